"""AdamW where eps is far below the usual: steps that roots below fp32's normal range decide."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_adamw import DEV, T32, expected, step, tensor, verify

pytestmark = pytest.mark.gpu


def zeroed(n, bits, off, seed=9):
    """A first step of values that are zero, so that nothing but the step is compared."""
    d = tensor(n, seed, T32, T32, False, bits, off)
    for k in ("param", "m", "v") + (("scales",) if bits == 8 else ()):
        d[k].zero_()
    return d


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("lr", [1e-3, 1.0, 1e4])
@pytest.mark.parametrize("eps", [1e-8, 1e-12, 1e-15, 1e-20, 1e-30, 2e-38, 1.0, 1e30])
def test_small_gradients_beside_ordinary_ones(moe, eps, lr, off, bits):
    d = zeroed(256 * 6, bits, off)
    g = d["grad"]
    g[3], g[4], g[5], g[6] = 1e-18, -3e-19, 1e-22, 0.0  # squares below the normal range, below all, and none
    g[256:512] = torch.where(torch.arange(256, device=DEV) % 2 == 0, g[256:512], torch.zeros(256, device=DEV))
    g[512:768] = torch.logspace(-24, -3, 256, device=DEV)
    want = expected(d, step=1, beta2=0.999, eps=eps, lr=lr)
    step([d], step=1, beta2=0.999, eps=eps, lr=lr)
    verify(d, want)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("beta2", [0.0, 1 - 1e-6, 1 - 1e-9, 1 - 1e-13])
def test_corrections_of_any_size(moe, beta2, bits):
    for eps in (1e-8, 1e-20):
        d = zeroed(256 * 4, bits, 0)
        d["grad"][3], d["grad"][4], d["grad"][5] = 1e-18, 0.0, 1e-15
        want = expected(d, step=1, beta2=beta2, eps=eps)
        step([d], step=1, beta2=beta2, eps=eps)
        verify(d, want)


@pytest.mark.parametrize("lr", [1e-20, 1e-36, 1e20])
def test_rates_beside_values_of_zero(moe, lr):
    """However small a step, it is taken the same way with and without a wide access."""
    a, b = zeroed(256 * 4, 8, 0), zeroed(256 * 4, 8, 1)
    for d in (a, b):
        want = expected(d, step=1, lr=lr)
        step([d], step=1, lr=lr)
        verify(d, want)


@pytest.mark.parametrize("off", [0, 1])
def test_no_rate_leaves_values_whatever_their_states(moe, off):
    d = tensor(256 * 4, 3, T32, T32, False, 32, off)
    d["m"][:] = 1e10
    d["v"].zero_()
    d["grad"].zero_()
    before = d["param"].clone()
    step([d], lr=0.0, eps=2e-38)
    assert torch.equal(d["param"], before)


def test_a_rate_on_the_device(moe):
    """The rate that a replayed step finds decides like the one that is given."""
    lr = torch.tensor([1.0], device=DEV)
    d = zeroed(256 * 4, 8, 0)
    d["grad"][3], d["grad"][4] = 1e-18, 0.0
    want = expected(d, step=1, beta2=0.999, eps=2e-38, lr=1.0)
    step([d], step=5, beta2=0.999, eps=2e-38, lr=9.0, lr_dev=lr.data_ptr(), step_dev=(n := torch.ones(1, dtype=torch.int64, device=DEV)).data_ptr())
    assert int(n) == 1
    x, tol, states, alone = want
    # (the corrections on the device are taken in fp32: 2^-21 of the step more)
    verify(d, (x, tol + 2.0 ** -21 * abs(x), states, alone))
