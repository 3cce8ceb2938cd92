"""Gradients of the cross entropy where tokens' weights are not finite: they show in what they reach, and nowhere else."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_cross_entropy import DEV, backward, forward, inputs
from training_ref import check, cross_entropy

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def setup(T, H, V, dtype, seed):
    h, w, labels, dloss = inputs(T, H, V, dtype, seed)
    labels.clamp_(min=0)
    labels[1] = -1
    _, lse, st = forward(h, w, labels, dtype)
    assert st == 0
    return h, w, labels, dloss, lse


@pytest.mark.parametrize("dtype", [m.MOE_BF16, m.MOE_F16])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("others", ["ordinary", "zero", "as bad"])
@pytest.mark.parametrize("which", ["dloss", "dlse"])
def test_a_weight_that_is_not_finite(moe, which, others, bad, dtype):
    T, H, V = 150, 72, 600
    h, w, labels, dloss, lse = setup(T, H, V, dtype, 11)
    dlse = torch.randn(T, device=DEV) * 1e-3
    hit = torch.zeros(T, dtype=torch.bool, device=DEV)
    hit[7] = hit[140] = True
    if others == "zero":
        dloss.zero_(), dlse.zero_()
    if others == "as bad":
        hit[:] = True
    weights = {"dloss": dloss, "dlse": dlse}
    weights[which][hit] = bad
    if which == "dloss":
        hit[1] = False  # a token without a label has no weight there
    dh, dw = backward(h, w, labels, dtype, lse, dloss, dlse)
    assert not torch.isfinite(dh[hit]).any() and not torch.isfinite(dw).any()
    if bad != bad:
        assert torch.isnan(dh[hit]).all() and torch.isnan(dw).all()
    # the other tokens' rows: as if the weights that are not finite, and they alone, were zero (d's rounding goes by all others)
    weights[which][~torch.isfinite(weights[which])] = 0
    only, _ = backward(h, w, labels, dtype, lse, dloss, dlse)
    assert torch.equal(dh[~hit], only[~hit])
    want = cross_entropy(h, w, labels, dloss, dlse)
    check(only, want["dh"], want["dh_tol"], "dh")


def test_a_weight_of_no_token(moe):
    """What a token without a label has in its place is not a weight."""
    h, w, labels, dloss, lse = setup(150, 72, 600, m.MOE_BF16, 12)
    want = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    for bad in (NAN, INF, 1e30):
        dloss[1] = bad
        got = backward(h, w, labels, m.MOE_BF16, lse, dloss)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("at", [0, 255, 256, 2047, 2048, 4095, 4999])
@pytest.mark.parametrize("which", ["dloss", "dlse"])
def test_the_largest_weight_in_any_place(moe, which, at):
    """In fp16 a weight 10,000 times the others' would leave the range, were it not found."""
    T, H, V = 5000, 64, 300
    h, w, labels, dloss, lse = setup(T, H, V, m.MOE_F16, 13)
    dloss[:] = 1e-4
    dlse = torch.full((T,), 1e-4, device=DEV)
    {"dloss": dloss, "dlse": dlse}[which][at] = -1.0
    want = cross_entropy(h, w, labels, dloss, dlse)
    dh, dw = backward(h, w, labels, m.MOE_F16, lse, dloss, dlse)
    check(dh, want["dh"], want["dh_tol"], "dh")
    check(dw, want["dw"], want["dw_tol"], "dw")
