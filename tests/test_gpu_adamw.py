"""moe_adamw_step and moe_adamw_states: m, v and the 8-bit codes bit for bit, the values within derived bounds."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
from training_ref import adamw, check, decode, encode

pytestmark = pytest.mark.gpu
DEV = "cuda"
T32, BF, HF = torch.float32, torch.bfloat16, torch.float16
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=7)


def tensor(n, seed, param=T32, grad=T32, master=False, bits=32, off=0, **more):
    """A tensor's dict on the GPU, `off` elements into its buffers."""
    r = np.random.default_rng(seed)

    def put(a, t):
        b = torch.zeros(n + off, dtype=t, device=DEV)
        b[off:] = torch.from_numpy(a).to(DEV).to(t)
        return b[off:]

    x = r.standard_normal(n).astype(np.float32) * 0.05
    spread = np.exp(r.standard_normal(n)).astype(np.float32)
    mm, vv = (r.standard_normal(n).astype(np.float32) * 1e-3 * spread), np.square(2e-3 * spread * (0.5 + r.random(n))).astype(np.float32)
    d = {"param": put(x, param), "grad": put(r.standard_normal(n).astype(np.float32) * 1e-3 * spread, grad),
         "master": put(x, T32) if master else None, **more}
    if bits == 8:
        mc, vc, s = encode(mm, vv)
        d.update(m=put(mc, torch.uint8), v=put(vc, torch.uint8), scales=torch.from_numpy(s).to(DEV))
    else:
        d.update(m=put(mm, T32), v=put(vv, T32))
    return d


def expected(d, scale=1.0, **h):
    """What a step should leave: x64, tolerance, m, v (or codes and scales)."""
    h = {**HYPER, **h}
    x = (d["master"] if d.get("master") is not None else d["param"]).cpu().double().numpy()
    g = d["grad"].cpu().float().numpy()
    held = d.get("scales") is not None
    mm, vv = d["m"].cpu().numpy(), d["v"].cpu().numpy()
    if held:
        s = d["scales"].cpu().numpy()
        mm, vv = decode(mm, vv, s)
    lr = h["lr"] * d.get("lr_factor", 1.0)
    xn, mn, vn, tol, alone = adamw(x, g, mm, vv, lr, h["beta1"], h["beta2"], h["eps"], h["step"], d.get("weight_decay", 0.0), scale)
    return xn, tol, (encode(mn, vn) if held else (mn, vn)), alone


def verify(d, want):
    x, tol, states, _ = want
    if d.get("master") is not None:
        check(d["master"], torch.from_numpy(x), torch.from_numpy(tol), "master")
        assert torch.equal(d["param"], d["master"].to(d["param"].dtype))
    else:
        check(d["param"], torch.from_numpy(x), torch.from_numpy(tol), "param")
    for name, s in zip(("m", "v", "scales"), states):
        got = d[name].cpu().numpy()
        assert np.array_equal(got.reshape(-1), s.reshape(-1)), (name, np.argwhere(got.reshape(-1) != s.reshape(-1))[:5])


def step(ds, status=None, **kw):
    t = m.make_adamw_tensors(ds)
    m.moe_adamw_step(t, m.moe_adamw_options(**{**HYPER, **kw}), status)
    torch.cuda.synchronize()
    return t


KINDS = [(T32, T32, False), (T32, BF, False), (BF, BF, True), (BF, BF, False), (HF, T32, True), (HF, HF, False), (BF, T32, True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", KINDS)
def test_types_and_sizes(moe, param, grad, master, bits):
    ds = [tensor(n, n, param, grad, master, bits, weight_decay=0.1 * (n % 2), lr_factor=1.0 + n % 3)
          for n in (1, 2, 31, 255, 256, 257, 1000, 4096, 40009)]
    want = [expected(d) for d in ds]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    step(ds, st)
    assert m.moe_check_status(st) == 0
    for d, w in zip(ds, want):
        verify(d, w)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_tensors_at_any_alignment(moe, bits, off):
    ds = [tensor(n, n, BF, BF, True, bits, off) for n in (5, 300, 5000)]
    want = [expected(d) for d in ds]
    step(ds)
    for d, w in zip(ds, want):
        verify(d, w)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(moe, bits):
    """More than a launch holds; some empty."""
    ds = [tensor(0 if i % 50 == 9 else 1 + i * 7 % 700, i, BF, BF, False, bits) for i in range(900)]
    want = [expected(d) if d["param"].numel() else None for d in ds]
    step(ds)
    for d, w in zip(ds, want):
        if w:
            verify(d, w)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_and_small_tensors_together(moe, bits):
    ds = [tensor(n, n, T32, T32, False, bits) for n in (3_000_001, 12, 700_000)]
    want = [expected(d) for d in ds]
    step(ds)
    for d, w in zip(ds, want):
        verify(d, w)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(moe, bits):
    for off in (0, 1):
        d = tensor(2000, 3, T32, T32, False, bits, off)
        d["grad"][3], d["grad"][700], d["grad"][1999] = float("nan"), float("inf"), 1e25  # the last: its square is infinite
        d["grad"][256:512] = float("nan")  # a whole block
        before = {k: v.clone() for k, v in d.items() if v is not None}
        want = expected(d)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        step([d], st)
        assert m.moe_check_status(st) == m.MOE_ERR_NONFINITE
        x, tol, states, alone = want
        check(d["param"], torch.from_numpy(x), torch.from_numpy(tol))
        keep = torch.from_numpy(alone).to(DEV)
        assert int(keep.sum()) == 259 and torch.equal(d["param"][keep], before["param"][keep])
        if bits == 32:
            verify(d, want)
            assert torch.equal(d["m"][keep], before["m"][keep])
        else:  # a block without a good gradient keeps its bits; the others are held anew
            sl = slice(256, 512)
            assert torch.equal(d["m"][sl], before["m"][sl]) and torch.equal(d["v"][sl], before["v"][sl])
            assert torch.equal(d["scales"][1], before["scales"][1])
            for name, s in zip(("m", "v", "scales"), states):
                got = d[name].cpu().numpy().copy()
                rows = sl if name != "scales" else slice(1, 2)
                s = s.copy()
                s[rows] = got[rows]
                assert np.array_equal(got, s), name


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_scale_that_is_not_finite_leaves_everything(moe, bits, bad):
    d = tensor(3000, 4, BF, BF, True, bits)
    before = {k: v.clone() for k, v in d.items() if v is not None}
    s = torch.tensor([bad], device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    step([d], st, grad_scale=s.data_ptr())
    assert m.moe_check_status(st) == m.MOE_ERR_NONFINITE
    for k, v in before.items():
        assert torch.equal(d[k], v), k


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_tiny_and_huge_states(moe, bits):
    n = 256 * 8
    d = tensor(n, 5, T32, T32, False, bits)
    g = torch.zeros(n, device=DEV)
    g[256:512] = 1e-25   # squares below fp32
    g[512:768] = 1e18
    g[768:1024] = torch.logspace(-20, 10, 256, device=DEV)
    g[1024:1280] = -torch.logspace(-3, 3, 256, device=DEV)
    g[1300] = 1.0
    d["grad"] = g
    for k in ("m", "v") + (("scales",) if bits == 8 else ()):
        d[k].zero_()
    want = expected(d, step=1)
    step([d], step=1)
    verify(d, want)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr", [0.0, 1e-38, 1e-30, -1e-3, 100.0])
def test_rates_of_any_size(moe, bits, lr):
    d = tensor(5000, 8, T32, T32, False, bits, weight_decay=0.01)
    if bits == 32:
        d["m"][:256].zero_(), d["v"][:256].zero_()
    else:
        d["scales"][0].zero_()
    d["grad"][:256].zero_()  # 0 / eps
    want = expected(d, lr=lr)
    before = d["param"].clone()
    step([d], lr=lr)
    verify(d, want)
    assert lr != 0 or torch.equal(d["param"], before)


def test_scalars_on_the_device_and_a_replayed_step(moe):
    ds = [tensor(5000, 6, BF, BF, True, 8, weight_decay=0.1), tensor(777, 7, T32, T32, False, 32, lr_factor=0.5)]
    lr = torch.tensor([1.0], device=DEV)
    n = torch.tensor([1], dtype=torch.int64, device=DEV)
    scale = torch.tensor([1.0], device=DEV)
    t = m.make_adamw_tensors(ds)
    o = m.moe_adamw_options(lr=9.0, beta1=0.9, beta2=0.99, eps=1e-8, step=99, lr_dev=lr.data_ptr(), step_dev=n.data_ptr(),
                            grad_scale=scale.data_ptr())
    s = torch.cuda.Stream()
    saved = [{k: v.clone() for k, v in d.items() if isinstance(v, torch.Tensor)} for d in ds]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_adamw_step(t, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_adamw_step(t, o)
    for d, b in zip(ds, saved):
        for k, v in b.items():
            d[k].copy_(v)
    for step_, rate, factor in ((1, 1e-3, 1.0), (2, 5e-4, 0.25), (1000, 2e-3, 4.0)):
        lr.fill_(rate), n.fill_(step_), scale.fill_(factor)
        want = [expected(d, factor, step=step_, lr=float(lr)) for d in ds]
        graph.replay()
        torch.cuda.synchronize()
        # the corrections on the device are taken in fp32: 2^-21 of the step more
        for d, w in zip(ds, want):
            x, tol, states, alone = w
            old = (np.abs(x) + 1) * 0.0 + 2.0 ** -21 * 2e-3 * 4 * np.sqrt(1 / (1 - 0.99))
            verify(d, (x, tol + old, states, alone))


@pytest.mark.parametrize("off", [0, 1])
def test_values_of_the_states(moe, off):
    ds = [tensor(n, n, BF, BF, True, bits, off) for n in (3, 256, 5001) for bits in (8, 32)] + [tensor(0, 1)]
    t = m.make_adamw_tensors(ds)
    mv = [torch.full((d["param"].numel() + off,), 7.0, device=DEV)[off:] for d in ds]
    vv = [torch.full((d["param"].numel() + off,), 7.0, device=DEV)[off:] for d in ds]
    vv[1] = None
    m.moe_adamw_states(t, m.make_adamw_values(mv, vv))
    for d, a, b in zip(ds, mv, vv):
        want = d["m"].cpu().numpy(), d["v"].cpu().numpy()
        if d.get("scales") is not None:
            want = decode(*want, d["scales"].cpu().numpy())
        assert np.array_equal(a.cpu().numpy(), want[0])
        assert b is None or np.array_equal(b.cpu().numpy(), want[1])
    only = torch.empty_like(mv[0])
    m.moe_adamw_states(m.make_adamw_tensors(ds[:1]), m.make_adamw_values([only], None))
    assert torch.equal(only, mv[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_one_large_tensor_as_its_pieces(moe, bits):
    """One tensor of 90 million values, whose CTAs take 16,384 each, and the same in pieces whose CTAs take 2,048: the same bits."""
    n, piece = 90_000_128, 1 << 24
    g = torch.Generator(device=DEV).manual_seed(1)

    def make():
        g.manual_seed(1)
        d = {"param": torch.randn(n, generator=g, device=DEV).bfloat16(), "grad": torch.randn(n, generator=g, device=DEV).bfloat16()}
        if bits == 32:
            d["m"], d["v"] = torch.randn(n, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV)
        else:
            d["m"] = torch.randint(0, 126, (n,), generator=g, device=DEV).to(torch.uint8)
            d["v"] = torch.randint(0, 256, (n,), generator=g, device=DEV).to(torch.uint8)
            d["scales"] = torch.rand((n + 255) // 256, 2, generator=g, device=DEV)
        return d

    a, b = make(), make()
    step([a])
    for at in range(0, n, piece):
        end = min(n, at + piece)
        step([{k: (t[at // 256:(end + 255) // 256] if k == "scales" else t[at:end]) for k, t in b.items()}])
    for k in a:
        assert torch.equal(a[k], b[k]), k
