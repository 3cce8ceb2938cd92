"""moe_router_loss and its gradient against their 64-bit forms."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from training_ref import check, router_loss

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {m.MOE_F32: torch.float32, m.MOE_BF16: torch.bfloat16, m.MOE_F16: torch.float16}


def inputs(T, E, k, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = (torch.randn(T, E, generator=g, device=DEV) * 2).to(TYPES[dtype])
    top = torch.topk(logits.float(), k, dim=1)
    w = torch.softmax(top.values, 1)
    dw = torch.randn(T, k, generator=g, device=DEV)
    return logits, top.indices.int(), w, dw


def run(logits, ids, k, dtype, keep=None, dloss=None, w=None, dw=None, in_place=False):
    T, E = logits.shape
    f = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    out = {"loss": f(2), "mean": f(E), "lse": f(max(T, 1))[:T], "counts": torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)}
    nb = m.moe_router_loss_workspace_size(T, E)
    ws = torch.full((max(nb, 1),), 0xA5, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_router_loss(logits, dtype, T, E, ids, k, keep, out["loss"], out["counts"], out["mean"], out["lse"], ws, nb, st)
    out["dlogits"] = logits if in_place else torch.full_like(logits, 7.0)
    m.moe_router_loss_backward(logits, dtype, T, E, ids, k, out["counts"], out["lse"], dloss, w, dw, out["dlogits"])
    out["status"] = m.moe_check_status(st)
    return out


def compare(got, want, keys=("loss", "mean", "lse", "dlogits")):
    assert torch.equal(got["counts"], want["counts"])
    for key in keys:
        check(got[key], want[key], want[key + "_tol"], key)


DLOSS = (0.3, 0.07)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 10), (2, 2, 2), (7, 61, 4), (32, 512, 10), (33, 100, 3), (129, 128, 16),
                                   (300, 256, 8), (384, 1024, 2), (385, 512, 10), (1024, 60, 4), (1025, 64, 6), (4099, 513, 10), (2500, 1024, 16), (1500, 1021, 1)])
def test_sizes(moe, T, E, k, dtype):
    logits, ids, w, dw = inputs(T, E, k, dtype, T)
    d = torch.tensor(DLOSS, device=DEV)
    want = router_loss(logits, ids, k, None, d, w, dw)
    got = run(logits, ids, k, dtype, None, d, w, dw)
    assert got["status"] == 0
    compare(got, want)


@pytest.mark.parametrize("T", [50, 3000])
def test_parts_of_the_gradient(moe, T):
    logits, ids, w, dw = inputs(T, 96, 5, m.MOE_F32, 1)
    for d in (None, torch.tensor([1.0, 0.0], device=DEV), torch.tensor([0.0, 1.0], device=DEV)):
        for ww, dd in ((None, None), (w, dw)):
            compare(run(logits, ids, 5, m.MOE_F32, None, d, ww, dd), router_loss(logits, ids, 5, None, d, ww, dd))


@pytest.mark.parametrize("T", [40, 2000])
@pytest.mark.parametrize("kind", ["some", "none", "one"])
def test_tokens_left_out(moe, T, kind):
    logits, ids, w, dw = inputs(T, 512, 10, m.MOE_BF16, 2)
    keep = torch.rand(T, device=DEV) < 0.5 if kind == "some" else torch.zeros(T, dtype=torch.bool, device=DEV)
    if kind == "one":
        keep[T - 1] = True
    d = torch.tensor(DLOSS, device=DEV)
    got = run(logits, ids, 10, m.MOE_BF16, keep, d, w, dw)
    compare(got, router_loss(logits, ids, 10, keep, d, w, dw))
    if kind == "none":
        assert (got["loss"] == 0).all() and (got["counts"] == 0).all() and (got["mean"] == 0).all()
    bytes_ = keep.to(torch.uint8) * 255  # any byte but zero counts
    assert torch.equal(run(logits, ids, 10, m.MOE_BF16, bytes_, d, w, dw)["dlogits"], got["dlogits"])


@pytest.mark.parametrize("T", [20, 1100])
def test_infinite_and_nan_logits(moe, T):
    logits, ids, w, dw = inputs(T, 130, 4, m.MOE_F32, 3)
    d = torch.tensor(DLOSS, device=DEV)
    logits[1, :100] = -float("inf")   # experts that cannot be chosen
    logits[2] = -float("inf")         # ... and nothing left: the token does not count
    logits[3] = -3.0e38               # finite, however large
    logits[3, 7] = 3.0e38
    logits[4] *= 1e30
    got = run(logits, ids, 4, m.MOE_F32, None, d, w, dw)
    want = router_loss(logits, ids, 4, None, d, w, dw)
    assert got["status"] == 0 and got["lse"][2] == -float("inf")
    # (the squares of such logits leave fp32; the loss is infinite, as its definition in fp32 is)
    assert torch.equal(got["counts"], want["counts"]) and torch.isinf(got["loss"][1])
    check(got["mean"], want["mean"], want["mean_tol"])
    rows = torch.tensor([i for i in range(T) if i not in (3, 4)], device=DEV)
    check(got["dlogits"][rows], want["dlogits"][rows], want["dlogits_tol"][rows])
    logits[3:5] = 0.5
    logits[5, 3] = float("nan")
    logits[6, 5] = float("inf")
    got = run(logits, ids, 4, m.MOE_F32, None, d, w, dw)
    assert got["status"] == m.MOE_ERR_NONFINITE
    compare(got, router_loss(logits, ids, 4, None, d, w, dw))


@pytest.mark.parametrize("T", [30, 1500])
def test_ids_of_no_expert_and_repeated_ones(moe, T):
    logits, ids, w, dw = inputs(T, 70, 6, m.MOE_F32, 4)
    d = torch.tensor(DLOSS, device=DEV)
    ids[1, 2] = m.MOE_ID_NOT_LOCAL
    ids[2] = m.MOE_ID_NOT_LOCAL
    ids[3, 4] = ids[3, 1]
    ids[4] = 5
    got = run(logits, ids, 6, m.MOE_F32, None, d, w, dw)
    assert got["status"] == 0
    compare(got, router_loss(logits, ids, 6, None, d, w, dw))
    ids[5, 0], ids[6, 1] = 70, -5
    got = run(logits, ids, 6, m.MOE_F32, None, d, w, dw)
    assert got["status"] == m.MOE_ERR_BOUNDS
    compare(got, router_loss(logits, ids, 6, None, d, w, dw))


def test_no_tokens(moe):
    got = run(torch.zeros(0, 33, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV), 2, m.MOE_F32)
    assert (got["loss"] == 0).all() and (got["counts"] == 0).all() and (got["mean"] == 0).all()


@pytest.mark.parametrize("E", [64, 61])
def test_rows_off_sixteen_bytes_and_in_place(moe, E):
    T, k = 700, 4
    logits, ids, w, dw = inputs(T, E, k, m.MOE_F32, 5)
    d = torch.tensor(DLOSS, device=DEV)
    want = run(logits, ids, k, m.MOE_F32, None, d, w, dw)
    flat = torch.empty(T * E + 1, device=DEV)
    off = flat[1:].view(T, E).copy_(logits)
    got = run(off, ids, k, m.MOE_F32, None, d, w, dw, in_place=True)
    compare(got, router_loss(logits, ids, k, None, d, w, dw))
    assert torch.equal(got["counts"], want["counts"])


def test_same_bits_twice_and_on_another_stream(moe):
    logits, ids, w, dw = inputs(5000, 512, 10, m.MOE_F32, 6)
    d = torch.tensor(DLOSS, device=DEV)
    a = run(logits, ids, 10, m.MOE_F32, None, d, w, dw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = run(logits, ids, 10, m.MOE_F32, None, d, w, dw)
    s.synchronize()
    for key in ("loss", "mean", "lse", "counts", "dlogits"):
        assert torch.equal(a[key], b[key]), key


def test_captured_and_replayed(moe):
    T, E, k = 2100, 128, 8
    logits, ids, w, dw = inputs(T, E, k, m.MOE_F32, 7)
    d = torch.tensor(DLOSS, device=DEV)
    f = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    loss, counts, mean, lse, dl = f(2), torch.empty(E + 1, dtype=torch.int32, device=DEV), f(E), f(T), f(T, E)
    nb = m.moe_router_loss_workspace_size(T, E)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)

    def step():
        m.moe_router_loss(logits, m.MOE_F32, T, E, ids, k, None, loss, counts, mean, lse, ws, nb)
        m.moe_router_loss_backward(logits, m.MOE_F32, T, E, ids, k, counts, lse, d, w, dw, dl)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = inputs(T, E, k, m.MOE_F32, 8)
    for dst, src in zip((logits, ids, w, dw), other):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    want = run(*other[:2], k, m.MOE_F32, None, d, *other[2:])
    for a, b in ((loss, "loss"), (counts, "counts"), (mean, "mean"), (lse, "lse"), (dl, "dlogits")):
        assert torch.equal(a, want[b]), b


def test_agrees_with_the_routers_own_choice(moe):
    """The calls as they are used: moe_topk_from_logits gives ids and weights, the losses' gradient goes back to its logits."""
    T, E, k = 257, 96, 6
    logits = torch.randn(T, E, device=DEV)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    m.moe_topk_from_logits(logits, T, E, k, ids, w)
    dw = torch.randn(T, k, device=DEV)
    l = logits.double().requires_grad_()
    kept = torch.softmax(l.gather(1, ids.long()), 1)
    p = torch.softmax(l, 1)
    f = torch.bincount(ids.reshape(-1).long(), minlength=E).double() / (T * k)
    loss = torch.stack([E * (f * p.mean(0)).sum(), torch.logsumexp(l, 1).square().mean()])
    d = torch.tensor(DLOSS, device=DEV)
    grad, = torch.autograd.grad((loss * d.double()).sum() + (kept * dw.double()).sum(), l)
    got = run(logits, ids, k, m.MOE_F32, None, d, w, dw)
    want = router_loss(logits, ids, k, None, d, w, dw)
    check(got["loss"], loss.detach(), want["loss_tol"])
    # the weights themselves carry 1e-6 of the kept softmax
    check(got["dlogits"], grad, want["dlogits_tol"] + 4e-6 * dw.abs().max())
