"""moe_cross_entropy and its gradients against their 64-bit forms."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from training_ref import check, cross_entropy

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {m.MOE_BF16: torch.bfloat16, m.MOE_F16: torch.float16, m.MOE_F32: torch.float32}


def inputs(T, H, V, dtype, seed=0, scale=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn(V, H, generator=g, device=DEV) * scale / H ** 0.5).to(TYPES[dtype])
    labels = torch.randint(0, V, (T,), generator=g, device=DEV)
    h = (torch.randn(T, H, generator=g, device=DEV) + torch.rand(T, 1, generator=g, device=DEV) * 2 * w[labels].float()).to(TYPES[dtype])
    labels[torch.rand(T, generator=g, device=DEV) < 0.15] = -100
    dloss = torch.rand(T, generator=g, device=DEV) / T
    return h, w, labels.int(), dloss


def forward(h, w, labels, dtype):
    (T, H), V = h.shape, w.shape[0]
    loss, lse = torch.full((T,), 7.0, device=DEV), torch.full((T,), 7.0, device=DEV)
    nb = m.moe_cross_entropy_workspace_size(T, H, V)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN bit patterns
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_cross_entropy(h, dtype, T, H, w, V, labels, loss, lse, ws, nb, st)
    return loss, lse, m.moe_check_status(st)


def backward(h, w, labels, dtype, lse, dloss, dlse=None, want=(True, True), dw_dtype=None, dw0=None):
    (T, H), V = h.shape, w.shape[0]
    dh = torch.full_like(h, 7.0) if want[0] else None
    wt = dtype if dw_dtype is None else dw_dtype
    dw = (torch.full((V, H), 7.0, dtype=TYPES[wt], device=DEV) if dw0 is None else dw0.clone()) if want[1] else None
    nb = m.moe_cross_entropy_backward_workspace_size(T, H, V)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_cross_entropy_backward(h, dtype, T, H, w, V, labels, lse, dloss, dlse, dh, dw, wt, dw0 is not None, ws, nb, st)
    assert m.moe_check_status(st) == 0 or bool((labels >= V).any())
    return dh, dw


SIZES = [(1, 8, 1), (1, 64, 7), (2, 72, 255), (3, 256, 256), (31, 264, 257), (4, 2048, 5003), (129, 64, 1000), (128, 128, 512),
         (300, 1056, 4099), (257, 8, 70), (513, 520, 2049), (1111, 200, 3001),
         (16, 136, 5000), (17, 64, 4865), (33, 320, 20011), (63, 72, 9001), (64, 128, 31), (65, 128, 5001)]


@pytest.mark.parametrize("dtype", [m.MOE_BF16, m.MOE_F16])
@pytest.mark.parametrize("T,H,V", SIZES)
def test_sizes(moe, T, H, V, dtype):
    h, w, labels, dloss = inputs(T, H, V, dtype, T + V)
    loss, lse, st = forward(h, w, labels, dtype)
    want = cross_entropy(h, w, labels, dloss)
    assert st == 0
    check(loss, want["loss"], want["loss_tol"], "loss")
    check(lse, want["lse"], want["lse_tol"], "lse")
    assert (loss[labels < 0] == 0).all()
    dh, dw = backward(h, w, labels, dtype, lse, dloss)
    check(dh, want["dh"], want["dh_tol"], "dh")
    check(dw, want["dw"], want["dw_tol"], "dw")


@pytest.mark.parametrize("dtype", [m.MOE_BF16, m.MOE_F16])
def test_gradient_of_lse_types_and_accumulation(moe, dtype):
    T, H, V = 200, 136, 777
    h, w, labels, dloss = inputs(T, H, V, dtype, 1)
    dlse = torch.randn(T, device=DEV) * 3e-3
    _, lse, _ = forward(h, w, labels, dtype)
    want = cross_entropy(h, w, labels, dloss, dlse)
    dh, dw = backward(h, w, labels, dtype, lse, dloss, dlse, dw_dtype=m.MOE_F32)
    check(dh, want["dh"], want["dh_tol"], "dh")
    check(dw, want["dw"], want["dw_tol"], "dw")
    start = torch.randn(V, H, device=DEV)
    _, more = backward(h, w, labels, dtype, lse, dloss, dlse, dw_dtype=m.MOE_F32, dw0=start)
    assert torch.equal(more, start + dw)  # one addition per value
    only, none = backward(h, w, labels, dtype, lse, dloss, dlse, want=(True, False))
    assert none is None and torch.equal(only, dh)
    none, only = backward(h, w, labels, dtype, lse, dloss, dlse, want=(False, True), dw_dtype=m.MOE_F32)
    assert none is None and torch.equal(only, dw)


def test_labels_left_out(moe):
    T, H, V = 140, 64, 300
    h, w, labels, dloss = inputs(T, H, V, m.MOE_BF16, 2)
    labels[:] = -1
    loss, lse, st = forward(h, w, labels, m.MOE_BF16)
    want = cross_entropy(h, w, labels)
    assert st == 0 and (loss == 0).all()
    check(lse, want["lse"], want["lse_tol"])
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    assert (dh == 0).all() and (dw == 0).all()
    labels[3], labels[5], labels[6] = 299, 300, 2 ** 31 - 1
    loss, lse, st = forward(h, w, labels, m.MOE_BF16)
    want = cross_entropy(h, w, labels, dloss)
    assert st == m.MOE_ERR_BOUNDS
    check(loss, want["loss"], want["loss_tol"])
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    check(dh, want["dh"], want["dh_tol"])
    check(dw, want["dw"], want["dw_tol"])


def test_weights_of_zero_and_tokens_that_are_not_finite(moe):
    """A token left out by its weight takes no part, even where its hidden state is not a number."""
    T, H, V = 150, 64, 500
    h, w, labels, dloss = inputs(T, H, V, m.MOE_BF16, 3)
    labels.clamp_(min=0)
    dloss[10:20] = 0
    _, lse, _ = forward(h, w, labels, m.MOE_BF16)
    want = cross_entropy(h, w, labels, dloss)
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    check(dh, want["dh"], want["dh_tol"])
    check(dw, want["dw"], want["dw_tol"])
    assert (dh[10:20] == 0).all()
    h[40] = float("nan")
    loss, lse, _ = forward(h, w, labels, m.MOE_BF16)
    assert torch.isnan(loss[40]) and torch.isfinite(loss[torch.arange(T, device=DEV) != 40]).all()


def test_extreme_logits(moe):
    """A certain label, a hopeless one, and logits of some thousands."""
    T, H, V = 130, 64, 600
    h, w, labels, dloss = inputs(T, H, V, m.MOE_BF16, 4, scale=400.0)
    labels.clamp_(min=0)
    z = h.float() @ w.float().T
    labels[:50] = z[:50].argmax(1).int()
    labels[50:60] = z[50:60].argmin(1).int()
    loss, lse, _ = forward(h, w, labels, m.MOE_BF16)
    want = cross_entropy(h, w, labels, dloss)
    check(loss, want["loss"], want["loss_tol"])
    assert (loss[:50] >= 0).all()


def test_huge_logits(moe):
    """Logits of 10^30 beside ordinary rows: the largest takes all."""
    T, H, V = 40, 64, 300
    h, w, labels, dloss = inputs(T, H, V, m.MOE_BF16, 9)
    labels.clamp_(min=0)
    h[5] *= 1e30
    h[6] *= 1e6
    loss, lse, _ = forward(h, w, labels, m.MOE_BF16)
    want = cross_entropy(h, w, labels, dloss)
    check(loss, want["loss"], want["loss_tol"])
    check(lse, want["lse"], want["lse_tol"])
    best = (h[5].double() @ w.double().T).argmax()
    labels[5] = int(best)
    loss, lse, _ = forward(h, w, labels, m.MOE_BF16)
    assert loss[5] == 0
    dloss[6] = 0
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    assert (dh[5] == 0).all() and torch.isfinite(dw).all()


def test_several_pieces_of_the_vocabulary(moe):
    T, H, V = 2048, 64, 70001
    h, w, labels, dloss = inputs(T, H, V, m.MOE_BF16, 5)
    _, lse, _ = forward(h, w, labels, m.MOE_BF16)
    assert m.moe_cross_entropy_backward_workspace_size(T, H, V) < (258 << 20)
    want = cross_entropy(h, w, labels, dloss, pieces=2)
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    check(dh, want["dh"], want["dh_tol"], "dh")
    check(dw, want["dw"], want["dw_tol"], "dw")
    dh2, dw32 = backward(h, w, labels, m.MOE_BF16, lse, dloss, dw_dtype=m.MOE_F32)
    assert torch.equal(dh2, dh)  # the same bits again
    check(dw32, want["dw"], want["dw_tol"], "dw fp32")


def test_rows_before_and_behind_stay_as_they_were(moe):
    T, H, V = 33, 72, 333
    h, w, labels, dloss = inputs(T, H, V, m.MOE_F16, 6)
    _, lse, _ = forward(h, w, labels, m.MOE_F16)
    want = backward(h, w, labels, m.MOE_F16, lse, dloss)
    bigh, bigw = torch.full((T + 8, H), 3.0, dtype=torch.float16, device=DEV), torch.full((V + 8, H), 3.0, dtype=torch.float16, device=DEV)
    nb = m.moe_cross_entropy_backward_workspace_size(T, H, V)
    ws = torch.empty(nb + 64, dtype=torch.uint8, device=DEV)
    ws[nb:] = 77
    m.moe_cross_entropy_backward(h, m.MOE_F16, T, H, w, V, labels, lse, dloss, None, bigh[4:4 + T], bigw[4:4 + V], m.MOE_F16, False,
                                 ws[:nb], nb)
    assert torch.equal(bigh[4:4 + T], want[0]) and torch.equal(bigw[4:4 + V], want[1])
    for t, n in ((bigh, T), (bigw, V)):
        assert (t[:4] == 3).all() and (t[4 + n:] == 3).all()
    assert (ws[nb:] == 77).all()


def test_no_tokens(moe):
    H, V = 16, 40
    e = torch.zeros(0, H, dtype=torch.bfloat16, device=DEV)
    w = torch.randn(V, H, device=DEV).bfloat16()
    none_i, none_f = torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(0, device=DEV)
    m.moe_cross_entropy(e, m.MOE_BF16, 0, H, w, V, none_i, none_f, none_f)
    dw = torch.full((V, H), 7.0, device=DEV)
    m.moe_cross_entropy_backward(e, m.MOE_BF16, 0, H, w, V, none_i, none_f, none_f, None, e, dw, m.MOE_F32, True)
    assert (dw == 7).all()
    m.moe_cross_entropy_backward(e, m.MOE_BF16, 0, H, w, V, none_i, none_f, none_f, None, e, dw, m.MOE_F32, False)
    assert (dw == 0).all()


def test_captured_and_replayed_on_two_streams(moe):
    T, H, V = 260, 128, 1500
    sets = [inputs(T, H, V, m.MOE_BF16, s) for s in (7, 8)]
    nb = max(m.moe_cross_entropy_workspace_size(T, H, V), m.moe_cross_entropy_backward_workspace_size(T, H, V))
    graphs = []
    for h, w, labels, dloss in sets:
        b = dict(h=torch.zeros_like(h), w=torch.zeros_like(w), labels=torch.zeros_like(labels), dloss=torch.zeros_like(dloss),
                 loss=torch.empty(T, device=DEV), lse=torch.empty(T, device=DEV), dh=torch.empty_like(h), dw=torch.empty_like(w),
                 ws=torch.empty(nb, dtype=torch.uint8, device=DEV))

        def step(b=b):
            m.moe_cross_entropy(b["h"], m.MOE_BF16, T, H, b["w"], V, b["labels"], b["loss"], b["lse"], b["ws"], nb)
            m.moe_cross_entropy_backward(b["h"], m.MOE_BF16, T, H, b["w"], V, b["labels"], b["lse"], b["dloss"], None, b["dh"],
                                         b["dw"], m.MOE_BF16, False, b["ws"], nb)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, b, torch.cuda.Stream()))
    for (g, b, s), (h, w, labels, dloss) in zip(graphs, sets):
        b["h"].copy_(h), b["w"].copy_(w), b["labels"].copy_(labels), b["dloss"].copy_(dloss)
    torch.cuda.synchronize()
    for g, b, s in graphs:
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for (g, b, s), (h, w, labels, dloss) in zip(graphs, sets):
        loss, lse, _ = forward(h, w, labels, m.MOE_BF16)
        dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
        assert torch.equal(b["loss"], loss) and torch.equal(b["lse"], lse)
        assert torch.equal(b["dh"], dh) and torch.equal(b["dw"], dw)
