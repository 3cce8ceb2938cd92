"""The gradients of the plain forms against differences (CPU)."""
import numpy as np
import torch

from training_ref import ROOTS, E4M3, adamw, cross_entropy, decode, encode, router_loss


def test_router_loss_gradient():
    g = torch.Generator().manual_seed(0)
    T, E, k = 5, 7, 3
    logits = torch.randn(T, E, generator=g, dtype=torch.float64)
    ids = torch.topk(logits, k, dim=1).indices.int()
    keep = torch.tensor([1, 1, 0, 1, 1], dtype=torch.uint8)
    d, dw = torch.tensor([0.7, 0.2], dtype=torch.float64), torch.randn(T, k, generator=g, dtype=torch.float64)
    weights = lambda l: torch.softmax(l.gather(1, ids.long()), 1)  # noqa: E731

    def total(l):
        return float((router_loss(l, ids, k, keep)["loss"] * d).sum() + (weights(l) * dw).sum())

    grad = router_loss(logits, ids, k, keep, d, weights(logits), dw)["dlogits"]
    for t in range(T):
        for e in range(E):
            step = torch.zeros_like(logits)
            step[t, e] = 1e-5
            diff = (total(logits + step) - total(logits - step)) / 2e-5
            assert abs(diff - float(grad[t, e])) < 1e-8


def test_cross_entropy_gradient():
    g = torch.Generator().manual_seed(1)
    T, H, V = 4, 8, 6
    h, w = torch.randn(T, H, generator=g, dtype=torch.float64), torch.randn(V, H, generator=g, dtype=torch.float64)
    labels = torch.tensor([2, -1, 5, 6], dtype=torch.int32)
    dloss, dlse = torch.rand(T, generator=g, dtype=torch.float64), torch.randn(T, generator=g, dtype=torch.float64)

    def total(a, b):
        r = cross_entropy(a, b, labels)
        return float((r["loss"] * dloss).sum() + (r["lse"] * dlse).sum())

    # (types other than the three have no rounding; the bounds are not looked at)
    import training_ref

    training_ref.HALF[torch.float64] = 0.0
    r = cross_entropy(h, w, labels, dloss, dlse)
    del training_ref.HALF[torch.float64]
    for x, grad, which in ((h, r["dh"], 0), (w, r["dw"], 1)):
        for i in range(x.shape[0]):
            for j in range(H):
                step = torch.zeros_like(x)
                step[i, j] = 1e-5
                a = (total(h + step, w) - total(h - step, w)) if which == 0 else (total(h, w + step) - total(h, w - step))
                assert abs(a / 2e-5 - float(grad[i, j])) < 1e-8


def test_adamw_against_torch():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(100, generator=g)
    p = x.double().requires_grad_()
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    m, v, mine = np.zeros(100, np.float32), np.zeros(100, np.float32), x.double().numpy()
    for step in range(1, 6):
        grad = torch.randn(100, generator=g)
        p.grad = grad.double()
        opt.step()
        mine, m, v, _, _ = adamw(mine, grad.numpy(), m, v, 1e-2, 0.9, 0.99, 1e-8, step, 0.1)
    assert np.abs(mine - p.detach().numpy()).max() < 1e-7


def test_codes():
    assert E4M3[-1] == 448 and ROOTS[255] == 1.9375 and ROOTS[1] == 17 * 2.0 ** -19 and len(E4M3) == 127
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, E4M3)
    r = np.random.default_rng(0)
    m = (r.standard_normal(1000) * np.exp(r.standard_normal(1000) * 3)).astype(np.float32)
    v = np.square(m * r.random(1000).astype(np.float32))
    m[256:512] = 0
    v[512:768] = 0
    mc, vc, s = encode(m, v)
    dm, dv = decode(mc, vc, s)
    top = np.repeat(np.abs(np.concatenate([m, np.zeros(24, np.float32)])).reshape(-1, 256).max(1), 256)[:1000]
    assert (np.abs(dm - m) <= 2.0 ** -4 * np.abs(m) + top * 2.0 ** -10 / 448 + 1e-30).all()
    assert ((dv == 0) == (v == 0)).all()
    root_top = np.sqrt(np.repeat(np.concatenate([v, np.zeros(24, np.float32)]).reshape(-1, 256).max(1), 256)[:1000])
    assert (np.abs(np.sqrt(dv) - np.sqrt(v)) <= 2.0 ** -5 * 1.001 * np.sqrt(v) + root_top * 17 / 16 * 2.0 ** -15 / 1.9375).all()
    mc2, vc2, s2 = encode(dm, dv)  # what is held stays what it is
    assert np.array_equal(mc2, mc) and np.array_equal(vc2, vc) and np.allclose(s2, s, rtol=1e-6)
