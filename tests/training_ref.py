"""Plain 64-bit forms of the router's losses, the cross entropy and AdamW (torch, on any device), and error bounds for
kernels that compute them with 32-bit sums."""
import numpy as np
import torch

from operators_ref import HALF, TINY, U32  # noqa: F401


def check(got, want, slack, what=""):
    """|got - want| <= slack (error before the rounding) + half a step of got's type; NaN where want is NaN."""
    g, w = got.double(), want.double().to(got.device)
    s = torch.as_tensor(slack, dtype=torch.float64, device=got.device)
    tol = s + HALF[got.dtype] * (w.abs() + s) + TINY[got.dtype]
    bad = ~(((g - w).abs() <= tol) | (torch.isnan(g) & torch.isnan(w)) | (g == w))
    if bad.any():
        i = tuple(int(x[0]) for x in torch.nonzero(bad, as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {float(g[i])!r}, want "
                             f"{float(w[i])!r} +- {float(tol.expand_as(g)[i]):.3e}")


# ---------------------------------------------------------------- the router's losses

def router_loss(logits, ids, k, keep, dloss=None, w=None, dw=None):
    """A dict of loss, counts, mean, lse (and dlogits), and of a bound for each (key + "_tol")."""
    l = logits.double()
    T, E = l.shape
    dev = l.device
    top = l.amax(1) if T else l.new_zeros(0)
    counts_in = torch.isfinite(top) & ~torch.isnan(l).any(1) if T else torch.zeros(0, dtype=torch.bool, device=dev)
    if keep is not None:
        counts_in &= keep.bool()
    safe = torch.where(counts_in[:, None], l, torch.zeros_like(l))
    lse = torch.logsumexp(safe, 1) if T else l.new_zeros(0)
    p = torch.exp(safe - lse[:, None]) * counts_in[:, None]
    n = int(counts_in.sum())
    pick = ids.long()[counts_in].reshape(-1)
    pick = pick[(pick >= 0) & (pick < E)]
    count = torch.bincount(pick, minlength=E)
    mean = p.sum(0) / max(n, 1)
    lse_in = torch.where(counts_in, lse, torch.zeros_like(lse))
    loss = torch.stack([E * (count.double() * mean).sum() / (max(n, 1) * k), lse_in.square().sum() / max(n, 1)])
    # an exponential: 2^-22 of its own, and two roundings of an argument of at most 88 that matters; then 40 additions
    span = torch.where(torch.isfinite(safe), safe.amax(1, keepdim=True) - safe, torch.zeros_like(safe)).clamp(0, 88).amax(1) if T else top
    u = (44 + 3 * span) * U32 * counts_in
    e_lse = u + 4 * U32 * (lse_in.abs() + np.log(E) + 1)
    rel = 2 * (u.amax() if n else 0.0) + 500 * U32  # of a mean of probabilities
    out = {"loss": loss, "counts": torch.cat([count, torch.tensor([n], device=dev)]).int(), "mean": mean,
           "lse": torch.where(counts_in, lse, torch.full_like(lse, -float("inf"))), "mean_tol": rel * mean,
           "lse_tol": e_lse, "loss_tol": torch.stack([(rel + 100 * U32) * loss[0],
                                                      (2 * lse_in.abs() * e_lse).sum() / max(n, 1) + 600 * U32 * loss[1]])}
    grad, tol = torch.zeros_like(l), torch.zeros_like(l)
    if dloss is not None:
        d = dloss.double().to(dev)
        g = d[0] * E * count.double() / (max(n, 1) ** 2 * k)
        z = 2 * d[1] / max(n, 1)
        grad = p * (g - (p * g).sum(1, keepdim=True) + (z * lse_in)[:, None]) * counts_in[:, None]
        size = g.abs() + (p * g.abs()).sum(1, keepdim=True) + (z * lse_in).abs()[:, None]
        tol = p * size * (2 * u + e_lse + 100 * U32)[:, None]
    if w is not None:
        wd, dd = w.double(), dw.double()
        v = wd * (dd - (wd * dd).sum(1, keepdim=True))
        e = 24 * U32 * wd * (dd.abs() + (wd * dd.abs()).sum(1, keepdim=True))
        ok = (ids >= 0) & (ids < E)
        at = torch.where(ok, ids, torch.zeros_like(ids)).long()
        grad = grad.scatter_add(1, at, v * ok)
        tol = tol.scatter_add(1, at, e * ok) + U32 * grad.abs() * 16
    out["dlogits"], out["dlogits_tol"] = grad, tol
    return out


# ---------------------------------------------------------------- cross entropy

def cross_entropy(h, w, labels, dloss=None, dlse=None, pieces=1):
    """loss, lse (and dh, dw) with bounds."""
    hd, wd = h.double(), w.double()
    T, H = hd.shape
    V = wd.shape[0]
    z = hd @ wd.T
    # each instruction sums 16 products and the running sum: at most 2^-23 of the magnitudes each
    e_z = ((H / 16 + 8) * 2.0 ** -23 * (hd.abs() @ wd.abs().T)).amax(1)
    big = z.abs().amax(1)
    lse = torch.logsumexp(z, 1)
    there = (labels >= 0) & (labels < V)
    at = torch.where(there, labels, torch.zeros_like(labels)).long()[:, None]
    loss = torch.where(there, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    # the exponentials' arguments are rounded at the size of the logits, sums of 64 + 8 + a sum per tile
    e_exp = U32 * (8 * big + 96 + V / 256)
    out = {"loss": loss, "lse": lse, "loss_tol": (2 * e_z + e_exp + 4 * U32 * (lse.abs() + big)) * there,
           "lse_tol": e_z + e_exp + 4 * U32 * lse.abs()}
    if dloss is None:
        return out
    b = torch.where(there, dloss.double(), torch.zeros_like(lse))
    a = b + (dlse.double() if dlse is not None else 0.0)
    p = torch.exp(z - lse[:, None])
    d = p * a[:, None]
    d.scatter_add_(1, at, -b[:, None])
    top = max(float(b.abs().max()), float(dlse.abs().max()) if dlse is not None else 0.0)
    rel = (e_z + out["lse_tol"] + e_exp + 16 * U32)[:, None]
    e_d = p * a.abs()[:, None] * rel + 8 * U32 * b.abs()[:, None] * torch.zeros_like(p).scatter_(1, at, 1.0)
    e_d += HALF[h.dtype] * (d.abs() + e_d)
    if h.dtype == torch.float16:
        e_d += 2.0 ** -24 / 16384.0 * top
    m = d.abs() + e_d
    k = 2.0 ** -23
    out["dh"], out["dh_tol"] = d @ wd, e_d @ wd.abs() + ((V / 16 + 8 + 2 * pieces) * k) * (m @ wd.abs())
    out["dw"], out["dw_tol"] = d.T @ hd, e_d.T @ hd.abs() + ((T / 16 + 8) * k) * (m.T @ hd.abs())
    return out


# ---------------------------------------------------------------- AdamW (numpy, 32-bit steps as the header defines them)

F = np.float32
ROOTS = np.concatenate([[0.0], [(16 + c % 16) * 2.0 ** (c // 16 - 19) for c in range(1, 256)]])
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def nearest(x, grid):
    """The index of the nearest value; a tie goes to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, side="left"), np.searchsorted(mid, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def encode(m, v):
    """Codes and scales of fp32 m and v (1D)."""
    n = m.size
    pad = (-n) % 256
    mb = np.concatenate([m, np.zeros(pad, F)]).reshape(-1, 256)
    rb = np.sqrt(np.concatenate([v, np.zeros(pad, F)])).reshape(-1, 256)
    assert rb.dtype == F
    codes, scales = [], []
    for b, grid, full in ((mb, E4M3, F(448)), (rb, ROOTS, F(1.9375))):
        top = np.abs(b).max(1)
        some = top >= F(2.0 ** -100)
        safe = np.where(some, top, F(1))
        x = np.abs(b) * (full / safe)[:, None]
        c = nearest(np.minimum(x, full).astype(np.float64), grid)
        if full != 448:
            c = np.where(b > 0, np.maximum(c, 1), c)
        else:
            c = c + 128 * np.signbit(b)
        codes.append(np.where(some[:, None], c, 128 * np.signbit(b) if full == 448 else 0).astype(np.uint8).reshape(-1)[:n])
        scales.append(np.where(some, safe / full, F(0)))
    return codes[0], codes[1], np.stack(scales, 1).astype(F)


def decode(mc, vc, scales):
    u = np.repeat(scales, 256, 0)[:mc.size]
    mag = E4M3[np.minimum(mc & 127, 126)].astype(F)
    m = np.where(mc >= 128, -mag, mag) * u[:, 0]
    r = ROOTS[vc].astype(F) * u[:, 1]
    return m, r * r


def adamw(x, g, m, v, lr, b1, b2, eps, step, decay, scale=1.0):
    """x (float64), m and v (fp32) after a step, a bound for x, and which elements were left alone."""
    with np.errstate(all="ignore"):
        g = (g.astype(F) * F(scale)).astype(F)
        g2 = g * g
        ok = g2 < np.inf
        mn = m * F(b1) + g * F(1 - b1)
        vn = v * F(b2) + g2 * F(1 - b2)
    assert mn.dtype == F and vn.dtype == F
    mn, vn = np.where(ok, mn, m), np.where(ok, vn, v)
    b = lambda t: -np.expm1(step * np.log(t)) if t else 1.0  # noqa: E731
    to = lr * mn.astype(np.float64) / b(b1) / (np.sqrt(vn.astype(np.float64) / b(b2)) + eps)
    xn = np.where(ok, x * (1 - lr * decay) - to, x)
    tol = np.where(ok, 16 * U32 * np.abs(to) + 3 * U32 * np.abs(x), 0.0)
    return xn, mn, vn, tol, ~ok
