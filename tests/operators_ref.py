"""Plain 64-bit forms of the row, 4-bit and norm operators (numpy), and error
bounds for kernels that compute them with 32-bit sums."""
import numpy as np
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # smallest subnormal
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, slack, dtype):
    """|got - want| <= slack (error before the rounding) + half a step of the output's type."""
    got, want = f64(got), np.asarray(want, np.float64)
    tol = slack + HALF[dtype] * (np.abs(want) + slack) + TINY[dtype]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside; first at {np.argwhere(bad)[0]}: got {got[bad][0]!r}, "
                           f"want {want[bad][0]!r} +- {np.broadcast_to(tol, got.shape)[bad][0]:.3e}")


def sorted_pairs(ids, E):
    """offsets, perm and inverse of the stable sort of the (token, slot) pairs; ids outside [0, E) are left out."""
    flat = np.asarray(ids).reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")
    n = int(ok.sum())
    perm = np.full(flat.size, -1, np.int32)
    perm[:n] = order[:n]
    inv = np.full(flat.size, -1, np.int32)
    inv[perm[:n]] = np.arange(n)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))]).astype(np.int32)
    return offsets, perm, inv


def quantise(x):
    """codes (one per entry, sign at bit 3) and scale bytes per 32, from values held exactly in x (float64)."""
    r, c = x.shape
    b = x.reshape(r, c // 32, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(np.isfinite(b), b, 0.0)
    m = np.abs(b).max(2)
    _, e = np.frexp(m)
    e = np.where(m > 0, np.maximum(e - 3, -127), -127)
    a = np.ldexp(np.abs(b), -e[:, :, None])
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    code = np.where(lo % 2 == 0, lo, hi)  # a tie goes to the even mantissa
    code = code + 8 * np.signbit(b)
    code = np.where(bad[:, :, None], 0, code)
    byte = np.where(bad, 255, e + 127)
    return code.reshape(r, c).astype(np.uint8), byte.astype(np.uint8)


def pack(code, byte):
    """The stored form: two codes per byte, scale rows padded with zeros to a multiple of 32 bytes."""
    r = code.shape[0]
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    scales = np.zeros((r, (byte.shape[1] + 31) // 32 * 32), np.uint8)
    scales[:, :byte.shape[1]] = byte
    return codes, scales


def values(code, byte):
    r, c = code.shape
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return (v.reshape(r, -1, 32) * s[:, :, None]).reshape(r, c)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def matmul(x, w, offsets, swiglu):
    """Rows times their group's weights [E][rows][K], and a bound of the error of the same sums in 32 bits: each of
    the K/64 steps may round the running sum and its own 64 products' sum, at most 2^-23 of the magnitudes each."""
    E, wr, K = w.shape
    N = wr // 2 if swiglu else wr
    out, slack = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N))
    u = (K / 64 + 8) * 2.0 ** -23
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        y, m = x[a:b] @ w[e].T, np.abs(x[a:b]) @ np.abs(w[e].T)
        if not swiglu:
            out[a:b], slack[a:b] = y, u * m
            continue
        g, up, dg, du = y[:, :N], y[:, N:], u * m[:, :N], u * m[:, N:]
        out[a:b] = silu(g) * up
        slack[a:b] = 1.1 * dg * np.abs(up) + (np.abs(silu(g)) + 1.1 * dg) * du + 16 * U32 * np.abs(out[a:b])
    return out, slack


def block_norm(x, b, w_post, w_pre, gate, alpha, eps):
    """v' = alpha gate v, y, u, r1, r2; gate broadcasts over [T][H]."""
    r1 = 1.0 / np.sqrt((b * b).mean(1, keepdims=True) + eps)
    v = b * r1 * w_post
    y = x + alpha * gate * v
    r2 = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    return v, y, y * r2 * w_pre, r1, r2


def block_norm_backward(x, b, w_post, w_pre, gate, alpha, eps, dy, du):
    """The gradients, and the sums of the magnitudes that each is made of."""
    v, y, _, r1, r2 = block_norm(x, b, w_post, w_pre, gate, alpha, eps)

    def parts(sgn):
        f = (lambda a: a) if sgn else np.abs
        m = 1.0 if sgn else -1.0
        x_ = y if sgn else np.abs(x) + np.abs(alpha * gate * v)
        d2 = f(du) * f(w_pre)
        t = f(dy) + r2 * d2 - m * x_ * r2 ** 3 * (d2 * x_).mean(1, keepdims=True)
        dv = f(alpha * gate * np.ones_like(x)) * t
        d1 = dv * f(w_post)
        db = r1 * d1 - m * f(b) * r1 ** 3 * (d1 * f(b)).mean(1, keepdims=True)
        return t, db, dv * f(b) * r1, f(du) * x_ * r2, f(np.float64(alpha)) * t * f(v)

    return parts(True), parts(False)
