"""moe_dispatch, moe_combine and their gradients against plain 64-bit forms: types, odd widths, strides, left-out
pairs and tokens, tails past the last pair, and buffers' ends."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {torch.float32: m.MOE_F32, torch.bfloat16: m.MOE_BF16, torch.float16: m.MOE_F16}
SHAPES = [  # T, H, E, k, part of the pairs left out
    (1, 8, 2, 1, 0.0), (1, 2048, 512, 10, 0.0), (4, 2048, 512, 10, 0.3), (3, 1, 4, 2, 0.0), (5, 33, 4, 3, 0.5),
    (7, 250, 1, 1, 0.0), (64, 1001, 60, 4, 0.5), (33, 264, 16, 16, 0.1), (700, 768, 64, 6, 0.0), (129, 8192, 8, 2, 0.9),
    (40, 100, 8, 8, 1.0), (300, 2046, 24, 5, 0.2), (9, 6, 4, 2, 0.0),
]


def case(T, H, E, k, out, seed):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < out] = -1
    if T > 2:
        ids[1] = -1  # a token with no pair at all
    return rng, ids, R.sorted_pairs(ids, E)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def guarded(n, dtype, fill=float("nan")):
    """A buffer of n elements with a guard behind it."""
    buf = torch.full((n + 64,), 7.0, dtype=dtype, device=DEV)
    buf[:n] = fill
    return buf, buf[:n]


def unhurt(buf, n):
    assert bool((buf[n:] == 7.0).all()), "wrote past the end"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_dispatch_and_its_gradient(moe, shape, dtype):
    T, H, E, k, out = shape
    rng, ids, (offsets, perm, inv) = case(*shape, seed=1)
    x = dev(rng.standard_normal((T, H), np.float32)).to(dtype)
    buf, rows = guarded(T * k * H, dtype)
    m.moe_dispatch(x, TYPES[dtype], T, H, k, E, dev(offsets), dev(inv), rows)
    want = np.zeros((T * k, H))
    n = offsets[-1]
    want[:n] = R.f64(x)[perm[:n] // k]
    assert np.array_equal(R.f64(rows).reshape(T * k, H), want)
    unhurt(buf, T * k * H)

    dr = dev(rng.standard_normal((T * k, H), np.float32)).to(dtype)
    dr[int(n):] = float("nan")  # rows of no pair must not be read into a sum
    buf, dx = guarded(T * H, dtype)
    m.moe_dispatch_backward(dr, TYPES[dtype], T, H, k, dev(inv), dx)
    d = np.nan_to_num(R.f64(dr))
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(want, perm[:n] // k, d[:n])
    np.add.at(mag, perm[:n] // k, np.abs(d[:n]))
    R.within(dx.view(T, H), want, k * R.U32 * mag, dtype)
    unhurt(buf, T * H)


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_combine(moe, shape, dtype, accumulate, out_f32):
    T, H, E, k, out = shape
    rng, ids, (offsets, perm, inv) = case(*shape, seed=2)
    y = dev(rng.standard_normal((T * k, H), np.float32)).to(dtype)
    y[int(offsets[-1]):] = float("nan")
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[ids < 0] = np.inf  # the weight of a left-out pair is not looked at
    ot = torch.float32 if out_f32 else dtype
    buf, o = guarded(T * H, ot)
    old = dev(rng.standard_normal((T, H), np.float32)).to(ot)
    if accumulate:
        o.copy_(old.view(-1))
    m.moe_combine(y, TYPES[dtype], T, H, k, dev(w), dev(inv), o, TYPES[ot], accumulate)
    want = R.f64(old) if accumulate else np.zeros((T, H))
    mag = np.abs(want)
    yv = R.f64(y)
    for t in range(T):
        for j in range(k):
            if inv[t * k + j] >= 0:
                want[t] += float(w[t, j]) * yv[inv[t * k + j]]
                mag[t] += abs(float(w[t, j])) * np.abs(yv[inv[t * k + j]])
    R.within(o.view(T, H), want, (k + 1) * R.U32 * mag, ot)
    unhurt(buf, T * H)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_gradients(moe, shape, dtype):
    T, H, E, k, out = shape
    rng, ids, (offsets, perm, inv) = case(*shape, seed=3)
    n = int(offsets[-1])
    y = dev(rng.standard_normal((T * k, H), np.float32)).to(dtype)
    y[n:] = float("nan")
    dout = dev(rng.standard_normal((T, H), np.float32)).to(dtype)
    w = rng.standard_normal((T, k)).astype(np.float32)
    b1, dy = guarded(T * k * H, dtype)
    b2, dw = guarded(T * k, torch.float32)
    m.moe_combine_backward(dout, y, TYPES[dtype], T, H, k, E, dev(offsets), dev(w), dev(inv), dy, dw)
    d, yv = R.f64(dout), R.f64(y)
    want = np.zeros((T * k, H))
    want[:n] = d[perm[:n] // k] * w.astype(np.float64).reshape(-1)[perm[:n], None]
    R.within(dy.view(T * k, H), want, 0.0, dtype)
    wd, mag = np.zeros(T * k), np.zeros(T * k)
    wd[perm[:n]] = (d[perm[:n] // k] * yv[:n]).sum(1)
    mag[perm[:n]] = np.abs(d[perm[:n] // k] * yv[:n]).sum(1)
    # a lane adds at most H/32 + 8 terms in turn, then a tree of five
    R.within(dw, wd, (H / 32 + 14) * R.U32 * mag, torch.float32)
    unhurt(b1, T * k * H)
    unhurt(b2, T * k)


def test_combine_gradient_is_the_difference_quotient(moe):
    """<dy, a> + <dw, c> against the 64-bit combine moved along (a, c): it is linear in each, so the central
    difference is exact but for its own rounding."""
    T, H, E, k = 9, 72, 6, 3
    rng, ids, (offsets, perm, inv) = case(T, H, E, k, 0.2, seed=4)
    y, w = rng.standard_normal((T * k, H)).astype(np.float32), rng.random((T, k)).astype(np.float32)
    g = rng.standard_normal((T, H)).astype(np.float32)
    dy, dw = torch.empty(T * k, H, device=DEV), torch.empty(T, k, device=DEV)
    m.moe_combine_backward(dev(g), dev(y), m.MOE_F32, T, H, k, E, dev(offsets), dev(w), dev(inv), dy, dw)
    a, c = rng.standard_normal((T * k, H)), rng.standard_normal((T, k))

    def loss(s):
        yy, ww = y + s * a, (w + s * c).reshape(-1)
        n = offsets[-1]
        return (g[perm[:n] // k] * yy[:n] * ww[perm[:n], None]).sum()

    h = 1e-3
    want = (loss(h) - loss(-h)) / (2 * h)
    got = (R.f64(dy) * a).sum() + (R.f64(dw) * c).sum()
    mag = np.abs(R.f64(dy) * a).sum() + (np.abs(c) * np.abs(g).sum(1, keepdims=True)).sum() * np.abs(y).max()
    assert abs(got - want) <= (H / 32 + 14) * R.U32 * mag + 1e-9 * mag


@pytest.mark.parametrize("dtype", TYPES)
def test_dispatch_gradient_is_its_adjoint(moe, dtype):
    """<dispatch(x), g> = <x, dispatch_backward(g)>: the difference quotient of a linear map, without its rounding."""
    T, H, E, k = 21, 136, 9, 4
    rng, ids, (offsets, perm, inv) = case(T, H, E, k, 0.3, seed=8)
    x, g = (dev(rng.standard_normal(s).astype(np.float32)).to(dtype) for s in ((T, H), (T * k, H)))
    rows, dx = torch.empty_like(g), torch.empty_like(x)
    m.moe_dispatch(x, TYPES[dtype], T, H, k, E, dev(offsets), dev(inv), rows)
    m.moe_dispatch_backward(g, TYPES[dtype], T, H, k, dev(inv), dx)
    a, b = (R.f64(rows) * R.f64(g)).sum(), (R.f64(x) * R.f64(dx)).sum()
    mag = np.abs(R.f64(rows) * R.f64(g)).sum()  # dx is off by k roundings of its sum and one to its type, at most of mag
    assert abs(a - b) <= (k * R.U32 + R.HALF[dtype]) * mag * 1.01


def test_dispatch_takes_rows_at_a_stride_and_one_row_for_all(moe):
    T, H, E, k = 13, 48, 5, 2
    rng, ids, (offsets, perm, inv) = case(T, H, E, k, 0.0, seed=5)
    n = int(offsets[-1])
    wide = dev(rng.standard_normal((T, 3 * H + 1), np.float32))
    for x in (wide[:, H:2 * H], wide[:, 1:H + 1], wide[2:3, :H].expand(T, H)):
        rows = torch.empty(T * k, H, device=DEV)
        m.moe_dispatch(x, m.MOE_F32, T, H, k, E, dev(offsets), dev(inv), rows)
        assert torch.equal(rows[:n], x[dev(perm[:n]).long() // k])


def test_entries_out_of_range_count_as_left_out(moe):
    T, H, E, k = 6, 40, 4, 2
    rng, ids, (offsets, perm, inv) = case(T, H, E, k, 0.0, seed=6)
    inv[0], inv[5] = T * k, -2 ** 31
    y = rng.standard_normal((T * k, H)).astype(np.float32)
    o = torch.empty(T, H, device=DEV)
    m.moe_dispatch_backward(dev(y), m.MOE_F32, T, H, k, dev(inv), o)
    want = np.zeros((T, H))
    for i, p in enumerate(inv):
        if 0 <= p < T * k:
            want[i // k] += y[p]
    R.within(o, want, k * R.U32 * np.abs(y).max(), torch.float32)
    offsets[-1] = 10 ** 9  # nothing to clear: clipped to the rows
    m.moe_dispatch(dev(y[:T].copy()), m.MOE_F32, T, H, k, E, dev(offsets), dev(inv), torch.empty(T * k, H, device=DEV))


def test_same_bits_every_time_and_on_another_stream(moe):
    T, H, E, k = 300, 520, 32, 8
    rng, ids, (offsets, perm, inv) = case(T, H, E, k, 0.1, seed=7)
    y, w, g = (dev(rng.standard_normal(s).astype(np.float32)) for s in ((T * k, H), (T, k), (T, H)))
    got = []
    torch.cuda.synchronize()
    for s in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            o, dy, dw = torch.empty(T, H, device=DEV), torch.empty(T * k, H, device=DEV), torch.empty(T, k, device=DEV)
            m.moe_combine(y, m.MOE_F32, T, H, k, w, dev(inv), o)
            m.moe_combine_backward(g, y, m.MOE_F32, T, H, k, E, dev(offsets), w, dev(inv), dy, dw)
        s.synchronize()
        got.append((o, dy, dw))
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (3, 2, 1024), (32, 16, 1024), (256, 16, 1024), (409, 10, 1024), (410, 10, 1000),
                                   (1365, 3, 375), (1366, 3, 375), (4096, 1, 7), (5000, 3, 33), (3276, 10, 512),
                                   (3277, 10, 512), (8200, 10, 1000), (40000, 10, 1024), (70000, 3, 5)])
def test_sort_of_the_pairs(moe, T, k, E):
    """The sort that the rows go by, at the sizes where its runs and chunks change, with pairs left out."""
    rng = np.random.default_rng(T * k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    off, perm, inv = (torch.full((n,), -7, dtype=torch.int32, device=DEV) for n in (E + 1, T * k, T * k))
    nb = m.moe_permute_workspace_size(T, k, E)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_permute(dev(ids), T, k, E, off, perm, inv, torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV), nb, st)
    assert m.moe_check_status(st) == m.MOE_OK
    for got, want in zip((off, perm, inv), R.sorted_pairs(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_no_tokens(moe):
    m.moe_dispatch(torch.empty(0, 8, device=DEV), m.MOE_F32, 0, 8, 2, 4, torch.zeros(5, dtype=torch.int32, device=DEV),
                   torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 8, device=DEV))
    m.moe_combine(torch.empty(0, 8, device=DEV), m.MOE_F32, 0, 8, 2, torch.empty(0, 2, device=DEV),
                  torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 8, device=DEV))


def test_offsets_past_32_bits(moe):
    """Rows whose element index passes 2^31."""
    T, H, k = 270_000, 8192, 1
    inv = torch.arange(T, dtype=torch.int32, device=DEV).flip(0).contiguous()
    offsets = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x[:] = (torch.arange(T, device=DEV) % 251).to(torch.bfloat16)[:, None]
    rows = torch.empty_like(x)
    m.moe_dispatch(x, m.MOE_BF16, T, H, k, 1, offsets, inv, rows)
    assert torch.equal(rows[:, 0], x[:, 0].flip(0)) and torch.equal(rows[:, -1], x[:, -1].flip(0))
    back = torch.empty_like(x)
    m.moe_dispatch_backward(rows, m.MOE_BF16, T, H, k, inv, back)
    assert torch.equal(back, x)
