"""The 4-bit format and its products against plain 64-bit forms: values at every border of the format, blocks that
hold infinities or NaN, every group size that takes another number of tiles, odd widths, K from one block up."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {torch.float32: m.MOE_F32, torch.bfloat16: m.MOE_BF16, torch.float16: m.MOE_F16}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def quantise(x, rows, cols):
    cb, sb = m.moe_mx4_size(rows, cols)
    codes = torch.full((cb + 32,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((sb + 32,), 0xA5, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_mx4_quantise(x, TYPES[x.dtype], rows, cols, codes, scales, st)
    assert bool((codes[cb:] == 0xA5).all()) and bool((scales[sb:] == 0xA5).all()), "wrote past the end"
    return codes[:cb].clone(), scales[:sb].clone(), m.moe_check_status(st)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (5, 96), (2, 256), (7, 288), (130, 800), (33, 2048), (1, 8192)])
def test_quantise_and_back(moe, rows, cols, dtype):
    rng = np.random.default_rng(rows * cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 12, (rows, cols // 32)).repeat(32, 1))
    x = dev(x.astype(np.float32)).to(dtype)
    codes, scales, st = quantise(x, rows, cols)
    assert st == m.MOE_OK
    code, byte = R.quantise(R.f64(x))
    wc, ws = R.pack(code, byte)
    assert np.array_equal(codes.cpu().numpy().reshape(wc.shape), wc)
    assert np.array_equal(scales.cpu().numpy().reshape(ws.shape), ws)
    for t in (torch.float32, torch.bfloat16):  # exact in both
        out = torch.full((rows, cols), float("nan"), dtype=t, device=DEV)
        m.moe_mx4_dequantise(codes, scales, rows, cols, out, TYPES[t])
        assert np.array_equal(R.f64(out), R.values(code, byte))


def test_borders_of_the_format(moe):
    """Every midpoint between two values, its neighbours in fp32, and saturation, at scales from the smallest to the
    largest."""
    mid = (R.E2M1[1:] + R.E2M1[:-1]) / 2
    probe = np.concatenate([R.E2M1, mid, [6.5, 7.0, 7.96875]])
    probe = np.unique(np.concatenate([probe, np.nextafter(probe.astype(np.float32), np.float32(9)).astype(np.float64),
                                      np.nextafter(probe.astype(np.float32), np.float32(-9)).astype(np.float64)]))
    probe = probe[probe >= 0]
    rows = []
    for e in (-127, -126, -100, -3, 0, 5, 100, 125):
        for a in range(0, len(probe), 30):
            blk = np.zeros(32)
            part = probe[a:a + 30]
            blk[1:1 + len(part)] = part * np.where(np.arange(len(part)) % 2, -1, 1)
            blk[0] = 4.0  # fixes the block's exponent
            rows.append(np.ldexp(blk, e).astype(np.float32))
    rows += [np.zeros(32, np.float32), np.full(32, -0.0, np.float32), np.full(32, 2.0 ** -149, np.float32),
             np.full(32, 2.0 ** -130, np.float32), np.full(32, np.finfo(np.float32).max, np.float32)]
    x = dev(np.stack(rows))
    codes, scales, st = quantise(x, len(rows), 32)
    assert st == m.MOE_OK
    wc, ws = R.pack(*R.quantise(R.f64(x)))
    assert np.array_equal(scales.cpu().numpy().reshape(ws.shape), ws)
    assert np.array_equal(codes.cpu().numpy().reshape(wc.shape), wc)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_block_that_is_not_finite(moe, dtype, bad):
    x = torch.ones(4, 128, dtype=dtype, device=DEV)
    x[2, 70] = bad
    codes, scales, st = quantise(x, 4, 128)
    assert st == m.MOE_ERR_NONFINITE
    out = torch.zeros(4, 128, device=DEV)
    m.moe_mx4_dequantise(codes, scales, 4, 128, out, m.MOE_F32)
    want = torch.ones(4, 128, device=DEV)
    want[2, 64:96] = float("nan")
    assert torch.equal(torch.nan_to_num(out, nan=-1.0), torch.nan_to_num(want, nan=-1.0))


def test_rows_at_a_stride(moe):
    rng = np.random.default_rng(5)
    wide = dev(rng.standard_normal((9, 300)).astype(np.float32))
    for x in (wide[:, 8:8 + 96], wide[:, 3:3 + 96], wide[1:2, :96].expand(9, 96), wide.bfloat16()[:, 1:97]):
        c, s, _ = quantise(x, 9, 96)
        c2, s2, _ = quantise(x.contiguous(), 9, 96)
        assert torch.equal(c, c2) and torch.equal(s, s2)


# ---------------------------------------------------------------- products

def product(rng, E, N, K, offsets, rows, dtype, swiglu, spread=3):
    wr = N * (2 if swiglu else 1)
    xc, xb = rng.integers(0, 16, (rows, K)).astype(np.uint8), rng.integers(127 - spread, 128 + spread, (rows, K // 32)).astype(np.uint8)
    wc, wb = rng.integers(0, 16, (E * wr, K)).astype(np.uint8), rng.integers(120 - spread, 121 + spread, (E * wr, K // 32)).astype(np.uint8)
    x, w = R.values(xc, xb), R.values(wc, wb).reshape(E, wr, K)
    bufs = [dev(a) for a in (*R.pack(wc, wb), *R.pack(xc, xb))]
    out = torch.full((rows * N + 64,), 7.0, dtype=dtype, device=DEV)
    out[:rows * N] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_mx4_matmul(bufs[0], bufs[1], E, N, K, bufs[2], bufs[3], rows, None if offsets is None else dev(offsets),
                     out, TYPES[dtype], m.MOE_MX4_SWIGLU if swiglu else m.MOE_MX4_PLAIN, st)
    assert m.moe_check_status(st) == m.MOE_OK
    assert bool((out[rows * N:] == 7.0).all()), "wrote past the end"
    want, slack = R.matmul(x, w, [0, rows] if offsets is None else offsets, swiglu)
    R.within(out[:rows * N].view(rows, N), want, slack, dtype)
    return bufs, out[:rows * N].view(rows, N)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows,N,K", [
    (1, 1, 32), (1, 128, 256), (2, 7, 64), (1, 2048, 2048), (3, 100, 96), (16, 129, 288), (17, 64, 800), (31, 333, 512),
    (33, 128, 4096), (96, 65, 160), (129, 130, 2048), (224, 256, 256), (225, 96, 544), (449, 200, 320), (1111, 501, 96),
])
def test_one_matrix(moe, rows, N, K, swiglu):
    rng = np.random.default_rng(rows + N + K)
    for dtype in TYPES:
        product(rng, 1, N, K, None, rows, dtype, swiglu)


GROUPS = [
    [1], [0, 0, 5], [3, 0, 0, 1], [0, 0, 0], [17, 1, 0, 31, 2], [40, 0, 300, 1], [225, 224, 223], [1] * 40, [0] * 63 + [9],
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("tail", [0, 6])
@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: f"{len(c)}g{sum(c)}")
def test_groups(moe, counts, tail, swiglu):
    rng = np.random.default_rng(sum(counts) + tail)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(offsets[-1]) + tail
    if rows == 0:
        return
    for N, K, dtype in ((96, 160, torch.float32), (300, 544, torch.bfloat16), (70, 1056, torch.float16)):
        product(rng, len(counts), N, K, offsets, rows, dtype, swiglu)


def test_more_tiles_than_processors(moe):
    rng = np.random.default_rng(9)
    counts = rng.integers(0, 90, 48)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    product(rng, 48, 1100, 320, offsets, int(offsets[-1]), torch.bfloat16, False)
    product(rng, 48, 520, 320, offsets, int(offsets[-1]), torch.bfloat16, True)


def test_most_experts(moe):
    rng = np.random.default_rng(10)
    counts = (rng.random(1024) < 0.02).astype(np.int64) * rng.integers(1, 4, 1024)
    counts[1023] = 2
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    product(rng, 1024, 40, 64, offsets, int(offsets[-1]), torch.float32, False)


def test_scales_far_apart(moe):
    rng = np.random.default_rng(11)
    product(rng, 1, 140, 512, None, 50, torch.float32, False, spread=30)


def test_nan_stays_in_its_row_and_column(moe):
    rng = np.random.default_rng(12)
    rows, N, K = 40, 150, 320
    (wc, ws, xc, xs), ok = product(rng, 1, N, K, None, rows, torch.float32, False)
    ws.view(N, -1)[77, 3] = 255
    xs.view(rows, -1)[11, 9] = 255
    out = torch.zeros(rows, N, device=DEV)
    m.moe_mx4_matmul(wc, ws, 1, N, K, xc, xs, rows, None, out)
    want = ok.clone()
    want[11, :] = float("nan")
    want[:, 77] = float("nan")
    assert torch.equal(torch.nan_to_num(out, nan=-1.0), torch.nan_to_num(want, nan=-1.0))


def test_a_row_does_not_depend_on_its_company(moe):
    """The same row alone, in a batch and in another group's company: the same bits where the same K is summed in
    one piece."""
    rng = np.random.default_rng(13)
    N, K, rows = 200, 256, 300
    (wc, ws, xc, xs), all_rows = product(rng, 1, N, K, None, rows, torch.float32, False)
    for r in (0, 7, 299):
        one = torch.empty(1, N, device=DEV)
        m.moe_mx4_matmul(wc, ws, 1, N, K, xc.view(rows, -1)[r].clone(), xs.view(rows, -1)[r].clone(), 1, None, one)
        assert torch.equal(one[0], all_rows[r])


def test_same_bits_every_time(moe):
    rng = np.random.default_rng(14)
    (wc, ws, xc, xs), first = product(rng, 1, 300, 2048, None, 5, torch.float32, False)
    for _ in range(3):
        again = torch.empty_like(first)
        m.moe_mx4_matmul(wc, ws, 1, 300, 2048, xc, xs, 5, None, again)
        assert torch.equal(again, first)


def test_many_steps_through_few_stages(moe):
    """The widest tiles leave four stages, which a long K passes through many times: the same bits every time."""
    rng = np.random.default_rng(17)
    for rows, N in ((449, 2501), (1111, 300)):
        (wc, ws, xc, xs), first = product(rng, 1, N, 4064, None, rows, torch.float32, False)
        for _ in range(40):
            again = torch.empty_like(first)
            m.moe_mx4_matmul(wc, ws, 1, N, 4064, xc, xs, rows, None, again)
            assert torch.equal(again, first)


def test_bad_offsets_are_clipped_and_reported(moe):
    rng = np.random.default_rng(15)
    for bad in ([0, 3, 2, 6], [-4, 2, 3, 6], [0, 2, 3, 1000], [2 ** 31 - 1, -2 ** 31, 0, 6]):
        rows, N, K = 6, 64, 64
        code, byte = rng.integers(0, 16, (rows, K)).astype(np.uint8), np.full((rows, 2), 127, np.uint8)
        wcode, wbyte = rng.integers(0, 16, (3 * N, K)).astype(np.uint8), np.full((3 * N, 2), 127, np.uint8)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.zeros(rows * N + 64, device=DEV)
        args = [dev(a) for a in (*R.pack(wcode, wbyte), *R.pack(code, byte))]
        m.moe_mx4_matmul(args[0], args[1], 3, N, K, args[2], args[3], rows, dev(np.array(bad, np.int32)), out,
                         dev_status=st)
        assert m.moe_check_status(st) == m.MOE_ERR_BOUNDS
        assert bool((out[rows * N:] == 0).all())


def test_outputs_past_32_bits(moe):
    """More than 2^31 values out (and in), the last rows against the same rows alone."""
    rows, N, K = 1_060_000, 2050, 32
    rng = np.random.default_rng(19)
    wc, ws = [dev(a) for a in R.pack(rng.integers(0, 16, (N, K)).astype(np.uint8), rng.integers(125, 130, (N, 1)).astype(np.uint8))]
    x = torch.randn(rows, K, device=DEV)
    cb, sb = m.moe_mx4_size(rows, K)
    xc, xs = torch.empty(rows, cb // rows, dtype=torch.uint8, device=DEV), torch.empty(rows, sb // rows, dtype=torch.uint8, device=DEV)
    m.moe_mx4_quantise(x, m.MOE_F32, rows, K, xc, xs)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    m.moe_mx4_matmul(wc, ws, 1, N, K, xc, xs, rows, None, out, m.MOE_BF16)
    assert out.numel() > 2 ** 31
    for a in (0, 524_288, rows - 40):
        one = torch.empty(40, N, dtype=torch.bfloat16, device=DEV)
        m.moe_mx4_matmul(wc, ws, 1, N, K, xc[a:a + 40].contiguous(), xs[a:a + 40].contiguous(), 40, None, one, m.MOE_BF16)
        assert torch.equal(out[a:a + 40], one)
    wide = torch.empty(rows, 2048, dtype=torch.bfloat16, device=DEV)  # quantise and back past 2^31 values
    wide[:] = out[:, :2048]
    cb, sb = m.moe_mx4_size(rows, 2048)
    c, s = torch.empty(cb, dtype=torch.uint8, device=DEV), torch.empty(sb, dtype=torch.uint8, device=DEV)
    m.moe_mx4_quantise(wide, m.MOE_BF16, rows, 2048, c, s)
    back = torch.empty_like(wide)
    m.moe_mx4_dequantise(c, s, rows, 2048, back)
    for a in (0, rows - 8):
        code, byte = R.quantise(R.f64(wide[a:a + 8]))
        assert np.array_equal(R.f64(back[a:a + 8]), R.values(code, byte))


def test_products_on_several_streams(moe):
    rng = np.random.default_rng(18)
    cases = [product(rng, 1, 700, 1024, None, 300, torch.float32, False), product(rng, 1, 256, 4096, None, 3, torch.float32, False)]
    sizes = [(1, 700, 1024, 300), (1, 256, 4096, 3)]
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(4)]
    for i in range(24):
        (wc, ws, xc, xs), want = cases[i % 2]
        E, N, K, rows = sizes[i % 2]
        with torch.cuda.stream(streams[i % 4]):
            o = torch.empty_like(want)
            m.moe_mx4_matmul(wc, ws, E, N, K, xc, xs, rows, None, o)
        outs.append((o, want))
    torch.cuda.synchronize()
    for o, want in outs:
        assert torch.equal(o, want)


def test_captured_in_a_graph(moe):
    rng = np.random.default_rng(16)
    rows, N, K = 12, 256, 512
    x = dev(rng.standard_normal((rows, K)).astype(np.float32))
    (wc, ws, _, _), _ = product(rng, 1, N, K, None, rows, torch.float32, False)
    cb, sb = m.moe_mx4_size(rows, K)
    codes, scales = torch.empty(cb, dtype=torch.uint8, device=DEV), torch.empty(sb, dtype=torch.uint8, device=DEV)
    out = torch.empty(rows, N, device=DEV)

    def step():
        m.moe_mx4_quantise(x, m.MOE_F32, rows, K, codes, scales)
        m.moe_mx4_matmul(wc, ws, 1, N, K, codes, scales, rows, None, out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(dev(rng.standard_normal((rows, K)).astype(np.float32)))
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    step()
    assert torch.equal(got, out)
