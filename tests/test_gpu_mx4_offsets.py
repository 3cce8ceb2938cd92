"""Group offsets of the 4-bit product at their limits: more tiles than fit a count of every group with all rows, and
offsets that are not in order."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R
from test_gpu_mx4 import DEV, dev, product

pytestmark = pytest.mark.gpu


def test_many_groups_of_a_wide_matrix(moe):
    """1,024 groups of 16,384 rows, 2,049 column tiles: two million tiles, though groups x row tiles x column tiles
    pass 2^30.  Columns at both ends and between, all rows, against 64 bits."""
    E, rows, N, K = 1024, 16384, 262_272, 32
    rng = np.random.default_rng(21)
    offsets = np.concatenate([[0], np.sort(rng.integers(0, rows, E - 1)), [rows - 5]]).astype(np.int32)
    offsets = np.minimum(offsets, rows - 5)
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    wc = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.zeros(E, N, 32, dtype=torch.uint8, device=DEV)
    ws[:, :, 0] = torch.randint(117, 124, (E, N), generator=g, device=DEV, dtype=torch.uint8)
    xc, xb = rng.integers(0, 16, (rows, K)).astype(np.uint8), rng.integers(124, 131, (rows, 1)).astype(np.uint8)
    bufs = [dev(a) for a in R.pack(xc, xb)]
    out = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_mx4_matmul(wc, ws, E, N, K, bufs[0], bufs[1], rows, dev(offsets), out, m.MOE_BF16, dev_status=st)
    assert m.moe_check_status(st) == m.MOE_OK
    cols = torch.tensor([0, 1, 127, 128, 131_071, 200_000, N - 129, N - 128, N - 1], device=DEV)
    c = wc[:, cols].cpu().numpy().reshape(-1, K // 2)
    code = np.empty((c.shape[0], K), np.uint8)
    code[:, 0::2], code[:, 1::2] = c & 15, c >> 4
    w = R.values(code, ws[:, cols, :1].cpu().numpy().reshape(-1, 1)).reshape(E, len(cols), K)
    want, slack = R.matmul(R.values(xc, xb), w, offsets, False)
    R.within(out[:, cols], want, slack, torch.bfloat16)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("bad,good", [
    ([0, 90, 0, 90, 0, 90], [0, 90, 90, 90, 90, 90]),          # every other group asks for all rows
    ([0, 40, 20, 60, 50, 90], [0, 40, 40, 60, 60, 90]),
    ([-7, 30, 200, 10, 20, 80], [0, 30, 90, 90, 90, 90]),
    ([2 ** 31 - 1, -2 ** 31, 0, 6, 90, 3], [90, 90, 90, 90, 90, 90]),
    ([0, 10, 20, 30, 40, -1], [0, 10, 20, 30, 40, 40]),
])
def test_offsets_out_of_order(moe, bad, good, swiglu):
    """Reported, and each group begins no earlier than the one before it ends: the bits of those offsets."""
    E, N, K, rows = 5, 200, 96, 90
    rng = np.random.default_rng(22)
    bufs, _ = product(rng, E, N, K, np.array([0, 20, 40, 60, 80, 90], np.int32), rows, torch.float32, swiglu)
    outs = []
    for off, status in ((bad, m.MOE_ERR_BOUNDS), (good, m.MOE_OK)):
        out = torch.full((rows, N), float("nan"), device=DEV)
        out[:good[0]] = 0
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        m.moe_mx4_matmul(*bufs[:2], E, N, K, *bufs[2:], rows, dev(np.array(off, np.int32)), out,
                         epilogue=m.MOE_MX4_SWIGLU if swiglu else m.MOE_MX4_PLAIN, dev_status=st)
        assert m.moe_check_status(st) == status
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and not bool(outs[0].isnan().any())


def test_most_groups_out_of_order(moe):
    rng = np.random.default_rng(23)
    E, N, K, rows = 1024, 40, 64, 3000
    bufs, want = product(rng, E, N, K, np.array([0] + [rows] * E, np.int32), rows, torch.float32, False)
    out = torch.full_like(want, float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_mx4_matmul(*bufs[:2], E, N, K, *bufs[2:], rows, dev(np.array([0, rows] * (E // 2) + [0], np.int32)), out, dev_status=st)
    assert m.moe_check_status(st) == m.MOE_ERR_BOUNDS
    assert torch.equal(out, want)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("offsets,rows,N,K", [
    ([3, 7, 7, 12], 12, 96, 160), ([1, 1, 2, 2], 5, 33, 288), ([40, 300, 300, 301], 310, 70, 64), ([6, 6, 6, 6], 6, 130, 96),
    ([1000, 1002, 1003, 1040], 1040, 257, 4096),
])
def test_a_slice_of_offsets(moe, offsets, rows, N, K, dtype, swiglu):
    """The first group begins past row 0: the rows before it are zero as those after the last."""
    rng = np.random.default_rng(rows + N)
    product(rng, 3, N, K, np.array(offsets, np.int32), rows, dtype, swiglu, spread=0)
