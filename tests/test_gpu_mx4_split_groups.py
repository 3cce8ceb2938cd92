"""Grouped products of few rows and a long K, whose K a cluster of CTAs shares: groups empty, of one to three rows, of
more rows than a tile, fewer rows than CTAs, rows of no group.  (On 152 SMs the plan gives 64 of the 90 shapes eight
CTAs, 20 four and 5 two, 78 of the 90 at less than 0.75 of the unsplit cost.)"""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_mx4 import DEV, TYPES, dev, product

pytestmark = pytest.mark.gpu
GROUPS = [([1, 0, 3], 0), ([0, 2, 0, 1, 0, 0, 5, 0], 6), ([3], 6), ([40, 0, 1], 0), ([1] * 10, 6), ([0] * 15 + [2], 3),
          ([0, 0, 0], 4), ([70, 2], 0), ([0, 3, 1, 0, 0, 0, 0, 0], 1)]


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N,K", [(200, 4096), (512, 4096), (70, 8192), (33, 4128), (65, 16384)])
@pytest.mark.parametrize("counts,tail", GROUPS, ids=str)
def test_split_groups(moe, counts, tail, N, K, swiglu):
    rng = np.random.default_rng(sum(counts) + 7 * tail + N + K)
    for dtype in TYPES:  # (scales that keep fp16 outputs in range)
        product(rng, len(counts), N, K, offsets_of(counts), sum(counts) + tail, dtype, swiglu, spread=0)


@pytest.mark.parametrize("swiglu", [False, True])
def test_split_groups_have_the_same_bits_every_time(moe, swiglu):
    rng = np.random.default_rng(31)
    offsets = offsets_of([0, 3, 1, 0, 0, 2, 0, 0])
    E, N, K, rows = 8, 300, 8192, 8
    bufs, first = product(rng, E, N, K, offsets, rows, torch.float32, swiglu)
    off = dev(offsets)
    for _ in range(200):
        again = torch.full_like(first, float("nan"))
        m.moe_mx4_matmul(*bufs[:2], E, N, K, *bufs[2:], rows, off, again, epilogue=m.MOE_MX4_SWIGLU if swiglu else m.MOE_MX4_PLAIN)
        assert torch.equal(again, first)


@pytest.mark.parametrize("swiglu", [False, True])
def test_split_groups_from_the_end_of_a_slice_and_out_of_order(moe, swiglu):
    rng = np.random.default_rng(32)
    E, N, K, rows = 4, 200, 8192, 9
    good = np.array([2, 2, 5, 6, 8], np.int32)
    bufs, want = product(rng, E, N, K, good, rows, torch.float32, swiglu)
    out = torch.full_like(want, float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_mx4_matmul(*bufs[:2], E, N, K, *bufs[2:], rows, dev(np.array([2, 1, 5, 6, 8], np.int32)), out,
                     epilogue=m.MOE_MX4_SWIGLU if swiglu else m.MOE_MX4_PLAIN, dev_status=st)
    assert m.moe_check_status(st) == m.MOE_ERR_BOUNDS
    assert torch.equal(out, want)
