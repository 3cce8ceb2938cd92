"""The sort of the pairs at every size where its form changes, without a workspace where none is asked for, with and
without the library's own scratch: left-out pairs, ids that are out of range, buffers' ends."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [(1, 1, 1), (1, 1, 1024), (1, 10, 512), (4, 10, 512), (31, 1, 3), (3, 11, 128), (16, 4, 127), (13, 5, 2), (127, 1, 1024),
         (32, 4, 1), (8, 16, 512), (43, 3, 129), (256, 4, 1024), (1025, 1, 60), (4097, 1, 512), (2048, 16, 1024), (32768, 1, 7)]


def sort(fn, ids, T, k, E):
    n = T * k
    bufs = [torch.full((x + 8,), -7, dtype=torch.int32, device=DEV) for x in (E + 1, n, n)]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    fn(torch.from_numpy(ids).to(DEV), T, k, E, *bufs, dev_status=st)
    status = m.moe_check_status(st)
    got = [b.cpu().numpy() for b in bufs]
    assert all((b[-8:] == -7).all() for b in got), "wrote past the end"
    return status, [b[:-8] for b in got]


@pytest.mark.parametrize("left_out", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_without_a_workspace(moe, T, k, E, left_out):
    rng = np.random.default_rng(T * k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < left_out] = -1
    for fn in (m.moe_permute, m.moe_permute_noalloc):
        status, got = sort(fn, ids, T, k, E)
        assert status == m.MOE_OK
        for a, b in zip(got, R.sorted_pairs(ids, E)):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("bad", ["E", -2, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_ids_out_of_range(moe, T, k, E, bad):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[T // 2, k - 1] = E if bad == "E" else bad
    for fn in (m.moe_permute, m.moe_permute_noalloc):
        status, got = sort(fn, ids, T, k, E)
        assert status == m.MOE_ERR_BOUNDS
        for a, b in zip(got, R.sorted_pairs(ids, E)):
            assert np.array_equal(a, b)
