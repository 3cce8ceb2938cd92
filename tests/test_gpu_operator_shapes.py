"""Seeded random shapes through the row, 4-bit and norm operators, each against its plain 64-bit form: sizes over
their whole ranges, spread over their logarithm, groups empty, small, even or all in one."""
import numpy as np
import pytest
import torch

import test_gpu_block_norm as norms
import test_gpu_mx4 as mx4
import test_gpu_rows as rows

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def spread(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(40))
def test_products(moe, seed):
    rng = np.random.default_rng(seed)
    E = 1 if rng.random() < 0.35 else spread(rng, 2, 300)
    N, K, swiglu = spread(rng, 1, 700), 32 * spread(rng, 1, 90), bool(rng.random() < 0.5)
    while E * N * K > 3e7:
        E, N = max(1, E // 2), max(1, N * 2 // 3)
    counts = [np.array([spread(rng, 1, 900)]) if E == 1 else rng.integers(0, 4, E),
              (rng.random(E) < 0.2) * rng.integers(0, 300, E), rng.integers(0, 60, E),
              np.where(np.arange(E) == rng.integers(0, E), spread(rng, 1, 900), 0)][seed % 4]
    while counts.sum() * K * N > 2e9:
        counts = counts // 2
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(offsets[-1]) + int(rng.integers(0, 9))
    dtype = TYPES[seed % 3]
    if n:  # (fp16 outputs: scales that keep them in its range)
        mx4.product(rng, E, N, K, offsets, n, dtype, swiglu, spread=0 if dtype == torch.float16 else int(rng.integers(0, 8)))


@pytest.mark.parametrize("seed", range(40))
def test_rows(moe, seed):
    rng = np.random.default_rng(1000 + seed)
    T, H, E = spread(rng, 1, 400), spread(rng, 1, 3000), spread(rng, 1, 400)
    shape = (T, H, E, int(rng.integers(1, min(E, 16) + 1)), [0.0, 0.2, 0.7, 1.0][seed % 4])
    rows.test_dispatch_and_its_gradient(moe, shape, TYPES[seed % 3])
    rows.test_combine(moe, shape, TYPES[seed % 3], bool(seed & 1), bool(seed & 2))
    rows.test_combine_gradients(moe, shape, TYPES[seed % 3])
    rows.test_sort_of_the_pairs(moe, spread(rng, 1, 6000), shape[3], E)


@pytest.mark.parametrize("seed", range(60))
def test_norms_and_quantisation(moe, seed):
    rng = np.random.default_rng(2000 + seed)
    T, H = spread(rng, 1, 300), spread(rng, 1, 16384 if seed % 3 == 0 else 2500)
    (res, act), gate = norms.PAIRS[seed % 5], list(norms.GATES)[seed % 3]
    norms.test_forward(moe, T, H, res, act, gate)
    norms.test_gradients(moe, T, H, res, act, gate)
    mx4.test_quantise_and_back(moe, spread(rng, 1, 300), 32 * spread(rng, 1, 100), TYPES[seed % 3])
