"""Seeded random shapes, types and options through the training operators, against their 64-bit forms."""
import math
import random

import pytest
import torch

import bit_expert_ffn_gb300 as m
import test_gpu_adamw as aw
import test_gpu_cross_entropy as ce
import test_gpu_router_loss as rl
from training_ref import check, cross_entropy, router_loss

pytestmark = pytest.mark.gpu
DEV = "cuda"


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


@pytest.mark.parametrize("seed", range(24))
def test_cross_entropy(moe, seed):
    rng = random.Random(seed)
    T, H = log_uniform(rng, 1, 2500), 8 * log_uniform(rng, 1, 140)
    V = log_uniform(rng, 1, min(20000, 10_000_000 // T))
    dtype = rng.choice([m.MOE_BF16, m.MOE_F16])
    h, w, labels, dloss = ce.inputs(T, H, V, dtype, seed, rng.choice([0.5, 2.0, 6.0]))
    dlse = torch.randn(T, device=DEV) * float(dloss.max()) if rng.random() < 0.4 else None
    loss, lse, _ = ce.forward(h, w, labels, dtype)
    want = cross_entropy(h, w, labels, dloss, dlse)
    check(loss, want["loss"], want["loss_tol"], "loss")
    check(lse, want["lse"], want["lse_tol"], "lse")
    wide = rng.random() < 0.5
    start = torch.randn(V, H, device=DEV) if wide and rng.random() < 0.5 else None
    dh, dw = ce.backward(h, w, labels, dtype, lse, dloss, dlse, dw_dtype=m.MOE_F32 if wide else None, dw0=start)
    check(dh, want["dh"], want["dh_tol"], "dh")
    check(dw, want["dw"] if start is None else want["dw"] + start.double(), want["dw_tol"], "dw")


@pytest.mark.parametrize("seed", range(24))
def test_router_loss(moe, seed):
    rng = random.Random(100 + seed)
    E, T = log_uniform(rng, 1, 1024), log_uniform(rng, 1, 6000)
    k = rng.randint(1, min(E, 16))
    dtype = rng.choice(list(rl.TYPES))
    logits, ids, w, dw = rl.inputs(T, E, k, dtype, seed)
    keep = torch.rand(T, device=DEV) < rng.random() if rng.random() < 0.5 else None
    d = torch.tensor([rng.random(), rng.random()], device=DEV)
    rl.compare(rl.run(logits, ids, k, dtype, keep, d, w, dw), router_loss(logits, ids, k, keep, d, w, dw))


@pytest.mark.parametrize("seed", range(16))
def test_adamw(moe, seed):
    rng = random.Random(200 + seed)
    bits, (param, grad, master) = rng.choice([8, 32]), rng.choice(aw.KINDS)
    ds = [aw.tensor(log_uniform(rng, 1, 60000), 100 * seed + j, param, grad, master, bits, rng.choice([0, 0, 1, 8]),
                    weight_decay=rng.random(), lr_factor=2 * rng.random()) for j in range(rng.randint(1, 6))]
    h = dict(lr=10 ** rng.uniform(-5, -1), beta1=rng.choice([0.0, 0.9, 0.95]), beta2=rng.choice([0.0, 0.95, 0.999]),
             step=rng.randint(1, 5000))
    want = [aw.expected(d, **h) for d in ds]
    aw.step(ds, **h)
    for d, expect in zip(ds, want):
        aw.verify(d, expect)
