"""Cross entropy of more tokens than the tiles' order takes in one band of rows (4,096)."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_cross_entropy import backward, forward, inputs
from training_ref import check, cross_entropy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,V", [(5000, 64, 700), (4097, 72, 300), (8200, 264, 1030), (13000, 8, 2049)])
def test_more_than_a_band(moe, T, H, V):
    h, w, labels, dloss = inputs(T, H, V, m.MOE_BF16, T)
    loss, lse, st = forward(h, w, labels, m.MOE_BF16)
    want = cross_entropy(h, w, labels, dloss)
    assert st == 0
    check(loss, want["loss"], want["loss_tol"], "loss")
    check(lse, want["lse"], want["lse_tol"], "lse")
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    check(dh, want["dh"], want["dh_tol"], "dh")
    check(dw, want["dw"], want["dw_tol"], "dw")
    # (the fp32 form's sums are the same ones, rounded)
    _, dw32 = backward(h, w, labels, m.MOE_BF16, lse, dloss, want=(False, True), dw_dtype=m.MOE_F32)
    check(dw32, want["dw"], want["dw_tol"], "dw fp32")
    assert torch.equal(dw32.bfloat16(), dw)
