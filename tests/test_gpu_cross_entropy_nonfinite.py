"""Cross entropy of hidden states and weights that are not finite: where they show."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_cross_entropy import DEV, backward, forward, inputs
from training_ref import check, cross_entropy

pytestmark = pytest.mark.gpu
T, H, V = 140, 64, 500
NAN, INF = float("nan"), float("inf")


def setup(dtype, seed=31):
    h, w, labels, dloss = inputs(T, H, V, dtype, seed)
    h[:, 3] = h[:, 3].abs() + 0.25  # the sign of an infinity there is w's
    labels[labels == 5] = 6
    return h, w, labels, dloss


def without(w, labels, row):
    """The vocabulary without a row, and the labels in it."""
    return torch.cat([w[:row], w[row + 1:]]), torch.where(labels > row, labels - 1, labels)


@pytest.mark.parametrize("dtype", [m.MOE_BF16, m.MOE_F16])
def test_a_logit_of_minus_infinity_is_a_probability_of_zero(moe, dtype):
    h, w, labels, dloss = setup(dtype)
    less, place = without(w, labels, 5)
    want = cross_entropy(h, less, place, dloss)
    w[5, 3] = -INF
    loss, lse, st = forward(h, w, labels, dtype)
    assert st == 0
    check(loss, want["loss"], want["loss_tol"], "loss")
    check(lse, want["lse"], want["lse_tol"], "lse")
    dh, dw = backward(h, w, labels, dtype, lse, dloss)
    rest = [i for i in range(H) if i != 3]
    assert torch.isnan(dh[:, 3]).all()  # zero times infinity, of every token
    check(dh[:, rest], want["dh"][:, rest], want["dh_tol"][:, rest], "dh")
    assert (dw[5] == 0).all()
    check(torch.cat([dw[:5], dw[6:]]), want["dw"], want["dw_tol"], "dw")
    labels[9] = 5  # a label that cannot be
    loss, lse, _ = forward(h, w, labels, dtype)
    assert loss[9] == INF and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [m.MOE_BF16, m.MOE_F16])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_other_logits_that_are_not_finite(moe, bad, dtype):
    h, w, labels, dloss = setup(dtype)
    labels[2], dloss[4] = -1, 0.0
    w[5, 3] = bad
    loss, lse, _ = forward(h, w, labels, dtype)
    there = labels >= 0
    assert torch.isnan(loss[there]).all() and (loss[~there] == 0).all() and torch.isnan(lse).all()
    dh, dw = backward(h, w, labels, dtype, lse, dloss)
    took = there & (dloss != 0)
    assert torch.isnan(dh[took]).all() and torch.isnan(dw).all()
    rest = [i for i in range(H) if i != 3]
    assert (dh[~took][:, rest] == 0).all() and torch.isnan(dh[~took][:, 3]).all()


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_a_hidden_value_that_is_not_finite(moe, bad):
    h, w, labels, dloss = setup(m.MOE_BF16)
    labels[7] = 11
    h[7, 20] = bad
    dloss[7] = 0  # its token takes no part
    loss, lse, _ = forward(h, w, labels, m.MOE_BF16)
    others = torch.arange(T, device=DEV) != 7
    assert torch.isnan(loss[7]) and torch.isfinite(loss[others]).all()
    want = cross_entropy(h[others], w, labels[others], dloss[others])
    check(loss[others], want["loss"], want["loss_tol"], "loss")
    dh, dw = backward(h, w, labels, m.MOE_BF16, lse, dloss)
    assert (dh[7] == 0).all()
    check(dh[others], want["dh"], want["dh_tol"], "dh")
    rest = [i for i in range(H) if i != 20]
    assert torch.isnan(dw[:, 20]).all()  # zero times it
    check(dw[:, rest], want["dw"][:, rest], want["dw_tol"][:, rest], "dw")
