"""Router losses of fewer experts than the cluster has CTAs: some of them have no columns to sum."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_router_loss import DEV, DLOSS, compare, inputs, run
from training_ref import router_loss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [m.MOE_F32, m.MOE_BF16])
@pytest.mark.parametrize("T", [13, 32, 60, 212, 384, 385])
@pytest.mark.parametrize("E", [1, 2, 3, 4, 5, 7, 8])
def test_fewer_experts_than_ctas(moe, E, T, dtype):
    k = min(E, 2)
    logits, ids, w, dw = inputs(T, E, k, dtype, 17 * E + T)
    d = torch.tensor(DLOSS, device=DEV)
    got = run(logits, ids, k, dtype, None, d, w, dw)
    assert got["status"] == 0
    compare(got, router_loss(logits, ids, k, None, d, w, dw))
