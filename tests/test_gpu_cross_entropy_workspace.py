"""One workspace, of the largest batch's size, for every smaller one."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from test_gpu_cross_entropy import DEV, backward, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,V", [(2048, 32000), (64, 9001), (72, 70001)])
def test_smaller_batches(moe, H, V):
    top = 500
    h, w, labels, dloss = inputs(top, H, V, m.MOE_BF16, 21)
    nf, nb = m.moe_cross_entropy_workspace_size(top, H, V), m.moe_cross_entropy_backward_workspace_size(top, H, V)
    wf, wb = (torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV) for n in (nf, nb))
    for T in (500, 386, 379, 129, 22, 15, 1):
        want = forward(h[:T], w, labels[:T], m.MOE_BF16)
        grads = backward(h[:T], w, labels[:T], m.MOE_BF16, want[1], dloss[:T])
        loss, lse, dh, dw = torch.empty(T, device=DEV), torch.empty(T, device=DEV), torch.empty_like(h[:T]), torch.empty_like(w)
        m.moe_cross_entropy(h[:T], m.MOE_BF16, T, H, w, V, labels[:T], loss, lse, wf[:nf], nf)
        m.moe_cross_entropy_backward(h[:T], m.MOE_BF16, T, H, w, V, labels[:T], lse, dloss[:T], None, dh, dw, m.MOE_BF16, False, wb[:nb], nb)
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(dh, grads[0]) and torch.equal(dw, grads[1])
        assert (wf[nf:] == 0xFF).all() and (wb[nb:] == 0xFF).all()
