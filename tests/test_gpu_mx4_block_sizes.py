"""The block of MXFP4 experts with no tokens, and with fewer than its buffers hold: as with buffers of just that size."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300.model import LayerShape
from bit_expert_ffn_gb300.mx4_block import Mx4BlockBuffers, random_block

pytestmark = pytest.mark.gpu
DEV = "cuda"
S = LayerShape(H=256, I=96, E=12, k=3)


def tokens(T, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [torch.randn(T, S.H, generator=g, device=DEV).to(t) for t in (torch.float32, torch.bfloat16) * 2]


def test_no_tokens(moe):
    blk = random_block(S, seed=1)
    x, u, dy, du = tokens(0, 0)
    for bufs in (Mx4BlockBuffers(S, 0), Mx4BlockBuffers(S, 4)):
        blk.forward(x, u, 0, torch.empty_like(x), torch.empty_like(u), bufs)
        g = blk.backward(x, 0, bufs, dy, du, torch.empty(0, S.H, dtype=torch.bfloat16, device=DEV))
        assert m.moe_check_status(blk.status) == m.MOE_OK
        for n in ("w_post", "w_pre", "gate"):
            assert torch.equal(g[n], torch.zeros(S.H, device=DEV))
        assert g["x"].shape == (0, S.H) and g["rows"].shape == (0, S.H) and g["w"].shape == (0, S.k)


@pytest.mark.parametrize("T", [1, 5, 31])
def test_fewer_tokens_than_the_buffers_hold(moe, T):
    blk = random_block(S, seed=2)
    x, u, dy, du = tokens(T, T)
    dr = torch.randn(T * S.k, S.H, device=DEV).bfloat16()
    got = []
    for bufs in (Mx4BlockBuffers(S, T), Mx4BlockBuffers(S, 32)):
        bufs.h.fill_(float("nan"))  # what a pass does not write, it does not read
        bufs.rows.fill_(float("nan"))
        y, un = torch.empty_like(x), torch.empty_like(u)
        blk.forward(x, u, T, y, un, bufs)
        g = blk.backward(x, T, bufs, dy, du, dr)
        assert m.moe_check_status(blk.status) == m.MOE_OK
        got.append({"y": y, "u_next": un, **{"d" + n: t for n, t in g.items()}})
    for n in got[0]:
        assert torch.equal(got[0][n], got[1][n]), n
