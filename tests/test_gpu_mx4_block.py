"""A block with MXFP4 experts, stage by stage: what each call made of what the one before it wrote, against the plain
64-bit forms."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R
from bit_expert_ffn_gb300.model import LayerShape
from bit_expert_ffn_gb300.mx4_block import Mx4BlockBuffers, random_block

pytestmark = pytest.mark.gpu
DEV = "cuda"


def stored(q):
    """The values a Mx4Matrix holds."""
    c = q.codes.cpu().numpy().reshape(q.rows, -1)
    code = np.empty((q.rows, q.cols), np.uint8)
    code[:, 0::2], code[:, 1::2] = c & 15, c >> 4
    return R.values(code, q.scales.cpu().numpy().reshape(q.rows, -1)[:, :q.cols // 32])


def same(q, x):
    wc, ws = R.pack(*R.quantise(x))
    assert np.array_equal(q.codes.cpu().numpy().reshape(wc.shape), wc)
    assert np.array_equal(q.scales.cpu().numpy().reshape(ws.shape), ws)


@pytest.mark.parametrize("T", [1, 4, 37, 300])
@pytest.mark.parametrize("H,I,E,k", [(256, 96, 12, 3), (512, 160, 40, 8)])
def test_block(moe, T, H, I, E, k):
    s = LayerShape(H=H, I=I, E=E, k=k)
    blk = random_block(s, seed=T + H)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x = torch.randn(T, H, generator=g, device=DEV)
    u = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    y, un, B = torch.empty_like(x), torch.empty_like(u), Mx4BlockBuffers(s, T)
    blk.forward(x, u, T, y, un, B)
    assert m.moe_check_status(blk.status) == m.MOE_OK

    ids = B.ids.cpu().numpy()
    offsets, perm, inv = R.sorted_pairs(ids, E)
    for got, want in ((B.offsets, offsets), (B.perm, perm), (B.inv, inv)):
        assert np.array_equal(got.cpu().numpy()[:want.size], want)
    same(B.u_q, R.f64(u))
    rows = stored(B.rows_q)
    assert np.array_equal(rows, stored(B.u_q)[perm // k])
    wgu, wd = stored(blk.gate_up).reshape(E, 2 * I, H), stored(blk.down).reshape(E, H, I)
    h, slack = R.matmul(rows, wgu, offsets, True)
    R.within(B.h, h, slack, torch.bfloat16)
    same(B.h_q, R.f64(B.h))
    o, slack = R.matmul(stored(B.h_q), wd, offsets, False)
    R.within(B.rows, o, slack, torch.bfloat16)
    w, ov = R.f64(B.w), R.f64(B.rows)
    terms = w.reshape(-1)[:, None] * ov[inv]
    R.within(B.b, terms.reshape(T, k, H).sum(1), (k + 1) * R.U32 * np.abs(terms).reshape(T, k, H).sum(1), torch.bfloat16)
    xv, bv, wp, wn, gt = R.f64(x), R.f64(B.b), R.f64(blk.w_post), R.f64(blk.w_pre), R.f64(blk.gate)
    v, wy, wu, r1, r2 = R.block_norm(xv, bv, wp, wn, gt, blk.alpha, m.RMS_EPS)
    c = 80 * R.U32
    dy = c * np.abs(blk.alpha * gt * v) + R.U32 * np.abs(xv)
    R.within(y, wy, dy, torch.float32)
    dr = c + (np.abs(wy) * dy).mean(1, keepdims=True) * r2 ** 2
    R.within(un, wu, np.abs(wu) * dr + r2 * np.abs(wn) * dy, torch.bfloat16)

    gy, gu = torch.randn(T, H, generator=g, device=DEV), torch.randn(T, H, generator=g, device=DEV).bfloat16()
    dr_in = torch.randn(T * k, H, generator=g, device=DEV).bfloat16()
    got = blk.backward(x, T, B, gy, gu, dr_in)
    want, mag = R.block_norm_backward(xv, bv, wp, wn, gt, blk.alpha, m.RMS_EPS, R.f64(gy), R.f64(gu))
    R.within(got["x"], want[0], 6 * c * mag[0], torch.float32)
    for n, i in (("w_post", 2), ("w_pre", 3), ("gate", 4)):
        R.within(got[n], want[i].sum(0), (6 * c + (T + 60) * R.U32) * mag[i].sum(0), torch.float32)
    # the gradient of b is rounded to bf16 before it goes on
    half = 2.0 ** -8
    db, ddb = want[1], 6 * c * mag[1] + half * np.abs(want[1])
    R.within(got["rows"], w.reshape(-1)[perm, None] * db[perm // k], w.reshape(-1)[perm, None] * 1.01 * ddb[perm // k],
             torch.bfloat16)
    dots = (db[:, None] * ov[inv].reshape(T, k, H)).sum(2)
    R.within(got["w"], dots, (1.01 * ddb[:, None] * np.abs(ov[inv].reshape(T, k, H))).sum(2)
             + (H / 32 + 14) * R.U32 * (np.abs(db[:, None] * ov[inv].reshape(T, k, H))).sum(2), torch.float32)
    d = R.f64(dr_in)[inv].reshape(T, k, H)
    R.within(got["u"], d.sum(1), k * R.U32 * np.abs(d).sum(1), torch.bfloat16)


def test_block_in_place_and_from_a_graph(moe):
    s = LayerShape(H=256, I=128, E=16, k=4)
    blk = random_block(s, seed=3)
    T = 20
    x = torch.randn(T, 256, device=DEV)
    u = torch.randn(T, 256, device=DEV).bfloat16()
    B = Mx4BlockBuffers(s, T)
    y, un = torch.empty_like(x), torch.empty_like(u)
    blk.forward(x, u, T, y, un, B)
    y2, un2 = x.clone(), u.clone()
    blk.forward(y2, un2, T, y2, un2, B)
    assert torch.equal(y, y2) and torch.equal(un, un2)
    y3, un3 = x.clone(), u.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.forward(y3, un3, T, y3, un3, B)
    y3.copy_(x), un3.copy_(u)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y3) and torch.equal(un, un3)
