"""Gradients of the block norms for rows far from one in size, against the plain 64-bit form: the cube of a row's
reciprocal root leaves the range of 32 bits long before the row's squares do."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R
from test_gpu_block_norm import C, DEV, GATES, TYPES, dev, wide_gate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("size_x,size_b,alpha,eps", [
    (1.0, 1.0, 0.75, 1e-6), (1e15, 1e15, 0.75, 1e-6), (1e15, 1e15, 1e15, 1e-6), (1.0, 1e15, 0.75, 1e-6), (3e14, 1.0, 1e14, 1e-6),
    (1e-13, 1e-13, 1e-13, 0.0), (1.0, 1e-13, 0.75, 0.0), (1e-13, 1.0, 1e-13, 0.0),
])
@pytest.mark.parametrize("act", [torch.float32, torch.bfloat16], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,H", [(5, 64), (3, 33), (4, 500), (3, 2048), (2, 6001), (2, 16384)])
def test_gradients(moe, T, H, act, size_x, size_b, alpha, eps, gate):
    rng = np.random.default_rng(T * H)
    b = rng.standard_normal((T, H))
    s = {"x": dev((size_x * rng.standard_normal((T, H))).astype(np.float32)), "b": dev((size_b * b).astype(np.float32)).to(act),
         "w_post": dev((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)),
         "w_pre": dev((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)),
         # in step with the rows, so that the mean terms carry weight
         "du": dev((b + 0.3 * rng.standard_normal((T, H))).astype(np.float32)).to(act)}
    n = {"none": 0, "token": T, "channel": H}[gate]
    s["gate"] = dev(rng.uniform(0.5, 1.5, n).astype(np.float32)) if n else None
    nb = m.moe_block_norm_backward_workspace_size(T, H, GATES[gate])
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    dx, db = torch.empty(T, H, device=DEV), torch.empty(T, H, dtype=act, device=DEV)
    dwp, dwn = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    dg = None if s["gate"] is None else torch.empty_like(s["gate"])
    m.moe_block_norm_backward(s["x"], m.MOE_F32, s["b"], TYPES[act], T, H, s["w_post"], s["w_pre"], s["gate"], GATES[gate],
                              alpha, eps, None, s["du"], dx, db, dwp, dwn, dg, ws, nb)
    x, b, wp, wn, du = (R.f64(s[n]) for n in ("x", "b", "w_post", "w_pre", "du"))
    a32 = float(np.float32(alpha))
    got, mag = R.block_norm_backward(x, b, wp, wn, wide_gate(s, gate), a32, float(np.float32(eps)), np.zeros((T, H)), du)
    c = 6 * C  # three means, each of quantities that carry the ones before
    R.within(dx, got[0], c * mag[0], torch.float32)
    R.within(db, got[1], c * mag[1], act)
    cs = c + T * R.U32
    R.within(dwp, got[2].sum(0), cs * mag[2].sum(0), torch.float32)
    R.within(dwn, got[3].sum(0), cs * mag[3].sum(0), torch.float32)
    if dg is not None:
        ax = 1 if gate == "token" else 0
        R.within(dg, got[4].sum(ax), (cs + 60 * R.U32) * mag[4].sum(ax), torch.float32)
