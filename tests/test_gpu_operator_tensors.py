"""Operands of the row, 4-bit and norm calls in the other types that hold them: bit patterns of 16-bit values, bytes."""
import pytest
import torch

import bit_expert_ffn_gb300 as m

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [torch.int16, torch.uint16])
@pytest.mark.parametrize("t,dtype", [(torch.bfloat16, m.MOE_BF16), (torch.float16, m.MOE_F16)])
def test_bit_patterns(moe, t, dtype, bits):
    x = torch.randn(6, 64, device=DEV).to(t)
    inv = torch.randperm(12, device=DEV).int()
    off = torch.tensor([0, 5, 12], dtype=torch.int32, device=DEV)
    a, b = torch.empty(12, 64, dtype=t, device=DEV), torch.empty(12, 64, dtype=bits, device=DEV)
    m.moe_dispatch(x, dtype, 6, 64, 2, 2, off, inv, a)
    m.moe_dispatch(x.view(bits), dtype, 6, 64, 2, 2, off, inv, b)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_bytes(moe):
    x = torch.randn(6, 64, device=DEV)
    cb, sb = m.moe_mx4_size(6, 64)
    got = []
    for t in [torch.uint8, torch.int8] + [getattr(torch, n) for n in ("float8_e8m0fnu",) if hasattr(torch, n)]:
        codes, scales = torch.zeros(cb, dtype=torch.uint8, device=DEV), torch.zeros(sb, dtype=torch.uint8, device=DEV).view(t)
        m.moe_mx4_quantise(x, m.MOE_F32, 6, 64, codes, scales)
        out = torch.empty(6, 64, device=DEV)
        m.moe_mx4_dequantise(codes, scales, 6, 64, out, m.MOE_F32)
        got.append(out)
    assert all(torch.equal(got[0], o) for o in got[1:]) and bool(((got[0] - x).abs() <= 0.26 * x.abs().max()).all())
