"""What the row, 4-bit and norm calls refuse, before anything is launched (no GPU needed)."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B

A = 1 << 20  # an aligned address that no refused call may touch


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


def refused(status, word, fn, *args, **kw):
    with pytest.raises(m.MoeError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)
    assert word in str(e.value), str(e.value)


BAD = m.MOE_ERR_INVALID_ARG


def test_rows():
    refused(BAD, "k", m.moe_dispatch, A, m.MOE_F32, 1, 8, 17, 32, A, A, A)
    refused(BAD, "k", m.moe_dispatch, A, m.MOE_F32, 1, 8, 0, 32, A, A, A)
    refused(BAD, "H", m.moe_dispatch, A, m.MOE_F32, 1, 0, 2, 32, A, A, A)
    refused(BAD, "T", m.moe_dispatch, A, m.MOE_F32, -1, 8, 2, 32, A, A, A)
    refused(BAD, "dtype", m.moe_dispatch, A, 3, 1, 8, 2, 32, A, A, A)
    refused(BAD, "E", m.moe_dispatch, A, m.MOE_F32, 1, 8, 2, 1025, A, A, A)
    refused(BAD, "NULL", m.moe_dispatch, A, m.MOE_F32, 1, 8, 2, 32, A, None, A)
    refused(BAD, "aligned", m.moe_dispatch, A + 1, m.MOE_BF16, 1, 8, 2, 32, A, A, A)
    refused(BAD, "too large", m.moe_dispatch, A, m.MOE_F32, 2 ** 30, 8, 2, 32, A, A, A)
    refused(BAD, "aligned", m.moe_dispatch_backward, A + 2, m.MOE_F32, 1, 8, 2, A, A)
    refused(BAD, "out_dtype", m.moe_combine, A, m.MOE_BF16, 1, 8, 2, A, A, A, m.MOE_F16)
    refused(BAD, "out_dtype", m.moe_combine, A, m.MOE_F32, 1, 8, 2, A, A, A, m.MOE_BF16)
    refused(BAD, "NULL", m.moe_combine, A, m.MOE_F32, 1, 8, 2, None, A, A)
    refused(BAD, "NULL", m.moe_combine_backward, A, A, m.MOE_F32, 1, 8, 2, 4, A, A, A, None, A)
    assert m.moe_combine(A, m.MOE_F32, 0, 8, 2, A, A, A) is None
    with pytest.raises(m.MoeError, match="x_stride"):
        m._check(m.lib().moe_dispatch(A, m.MOE_F32, 7, 1, 8, 2, 32, A, A, A, None), "moe_dispatch")


def test_existing_calls_still_refuse_fp16():
    refused(BAD, "out_dtype", m.moe_shared_expert, A, A, A, 64, 64, A, 1, A, m.MOE_F16, 0, A, 1 << 20)


def test_mx4():
    assert m.moe_mx4_size(3, 32) == (48, 96)
    assert m.moe_mx4_size(1, 256) == (128, 32)
    assert m.moe_mx4_size(2, 288) == (288, 64)
    assert m.moe_mx4_size(1, 1056) == (528, 64)
    assert m.moe_mx4_size(0, 64) == (0, 0)
    refused(BAD, "cols", m.moe_mx4_size, 1, 33)
    refused(BAD, "cols", m.moe_mx4_size, 1, 0)
    refused(BAD, "too many", m.moe_mx4_size, 2 ** 50, 64)
    refused(BAD, "cols", m.moe_mx4_quantise, A, m.MOE_F32, 1, 48, A, A)
    refused(BAD, "dtype", m.moe_mx4_quantise, A, 7, 1, 64, A, A)
    refused(BAD, "16-byte", m.moe_mx4_quantise, A, m.MOE_F32, 1, 64, A + 8, A)
    refused(BAD, "aligned", m.moe_mx4_quantise, A + 2, m.MOE_F32, 1, 64, A, A)
    refused(BAD, "NULL", m.moe_mx4_quantise, None, m.MOE_F32, 1, 64, A, A)
    refused(BAD, "NULL", m.moe_mx4_dequantise, A, A, 1, 64, None)
    refused(BAD, "32-byte", m.moe_mx4_dequantise, A, A + 16, 1, 64, A)
    args = dict(out_dtype=m.MOE_F32)
    refused(BAD, "E", m.moe_mx4_matmul, A, A, 0, 8, 64, A, A, 1, A, A, **args)
    refused(BAD, "E", m.moe_mx4_matmul, A, A, 1025, 8, 64, A, A, 1, A, A, **args)
    refused(BAD, "N", m.moe_mx4_matmul, A, A, 1, 0, 64, A, A, 1, None, A, **args)
    refused(BAD, "K", m.moe_mx4_matmul, A, A, 1, 8, 40, A, A, 1, None, A, **args)
    refused(BAD, "rows", m.moe_mx4_matmul, A, A, 1, 8, 64, A, A, -1, None, A, **args)
    refused(BAD, "offsets", m.moe_mx4_matmul, A, A, 2, 8, 64, A, A, 1, None, A, **args)
    refused(BAD, "NULL", m.moe_mx4_matmul, A, A, 1, 8, 64, A, None, 1, None, A, **args)
    refused(BAD, "16-byte", m.moe_mx4_matmul, A, A, 1, 8, 64, A + 8, A, 1, None, A, **args)
    refused(BAD, "epilogue", m.moe_mx4_matmul, A, A, 1, 8, 64, A, A, 1, None, A, epilogue=2)
    refused(BAD, "out_dtype", m.moe_mx4_matmul, A, A, 1, 8, 64, A, A, 1, None, A, out_dtype=5)
    assert m.moe_mx4_matmul(A, A, 1, 8, 64, A, A, 0, None, A) is None


def norm(**kw):
    a = dict(x=A, res_dtype=m.MOE_F32, b=A, dtype=m.MOE_BF16, T=2, H=64, w_post=None, w_pre=None, gate=None,
             gate_kind=m.MOE_GATE_NONE, alpha=1.0, eps=1e-6)
    a.update(kw)
    return a


def test_block_norm():
    out = dict(y=A, u=A)
    refused(BAD, "residual", m.moe_block_norm, **norm(res_dtype=m.MOE_F16), **out)
    refused(BAD, "residual", m.moe_block_norm, **norm(dtype=4), **out)
    refused(m.MOE_ERR_UNSUPPORTED, "16384", m.moe_block_norm, **norm(H=16385), **out)
    refused(BAD, "H", m.moe_block_norm, **norm(H=0), **out)
    refused(BAD, "gate_kind", m.moe_block_norm, **norm(gate_kind=3), **out)
    refused(BAD, "gate", m.moe_block_norm, **norm(gate_kind=m.MOE_GATE_TOKEN), **out)
    refused(BAD, "gate", m.moe_block_norm, **norm(gate=A), **out)
    refused(BAD, "eps", m.moe_block_norm, **norm(eps=-1.0), **out)
    refused(BAD, "NULL", m.moe_block_norm, **norm(), y=None, u=A)
    refused(BAD, "aligned", m.moe_block_norm, **norm(x=A + 2), **out)
    back = dict(dy=A, du=A, dx=A, db=A)
    need = m.moe_block_norm_backward_workspace_size(2, 64)
    refused(m.MOE_ERR_WORKSPACE, str(need), m.moe_block_norm_backward, **norm(), **back, ws=A, ws_bytes=need - 1)
    refused(BAD, "dgate", m.moe_block_norm_backward, **norm(), **back, dgate=A, ws=A, ws_bytes=need)
    refused(BAD, "NULL", m.moe_block_norm_backward, **norm(), dy=A, du=A, dx=None, db=A, ws=A, ws_bytes=need)
    refused(BAD, "16-byte", m.moe_block_norm_backward, **norm(), **back, ws=A + 4, ws_bytes=need)
    refused(BAD, "gate_kind", m.moe_block_norm_backward_workspace_size, 2, 64, 9)


def test_tensors_that_are_too_small_or_not_packed():
    i32 = torch.int32
    x, off, inv, out = torch.zeros(4, 8), torch.zeros(5, dtype=i32), torch.zeros(8, dtype=i32), torch.zeros(8, 8)
    refused(BAD, "out", m.moe_dispatch, x, m.MOE_F32, 4, 8, 2, 4, off, inv, out[:7])
    refused(BAD, "out", m.moe_dispatch, x, m.MOE_F32, 4, 8, 2, 4, off, inv, torch.zeros(8, 16)[:, ::2])
    refused(BAD, "x ", m.moe_dispatch, x[:3], m.MOE_F32, 4, 8, 2, 4, off, inv, out)
    refused(BAD, "x ", m.moe_dispatch, x.t(), m.MOE_F32, 4, 8, 2, 4, off, inv, out)
    refused(BAD, "x ", m.moe_dispatch, x.half(), m.MOE_F32, 4, 8, 2, 4, off, inv, out)
    refused(BAD, "offsets", m.moe_dispatch, x, m.MOE_F32, 4, 8, 2, 4, off[:4], inv, out)
    refused(BAD, "inv_perm", m.moe_dispatch, x, m.MOE_F32, 4, 8, 2, 4, off, inv.long(), out)
    refused(BAD, "codes", m.moe_mx4_quantise, torch.zeros(2, 64), m.MOE_F32, 2, 64, torch.zeros(63, dtype=torch.uint8),
            torch.zeros(64, dtype=torch.uint8))
    refused(BAD, "w_post", m.moe_block_norm, **norm(w_post=torch.zeros(63)), y=A, u=A)
