"""Tensors of another type than the call says, or on the host, are refused before anything is launched (no GPU needed)."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B

f32, bf16, f16, i16, i32, i64, u8 = (torch.float32, torch.bfloat16, torch.float16, torch.int16, torch.int32, torch.int64,
                                     torch.uint8)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


def z(*shape, t=bf16):
    return torch.zeros(*shape, dtype=t)


def operands(t=bf16):
    """T = 4 tokens, H = 64 columns, k = 2 pairs each, E = 3 groups."""
    return {
        "dispatch": (m.moe_dispatch, dict(x=z(4, 64, t=t), dtype=m.MOE_BF16, T=4, H=64, k=2, E=3, offsets=z(4, t=i32),
                                          inv_perm=z(8, t=i32), out=z(8, 64, t=t))),
        "dispatch_backward": (m.moe_dispatch_backward, dict(drows=z(8, 64, t=t), dtype=m.MOE_BF16, T=4, H=64, k=2,
                                                            inv_perm=z(8, t=i32), dx=z(4, 64, t=t))),
        "combine": (m.moe_combine, dict(y=z(8, 64, t=t), dtype=m.MOE_BF16, T=4, H=64, k=2, w=z(4, 2, t=f32),
                                        inv_perm=z(8, t=i32), out=z(4, 64, t=f32))),
        "combine_backward": (m.moe_combine_backward, dict(dout=z(4, 64, t=t), y=z(8, 64, t=t), dtype=m.MOE_BF16, T=4, H=64, k=2,
                                                          E=3, offsets=z(4, t=i32), w=z(4, 2, t=f32), inv_perm=z(8, t=i32),
                                                          dy=z(8, 64, t=t), dw=z(4, 2, t=f32))),
        "quantise": (m.moe_mx4_quantise, dict(x=z(4, 64, t=t), dtype=m.MOE_BF16, rows=4, cols=64, codes=z(4, 32, t=u8),
                                              scales=z(4, 32, t=u8), dev_status=z(1, t=i32))),
        "dequantise": (m.moe_mx4_dequantise, dict(codes=z(4, 32, t=u8), scales=z(4, 32, t=u8), rows=4, cols=64, out=z(4, 64, t=t))),
        "matmul": (m.moe_mx4_matmul, dict(w_codes=z(24, 32, t=u8), w_scales=z(24, 32, t=u8), E=3, N=8, K=64, x_codes=z(4, 32, t=u8),
                                          x_scales=z(4, 32, t=u8), rows=4, offsets=z(4, t=i32), out=z(4, 8, t=t),
                                          out_dtype=m.MOE_BF16, dev_status=z(1, t=i32))),
        "block_norm": (m.moe_block_norm, dict(x=z(4, 64, t=f32), res_dtype=m.MOE_F32, b=z(4, 64, t=t), dtype=m.MOE_BF16, T=4, H=64,
                                              w_post=z(64, t=f32), w_pre=z(64, t=f32), gate=z(4, t=f32),
                                              gate_kind=m.MOE_GATE_TOKEN, alpha=1.0, eps=1e-6, y=z(4, 64, t=f32), u=z(4, 64, t=t))),
        "block_norm_backward": (m.moe_block_norm_backward, dict(
            x=z(4, 64, t=f32), res_dtype=m.MOE_F32, b=z(4, 64, t=t), dtype=m.MOE_BF16, T=4, H=64, w_post=z(64, t=f32),
            w_pre=z(64, t=f32), gate=z(64, t=f32), gate_kind=m.MOE_GATE_CHANNEL, alpha=1.0, eps=1e-6, dy=z(4, 64, t=f32),
            du=z(4, 64, t=t), dx=z(4, 64, t=f32), db=z(4, 64, t=t), dw_post=z(64, t=f32), dw_pre=z(64, t=f32),
            dgate=z(64, t=f32), ws=z(1 << 16, t=u8), ws_bytes=1 << 16)),
    }


def refused(fn, args, *words):
    with pytest.raises(m.MoeError) as e:
        fn(**args)
    assert e.value.status == m.MOE_ERR_INVALID_ARG and all(w in str(e.value) for w in words), str(e.value)


SAME_SIZE = {bf16: f16, f32: i32, i32: f32, u8: torch.bool}  # another type of the same bytes
TENSORS = [(c, n) for c, (_, a) in operands().items() for n, t in a.items() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("call,name", TENSORS)
def test_another_type_of_the_same_size(call, name):
    fn, args = operands()[call]
    if name != "ws":  # (bytes of any type)
        args[name] = args[name].to(SAME_SIZE[args[name].dtype])
        refused(fn, args, f"{name} must", str(args[name].dtype))


@pytest.mark.parametrize("call,name", TENSORS)
def test_a_tensor_on_the_host(call, name):
    """Everything else is an address that no call may come as far as using."""
    fn, args = operands()[call]
    host = args[name]
    args = {n: 1 << 20 if isinstance(t, torch.Tensor) else t for n, t in args.items()}
    args[name] = host
    refused(fn, args, f"{name} must be on the GPU")


def test_rows_at_a_stride_on_the_host():
    fn, args = operands()["dispatch"]
    args["x"] = z(4, 80)[:, :64]
    refused(fn, args, "must be on the GPU")


@pytest.mark.parametrize("call", operands())
def test_bit_patterns_are_the_right_type(call):
    """16-bit values as int16 or uint16: no complaint but that they are the host's."""
    for t in (i16, torch.uint16):
        fn, args = operands(t)[call]
        refused(fn, args, "must be on the GPU")


def test_workspace_smaller_than_it_is_said_to_be():
    fn, args = operands()["block_norm_backward"]
    args["ws"] = args["ws"][:-1]
    refused(fn, args, "ws must", "65536")
