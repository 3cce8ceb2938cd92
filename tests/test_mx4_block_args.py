"""What the block of MXFP4 experts refuses before its first launch (no GPU needed: the tensors are the host's, and no
call of the block may come as far as looking at them)."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B
from bit_expert_ffn_gb300.model import LayerShape, Workspace
from bit_expert_ffn_gb300.mx4_block import Mx4Block, Mx4BlockBuffers, Mx4Matrix

S = LayerShape(H=64, I=32, E=4, k=2)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


def block(s=S):
    """A block as its constructor leaves it, but for the quantising."""
    b = object.__new__(Mx4Block)
    b.s, b.dev, b.alpha, b.status = s, torch.device("cpu"), 1.0, torch.zeros(1, dtype=torch.int32)
    b.gate_up, b.down = Mx4Matrix(s.E * 2 * s.I, s.H, "cpu"), Mx4Matrix(s.E * s.H, s.I, "cpu")
    b.router_w, b.w_post, b.w_pre, b.gate = torch.zeros(s.E, s.H), torch.ones(s.H), torch.ones(s.H), torch.ones(s.H)
    b.ws = Workspace(b.dev)
    return b


def tokens(T):
    return torch.zeros(T, S.H), torch.zeros(T, S.H, dtype=torch.bfloat16)


def refused(word, fn, *args):
    with pytest.raises(m.MoeError) as e:
        fn(*args)
    assert e.value.status == m.MOE_ERR_INVALID_ARG and word in str(e.value), str(e.value)


def test_more_tokens_than_the_buffers_hold():
    x, u = tokens(5)
    bufs = Mx4BlockBuffers(S, 4, "cpu")
    refused("at most 4", block().forward, x, u, 5, x, u, bufs)
    refused("at most 4", block().backward, x, 5, bufs, x, u)
    refused("at most 4", block().forward, x, u, -1, x, u, bufs)


def test_buffers_of_another_layer():
    x, u = tokens(3)
    for other in (LayerShape(H=64, I=32, E=3, k=2), LayerShape(H=64, I=32, E=4, k=1), LayerShape(H=32, I=32, E=4, k=2),
                  LayerShape(H=64, I=64, E=4, k=2)):
        refused("the block has", block().forward, x, u, 3, x, u, Mx4BlockBuffers(other, 3, "cpu"))


def test_too_few_rows_for_the_router():
    x, u = tokens(4)
    bufs = Mx4BlockBuffers(S, 4, "cpu")
    refused("u must", block().forward, x, u[:3], 4, x, u, bufs)
    refused("u must", block().forward, x, u.float(), 4, x, u, bufs)
    refused("u must", block().forward, x, u.t(), 4, x, u, bufs)
    refused("router_w", Mx4Block, S, u, u, torch.zeros(3, 64), x[0], x[0], x[0])
    refused("router_w", Mx4Block, S, u, u, torch.zeros(4, 64).double(), x[0], x[0], x[0])


def test_a_matrix_of_no_rows_keeps_its_width():
    q = Mx4Matrix(0, 1056, "cpu")
    assert q.codes.shape == (0, 528) and q.scales.shape == (0, 64)
    assert q.codes.view(torch.bfloat16).shape == (0, 264)
