"""A training step around a block with frozen MXFP4 experts, driven through the C ABI.

    python -m bit_expert_ffn_gb300.mx4_train [tokens]

:class:`Mx4Training` puts a head (bf16 with an fp32 copy) behind an
:class:`~bit_expert_ffn_gb300.mx4_block.Mx4Block` and trains what is not
quantised: the head, the router, the norms' weights and the gate.  A step is

    block.forward -> router_loss -> cross_entropy -> cross_entropy_backward
      -> block.backward (norms, combine, router) -> adamw_step

All of it is enqueued on the current stream, with the learning rate and the
step's number on the device, so that a step can be captured and replayed.  The
router's weights get their gradient from the logits' by a product of the
caller's library (fp32).
"""
from __future__ import annotations

import sys

import torch

from . import (MOE_BF16, MOE_ERR_INVALID_ARG, RMS_EPS, MoeError, make_adamw_tensors, moe_adamw_options, moe_adamw_step,
               moe_check_status, moe_cross_entropy, moe_cross_entropy_backward, moe_cross_entropy_backward_workspace_size,
               moe_cross_entropy_workspace_size)
from .model import LayerShape, Workspace
from .mx4_block import Mx4Block, Mx4BlockBuffers, random_block


class Mx4Training:
    """block, and a head [V][H] in fp32, for T tokens a step; balance and square weigh the router's losses."""

    def __init__(self, block: Mx4Block, head: torch.Tensor, T: int, lr: float = 1e-3, weight_decay: float = 0.1,
                 balance: float = 0.01, square: float = 0.001, beta1: float = 0.9, beta2: float = 0.95):
        s, d, f32 = block.s, block.dev, torch.float32
        if head.dtype != f32 or head.dim() != 2 or head.shape[1] != s.H or T < 1:
            raise MoeError(MOE_ERR_INVALID_ARG, f"Mx4Training: head must be [V][{s.H}] in fp32 and T positive (got {tuple(head.shape)}, "
                                                f"{head.dtype}, T={T})")
        self.block, self.T, self.V = block, T, head.shape[0]
        self.bufs, self.ws = Mx4BlockBuffers(s, T, d), Workspace(d)
        self.head32 = head.contiguous().clone()
        self.head = self.head32.to(torch.bfloat16)
        self.y, self.u = torch.empty(T, s.H, dtype=f32, device=d), torch.empty(T, s.H, dtype=torch.bfloat16, device=d)
        self.du = torch.empty_like(self.u)
        self.loss, self.lse, self.dloss = (torch.empty(T, dtype=f32, device=d) for _ in range(3))
        self.router_dloss = torch.tensor([balance, square], dtype=f32, device=d)
        self.lr = torch.tensor([lr], dtype=f32, device=d)
        self.step_number = torch.zeros(1, dtype=torch.int64, device=d)
        self.grads = {"head": torch.empty_like(self.head), "router": torch.empty_like(block.router_w),
                      "w_post": torch.empty_like(block.w_post), "w_pre": torch.empty_like(block.w_pre),
                      "gate": torch.empty_like(block.gate)}
        n, blocks = self.head.numel(), (self.head.numel() + 255) // 256
        byte = lambda: torch.zeros(n, dtype=torch.uint8, device=d)  # noqa: E731
        self.states = {"head": dict(m=byte(), v=byte(), scales=torch.zeros(blocks, 2, dtype=f32, device=d), master=self.head32)}
        params = {"head": self.head, "router": block.router_w, "w_post": block.w_post, "w_pre": block.w_pre, "gate": block.gate}
        for name in ("router", "w_post", "w_pre", "gate"):
            self.states[name] = dict(m=torch.zeros_like(params[name]), v=torch.zeros_like(params[name]))
        decay = {"head": weight_decay, "router": weight_decay}
        self.tensors = make_adamw_tensors([dict(param=p, grad=self.grads[name], weight_decay=decay.get(name, 0.0), **self.states[name])
                                           for name, p in params.items()])
        self.options = moe_adamw_options(lr=lr, beta1=beta1, beta2=beta2, eps=1e-8, step=1, lr_dev=self.lr.data_ptr(),
                                         step_dev=self.step_number.data_ptr())

    def gradients(self, x, u, labels):
        """The losses and all gradients of a step on x [T][H] fp32, u [T][H] bf16 and labels [T] (int32, negative: none): per
        token self.loss, the router's self.bufs.loss, and self.grads; returns block.backward's dict."""
        b, T, H = self.block, self.T, self.block.s.H
        if labels.dtype != torch.int32 or labels.numel() != T or x.numel() != T * H:
            raise MoeError(MOE_ERR_INVALID_ARG, f"Mx4Training: a step takes {T} tokens and int32 labels (got {tuple(x.shape)}, "
                                                f"{tuple(labels.shape)}, {labels.dtype})")
        there = labels >= 0
        b.forward(x, u, T, self.y, self.u, self.bufs)
        b.router_loss(T, self.bufs, there)
        nf, nb = moe_cross_entropy_workspace_size(T, H, self.V), moe_cross_entropy_backward_workspace_size(T, H, self.V)
        ws = self.ws.get(max(nf, nb))
        moe_cross_entropy(self.u, MOE_BF16, T, H, self.head, self.V, labels, self.loss, self.lse, ws, nf, b.status)
        torch.div(there, there.sum().clamp_min(1), out=self.dloss)  # the mean over the tokens that have a label
        moe_cross_entropy_backward(self.u, MOE_BF16, T, H, self.head, self.V, labels, self.lse, self.dloss, None, self.du,
                                   self.grads["head"], MOE_BF16, False, ws, nb, b.status)
        into = {n: self.grads[n] for n in ("w_post", "w_pre", "gate")}
        g = b.backward(x, T, self.bufs, None, self.du, dloss=self.router_dloss, into=into)
        torch.mm(g["logits"].t(), u.view(T, H).float(), out=self.grads["router"].view(b.s.E, H))
        return g

    def step(self, x, u, labels):
        """One training step; returns the losses per token (0 where there is no label)."""
        self.gradients(x, u, labels)
        self.step_number += 1
        moe_adamw_step(self.tensors, self.options, self.block.status)
        return self.loss


def main(T: int, V: int = 8192) -> None:
    s = LayerShape()
    block = random_block(s)
    train = Mx4Training(block, torch.randn(V, s.H, device="cuda") * s.H ** -0.5, T)
    x = torch.randn(T, s.H, device="cuda")
    u = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + RMS_EPS)).bfloat16()
    labels = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    times = []
    for i in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        loss = train.step(x, u, labels)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
        if i in (0, 11):
            lb, sq = train.bufs.loss.tolist()
            print(f"step {i + 1}: cross entropy {float(loss.mean()):.4f}, balance {lb:.4f}, squared log-sum {sq:.4f}")
    assert moe_check_status(block.status) == 0
    ms = sorted(times[2:])[5]
    print(f"{T} tokens a step through a block of {s.E} frozen MXFP4 experts and a head of {V}: {ms * 1e3:.0f} us a step")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8192)
