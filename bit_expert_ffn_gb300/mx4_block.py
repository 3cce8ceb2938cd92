"""A MoE block with MXFP4 experts between its norms, driven through the C ABI.

    python -m bit_expert_ffn_gb300.mx4_block [tokens]

:class:`Mx4Block` keeps a layer's experts as e2m1 codes with e8m0 scales and
runs one block as the sequence of library calls

    router_topk -> permute -> mx4_quantise -> dispatch -> mx4_matmul (SwiGLU)
      -> mx4_quantise -> mx4_matmul -> combine -> block_norm

from the residual stream x (fp32) and its normalised input u (bf16) to the next
block's: y = x + alpha gate w_post rmsnorm(experts(u)), u' = w_pre rmsnorm(y).
:meth:`Mx4Block.backward` gives the gradients of what is trained around frozen
quantised experts: the norms' weights, the gate, the routing weights and the
router's logits (with the router's own losses, :meth:`Mx4Block.router_loss`),
and the residual stream's own.  Nothing here computes any part of the block
itself.
"""
from __future__ import annotations

import sys

import torch

from . import (MOE_BF16, MOE_ERR_INVALID_ARG, MOE_F32, MOE_GATE_CHANNEL, MOE_MX4_PLAIN, MOE_MX4_SWIGLU, RMS_EPS, MoeError,
               load, moe_block_norm, moe_block_norm_backward, moe_block_norm_backward_workspace_size, moe_check_status,
               moe_combine, moe_combine_backward, moe_dispatch, moe_dispatch_backward, moe_mx4_matmul, moe_mx4_quantise,
               moe_mx4_size, moe_permute, moe_permute_workspace_size, moe_router_loss, moe_router_loss_backward, moe_router_loss_workspace_size,
               moe_router_topk, moe_router_workspace_size)
from .model import LayerShape, Workspace


class Mx4Matrix:
    """[rows][cols] in MXFP4 on the device, quantised from fp32, bf16 or fp16 values."""

    def __init__(self, rows: int, cols: int, dev="cuda"):
        cb, sb = moe_mx4_size(1, cols)  # a row's bytes
        self.rows, self.cols = rows, cols
        self.codes = torch.empty(rows, cb, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(rows, sb, dtype=torch.uint8, device=dev)

    def put(self, values: torch.Tensor, dtype: int, status=None, rows=None) -> "Mx4Matrix":
        """Quantises values into the first `rows` rows (all of them by default)."""
        moe_mx4_quantise(values, dtype, self.rows if rows is None else rows, self.cols, self.codes, self.scales, status)
        return self


class Mx4BlockBuffers:
    """What a block's forward pass writes for up to T tokens, and its backward pass reads."""

    def __init__(self, s: LayerShape, T: int, dev="cuda"):
        d, P, n = torch.device(dev), T * s.k, max(T, 1)
        i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
        self.s, self.T = s, T
        self.logits = torch.empty(n, s.E, dtype=f32, device=d)
        self.ids = torch.empty(n, s.k, dtype=i32, device=d)
        self.w = torch.empty(n, s.k, dtype=f32, device=d)
        self.loss = torch.empty(2, dtype=f32, device=d)  # the router's losses: balance, squared log-sum
        self.counts = torch.empty(s.E + 1, dtype=i32, device=d)
        self.mean_prob = torch.empty(s.E, dtype=f32, device=d)
        self.lse = torch.empty(n, dtype=f32, device=d)
        self.offsets = torch.empty(s.E + 1, dtype=i32, device=d)
        self.perm = torch.empty(max(P, 1), dtype=i32, device=d)
        self.inv = torch.empty(max(P, 1), dtype=i32, device=d)
        self.u_q = Mx4Matrix(T, s.H, d)     # the tokens, quantised once
        self.rows_q = Mx4Matrix(P, s.H, d)  # ... at their pairs' places
        self.h = torch.empty(P, s.I, dtype=bf16, device=d)
        self.h_q = Mx4Matrix(P, s.I, d)
        self.rows = torch.empty(P, s.H, dtype=bf16, device=d)
        self.b = torch.empty(T, s.H, dtype=bf16, device=d)


class Mx4Block:
    """One block: s.E experts of s.I columns on s.H, the top s.k of a token; H and I multiples of 32."""

    def __init__(self, s: LayerShape, gate_up: torch.Tensor, down: torch.Tensor, router_w: torch.Tensor,
                 w_post: torch.Tensor, w_pre: torch.Tensor, gate: torch.Tensor, alpha: float = 1.0):
        """gate_up [E][2I][H] (gate rows first) and down [E][H][I] in bf16, quantised here; router_w [E][H], w_post, w_pre
        and gate [H] in fp32."""
        load()
        self._require(router_w.dtype == torch.float32 and router_w.is_contiguous() and router_w.numel() >= s.E * s.H,
                      f"router_w must be a packed fp32 tensor of {s.E} x {s.H} (got {tuple(router_w.shape)}, {router_w.dtype})")
        self.s, self.dev, self.alpha = s, gate_up.device, float(alpha)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.dev)
        self.gate_up = Mx4Matrix(s.E * 2 * s.I, s.H, self.dev).put(gate_up, MOE_BF16, self.status)
        self.down = Mx4Matrix(s.E * s.H, s.I, self.dev).put(down, MOE_BF16, self.status)
        self.router_w, self.w_post, self.w_pre, self.gate = router_w, w_post, w_pre, gate
        self.ws = Workspace(self.dev)

    @staticmethod
    def _require(ok: bool, what: str):
        if not ok:
            raise MoeError(MOE_ERR_INVALID_ARG, f"Mx4Block: {what}")

    def _check(self, T: int, bufs: Mx4BlockBuffers):
        """Before the first launch: some of the calls take addresses and could not tell that a buffer ends too early."""
        s, b = self.s, bufs.s
        self._require(0 <= T <= bufs.T, f"T={T}, but the buffers are for at most {bufs.T} tokens")
        self._require((s.H, s.I, s.E, s.k) == (b.H, b.I, b.E, b.k),
                      f"the buffers are for H={b.H} I={b.I} E={b.E} k={b.k}, the block has H={s.H} I={s.I} E={s.E} k={s.k}")

    def forward(self, x, u, T, y, u_next, bufs: Mx4BlockBuffers):
        """y, u_next <- the block on x [T][H] fp32 and u [T][H] bf16 (y may be x, u_next may be u); T at most the buffers'."""
        s, B = self.s, bufs
        self._check(T, B)
        self._require(u.dtype == torch.bfloat16 and u.is_contiguous() and u.numel() >= T * s.H,
                      f"u must be a packed bf16 tensor of at least {T} x {s.H} (got {tuple(u.shape)}, {u.dtype})")
        rws, pws = moe_router_workspace_size(T, s.H, s.E, True), moe_permute_workspace_size(T, s.k, s.E)
        ws = self.ws.get(max(rws, pws))
        moe_router_topk(u, T, s.H, self.router_w, None, s.E, s.k, B.logits, B.ids, B.w, ws, rws, self.status)
        moe_permute(B.ids, T, s.k, s.E, B.offsets, B.perm, B.inv, ws, pws, self.status)
        # a token's codes and scales are rows of bytes like any other: a tenth of the quantising, a quarter of the
        # bytes that its bf16 rows would be
        B.u_q.put(u, MOE_BF16, self.status, T)
        for a, b in ((B.u_q.codes, B.rows_q.codes), (B.u_q.scales, B.rows_q.scales)):
            moe_dispatch(a.view(torch.bfloat16), MOE_BF16, T, a.shape[1] // 2, s.k, s.E, B.offsets, B.inv,
                         b.view(torch.bfloat16))
        P = T * s.k
        moe_mx4_matmul(self.gate_up.codes, self.gate_up.scales, s.E, s.I, s.H, B.rows_q.codes, B.rows_q.scales, P, B.offsets,
                       B.h, MOE_BF16, MOE_MX4_SWIGLU, self.status)
        B.h_q.put(B.h, MOE_BF16, self.status, P)
        moe_mx4_matmul(self.down.codes, self.down.scales, s.E, s.H, s.I, B.h_q.codes, B.h_q.scales, P, B.offsets, B.rows,
                       MOE_BF16, MOE_MX4_PLAIN, self.status)
        moe_combine(B.rows, MOE_BF16, T, s.H, s.k, B.w, B.inv, B.b, MOE_BF16)
        moe_block_norm(x, MOE_F32, B.b, MOE_BF16, T, s.H, self.w_post, self.w_pre, self.gate, MOE_GATE_CHANNEL, self.alpha,
                       RMS_EPS, y, u_next)

    def router_loss(self, T, bufs: Mx4BlockBuffers, keep=None):
        """The router's losses of a forward pass that filled bufs, over its T tokens or those that keep [T] (bytes or truth
        values) marks: bufs.loss [2], counts [E + 1], mean_prob [E]; returns bufs.loss."""
        s, B = self.s, bufs
        self._check(T, B)
        nb = moe_router_loss_workspace_size(T, s.E)
        moe_router_loss(B.logits, MOE_F32, T, s.E, B.ids, s.k, keep, B.loss, B.counts, B.mean_prob, B.lse, self.ws.get(nb), nb,
                        self.status)
        return B.loss

    def backward(self, x, T, bufs: Mx4BlockBuffers, dy, du_next, drows=None, dloss=None, into=None):
        """Gradients of a forward pass on x (as it was) that filled bufs, for dy [T][H] fp32 and du_next [T][H] bf16 (either may
        be None): a dict of x, w_post, w_pre, gate, w (routing weights) and rows (the experts' outputs); with drows, the
        gradient of the dispatched rows as the caller's own experts give it, also u; with dloss [2], the gradient of what
        router_loss gave, also logits, from the losses and the routing weights.  into: tensors to write w_post, w_pre and
        gate to."""
        s, B, d = self.s, bufs, self.dev
        self._check(T, B)
        f32 = torch.float32
        g = {"x": torch.empty_like(x), "w_post": torch.empty(s.H, dtype=f32, device=d),
             "w_pre": torch.empty(s.H, dtype=f32, device=d), "gate": torch.empty(s.H, dtype=f32, device=d),
             "rows": torch.empty_like(B.rows[:T * s.k]), "w": torch.empty_like(B.w[:T])}
        g.update(into or {})
        db = torch.empty_like(B.b[:T])
        nb = moe_block_norm_backward_workspace_size(T, s.H, MOE_GATE_CHANNEL)
        moe_block_norm_backward(x, MOE_F32, B.b, MOE_BF16, T, s.H, self.w_post, self.w_pre, self.gate, MOE_GATE_CHANNEL,
                                self.alpha, RMS_EPS, dy, du_next, g["x"], db, g["w_post"], g["w_pre"], g["gate"],
                                self.ws.get(nb), nb)
        moe_combine_backward(db, B.rows, MOE_BF16, T, s.H, s.k, s.E, B.offsets, B.w, B.inv, g["rows"], g["w"])
        if drows is not None:
            g["u"] = torch.empty(T, s.H, dtype=torch.bfloat16, device=d)
            moe_dispatch_backward(drows, MOE_BF16, T, s.H, s.k, B.inv, g["u"])
        if dloss is not None:
            g["logits"] = torch.empty_like(B.logits[:T])
            moe_router_loss_backward(B.logits, MOE_F32, T, s.E, B.ids, s.k, B.counts, B.lse, dloss, B.w, g["w"], g["logits"])
        return g


def random_block(s: LayerShape, seed: int = 0, dev="cuda") -> Mx4Block:
    """A block of normal weights (sigma 1/sqrt(inputs)), norms and gate near one."""
    r = torch.Generator(device=dev)
    r.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=r, device=dev) * scale).to(dtype)

    gate_up = torch.empty(s.E, 2 * s.I, s.H, dtype=torch.bfloat16, device=dev)
    down = torch.empty(s.E, s.H, s.I, dtype=torch.bfloat16, device=dev)
    for e in range(s.E):
        gate_up[e] = normal(2 * s.I, s.H, scale=s.H ** -0.5)
        down[e] = normal(s.H, s.I, scale=s.I ** -0.5)
    return Mx4Block(s, gate_up, down, normal(s.E, s.H, scale=0.02), 1 + normal(s.H, scale=0.1), 1 + normal(s.H, scale=0.1),
                    torch.sigmoid(normal(s.H)), alpha=0.5)


def main(T: int) -> None:
    s = LayerShape()
    block = random_block(s)
    x = torch.randn(T, s.H, device="cuda")
    u, y, un = x.bfloat16(), torch.empty_like(x), torch.empty(T, s.H, dtype=torch.bfloat16, device="cuda")
    bufs = Mx4BlockBuffers(s, T)
    block.forward(x, u, T, y, un, bufs)
    assert moe_check_status(block.status) == 0
    times = []
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        block.forward(x, u, T, y, un, bufs)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    ms = sorted(times[2:])[5]
    print(f"{T} tokens through a block of {s.E} MXFP4 experts (H={s.H}, I={s.I}, top-{s.k}): {ms * 1e3:.0f} us, "
          f"{T / ms * 1e3:.0f} tokens/s")
    grads = block.backward(x, T, bufs, torch.randn_like(y), torch.randn_like(un))
    torch.cuda.synchronize()
    print("gradients:", ", ".join(f"{n} {tuple(t.shape)}" for n, t in grads.items()))


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8192)
