"""The training step around a block with MXFP4 experts: its calls together, its gradients, its update, and as a graph."""
import pytest
import torch

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300.model import LayerShape
from bit_expert_ffn_gb300.mx4_block import random_block
from bit_expert_ffn_gb300.mx4_train import Mx4Training
from test_gpu_adamw import expected, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(T, V, seed=0, s=LayerShape(H=256, I=128, E=24, k=4)):
    g = torch.Generator(device=DEV).manual_seed(seed)
    head = torch.randn(V, s.H, generator=g, device=DEV) * s.H ** -0.5
    train = Mx4Training(random_block(s, seed), head, T)
    x = torch.randn(T, s.H, generator=g, device=DEV)
    u = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + m.RMS_EPS)).bfloat16()
    labels = torch.randint(-1, V, (T,), generator=g, device=DEV).int()
    return train, x, u, labels


@pytest.mark.parametrize("T,V", [(1, 50), (37, 333), (700, 1000)])
def test_gradients(moe, T, V):
    train, x, u, labels = make(T, V, T)
    labels[0] = 3
    b, B, s = train.block, train.bufs, train.block.s
    g = train.gradients(x, u, labels)
    assert m.moe_check_status(b.status) == 0
    # the same function in 64 bits, from the experts' rows and the logits as they came
    leaf = {n: t.double().detach().requires_grad_() for n, t in (("logits", B.logits[:T]), ("w_post", b.w_post), ("w_pre", b.w_pre),
                                                                 ("gate", b.gate), ("head", train.head), ("x", x))}
    ids, there = B.ids[:T].long(), labels >= 0
    w = torch.softmax(leaf["logits"].gather(1, ids), 1)
    rows = B.rows[B.inv[:T * s.k].long()].double().view(T, s.k, s.H)
    rms = lambda t: t * torch.rsqrt(t.square().mean(1, keepdim=True) + m.RMS_EPS)  # noqa: E731
    out = (w[:, :, None] * rows).sum(1)
    y = leaf["x"] + b.alpha * leaf["gate"] * leaf["w_post"] * rms(out)
    hidden = leaf["w_pre"] * rms(y)
    ce = torch.nn.functional.cross_entropy(hidden @ leaf["head"].t(), labels.long().clamp_min(0), reduction="none")[there]
    p, lse = torch.softmax(leaf["logits"], 1)[there], torch.logsumexp(leaf["logits"], 1)[there]
    f = torch.bincount(ids[there].reshape(-1), minlength=s.E).double() / ids[there].numel()
    c = train.router_dloss.double()
    total = ce.mean() + c[0] * s.E * (f * p.mean(0)).sum() + c[1] * lse.square().mean()
    want = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    got = {"logits": g["logits"], "x": g["x"], "head": train.grads["head"], **{n: train.grads[n] for n in ("w_post", "w_pre", "gate")}}
    # four values on the way are rounded to bf16 (the experts' sum, the hidden states, their gradient and the sum's), and the
    # logits' gradient in the products; each by at most 2^-8 of itself
    for n, t in got.items():
        err = float((t.double() - want[n]).norm() / want[n].norm())
        assert err <= 5 * 2.0 ** -8, (n, err)
    router = want["logits"].t() @ u.double()
    assert float((train.grads["router"].double() - router).norm() / router.norm()) <= 5 * 2.0 ** -8
    assert abs(float(train.loss[there].double().mean()) - float(ce.detach().mean())) <= 2.0 ** -6 * float(ce.detach().mean())
    assert (train.loss[~there] == 0).all()


def test_update(moe):
    train, x, u, labels = make(130, 500, 5)
    for i in range(3):
        train.gradients(x, u, labels)
        ds, params = [], {"head": train.head, "router": train.block.router_w, "w_post": train.block.w_post, "w_pre": train.block.w_pre,
                          "gate": train.block.gate}
        for name, p in params.items():
            flat = {k: t.view(-1) if k != "scales" else t for k, t in train.states[name].items()}
            ds.append({"param": p.view(-1), "grad": train.grads[name].view(-1),
                       "weight_decay": 0.1 if name in ("head", "router") else 0.0, **flat})
        want = [expected(d, step=i + 1, lr=float(train.lr), beta1=0.9, beta2=0.95) for d in ds]
        train.step_number += 1
        m.moe_adamw_step(train.tensors, train.options)
        for d, (xw, tol, st, alone) in zip(ds, want):
            # (the corrections on the device are taken in fp32: 2^-21 of the step, at most lr / sqrt(1 - beta2) times 4)
            verify(d, (xw, tol + 2.0 ** -21 * 1e-3 * 4 * 4.5, st, alone))


def test_captured_and_replayed(moe):
    a, x, u, labels = make(257, 400, 6)
    b, _, _, _ = make(257, 400, 6)
    for t in (a, b):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            t.step(x, u, labels)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(x, u, labels)
    for _ in range(3):
        graph.replay()
        b.step(x, u, labels)
    torch.cuda.synchronize()
    assert int(a.step_number) == int(b.step_number) == 4
    assert torch.equal(a.loss, b.loss) and torch.equal(a.head, b.head) and torch.equal(a.block.router_w, b.block.router_w)
    for n in a.states:
        for k in a.states[n]:
            assert torch.equal(a.states[n][k], b.states[n][k]), (n, k)


def test_refusals(moe):
    train, x, u, labels = make(20, 60)
    with pytest.raises(m.MoeError, match="labels"):
        train.gradients(x, u, labels.long())
    with pytest.raises(m.MoeError, match="tokens"):
        train.gradients(x[:10], u, labels)
    with pytest.raises(m.MoeError, match="head"):
        Mx4Training(train.block, torch.zeros(10, 8, device=DEV), 4)
