"""What the router's losses, the cross entropy and AdamW refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B

A = 1 << 20  # an aligned address that no refused call may touch
BAD = m.MOE_ERR_INVALID_ARG
f32, bf16, f16, i32, u8 = torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


def refused(status, word, fn, *args, **kw):
    with pytest.raises(m.MoeError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)
    assert word in str(e.value), str(e.value)


def loss(**kw):
    a = dict(logits=A, dtype=m.MOE_F32, T=2, E=8, ids=A, k=2, keep=None, loss=A, counts=A, mean_prob=A, lse=A)
    return {**a, **kw}


def test_router_loss():
    f, b = m.moe_router_loss, m.moe_router_loss_backward
    for kw, word in ((dict(dtype=3), "dtype"), (dict(E=0), "E"), (dict(E=1025), "E"), (dict(k=0), "k"), (dict(k=9), "k"),
                     (dict(E=64, k=17), "k"), (dict(T=-1), "T"), (dict(T=2 ** 30), "T"), (dict(logits=None), "NULL"),
                     (dict(ids=None), "NULL"), (dict(loss=None), "NULL"), (dict(lse=None), "NULL"), (dict(logits=A + 2), "aligned"),
                     (dict(counts=A + 1), "aligned"), (dict(dev_status=A + 2), "aligned")):
        refused(BAD, word, f, **loss(**kw))
    need = m.moe_router_loss_workspace_size(5000, 8)
    assert need > 0 and m.moe_router_loss_workspace_size(384, 1024) == 0
    refused(m.MOE_ERR_WORKSPACE, str(need), f, **loss(T=5000), ws=A, ws_bytes=need - 1)
    refused(m.MOE_ERR_WORKSPACE, str(need), f, **loss(T=5000))
    refused(BAD, "16-byte", f, **loss(T=5000), ws=A + 4, ws_bytes=need)
    refused(BAD, "E", m.moe_router_loss_workspace_size, 1, 2000)
    back = dict(logits=A, dtype=m.MOE_F32, T=2, E=8, ids=A, k=2, counts=A, lse=A, dloss=A, w=A, dw=A, dlogits=A)
    for kw, word in ((dict(dlogits=None), "NULL"), (dict(lse=None), "NULL"), (dict(w=None), "together"), (dict(dw=None), "together"),
                     (dict(ids=None), "ids"), (dict(dlogits=A + 1), "aligned"), (dict(dtype=-1), "dtype"), (dict(k=11), "k")):
        refused(BAD, word, b, **{**back, **kw})
    assert b(**{**back, "T": 0}) is None


def ce(**kw):
    return {**dict(h=A, dtype=m.MOE_BF16, T=2, H=64, w=A, V=100, labels=A, loss=A, lse=A, ws=A, ws_bytes=1 << 30), **kw}


def test_cross_entropy():
    f, b = m.moe_cross_entropy, m.moe_cross_entropy_backward
    for kw, word in ((dict(dtype=m.MOE_F32), "dtype"), (dict(H=0), "H"), (dict(H=12), "H"), (dict(V=0), "V"), (dict(T=-1), "T"),
                     (dict(V=2 ** 24 + 1), "V"), (dict(T=2 ** 24, V=2 ** 24), "tiles"), (dict(h=None), "NULL"), (dict(labels=None), "NULL"),
                     (dict(lse=None), "NULL"), (dict(h=A + 8), "16-byte"), (dict(w=A + 2), "16-byte"), (dict(labels=A + 2), "aligned"),
                     (dict(loss=A + 2), "aligned"), (dict(ws=A + 8), "16-byte")):
        refused(BAD, word, f, **ce(**kw))
    need = m.moe_cross_entropy_workspace_size(2, 64, 100)
    refused(m.MOE_ERR_WORKSPACE, str(need), f, **ce(ws_bytes=need - 1))
    refused(m.MOE_ERR_WORKSPACE, str(need), f, **ce(ws=None))
    assert f(**ce(T=0)) is None
    back = dict(h=A, dtype=m.MOE_F16, T=2, H=64, w=A, V=100, labels=A, lse=A, dloss=A, dlse=None, dh=A, dw=A, dw_dtype=m.MOE_F16,
                accumulate=False, ws=A, ws_bytes=1 << 30)
    for kw, word in ((dict(dw_dtype=m.MOE_BF16), "dw_dtype"), (dict(accumulate=True), "accumulated"), (dict(dh=A + 2), "16-byte"),
                     (dict(dw=A + 4), "16-byte"), (dict(lse=None), "NULL"), (dict(dloss=None), "NULL"), (dict(dlse=A + 1), "aligned"),
                     (dict(ws=A + 4), "16-byte")):
        refused(BAD, word, b, **{**back, **kw})
    need = m.moe_cross_entropy_backward_workspace_size(2, 64, 100)
    refused(m.MOE_ERR_WORKSPACE, str(need), b, **{**back, "ws_bytes": need - 1})
    assert b(**{**back, "dh": None, "dw": None}) is None
    # the logits' gradient is held for a piece of the vocabulary only
    assert m.moe_cross_entropy_backward_workspace_size(8192, 2048, 200_000) < (257 << 20) + 8192 * 2048 * 4


def a_tensor(n=300, **kw):
    return {**dict(param=torch.zeros(n), grad=torch.zeros(n), m=torch.zeros(n), v=torch.zeros(n)), **kw}


OPT = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)


def raw(**kw):
    """One tensor of made-up addresses, as AdamwTensors holds it."""
    a = dict(param=A, grad=2 * A, master=None, m=3 * A, v=4 * A, scales=None, n=16, param_dtype=m.MOE_F32, grad_dtype=m.MOE_F32,
             lr_factor=1.0, weight_decay=0.0)
    arr = (m.moe_adamw_tensor * 1)()
    for k, v in {**a, **kw}.items():
        setattr(arr[0], k, v)
    return m.AdamwTensors(arr, [])


def test_adamw():
    f = m.moe_adamw_step
    o = lambda **kw: m.moe_adamw_options(**{**OPT, **kw})  # noqa: E731
    for kw, word in ((dict(param=None), "NULL"), (dict(grad=None), "NULL"), (dict(m=None), "NULL"), (dict(v=None), "NULL"), (dict(n=-1), "n "),
                     (dict(param_dtype=5), "param_dtype"), (dict(grad_dtype=-2), "grad_dtype"), (dict(param=A + 2), "aligned"),
                     (dict(master=A + 2), "aligned"), (dict(m=A + 1), "aligned"), (dict(scales=A + 4), "scales"),
                     (dict(lr_factor=float("nan")), "finite"), (dict(weight_decay=float("inf")), "finite")):
        refused(BAD, word, f, raw(**kw), o())
    for kw, word in ((dict(beta1=1.0), "beta1"), (dict(beta2=-0.1), "beta2"), (dict(eps=0.0), "eps"), (dict(eps=1e-60), "eps"), (dict(eps=1e-40), "eps"),
                     (dict(step=0), "step"), (dict(lr=float("nan")), "lr"), (dict(lr_dev=A + 2), "aligned"), (dict(step_dev=A + 4), "aligned")):
        refused(BAD, word, f, raw(), o(**kw))
    two = (m.moe_adamw_tensor * 2)(raw().array[0], raw().array[0])
    refused(BAD, "overlap", f, m.AdamwTensors(two, []), o())
    with pytest.raises(m.MoeError, match="options"):
        m._check(m.lib().moe_adamw_step(raw().array, 1, None, None, None), "moe_adamw_step")
    with pytest.raises(m.MoeError, match="n_tensors"):
        m._check(m.lib().moe_adamw_step(raw().array, -1, ctypes.byref(o()), None, None), "moe_adamw_step")
    assert f(m.make_adamw_tensors([]), o()) is None
    assert f(raw(n=0), o()) is None
    refused(BAD, "aligned", m.moe_adamw_states, raw(), m.AdamwValues((ctypes.c_void_p * 1)(A + 2), None, [None, None], None))


def test_adamw_tensors():
    f = m.make_adamw_tensors
    refused(BAD, "on the GPU", f, [a_tensor()])
    refused(BAD, "needed", f, [a_tensor(grad=None)])
    refused(BAD, "needed", f, [a_tensor(decay=0.1)])
    refused(BAD, "grad", f, [a_tensor(grad=torch.zeros(299))])
    refused(BAD, "301", f, [a_tensor(grad=torch.zeros(301))])
    refused(BAD, "param", f, [a_tensor(param=torch.zeros(300, dtype=torch.float64))])
    refused(BAD, "m must", f, [a_tensor(m=torch.zeros(300, dtype=u8))])
    refused(BAD, "m must", f, [a_tensor(scales=torch.zeros(2, 2))])
    eight = dict(m=torch.zeros(300, dtype=u8), v=torch.zeros(300, dtype=u8))
    refused(BAD, "scales", f, [a_tensor(**eight, scales=torch.zeros(1, 2))])
    refused(BAD, "packed", f, [a_tensor(v=torch.zeros(600)[::2])])
    x = torch.zeros(700)
    refused(BAD, "overlaps", f, [a_tensor(param=x[:300]), a_tensor(param=x[299:599])])
    refused(BAD, "overlaps", f, [a_tensor(param=x[:300]), a_tensor(m=x[100:400])])
    refused(BAD, "overlaps", f, [a_tensor(param=x[:300]), a_tensor(grad=x[200:500])])
    refused(BAD, "on the GPU", f, [a_tensor(grad=x[:300]), a_tensor(grad=x[:300])])  # gradients are only read


def operands():
    z = lambda *s, t=f32: torch.zeros(*s, dtype=t)  # noqa: E731
    return {
        "router_loss": (m.moe_router_loss, dict(logits=z(4, 8), dtype=m.MOE_F32, T=4, E=8, ids=z(4, 2, t=i32), k=2, keep=z(4, t=u8),
                                                loss=z(2), counts=z(9, t=i32), mean_prob=z(8), lse=z(4), ws=z(64, t=u8), ws_bytes=64,
                                                dev_status=z(1, t=i32))),
        "router_loss_backward": (m.moe_router_loss_backward, dict(
            logits=z(4, 8), dtype=m.MOE_F32, T=4, E=8, ids=z(4, 2, t=i32), k=2, counts=z(9, t=i32), lse=z(4), dloss=z(2), w=z(4, 2),
            dw=z(4, 2), dlogits=z(4, 8))),
        "cross_entropy": (m.moe_cross_entropy, dict(h=z(4, 16, t=bf16), dtype=m.MOE_BF16, T=4, H=16, w=z(9, 16, t=bf16), V=9,
                                                    labels=z(4, t=i32), loss=z(4), lse=z(4), ws=z(4096, t=u8), ws_bytes=4096,
                                                    dev_status=z(1, t=i32))),
        "cross_entropy_backward": (m.moe_cross_entropy_backward, dict(
            h=z(4, 16, t=bf16), dtype=m.MOE_BF16, T=4, H=16, w=z(9, 16, t=bf16), V=9, labels=z(4, t=i32), lse=z(4), dloss=z(4),
            dlse=z(4), dh=z(4, 16, t=bf16), dw=z(9, 16), dw_dtype=m.MOE_F32, accumulate=True, ws=z(8192, t=u8), ws_bytes=8192,
            dev_status=z(1, t=i32))),
    }


TENSORS = [(c, n) for c, (_, a) in operands().items() for n, t in a.items() if isinstance(t, torch.Tensor)]
SAME_SIZE = {bf16: f16, f32: i32, i32: f32, u8: torch.float8_e4m3fn}


@pytest.mark.parametrize("call,name", TENSORS)
def test_another_type_or_too_short(call, name):
    fn, args = operands()[call]
    full = args[name]
    args[name] = full.reshape(-1)[:-1]
    refused(BAD, name, fn, **args)
    if name != "ws":
        args[name] = full.to(SAME_SIZE[full.dtype])
        refused(BAD, f"{name} must", fn, **args)


@pytest.mark.parametrize("call,name", TENSORS)
def test_a_tensor_on_the_host(call, name):
    """Everything else is an address that no call may come as far as using."""
    fn, args = operands()[call]
    host = args[name]
    args = {n: A if isinstance(t, torch.Tensor) else t for n, t in args.items()}
    args[name] = host
    refused(BAD, f"{name} must be on the GPU", fn, **args)
