"""Cases of the framework's operators of a training step around its blocks.

    router_loss     balance loss, squared log-sum loss and counts per expert from the router's logits; and the logits'
                    gradient from both losses and from the routing weights
    cross_entropy   softmax cross entropy of hidden states against a head's weights, logits not kept; and the gradients
    adamw           one AdamW step over many tensors, states in 32 bits or in 8 bits with scales per 256

``run`` computes a case in elementary torch operations, or, where ``own`` is true, by the framework's calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
DEV = "cuda"
BLOCK = 256  # values that share a scale
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.1, 1000


def listed():
    return [
        # the tokens of a small evaluation batch over the layer's 512 experts: all latency
        {"name": "router_loss_small", "op": "router_loss", "dir": "fwd", "T": 32, "E": 512, "k": 10, "pad": False, "type": "f32"},
        # a 32K-token batch watched for its balance
        {"name": "router_loss_batch", "op": "router_loss", "dir": "fwd", "T": 32768, "E": 512, "k": 10, "pad": False, "type": "f32"},
        # the same batch trained: losses, and the logits' gradient
        {"name": "router_loss_gradient", "op": "router_loss", "dir": "train", "T": 32768, "E": 512, "k": 10, "pad": False, "type": "f32"},
        # a padded batch of odd size, logits in 16 bits
        {"name": "router_loss_padded", "op": "router_loss", "dir": "train", "T": 9973, "E": 61, "k": 4, "pad": True, "type": "bf16"},
        # scoring a verify window of four tokens: the head's weights are read once
        {"name": "cross_entropy_window", "op": "cross_entropy", "dir": "fwd", "T": 4, "H": 2048, "V": 100003, "type": "bf16"},
        # the loss of a 4K-token evaluation batch
        {"name": "cross_entropy_batch", "op": "cross_entropy", "dir": "fwd", "T": 4096, "H": 2048, "V": 65536, "type": "bf16"},
        # a training batch: loss, gradients of the hidden states and of the head
        {"name": "cross_entropy_gradient", "op": "cross_entropy", "dir": "train", "T": 4096, "H": 2048, "V": 65536, "type": "bf16"},
        # a short batch on a small head, nothing a multiple of a tile
        {"name": "cross_entropy_odd", "op": "cross_entropy", "dir": "train", "T": 1111, "H": 1056, "V": 8191, "type": "bf16"},
        # the norms and the gate of one block: all latency
        {"name": "adamw_norms", "op": "adamw", "groups": 1, "big": 0, "small": 2048, "param": "f32", "master": False, "grad": "f32", "states": 32},
        # the routers, norms and gates of 48 layers
        {"name": "adamw_routers", "op": "adamw", "groups": 48, "big": 512 * 2048, "small": 2048, "param": "f32", "master": False, "grad": "f32", "states": 32},
        # 40 experts of 3 x 768 x 2048 in 16 bits with a 32-bit copy, states in 8 bits
        {"name": "adamw_experts", "op": "adamw", "groups": 40, "big": 3 * 768 * 2048, "small": 0, "param": "bf16", "master": True, "grad": "bf16", "states": 8},
        # many small tensors of odd sizes without a copy
        {"name": "adamw_odd", "op": "adamw", "groups": 100, "big": 40009, "small": 333, "param": "bf16", "master": False, "grad": "bf16", "states": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router_loss", "cross_entropy", "adamw"])
    if op == "router_loss":
        E = rng.choice([_log(rng, 2, 1024), 4 * _log(rng, 1, 256)])
        k = rng.randint(1, min(E, 16))
        return {"op": op, "dir": rng.choice(["fwd", "train"]), "T": _log(rng, 1, min(65536, 16_000_000 // E)), "E": E, "k": k,
                "pad": rng.random() < 0.4, "type": rng.choice(["f32", "f32", "bf16", "f16"])}
    if op == "cross_entropy":
        H = 8 * _log(rng, 8, 512)
        V = _log(rng, 64, 130000)
        top = max(1, min(16384, 500_000_000_000 // (H * V), 250_000_000 // V))
        return {"op": op, "dir": rng.choice(["fwd", "train"]), "T": _log(rng, 1, top), "H": H, "V": V,
                "type": rng.choice(["bf16", "bf16", "f16"])}
    groups = _log(rng, 1, 120)
    param = rng.choice(["f32", "bf16", "f16"])
    return {"op": op, "groups": groups, "big": _log(rng, 100, 150_000_000 // groups), "small": rng.choice([0, _log(rng, 1, 8192)]),
            "param": param, "master": param != "f32" and rng.random() < 0.5, "grad": rng.choice(["f32", param]),
            "states": rng.choice([8, 32])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    """Normal values, made in pieces so that large ones need no second copy in 32 bits."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        b = min(flat.numel(), a + (1 << 27))
        flat[a:b] = torch.randn(b - a, generator=g, device=DEV) * scale
    return out


def _sizes(c):
    """The tensors of a group: one big one, three small ones."""
    out = []
    for _ in range(c["groups"]):
        out += [c["big"]] * (c["big"] > 0) + [c["small"]] * (3 * (c["small"] > 0))
    return out


def _places(c):
    """Where each tensor lies in a flat buffer (each begins at a multiple of 256 values, as an allocator would place
    it), and the buffer's length."""
    at, out = 0, []
    for n in _sizes(c):
        out.append((at, n))
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return out, at


def _inputs(c, seed):
    """What both sides are given: tensors made from the seed alone."""
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "router_loss":
        T, E, k = c["T"], c["E"], c["k"]
        pop = torch.randn(E, generator=g, device=DEV)  # some experts are more popular than others
        s["logits"] = (torch.randn(T, E, generator=g, device=DEV) + pop).to(TYPES[c["type"]])
        top = torch.topk(s["logits"].float(), k, dim=1)
        s["ids"] = top.indices.int()
        w = torch.exp(top.values - top.values[:, :1])
        s["w"] = w / w.sum(1, keepdim=True)
        # sequences of 1,000 places, each filled to a length of its own
        ends = torch.randint(1, 1001, ((T + 999) // 1000,), generator=g, device=DEV)
        place = torch.arange(T, device=DEV)
        s["keep"] = (place % 1000 < ends[place // 1000]).to(torch.uint8) if c["pad"] else None
        s["dloss"] = torch.tensor([0.01, 0.001], device=DEV)
        s["dw"] = torch.randn(T, k, generator=g, device=DEV) / T if c["dir"] == "train" else None
    elif c["op"] == "cross_entropy":
        T, H, V, t = c["T"], c["H"], c["V"], TYPES[c["type"]]
        s["w"] = _normal(g, V, H, dtype=t, scale=2.5 / math.sqrt(H))
        labels = torch.randint(0, V, (T,), generator=g, device=DEV)
        # hidden states that know something of their labels; a tenth of the places have none
        lean = 2.4 * torch.rand(T, 1, generator=g, device=DEV)
        s["h"] = (torch.randn(T, H, generator=g, device=DEV) + lean * s["w"][labels].float()).to(t)
        none = torch.rand(T, generator=g, device=DEV) < 0.1
        s["labels"] = torch.where(none, -100, labels).int()
        s["dloss"] = torch.full((T,), 1.0 / max(1, T - int(none.sum())), device=DEV)
    else:
        s["places"], n = _places(c)
        inside = torch.zeros(n, dtype=torch.bool, device=DEV)
        for at, size in s["places"]:
            inside[at:at + size] = True
        master = _normal(g, n, scale=0.02) * inside
        s["param"] = master.to(TYPES[c["param"]])
        s["master"] = master if c["master"] else None
        spread = torch.exp(_normal(g, n))  # values of unlike gradients
        s["grad"] = (_normal(g, n, scale=1e-3) * spread * inside).to(TYPES[c["grad"]])
        m = _normal(g, n, scale=3e-4) * spread * inside
        v = (1e-3 * spread * inside) ** 2 * (0.5 + torch.rand(n, generator=g, device=DEV))
        if c["states"] == 32:
            s["m"], s["v"] = m, v
        else:
            s["m"], s["v"], s["scales"] = _encode(m, v)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import bit_expert_ffn_gb300 as moe

    c = case
    s["moe"] = moe
    D = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "f16": moe.MOE_F16}
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"] == "router_loss":
        T, E = c["T"], c["E"]
        s["t"] = D[c["type"]]
        s["loss"], s["counts"], s["mean"], s["lse"] = new(2), new(E + 1, dtype=torch.int32), new(E), new(T)
        s["ws_bytes"] = moe.moe_router_loss_workspace_size(T, E)
        s["ws"] = new(max(1, s["ws_bytes"]), dtype=torch.uint8)
        if c["dir"] == "train":
            s["dlogits"] = torch.empty_like(s["logits"])
    elif c["op"] == "cross_entropy":
        T, H, V = c["T"], c["H"], c["V"]
        s["t"] = D[c["type"]]
        s["loss"], s["lse"] = new(T), new(T)
        s["ws_bytes"] = moe.moe_cross_entropy_workspace_size(T, H, V)
        if c["dir"] == "train":
            s["dh"], s["dhead"] = torch.empty_like(s["h"]), torch.empty_like(s["w"])
            s["back_bytes"] = moe.moe_cross_entropy_backward_workspace_size(T, H, V)
        s["ws"] = new(max(1, s["ws_bytes"], s.get("back_bytes", 0)), dtype=torch.uint8)
    else:
        part = lambda t, at, n: t[at:at + n]  # noqa: E731
        tensors = []
        s["m_values"], s["v_values"] = torch.zeros_like(s["m"], dtype=torch.float32), torch.zeros_like(s["v"], dtype=torch.float32)
        for at, n in s["places"]:
            tensors.append(dict(
                param=part(s["param"], at, n), grad=part(s["grad"], at, n), m=part(s["m"], at, n), v=part(s["v"], at, n),
                master=part(s["master"], at, n) if c["master"] else None,
                scales=s["scales"][at // BLOCK:(at + n + BLOCK - 1) // BLOCK] if c["states"] == 8 else None,
                weight_decay=DECAY if n == c["big"] else 0.0))
        s["tensors"] = moe.make_adamw_tensors(tensors)
        s["options"] = moe.moe_adamw_options(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, step=STEP)
        if c["states"] == 8:
            s["values"] = moe.make_adamw_values([part(s["m_values"], at, n) for at, n in s["places"]],
                                                [part(s["v_values"], at, n) for at, n in s["places"]])
    return s


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    c, moe = s["c"], s["moe"]
    if c["op"] == "router_loss":
        T, E, k = c["T"], c["E"], c["k"]
        moe.moe_router_loss(s["logits"], s["t"], T, E, s["ids"], k, s["keep"], s["loss"], s["counts"], s["mean"], s["lse"],
                            s["ws"], s["ws_bytes"])
        out = {"loss": s["loss"], "counts": s["counts"], "mean": s["mean"]}
        if c["dir"] == "train":
            moe.moe_router_loss_backward(s["logits"], s["t"], T, E, s["ids"], k, s["counts"], s["lse"], s["dloss"], s["w"],
                                         s["dw"], s["dlogits"])
            out["dlogits"] = s["dlogits"]
        return out
    if c["op"] == "cross_entropy":
        T, H, V = c["T"], c["H"], c["V"]
        moe.moe_cross_entropy(s["h"], s["t"], T, H, s["w"], V, s["labels"], s["loss"], s["lse"], s["ws"], s["ws_bytes"])
        if c["dir"] == "fwd":
            return s["loss"]
        moe.moe_cross_entropy_backward(s["h"], s["t"], T, H, s["w"], V, s["labels"], s["lse"], s["dloss"], None, s["dh"],
                                       s["dhead"], s["t"], False, s["ws"], s["back_bytes"])
        return {"loss": s["loss"], "dh": s["dh"], "dw": s["dhead"]}
    moe.moe_adamw_step(s["tensors"], s["options"])
    out = {"param": s["param"]}
    if c["master"]:
        out["master"] = s["master"]
    if c["states"] == 32:
        out["m"], out["v"] = s["m"], s["v"]
    else:
        moe.moe_adamw_states(s["tensors"], s["values"])
        out["m"], out["v"] = s["m_values"], s["v_values"]
    return out


# ---------------------------------------------------------------- plain form

def _encode(m, v):
    """8-bit codes of m (e4m3) and of the root of v (an unsigned float: 4 exponent and 4 mantissa bits, code 0 for zero
    alone), and the scales [blocks][2]."""
    mb, r = m.view(-1, BLOCK), torch.sqrt(v).view(-1, BLOCK)
    tops = torch.stack([mb.abs().amax(1), r.amax(1)], 1)
    tops = torch.where(tops < 2.0 ** -100, torch.zeros_like(tops), tops)
    top = torch.tensor([448.0, 1.9375], device=m.device)
    inv = torch.where(tops > 0, top / tops, torch.zeros_like(tops))
    mc = (mb * inv[:, :1]).to(torch.float8_e4m3fn).view(torch.uint8)
    bits = (r * inv[:, 1:]).view(torch.int32)
    near = (bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19  # to nearest of 4 mantissa bits, ties to even
    vc = (near - (112 << 4)).clamp(1, 255)
    vc = torch.where((r > 0) & (tops[:, 1:] > 0), vc, torch.zeros_like(vc)).to(torch.uint8)
    return mc.view(-1), vc.view(-1), tops / top


def _decode(mc, vc, scales):
    """The values that codes and scales stand for."""
    m = mc.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scales[:, :1]
    code = vc.view(-1, BLOCK).int()
    r = torch.where(code > 0, (code + (112 << 4)) << 19, torch.zeros_like(code)).view(torch.float32) * scales[:, 1:]
    return m.view(-1), (r * r).view(-1)


def run(s):
    if own:
        return _run_own(s)
    c = s["c"]
    if c["op"] == "router_loss":
        T, E, k = c["T"], c["E"], c["k"]
        l = s["logits"].float()
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - top)
        z = e.sum(1, keepdim=True)
        p, lse = e / z, (top + torch.log(z))[:, 0]
        f = torch.ones(T, device=l.device) if s["keep"] is None else (s["keep"] != 0).float()
        n = f.sum()
        n1 = n.clamp_min(1.0)
        count = torch.zeros(E, device=l.device)
        count.index_add_(0, s["ids"].reshape(-1).long(), f[:, None].expand(T, k).reshape(-1))
        mean = (p * f[:, None]).sum(0) / n1
        loss = torch.stack([E * (count / (n1 * k) * mean).sum(), (lse * lse * f).sum() / n1])
        out = {"loss": loss, "counts": torch.cat([count, n[None]]).int(), "mean": mean}
        if c["dir"] == "train":
            d = s["dloss"]
            ge = d[0] * E * count / (n1 * n1 * k)
            grad = p * (ge - (p * ge).sum(1, keepdim=True) + (2.0 * d[1] / n1) * lse[:, None]) * f[:, None]
            dv = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True))
            out["dlogits"] = grad.scatter_add_(1, s["ids"].long(), dv).to(s["logits"].dtype)
        return out
    if c["op"] == "cross_entropy":
        h, w = s["h"].float(), s["w"].float()
        there = (s["labels"] >= 0).float()
        label = s["labels"].clamp_min(0).long()[:, None]
        z = h @ w.T
        top = z.amax(1, keepdim=True)
        own_z = z.gather(1, label)
        p = torch.exp(z.sub_(top))
        total = p.sum(1, keepdim=True)
        loss = (torch.log(total) + top - own_z)[:, 0] * there
        if c["dir"] == "fwd":
            return loss
        p /= total
        p.scatter_add_(1, label, torch.full_like(total, -1.0))
        p *= (s["dloss"] * there)[:, None]
        return {"loss": loss, "dh": (p @ w).to(s["h"].dtype), "dw": (p.T @ h).to(s["w"].dtype)}
    old = (s["m"], s["v"]) if c["states"] == 32 else _decode(s["m"], s["v"], s["scales"])
    g = s["grad"].float()
    m = old[0] * BETA1 + g * (1.0 - BETA1)
    v = old[1] * BETA2 + (g * g) * (1.0 - BETA2)
    b1, b2 = 1.0 - BETA1 ** STEP, 1.0 - BETA2 ** STEP
    x = s["master"] if c["master"] else s["param"].float()
    step = m / (torch.sqrt(v) / math.sqrt(b2) + EPS) * (LR / b1)
    x = _shrink(s, x) - step
    out = {}
    if c["master"]:
        out["master"] = s["master"].copy_(x)
    out["param"] = s["param"].copy_(x)
    if c["states"] == 32:
        out["m"], out["v"] = s["m"].copy_(m), s["v"].copy_(v)
    else:
        s["m"], s["v"], s["scales"] = _encode(m, v)
        out["m"], out["v"] = _decode(s["m"], s["v"], s["scales"])
    return out


def _shrink(s, x):
    """x (1 - lr decay), where a tensor decays."""
    c = s["c"]
    x = x.clone()
    for at, n in s["places"]:
        if n == c["big"]:
            x[at:at + n] *= 1.0 - LR * DECAY
    return x


# ---------------------------------------------------------------- the definition in 64 bits

def _grid():
    """The values of the 8-bit codes of the root, in order."""
    code = torch.arange(1, 256, device=DEV)
    return torch.cat([torch.zeros(1, dtype=torch.float64, device=DEV), (16 + code % 16).double() * 2.0 ** (code // 16 - 19).double()])


def _e4m3():
    """The values of the e4m3 codes 0 .. 126."""
    code = torch.arange(127, device=DEV)
    e, f = code // 8, (code % 8).double()
    return torch.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10).double())


def _nearest(x, grid):
    """The index of the nearest grid value; a tie goes to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(x, mid), torch.bucketize(x, mid, right=True)
    return torch.where(low % 2 == 0, low, high)


def _r32(x):
    """Rounded to 32 bits.  States in 8 bits are defined by 32-bit steps, each rounded to nearest, so that codes next to
    a border are the same everywhere: a product, sum, quotient or root of 32-bit numbers taken in 64 bits and rounded
    is that step."""
    return x.float().double()


def _held(m, v):
    """m and v (32-bit numbers) as 8 bits hold them."""
    out_m, out_v, e4m3, grid = torch.empty_like(m), torch.empty_like(v), _e4m3(), _grid()
    for a in range(0, m.numel(), 1 << 22):
        x, r = m[a:a + (1 << 22)].view(-1, BLOCK), _r32(torch.sqrt(v[a:a + (1 << 22)])).view(-1, BLOCK)
        for src, dst, g, root in ((x, out_m, e4m3, False), (r, out_v, grid, True)):
            top = src.abs().amax(1, keepdim=True)
            some = top >= 2.0 ** -100
            top = torch.where(some, top, torch.ones_like(top))
            code = _nearest(_r32(src.abs() * _r32(g[-1] / top)), g)
            if root:  # only zero is held as zero
                code = torch.where(src > 0, code.clamp_min(1), code)
            val = torch.sign(src) * _r32(g[code] * _r32(top / g[-1])) * some
            dst[a:a + (1 << 22)] = (_r32(val * val) if root else val).view(-1)
    return out_m, out_v


def _values64(s):
    c = s["c"]
    if c["states"] == 32:
        return s["m"].double(), s["v"].double()
    unit = s["scales"].double().repeat_interleave(BLOCK, 0)
    mag = _e4m3()[(s["m"] & 127).long()]
    m = _r32(torch.where(s["m"] >= 128, -mag, mag) * unit[:, 0])
    return m, _r32(_r32(_grid()[s["v"].long()] * unit[:, 1]) ** 2)


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "router_loss":
        E, k, T = c["E"], c["k"], c["T"]
        l = s["logits"].double().requires_grad_()
        kept = torch.ones(T, dtype=torch.bool, device=DEV) if s["keep"] is None else s["keep"].bool()
        n = int(kept.sum())
        picks = s["ids"][kept].reshape(-1).long()
        count = torch.bincount(picks, minlength=E)
        counts = torch.cat([count, torch.tensor([n], device=DEV)]).int()
        if n:
            lse = torch.logsumexp(l[kept], 1)
            mean = torch.softmax(l[kept], 1).mean(0)
            balance, square = E * torch.dot(count.double() / (n * k), mean), lse.square().mean()
        else:
            mean = torch.zeros(E, dtype=torch.float64, device=DEV)
            balance = square = (l * 0.0).sum()
        out = {"loss": torch.stack([balance, square]).detach(), "counts": counts, "mean": mean.detach()}
        if c["dir"] == "train":
            w = s["w"].double()  # the kept experts' softmax, as given: dl = w (dw - <w, dw>) at their places
            dv = w * s["dw"].double()
            dv = dv - w * dv.sum(1, keepdim=True)
            grad = torch.autograd.grad(balance * s["dloss"][0].double() + square * s["dloss"][1].double(), l)[0]
            rows = torch.arange(T, device=DEV)[:, None].expand(T, k)
            out["dlogits"] = grad.index_put((rows, s["ids"].long()), dv, accumulate=True)
        return out
    if c["op"] == "cross_entropy":
        T, V = c["T"], c["V"]
        if T * V * c["H"] > 600_000_000_000:
            return None
        h, w = s["h"].double(), s["w"].double()
        loss = torch.zeros(T, dtype=torch.float64, device=DEV)
        dh, dw = torch.zeros_like(h), torch.zeros_like(w)
        for a in range(0, T, 1024):
            b = min(T, a + 1024)
            rows = torch.nonzero(s["labels"][a:b] >= 0)[:, 0]
            label = s["labels"][a:b][rows].long()
            logp = torch.log_softmax(torch.matmul(h[a:b][rows], w.t()), dim=1)
            at = torch.arange(rows.numel(), device=DEV)
            loss[a + rows] = -logp[at, label]
            if c["dir"] == "train":
                dz = logp.exp_()
                dz[at, label] -= 1.0
                dz *= s["dloss"][a:b][rows].double().unsqueeze(1)
                dh[a + rows] = torch.matmul(dz, w)
                dw.addmm_(dz.t(), h[a:b][rows])
        return loss if c["dir"] == "fwd" else {"loss": loss, "dh": dh, "dw": dw}
    old_m, old_v = _values64(s)
    g = s["grad"].double()
    if c["states"] == 32:
        m, v = torch.lerp(g, old_m, BETA1), torch.lerp(g.square(), old_v, BETA2)
    else:
        f1, f2, o1, o2 = _r32(torch.tensor([BETA1, BETA2, 1.0 - BETA1, 1.0 - BETA2], dtype=torch.float64)).tolist()
        m = _r32(_r32(old_m * f1) + _r32(g * o1))
        v = _r32(_r32(old_v * f2) + _r32(_r32(g.square()) * o2))
    x = (s["master"] if c["master"] else s["param"]).double()
    rate = torch.ones_like(x)
    for at, n in s["places"]:
        if n == c["big"]:
            rate[at:at + n] = 1.0 - LR * DECAY
    x = x * rate - LR * (m / (1.0 - BETA1 ** STEP)) / (torch.sqrt(v / (1.0 - BETA2 ** STEP)) + EPS)
    if c["states"] == 8:
        m, v = _held(m, v)
    out = {"master": x} if c["master"] else {}
    out.update(param=x, m=m, v=v)
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(c):
    if c["op"] == "router_loss":
        T, E, k, b = c["T"], c["E"], c["k"], SIZE[c["type"]]
        fwd = T * E * b + T * k * 4 + (T if c["pad"] else 0) + 8 * E + 12
        if c["dir"] == "fwd":
            return {"bytes": fwd, "flops": 5 * T * E}
        # the losses need every logit before any gradient: the logits come twice
        return {"bytes": fwd + 2 * T * E * b + 8 * T * k, "flops": 12 * T * E}
    if c["op"] == "cross_entropy":
        T, H, V, b = c["T"], c["H"], c["V"], SIZE[c["type"]]
        if c["dir"] == "fwd":
            return {"bytes": (T + V) * H * b + 8 * T, "flops": 2 * T * H * V}
        # the product again (its logits are not kept), and the two gradients
        return {"bytes": 2 * (T + V) * H * b + 12 * T, "flops": 8 * T * H * V}
    n, p, g = sum(_sizes(c)), SIZE[c["param"]], SIZE[c["grad"]]
    held = (p if not c["master"] else 4 + 4) + p + g  # 16-bit parameters beside a copy are only written
    # 8-bit states: read and written, scales too, and their values given out
    return {"bytes": n * (held + 16) if c["states"] == 32 else n * (held + 4 + 8) + n * 16 // BLOCK, "flops": 14 * n}
