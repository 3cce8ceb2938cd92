"""moe_block_norm and its gradients against plain 64-bit forms: types, widths that are not a multiple of a vector,
gates of every kind, zero rows, strides, gradients that are absent."""
import numpy as np
import pytest
import torch

import bit_expert_ffn_gb300 as m
import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
TYPES = {torch.float32: m.MOE_F32, torch.bfloat16: m.MOE_BF16, torch.float16: m.MOE_F16}
PAIRS = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
         (torch.float32, torch.bfloat16), (torch.float32, torch.float16)]
SHAPES = [(1, 1), (1, 2048), (3, 8), (2, 33), (5, 264), (4, 1001), (700, 128), (6, 4096), (3, 4104), (2, 8200), (2, 16384),
          (2, 16383), (470, 24), (9, 256), (9, 257), (6, 512), (6, 513), (2, 8192), (5, 1002), (7, 70), (2, 6006),
          # where the rows ahead take just below 48 KB of shared memory, for one pair of types or another
          (4, 366), (5, 486), (2, 1532), (2, 2040), (2, 3064), (2, 4088), (2, 6136)]
GATES = {"none": m.MOE_GATE_NONE, "token": m.MOE_GATE_TOKEN, "channel": m.MOE_GATE_CHANNEL}
# A mean's 32-bit sum: at most 32 terms per thread, a tree of 5, 16 warps in turn; the root and the products after
# it are a few roundings more.
C = 80 * R.U32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def inputs(T, H, res, act, gate, seed):
    rng = np.random.default_rng(seed)
    s = {"x": dev((2 * rng.standard_normal((T, H))).astype(np.float32)).to(res),
         "b": dev(rng.standard_normal((T, H)).astype(np.float32)).to(act),
         "dy": dev(rng.standard_normal((T, H)).astype(np.float32)).to(res),
         "du": dev(rng.standard_normal((T, H)).astype(np.float32)).to(act),
         "w_post": dev((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)),
         "w_pre": dev((1 + 0.3 * rng.standard_normal(H)).astype(np.float32))}
    n = {"none": 0, "token": T, "channel": H}[gate]
    s["gate"] = dev(rng.standard_normal(n).astype(np.float32)) if n else None
    if T > 2:
        s["b"][1] = 0  # a block that gives nothing
    if T > 3:
        s["x"][2] = 0
        s["b"][2] = 0  # nothing at all: eps alone under the root
    return s


def wide_gate(s, gate):
    g = 1.0 if s["gate"] is None else R.f64(s["gate"])
    return g[:, None] if gate == "token" else g


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("res,act", PAIRS, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(moe, T, H, res, act, gate):
    s = inputs(T, H, res, act, gate, T + H)
    alpha = 0.75
    y = torch.full((T * H + 64,), 7.0, dtype=res, device=DEV)
    u = torch.full((T * H + 64,), 7.0, dtype=act, device=DEV)
    m.moe_block_norm(s["x"], TYPES[res], s["b"], TYPES[act], T, H, s["w_post"], s["w_pre"], s["gate"], GATES[gate],
                     alpha, EPS, y, u)
    assert bool((y[T * H:] == 7).all()) and bool((u[T * H:] == 7).all())
    g = wide_gate(s, gate)
    x, b, wp, wn = (R.f64(s[n]) for n in ("x", "b", "w_post", "w_pre"))
    v, wy, wu, r1, r2 = R.block_norm(x, b, wp, wn, g, alpha, EPS)
    dy = C * np.abs(alpha * g * v) + R.U32 * np.abs(x)
    R.within(y[:T * H].view(T, H), wy, dy, res)
    # the mean of y^2 moves by the rows' own errors
    dr = C + (np.abs(wy) * dy).mean(1, keepdims=True) * r2 ** 2
    R.within(u[:T * H].view(T, H), wu, np.abs(wu) * dr + r2 * np.abs(wn) * dy, act)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("res,act", PAIRS, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,H", SHAPES)
def test_gradients(moe, T, H, res, act, gate):
    s = inputs(T, H, res, act, gate, T * H)
    if T > 3:
        s["x"][2] = 1  # (a row of zeros has gradients of size 1 / sqrt(eps))
    alpha = 0.75
    nb = m.moe_block_norm_backward_workspace_size(T, H, GATES[gate])
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    dx = torch.full((T * H + 64,), 7.0, dtype=res, device=DEV)
    db = torch.full((T * H + 64,), 7.0, dtype=act, device=DEV)
    dwp, dwn = torch.full((H,), 9.0, device=DEV), torch.full((H,), 9.0, device=DEV)
    dg = None if s["gate"] is None else torch.full_like(s["gate"], 9.0)
    m.moe_block_norm_backward(s["x"], TYPES[res], s["b"], TYPES[act], T, H, s["w_post"], s["w_pre"], s["gate"], GATES[gate],
                              alpha, EPS, s["dy"], s["du"], dx, db, dwp, dwn, dg, ws, nb)
    assert bool((dx[T * H:] == 7).all()) and bool((db[T * H:] == 7).all())
    x, b, wp, wn, dy, du = (R.f64(s[n]) for n in ("x", "b", "w_post", "w_pre", "dy", "du"))
    got, mag = R.block_norm_backward(x, b, wp, wn, wide_gate(s, gate), alpha, EPS, dy, du)
    c = 6 * C  # three means, each of quantities that carry the ones before
    R.within(dx[:T * H].view(T, H), got[0], c * mag[0], res)
    R.within(db[:T * H].view(T, H), got[1], c * mag[1], act)
    cs = c + T * R.U32
    R.within(dwp, got[2].sum(0), cs * mag[2].sum(0), torch.float32)
    R.within(dwn, got[3].sum(0), cs * mag[3].sum(0), torch.float32)
    if dg is not None:
        ax = 1 if gate == "token" else 0
        R.within(dg, got[4].sum(ax), (cs + 60 * R.U32) * mag[4].sum(ax), torch.float32)


@pytest.mark.parametrize("gate", GATES)
def test_gradients_are_difference_quotients(moe, gate):
    T, H, alpha = 5, 72, 0.6
    s = inputs(T, H, torch.float32, torch.float32, gate, 3)
    s["b"][1] = 0.5
    s["x"][2] = 1
    nb = m.moe_block_norm_backward_workspace_size(T, H, GATES[gate])
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    out = {n: torch.empty_like(s[n]) for n in ("x", "b", "w_post", "w_pre")}
    out["gate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    m.moe_block_norm_backward(s["x"], m.MOE_F32, s["b"], m.MOE_F32, T, H, s["w_post"], s["w_pre"], s["gate"], GATES[gate],
                              alpha, EPS, s["dy"], s["du"], out["x"], out["b"], out["w_post"], out["w_pre"], out["gate"],
                              ws, nb)
    a = {n: R.f64(t) for n, t in s.items() if t is not None}
    rng = np.random.default_rng(4)
    for n in ("x", "b", "w_post", "w_pre", "gate"):
        if out.get(n) is None:
            continue
        d = rng.standard_normal(a[n].shape)

        def loss(h):
            z = dict(a)
            z[n] = a[n] + h * d
            g = z.get("gate", 1.0)
            g = g[:, None] if gate == "token" else g
            _, y, u, _, _ = R.block_norm(z["x"], z["b"], z["w_post"], z["w_pre"], g, alpha, EPS)
            return (a["dy"] * y).sum() + (a["du"] * u).sum()

        # fourth-order central difference: its own error is about (h / sqrt(eps))^4 at the row where b = 0, whose
        # curvature has the length sqrt(eps) = 1e-3
        h = 1e-5
        want = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
        got = R.f64(out[n])
        assert abs((got * d).sum() - want) <= 1e-5 * np.abs(got * d).sum() + 1e-6


def test_absent_gradients_and_weights(moe):
    T, H = 9, 200
    s = inputs(T, H, torch.float32, torch.bfloat16, "token", 8)
    s["x"][2] = 1
    nb = m.moe_block_norm_backward_workspace_size(T, H, m.MOE_GATE_TOKEN)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    one, zero_y, zero_u = torch.ones(H, device=DEV), torch.zeros_like(s["dy"]), torch.zeros_like(s["du"])

    def run(w, dy, du, sums):
        dx, db = torch.empty_like(s["x"]), torch.empty_like(s["b"])
        dw = [torch.empty(H, device=DEV) if sums else None for _ in range(2)]
        m.moe_block_norm_backward(s["x"], m.MOE_F32, s["b"], m.MOE_BF16, T, H, w, w, s["gate"], m.MOE_GATE_TOKEN, 1.0,
                                  EPS, dy, du, dx, db, dw[0], dw[1], None, ws, nb)
        return [t for t in (dx, db, *dw) if t is not None]

    for dy, du in ((s["dy"], None), (None, s["du"]), (None, None)):
        want = run(one, dy if dy is not None else zero_y, du if du is not None else zero_u, True)
        for a, b in zip(want, run(None, dy, du, True)):
            assert torch.equal(a, b)
        for a, b in zip(want, run(None, dy, du, False)):
            assert torch.equal(a, b)


def test_in_place_and_strides(moe):
    T, H = 21, 520
    s = inputs(T, H, torch.float32, torch.bfloat16, "channel", 9)
    args = (T, H, s["w_post"], s["w_pre"], s["gate"], m.MOE_GATE_CHANNEL, 0.5, EPS)
    y, u = torch.empty_like(s["x"]), torch.empty_like(s["b"])
    m.moe_block_norm(s["x"], m.MOE_F32, s["b"], m.MOE_BF16, *args, y, u)
    for pad in (8, 3):
        x2 = torch.zeros(T, H + pad, device=DEV)
        b2 = torch.zeros(T, H + pad, device=DEV, dtype=torch.bfloat16)
        x2[:, :H], b2[:, :H] = s["x"], s["b"]
        y2, u2 = torch.empty_like(y), torch.empty_like(u)
        m.moe_block_norm(x2[:, :H], m.MOE_F32, b2[:, :H], m.MOE_BF16, *args, y2, u2)
        if pad == 8:  # the same kernel
            assert torch.equal(y, y2) and torch.equal(u, u2)
        else:  # sums in another order
            assert torch.allclose(y, y2, rtol=1e-5, atol=1e-5)
            assert torch.allclose(u.float(), u2.float(), rtol=2 ** -7, atol=1e-5)
    x3, b3 = s["x"].clone(), s["b"].clone()
    m.moe_block_norm(x3, m.MOE_F32, b3, m.MOE_BF16, *args, x3, b3)
    assert torch.equal(x3, y) and torch.equal(b3, u)
    nb = m.moe_block_norm_backward_workspace_size(T, H, m.MOE_GATE_CHANNEL)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    dx, db = torch.empty_like(y), torch.empty_like(u)
    m.moe_block_norm_backward(s["x"], m.MOE_F32, s["b"], m.MOE_BF16, *args, s["dy"], s["du"], dx, db, ws=ws, ws_bytes=nb)
    dy, du = s["dy"].clone(), s["du"].clone()
    m.moe_block_norm_backward(s["x"], m.MOE_F32, s["b"], m.MOE_BF16, *args, dy, du, dy, du, ws=ws, ws_bytes=nb)
    assert torch.equal(dx, dy) and torch.equal(db, du)


def test_infinities_and_nan_stay_in_their_rows(moe):
    T, H = 6, 96
    s = inputs(T, H, torch.float32, torch.float32, "none", 10)
    args = (T, H, s["w_post"], s["w_pre"], None, m.MOE_GATE_NONE, 1.0, EPS)
    y, u = torch.empty_like(s["x"]), torch.empty_like(s["b"])
    m.moe_block_norm(s["x"], m.MOE_F32, s["b"], m.MOE_F32, *args, y, u)
    s["x"][0, 3], s["b"][4, 5] = float("inf"), float("nan")
    y2, u2 = torch.empty_like(y), torch.empty_like(u)
    m.moe_block_norm(s["x"], m.MOE_F32, s["b"], m.MOE_F32, *args, y2, u2)
    keep = [1, 2, 3, 5]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(u[keep], u2[keep])
    assert bool(torch.isnan(u2[4]).all()) and bool(torch.isinf(y2[0, 3]))


def test_no_tokens(moe):
    H = 40
    e = torch.empty(0, H, device=DEV)
    m.moe_block_norm(e, m.MOE_F32, e, m.MOE_F32, 0, H, None, None, None, m.MOE_GATE_NONE, 1.0, EPS, e, e)
    sums = [torch.full((H,), 5.0, device=DEV) for _ in range(3)]
    gate = torch.ones(H, device=DEV)
    m.moe_block_norm_backward(e, m.MOE_F32, e, m.MOE_F32, 0, H, None, None, gate, m.MOE_GATE_CHANNEL, 1.0, EPS, e, e, e, e,
                              *sums)
    assert all(bool((t == 0).all()) for t in sums)
