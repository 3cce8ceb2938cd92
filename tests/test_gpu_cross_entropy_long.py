"""A cross entropy that takes longer than any of its waits may."""
import pytest
import torch

import bit_expert_ffn_gb300 as m

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_a_product_of_seconds(moe):
    """786,432 tokens against 524,288 words, H = 8,192: 6.8 * 10^15 operations, some 3.5 s by pairs of CTAs, of which each wait takes
    microseconds.  No wait runs out, and the losses are right."""
    T, H, V = 3 << 18, 8192, 1 << 19
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    g = torch.Generator(device=DEV).manual_seed(0)

    def normal(rows, scale):
        t = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
        for a in range(0, rows, 1 << 16):
            t[a:a + (1 << 16)] = torch.randn(min(1 << 16, rows - a), H, generator=g, device=DEV) * scale
        return t

    h, w = normal(T, 1.0), normal(V, 2.0 / H ** 0.5)
    labels = torch.randint(0, V, (T,), generator=g, device=DEV).int()
    loss, lse = torch.full((T,), 7.0, device=DEV), torch.full((T,), 7.0, device=DEV)
    nb = m.moe_cross_entropy_workspace_size(T, H, V)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    m.moe_cross_entropy(h, m.MOE_BF16, T, H, w, V, labels, loss, lse, ws, nb, st)
    b.record()
    assert m.moe_check_status(st) == 0
    assert a.elapsed_time(b) > 2100.0  # (longer than a wait's limit)
    # some tokens of every part of the batch, in 64 bits
    some = torch.cat([torch.arange(0, T, T // 60, device=DEV), torch.tensor([T - 1], device=DEV)])
    hs, sums, size = h[some].double(), [], torch.zeros(len(some), device=DEV)
    for i in range(0, V, 1 << 15):
        piece = w[i:i + (1 << 15)]
        sums.append(torch.logsumexp(hs @ piece.double().T, 1))
        size = torch.maximum(size, (hs.float().abs() @ piece.float().abs().T).amax(1))
    want = torch.logsumexp(torch.stack(sums), 0)
    z = (hs * w[labels[some].long()].double()).sum(1)
    # each instruction sums 16 products and the running sum, at most 2^-23 of the magnitudes each; then the exponentials, whose
    # arguments are at most 40, and their sums of 64 + 8 + one per tile
    tol = (H / 16 + 8) * 2.0 ** -23 * size.double() + 2.0 ** -24 * (8 * 40 + 96 + V / 256 + 4 * 60)
    assert ((lse[some].double() - want).abs() <= tol).all()
    assert ((loss[some].double() - (want - z)).abs() <= 2 * tol).all()
