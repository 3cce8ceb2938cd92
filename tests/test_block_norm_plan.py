"""The norm gradient's plan at the largest token counts (host arithmetic, no GPU needed)."""
import pytest

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


@pytest.mark.parametrize("H", [1, 64, 512])
def test_token_counts_up_to_the_largest_int(H):
    """Four rows a CTA: the count of CTAs is the same for all of these, and so is the workspace."""
    want = m.moe_block_norm_backward_workspace_size(1 << 30, H)
    assert 0 < want < 1 << 30
    for T in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 3, 2 ** 31 - 4):
        assert m.moe_block_norm_backward_workspace_size(T, H) == want
