"""The sort asks for a workspace only where it uses one (host side, no GPU needed)."""
import pytest

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B

A = 1 << 20  # an address that no refused call may touch


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


def test_sizes():
    for T, k, E in ((1, 1, 1), (4097, 1, 512), (2048, 16, 1024), (32768, 1, 7)):
        assert m.moe_permute_workspace_size(T, k, E) == 0
    assert m.moe_permute_workspace_size(32769, 1, 7) == 2 * 512  # 17 chunks of 7 counters, twice, in 256-byte pieces
    assert m.moe_permute_workspace_size(3277, 10, 512) == 2 * 17 * 512 * 4


def test_refused_without_one():
    for ws, nb in ((None, 0), (A, 2 * 17 * 512 * 4 - 1), (None, 1 << 20)):
        with pytest.raises(m.MoeError) as e:
            m.moe_permute(A, 3277, 10, 512, A, A, A, ws, nb)
        assert e.value.status == m.MOE_ERR_WORKSPACE and str(2 * 17 * 512 * 4) in str(e.value)
