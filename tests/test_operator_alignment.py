"""Index, weight and status words off their 4 bytes are refused before anything is launched (no GPU needed: the
addresses are made up, and no call may come as far as using them)."""
import pytest

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B

A = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


CALLS = {  # the call with every address in place, and the arguments that may not move
    "dispatch": (lambda p: m.moe_dispatch(A, m.MOE_BF16, 1, 8, 2, 4, p["offsets"], p["inv_perm"], A), ("offsets", "inv_perm")),
    "dispatch_backward": (lambda p: m.moe_dispatch_backward(A, m.MOE_BF16, 1, 8, 2, p["inv_perm"], A), ("inv_perm",)),
    "combine": (lambda p: m.moe_combine(A, m.MOE_BF16, 1, 8, 2, p["w"], p["inv_perm"], A), ("w", "inv_perm")),
    "combine_backward": (lambda p: m.moe_combine_backward(A, A, m.MOE_BF16, 1, 8, 2, 4, p["offsets"], p["w"], p["inv_perm"],
                                                          A, p["dw"]), ("offsets", "w", "inv_perm", "dw")),
    "quantise": (lambda p: m.moe_mx4_quantise(A, m.MOE_BF16, 1, 64, A, A, p["dev_status"]), ("dev_status",)),
    "matmul": (lambda p: m.moe_mx4_matmul(A, A, 1, 8, 64, A, A, 1, p["offsets"], A, dev_status=p["dev_status"]),
               ("offsets", "dev_status")),
}


@pytest.mark.parametrize("call,arg", [(c, a) for c, (_, names) in CALLS.items() for a in names])
@pytest.mark.parametrize("off", [1, 2])
def test_words_off_their_place(call, arg, off):
    fn, names = CALLS[call]
    with pytest.raises(m.MoeError) as e:
        fn({n: A + off if n == arg else A for n in names})
    assert e.value.status == m.MOE_ERR_INVALID_ARG and "aligned" in str(e.value) and arg in str(e.value), str(e.value)
