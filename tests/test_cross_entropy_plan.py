"""How the cross entropy is cut up, and its workspaces (host arithmetic, no GPU needed)."""
import os
import random
import subprocess

import pytest

import bit_expert_ffn_gb300 as m
from bit_expert_ffn_gb300 import build as B
from conftest import ROOT

SIZES = (m.moe_cross_entropy_workspace_size, m.moe_cross_entropy_backward_workspace_size)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    m.load()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("H,V", [(2048, 32000), (8, 1), (64, 70001), (1056, 8191), (2048, 65536), (4096, 128000), (136, 300), (80, 109558)])
def test_a_workspace_is_enough_for_every_smaller_batch(size, H, V):
    last = 0
    for T in list(range(0, 3000)) + list(range(3000, 40000, 97)) + [1 << 17, 1 << 20]:
        now = size(T, H, V)
        assert now >= last, T
        last = now


def test_sizes_stay_small():
    """What the header says of d, and little beside it for a split into parts."""
    back = SIZES[1]
    for T, H, V in ((4096, 2048, 65536), (8192, 2048, 200_000), (1000, 2048, 32000)):
        assert back(T, H, V) <= (256 << 20) + (1 << 20) + max(64 << 20, (T + 255) // 256 * 256 * H * 4)
    assert back(1, 2048, 1000) <= 65 << 20


PROGRAM = r"""
#include <cstddef>
namespace moe {
inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }
}
#include "cross_entropy_plan.cuh"

#include <cstdio>
#include <cstdlib>

using namespace moe;
using namespace moe::ce;

int main(int argc, char **argv)
{
    for (int i = 1; i + 3 < argc; i += 4) {
        const int T = std::atoi(argv[i]), H = std::atoi(argv[i + 1]), V = std::atoi(argv[i + 2]), sms = std::atoi(argv[i + 3]);
        const Layout l = layout(T, H, V, sms);
        const size_t end = l.sums + (l.pieces > 1 || l.parts > 1 ? align256((size_t)l.parts * l.part_rows * H * 4) : 0);
        const Cut cut = cut_logits(T, V, sms);
        const bool ok = end <= l.total && l.total == layout_bytes(T, H, V) && l.parts >= 1 && l.parts <= MOST_PARTS && l.columns % BN == 0 &&
                        (int64_t)l.columns * l.pieces >= V && (int64_t)l.columns * (l.pieces - 1) < V && l.part_rows >= T &&
                        l.parts <= tiles(std::min(V, l.columns), BK) && align256((size_t)tiles(V, cut.bn) * T * 16) <= stats_bytes(T, V, sms);
        bool all = true;  // every item of both jobs is somebody's
        for (int s = 1; s <= 3; s++) {
            const int64_t a = (int64_t)tiles(T, BN) * s, b = tiles(V, BN), G = std::min<int64_t>(a + b, sms / l.C);
            const Deal d = deal(a, 1 + T % 50, b, 1 + V % 70, G);
            all = all && d.longer == a % G && (int64_t)d.longer * d.long_items + (G - d.longer) * d.short_items >= b;
        }
        if (!ok || !all) {
            std::printf("T=%d H=%d V=%d sms=%d: needs %zu of %zu, columns %d pieces %d parts %d C %d bn %d\n", T, H, V, sms, end, l.total,
                        l.columns, l.pieces, l.parts, l.C, cut.bn);
            return 1;
        }
    }
    return 0;
}
"""


def test_what_a_plan_uses_is_within_its_workspace(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "bit_expert_ffn_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    rng = random.Random(0)
    shapes = [(1 << 24, 8, 1), (1, 1 << 20, 1 << 19), (1 << 20, 1 << 19, 1 << 10), (3660, 80, 109558), (1, 7752, 15728), (2, 64, 65)]
    for _ in range(6000):
        shapes.append((int(2 ** rng.uniform(0, 18)), 8 * int(2 ** rng.uniform(0, 11)), int(2 ** rng.uniform(0, 19))))
    for i in range(0, len(shapes), 500):
        args = [str(x) for k, s in enumerate(shapes[i:i + 500]) for x in (*s, (152, 148, 20)[k % 3])]
        r = subprocess.run([str(exe)] + args, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
