"""How the router loss's last sums are shared out (host arithmetic, no GPU needed)."""
import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>

#include "router_loss_deal.cuh"

using moe::rl::Deal;
using moe::rl::deal;

// (a division by zero is no constant)
static_assert(deal(0, 384, 8, 1).per == 0 && deal(0, 384, 8, 1).groups == 1 && !deal(0, 1024, 304, 4).twice, "a CTA without columns");

int main()
{
    const int threads[] = {384, 1024}, clusters[] = {1, 2, 4, 8}, all[] = {1, 2, 4, 8, 33, 304};
    for (int T : threads)
        for (int V = 1; V <= 4; V += 3)
            for (int C : clusters)
                for (int parts : all)
                    for (int E = 1; E <= 1024; E++) {
                        if (E % V) continue;
                        int units = E / V, seen = 0;
                        for (int r = 0; r < C; r++) {
                            const int w = units * (r + 1) / C - units * r / C;
                            const Deal d = deal(w, T, parts, V);
                            seen += w;
                            const bool none = w == 0 && d.per == 0 && !d.twice;
                            const bool some = w > 0 && d.per == (w < T ? w : T) && d.groups >= 1 && d.groups <= parts &&
                                              d.per * d.groups <= T && (!d.twice || (d.turns >= 2 && d.turns * d.values <= T));
                            if (!none && !some) {
                                std::printf("T=%d V=%d C=%d parts=%d E=%d r=%d\n", T, V, C, parts, E, r);
                                return 1;
                            }
                        }
                        if (seen != units) return 2;
                    }
    return 0;
}
"""


def test_every_slice_of_every_cluster(tmp_path):
    src, exe = tmp_path / "deal.cpp", tmp_path / "deal"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "bit_expert_ffn_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
