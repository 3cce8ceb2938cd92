// router_loss_deal.cuh -- how the threads of a CTA share the sums over parts of
// its slice of the experts (router_loss.cu's finish; plain arithmetic, for host
// and device).
#pragma once

namespace moe {
namespace rl {

struct Deal {
    int per, groups;  // threads a row of units, and rows of them: every groups-th part each
    int values;       // the sums of a unit's row: probabilities and counts
    int turns;        // into how many sums the groups' are joined by all threads, where that is done
    bool twice;       // many groups: their sums by all threads, then the threads'
};

// w units of V columns (none, where there are fewer units than CTAs), summed over `parts` parts.
#if defined(__CUDACC__)
__host__ __device__
#endif
constexpr Deal deal(int w, int threads, int parts, int V)
{
    Deal d = {};
    d.per = w < threads ? w : threads;
    if (d.per == 0) {
        d.groups = 1;
        return d;
    }
    d.groups = threads / d.per < parts ? threads / d.per : parts;
    if (d.groups < 1) d.groups = 1;
    d.values = 2 * V * d.per;
    d.turns = threads / d.values;
    d.twice = d.groups >= 16 && d.turns >= 2;
    return d;
}

}  // namespace rl
}  // namespace moe
