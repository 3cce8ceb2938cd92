// cross_entropy.cu -- moe_cross_entropy: softmax cross entropy of hidden states
// against a head's weights, and its gradients, on the tensor cores, without the
// tokens x vocabulary logits.
//
//   z = h W^T, lse_t = log sum_v exp z_tv, loss_t = lse_t - z_t,label
//   d = exp(z - lse) (dloss + dlse) - onehot dloss
//   dh = d W, dW = d^T h
//
// How they are cut into tiles, pieces and parts is cross_entropy_plan.cuh's.
// Three kinds of product share one kernel:
//   LOSS   z's tiles; each row's maximum and sum of exponentials over the
//          tile's columns leave (8 bytes a warp's half of them), and its label's z
//   GRAD   z's tiles again, for a piece of the vocabulary; d leaves in 16 bits
//   PROD   both gradients of a piece in one launch: dh (K over the piece's
//          columns) and dW (K over the tokens)
// d is divided by the call's largest |dloss| or |dlse| that is finite before its
// rounding (so fp16 holds it, and the usual equal weights leave no rounding of
// their own) and the gradients are multiplied by it.  A weight that is not finite
// so stays in what its token reaches.
//
// d is row-major [T][piece]: for dh it is the A operand as it lies (K inner), for
// dW it is A with M inner, and W and h are B with N inner: the tensor cores take
// both, so nothing is transposed.  A tile is 128 x 256 of one CTA, or 256 x 256 of
// a pair of CTAs whose tensor cores work as one (each loads its 128 rows of A and
// its half of B's columns: two thirds of the shared-memory traffic per product,
// and six steps of K = 64 on their way instead of four).  Operands come by TMA
// (128-byte swizzle), sums lie in two accumulators of 256 columns of tensor memory
// in turn, so that a tile's way out runs under the next tile's products; results
// leave through shared memory by TMA.  Tiles of both jobs of PROD are dealt out so
// that all CTAs end together; dh's long sums are split into parts where they are
// too few for that.
//
// Measured on one GB300 (bf16, H = 2,048): 4,096 tokens against 65,536 words 612
// to 622 us in a long run (1.8 PFLOP/s, power-bound), 523 while the clocks are
// still up (by single CTAs 557); with both gradients 2.57 to 2.64 ms (1.7 PFLOP/s),
// 2.44 at first (by single CTAs 2.61); four tokens against 100,003 words 67 us (410
// MB of W, 6.1 TB/s); 1,111 tokens, H = 1,056, 8,191 words with gradients 71 us.
// Tried without gain: W on its way to L2 in boxes of 512 bytes a row (four tokens,
// 10 us more), results straight from the registers, the next columns loaded from
// tensor memory ahead, four blocks of results on their way instead of two.
//
// Every wait is bounded: after about 2 s the CTA records MOE_ERR_TIMEOUT and
// stops.
#include "cluster.cuh"
#include "common.cuh"
#include "cross_entropy_plan.cuh"
#include "dense_tc.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace moe {
namespace ce {

using tc::elect_one;
using tc::mbar_test;
using tc::uniform;

enum Kind { LOSS, GRAD, PROD };

constexpr int A_BYTES = ROWS * BK * 2;

// A tile is one CTA's (C = 1: 128 rows) or a pair's (C = 2: 256 rows), each with its rows of A and its half of B's columns.
template <int C>
struct Tile {
    static constexpr int BM = ROWS * C, B_BYTES = BN / C * BK * 2, STAGES = C == 1 ? 4 : 6;
};
constexpr int MAX_STAGES = 6;
constexpr int EPI_WARP0 = 2, EPI_WARPS = 8;  // two per quarter of the lanes: every other 32 columns each
constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int OUT_BYTES = 32 * 128;  // a warp's 32 rows of 32 fp32 values on their way out, or two blocks of 16-bit ones in turn
constexpr size_t SMEM = 192 * 1024 + EPI_WARPS * OUT_BYTES + 1024;
constexpr int BAND_ROWS = 4096;  // rows that pass over the columns together
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float FUSED = 1e6f;  // below it x log2 e is rounded by at most 1/16
constexpr float F16_ROOM = 16384.f;  // |d| <= 1 after the division: as fp16, 2^14 times that

struct Job {
    int m_tiles, n_tiles, bn;  // columns of a tile: a multiple of 32, at most BN
    int K, parts;              // the sum's length, and into how many parts it is split
    int mn_a;                  // A with M inner
    int b_y0, out_y0;          // added to B's and the output's row coordinates
    int part_rows;             // rows of the output from one part to the next
    int add, out_f32;
    // Rows of the operands' boxes: as many as there are tokens, where they are few.  (Rows past the end that TMA has to fill
    // with zeros take their time: four tokens against 100,003 x 2,048 82 us with boxes of 128, 69 with boxes of 8.)  Past
    // a box of A with K inner lies what was there: rows of the result that nobody takes.
    int a_rows, b_rows;
};

// Which items a CTA or pair takes: of the first job every G-th (G of them in all), then of the
// second what evens them out: `long_items` each for those with one more of the first,
// `short_items` for the others.
struct Params {
    Job job[2];
    int items0, items1, longer, long_items, short_items;
    uint32_t idesc;     // but for N and the operands' order
    int T, V;           // rows, columns that there are (LOSS: of the vocabulary; GRAD: of the piece)
    int v0, all;        // the piece's first column, columns of the whole vocabulary
    int f16;
    const int32_t *labels;
    float2 *stats;      // [T][n tiles][2]
    float *label_z;
    const float *lse, *dloss, *dlse;
    float *top;         // the largest finite |dloss| or |dlse|, 1 where there is none above zero: written by GRAD, for PROD
    int32_t *status;
};

struct Maps {
    CUtensorMap a[2], b[2], out[2];
};

// What a row of the logits' gradient needs.
struct Row {
    int label;
    float lse, dloss, dlse;
};

struct Shared {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem;
    float top[EPI_WARPS];
    volatile int abort;
};

struct Item {
    int j, m, n, part;  // job, tiles, part of K
    int kb0, kb1;       // steps
};

// The CTA's or pair's i-th item; false when there are no more.  Row tiles first, within bands of BAND: the tiles at work
// share the columns' operand, and a band's rows stay in L2.
template <int C>
__device__ __forceinline__ bool item_of(const Params &p, int i, Item &it)
{
    constexpr int BAND = BAND_ROWS / Tile<C>::BM;
    const int c = blockIdx.x / C, G = gridDim.x / C;
    int t = c + i * G;
    it.j = 0;
    if (t >= p.items0) {
        i -= (p.items0 - c + G - 1) / G;
        const bool more = c < p.longer;  // of the first job
        const int even = min(p.long_items, p.short_items);
        it.j = 1;
        if (i < even) t = i * G + c;
        else if (i < (more ? p.long_items : p.short_items)) t = even * G + (more ? (i - even) * p.longer + c : (i - even) * (G - p.longer) + c - p.longer);
        else return false;
        if (t >= p.items1) return false;
    }
    const Job &g = p.job[it.j];
    it.part = it.kb0 = 0;
    it.kb1 = (g.K + BK - 1) / BK;
    if (g.parts > 1) {  // (quotients take some hundred cycles each, of every warp and tile: only where there is need)
        const uint32_t whole = g.m_tiles * g.n_tiles, nk = it.kb1;
        it.part = (uint32_t)t / whole;
        t -= it.part * whole;
        it.kb0 = nk * it.part / (uint32_t)g.parts;
        it.kb1 = nk * (it.part + 1) / (uint32_t)g.parts;
    }
    int m0 = 0, rows = g.m_tiles;
    if (rows > BAND) {
        const uint32_t band = (uint32_t)t / (uint32_t)(BAND * g.n_tiles);
        m0 = band * BAND;
        rows = min(BAND, g.m_tiles - m0);
        t -= m0 * g.n_tiles;
    }
    it.n = (uint32_t)t / (uint32_t)rows;
    it.m = m0 + t - it.n * rows;
    return true;
}

__device__ __forceinline__ bool warp_wait(Shared &S, uint64_t *bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    const bool ok = tc::mbar_wait(bar, parity, kWaitNs);
    return __all_sync(0xffffffffu, ok && !S.abort);
}

// The shared-memory address of the pair's first CTA that corresponds to this CTA's.
__device__ __forceinline__ uint32_t leaders(const void *p)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(tc::smem_u32(p)));
    return a;
}

// Arrive on the first CTA's barrier, and its wait for both CTAs' arrivals.
template <int C>
__device__ __forceinline__ void arrive_leader(uint64_t *bar)
{
    if (C == 1) return tc::mbar_arrive(bar);
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leaders(bar)) : "memory");
}

__device__ __forceinline__ bool cluster_try_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool warp_wait_pair(Shared &S, uint64_t *bar, uint32_t parity)
{
    bool ok = cluster_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    const unsigned long long t0 = tc::now_ns();
    while (!ok && tc::now_ns() - t0 <= kWaitNs) ok = cluster_try_wait(bar, parity);
    return __all_sync(0xffffffffu, ok && !S.abort);
}

// A box into this CTA's shared memory, its bytes counted by the first CTA's barrier.
template <int C>
__device__ __forceinline__ void load(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar, uint32_t leader_bar)
{
    if (C == 1) return tc::tma_load_2d(dst, map, x, y, bar);
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader_bar)
        : "memory");
}

// D[tmem] (+)= A B^T; a pair's, each CTA's part of the operands at the same places of its shared memory.
template <int C>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (C == 1) return tc::mma_f16_ss(d, a, b, idesc, accumulate);
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the CTA's or both CTAs' barriers once the MMAs issued so far are done.
template <int C>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if (C == 1) return tc::mma_commit(bar);
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     tc::smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

// Descriptor of an operand with M or N inner, 128-byte swizzle: 64 elements (128 bytes) a row, eight K rows
// (1,024 bytes) an atom; the next atom of K follows, the next 64 elements of M or N come a whole step (8 KB) on.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t smem_addr)
{
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | (uint64_t)(BK * 128 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int f16)
{
    uint32_t w;
    if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

__device__ __forceinline__ void tma_add_2d(const CUtensorMap *map, int x, int y, const void *src)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(tc::smem_u32(src))
                 : "memory");
}

// A lane's row of 32 fp32 (128 bytes) or 16-bit (64 bytes) values into the warp's block, swizzled as TMA expects it.
__device__ __forceinline__ void put_row(char *buf, int lane, const uint32_t (&w)[32], bool f32)
{
    if (f32) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            *reinterpret_cast<uint4 *>(buf + lane * 128 + ((j ^ (lane & 7)) * 16)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            *reinterpret_cast<uint4 *>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
}

// All threads of the CTA or pair.
template <int C>
__device__ __forceinline__ void tile_sync()
{
    if (C == 1) __syncthreads();
    else cluster_sync();
}

template <Kind K, int C>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps)
{
    using Z = Tile<C>;
    constexpr int BM = Z::BM, STAGES = Z::STAGES, B_BYTES = Z::B_BYTES;
    extern __shared__ __align__(1024) char dyn_raw[];
    char *dyn = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    char *sA = dyn, *sB = sA + STAGES * A_BYTES, *sO = sB + STAGES * B_BYTES;
    __shared__ Shared S;
    const int warp = uniform(warp_id()), lane = lane_id();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            tc::mbar_init(&S.full[s], 1);
            tc::mbar_init(&S.empty[s], 1);
        }
        for (int i = 0; i < 2; i++) {
            tc::mbar_init(&S.acc_full[i], 1);
            tc::mbar_init(&S.acc_empty[i], C * EPI_WARPS);  // both CTAs'; the first one's barrier is the one waited for
        }
        tc::mbar_init(&S.mma_done, 1);
        S.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == EPI_WARP0 && C == 1) tc::tmem_alloc(&S.tmem, 512);
    if (warp == EPI_WARP0 && C == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(&S.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    // (launched while the kernel before it may still run, and lets the next one come as soon: nothing above reads what that one writes)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::tc_fence_before();
    tile_sync<C>();  // both CTAs' barriers are there
    tc::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)S.tmem);
    const int rank = C == 1 ? 0 : uniform((int)cluster_rank());

    if (warp == 0) {
        // ---------------- operands
        int it = 0, s = 0;
        uint32_t phase = 1;
        bool ok = true;
        Item m;
        for (int i = 0; ok && item_of<C>(p, i, m); i++) {
            const Job &g = p.job[m.j];
            const int half = g.bn / C, boxes = (half + 63) / 64;
            const uint32_t bytes = (K == PROD && g.mn_a ? ROWS / 64 : 1) * g.a_rows * 128 + (K == PROD ? boxes * g.b_rows : half) * 128;
            for (int kb = m.kb0; kb < m.kb1; kb++, it++) {
                if (it >= STAGES) ok = warp_wait(S, &S.empty[s], phase);
                if (!ok) break;
                if (elect_one()) {
                    if (rank == 0) tc::mbar_arrive_expect_tx(&S.full[s], C * bytes);
                    uint64_t *own = &S.full[s];
                    const uint32_t bar = C == 1 ? 0 : leaders(own);
                    char *a = sA + s * A_BYTES, *b = sB + s * B_BYTES;
                    if (K == PROD && g.mn_a) {
#pragma unroll
                        for (int h = 0; h < ROWS / 64; h++)
                            load<C>(a + h * BK * 128, &maps.a[m.j], m.m * BM + rank * ROWS + h * 64, kb * BK, own, bar);
                    } else {
                        load<C>(a, &maps.a[m.j], kb * BK, m.m * BM + rank * ROWS, own, bar);
                    }
                    if (K == PROD) {
                        for (int h = 0; h < boxes; h++)
                            load<C>(b + h * BK * 128, &maps.b[m.j], m.n * g.bn + rank * half + h * 64, g.b_y0 + kb * BK, own, bar);
                    } else {
                        load<C>(b, &maps.b[m.j], kb * BK, g.b_y0 + m.n * g.bn + rank * half, own, bar);
                    }
                }
                if (++s == STAGES) s = 0, phase ^= 1;
            }
        }
        if (lane == 0) {
            if (!ok) {
                set_status(p.status, MOE_ERR_TIMEOUT);
                S.abort = 1;
            }
            // no copy, and no arrival from the products, may still be on its way when the pair leaves: every stage's last
            // use is over (after a stop: every copy has landed, in the first CTA's count of both CTAs')
            for (int i = 0; i < STAGES && i < it; i++) {
                const int u = (it - 1 - i) / STAGES, at = (it - 1 - i) % STAGES;
                bool over = true;
                if (ok && !S.abort) over = tc::mbar_wait(&S.empty[at], u & 1, kWaitNs);
                else if (rank == 0) over = tc::mbar_wait(&S.full[at], u & 1, kWaitNs / 100);
                if (!over) {
                    set_status(p.status, MOE_ERR_TIMEOUT);
                    S.abort = 1;
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA, by the pair's first CTA
        int j = 0, s = 0;
        uint32_t phase = 0;
        bool ok = true;
        Item m;
        for (int i = 0; rank == 0 && ok && item_of<C>(p, i, m); i++) {
            const Job &g = p.job[m.j];
            if (m.kb0 == m.kb1) continue;  // a part of nothing
            const int acc = j & 1, v = j >> 1;
            j++;
            if (v > 0) ok = (C == 1 ? warp_wait : warp_wait_pair)(S, &S.acc_empty[acc], (v - 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(acc * BN);
            const uint32_t idesc = p.idesc | (uint32_t)(g.bn >> 3) << 17 | (K == PROD ? (uint32_t)g.mn_a << 15 | 1u << 16 : 0u);
            bool ready = mbar_test(&S.full[s], phase);
            for (int kb = m.kb0; kb < m.kb1; kb++) {
                if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(S, &S.full[s], phase);
                if (!ok) break;
                tc::tc_fence_after();
                const int sn = s + 1 == STAGES ? 0 : s + 1;
                const uint32_t phase_n = sn ? phase : phase ^ 1;
                ready = mbar_test(&S.full[sn], phase_n);
                if (elect_one()) {
                    const uint32_t a = tc::smem_u32(sA + s * A_BYTES), b = tc::smem_u32(sB + s * B_BYTES);
                    const bool ma = K == PROD && g.mn_a;
                    const uint64_t da = ma ? desc_mnmajor_sw128(a) : tc::desc_kmajor_sw128(a);
                    const uint64_t db = K == PROD ? desc_mnmajor_sw128(b) : tc::desc_kmajor_sw128(b);
                    // K = 16 an instruction: 32 bytes of a row, or 16 rows of 128 bytes
                    const uint64_t ka = ma ? 128 : 2, kbs = K == PROD ? 128 : 2;
                    const int left = K == PROD ? g.K - kb * BK : BK;  // (d's columns past K's last sixteen may never have been written)
#pragma unroll
                    for (int k = 0; k < BK / 16; k++)
                        if (k * 16 < left) mma<C>(d, da + k * ka, db + k * kbs, idesc, (kb > m.kb0 || k > 0) ? 1u : 0u);
                    commit<C>(&S.empty[s]);
                    if (kb + 1 == m.kb1) commit<C>(&S.acc_full[acc]);
                }
                s = sn;
                phase = phase_n;
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, MOE_ERR_TIMEOUT);
            S.abort = 1;
        }
        if (rank == 0 && elect_one()) commit<C>(&S.mma_done);
        if (rank == 0 && !tc::mbar_wait(&S.mma_done, 0, kWaitNs) && lane == 0) set_status(p.status, MOE_ERR_TIMEOUT);
    } else {
        // ---------------- sums out
        const int q = warp & 3, side = (warp - EPI_WARP0) >> 2;
        char *out = sO + (warp - EPI_WARP0) * OUT_BYTES;
        int j = 0, turn = 0;
        bool was32 = false;
        // the largest finite |dloss| or |dlse| of the tokens that count, by every CTA for itself, under its first tile's products
        float top = K == PROD ? *p.top : 0.f;
        auto finite = [](float x, bool there) { return there && fabsf(x) < INFINITY ? fabsf(x) : 0.f; };
        if (K == GRAD) {
            // (all loads of a turn before the first use, and none that waits for a label)
            constexpr int AT_ONCE = 8, STEP = EPI_WARPS * 32;
            for (int t0 = threadIdx.x - EPI_WARP0 * 32; t0 < p.T; t0 += AT_ONCE * STEP) {
                int label[AT_ONCE];
                float b[AT_ONCE], e[AT_ONCE];
#pragma unroll
                for (int i = 0; i < AT_ONCE; i++) {
                    const int t = t0 + i * STEP;
                    label[i] = t < p.T ? p.labels[t] : -1;
                    b[i] = t < p.T ? p.dloss[t] : 0.f;
                    e[i] = t < p.T && p.dlse ? p.dlse[t] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < AT_ONCE; i++)
                    top = fmaxf(top, fmaxf(finite(b[i], label[i] >= 0 && label[i] < p.all), finite(e[i], true)));
            }
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            if (lane == 0) S.top[warp - EPI_WARP0] = top;
            tc::named_sync(1, EPI_WARPS * 32);
#pragma unroll
            for (int w = 0; w < EPI_WARPS; w++) top = fmaxf(top, S.top[w]);
            if (top == 0.f) top = 1.f;
            if (blockIdx.x == 0 && threadIdx.x == EPI_WARP0 * 32) *p.top = top;
        }
        const float up = K == PROD ? (p.f16 ? top / F16_ROOM : top) : 0.f;
        const float down = p.f16 ? F16_ROOM : 1.f;
        // what a row needs comes while the tile before is on its way out
        Item m, next;
        Row in = {}, ahead = {};
        auto row_of = [&](const Item &m) { return m.m * BM + rank * ROWS + q * 32 + lane; };
        auto fetch = [&](const Item &m, Row &r) {
            const int row = row_of(m);
            r.label = -1;
            if (K == PROD || row >= p.T) return;
            r.label = p.labels[row];
            if (K == GRAD) {
                r.lse = p.lse[row];
                r.dloss = p.dloss[row];
                if (p.dlse) r.dlse = p.dlse[row];
            }
        };
        bool more = item_of<C>(p, 0, m);
        if (more) fetch(m, in);
        for (int i = 1; more; i++, m = next, in = ahead) {
            more = item_of<C>(p, i, next);
            if (more) fetch(next, ahead);
            const Job &g = p.job[m.j];
            if (m.kb0 == m.kb1) continue;
            const int acc = j & 1, v = j >> 1;
            j++;
            const int row = row_of(m), n0 = m.n * g.bn;
            int label = in.label;
            float lse = 0.f, nl = 0.f, a = 0.f, b = 0.f;
            if (K == GRAD && row < p.T) {
                const bool there = label >= 0 && label < p.all;
                b = there ? in.dloss : 0.f;
                a = b + (p.dlse ? in.dlse : 0.f);
                a = a / top * down;
                b = b / top * down;
                lse = in.lse;
                nl = -lse * LOG2E;
                if (fabsf(lse) < FUSED) a *= ex2(-fmaf(lse, LOG2E, nl));  // (what the product's rounding left out)
                label -= p.v0;
            }
            if (!warp_wait(S, &S.acc_full[acc], v & 1)) {
                if (lane == 0) set_status(p.status, MOE_ERR_TIMEOUT);
                S.abort = 1;
                break;
            }
            tc::tc_fence_after();
            const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
            if (K == LOSS) {
                float mx = -INFINITY, sum = 0.f, zl = 0.f;
                bool mine = false;
#pragma unroll 1
                for (int c = side * 32; c < g.bn; c += 64) {
                    const int left = p.V - n0 - c;
                    if (left <= 0) break;
                    uint32_t r[32];
                    __syncwarp();
                    tc::tmem_ld_32x32b_x32(tbase + c, r);
                    tc::tmem_ld_wait();
                    if (left < 32) {
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            if (i >= left) r[i] = 0xff800000u;
                    }
                    const int at = label - n0 - c;
                    if ((unsigned)at < 32u) {
                        mine = at < left;
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            if (i == at) zl = __uint_as_float(r[i]);
                    }
                    float cm = mx;
#pragma unroll
                    for (int i = 0; i < 32; i++) cm = fmaxf(cm, __uint_as_float(r[i]));
                    const float ref = cm == -INFINITY ? 0.f : cm;
                    float t[4] = {0.f, 0.f, 0.f, 0.f}, right = 1.f;
                    if (fabsf(ref) < FUSED) {  // exponents as products and sums in one; the maximum's rounding put right after
                        const float off = ref * LOG2E;
                        right = ex2(-fmaf(ref, LOG2E, -off));
#pragma unroll
                        for (int i = 0; i < 32; i++) t[i & 3] += ex2(fmaf(__uint_as_float(r[i]), LOG2E, -off));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i++) t[i & 3] += ex2((__uint_as_float(r[i]) - ref) * LOG2E);
                    }
                    sum = fmaf((t[0] + t[1]) + (t[2] + t[3]), right, sum * ex2((mx - ref) * LOG2E));
                    mx = cm;
                }
                if (row < p.T) {
                    p.stats[((int64_t)row * g.n_tiles + m.n) * 2 + side] = make_float2(mx, sum);
                    if (mine) p.label_z[row] = zl;
                }
            } else {
#pragma unroll 1
                for (int c = side * 32; c < g.bn; c += 64) {
                    uint32_t r[32];
                    __syncwarp();
                    tc::tmem_ld_32x32b_x32(tbase + c, r);
                    tc::tmem_ld_wait();
                    const bool f32 = K == PROD && g.out_f32;
                    if (K == GRAD) {
                        const int left = p.V - n0 - c, at = label - n0 - c;
                        if (!(fabsf(lse) < FUSED)) {
#pragma unroll
                            for (int i = 0; i < 32; i++) r[i] = __float_as_uint(ex2((__uint_as_float(r[i]) - lse) * LOG2E) * a);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i++) r[i] = __float_as_uint(ex2(fmaf(__uint_as_float(r[i]), LOG2E, nl)) * a);
                        }
                        if ((unsigned)at < 32u) {
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                if (i == at) r[i] = __float_as_uint(__uint_as_float(r[i]) - b);
                        }
                        if (left < 32 || (a == 0.f && b == 0.f)) {  // past the vocabulary; a token that takes no part, whatever its logits
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                if (i >= left || (a == 0.f && b == 0.f)) r[i] = 0;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__uint_as_float(r[i]) * up);
                    }
                    if (!f32) {
#pragma unroll
                        for (int i = 0; i < 16; i++) r[i] = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), p.f16);
                    }
                    char *buf = out + (f32 ? 0 : (turn & 1) * (OUT_BYTES / 2));
                    turn++;
                    if (lane == 0) {
                        if (K == PROD && (f32 || was32)) tc::bulk_wait_read<0>();
                        else tc::bulk_wait_read<1>();
                    }
                    was32 = f32;
                    __syncwarp();
                    put_row(buf, lane, r, f32);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int x = n0 + c, y = g.out_y0 + m.part * g.part_rows + m.m * BM + rank * ROWS + q * 32;
                        if (K == PROD && g.add) tma_add_2d(&maps.out[m.j], x, y, buf);
                        else tc::tma_store_2d(&maps.out[m.j], x, y, buf);
                        tc::bulk_commit();
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<C>(&S.acc_empty[acc]);
        }
        if (K != LOSS && lane == 0) tc::bulk_wait_all();
        // the pair's second CTA issues no products: its wait for their end, and with it the limit, begins where its last tile is out
        if (rank == 1 && warp == EPI_WARP0 && !tc::mbar_wait(&S.mma_done, 0, kWaitNs) && lane == 0) set_status(p.status, MOE_ERR_TIMEOUT);
    }
    tc::tc_fence_before();
    tile_sync<C>();  // neither CTA leaves while the other's products read its operands or write its sums
    if (warp == EPI_WARP0) {
        tc::tc_fence_after();
        if (C == 1) tc::tmem_dealloc(tmem, 512);
        else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// lse and loss from the tiles' maxima and sums: a warp per token.
constexpr int COMBINE_WARPS = 8;

__global__ void __launch_bounds__(COMBINE_WARPS * 32) combine_kernel(const float2 *stats, const float *label_z, const int32_t *labels,
                                                                     int T, int V, int tiles, float *loss, float *lse, int32_t *status)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = blockIdx.x * COMBINE_WARPS + warp_id(), lane = lane_id();
    if (t >= T) return;
    const float2 *row = stats + (int64_t)t * tiles;
    float m = -INFINITY, s = 0.f;
    for (int i = lane; i < tiles; i += 256) {  // eight a lane at once
        float2 v[8];
        float top = m;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            v[j] = i + 32 * j < tiles ? row[i + 32 * j] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) top = fmaxf(top, v[j].x);
        const float off = top == -INFINITY ? 0.f : top;
        s *= ex2((m - off) * LOG2E);
#pragma unroll
        for (int j = 0; j < 8; j++) s = fmaf(v[j].y, ex2((v[j].x - off) * LOG2E), s);
        m = top;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        const float top = fmaxf(m, m2), off = top == -INFINITY ? 0.f : top;
        // (the smaller lane's term first, so that both lanes have the same sum)
        const float a = s * ex2((m - off) * LOG2E), b = s2 * ex2((m2 - off) * LOG2E);
        s = lane & o ? b + a : a + b;
        m = top;
    }
    if (lane != 0) return;
    const int label = labels[t];
    const float l = logf(s);
    lse[t] = m + l;
    if (label >= V) set_status(status, MOE_ERR_BOUNDS);
    // (the differences first: a label that is nearly certain leaves a small loss; s may round to just below 1)
    const float v = label < 0 || label >= V ? 0.f : (m - label_z[t]) + l;
    loss[t] = v < 0.f ? 0.f : v;
}

// The parts' fp32 sums, in order, to 16 bits, eight values at a time (a part's n values are a multiple of eight).
template <class A>
__global__ void __launch_bounds__(256) round_kernel(const float *in, int parts, int64_t part, typename A::T *out, int64_t n)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
        float v[8];
        F32::load4(in + i, v);
        F32::load4(in + i + 4, v + 4);
#pragma unroll 4
        for (int s = 1; s < parts; s++) {
            float u[8];
            F32::load4(in + s * part + i, u);
            F32::load4(in + s * part + i + 4, u + 4);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] += u[j];
        }
        A::store8(out + i, v);
    }
}

static moe_status check(int T, int H, int V)
{
    MOE_REQUIRE(T >= 0 && T <= (1 << 24), "T must be in [0, 2^24] (got %d)", T);
    MOE_REQUIRE(H >= 8 && H % 8 == 0 && H <= (1 << 20), "H must be a multiple of 8 in [8, 2^20] (got %d)", H);
    MOE_REQUIRE(V >= 1 && V <= (1 << 24), "V must be in [1, 2^24] (got %d)", V);
    MOE_REQUIRE((int64_t)tiles(T, ROWS) * tiles(V, BN / 2) < (1 << 30) && (int64_t)std::max(T, V) * H < (1ll << 40),
                "too many tiles (T=%d H=%d V=%d)", T, H, V);
    return MOE_OK;
}

static moe_status check_types(const void *h, moe_dtype dtype, int T, int H, const void *w, int V, const int32_t *labels, int32_t *status)
{
    MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "dtype must be MOE_BF16 or MOE_F16 (got %d)", (int)dtype);
    moe_status st = check(T, H, V);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(T == 0 || (h && w && labels), "NULL pointer");
    MOE_REQUIRE(aligned16(h) && aligned16(w), "h and w must be 16-byte aligned");
    MOE_REQUIRE(aligned_to(labels, 4) && aligned_to(status, 4), "labels and dev_status must be 4-byte aligned");
    return MOE_OK;
}

template <class F, class... A>
moe_status launch(const char *what, F kernel, int cluster, int grid, int threads, size_t smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];  // the set-up overlaps the end of the kernel before
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    return check_launch(what);
}

template <Kind K, int C>
moe_status product(Params &p, const Maps &maps, cudaStream_t s)
{
    auto items = [](const Job &g) { return g.m_tiles * g.n_tiles * g.parts; };
    p.items0 = items(p.job[0]);
    p.items1 = items(p.job[1]);
    const int at_once = (int)std::min<int64_t>((int64_t)p.items0 + p.items1, sm_count() / C);
    const Deal d = deal(p.items0, tiles(tiles(p.job[0].K, BK), p.job[0].parts), p.items1, tiles(p.job[1].K, BK), at_once);
    p.longer = d.longer, p.long_items = d.long_items, p.short_items = d.short_items;
    MOE_CUDA_TRY(cudaFuncSetAttribute(product_kernel<K, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM));
    return launch("cross_entropy", product_kernel<K, C>, C, C * at_once, THREADS, SMEM, s, p, maps);
}

template <Kind K>
moe_status product(int C, Params &p, const Maps &maps, cudaStream_t s)
{
    return C == 1 ? product<K, 1>(p, maps, s) : product<K, 2>(p, maps, s);
}

static CUtensorMapDataType map_type(moe_dtype t)
{
    return t == MOE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : t == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

}  // namespace ce
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_cross_entropy_workspace_size(int T, int H, int V, size_t *bytes)
{
    using namespace ce;
    MOE_REQUIRE(bytes, "bytes must not be NULL");
    moe_status st = check(T, H, V);
    if (st != MOE_OK) return st;
    *bytes = align256((size_t)T * 4) + stats_bytes(T, V, sm_count());
    return MOE_OK;
}

extern "C" moe_status moe_cross_entropy(const void *h, moe_dtype dtype, int T, int H, const void *w, int V,
                                        const int32_t *labels, float *loss, float *lse, void *ws, size_t ws_bytes,
                                        int32_t *dev_status, moe_stream_t stream)
{
    using namespace ce;
    moe_status st = check_types(h, dtype, T, H, w, V, labels, dev_status);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(loss && lse, "NULL pointer");
    MOE_REQUIRE(aligned_to(loss, 4) && aligned_to(lse, 4), "loss and lse must be 4-byte aligned");
    size_t need = 0;
    st = moe_cross_entropy_workspace_size(T, H, V, &need);
    if (st != MOE_OK) return st;
    if (ws_bytes < need || !ws)
        return fail(MOE_ERR_WORKSPACE, "moe_cross_entropy needs %zu bytes of workspace (got %zu)", need, ws ? ws_bytes : (size_t)0);
    MOE_REQUIRE(aligned16(ws), "ws must be 16-byte aligned");
    Params p = {};
    Maps maps = {};
    const Cut cut = cut_logits(T, V, sm_count());
    const int n_tiles = tiles(V, cut.bn);
    p.job[0] = {tiles(T, ROWS * cut.C), n_tiles, cut.bn, H, 1, 0, 0, 0, 0, 0, 0, box_rows(T, cut.C), 0};
    p.idesc = tc::idesc_f16_f32(ROWS * cut.C, 0, dtype == MOE_BF16);
    p.T = T, p.V = V, p.labels = labels, p.status = dev_status;
    p.label_z = static_cast<float *>(ws);
    p.stats = reinterpret_cast<float2 *>(static_cast<char *>(ws) + align256((size_t)T * 4));
    st = make_tmap_2d(&maps.a[0], h, map_type(dtype), 2, T, H, BK, box_rows(T, cut.C));
    if (st == MOE_OK) st = make_tmap_2d(&maps.b[0], w, map_type(dtype), 2, V, H, BK, cut.bn / cut.C);
    if (st != MOE_OK) return st;
    const cudaStream_t s = to_cuda(stream);
    st = product<LOSS>(cut.C, p, maps, s);
    if (st != MOE_OK) return st;
    return launch("cross_entropy_combine", combine_kernel, 1, tiles(T, COMBINE_WARPS), COMBINE_WARPS * 32, 0, s, p.stats, p.label_z, labels, T,
                  V, 2 * n_tiles, loss, lse, dev_status);
}

extern "C" moe_status moe_cross_entropy_backward_workspace_size(int T, int H, int V, size_t *bytes)
{
    using namespace ce;
    MOE_REQUIRE(bytes, "bytes must not be NULL");
    moe_status st = check(T, H, V);
    if (st != MOE_OK) return st;
    *bytes = T ? layout_bytes(T, H, V) : 0;
    return MOE_OK;
}

extern "C" moe_status moe_cross_entropy_backward(const void *h, moe_dtype dtype, int T, int H, const void *w, int V,
                                                 const int32_t *labels, const float *lse, const float *dloss,
                                                 const float *dlse, void *dh, void *dw, moe_dtype dw_dtype, int accumulate,
                                                 void *ws, size_t ws_bytes, int32_t *dev_status, moe_stream_t stream)
{
    using namespace ce;
    moe_status st = check_types(h, dtype, T, H, w, V, labels, dev_status);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(!dw || dw_dtype == dtype || dw_dtype == MOE_F32, "dw_dtype must be dtype or MOE_F32 (got %d)", (int)dw_dtype);
    MOE_REQUIRE(!dw || !accumulate || dw_dtype == MOE_F32, "dw is accumulated in MOE_F32 only");
    MOE_REQUIRE(aligned16(dh) && aligned16(dw), "dh and dw must be 16-byte aligned");
    const cudaStream_t s = to_cuda(stream);
    if (T == 0) {
        if (dw && !accumulate) MOE_CUDA_TRY(cudaMemsetAsync(dw, 0, (size_t)V * H * dtype_bytes(dw_dtype), s));
        return MOE_OK;
    }
    if (!dh && !dw) return MOE_OK;
    MOE_REQUIRE(lse && dloss, "NULL pointer");
    MOE_REQUIRE(aligned_to(lse, 4) && aligned_to(dloss, 4) && aligned_to(dlse, 4), "lse, dloss and dlse must be 4-byte aligned");
    const Layout l = layout(T, H, V, sm_count());
    if (ws_bytes < l.total || !ws)
        return fail(MOE_ERR_WORKSPACE, "moe_cross_entropy_backward needs %zu bytes of workspace (got %zu)", l.total,
                    ws ? ws_bytes : (size_t)0);
    MOE_REQUIRE(aligned16(ws), "ws must be 16-byte aligned");
    char *base = static_cast<char *>(ws);
    float *top = reinterpret_cast<float *>(base), *sums = reinterpret_cast<float *>(base + l.sums);
    void *d = base + l.d;

    Params gp = {}, pp = {};
    Maps gm = {}, pm = {};
    const int f16 = dtype == MOE_F16;
    const Cut cut = cut_logits(T, std::min(V, l.columns), sm_count());  // (of every piece)
    gp.idesc = tc::idesc_f16_f32(ROWS * cut.C, 0, !f16);
    pp.idesc = tc::idesc_f16_f32(ROWS * l.C, 0, !f16);
    gp.T = T, gp.all = V, gp.labels = labels, gp.lse = lse, gp.dloss = dloss, gp.dlse = dlse, gp.top = pp.top = top;
    gp.status = pp.status = dev_status;
    gp.f16 = pp.f16 = f16;
    const bool direct = l.pieces == 1 && l.parts == 1;  // dh leaves as it is: no sums of pieces or parts
    const int k_rows = std::min(BK, round_up(T, 16));   // of a step over the tokens
    const auto half = CU_TENSOR_MAP_SWIZZLE_64B;        // boxes of 32 16-bit columns
    st = make_tmap_2d(&gm.a[0], h, map_type(dtype), 2, T, H, BK, box_rows(T, cut.C));
    if (st == MOE_OK) st = make_tmap_2d(&gm.b[0], w, map_type(dtype), 2, V, H, BK, cut.bn / cut.C);
    if (st == MOE_OK) st = make_tmap_2d(&gm.out[0], d, map_type(dtype), 2, T, l.columns, 32, 32, half);
    CUtensorMap d_k, d_m, w_n, h_n, out_h, out_w;
    if (st == MOE_OK) st = make_tmap_2d(&d_k, d, map_type(dtype), 2, T, l.columns, BK, box_rows(T, l.C));
    if (st == MOE_OK) st = make_tmap_2d(&d_m, d, map_type(dtype), 2, T, l.columns, 64, k_rows);
    if (st == MOE_OK) st = make_tmap_2d(&w_n, w, map_type(dtype), 2, V, H, 64, BK);
    if (st == MOE_OK) st = make_tmap_2d(&h_n, h, map_type(dtype), 2, T, H, 64, k_rows);
    if (st == MOE_OK && dh)
        st = direct ? make_tmap_2d(&out_h, dh, map_type(dtype), 2, T, H, 32, 32, half)
                    : make_tmap_2d(&out_h, sums, map_type(MOE_F32), 4, l.parts * l.part_rows, H, 32, 32);
    if (st == MOE_OK && dw)
        st = dw_dtype == MOE_F32 ? make_tmap_2d(&out_w, dw, map_type(MOE_F32), 4, V, H, 32, 32)
                                 : make_tmap_2d(&out_w, dw, map_type(dtype), 2, V, H, 32, 32, half);
    if (st != MOE_OK) return st;
    const int nt = tiles(H, BN), bn = tile_columns(H);
    for (int i = 0; i < l.pieces; i++) {
        const int v0 = i * l.columns, n = std::min(l.columns, V - v0);
        gp.v0 = v0;
        gp.V = n;
        gp.job[0] = {tiles(T, ROWS * cut.C), tiles(n, cut.bn), cut.bn, H, 1, 0, v0, 0, 0, 0, 0, box_rows(T, cut.C), 0};
        st = product<GRAD>(cut.C, gp, gm, s);
        if (st != MOE_OK) return st;
        int j = 0;
        if (dh) {
            pp.job[j] = {tiles(T, ROWS * l.C), nt, bn, n, l.parts, 0, v0, 0, (int)l.part_rows, !direct && i > 0, !direct, box_rows(T, l.C), BK};
            pm.a[j] = d_k, pm.b[j] = w_n, pm.out[j] = out_h;
            j++;
        }
        if (dw) {
            pp.job[j] = {tiles(n, ROWS * l.C), nt, bn, T, 1, 1, 0, v0, 0, accumulate != 0, dw_dtype == MOE_F32, k_rows, k_rows};
            pm.a[j] = d_m, pm.b[j] = h_n, pm.out[j] = out_w;
            j++;
        }
        st = product<PROD>(l.C, pp, pm, s);
        if (st != MOE_OK) return st;
    }
    if (dh && !direct) {
        const int64_t n = (int64_t)T * H;
        const int grid = (int)std::min<int64_t>((n + 2047) / 2048, (int64_t)sm_count() * 8);
        return f16 ? launch("cross_entropy_round", round_kernel<Fp16>, 1, grid, 256, 0, s, sums, l.parts, l.part_rows * H, static_cast<uint16_t *>(dh), n)
                   : launch("cross_entropy_round", round_kernel<Bf16>, 1, grid, 256, 0, s, sums, l.parts, l.part_rows * H, static_cast<uint16_t *>(dh), n);
    }
    return MOE_OK;
}
