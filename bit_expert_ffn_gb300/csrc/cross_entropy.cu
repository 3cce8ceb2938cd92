// cross_entropy.cu -- moe_cross_entropy: softmax cross entropy of hidden states
// against a head's weights, and its gradients, on the tensor cores, without the
// tokens x vocabulary logits.
//
//   z = h W^T, lse_t = log sum_v exp z_tv, loss_t = lse_t - z_t,label
//   d = exp(z - lse) (dloss + dlse) - onehot dloss
//   dh = d W, dW = d^T h
//
// Three kinds of product share one kernel (128 x 256 tiles, K in steps of 64):
//   LOSS   z's tiles; each row's maximum and sum of exponentials over the
//          tile's 256 columns leave (8 bytes instead of 1 KB), and its label's z
//   GRAD   z's tiles again, for a piece of the vocabulary; d leaves in 16 bits
//   PROD   both gradients of a piece in one launch: dh (K over the piece's
//          columns) and dW (K over the tokens)
// d is divided by the call's largest |dloss| or |dlse| before its rounding (so
// fp16 holds it, and the usual equal weights leave no rounding of their own) and
// the gradients are multiplied by it.
//
// d is row-major [T][piece]: for dh it is the A operand as it lies (K inner), for
// dW it is A with M inner, and W and h are B with N inner: the tensor cores take
// both, so nothing is transposed.  Operands come by TMA (128-byte swizzle), sums
// lie in two accumulators of 256 columns of tensor memory in turn, so that a
// tile's epilogue runs under the next tile's products; results leave through
// shared memory by TMA.
//
// Every wait is bounded: after about 2 s the CTA records MOE_ERR_TIMEOUT and
// stops.
#include "dense_tc.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace moe {
namespace ce {

using tc::elect_one;
using tc::mbar_test;
using tc::uniform;

enum Kind { LOSS, GRAD, PROD };

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
constexpr int STAGES = 4;
constexpr int EPI_WARP0 = 2, EPI_WARPS = 4;
constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int OUT_BYTES = 32 * 128;  // a warp's 32 rows of 32 values on their way out, two in turn
constexpr size_t SMEM = STAGES * (A_BYTES + B_BYTES) + EPI_WARPS * 2 * OUT_BYTES + 1024;
constexpr int BAND = 32;  // row tiles that pass over the columns together
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float FUSED = 1e6f;  // below it x log2 e is rounded by at most 1/16
constexpr size_t PIECE_BYTES = 256u << 20;
constexpr float F16_ROOM = 16384.f;  // |d| <= 1 after the division: as fp16, 2^14 times that

struct Job {
    int m_tiles, n_tiles, bn;  // columns of a tile: a multiple of 32, at most BN
    int K, parts;              // the sum's length, and into how many parts it is split
    int mn_a;                  // A with M inner
    int b_y0, out_y0;          // added to B's and the output's row coordinates
    int part_rows;             // rows of the output from one part to the next
    int add, out_f32;
};

// Which items a CTA takes: of the first job every G-th (G the grid), then of the
// second what evens the CTAs out: `long_items` each for those with one more of the first,
// `short_items` for the others.
struct Params {
    Job job[2];
    int items0, items1, longer, long_items, short_items;
    uint32_t idesc;     // but for N and the operands' order
    int T, V;           // rows, columns that there are (LOSS: of the vocabulary; GRAD: of the piece)
    int v0, all;        // the piece's first column, columns of the whole vocabulary
    int f16;
    const int32_t *labels;
    float2 *stats;      // [T][n tiles]
    float *label_z;
    const float *lse, *dloss, *dlse, *top;
    int32_t *status;
};

struct Maps {
    CUtensorMap a[2], b[2], out[2];
};

struct Shared {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem;
    volatile int abort;
};

struct Item {
    int j, m, n, part;  // job, tiles, part of K
    int kb0, kb1;       // steps
};

// The CTA's i-th item; false when there are no more.  Row tiles first, within bands of BAND: the tiles at work
// share the columns' operand, and a band's rows stay in L2.
__device__ __forceinline__ bool item_of(const Params &p, int i, Item &it)
{
    const int c = blockIdx.x, G = gridDim.x;
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
    const int whole = g.m_tiles * g.n_tiles;
    it.part = t / whole;
    t -= it.part * whole;
    const int band = t / (BAND * g.n_tiles), m0 = band * BAND, rows = min(BAND, g.m_tiles - m0);
    t -= band * BAND * g.n_tiles;
    it.n = t / rows;
    it.m = m0 + t - it.n * rows;
    const int nk = (g.K + BK - 1) / BK;
    it.kb0 = (int)((int64_t)nk * it.part / g.parts);
    it.kb1 = (int)((int64_t)nk * (it.part + 1) / g.parts);
    return true;
}

__device__ __forceinline__ bool warp_wait(Shared &S, uint64_t *bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    const bool ok = tc::mbar_wait(bar, parity, kWaitNs);
    return __all_sync(0xffffffffu, ok && !S.abort);
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

template <Kind K>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps)
{
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
            tc::mbar_init(&S.acc_empty[i], EPI_WARPS);
        }
        tc::mbar_init(&S.mma_done, 1);
        S.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == EPI_WARP0) tc::tmem_alloc(&S.tmem, 512);
    // (launched while the kernel before it may still run, and lets the next one come as soon: nothing above reads what that one writes)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)S.tmem);

    if (warp == 0) {
        // ---------------- operands
        int it = 0, s = 0;
        uint32_t phase = 1;
        bool ok = true;
        Item m;
        for (int i = 0; ok && item_of(p, i, m); i++) {
            const Job &g = p.job[m.j];
            const int boxes = (g.bn + 63) / 64;
            const uint32_t bytes = A_BYTES + (K == PROD ? boxes * (BK * 128) : g.bn * 128);
            for (int kb = m.kb0; kb < m.kb1; kb++, it++) {
                if (it >= STAGES) ok = warp_wait(S, &S.empty[s], phase);
                if (!ok) break;
                if (elect_one()) {
                    tc::mbar_arrive_expect_tx(&S.full[s], bytes);
                    char *a = sA + s * A_BYTES, *b = sB + s * B_BYTES;
                    if (K == PROD && g.mn_a) {
#pragma unroll
                        for (int h = 0; h < BM / 64; h++)
                            tc::tma_load_2d(a + h * BK * 128, &maps.a[m.j], m.m * BM + h * 64, kb * BK, &S.full[s]);
                    } else {
                        tc::tma_load_2d(a, &maps.a[m.j], kb * BK, m.m * BM, &S.full[s]);
                    }
                    if (K == PROD) {
                        for (int h = 0; h < boxes; h++)
                            tc::tma_load_2d(b + h * BK * 128, &maps.b[m.j], m.n * g.bn + h * 64, g.b_y0 + kb * BK, &S.full[s]);
                    } else {
                        tc::tma_load_2d(b, &maps.b[m.j], kb * BK, g.b_y0 + m.n * g.bn, &S.full[s]);
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
            // no copy may still be in flight when the CTA leaves
            for (int i = 0; i < STAGES && i < it; i++) {
                const int u = (it - 1 - i) / STAGES;
                if (!tc::mbar_wait(&S.full[(it - 1 - i) % STAGES], u & 1, kWaitNs)) set_status(p.status, MOE_ERR_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA
        int j = 0, s = 0;
        uint32_t phase = 0;
        bool ok = true;
        Item m;
        for (int i = 0; ok && item_of(p, i, m); i++) {
            const Job &g = p.job[m.j];
            if (m.kb0 == m.kb1) continue;  // a part of nothing
            const int acc = j & 1, v = j >> 1;
            j++;
            if (v > 0) ok = warp_wait(S, &S.acc_empty[acc], (v - 1) & 1);
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
                        if (k * 16 < left) tc::mma_f16_ss(d, da + k * ka, db + k * kbs, idesc, (kb > m.kb0 || k > 0) ? 1u : 0u);
                    tc::mma_commit(&S.empty[s]);
                    if (kb + 1 == m.kb1) tc::mma_commit(&S.acc_full[acc]);
                }
                s = sn;
                phase = phase_n;
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, MOE_ERR_TIMEOUT);
            S.abort = 1;
        }
        if (elect_one()) tc::mma_commit(&S.mma_done);
        if (!tc::mbar_wait(&S.mma_done, 0, kWaitNs) && lane == 0) set_status(p.status, MOE_ERR_TIMEOUT);
    } else {
        // ---------------- sums out
        const int q = warp & 3;
        char *out = sO + (warp - EPI_WARP0) * 2 * OUT_BYTES;
        int j = 0, turn = 0;
        const float top = K == LOSS ? 0.f : *p.top;
        const float up = K == PROD ? (p.f16 ? top / F16_ROOM : top) : 0.f;
        const float down = K == GRAD && top > 0.f ? (p.f16 ? F16_ROOM : 1.f) : 0.f;
        Item m;
        for (int i = 0; item_of(p, i, m); i++) {
            const Job &g = p.job[m.j];
            if (m.kb0 == m.kb1) continue;
            const int acc = j & 1, v = j >> 1;
            j++;
            const int row = m.m * BM + q * 32 + lane, n0 = m.n * g.bn;
            int label = -1;
            float lse = 0.f, nl = 0.f, a = 0.f, b = 0.f;
            if (K != PROD && row < p.T) label = p.labels[row];
            if (K == GRAD && row < p.T) {
                const bool there = label >= 0 && label < p.all;
                b = there ? p.dloss[row] : 0.f;
                a = b + (p.dlse ? p.dlse[row] : 0.f);
                a = down > 0.f ? a / top * down : 0.f;
                b = down > 0.f ? b / top * down : 0.f;
                lse = p.lse[row];
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
                for (int c = 0; c < g.bn; c += 32) {
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
                    p.stats[(int64_t)row * g.n_tiles + m.n] = make_float2(mx, sum);
                    if (mine) p.label_z[row] = zl;
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < g.bn; c += 32) {
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
                    char *buf = out + (turn & 1) * OUT_BYTES;
                    turn++;
                    if (lane == 0) tc::bulk_wait_read<1>();
                    __syncwarp();
                    put_row(buf, lane, r, f32);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int x = n0 + c, y = g.out_y0 + m.part * g.part_rows + m.m * BM + q * 32;
                        if (K == PROD && g.add) tma_add_2d(&maps.out[m.j], x, y, buf);
                        else tc::tma_store_2d(&maps.out[m.j], x, y, buf);
                        tc::bulk_commit();
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.acc_empty[acc]);
        }
        if (K != LOSS && lane == 0) tc::bulk_wait_all();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == EPI_WARP0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
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

// The largest |dloss| or |dlse| of the tokens that count; one CTA.
__global__ void __launch_bounds__(1024) top_kernel(const float *dloss, const float *dlse, const int32_t *labels, int T, int V, float *top)
{
    __shared__ float part[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float m = 0.f;
    for (int t = threadIdx.x; t < T; t += 1024) {
        const int label = labels[t];
        if (label >= 0 && label < V) m = fmaxf(m, fabsf(dloss[t]));
        if (dlse) m = fmaxf(m, fabsf(dlse[t]));
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if (lane_id() == 0) part[warp_id()] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(part[threadIdx.x])));
        if (threadIdx.x == 0) *top = m;
    }
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

static int tiles(int n, int b) { return (n + b - 1) / b; }

// Columns of a piece: what 256 MiB hold, in whole tiles, and pieces of nearly equal size.
static int piece_columns(int T, int V)
{
    const int64_t most = std::max<int64_t>(BN, (int64_t)(PIECE_BYTES / 2 / std::max(T, 1)) / BN * BN);
    const int64_t pieces = (V + most - 1) / most;
    return (int)((V + pieces - 1) / pieces + BN - 1) / BN * BN;
}

static int round_up(int n, int b) { return tiles(n, b) * b; }

// Columns of a tile: equal ones over all n.
static int tile_columns(int n) { return round_up(tiles(n, tiles(n, BN)), 32); }

// The vocabulary's tiles for the logits: as wide as they go, unless narrower ones fill the last round of CTAs better
// (100,003 columns for one row tile on 152 SMs: three rounds of 224 instead of 256).
static int vocabulary_columns(int rows, int V, int sms)
{
    int best = BN;
    int64_t least = INT64_MAX;
    for (int bn = BN; bn >= 128; bn -= 32) {
        const int64_t rounds = ((int64_t)tiles(rows, BM) * tiles(V, bn) + sms - 1) / sms, cost = rounds * (bn + 16);
        if (cost < least) least = cost, best = bn;
    }
    return best;
}

// What a CTA of the gradients takes, in steps of BK: dh's items (nk0 each) dealt out first, dW's (nk1 each) so that the
// longest CTA is as short as it gets.
struct Deal {
    int longer, long_items, short_items;
    int64_t steps;
};

static Deal deal(int64_t items0, int64_t nk0, int64_t items1, int64_t nk1, int64_t G)
{
    Deal best = {0, 0, 0, INT64_MAX};
    const int64_t q = items0 / G, r = items0 % G;
    auto with = [&](int64_t s) {  // s items of the second job for a CTA without an extra one of the first
        const int64_t rest = std::max<int64_t>(0, items1 - (G - r) * s);
        if (s < 0 || (r == 0 && rest > 0)) return;
        const int64_t l = r ? (rest + r - 1) / r : s;
        const int64_t steps = std::max(r ? (q + 1) * nk0 + l * nk1 : 0, q * nk0 + s * nk1);
        if (steps < best.steps) best = {(int)r, (int)l, (int)s, steps};
    };
    with((items1 + G - r - 1) / (G - r));
    if (nk1 > 0) {  // about where all have the same
        const int64_t s = ((items0 * nk0 + items1 * nk1) / G - q * nk0) / nk1;
        for (int64_t i = s - 1; i <= s + 2; i++) with(i);
    }
    return best;
}

struct Layout {
    int columns, pieces, parts;  // dh's sums over a piece are split into parts
    int64_t part_rows;
    size_t d, sums, total;  // bytes: d after the top value, fp32 sums of dh when there are several pieces or parts
};

// Splitting dh's sums pays where its few, long items would leave the other CTAs waiting: steps of 0.27 us are weighed
// against a part's sums, written and read (8 bytes a value at 6 TB/s), and a launch for them.
static Layout layout(int T, int H, int V)
{
    Layout l;
    const int sms = sm_count();
    l.columns = piece_columns(T, V);
    l.pieces = tiles(V, l.columns);
    const int n = std::min(V, l.columns), nk0 = tiles(n, BK), nk1 = tiles(T, BK), nt = tiles(H, BN);
    const int64_t items0 = (int64_t)tiles(T, BM) * nt, items1 = (int64_t)tiles(n, BM) * nt;
    l.part_rows = round_up(T, BM);
    l.parts = 1;
    double least = 0;
    for (int s = 1; s <= 32 && s <= nk0; s++) {
        const Deal d = deal(items0 * s, tiles(nk0, s), items1, nk1, std::min<int64_t>(items0 * s + items1, sms));
        const double us = 0.27 * d.steps + (s > 1 || l.pieces > 1 ? 3.0 / l.pieces + 1.3e-6 * s * T * H * (l.pieces > 1 ? 2 : 1) : 0);
        if (s == 1 || us < least) least = us, l.parts = s;
    }
    l.d = 256;
    l.sums = l.d + align256((size_t)T * l.columns * 2);
    l.total = l.sums + (l.pieces > 1 || l.parts > 1 ? align256((size_t)l.parts * l.part_rows * H * 4) : 0);
    return l;
}

static moe_status check(int T, int H, int V)
{
    MOE_REQUIRE(T >= 0 && T <= (1 << 24), "T must be in [0, 2^24] (got %d)", T);
    MOE_REQUIRE(H >= 8 && H % 8 == 0 && H <= (1 << 20), "H must be a multiple of 8 in [8, 2^20] (got %d)", H);
    MOE_REQUIRE(V >= 1 && V <= (1 << 24), "V must be in [1, 2^24] (got %d)", V);
    MOE_REQUIRE((int64_t)tiles(T, BM) * tiles(V, BN / 2) < (1 << 30) && (int64_t)std::max(T, V) * H < (1ll << 40),
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
moe_status launch(const char *what, F kernel, int grid, int threads, size_t smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];  // the set-up overlaps the end of the kernel before
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    return check_launch(what);
}

template <Kind K>
moe_status product(Params &p, const Maps &maps, cudaStream_t s)
{
    auto items = [](const Job &g) { return g.m_tiles * g.n_tiles * g.parts; };
    p.items0 = items(p.job[0]);
    p.items1 = items(p.job[1]);
    const int grid = (int)std::min<int64_t>((int64_t)p.items0 + p.items1, sm_count());
    const Deal d = deal(p.items0, tiles(tiles(p.job[0].K, BK), p.job[0].parts), p.items1, tiles(p.job[1].K, BK), grid);
    p.longer = d.longer, p.long_items = d.long_items, p.short_items = d.short_items;
    MOE_CUDA_TRY(cudaFuncSetAttribute(product_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM));
    return launch("cross_entropy", product_kernel<K>, grid, THREADS, SMEM, s, p, maps);
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
    *bytes = align256((size_t)T * 4) + align256((size_t)tiles(V, vocabulary_columns(T, V, sm_count())) * T * 8);
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
    const int bn = vocabulary_columns(T, V, sm_count()), n_tiles = tiles(V, bn);
    p.job[0] = {tiles(T, BM), n_tiles, bn, H, 1, 0, 0, 0, 0, 0, 0};
    p.idesc = tc::idesc_f16_f32(BM, 0, dtype == MOE_BF16);
    p.T = T, p.V = V, p.labels = labels, p.status = dev_status;
    p.label_z = static_cast<float *>(ws);
    p.stats = reinterpret_cast<float2 *>(static_cast<char *>(ws) + align256((size_t)T * 4));
    st = make_tmap_2d(&maps.a[0], h, map_type(dtype), 2, T, H, BK, BM);
    if (st == MOE_OK) st = make_tmap_2d(&maps.b[0], w, map_type(dtype), 2, V, H, BK, bn);
    if (st != MOE_OK) return st;
    const cudaStream_t s = to_cuda(stream);
    st = product<LOSS>(p, maps, s);
    if (st != MOE_OK) return st;
    return launch("cross_entropy_combine", combine_kernel, tiles(T, COMBINE_WARPS), COMBINE_WARPS * 32, 0, s, p.stats, p.label_z, labels, T,
                  V, n_tiles, loss, lse, dev_status);
}

extern "C" moe_status moe_cross_entropy_backward_workspace_size(int T, int H, int V, size_t *bytes)
{
    using namespace ce;
    MOE_REQUIRE(bytes, "bytes must not be NULL");
    moe_status st = check(T, H, V);
    if (st != MOE_OK) return st;
    *bytes = T ? layout(T, H, V).total : 0;
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
    const Layout l = layout(T, H, V);
    if (ws_bytes < l.total || !ws)
        return fail(MOE_ERR_WORKSPACE, "moe_cross_entropy_backward needs %zu bytes of workspace (got %zu)", l.total,
                    ws ? ws_bytes : (size_t)0);
    MOE_REQUIRE(aligned16(ws), "ws must be 16-byte aligned");
    char *base = static_cast<char *>(ws);
    float *top = reinterpret_cast<float *>(base), *sums = reinterpret_cast<float *>(base + l.sums);
    void *d = base + l.d;

    st = launch("cross_entropy_top", top_kernel, 1, 1024, 0, s, dloss, dlse, labels, T, V, top);
    if (st != MOE_OK) return st;
    Params gp = {}, pp = {};
    Maps gm = {}, pm = {};
    const int f16 = dtype == MOE_F16;
    gp.idesc = pp.idesc = tc::idesc_f16_f32(BM, 0, !f16);
    gp.T = T, gp.all = V, gp.labels = labels, gp.lse = lse, gp.dloss = dloss, gp.dlse = dlse, gp.top = pp.top = top;
    gp.status = pp.status = dev_status;
    gp.f16 = pp.f16 = f16;
    const bool direct = l.pieces == 1 && l.parts == 1;  // dh leaves as it is: no sums of pieces or parts
    const auto half = CU_TENSOR_MAP_SWIZZLE_64B;        // boxes of 32 16-bit columns
    st = make_tmap_2d(&gm.a[0], h, map_type(dtype), 2, T, H, BK, BM);
    if (st == MOE_OK) st = make_tmap_2d(&gm.b[0], w, map_type(dtype), 2, V, H, BK, BN);
    if (st == MOE_OK) st = make_tmap_2d(&gm.out[0], d, map_type(dtype), 2, T, l.columns, 32, 32, half);
    CUtensorMap d_k, d_m, w_n, h_n, out_h, out_w;
    if (st == MOE_OK) st = make_tmap_2d(&d_k, d, map_type(dtype), 2, T, l.columns, BK, BM);
    if (st == MOE_OK) st = make_tmap_2d(&d_m, d, map_type(dtype), 2, T, l.columns, 64, BK);
    if (st == MOE_OK) st = make_tmap_2d(&w_n, w, map_type(dtype), 2, V, H, 64, BK);
    if (st == MOE_OK) st = make_tmap_2d(&h_n, h, map_type(dtype), 2, T, H, 64, BK);
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
        gp.job[0] = {tiles(T, BM), tiles(n, BN), BN, H, 1, 0, v0, 0, 0, 0, 0};
        st = product<GRAD>(gp, gm, s);
        if (st != MOE_OK) return st;
        int j = 0;
        if (dh) {
            pp.job[j] = {tiles(T, BM), nt, bn, n, l.parts, 0, v0, 0, (int)l.part_rows, !direct && i > 0, !direct};
            pm.a[j] = d_k, pm.b[j] = w_n, pm.out[j] = out_h;
            j++;
        }
        if (dw) {
            pp.job[j] = {tiles(n, BM), nt, bn, T, 1, 1, 0, v0, 0, accumulate != 0, dw_dtype == MOE_F32};
            pm.a[j] = d_m, pm.b[j] = h_n, pm.out[j] = out_w;
            j++;
        }
        st = product<PROD>(pp, pm, s);
        if (st != MOE_OK) return st;
    }
    if (dh && !direct) {
        const int64_t n = (int64_t)T * H;
        const int grid = (int)std::min<int64_t>((n + 2047) / 2048, (int64_t)sm_count() * 8);
        return f16 ? launch("cross_entropy_round", round_kernel<Fp16>, grid, 256, 0, s, sums, l.parts, l.part_rows * H, static_cast<uint16_t *>(dh), n)
                   : launch("cross_entropy_round", round_kernel<Bf16>, grid, 256, 0, s, sums, l.parts, l.part_rows * H, static_cast<uint16_t *>(dh), n);
    }
    return MOE_OK;
}
