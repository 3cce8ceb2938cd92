// mx4_matmul.cu -- moe_mx4_matmul: products of 4-bit floating point matrices
// (e2m1 codes, e8m0 scales per 32) on the tensor cores, one expert's weights
// for each group of rows.
//
//   out[p][n] = sum_k X[p][k] W_e[n][k]     (e: the group that row p is in)
//
// tcgen05.mma kind::mxf4 takes the codes and the scales as they are stored, so
// nothing is dequantised: products and sums are the tensor cores' fp32.  The
// weights are the M operand (128 rows a tile) and an expert's rows are N (16
// to 224), so that an expert with few rows wastes little: a tile reads 128
// weight rows for whatever rows there are, and one or two rows cost the same
// as sixteen.
//
// A CTA walks (row tile, weight tile) items.  A step is 256 of K (128 bytes
// of codes per row).  Warp 0 loads the codes of both operands with TMA
// (128-byte swizzle); warps 2 and 3 load the scales (eight bytes per row and
// step, four steps at a time, taken in turn) and put them into shared memory
// in the order that tcgen05.cp spreads over tensor memory (row r of a
// 128-row, 128-K chunk at byte (r % 32) * 16 + (r / 32) * 4); warp 1 issues the
// copies of the scales and four MMAs of K = 64; warps 4..7 take the sums out
// of tensor memory, two accumulators in turn.
//
// With SwiGLU a tile holds 64 gate rows and their 64 up rows, 16 of each in
// turn, so that both of a column's sums lie in one warp's lanes.
//
// Few items leave SMs idle while each reads its whole K, so K is split over a
// cluster of up to eight CTAs, which add their parts through distributed
// shared memory, in order.
//
// Every wait is bounded: after about 2 s the CTA records MOE_ERR_TIMEOUT and
// stops.
#include "dense_tc.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace moe {
namespace mx {

constexpr int BM = 128;            // weight rows per tile
constexpr int BK = 256;            // K per step
constexpr int MAX_BN = 224;        // rows per tile: two accumulators and the scales fill tensor memory
constexpr int MAX_STAGES = 12;
constexpr int A_BYTES = BM * BK / 2;
constexpr int SF_BYTES = 2 * 512 + 4 * 512;  // scales of a step: weights, then rows (two chunks of 128 rows)
constexpr int SF_COL = 2 * MAX_BN;           // tensor memory columns of the scales (two sets of 32)
constexpr int THREADS = 256;
constexpr int EPI_WARP0 = 4;
constexpr int MAX_E = 1024;
constexpr unsigned long long kWaitNs = 2000000000ull;

struct Params {
    int E, N, w_rows, rows;      // w_rows: weight rows per expert (N or 2N)
    int nk, n_mma;               // steps, and MMAs of K = 64, over the whole K
    int n_tiles, bn, stages, splits, swiglu;
    const int32_t *offsets;      // NULL: one group of all rows
    const uint8_t *w_scales, *x_scales;
    int pitch;                   // bytes of scales per row
    void *out;
    int out_type;
    int32_t *status;
};

struct Shared {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem;
    volatile int abort;
    int warp_tot[THREADS / 32];
    int tile0[MAX_E + 1];  // row tiles before expert e
};

struct Item {
    int e, p0, cnt;  // expert, first row, rows
    int n0;          // first output column
    int kb0, kb1;    // steps of this CTA
};

__device__ __forceinline__ void group_of(const Params &p, int e, int &p0, int &cnt)
{
    if (!p.offsets) {
        p0 = 0;
        cnt = p.rows;
        return;
    }
    // both ends clipped first, so that no offsets lead out of the rows
    const int a = min(max(__ldg(p.offsets + e), 0), p.rows), b = min(max(__ldg(p.offsets + e + 1), 0), p.rows);
    p0 = a;
    cnt = max(0, b - a);
}

__device__ __forceinline__ Item item_of(const Params &p, const Shared &S, int item, int split)
{
    Item it;
    const int tt = item / p.n_tiles;
    it.n0 = (item % p.n_tiles) * (p.swiglu ? BM / 2 : BM);
    int lo = 0, hi = p.E - 1;  // the last expert with tile0 <= tt
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (S.tile0[mid] <= tt) lo = mid;
        else hi = mid - 1;
    }
    it.e = lo;
    int p0, cnt;
    group_of(p, lo, p0, cnt);
    const int nt = S.tile0[lo + 1] - S.tile0[lo], j = tt - S.tile0[lo];
    const int w = ((cnt + nt - 1) / nt + 15) & ~15;
    it.p0 = p0 + j * w;
    it.cnt = min(w, cnt - j * w);
    it.kb0 = p.nk * split / p.splits;
    it.kb1 = p.nk * (split + 1) / p.splits;
    return it;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

// The float at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
        : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes) to four columns, repeated in the
// four lane quadrants.  Runs in order with the MMAs of the issuing thread.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t smem_addr)
{
    const uint64_t d = (uint64_t)((smem_addr & 0x3FFFFu) >> 4)  // start; no swizzle
                       | (uint64_t)(128 >> 4) << 32             // next eight rows of 16 bytes
                       | (uint64_t)1 << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::mxf4 with e2m1 operands and e8m0 scales, K
// = 64; `id`: the first of the two scales within a column's four bytes.
__device__ __forceinline__ uint32_t idesc_mxf4(int n, uint32_t id)
{
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(BM >> 7) << 27) |
           (id << 29);
}

__device__ __forceinline__ void store_out(const Params &p, int64_t i, float v)
{
    if (p.out_type == MOE_F32) static_cast<float *>(p.out)[i] = v;
    else if (p.out_type == MOE_BF16) Bf16::store(static_cast<uint16_t *>(p.out) + i, v);
    else Fp16::store(static_cast<uint16_t *>(p.out) + i, v);
}

// Lane `lane` of quadrant q holds columns c .. c+31 of a tile's sums.
__device__ __forceinline__ void write_columns(const Params &p, const Item &it, int q, int lane, int c, const float (&v)[32])
{
    if (!p.swiglu) {
        const int n = it.n0 + q * 32 + lane;
#pragma unroll
        for (int i = 0; i < 32; i++)
            if (n < p.N && c + i < it.cnt) store_out(p, (int64_t)(it.p0 + c + i) * p.N + n, v[i]);
        return;
    }
    // lanes 0..15: gate, 16..31: the same columns' up.  Each pair of lanes
    // swaps one value, and then has both of one row.
    const bool up = lane >= 16;
    const int n = it.n0 + q * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 1], 16);
        const float g = up ? got : v[i], u = up ? v[i + 1] : got;
        const int r = c + i + (up ? 1 : 0);
        if (n < p.N && r < it.cnt) store_out(p, (int64_t)(it.p0 + r) * p.N + n, g / (1.0f + expf(-g)) * u);
    }
}

__global__ void __launch_bounds__(THREADS, 1) mx4_matmul_kernel(const __grid_constant__ Params p,
                                                                const __grid_constant__ CUtensorMap mw,
                                                                const __grid_constant__ CUtensorMap mx)
{
    extern __shared__ __align__(1024) char dyn_raw[];
    char *dyn = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    const int b_bytes = (p.bn + 31) / 32 * 32 * (BK / 2);
    char *sA = dyn, *sB = sA + p.stages * A_BYTES, *sF = sB + p.stages * b_bytes;
    __shared__ Shared S;
    const int warp = warp_id(), lane = lane_id();
    const int split = p.splits > 1 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / p.splits, step = gridDim.x / p.splits;

    // row tiles before each expert: four experts per thread, then a scan
    {
        int n[MAX_E / THREADS], sum = 0;
#pragma unroll
        for (int i = 0; i < MAX_E / THREADS; i++) {
            const int e = threadIdx.x * (MAX_E / THREADS) + i;
            int p0, cnt = 0;
            if (e < p.E) {
                group_of(p, e, p0, cnt);
                if (p.offsets && blockIdx.x == 0) {
                    const int a = p.offsets[e], b = p.offsets[e + 1];
                    if (a < 0 || b < a || b > p.rows) set_status(p.status, MOE_ERR_BOUNDS);
                }
            }
            n[i] = sum;
            sum += (cnt + p.bn - 1) / p.bn;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) S.warp_tot[warp] = incl;
        __syncthreads();
        int base = incl - sum;
        for (int i = 0; i < warp; i++) base += S.warp_tot[i];
#pragma unroll
        for (int i = 0; i < MAX_E / THREADS; i++) {
            const int e = threadIdx.x * (MAX_E / THREADS) + i;
            if (e <= p.E) S.tile0[e] = base + n[i];
        }
        if (p.E == MAX_E && threadIdx.x == THREADS - 1) S.tile0[MAX_E] = base + sum;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; s++) {
            tc::mbar_init(&S.full[s], 2);  // the producer's (with the bytes of its copies) and the scales'
            tc::mbar_init(&S.empty[s], 1);
        }
        for (int i = 0; i < 2; i++) {
            tc::mbar_init(&S.acc_full[i], 1);
            tc::mbar_init(&S.acc_empty[i], 4);
        }
        tc::mbar_init(&S.mma_done, 1);
        S.abort = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&mw);
        tc::tma_prefetch_desc(&mx);
    }
    if (warp == 2) tc::tmem_alloc(&S.tmem, 512);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = S.tmem;
    // (a cluster that splits K takes one item; the grid holds them all)
    const int total = p.splits > 1 ? min(S.tile0[p.E] * p.n_tiles, step) : S.tile0[p.E] * p.n_tiles;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- codes
            int it = 0;
            for (int item = first; item < total && !S.abort; item += step) {
                const Item m = item_of(p, S, item, split);
                const int boxes = (m.cnt + 31) / 32;
                for (int kb = m.kb0; kb < m.kb1; kb++, it++) {
                    const int s = it % p.stages, u = it / p.stages;
                    if (u > 0 && !tc::mbar_wait(&S.empty[s], (u - 1) & 1, kWaitNs)) {
                        set_status(p.status, MOE_ERR_TIMEOUT);
                        S.abort = 1;
                        break;
                    }
                    tc::mbar_arrive_expect_tx(&S.full[s], A_BYTES + boxes * 32 * (BK / 2));
                    char *a = sA + s * A_BYTES, *b = sB + s * b_bytes;
                    const int x = kb * (BK / 2);
                    if (p.swiglu) {
                        for (int i = 0; i < 8; i++)
                            tma_load_3d(a + i * 16 * (BK / 2), &mw, x, (i & 1) * p.N + m.n0 + (i >> 1) * 16, m.e, &S.full[s]);
                    } else {
                        tma_load_3d(a, &mw, x, m.n0, m.e, &S.full[s]);
                    }
                    for (int i = 0; i < boxes; i++)
                        tc::tma_load_2d(b + i * 32 * (BK / 2), &mx, x, m.p0 + i * 32, &S.full[s]);
                }
            }
            // no copy may still be in flight when the CTA leaves (a full
            // barrier that never got its scales' arrival runs out of time)
            for (int s = 0; s < p.stages && s < it; s++) {
                const int u = (it - 1 - s) / p.stages;
                if (!tc::mbar_wait(&S.full[s], u & 1, kWaitNs)) set_status(p.status, MOE_ERR_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA
            int it = 0, j = 0;
            bool stop = false;
            for (int item = first; item < total && !stop; item += step, j++) {
                const Item m = item_of(p, S, item, split);
                const int acc = j & 1, v = j >> 1;
                if (S.abort || (v > 0 && !tc::mbar_wait(&S.acc_empty[acc], (v - 1) & 1, kWaitNs))) {
                    stop = true;
                    break;
                }
                tc::tc_fence_after();
                const int n16 = (m.cnt + 15) & ~15;
                const uint32_t d = tmem + (uint32_t)(acc * MAX_BN);
                const uint32_t id0 = idesc_mxf4(n16, 0), id2 = idesc_mxf4(n16, 2);
                for (int kb = m.kb0; kb < m.kb1; kb++, it++) {
                    const int s = it % p.stages, u = it / p.stages;
                    if (!tc::mbar_wait(&S.full[s], u & 1, kWaitNs)) {
                        stop = true;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t sfa = tmem + SF_COL + (it & 1) * 32, sfb = sfa + 8;
                    const uint32_t f = tc::smem_u32(sF + s * SF_BYTES);
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        cp_scales(sfa + c * 4, f + c * 512);
                        cp_scales(sfb + c * 8, f + 1024 + c * 1024);
                        if (n16 > 128) cp_scales(sfb + c * 8 + 4, f + 1024 + c * 1024 + 512);
                    }
                    const uint64_t da = tc::desc_kmajor_sw128(tc::smem_u32(sA + s * A_BYTES));
                    const uint64_t db = tc::desc_kmajor_sw128(tc::smem_u32(sB + s * b_bytes));
                    const int nm = min(4, p.n_mma - kb * 4);
                    for (int i = 0; i < nm; i++)  // 32 bytes of the swizzled rows per MMA
                        mma_mxf4(d, da + i * 2, db + i * 2, (i & 1) ? id2 : id0, sfa + (i >> 1) * 4, sfb + (i >> 1) * 8,
                                 (kb > m.kb0 || i > 0) ? 1u : 0u);
                    tc::mma_commit(&S.empty[s]);
                }
                if (!stop) tc::mma_commit(&S.acc_full[acc]);
            }
            if (stop) {
                set_status(p.status, MOE_ERR_TIMEOUT);
                S.abort = 1;
            }
            tc::mma_commit(&S.mma_done);
            if (!tc::mbar_wait(&S.mma_done, 0, kWaitNs)) set_status(p.status, MOE_ERR_TIMEOUT);
        }
    } else if (warp == 2 || warp == 3) {
        // ---------------- scales: four steps at a time, the two warps in turn
        int it = 0, turn = 0;
        for (int item = first; item < total; item += step) {
            const Item m = item_of(p, S, item, split);
            bool stop = false;
            for (int kb = m.kb0; kb < m.kb1; kb += 4, turn ^= 1) {
                const int n = min(4, m.kb1 - kb);
                if (turn == (warp & 1)) {
                    uint2 wv[4][4], xv[MAX_BN / 32][4];
#pragma unroll
                    for (int g = 0; g < 4; g++) {
                        const int r = g * 32 + lane;
                        const int row = p.swiglu ? m.n0 + g * 16 + (lane & 15) : m.n0 + r;
                        const bool in = row < p.N;
                        const uint8_t *src =
                            p.w_scales + ((int64_t)m.e * p.w_rows + (p.swiglu && lane >= 16 ? p.N : 0) + row) * p.pitch + kb * 8;
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            wv[g][i] = in && i < n ? __ldg(reinterpret_cast<const uint2 *>(src) + i) : make_uint2(0u, 0u);
                    }
#pragma unroll
                    for (int g = 0; g < MAX_BN / 32; g++) {
                        const int r = g * 32 + lane;
                        const uint8_t *src = p.x_scales + (int64_t)(m.p0 + r) * p.pitch + kb * 8;
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            xv[g][i] = r < m.cnt && i < n ? __ldg(reinterpret_cast<const uint2 *>(src) + i) : make_uint2(0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (i >= n || stop) break;
                        const int s = (it + i) % p.stages, u = (it + i) / p.stages;
                        bool ok = true;
                        if (lane == 0) ok = !S.abort && (u == 0 || tc::mbar_wait(&S.empty[s], (u - 1) & 1, kWaitNs));
                        if (!__shfl_sync(0xffffffffu, (int)ok, 0)) {
                            stop = true;
                            break;
                        }
                        char *f = sF + s * SF_BYTES;
#pragma unroll
                        for (int g = 0; g < 4; g++) {
                            *reinterpret_cast<uint32_t *>(f + lane * 16 + g * 4) = wv[g][i].x;
                            *reinterpret_cast<uint32_t *>(f + 512 + lane * 16 + g * 4) = wv[g][i].y;
                        }
#pragma unroll
                        for (int g = 0; g < MAX_BN / 32; g++) {
                            if (g * 32 >= p.bn) break;
                            char *b = f + 1024 + (g >> 2) * 512 + lane * 16 + (g & 3) * 4;
                            *reinterpret_cast<uint32_t *>(b) = xv[g][i].x;
                            *reinterpret_cast<uint32_t *>(b + 1024) = xv[g][i].y;
                        }
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&S.full[s]);
                    }
                }
                it += n;
                if (stop) break;
            }
            if (stop) break;
        }
    } else {
        // ---------------- sums out
        const int q = warp - EPI_WARP0;
        int j = 0;
        for (int item = first; item < total && !S.abort; item += step, j++) {
            const Item m = item_of(p, S, item, split);
            const int acc = j & 1, v = j >> 1;
            if (!tc::mbar_wait(&S.acc_full[acc], v & 1, kWaitNs)) {
                if (lane == 0) set_status(p.status, MOE_ERR_TIMEOUT);
                S.abort = 1;
                break;
            }
            tc::tc_fence_after();
            const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * MAX_BN);
            for (int c = 0; c < m.cnt; c += 32) {
                uint32_t r[32];
                __syncwarp();
                tc::tmem_ld_32x32b_x32(tbase + c, r);
                tc::tmem_ld_wait();
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; i++) f[i] = __uint_as_float(r[i]);
                if (p.splits > 1) {
                    // every copy of this (only) item has been consumed: its stages hold the part now
                    float *part = reinterpret_cast<float *>(dyn) + c * BM + q * 32 + lane;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (c + i < m.cnt) part[i * BM] = f[i];
                } else {
                    write_columns(p, m, q, lane, c, f);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.acc_empty[acc]);
        }
        if (p.offsets) {  // rows of no group
            const int z0 = max(0, min(p.rows, __ldg(p.offsets + p.E)));
            const int64_t n = (int64_t)(p.rows - z0) * p.N;
            for (int64_t i = (int64_t)blockIdx.x * 128 + (threadIdx.x - EPI_WARP0 * 32); i < n; i += (int64_t)gridDim.x * 128)
                store_out(p, (int64_t)z0 * p.N + i, 0.f);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (p.splits > 1) {
        // the cluster's parts, added in order; each CTA takes groups of 32 rows in turn
        cluster_sync();
        if (warp >= EPI_WARP0 && first < total) {
            const int q = warp - EPI_WARP0;
            const Item m = item_of(p, S, first, split);
            const int per = (m.cnt + p.splits - 1) / p.splits;  // rows of this CTA
            const int c1 = min(m.cnt, (split + 1) * per);
            for (int c = split * per; c < c1; c += 32) {
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; i++) {
                    f[i] = 0.f;
                    if (c + i < c1)
                        for (int r = 0; r < p.splits; r++)
                            f[i] += ld_cluster(tc::smem_u32(reinterpret_cast<float *>(dyn) + (c + i) * BM + q * 32 + lane), r);
                }
                Item mine = m;
                mine.cnt = c1;
                write_columns(p, mine, q, lane, c, f);
            }
        }
        cluster_sync();  // no CTA leaves while another reads its part
    }
}

}  // namespace mx

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mx4_matmul(const uint8_t *w_codes, const uint8_t *w_scales, int E, int N, int K,
                                     const uint8_t *x_codes, const uint8_t *x_scales, int rows, const int32_t *offsets,
                                     void *out, moe_dtype out_dtype, moe_mx4_epilogue epilogue, int32_t *dev_status,
                                     moe_stream_t stream)
{
    using namespace mx;
    MOE_REQUIRE(E >= 1 && E <= MAX_E, "E must be in [1, %d] (got %d)", MAX_E, E);
    MOE_REQUIRE(N >= 1 && N <= (1 << 24), "N must be in [1, 2^24] (got %d)", N);
    MOE_REQUIRE(K >= 32 && K % 32 == 0 && K <= (1 << 24), "K must be a multiple of 32 in [32, 2^24] (got %d)", K);
    MOE_REQUIRE(rows >= 0 && rows <= (1 << 30), "rows must be in [0, 2^30] (got %d)", rows);
    MOE_REQUIRE(dtype_ok(out_dtype), "out_dtype must be MOE_F32, MOE_BF16 or MOE_F16 (got %d)", (int)out_dtype);
    MOE_REQUIRE(epilogue == MOE_MX4_PLAIN || epilogue == MOE_MX4_SWIGLU, "epilogue must be a moe_mx4_epilogue (got %d)",
                (int)epilogue);
    MOE_REQUIRE(offsets || E == 1, "offsets may be NULL for E = 1 only (got E=%d)", E);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(w_codes && w_scales && x_codes && x_scales && out, "NULL pointer");
    MOE_REQUIRE(aligned16(w_codes) && aligned16(w_scales) && aligned16(x_codes) && aligned16(x_scales),
                "codes and scales must be 16-byte aligned");
    MOE_REQUIRE(aligned_to(out, dtype_bytes(out_dtype)) && aligned_to(offsets, 4), "out and offsets must be aligned to their types");
    const bool swiglu = epilogue == MOE_MX4_SWIGLU;
    Params p = {};
    p.E = E, p.N = N, p.w_rows = swiglu ? 2 * N : N, p.rows = rows;
    p.nk = (K + BK - 1) / BK, p.n_mma = (K + 63) / 64;
    const int tn = swiglu ? BM / 2 : BM;
    p.n_tiles = (N + tn - 1) / tn;
    p.swiglu = swiglu;
    p.offsets = offsets, p.w_scales = w_scales, p.x_scales = x_scales, p.pitch = p.nk * 8;
    p.out = out, p.out_type = out_dtype, p.status = dev_status;
    // Rows per tile: what one group needs, twice the mean where there are
    // several (the groups' sizes are known on the device only).
    const int64_t groups = std::min(E, rows);
    const int64_t want = groups == 1 ? rows : 2 * ((rows + groups - 1) / groups);
    p.bn = (int)std::min<int64_t>(MAX_BN, (want + 31) / 32 * 32);
    const int stage = A_BYTES + p.bn * (BK / 2) + SF_BYTES;
    p.stages = std::min(MAX_STAGES, (200 * 1024) / stage);
    // at most this many items: every group's last row tile may be short
    const int64_t row_tiles = offsets ? groups + rows / p.bn : (rows + p.bn - 1) / p.bn;
    const int64_t items = row_tiles * p.n_tiles;
    // (item numbers stay in 32 bits whatever the offsets say)
    MOE_REQUIRE((int64_t)E * ((rows + p.bn - 1) / p.bn) * p.n_tiles <= (1 << 30), "too many tiles (rows=%d N=%d E=%d)", rows,
                N, E);
    const int sms = sm_count();
    p.splits = 1;
    while (p.splits < 8 && items * p.splits * 2 <= sms && p.nk >= 2 * p.splits) p.splits *= 2;
    const int64_t grid = p.splits > 1 ? items * p.splits : std::min<int64_t>(items, sms);
    const size_t smem = (size_t)p.stages * stage + 1024;
    CUtensorMap mw, mxm;
    moe_status st = make_tmap_bytes_3d(&mw, w_codes, E, p.w_rows, K / 2, swiglu ? 16 : BM);
    if (st == MOE_OK)
        st = make_tmap_2d(&mxm, x_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, K / 2, BK / 2, 32);
    if (st != MOE_OK) return st;
    MOE_CUDA_TRY(cudaFuncSetAttribute(mx4_matmul_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = to_cuda(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)p.splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.splits > 1 ? 1 : 0;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, mx4_matmul_kernel, p, mw, mxm));
    return check_launch("mx4_matmul");
}
