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
// (128-byte swizzle); warps 2..5 load the scales (32 bytes of a row are four
// steps) and put them into shared memory in the order that tcgen05.cp spreads
// over tensor memory (row r of a 128-row, 128-K chunk at byte (r % 32) * 16 +
// (r / 32) * 4); warp 1 issues the copies of the scales and four MMAs of K = 64;
// warps 6..13 take the sums out of tensor memory, two accumulators in turn.
//
// With SwiGLU a tile holds 64 gate rows and their 64 up rows, 16 of each in
// turn, so that both of a column's sums lie in one warp's lanes.
//
// Few items leave SMs idle while each reads its whole K, so K is split over a
// cluster of up to eight CTAs, which add their parts through distributed
// shared memory, in order.
//
// Measured: 81,920 rows x 2048 x 768 over 512 experts 127 us (797 MB, 6.3 TB/s: the
// weights' bytes bound it), SwiGLU of 768 x 2048 176 us (1,070 MB, 6.1 TB/s); 8192 x
// 8192 x 8192 191 us (5.8 PFLOP/s: shared memory, a step moves 44 KB in and out of
// it in 730 cycles); one row x 2048 x 2048 4.8 us (a launch, the set-up and eight
// steps of 0.3 us in turn).
//
// Every wait is bounded: after about 2 s the CTA records MOE_ERR_TIMEOUT and
// stops.
#include "cluster.cuh"
#include "dense_tc.cuh"
#include "rows.cuh"
#include "tc.cuh"

#include <type_traits>

namespace moe {
namespace mx {

constexpr int BM = 128;            // weight rows per tile
constexpr int BK = 256;            // K per step
constexpr int MAX_BN = 224;        // rows per tile: two accumulators and the scales fill tensor memory
constexpr int MAX_STAGES = 12, MAX_STAGE_BYTES = 200 * 1024;
constexpr int A_BYTES = BM * BK / 2;
constexpr int SF_BYTES = 2 * 512 + 4 * 512;  // scales of a step: weights, then rows (two chunks of 128 rows)
constexpr int SF_COL = 2 * MAX_BN;           // tensor memory columns of the scales (two sets of 32)
constexpr int SF_WARP0 = 2, SF_WARPS = 4;
constexpr int THREADS = 448;
constexpr int EPI_WARP0 = SF_WARP0 + SF_WARPS, EPI_WARPS = 8;  // two per quarter of the lanes: alone in its quarter a warp mostly waits
constexpr int MAX_E = 1024;
constexpr int STAGE_PITCH = 80;  // 32 16-bit columns and 16 bytes, so that eight rows fall into different banks
constexpr unsigned long long kWaitNs = 2000000000ull;

struct Params {
    int E, N, w_rows, rows;      // w_rows: weight rows per expert (N or 2N)
    int nk, n_mma;               // steps, and MMAs of K = 64, over the whole K
    int n_tiles, bn, stages, splits, swiglu;
    uint32_t tiles_m, tiles_shift, bn_m, bn_shift;  // reciprocals of n_tiles and bn
    const int32_t *offsets;      // NULL: one group of all rows
    int total;                   // its items
    const uint8_t *w_scales, *x_scales;
    int pitch;                   // bytes of scales per row, a multiple of 32: four steps
    void *out;
    int unit;  // bytes of the units that rows of out are made of: 16, 4 or 2
    int32_t *status;
};

struct Shared {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem;
    volatile int abort;
    int warp_tot[MAX_E / 128];
    int tile0[MAX_E + 1];  // row tiles before expert e
    int start[MAX_E], count[MAX_E];
    alignas(16) char stage[EPI_WARPS][16 * STAGE_PITCH];  // epilogue warps: 16 rows on their way out
};

// The value of lane 0, which the compiler then knows to be the same in the
// whole warp: descriptors and coordinates stay in uniform registers, which the
// TMA and tcgen05 instructions take.  (With values that might differ between
// lanes each such instruction cost 120 to 140 cycles to issue.)
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

struct Item {
    int e, p0, cnt;  // expert, first row, rows
    int n0;          // first output column
    int kb0, kb1;    // steps of this CTA
};

// x / d for x < 2^31: the high half of x m, shifted (m 0: d is 1).
__device__ __forceinline__ int quotient(int x, uint32_t m, uint32_t shift)
{
    return m ? (int)(__umulhi((uint32_t)x, m) >> shift) : x;
}

// The whole warp finds the last expert with tile0 <= tt: 32 ranges, then one.
__device__ __forceinline__ Item item_of(const Params &p, const Shared &S, int item, int split)
{
    Item it;
    const int lane = lane_id();
    const int tt = quotient(item, p.tiles_m, p.tiles_shift);
    it.n0 = (item - tt * p.n_tiles) * (p.swiglu ? BM / 2 : BM);
    if (!p.offsets) {  // bn is a tile's rows as they are
        it.e = 0;
        it.p0 = tt * p.bn;
        it.cnt = min(p.bn, p.rows - it.p0);
    } else {
        int e = __popc(__ballot_sync(0xffffffffu, lane * 32 < p.E && S.tile0[min(lane * 32, p.E)] <= tt)) - 1;
        e *= 32;
        e += __popc(__ballot_sync(0xffffffffu, e + lane < p.E && S.tile0[min(e + lane, p.E)] <= tt)) - 1;
        const int cnt = S.count[e], t0 = S.tile0[e], nt = S.tile0[e + 1] - t0;
        it.p0 = S.start[e];
        it.cnt = cnt;
        if (nt > 1) {
            const int w = ((cnt + nt - 1) / nt + 15) & ~15;
            it.p0 += (tt - t0) * w;
            it.cnt = min(w, cnt - (tt - t0) * w);
        }
        it.e = uniform(e);
        it.p0 = uniform(it.p0);
        it.cnt = uniform(it.cnt);
    }
    it.kb0 = 0;
    it.kb1 = p.nk;
    if (p.splits > 1) {
        it.kb0 = p.nk * split / p.splits;
        it.kb1 = p.nk * (split + 1) / p.splits;
    }
    return it;
}

// Whether the phase is complete now (try_wait may sleep for microseconds).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A whole warp waits; false for all of it when the time is up or the CTA stops.
__device__ __forceinline__ bool warp_wait(Shared &S, uint64_t *bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    const bool ok = tc::mbar_wait(bar, parity, kWaitNs);
    return __all_sync(0xffffffffu, ok && !S.abort);
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

// silu(g) u.  With t = e^-|g| <= 1 nothing overflows, and the quotient's
// divisor lies in [1, 2], where the fast one is within 2 ulp.  16-bit outputs take
// the fast exponential too (some 2^-21 relative for |g| < 8).
template <class O>
__device__ __forceinline__ float swiglu(float g, float u)
{
    const float t = O::kBytes == 4 ? expf(-fabsf(g)) : __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + t);
    return g * (g >= 0.f ? r : t * r) * u;
}

// 16 lanes x 16 columns: thread t gets lanes t/4 and t/4 + 8, of each group j of
// eight columns 2 (t%4) and the next: r[4j], r[4j+1] and r[4j+2], r[4j+3].
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, float (&r)[8])
{
    uint32_t u[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; i++) r[i] = __uint_as_float(u[i]);
}

// 32 lanes x 16 columns, a lane per thread.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, float (&r)[16])
{
    uint32_t u[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; i++) r[i] = __uint_as_float(u[i]);
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

template <class O>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t w;
    if (std::is_same<O, Bf16>::value) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// 16 staged rows of W columns to their place, in units that the rows' length and
// alignment allow (so a unit is in the matrix or past its edge as a whole).
template <class U, class T, int W, int P>
__device__ __forceinline__ void copy_out(T *out, int N, int n0, int rows, int lane, const char *stage)
{
    if constexpr (sizeof(U) >= sizeof(T)) {
        constexpr int E = sizeof(U) / sizeof(T), L = W / E, R = 32 / L;  // elements of a unit, lanes of a row, rows at once
        const int row0 = lane / L, col = (lane % L) * E, in = n0 + col < N ? min(rows, 16) : 0;
        T *o = out + (int64_t)row0 * N + n0 + col;
#pragma unroll
        for (int i = 0; i < 16; i += R, o += (int64_t)R * N)
            if (i + row0 < in) *reinterpret_cast<U *>(o) = *reinterpret_cast<const U *>(stage + (i + row0) * P + (lane % L) * sizeof(U));
    }
}

// Rows c .. c+15 of a tile, whose sums lie in columns of tensor memory from
// `taddr` on, a weight row per lane: this warp's 32 (SwiGLU: 16) output
// columns.  16-bit outputs are transposed in shared memory (stmatrix) and leave
// in pieces of 16 bytes, fp32 ones of SwiGLU too (from the registers they left in
// pieces of 32 bytes, at a third of the speed); other fp32 sums leave from the
// registers, a row's 128 bytes at once.
template <class O, bool kSwiglu>
__device__ __forceinline__ void write_rows(const Params &p, const Item &m, int q, int lane, uint32_t taddr, int c, char *stage)
{
    constexpr int W = kSwiglu ? 16 : 32;  // output columns of the warp
    using T = typename O::T;
    const int n0 = m.n0 + q * W, rows = m.cnt - c;
    T *out = static_cast<T *>(p.out) + (int64_t)(m.p0 + c) * p.N;
    __syncwarp();
    if (!kSwiglu && O::kBytes == 4) {  // a row's 32 columns are 128 bytes as they lie
        float v[16];
        tmem_ld_32x32b_x16(taddr, v);
        tc::tmem_ld_wait();
        const int in = n0 + lane < p.N ? rows : 0;
        T *o = out + n0 + lane;
#pragma unroll
        for (int i = 0; i < 16; i++, o += p.N)
            if (i < in) O::store(o, v[i]);
        return;
    }
    float a[8], b[8];
    tmem_ld_16x256b_x2(taddr, a);
    tmem_ld_16x256b_x2(taddr + (16u << 16), b);
    tc::tmem_ld_wait();
    if (kSwiglu) {
#pragma unroll
        for (int i = 0; i < 8; i++) a[i] = swiglu<O>(a[i], b[i]);
    }
    // (fp32 with SwiGLU: 16 columns are 64 bytes, a row of the staging block with 16 bytes between)
    constexpr int P = kSwiglu && O::kBytes == 2 ? 48 : STAGE_PITCH;
    if (O::kBytes == 4) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            *reinterpret_cast<float *>(stage + ((i >> 2) * 8 + 2 * (lane & 3) + (i & 1)) * P + (lane / 4 + (i & 2) * 4) * 4) = a[i];
    } else {
        const uint32_t base = tc::smem_u32(stage) + ((lane >> 4) * 8 + (lane & 7)) * P + ((lane >> 3) & 1) * 16;
        stmatrix_x4_trans(base, pack2<O>(a[0], a[1]), pack2<O>(a[2], a[3]), pack2<O>(a[4], a[5]), pack2<O>(a[6], a[7]));
        if (!kSwiglu)
            stmatrix_x4_trans(base + 32, pack2<O>(b[0], b[1]), pack2<O>(b[2], b[3]), pack2<O>(b[4], b[5]), pack2<O>(b[6], b[7]));
    }
    __syncwarp();
    if (p.unit == 16) copy_out<uint4, T, W, P>(out, p.N, n0, rows, lane, stage);
    else if (p.unit == 4) copy_out<uint32_t, T, W, P>(out, p.N, n0, rows, lane, stage);
    else copy_out<uint16_t, T, W, P>(out, p.N, n0, rows, lane, stage);
    __syncwarp();
}

// One row's sums of this warp's lanes (the parts of a cluster, added up).
template <class O, bool kSwiglu>
__device__ __forceinline__ void write_row(const Params &p, const Item &m, int q, int lane, int row, float v)
{
    typename O::T *out = static_cast<typename O::T *>(p.out) + (int64_t)(m.p0 + row) * p.N;
    if (!kSwiglu) {
        const int n = m.n0 + q * 32 + lane;
        if (n < p.N) O::store(out + n, v);
        return;
    }
    const float u = __shfl_down_sync(0xffffffffu, v, 16);  // lanes 0..15: gate, 16..31: the same columns' up
    const int n = m.n0 + q * 16 + lane;
    if (lane < 16 && n < p.N) O::store(out + n, swiglu<O>(v, u));
}

// 32 bytes (four steps) of a row's scales, or zeros.
__device__ __forceinline__ void load32(const uint8_t *src, bool in, uint32_t (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0;
    if (in)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(src));
}

// Groups of offsets that decrease or leave the rows: each begins no earlier than
// the one before it ends, so no row is in two of them, and their tiles are no
// more than good offsets' (which the launch counts on).  One thread, from the
// clipped starts in S.
__device__ __noinline__ void end_to_end(const Params &p, Shared &S)
{
    if (blockIdx.x == 0) set_status(p.status, MOE_ERR_BOUNDS);
    const int last = min(max(__ldg(p.offsets + p.E), 0), p.rows);
    int end = S.start[0], tiles = 0;
    for (int e = 0; e < p.E; e++) {
        const int next = max(end, e + 1 < p.E ? S.start[e + 1] : last);
        S.start[e] = end;
        S.count[e] = next - end;
        S.tile0[e] = tiles;
        tiles += quotient(next - end + p.bn - 1, p.bn_m, p.bn_shift);
        end = next;
    }
    S.tile0[p.E] = tiles;
}

template <class O, bool kSwiglu>
__global__ void __launch_bounds__(THREADS, 1) mx4_matmul_kernel(const __grid_constant__ Params p,
                                                                const __grid_constant__ CUtensorMap mw,
                                                                const __grid_constant__ CUtensorMap mx)
{
    extern __shared__ __align__(1024) char dyn_raw[];
    char *dyn = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    const int b_bytes = (p.bn + 31) / 32 * 32 * (BK / 2);
    char *sA = dyn, *sB = sA + p.stages * A_BYTES, *sF = sB + p.stages * b_bytes;
    __shared__ Shared S;
    const int warp = uniform(warp_id()), lane = lane_id();
    const int split = p.splits > 1 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / p.splits, step = gridDim.x / p.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; s++) {
            tc::mbar_init(&S.full[s], 1 + SF_WARPS);  // the producer's (with the bytes of its copies) and the scales'
            tc::mbar_init(&S.empty[s], 1);
        }
        for (int i = 0; i < 2; i++) {
            tc::mbar_init(&S.acc_full[i], 1);
            tc::mbar_init(&S.acc_empty[i], EPI_WARPS);
        }
        tc::mbar_init(&S.mma_done, 1);
        S.abort = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&mw);
        tc::tma_prefetch_desc(&mx);
    }
    if (warp == THREADS / 32 - 1) tc::tmem_alloc(&S.tmem, 512);
    // (launched while the kernel before it may still run: nothing above reads what that one writes)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // row tiles before each expert: four experts per thread, then a scan
    if (p.offsets && threadIdx.x < MAX_E / 4) {
        int off[5], n[4], sum = 0;
        bool bad = false;
        const int e0 = threadIdx.x * 4;
#pragma unroll
        for (int i = 0; i < 5; i++) off[i] = e0 + i <= p.E ? __ldg(p.offsets + e0 + i) : 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            // both ends clipped first, so that no offsets lead out of the rows
            const int a = min(max(off[i], 0), p.rows), b = min(max(off[i + 1], 0), p.rows);
            const int cnt = e0 + i < p.E ? max(0, b - a) : 0;
            if (e0 + i < p.E) {
                bad |= off[i] < 0 || off[i + 1] < off[i] || off[i + 1] > p.rows;
                S.start[e0 + i] = a;
                S.count[e0 + i] = cnt;
            }
            n[i] = sum;
            sum += quotient(cnt + p.bn - 1, p.bn_m, p.bn_shift);
        }
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) S.warp_tot[warp] = (int)incl;
        if (tc::named_sync_or(1, MAX_E / 4, bad)) {
            if (threadIdx.x == 0) end_to_end(p, S);
        } else {
            int base = (int)incl - sum;
            for (int i = 0; i < warp; i++) base += S.warp_tot[i];
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (e0 + i <= p.E) S.tile0[e0 + i] = base + n[i];
            if (p.E == MAX_E && e0 + 4 == MAX_E) S.tile0[MAX_E] = base + sum;
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)S.tmem);
    // (a cluster that splits K takes one item; the grid holds them all)
    const int tiles = p.offsets ? uniform(S.tile0[p.E]) * p.n_tiles : p.total;
    const int total = p.splits > 1 ? min(tiles, step) : tiles;

    if (warp == 0) {
        // ---------------- codes
        int it = 0, s = 0;
        uint32_t phase = 1;  // parity of the stage's use before this one
        bool ok = true;
        for (int item = first; item < total && ok; item += step) {
            const Item m = item_of(p, S, item, split);
            const int boxes = (m.cnt + 31) / 32;
            for (int kb = m.kb0; kb < m.kb1; kb++, it++) {
                if (it >= p.stages) ok = warp_wait(S, &S.empty[s], phase);
                if (!ok) break;
                if (elect_one()) {
                    tc::mbar_arrive_expect_tx(&S.full[s], A_BYTES + boxes * 32 * (BK / 2));
                    char *a = sA + s * A_BYTES, *b = sB + s * b_bytes;
                    const int x = kb * (BK / 2);
                    if (kSwiglu) {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            tma_load_3d(a + i * 16 * (BK / 2), &mw, x, (i & 1) * p.N + m.n0 + (i >> 1) * 16, m.e, &S.full[s]);
                    } else {
                        tma_load_3d(a, &mw, x, m.n0, m.e, &S.full[s]);
                    }
                    for (int i = 0; i < boxes; i++)
                        tc::tma_load_2d(b + i * 32 * (BK / 2), &mx, x, m.p0 + i * 32, &S.full[s]);
                }
                if (++s == p.stages) s = 0, phase ^= 1;
            }
        }
        if (lane == 0) {
            if (!ok) {
                set_status(p.status, MOE_ERR_TIMEOUT);
                S.abort = 1;
            }
            // no copy may still be in flight when the CTA leaves (after a
            // stop a barrier may lack its scales' arrivals: the copies
            // themselves land long before the shorter limit)
            for (int i = 0; i < p.stages && i < it; i++) {
                const int u = (it - 1 - i) / p.stages;
                if (!tc::mbar_wait(&S.full[i], u & 1, ok && !S.abort ? kWaitNs : kWaitNs / 100)) set_status(p.status, MOE_ERR_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA
        int it = 0, j = 0, s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int item = first; item < total && ok; item += step, j++) {
            const Item m = item_of(p, S, item, split);
            const int acc = j & 1, v = j >> 1;
            if (v > 0) ok = warp_wait(S, &S.acc_empty[acc], (v - 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            const int n16 = (m.cnt + 15) & ~15;
            const uint32_t d = tmem + (uint32_t)(acc * MAX_BN);
            const uint32_t id0 = idesc_mxf4(n16, 0), id2 = idesc_mxf4(n16, 2);
            bool ready = mbar_test(&S.full[s], phase);
            for (int kb = m.kb0; kb < m.kb1; kb++, it++) {
                if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(S, &S.full[s], phase);
                if (!ok) break;
                tc::tc_fence_after();
                // (the next step's answer comes while this one's instructions are issued)
                const int sn = s + 1 == p.stages ? 0 : s + 1;
                const uint32_t phase_n = sn ? phase : phase ^ 1;
                ready = mbar_test(&S.full[sn], phase_n);
                if (elect_one()) {
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
                    const int nm = p.n_mma - kb * 4;
#pragma unroll
                    for (int i = 0; i < 4; i++)  // 32 bytes of the swizzled rows per MMA
                        if (i < nm)
                            mma_mxf4(d, da + i * 2, db + i * 2, (i & 1) ? id2 : id0, sfa + (i >> 1) * 4, sfb + (i >> 1) * 8,
                                     (kb > m.kb0 || i > 0) ? 1u : 0u);
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
    } else if (warp < EPI_WARP0) {
        // ---------------- scales.  Warp k takes rows 32 g + 8 k + l of each
        // chunk of 128 (g the lane's low two bits, l the others): its 128 bytes
        // of the chunk then lie in a row.  Four steps' scales are one load per
        // row, and the next four are on their way while these are stored.
        const int k = warp - SF_WARP0, r = (lane & 3) * 32 + k * 8 + (lane >> 2);
        // (SwiGLU: row r of the tile is 16 of gate, 16 of up in turn)
        const int wr = kSwiglu ? (r >> 5) * 16 + (r & 15) : r, up = kSwiglu && (r & 16) ? p.N : 0;
        int item = first, base = 0, it = 0;
        Item m, mn;
        uint32_t cur[3][8], nxt[3][8];
        auto fetch = [&](const Item &q, int b, uint32_t (&v)[3][8]) {
            load32(p.w_scales + ((int64_t)q.e * p.w_rows + up + q.n0 + wr) * p.pitch + b * 8, q.n0 + wr < p.N, v[0]);
            load32(p.x_scales + (int64_t)(q.p0 + r) * p.pitch + b * 8, r < q.cnt, v[1]);
            load32(p.x_scales + (int64_t)(q.p0 + 128 + r) * p.pitch + b * 8, 128 + r < q.cnt, v[2]);
        };
        bool ok = item < total;
        if (ok) {
            m = item_of(p, S, item, split);
            base = m.kb0 & ~3;  // (a part of K may begin within the four)
            fetch(m, base, cur);
        }
        while (ok) {
            // the four steps after these
            int bn = base + 4;
            bool more = true;
            mn = m;
            if (bn >= m.kb1) {
                item += step;
                more = item < total;
                if (more) mn = item_of(p, S, item, split);
                bn = mn.kb0 & ~3;
            }
            if (more) fetch(mn, bn, nxt);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (base + i < m.kb0 || base + i >= m.kb1 || !ok) continue;
                const int s = it % p.stages, u = it / p.stages;
                it++;
                if (u > 0) ok = warp_wait(S, &S.empty[s], (u - 1) & 1);
                char *f = sF + s * SF_BYTES + k * 128 + lane * 4;
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    *reinterpret_cast<uint32_t *>(f + c * 512) = cur[0][2 * i + c];
                    *reinterpret_cast<uint32_t *>(f + 1024 + c * 1024) = cur[1][2 * i + c];
                    if (p.bn > 128) *reinterpret_cast<uint32_t *>(f + 1536 + c * 1024) = cur[2][2 * i + c];
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.full[s]);
            }
            if (!more) break;
            m = mn;
            base = bn;
#pragma unroll
            for (int j = 0; j < 3; j++)
#pragma unroll
                for (int i = 0; i < 8; i++) cur[j][i] = nxt[j][i];
        }
    } else {
        // ---------------- sums out
        const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;
        int j = 0;
        for (int item = first; item < total; item += step, j++) {
            const Item m = item_of(p, S, item, split);
            const int acc = j & 1, v = j >> 1;
            if (!warp_wait(S, &S.acc_full[acc], v & 1)) {
                if (lane == 0) set_status(p.status, MOE_ERR_TIMEOUT);
                S.abort = 1;
                break;
            }
            tc::tc_fence_after();
            const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * MAX_BN);
            if (p.splits == 1) {
#pragma unroll 1
                for (int c = half * 16; c < m.cnt; c += 32)
                    write_rows<O, kSwiglu>(p, m, q, lane, tbase + c, c, S.stage[warp - EPI_WARP0]);
            }
            for (int c = half * 16; p.splits > 1 && c < m.cnt; c += 32) {
                float r[16];
                __syncwarp();
                tmem_ld_32x32b_x16(tbase + c, r);
                tc::tmem_ld_wait();
                // every copy of this (only) item has been consumed: its stages hold the part now
                float *part = reinterpret_cast<float *>(dyn) + c * BM + q * 32 + lane;
#pragma unroll
                for (int i = 0; i < 16; i++)
                    if (c + i < m.cnt) part[i * BM] = r[i];
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.acc_empty[acc]);
        }
        if (p.offsets) {  // rows of no group: before the first and after the last
            const int z0 = S.start[p.E - 1] + S.count[p.E - 1];
            const int64_t rank = (int64_t)blockIdx.x * (EPI_WARPS * 32) + (threadIdx.x - EPI_WARP0 * 32);
            const int64_t threads = (int64_t)gridDim.x * (EPI_WARPS * 32);
            auto *out = static_cast<typename O::T *>(p.out);
            zero_bytes(out + (int64_t)z0 * p.N, (int64_t)(p.rows - z0) * p.N * O::kBytes, rank, threads);
            if (S.start[0]) zero_bytes(out, (int64_t)S.start[0] * p.N * O::kBytes, rank, threads);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == THREADS / 32 - 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (p.splits > 1) {
        // the cluster's parts, added in order; each CTA takes its share of the rows
        cluster_sync();
        if (warp >= EPI_WARP0 && first < total) {
            const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;
            const Item m = item_of(p, S, first, split);
            const int per = (m.cnt + p.splits - 1) / p.splits;  // rows of this CTA
            const int c1 = min(m.cnt, (split + 1) * per);
            for (int c = split * per + half; c < c1; c += 2) {
                const uint32_t a = tc::smem_u32(reinterpret_cast<float *>(dyn) + c * BM + q * 32 + lane);
                float v = 0.f;
                for (int r = 0; r < p.splits; r++) v += __uint_as_float(ld_cluster(a, r));
                write_row<O, kSwiglu>(p, m, q, lane, c, v);
            }
        }
        cluster_sync();  // no CTA leaves while another reads its part
    }
}

// m = floor(2^(31 + s) / d) + 1 with s = ceil(log2 d): x m is at most 2^31 2^s off
// 2^(31 + s) x / d, less than its next multiple.
static void reciprocal(int d, uint32_t *m, uint32_t *shift)
{
    uint32_t s = 0;
    while ((1ll << s) < d) s++;
    *m = s ? (uint32_t)((1ull << (31 + s)) / (uint32_t)d + 1) : 0;
    *shift = s ? s - 1 : 0;
}

// Rows per tile (a multiple of 16, at most MAX_BN).  Several groups: twice the
// mean, since their sizes are known on the device only (a larger group takes
// more tiles), but no more than what gives every SM a tile.
static int grouped_rows(int rows, int E, int n_tiles, int sms)
{
    const int64_t groups = std::min(E, rows), want = 2 * ((rows + groups - 1) / groups);
    const int64_t share = ((int64_t)rows * n_tiles + sms - 1) / sms;
    return (int)std::min<int64_t>(MAX_BN, (std::min(want, std::max<int64_t>(share, 32)) + 31) / 32 * 32);
}

// What a plan costs, in units of 10 ns (measured).  A step of 256 K takes 0.29 us
// with few rows (its instructions, one after the other), more when its bytes
// take longer: 0.39 us for 160 rows, 0.47 for 224.  A row leaves tensor memory
// in some 8 ns, hidden but for the last tile's.  Splitting K over s CTAs adds
// 1.8 us and 25 ns a row; a cluster needs its SMs in one group of them, and all
// clusters are to be there at once.  (One row, 2048 columns: K = 2048 takes 5.0 us
// whole and 5.1 in four parts, K = 8192 11.9 and 7.7; 16 items in eight parts 8.7.)
static int64_t plan_cost(int64_t items, int bn, int nk, int splits, int sms)
{
    if (splits > 1 && (splits > nk || items * splits > (splits < 8 ? sms - 24 : sms - 56))) return INT64_MAX;
    const int64_t rounds = (items + sms - 1) / sms, step = std::max(29, (BM + 24 + bn) / 8);
    return rounds * ((nk + splits - 1) / splits) * step + 4 * bn / 5 + 30 * rounds + (splits > 1 ? 180 + 5 * bn / 2 : 0);
}

// Rows per tile (one group) and CTAs per item.
static void plan_dense(int rows, int n_tiles, int nk, int sms, int *bn, int *splits)
{
    int64_t best = INT64_MAX;
    for (int b = MAX_BN; b >= 16; b -= 16) {
        if (b - 16 >= rows) continue;  // wider than the rows
        for (int s = 1; s <= 8; s *= 2) {
            const int64_t cost = plan_cost((int64_t)((rows + b - 1) / b) * n_tiles, b, nk, s, sms);
            if (cost < best) {
                best = cost;
                *bn = b;
                *splits = s;
            }
        }
    }
}

static int plan_splits(int64_t items, int bn, int nk, int sms)
{
    int best = 1;
    for (int s = 2; s <= 8; s *= 2)
        if (plan_cost(items, bn, nk, s, sms) < plan_cost(items, bn, nk, best, sms)) best = s;
    return best;
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
    MOE_REQUIRE(aligned16(w_codes) && aligned16(x_codes), "codes must be 16-byte aligned");
    MOE_REQUIRE(aligned_to(w_scales, 32) && aligned_to(x_scales, 32), "scales must be 32-byte aligned");
    MOE_REQUIRE(aligned_to(out, dtype_bytes(out_dtype)) && aligned_to(offsets, 4) && aligned_to(dev_status, 4),
                "out, offsets and dev_status must be aligned to their types");
    const bool swiglu = epilogue == MOE_MX4_SWIGLU;
    Params p = {};
    p.E = E, p.N = N, p.w_rows = swiglu ? 2 * N : N, p.rows = rows;
    p.nk = (K + BK - 1) / BK, p.n_mma = (K + 63) / 64;
    const int tn = swiglu ? BM / 2 : BM;
    p.n_tiles = (N + tn - 1) / tn;
    p.swiglu = swiglu;
    p.offsets = offsets, p.w_scales = w_scales, p.x_scales = x_scales, p.pitch = (p.nk + 3) / 4 * 32;
    p.out = out, p.status = dev_status;
    const int64_t row_bytes = (int64_t)N * dtype_bytes(out_dtype);
    p.unit = aligned16(out) && row_bytes % 16 == 0 ? 16 : aligned_to(out, 4) && row_bytes % 4 == 0 ? 4 : 2;
    const int sms = sm_count();
    p.splits = 0;
    if (offsets) p.bn = grouped_rows(rows, E, p.n_tiles, sms);
    else plan_dense(rows, p.n_tiles, p.nk, sms, &p.bn, &p.splits);
    const int stage = A_BYTES + (p.bn + 31) / 32 * 32 * (BK / 2) + SF_BYTES;
    p.stages = std::min(MAX_STAGES, MAX_STAGE_BYTES / stage);
    // at most this many items: every group's last row tile may be short
    const int64_t row_tiles = offsets ? std::min(E, rows) + rows / p.bn : (rows + p.bn - 1) / p.bn;
    const int64_t items = row_tiles * p.n_tiles;
    MOE_REQUIRE(items <= (1 << 30), "too many tiles (rows=%d N=%d E=%d)", rows, N, E);
    p.total = (int)items;
    reciprocal(p.n_tiles, &p.tiles_m, &p.tiles_shift);
    reciprocal(p.bn, &p.bn_m, &p.bn_shift);
    if (offsets) p.splits = plan_splits(items, std::min(p.bn, rows), p.nk, sms);
    const int64_t grid = p.splits > 1 ? items * p.splits : std::min<int64_t>(items, sms);
    const size_t smem = (size_t)p.stages * stage + 1024;
    CUtensorMap mw, mxm;
    moe_status st = make_tmap_bytes_3d(&mw, w_codes, E, p.w_rows, K / 2, swiglu ? 16 : BM);
    if (st == MOE_OK)
        st = make_tmap_2d(&mxm, x_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, K / 2, BK / 2, 32);
    if (st != MOE_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = to_cuda(stream);
    // The set-up overlaps the end of the kernel before (as a rule the one that quantised the rows).
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return with_dtype(out_dtype, [&](auto o) {
        using O = decltype(o);
        auto fn = swiglu ? mx4_matmul_kernel<O, true> : mx4_matmul_kernel<O, false>;
        // (the most that any call takes: calls of several threads do not undo each other's)
        MOE_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_STAGE_BYTES + 1024));
        MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, fn, p, mw, mxm));
        return check_launch("mx4_matmul");
    });
}
