// rows.cu -- moe_dispatch, moe_combine and their gradients: token rows copied
// to their pairs' places in expert order, and the pairs' rows summed back.
//
// All four are bound by memory: a pair row crosses HBM once (written by
// dispatch, read by combine), a token row once.  The kernels walk tokens, not
// pairs: a warp takes one piece of one token's row and all k of its pairs, so
// the token's bytes are read (or summed) once and no atomics are needed.
// Measured, 2048 bf16 columns, ten places a token: dispatch of 32,768 tokens 220
// us (6.7 TB/s), combine 236 us (6.3 TB/s), combine's gradient for 8,192 tokens
// 106 us (6.7 TB/s).
#include "rows.cuh"

namespace moe {

constexpr int kRowThreads = 256;
// CTAs per SM that the kernels are built for.  combine's grid is that many, and
// a CTA takes several pieces; dispatch, which mostly writes, is faster with a
// CTA per eight pieces (32K tokens of 4 KB, ten places each: 220 against 250
// us), and combine's gradient with some (106 against 113 us at 8192 tokens).
// combine: more CTAs with a row or two on their way per lane each do better
// than fewer with four or five (16-bit rows: 64 against 83 us at 8192 tokens).
constexpr int kDispatchPerSm = 6, kBackPerSm = 4, kBackGrid = 32;
constexpr int combine_per_sm(int bytes, int unit) { return bytes == 2 && unit == 2 ? 6 : 8; }  // (63 against 97 us with eight, 2046 columns)
constexpr int kMaxK = 16;

// inv_perm of a token's slot (lane j of the warp), -1 for left-out pairs; an
// entry outside [0, n_pairs) counts as left out.
__device__ __forceinline__ int32_t pair_row(const int32_t *inv, int64_t t, int k, int64_t n_pairs, int lane)
{
    int32_t p = lane < k ? inv[t * k + lane] : -1;
    return p >= 0 && p < n_pairs ? p : -1;
}

__device__ __forceinline__ int64_t first_tail_row(const int32_t *offsets, int E, int64_t n_pairs)
{
    int64_t n = offsets[E];
    return n < 0 ? 0 : (n > n_pairs ? n_pairs : n);
}

// ---------------------------------------------------------------- dispatch
// A copy, whatever the type: V is the widest unit that row bytes and pointers
// allow.  Unit of work: kUnroll * 32 V's of one token's row, to its k places.
template <class V, int kUnroll>
__global__ void __launch_bounds__(kRowThreads, kDispatchPerSm) dispatch_kernel(const V *__restrict__ x, int64_t x_stride, int64_t T,
                                                               int row, int k, int E,
                                                               const int32_t *__restrict__ offsets,
                                                               const int32_t *__restrict__ inv, V *__restrict__ out)
{
    const int lane = lane_id();
    const int pieces = (row + 32 * kUnroll - 1) / (32 * kUnroll);
    const int64_t n_pairs = T * k, units = T * pieces;
    const int64_t w0 = (int64_t)blockIdx.x * (kRowThreads / 32) + warp_id(), wn = (int64_t)gridDim.x * (kRowThreads / 32);
    for (int64_t u = w0; u < units; u += wn) {
        const int64_t t = u / pieces;
        const int c0 = (int)(u % pieces) * 32 * kUnroll + lane;
        const int32_t p = pair_row(inv, t, k, n_pairs, lane);
        V v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; i++)
            if (c0 + 32 * i < row) v[i] = x[t * x_stride + c0 + 32 * i];
        for (int j = 0; j < k; j++) {
            const int32_t r = __shfl_sync(0xffffffffu, p, j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < kUnroll; i++)
                if (c0 + 32 * i < row) out[(int64_t)r * row + c0 + 32 * i] = v[i];
        }
    }
    // rows of no pair
    const int64_t z0 = first_tail_row(offsets, E, n_pairs);
    zero_bytes(out + z0 * row, (n_pairs - z0) * row * (int64_t)sizeof(V), w0 * 32 + lane, wn * 32);
}

// ---------------------------------------------------------------- combine
// out[t] = (out[t]) + sum_j w[t][j] y[inv[t][j]] in slot order, fp32 sums,
// one rounding at the end.  Unit of work: 256 columns of one token, eight per
// lane, in accesses of kUnit columns (8, or 2 or 1 where rows are not aligned).
// kBatch rows are on their way per lane: one where the pieces fill the GPU
// (more CTAs do better than more loads each), several where few warps run and
// each waits for its rows in turn otherwise.
template <class A, class O, int kUnit, int kBatch>
__global__ void __launch_bounds__(kRowThreads, kBatch == 1 ? combine_per_sm(A::kBytes, kUnit) : 2)
    combine_kernel(const typename A::T *__restrict__ y, int64_t T, int H, int k, const float *__restrict__ w,
                   const int32_t *__restrict__ inv, typename O::T *__restrict__ out, int accumulate)
{
    using UA = Unit<A, kUnit>;
    using UO = Unit<O, kUnit>;
    constexpr int P = 8 / kUnit;
    const int lane = lane_id();
    const int pieces = (H + 255) / 256;
    const int64_t n_pairs = T * k, units = T * pieces;
    const int64_t w0 = (int64_t)blockIdx.x * (kRowThreads / 32) + warp_id(), wn = (int64_t)gridDim.x * (kRowThreads / 32);
    for (int64_t u = w0; u < units; u += wn) {
        const int64_t t = u / pieces;
        const int32_t p = pair_row(inv, t, k, n_pairs, lane);
        const float f = w && lane < k ? w[t * k + lane] : 1.0f;
        const int c = (int)(u % pieces) * 256 + lane * kUnit;  // and every 32 kUnit from there
        float acc[P][kUnit] = {};
        typename O::T *o = out + t * H + c;
        if (accumulate) {
#pragma unroll
            for (int i = 0; i < P; i++)
                if (c + i * 32 * kUnit < H) UO::unpack(UO::raw(o + i * 32 * kUnit), acc[i]);
        }
        if constexpr (kBatch == 1) {
            for (int j = 0; j < k; j++) {
                const int32_t r = __shfl_sync(0xffffffffu, p, j);
                const float g = __shfl_sync(0xffffffffu, f, j);
                if (r < 0) continue;
                const typename A::T *row = y + (int64_t)r * H + c;
#pragma unroll
                for (int i = 0; i < P; i++) {
                    if (c + i * 32 * kUnit >= H) continue;
                    float v[kUnit];
                    UA::unpack(UA::raw(row + i * 32 * kUnit), v);
#pragma unroll
                    for (int e = 0; e < kUnit; e++) acc[i][e] = fmaf(g, v[e], acc[i][e]);
                }
            }
        }
        for (int j0 = 0; kBatch > 1 && j0 < k; j0 += kBatch) {
            typename UA::Raw q[kBatch][P];
            int32_t r[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; j++) {  // (lanes from k on hold -1)
                r[j] = __shfl_sync(0xffffffffu, p, min(j0 + j, 31));
                const typename A::T *row = y + (int64_t)r[j] * H + c;
#pragma unroll
                for (int i = 0; i < P; i++)
                    if (r[j] >= 0 && c + i * 32 * kUnit < H) q[j][i] = UA::raw(row + i * 32 * kUnit);
            }
#pragma unroll
            for (int j = 0; j < kBatch; j++) {
                const float g = __shfl_sync(0xffffffffu, f, min(j0 + j, 31));
                if (r[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < P; i++) {
                    if (c + i * 32 * kUnit >= H) break;
                    float v[kUnit];
                    UA::unpack(q[j][i], v);
#pragma unroll
                    for (int e = 0; e < kUnit; e++) acc[i][e] = fmaf(g, v[e], acc[i][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < P; i++)
            if (c + i * 32 * kUnit < H) UO::store(o + i * 32 * kUnit, acc[i]);
    }
}

// ---------------------------------------------------------------- combine's gradients
// One warp per (token, slot): dy[inv] = w dout[t] and dw = <dout[t], y[inv]>,
// the dot product in fp32 (lane sums over strided pieces, then a fixed tree).
template <class A, int kUnit>
__global__ void __launch_bounds__(kRowThreads, kBackPerSm) combine_backward_kernel(
    const typename A::T *__restrict__ dout, const typename A::T *__restrict__ y, int64_t T, int H, int k, int E,
    const int32_t *__restrict__ offsets, const float *__restrict__ w, const int32_t *__restrict__ inv,
    typename A::T *__restrict__ dy, float *__restrict__ dw)
{
    using U = Unit<A, kUnit>;
    constexpr int kBatch = kUnit < 8 ? 8 : A::kBytes == 2 ? 4 : 2;  // accesses of both rows on their way per lane
    const int lane = lane_id();
    const int64_t n_pairs = T * k;
    const int64_t w0 = (int64_t)blockIdx.x * (kRowThreads / 32) + warp_id(), wn = (int64_t)gridDim.x * (kRowThreads / 32);
    for (int64_t q = w0; q < n_pairs; q += wn) {
        const int32_t r = inv[q];
        if (r < 0 || r >= n_pairs) {
            if (lane == 0) dw[q] = 0.f;
            continue;
        }
        const float f = w[q];
        const typename A::T *d = dout + q / k * H, *yr = y + (int64_t)r * H;
        typename A::T *o = dy + (int64_t)r * H;
        float sum = 0.f;
        for (int c0 = lane * kUnit; c0 < H; c0 += kBatch * 32 * kUnit) {
            typename U::Raw dq[kBatch], yq[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (c0 + i * 32 * kUnit < H) {
                    yq[i] = U::raw(yr + c0 + i * 32 * kUnit);
                    dq[i] = U::raw(d + c0 + i * 32 * kUnit);
                }
#pragma unroll
            for (int i = 0; i < kBatch; i++) {
                if (c0 + i * 32 * kUnit >= H) break;
                float a[kUnit], b[kUnit];
                U::unpack(dq[i], a);
                U::unpack(yq[i], b);
#pragma unroll
                for (int e = 0; e < kUnit; e++) {
                    sum = fmaf(a[e], b[e], sum);
                    a[e] *= f;
                }
                U::store(o + c0 + i * 32 * kUnit, a);
            }
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) dw[q] = sum;
    }
    const int64_t z0 = first_tail_row(offsets, E, n_pairs);
    zero_bytes(dy + z0 * H, (n_pairs - z0) * H * A::kBytes, w0 * 32 + lane, wn * 32);
}

static unsigned row_grid(int64_t warps, int per_sm)
{
    const int64_t blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)sm_count() * per_sm));
}

// Elements per access that rows of H allow from p on: 8, 2 or 1.
static int row_unit(moe_dtype t, int H, const void *p)
{
    return H % 8 == 0 && aligned16(p) ? 8 : H % 2 == 0 && aligned_to(p, 2 * dtype_bytes(t)) ? 2 : 1;
}

static moe_status check_rows(int T, int H, int k, moe_dtype dtype)
{
    MOE_REQUIRE(T >= 0 && H >= 1 && H <= (1 << 24) && k >= 1 && k <= kMaxK,
                "T >= 0, H in [1, 2^24] and 1 <= k <= %d (got T=%d H=%d k=%d)", kMaxK, T, H, k);
    MOE_REQUIRE((int64_t)T * k <= INT32_MAX, "T*k too large (T=%d k=%d)", T, k);
    MOE_REQUIRE(dtype_ok(dtype), "dtype must be MOE_F32, MOE_BF16 or MOE_F16 (got %d)", (int)dtype);
    return MOE_OK;
}

template <class V>
static void launch_dispatch(const void *x, int64_t stride_bytes, int T, int64_t row_bytes, int k, int E,
                            const int32_t *offsets, const int32_t *inv, void *out, cudaStream_t s)
{
    const int row = (int)(row_bytes / (int64_t)sizeof(V));
    const int64_t units = (int64_t)T * ((row + 127) / 128);
    const unsigned grid = (unsigned)std::min<int64_t>((units + kRowThreads / 32 - 1) / (kRowThreads / 32), INT32_MAX);
    dispatch_kernel<V, 4><<<grid, kRowThreads, 0, s>>>(static_cast<const V *>(x),
                                                                  stride_bytes / (int64_t)sizeof(V), T, row, k, E,
                                                                  offsets, inv, static_cast<V *>(out));
}

static moe_status combine_any(const void *y, moe_dtype dtype, int T, int H, int k, const float *w,
                              const int32_t *inv, void *out, moe_dtype out_dtype, int accumulate, cudaStream_t s,
                              const char *what)
{
    const int unit = std::min(row_unit(dtype, H, y), row_unit(out_dtype, H, out));
    const int64_t pieces = (int64_t)T * ((H + 255) / 256);
    const unsigned grid = row_grid(pieces, combine_per_sm(dtype_bytes(dtype), unit));
    // (ten bf16 rows of 2048 columns: 3.6 against 4.4 us at 256 tokens, 5.6 against 5.0 at 512)
    const bool few = pieces <= (int64_t)sm_count() * 16;
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto go = [&](auto o) {
            using O = decltype(o);
            auto *yp = static_cast<const typename A::T *>(y);
            auto *op = static_cast<typename O::T *>(out);
            auto fn = unit == 1 ? combine_kernel<A, O, 1, 1> : unit == 2 ? combine_kernel<A, O, 2, 1>
                      : few ? combine_kernel<A, O, 8, 5> : combine_kernel<A, O, 8, 1>;
            fn<<<grid, kRowThreads, 0, s>>>(yp, T, H, k, w, inv, op, accumulate);
            return check_launch(what);
        };
        return out_dtype == dtype ? go(a) : go(F32{});
    });
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_dispatch(const void *x, moe_dtype dtype, int64_t x_stride, int T, int H, int k, int E,
                                   const int32_t *offsets, const int32_t *inv_perm, void *out, moe_stream_t stream)
{
    moe_status st = check_rows(T, H, k, dtype);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(E >= 1 && E <= 1024, "E must be in [1, 1024] (got %d)", E);
    MOE_REQUIRE(x_stride == 0 || x_stride >= H, "x_stride must be 0 (one row for every token) or >= H (got %lld, H=%d)",
                (long long)x_stride, H);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && offsets && inv_perm && out, "NULL pointer");
    const int b = dtype_bytes(dtype);
    const int64_t rb = (int64_t)H * b, sb = x_stride * b;
    MOE_REQUIRE(aligned_to(x, b) && aligned_to(out, b) && aligned_to(offsets, 4) && aligned_to(inv_perm, 4),
                "x, out, offsets and inv_perm must be aligned to their types");
    cudaStream_t s = to_cuda(stream);
    if (rb % 16 == 0 && sb % 16 == 0 && aligned16(x) && aligned16(out))
        launch_dispatch<uint4>(x, sb, T, rb, k, E, offsets, inv_perm, out, s);
    else if (rb % 4 == 0 && sb % 4 == 0 && aligned_to(x, 4) && aligned_to(out, 4))
        launch_dispatch<uint32_t>(x, sb, T, rb, k, E, offsets, inv_perm, out, s);
    else
        launch_dispatch<uint16_t>(x, sb, T, rb, k, E, offsets, inv_perm, out, s);
    return check_launch("dispatch");
}

extern "C" moe_status moe_dispatch_backward(const void *drows, moe_dtype dtype, int T, int H, int k,
                                            const int32_t *inv_perm, void *dx, moe_stream_t stream)
{
    moe_status st = check_rows(T, H, k, dtype);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(drows && inv_perm && dx, "NULL pointer");
    MOE_REQUIRE(aligned_to(drows, dtype_bytes(dtype)) && aligned_to(dx, dtype_bytes(dtype)) && aligned_to(inv_perm, 4),
                "drows, dx and inv_perm must be aligned to their types");
    return combine_any(drows, dtype, T, H, k, nullptr, inv_perm, dx, dtype, 0, to_cuda(stream), "dispatch_backward");
}

extern "C" moe_status moe_combine(const void *y, moe_dtype dtype, int T, int H, int k, const float *w,
                                  const int32_t *inv_perm, void *out, moe_dtype out_dtype, int accumulate,
                                  moe_stream_t stream)
{
    moe_status st = check_rows(T, H, k, dtype);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(out_dtype == dtype || out_dtype == MOE_F32, "out_dtype must be MOE_F32 or the rows' type (got %d, %d)",
                (int)out_dtype, (int)dtype);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(y && w && inv_perm && out, "NULL pointer");
    MOE_REQUIRE(aligned_to(y, dtype_bytes(dtype)) && aligned_to(out, dtype_bytes(out_dtype)) && aligned_to(w, 4) &&
                    aligned_to(inv_perm, 4),
                "y, out, w and inv_perm must be aligned to their types");
    return combine_any(y, dtype, T, H, k, w, inv_perm, out, out_dtype, accumulate, to_cuda(stream), "combine");
}

extern "C" moe_status moe_combine_backward(const void *dout, const void *y, moe_dtype dtype, int T, int H, int k, int E,
                                           const int32_t *offsets, const float *w, const int32_t *inv_perm, void *dy,
                                           float *dw, moe_stream_t stream)
{
    moe_status st = check_rows(T, H, k, dtype);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(E >= 1 && E <= 1024, "E must be in [1, 1024] (got %d)", E);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(dout && y && offsets && w && inv_perm && dy && dw, "NULL pointer");
    MOE_REQUIRE(aligned_to(dout, dtype_bytes(dtype)) && aligned_to(y, dtype_bytes(dtype)) &&
                    aligned_to(dy, dtype_bytes(dtype)) && aligned_to(offsets, 4) && aligned_to(w, 4) &&
                    aligned_to(inv_perm, 4) && aligned_to(dw, 4),
                "dout, y, dy, offsets, w, inv_perm and dw must be aligned to their types");
    const unsigned grid = row_grid((int64_t)T * k, kBackGrid);
    const int unit = std::min(std::min(row_unit(dtype, H, dout), row_unit(dtype, H, y)), row_unit(dtype, H, dy));
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        using E1 = typename A::T;
        auto fn = unit == 8 ? combine_backward_kernel<A, 8> : unit == 2 ? combine_backward_kernel<A, 2> : combine_backward_kernel<A, 1>;
        fn<<<grid, kRowThreads, 0, to_cuda(stream)>>>(static_cast<const E1 *>(dout), static_cast<const E1 *>(y), T, H, k,
                                                      E, offsets, w, inv_perm, static_cast<E1 *>(dy), dw);
        return check_launch("combine_backward");
    });
}
