// mx4.cu -- the microscaled 4-bit format (MXFP4): e2m1 codes, two to a byte,
// with one e8m0 scale byte per 32 values of a row.
//
// Both directions are one pass bound by memory: quantising reads a value once
// and writes 17/32 byte for it.  A thread takes eight values (four bytes of
// codes), four threads a block, whatever the rows' width: codes are one run
// over all rows, and the row that a block is in is a product with the width's
// reciprocal.  Each thread has two or four such pieces in flight, and a CTA takes
// no more than those (a grid of resident CTAs that loop was up to a fifth slower).
// 16-bit values find their largest magnitude two at a time: the conversion is
// otherwise bound by instructions.  Measured: 49,157 x 2208 fp32 quantised in 69
// us (7.2 TB/s), back to bf16 in 42 us (6.5 TB/s); 81,920 x 768 bf16 in 32 us (5.0
// TB/s).
#include "rows.cuh"

namespace moe {

constexpr int kMxThreads = 256, kQuantPieces = 2, kDequantPieces = 4;  // pieces in flight per thread

// Bytes of a row's scales: 32 for 1024 values, the unit the product loads.
__host__ __device__ constexpr int64_t mx4_pitch(int64_t cols) { return (cols + 1023) / 1024 * 32; }

// Eight values to e2m1 (nearest, ties to even, saturating at 6), the first in bits 0..3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float f)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0] * f), "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f), "f"(v[6] * f),
          "f"(v[7] * f));
    return r;
}

// fp32 bits of the largest magnitude of eight values as they lie; an infinity
// or a NaN is larger than any finite one.
__device__ __forceinline__ uint32_t abs_max(const F32::Raw8 &q)
{
    float v[8];
    F32::unpack8(q, v);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; k++) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ uint32_t abs_max16(const uint4 &q)
{
    const uint32_t m = __vmaxu2(__vmaxu2(q.x & 0x7fff7fffu, q.y & 0x7fff7fffu), __vmaxu2(q.z & 0x7fff7fffu, q.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}
template <class A>
__device__ __forceinline__ uint32_t block_max(const typename A::Raw8 &q);
template <>
__device__ __forceinline__ uint32_t block_max<F32>(const F32::Raw8 &q) { return abs_max(q); }
template <>
__device__ __forceinline__ uint32_t block_max<Bf16>(const uint4 &q) { return abs_max16(q) << 16; }
template <>
__device__ __forceinline__ uint32_t block_max<Fp16>(const uint4 &q) { return __float_as_uint(fp16_to_f32((uint16_t)abs_max16(q))); }

// The eight values of one piece, gathered where 16-byte loads cannot be used.
__device__ __forceinline__ F32::Raw8 gather8(const float *p)
{
    return {make_float4(p[0], p[1], p[2], p[3]), make_float4(p[4], p[5], p[6], p[7])};
}
__device__ __forceinline__ uint4 gather8(const uint16_t *p)
{
    return make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                      p[6] | (uint32_t)p[7] << 16);
}

// A launch takes fewer than 2^31 blocks of 32 values.  Block b is in row
// b / per_row: the high half of b times m = floor(2^(31 + s) / per_row) + 1, s =
// ceil(log2 per_row), shifted by s - 1 (b m is at most 2^31 2^s off 2^(31 + s) b
// / per_row, less than its next multiple).
struct Blocks {
    uint32_t total, per_row, m, shift;
    int pitch;
    __device__ __forceinline__ uint32_t row(uint32_t b) const { return per_row == 1 ? b : __umulhi(b, m) >> shift; }
};

// The block's exponent: e = floor(log2 m) - 2, at least -127; x 2^-e is exact,
// so each value is rounded once.
template <class A, bool kVec>
__global__ void __launch_bounds__(kMxThreads) mx4_quantise_kernel(const typename A::T *__restrict__ x, int64_t x_stride,
                                                                  Blocks n, uint8_t *__restrict__ codes,
                                                                  uint8_t *__restrict__ scales, int32_t *status)
{
    // A kernel that is launched to overlap this one (the product) may set itself up; it waits for the codes.
    asm volatile("griddepcontrol.launch_dependents;");
    // (the four threads of a block are in or out together)
    const uint32_t b0 = blockIdx.x * (kMxThreads / 4 * kQuantPieces) + threadIdx.x / 4, lane4 = threadIdx.x & 3;
    typename A::Raw8 q[kQuantPieces];
    uint32_t row[kQuantPieces], blk[kQuantPieces];
#pragma unroll
    for (int j = 0; j < kQuantPieces; j++) {
        const uint32_t b = b0 + j * (kMxThreads / 4);
        q[j] = {};
        if (b >= n.total) continue;
        row[j] = n.row(b);
        blk[j] = b - row[j] * n.per_row;
        const typename A::T *p = x + row[j] * x_stride + (blk[j] * 4 + lane4) * 8;
        if constexpr (kVec) q[j] = A::raw8(p);
        else q[j] = gather8(p);
    }
#pragma unroll
    for (int j = 0; j < kQuantPieces; j++) {
        const uint32_t b = b0 + j * (kMxThreads / 4);
        uint32_t m = block_max<A>(q[j]);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (b >= n.total) continue;
        const bool bad = m >= 0x7f800000u;
        const int byte = max((int)(m >> 23) - 2, 0);  // e + 127
        float v[8];
        A::unpack8(q[j], v);
        reinterpret_cast<uint32_t *>(codes)[(int64_t)b * 4 + lane4] =
            bad ? 0u : e2m1x8(v, __uint_as_float((uint32_t)(254 - byte) << 23));  // times 2^-e
        uint8_t *sc = scales + (int64_t)row[j] * n.pitch;
        if (lane4 == 0) {
            sc[blk[j]] = bad ? 255 : (uint8_t)byte;
            if (bad) set_status(status, MOE_ERR_NONFINITE);
        }
        if (blk[j] + 1 == n.per_row)  // the row's last block: the padding too
            for (int i = n.per_row + lane4; i < n.pitch; i += 4) sc[i] = 0;
    }
}

template <class A, bool kVec>
__global__ void __launch_bounds__(kMxThreads) mx4_dequantise_kernel(const uint8_t *__restrict__ codes,
                                                                    const uint8_t *__restrict__ scales, Blocks n,
                                                                    typename A::T *__restrict__ out)
{
    const uint32_t b0 = blockIdx.x * (kMxThreads / 4 * kDequantPieces) + threadIdx.x / 4, lane4 = threadIdx.x & 3;
    uint32_t q[kDequantPieces], byte[kDequantPieces];
#pragma unroll
    for (int j = 0; j < kDequantPieces; j++) {
        const uint32_t b = b0 + j * (kMxThreads / 4);
        if (b >= n.total) continue;
        const uint32_t row = n.row(b);
        q[j] = reinterpret_cast<const uint32_t *>(codes)[(int64_t)b * 4 + lane4];
        byte[j] = scales[(int64_t)row * n.pitch + (b - row * n.per_row)];
    }
#pragma unroll
    for (int j = 0; j < kDequantPieces; j++) {
        const uint32_t b = b0 + j * (kMxThreads / 4);
        if (b >= n.total) continue;
        const float f = byte[j] == 255u ? __uint_as_float(0x7fffffffu)
                                        : __uint_as_float(byte[j] ? byte[j] << 23 : 0x00400000u);
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            uint32_t h;
            asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(q[j] >> (8 * k)));
            v[2 * k] = fp16_to_f32((uint16_t)(h & 0xffffu)) * f;
            v[2 * k + 1] = fp16_to_f32((uint16_t)(h >> 16)) * f;
        }
        typename A::T *o = out + ((int64_t)b * 4 + lane4) * 8;
        if (kVec) {
            A::store8(o, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) A::store(o + k, v[k]);
        }
    }
}

static Blocks mx_blocks(int64_t rows, int64_t cols)
{
    Blocks n = {};
    n.per_row = (uint32_t)(cols / 32);
    n.total = (uint32_t)(rows * n.per_row);
    n.pitch = (int)mx4_pitch(cols);
    uint32_t s = 0;
    while ((1u << s) < n.per_row) s++;
    if (s > 0) {
        n.m = (uint32_t)((1ull << (31 + s)) / n.per_row + 1);
        n.shift = s - 1;
    }
    return n;
}

// Runs f(first row, blocks, grid) over ranges of fewer than 2^31 blocks.
template <class F>
static moe_status mx_ranges(int64_t rows, int64_t cols, int pieces, F f)
{
    const int64_t most = ((1ll << 31) - 1) / (cols / 32);
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t k = std::min(most, rows - r);
        const Blocks n = mx_blocks(k, cols);
        moe_status st = f(r, n, (unsigned)(((int64_t)n.total + kMxThreads / 4 * pieces - 1) / (kMxThreads / 4 * pieces)));
        if (st != MOE_OK) return st;
    }
    return MOE_OK;
}

static moe_status check_mx(int64_t rows, int64_t cols)
{
    MOE_REQUIRE(rows >= 0 && cols >= 32 && cols % 32 == 0 && cols <= (1 << 24),
                "rows >= 0 and cols a multiple of 32 in [32, 2^24] (got rows=%lld cols=%lld)", (long long)rows,
                (long long)cols);
    MOE_REQUIRE(rows <= (1ll << 45) / cols, "too many values (rows=%lld cols=%lld)", (long long)rows, (long long)cols);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mx4_size(int64_t rows, int64_t cols, size_t *code_bytes, size_t *scale_bytes)
{
    moe_status st = check_mx(rows, cols);
    if (st != MOE_OK) return st;
    if (code_bytes) *code_bytes = (size_t)(rows * (cols / 2));
    if (scale_bytes) *scale_bytes = (size_t)(rows * mx4_pitch(cols));
    return MOE_OK;
}

extern "C" moe_status moe_mx4_quantise(const void *x, moe_dtype dtype, int64_t x_stride, int64_t rows, int64_t cols,
                                       uint8_t *codes, uint8_t *scales, int32_t *dev_status, moe_stream_t stream)
{
    moe_status st = check_mx(rows, cols);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(dtype_ok(dtype), "dtype must be MOE_F32, MOE_BF16 or MOE_F16 (got %d)", (int)dtype);
    MOE_REQUIRE(x_stride == 0 || x_stride >= cols, "x_stride must be 0 or >= cols (got %lld, cols=%lld)",
                (long long)x_stride, (long long)cols);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(x && codes && scales, "NULL pointer");
    MOE_REQUIRE(aligned16(codes) && aligned_to(scales, 32), "codes must be 16-byte, scales 32-byte aligned");
    MOE_REQUIRE(aligned_to(x, dtype_bytes(dtype)) && aligned_to(dev_status, 4), "x and dev_status must be aligned to their types");
    const bool vec = aligned16(x) && (x_stride * dtype_bytes(dtype)) % 16 == 0;
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto fn = vec ? mx4_quantise_kernel<A, true> : mx4_quantise_kernel<A, false>;
        return mx_ranges(rows, cols, kQuantPieces, [&](int64_t r, const Blocks &n, unsigned grid) {
            fn<<<grid, kMxThreads, 0, to_cuda(stream)>>>(static_cast<const typename A::T *>(x) + r * x_stride, x_stride, n,
                                                         codes + r * (cols / 2), scales + r * mx4_pitch(cols), dev_status);
            return check_launch("mx4_quantise");
        });
    });
}

extern "C" moe_status moe_mx4_dequantise(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                                         void *out, moe_dtype dtype, moe_stream_t stream)
{
    moe_status st = check_mx(rows, cols);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(dtype_ok(dtype), "dtype must be MOE_F32, MOE_BF16 or MOE_F16 (got %d)", (int)dtype);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes && scales && out, "NULL pointer");
    MOE_REQUIRE(aligned16(codes) && aligned_to(scales, 32), "codes must be 16-byte, scales 32-byte aligned");
    MOE_REQUIRE(aligned_to(out, dtype_bytes(dtype)), "out must be aligned to its type");
    const bool vec = aligned16(out);
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto fn = vec ? mx4_dequantise_kernel<A, true> : mx4_dequantise_kernel<A, false>;
        return mx_ranges(rows, cols, kDequantPieces, [&](int64_t r, const Blocks &n, unsigned grid) {
            fn<<<grid, kMxThreads, 0, to_cuda(stream)>>>(codes + r * (cols / 2), scales + r * mx4_pitch(cols), n,
                                                         static_cast<typename A::T *>(out) + r * cols);
            return check_launch("mx4_dequantise");
        });
    });
}
