// mx4.cu -- the microscaled 4-bit format (MXFP4): e2m1 codes, two to a byte,
// with one e8m0 scale byte per 32 values of a row.
//
// Both directions are one pass bound by memory: quantising reads a value once
// and writes 17/32 byte for it.  A warp takes 256 columns of a row (eight
// values per lane, a block per four lanes), eight bytes of the row's scales;
// the last one of a row also clears the scales' padding.
#include "rows.cuh"

namespace moe {

constexpr int kMxThreads = 256;

// Bytes of a row's scales: 32 for 1024 values, the unit the product loads.
__host__ __device__ constexpr int64_t mx4_pitch(int64_t cols) { return (cols + 1023) / 1024 * 32; }

// Two fp32 values to e2m1 (nearest, ties to even, saturating at 6): lo in bits 0..3.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// Unit u = 256 columns of a row.  The block's exponent comes from the bits of
// its largest magnitude (an integer maximum, so an infinity or a NaN wins and
// marks the block): e = floor(log2 m) - 2, at least -127; x 2^-e is exact, so
// each value is rounded once.
template <class A, bool kVec>
__global__ void __launch_bounds__(kMxThreads) mx4_quantise_kernel(const typename A::T *__restrict__ x, int64_t x_stride,
                                                                  int64_t rows, int cols, uint8_t *__restrict__ codes,
                                                                  uint8_t *__restrict__ scales, int32_t *status)
{
    const int lane = lane_id();
    const int groups = (cols + 255) / 256;
    const int64_t units = rows * groups;
    const int64_t w0 = (int64_t)blockIdx.x * (kMxThreads / 32) + warp_id(), wn = (int64_t)gridDim.x * (kMxThreads / 32);
    for (int64_t u = w0; u < units; u += wn) {
        const int64_t r = u / groups;
        const int g = (int)(u % groups);
        const int c = g * 256 + lane * 8;
        float v[8] = {};
        if (c < cols) {
            const typename A::T *p = x + r * x_stride + c;
            if (kVec) {
                A::load8(p, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = A::load(p + i);
            }
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const bool bad = m >= 0x7f800000u;
        const int byte = max((int)(m >> 23) - 2, 0);  // e + 127
        const float f = __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^-e
        uint32_t q = 0;
        if (!bad) {
#pragma unroll
            for (int i = 0; i < 4; i++) q |= e2m1x2(v[2 * i] * f, v[2 * i + 1] * f) << (8 * i);
        }
        if (c < cols) *reinterpret_cast<uint32_t *>(codes + r * (cols / 2) + c / 2) = q;
        if (bad && (lane & 3) == 0) set_status(status, MOE_ERR_NONFINITE);
        uint8_t *sc = scales + r * mx4_pitch(cols);
        if ((lane & 3) == 0) sc[g * 8 + lane / 4] = bad ? 255 : (uint8_t)byte;
        if (g == groups - 1 && (groups + lane) * 8 < mx4_pitch(cols)) *reinterpret_cast<uint2 *>(sc + (groups + lane) * 8) = make_uint2(0, 0);
    }
}

template <class A, bool kVec>
__global__ void __launch_bounds__(kMxThreads) mx4_dequantise_kernel(const uint8_t *__restrict__ codes,
                                                                    const uint8_t *__restrict__ scales, int64_t rows,
                                                                    int cols, typename A::T *__restrict__ out)
{
    const int lane = lane_id();
    const int groups = (cols + 255) / 256;
    const int64_t units = rows * groups;
    const int64_t w0 = (int64_t)blockIdx.x * (kMxThreads / 32) + warp_id(), wn = (int64_t)gridDim.x * (kMxThreads / 32);
    for (int64_t u = w0; u < units; u += wn) {
        const int64_t r = u / groups;
        const int c = (int)(u % groups) * 256 + lane * 8;
        if (c >= cols) continue;
        const uint32_t q = *reinterpret_cast<const uint32_t *>(codes + r * (cols / 2) + c / 2);
        const uint32_t byte = scales[r * mx4_pitch(cols) + c / 32];
        const float f = byte == 255u ? __uint_as_float(0x7fffffffu) : byte ? __uint_as_float(byte << 23)
                                                                             : __uint_as_float(0x00400000u);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t h;
            asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(q >> (8 * i)));
            v[2 * i] = fp16_to_f32((uint16_t)(h & 0xffffu)) * f;
            v[2 * i + 1] = fp16_to_f32((uint16_t)(h >> 16)) * f;
        }
        typename A::T *o = out + r * cols + c;
        if (kVec) {
            A::store8(o, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) A::store(o + i, v[i]);
        }
    }
}

static unsigned mx_grid(int64_t units)
{
    const int64_t blocks = (units + kMxThreads / 32 - 1) / (kMxThreads / 32);
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)sm_count() * 8));
}

static moe_status check_mx(int64_t rows, int64_t cols)
{
    MOE_REQUIRE(rows >= 0 && cols >= 32 && cols % 32 == 0 && cols <= (1 << 24),
                "rows >= 0 and cols a multiple of 32 in [32, 2^24] (got rows=%lld cols=%lld)", (long long)rows,
                (long long)cols);
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
    MOE_REQUIRE(aligned_to(x, dtype_bytes(dtype)), "x must be aligned to its type");
    const bool vec = aligned16(x) && (x_stride * dtype_bytes(dtype)) % 16 == 0;
    const unsigned grid = mx_grid(rows * ((cols + 255) / 256));
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto fn = vec ? mx4_quantise_kernel<A, true> : mx4_quantise_kernel<A, false>;
        fn<<<grid, kMxThreads, 0, to_cuda(stream)>>>(static_cast<const typename A::T *>(x), x_stride, rows, (int)cols,
                                                     codes, scales, dev_status);
        return check_launch("mx4_quantise");
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
    const unsigned grid = mx_grid(rows * ((cols + 255) / 256));
    const bool vec = aligned16(out);
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto fn = vec ? mx4_dequantise_kernel<A, true> : mx4_dequantise_kernel<A, false>;
        fn<<<grid, kMxThreads, 0, to_cuda(stream)>>>(codes, scales, rows, (int)cols, static_cast<typename A::T *>(out));
        return check_launch("mx4_dequantise");
    });
}
