// mx4.cu -- the microscaled 4-bit format (MXFP4): e2m1 codes, two to a byte,
// with one e8m0 scale byte per 32 values of a row.
//
// Both directions are one pass bound by memory: quantising reads a value once
// and writes 17/32 byte for it.  A thread takes eight values (four bytes of
// codes), four threads a block, whatever the rows' width: codes are one run
// over all rows, and only the scales' place needs the row (a product with the
// width's reciprocal).  Each thread has four such pieces in flight.
#include "rows.cuh"

namespace moe {

constexpr int kMxThreads = 256, kMxUnroll = 4;

// Bytes of a row's scales: 32 for 1024 values, the unit the product loads.
__host__ __device__ constexpr int64_t mx4_pitch(int64_t cols) { return (cols + 1023) / 1024 * 32; }

// Two fp32 values to e2m1 (nearest, ties to even, saturating at 6): lo in bits 0..3.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// Piece i = eight values: row i / per_row by the reciprocal inv = floor(2^64 /
// per_row) + 1, exact while i * per_row < 2^64.
struct Pieces {
    int64_t total;
    int per_row;
    unsigned long long inv;
    __device__ __forceinline__ void at(int64_t i, int64_t &row, int &piece) const
    {
        row = (int64_t)__umul64hi((unsigned long long)i, inv);
        piece = (int)(i - row * per_row);
    }
};

// The block's exponent comes from the bits of its largest magnitude (an
// integer maximum, so an infinity or a NaN wins and marks the block):
// e = floor(log2 m) - 2, at least -127; x 2^-e is exact, so each value is
// rounded once.
template <class A, bool kVec>
__global__ void __launch_bounds__(kMxThreads) mx4_quantise_kernel(const typename A::T *__restrict__ x, int64_t x_stride,
                                                                  Pieces n, uint8_t *__restrict__ codes,
                                                                  uint8_t *__restrict__ scales, int32_t *status)
{
    const int cols = n.per_row * 8, pitch = (int)mx4_pitch(cols);
    for (int64_t i0 = (int64_t)blockIdx.x * (kMxThreads * kMxUnroll) + threadIdx.x; i0 - (int)threadIdx.x < n.total;
         i0 += (int64_t)gridDim.x * (kMxThreads * kMxUnroll)) {
        float v[kMxUnroll][8];
        int64_t row[kMxUnroll];
        int piece[kMxUnroll];
#pragma unroll
        for (int j = 0; j < kMxUnroll; j++) {
            const int64_t i = i0 + j * kMxThreads;
            n.at(i, row[j], piece[j]);
            if (i < n.total) {  // (the four threads of a block are in or out together)
                const typename A::T *p = x + row[j] * x_stride + piece[j] * 8;
                if (kVec) {
                    A::load8(p, v[j]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; k++) v[j][k] = A::load(p + k);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++) v[j][k] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < kMxUnroll; j++) {
            const int64_t i = i0 + j * kMxThreads;
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; k++) m = max(m, __float_as_uint(v[j][k]) & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (i >= n.total) continue;
            const bool bad = m >= 0x7f800000u;
            const int byte = max((int)(m >> 23) - 2, 0);                    // e + 127
            const float f = __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^-e
            uint32_t q = 0;
            if (!bad) {
#pragma unroll
                for (int k = 0; k < 4; k++) q |= e2m1x2(v[j][2 * k] * f, v[j][2 * k + 1] * f) << (8 * k);
            }
            reinterpret_cast<uint32_t *>(codes)[i] = q;
            uint8_t *sc = scales + row[j] * pitch;
            const int lane4 = threadIdx.x & 3, block = piece[j] >> 2;
            if (lane4 == 0) {
                sc[block] = bad ? 255 : (uint8_t)byte;
                if (bad) set_status(status, MOE_ERR_NONFINITE);
            }
            if (piece[j] - lane4 + 4 == n.per_row)  // the row's last block: the padding too
                for (int b = block + 1 + lane4; b < pitch; b += 4) sc[b] = 0;
        }
    }
}

template <class A, bool kVec>
__global__ void __launch_bounds__(kMxThreads) mx4_dequantise_kernel(const uint8_t *__restrict__ codes,
                                                                    const uint8_t *__restrict__ scales, Pieces n,
                                                                    typename A::T *__restrict__ out)
{
    const int pitch = (int)mx4_pitch(n.per_row * 8);
    for (int64_t i0 = (int64_t)blockIdx.x * (kMxThreads * kMxUnroll) + threadIdx.x; i0 < n.total;
         i0 += (int64_t)gridDim.x * (kMxThreads * kMxUnroll)) {
        uint32_t q[kMxUnroll], byte[kMxUnroll];
#pragma unroll
        for (int j = 0; j < kMxUnroll; j++) {
            const int64_t i = i0 + j * kMxThreads;
            int64_t row;
            int piece;
            n.at(i, row, piece);
            q[j] = i < n.total ? reinterpret_cast<const uint32_t *>(codes)[i] : 0u;
            byte[j] = i < n.total ? scales[row * pitch + (piece >> 2)] : 0u;
        }
#pragma unroll
        for (int j = 0; j < kMxUnroll; j++) {
            const int64_t i = i0 + j * kMxThreads;
            if (i >= n.total) break;
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
            typename A::T *o = out + i * 8;
            if (kVec) {
                A::store8(o, v);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++) A::store(o + k, v[k]);
            }
        }
    }
}

static Pieces mx_pieces(int64_t rows, int64_t cols)
{
    Pieces n;
    n.per_row = (int)(cols / 8);
    n.total = rows * n.per_row;
    n.inv = ~0ull / (unsigned)n.per_row + 1;  // floor(2^64 / d) + 1, or 2^64 / d itself where d is a power of two
    return n;
}

static unsigned mx_grid(const Pieces &n)
{
    const int64_t blocks = (n.total + kMxThreads * kMxUnroll - 1) / (kMxThreads * kMxUnroll);
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)sm_count() * 8));
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
    MOE_REQUIRE(aligned_to(x, dtype_bytes(dtype)), "x must be aligned to its type");
    const bool vec = aligned16(x) && (x_stride * dtype_bytes(dtype)) % 16 == 0;
    const Pieces n = mx_pieces(rows, cols);
    const unsigned grid = mx_grid(n);
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto fn = vec ? mx4_quantise_kernel<A, true> : mx4_quantise_kernel<A, false>;
        fn<<<grid, kMxThreads, 0, to_cuda(stream)>>>(static_cast<const typename A::T *>(x), x_stride, n, codes, scales,
                                                     dev_status);
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
    const Pieces n = mx_pieces(rows, cols);
    const unsigned grid = mx_grid(n);
    const bool vec = aligned16(out);
    return with_dtype(dtype, [&](auto a) {
        using A = decltype(a);
        auto fn = vec ? mx4_dequantise_kernel<A, true> : mx4_dequantise_kernel<A, false>;
        fn<<<grid, kMxThreads, 0, to_cuda(stream)>>>(codes, scales, n, static_cast<typename A::T *>(out));
        return check_launch("mx4_dequantise");
    });
}
