// rows.cuh -- element types of activation rows: fp32, bf16 and fp16 values to
// and from fp32 registers, one at a time or four or eight at once (raw8: eight
// as they lie, so that several loads fit into registers before any is used).
#pragma once

#include <type_traits>

#include "common.cuh"

namespace moe {

struct F32 {
    using T = float;
    static constexpr int kBytes = 4;
    struct Raw8 {
        float4 a, b;
    };
    __device__ static Raw8 raw8(const T *p) { return {reinterpret_cast<const float4 *>(p)[0], reinterpret_cast<const float4 *>(p)[1]}; }
    __device__ static void unpack8(const Raw8 &q, float (&v)[8])
    {
        v[0] = q.a.x, v[1] = q.a.y, v[2] = q.a.z, v[3] = q.a.w, v[4] = q.b.x, v[5] = q.b.y, v[6] = q.b.z, v[7] = q.b.w;
    }
    __device__ static float load(const T *p) { return *p; }
    __device__ static void store(T *p, float v) { *p = v; }
    __device__ static void store8(T *p, const float (&v)[8])
    {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ static void load4(const T *p, float *v)
    {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    }
    __device__ static void store4(T *p, const float *v) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
};

struct Bf16 {
    using T = uint16_t;
    static constexpr int kBytes = 2;
    using Raw8 = uint4;
    __device__ static Raw8 raw8(const T *p) { return *reinterpret_cast<const uint4 *>(p); }
    __device__ static float load(const T *p) { return bf16_to_f32(*p); }
    __device__ static void store(T *p, float v) { *p = f32_to_bf16(v); }
    __device__ static void unpack8(uint4 q, float (&v)[8])
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack8(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++)  // one rounding, to nearest even
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static void store8(T *p, const float (&v)[8]) { *reinterpret_cast<uint4 *>(p) = pack8(v); }
    __device__ static void load4(const T *p, float *v)
    {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static void store4(T *p, const float *v)
    {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; i++) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
};

struct Fp16 {
    using T = uint16_t;
    static constexpr int kBytes = 2;
    using Raw8 = uint4;
    __device__ static Raw8 raw8(const T *p) { return *reinterpret_cast<const uint4 *>(p); }
    __device__ static float load(const T *p) { return fp16_to_f32(*p); }
    __device__ static void store(T *p, float v) { *p = __half_as_ushort(__float2half_rn(v)); }
    __device__ static void unpack8(uint4 q, float (&v)[8])
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = fp16_to_f32((uint16_t)(w[i] & 0xffffu));
            v[2 * i + 1] = fp16_to_f32((uint16_t)(w[i] >> 16));
        }
    }
    __device__ static uint4 pack8(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static void store8(T *p, const float (&v)[8]) { *reinterpret_cast<uint4 *>(p) = pack8(v); }
    __device__ static void load4(const T *p, float *v)
    {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            v[2 * i] = fp16_to_f32((uint16_t)(w[i] & 0xffffu));
            v[2 * i + 1] = fp16_to_f32((uint16_t)(w[i] >> 16));
        }
    }
    __device__ static void store4(T *p, const float *v)
    {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; i++) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
};

// N = 8, 2 or 1 elements of a row as one access: as they lie (Raw), in fp32.
template <class A, int N>
struct Unit;
template <class A>
struct Unit<A, 8> {
    using Raw = typename A::Raw8;
    __device__ static Raw raw(const typename A::T *p) { return A::raw8(p); }
    __device__ static void unpack(const Raw &q, float (&v)[8]) { A::unpack8(q, v); }
    __device__ static void store(typename A::T *p, const float (&v)[8]) { A::store8(p, v); }
};
template <class A>
struct Unit<A, 2> {
    using Raw = std::conditional_t<A::kBytes == 4, uint2, uint32_t>;
    __device__ static Raw raw(const typename A::T *p) { return *reinterpret_cast<const Raw *>(p); }
    __device__ static void unpack(const Raw &q, float (&v)[2])
    {
        const typename A::T *e = reinterpret_cast<const typename A::T *>(&q);
        v[0] = A::load(e), v[1] = A::load(e + 1);
    }
    __device__ static void store(typename A::T *p, const float (&v)[2])
    {
        Raw q;
        A::store(reinterpret_cast<typename A::T *>(&q), v[0]);
        A::store(reinterpret_cast<typename A::T *>(&q) + 1, v[1]);
        *reinterpret_cast<Raw *>(p) = q;
    }
};
template <class A>
struct Unit<A, 1> {
    using Raw = typename A::T;
    __device__ static Raw raw(const typename A::T *p) { return *p; }
    __device__ static void unpack(const Raw &q, float (&v)[1]) { v[0] = A::load(&q); }
    __device__ static void store(typename A::T *p, const float (&v)[1]) { A::store(p, v[0]); }
};

// Zeros n bytes from p (both even) with the threads `rank` of `count`: 16 bytes
// at a time between the first and the last 16-byte boundary.
__device__ __forceinline__ void zero_bytes(void *p, int64_t n, int64_t rank, int64_t count)
{
    char *b = static_cast<char *>(p);
    const int64_t head = min(n, (int64_t)(-reinterpret_cast<uintptr_t>(b) & 15)), pieces = (n - head) / 16, tail = n - head - pieces * 16;
    for (int64_t i = rank; i < pieces; i += count) reinterpret_cast<uint4 *>(b + head)[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = rank; i < (head + tail) / 2; i += count)
        *reinterpret_cast<uint16_t *>(i * 2 < head ? b + i * 2 : b + pieces * 16 + i * 2) = 0;
}

inline bool dtype_ok(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16 || t == MOE_F16; }
inline int dtype_bytes(moe_dtype t) { return t == MOE_F32 ? 4 : 2; }
inline bool aligned_to(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0; }

// Calls F<A>() with the element type of `t`.
template <class F>
moe_status with_dtype(moe_dtype t, F f)
{
    if (t == MOE_F32) return f(F32{});
    if (t == MOE_BF16) return f(Bf16{});
    return f(Fp16{});
}

}  // namespace moe
