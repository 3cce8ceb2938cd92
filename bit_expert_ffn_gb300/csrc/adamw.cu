// adamw.cu -- moe_adamw_step: one AdamW step over many tensors, states in fp32
// or in 8 bits with two scales per 256 values; moe_adamw_states: their values.
//
//   m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2
//   x = x (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Memory bounds it: 28 bytes a value in fp32, 16 with 8-bit states, a 16-bit
// gradient and parameter and an fp32 copy.  The tensors' descriptors travel in the
// launch's parameters (up to 32 KB of constant memory), so a step needs no
// table in device memory; a CTA finds its tensor by bisection of the tensors'
// first chunks.  A warp takes 256 values at a time, the block of the 8-bit
// states, so that a block's largest values come from one warp's registers.  With
// fp32 states a lane has two groups of four (16-byte accesses), with 8-bit ones
// eight side by side (32 bytes of fp32; in fours as well 3% more time) and the next
// block on its way; or eight single ones where a tensor's pointers are not
// aligned for that.
//
// The 8-bit codes are defined by 32-bit arithmetic, each operation rounded:
// hence the explicit roundings below, where the compiler must not fuse a
// product with a sum.  (Pairs of fp32 operations in one instruction, mul and add
// .f32x2, were fused all the same, and brought 1%.)
//
// Measured on one GB300: 50 M fp32 values with fp32 states in 192 tensors 207 us
// (6.8 TB/s: memory); 189 M values, 8-bit states, 16-bit gradient and parameter
// and an fp32 copy 485 us (6.2 TB/s; some 70 instructions a value, 60% of the issue
// slots), their states' values in fp32 283 us (6.7 TB/s).
#include <new>

#include "rows.cuh"

namespace moe {
namespace aw {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int BLOCK = 256;                   // values that share scales, and of a warp's turn
constexpr int MIN_CHUNK = WARPS * BLOCK;     // values of a CTA
constexpr int FEW = 16, MANY = 428;          // tensors of a launch: its parameters hold 32,764 bytes
constexpr float SMALLEST = 7.888609052210118e-31f;  // 2^-100

struct Tensor {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *scales;
    int64_t n;
    float lr_factor, decay;
    int8_t pt, gt, vec, pad[5];
};

struct Common {
    float b1, o1, b2, o2, eps, lr, rate1, root2;  // o = 1 - b, rate1 = 1 / (1 - b1^t), root2 = 1 / sqrt(1 - b2^t)
    float log_b1, log_b2;
    const float *lr_dev, *grad_scale;
    const int64_t *step_dev;
    int32_t *status;
    int n, chunk;
};

template <int N>
struct Params {
    Common c;
    int32_t first[N];  // chunks before a tensor
    Tensor t[N];
};

// Four values as they lie: 16 bytes of fp32 or 8 of 16-bit types.
__device__ __forceinline__ uint4 raw4(const void *p, int64_t i, int type)
{
    if (type == MOE_F32) return *reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
    const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    return make_uint4(q.x, q.y, 0, 0);
}

__device__ __forceinline__ void unpack4(const uint4 &q, int type, float *v)
{
    if (type == MOE_F32) {
        v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
    } else if (type == MOE_BF16) {
        v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
        v[0] = fp16_to_f32((uint16_t)q.x), v[1] = fp16_to_f32((uint16_t)(q.x >> 16));
        v[2] = fp16_to_f32((uint16_t)q.y), v[3] = fp16_to_f32((uint16_t)(q.y >> 16));
    }
}

__device__ __forceinline__ void store4(void *p, int64_t i, int type, const float *v)
{
    if (type == MOE_F32) F32::store4(static_cast<float *>(p) + i, v);
    else if (type == MOE_BF16) Bf16::store4(static_cast<uint16_t *>(p) + i, v);
    else Fp16::store4(static_cast<uint16_t *>(p) + i, v);
}

constexpr int BYTES = 3;  // a type beside moe_dtype's: 8-bit codes

__device__ __forceinline__ float value(uint32_t raw, int type)
{
    return type == MOE_F32 ? __uint_as_float(raw) : type == MOE_BF16 ? __uint_as_float(raw << 16) : fp16_to_f32((uint16_t)raw);
}

__device__ __forceinline__ void store1(void *p, int64_t i, int type, float v)
{
    if (type == MOE_F32) F32::store(static_cast<float *>(p) + i, v);
    else if (type == MOE_BF16) Bf16::store(static_cast<uint16_t *>(p) + i, v);
    else Fp16::store(static_cast<uint16_t *>(p) + i, v);
}

// ---------------------------------------------------------------- 8-bit codes

// Four e4m3 codes to their values.
__device__ __forceinline__ void e4m3_values(uint32_t q, float *v)
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(q >> (16 * i))));
        v[2 * i] = fp16_to_f32((uint16_t)h), v[2 * i + 1] = fp16_to_f32((uint16_t)(h >> 16));
    }
}

__device__ __forceinline__ uint32_t e4m3_codes(const float *v)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Code c > 0: (16 + c % 16) 2^(c / 16 - 19), the code's bits at the head of an fp32's mantissa.
__device__ __forceinline__ float root_value(uint32_t c) { return c ? __uint_as_float((c + (112u << 4)) << 19) : 0.f; }

__device__ __forceinline__ uint32_t root_code(float x)
{
    const uint32_t b = __float_as_uint(x), near = (b + 0x3FFFFu + ((b >> 19) & 1u)) >> 19;
    return (uint32_t)min(max((int)near - (112 << 4), 1), 255);
}

// The largest of the warp's (non-negative) values.
__device__ __forceinline__ float warp_top(float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); }

// ---------------------------------------------------------------- a step

template <int N>
__device__ __forceinline__ int find(const Params<N> &p, int chunk)
{
    int lo = 0, hi = p.c.n;  // the last tensor whose first chunk is at most `chunk`
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A lane's eight values of 256 from `base`: two groups of four, or eight 32 apart.
template <bool kVec>
__device__ __forceinline__ int64_t place(int64_t base, int i, int lane)
{
    return kVec ? base + (i >> 2) * 128 + lane * 4 + (i & 3) : base + i * 32 + lane;
}

// A lane's eight values of 256 from `base`, as they lie, zero past the `left` that there are.
template <bool kVec>
__device__ __forceinline__ void load8(const void *p, int64_t base, int64_t left, int lane, int type, uint32_t (&r)[8])
{
    auto each = [&](auto unit) {
        const decltype(unit) *q = static_cast<const decltype(unit) *>(p) + base;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int e = (int)place<kVec>(0, i, lane);
            r[i] = e < left ? q[e] : 0;
        }
    };
    if (type == MOE_F32) each(uint32_t{});
    else if (type == BYTES) each(uint8_t{});
    else each(uint16_t{});
}

struct Scalars {
    float scale, shrink, rate, root2;
    float before, after;  // block: the rate multiplies m, or, where that could leave fp32's normal range, the quotient
    float root2_rate, eps_rate;  // for block8: root2 and eps over the rate (a product less a value); a rate of 0: 0 and infinity

    // Whether block8's steps are the exact ones to 2^-22: its roots of v below 2^-126 are 0, which counts for nothing beside eps
    // where root2 2^-63 is below eps 2^-24; and its reciprocals keep no number below 2^-126, so that root2 r / rate (r below
    // 2^64, since squares are finite) and eps / rate stay between 2^-79 and 2^125.
    __device__ bool fast(float eps) const
    {
        return eps >= root2 * 1.8189894e-12f && eps <= 1.2089258e24f && root2 <= 1048576.f &&  // (2^-39, 2^80, 2^20)
               (rate == 0.f || (fabsf(rate) >= 9.0949470e-13f && fabsf(rate) <= 1.0995116e12f));  // (2^-40, 2^40)
    }
};

// 256 values: with fp32 states (kVec: aligned for fours), or, k8, with 8-bit ones, value by value.
template <bool k8, bool kVec>
__device__ __forceinline__ void block(const Common &c, const Tensor &t, const Scalars &s, int64_t base, int lane)
{
    float x[8], g[8], m[8], v[8];
    const void *xp = t.master ? t.master : t.param;
    const int xt = t.master ? (int)MOE_F32 : t.pt;
    static_assert(!(k8 && kVec), "whole, aligned blocks with 8-bit states are block8's");
    const bool whole = kVec && base + BLOCK <= t.n;  // (a last, short block goes value by value)
    float um = 0.f, ur = 0.f;
    if (k8) {
        const float2 u = *reinterpret_cast<const float2 *>(t.scales + base / BLOCK * 2);
        um = u.x, ur = u.y;
    }
    if (whole) {
        uint4 rx[2], rg[2], rm[2], rv[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int64_t i = place<true>(base, 4 * j, lane);
            rg[j] = raw4(t.grad, i, t.gt);
            rx[j] = raw4(xp, i, xt);
            rm[j] = raw4(t.m, i, MOE_F32);
            rv[j] = raw4(t.v, i, MOE_F32);
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            unpack4(rg[j], t.gt, g + 4 * j);
            unpack4(rx[j], xt, x + 4 * j);
            unpack4(rm[j], MOE_F32, m + 4 * j);
            unpack4(rv[j], MOE_F32, v + 4 * j);
        }
    } else {  // (all loads before the first use)
        uint32_t rg[8], rx[8], rm[8], rv[8];
        const int64_t left = t.n - base;
        load8<kVec>(t.grad, base, left, lane, t.gt, rg);
        load8<kVec>(xp, base, left, lane, xt, rx);
        load8<kVec>(t.m, base, left, lane, k8 ? BYTES : (int)MOE_F32, rm);
        load8<kVec>(t.v, base, left, lane, k8 ? BYTES : (int)MOE_F32, rv);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            g[i] = value(rg[i], t.gt);
            x[i] = value(rx[i], xt);
            if (k8) {
                float q[4];
                e4m3_values(rm[i], q);
                m[i] = q[0];
                v[i] = root_value(rv[i]);
            } else {
                m[i] = __uint_as_float(rm[i]);
                v[i] = __uint_as_float(rv[i]);
            }
        }
    }
    float r[8], top_m = 0.f, top_r = 0.f;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if (k8) {
            m[i] = __fmul_rn(m[i], um);
            v[i] = __fmul_rn(v[i], ur);
            v[i] = __fmul_rn(v[i], v[i]);
        }
        const float gi = g[i] * s.scale, g2 = __fmul_rn(gi, gi);
        const bool ok = g2 < INFINITY;
        const float mn = __fadd_rn(__fmul_rn(m[i], c.b1), __fmul_rn(gi, c.o1));
        const float vn = __fadd_rn(__fmul_rn(v[i], c.b2), __fmul_rn(g2, c.o2));
        m[i] = ok ? mn : m[i];
        v[i] = ok ? vn : v[i];
        if (k8) r[i] = __fsqrt_rn(v[i]);
        else asm("sqrt.approx.f32 %0, %1;" : "=f"(r[i]) : "f"(v[i]));
        const float to = __fdividef(m[i] * s.before, fmaf(r[i], s.root2, c.eps)) * s.after;
        x[i] = ok ? fmaf(x[i], s.shrink, -to) : x[i];
        bad += !ok;
        if (k8) top_m = fmaxf(top_m, fabsf(m[i])), top_r = fmaxf(top_r, r[i]);
    }
    if (__any_sync(0xffffffffu, bad)) {
        if (bad) set_status(c.status, MOE_ERR_NONFINITE);
        // (a block without a good gradient keeps its scales' bits too; places past the end are good, but nobody's)
        bool good = false;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float gi = g[i] * s.scale;
            good |= place<kVec>(base, i, lane) < t.n && gi * gi < INFINITY;
        }
        if (!__any_sync(0xffffffffu, good)) return;
    }
    float im = 0.f, ir = 0.f;
    if (k8) {
        top_m = warp_top(top_m);
        top_r = warp_top(top_r);
        if (top_m < SMALLEST) top_m = 0.f;
        if (top_r < SMALLEST) top_r = 0.f;
        // the four quotients in four lanes at once: 448 / top, top / 448 and the root's
        const float top = lane & 1 ? top_r : top_m, full = lane & 1 ? 1.9375f : 448.f;
        const float q = top > 0.f ? (lane & 2 ? __fdiv_rn(top, full) : __fdiv_rn(full, top)) : 0.f;
        im = __shfl_sync(0xffffffffu, q, 0);
        ir = __shfl_sync(0xffffffffu, q, 1);
        const float2 u = make_float2(__shfl_sync(0xffffffffu, q, 2), __shfl_sync(0xffffffffu, q, 3));
        if (lane == 0) *reinterpret_cast<float2 *>(t.scales + base / BLOCK * 2) = u;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            m[i] = __fmul_rn(m[i], im);
            r[i] = __fmul_rn(r[i], ir);
        }
    }
    if (whole) {
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int64_t i = place<true>(base, 4 * j, lane);
            if (t.master) F32::store4(t.master + i, x + 4 * j);
            store4(t.param, i, t.pt, x + 4 * j);
            F32::store4(static_cast<float *>(t.m) + i, m + 4 * j);
            F32::store4(static_cast<float *>(t.v) + i, v + 4 * j);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t e = place<kVec>(base, i, lane);
            if (e >= t.n) continue;
            if (t.master) t.master[e] = x[i];
            store1(t.param, e, t.pt, x[i]);
            if (k8) {
                const float q[4] = {m[i], 0.f, 0.f, 0.f};
                static_cast<uint8_t *>(t.m)[e] = (uint8_t)e4m3_codes(q);
                static_cast<uint8_t *>(t.v)[e] = r[i] > 0.f ? (uint8_t)root_code(r[i]) : 0;
            } else {
                static_cast<float *>(t.m)[e] = m[i];
                static_cast<float *>(t.v)[e] = v[i];
            }
        }
    }
}

// Eight values of a type side by side as they lie (32 or 16 bytes), and in fp32.
template <class A>
struct Eight {
    uint32_t w[A::kBytes * 2];

    __device__ void load(const typename A::T *p)
    {
        if constexpr (A::kBytes == 4) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p));
        } else {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        }
    }
    __device__ void unpack(float (&v)[8]) const
    {
        if constexpr (A::kBytes == 4) {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = __uint_as_float(w[i]);
        } else {
            A::unpack8(make_uint4(w[0], w[1], w[2], w[3]), v);
        }
    }
};

template <class A>
__device__ __forceinline__ void store_eight(typename A::T *p, const float (&v)[8])
{
    if constexpr (A::kBytes == 4)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                     "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
    else A::store8(p, v);
}

// A lane's places in a chunk's tensors; blocks are `o` values further on.
template <class G, class X>
struct At {
    const typename G::T *g;
    typename X::T *x;  // the fp32 copy, or the parameter
    void *p;           // the parameter beside a copy, or NULL
    uint8_t *m, *v;
    float2 *scales;
    int pt;

    __device__ At(const Tensor &t, int64_t i, int lane)
        : g(static_cast<const typename G::T *>(t.grad) + i + lane * 8), m(static_cast<uint8_t *>(t.m) + i + lane * 8),
          v(static_cast<uint8_t *>(t.v) + i + lane * 8), scales(reinterpret_cast<float2 *>(t.scales) + i / BLOCK), pt(t.pt)
    {
        x = static_cast<typename X::T *>(t.master ? static_cast<void *>(t.master) : t.param) + i + lane * 8;
        p = t.master ? static_cast<char *>(t.param) + (i + lane * 8) * (pt == MOE_F32 ? 4 : 2) : nullptr;
    }
};

// What a lane loads of a block.
template <class G, class X>
struct Held8 {
    Eight<G> g;
    Eight<X> x;
    uint2 m, v;
    float2 u;

    __device__ void load(const At<G, X> &at, int o)
    {
        g.load(at.g + o);
        x.load(at.x + o);
        m = *reinterpret_cast<const uint2 *>(at.m + o);
        v = *reinterpret_cast<const uint2 *>(at.v + o);
        u = at.scales[o / BLOCK];
    }
};

// 256 values with 8-bit states, whole and aligned.  False, and nothing done, when the block wants block()'s exact steps: a
// gradient that is not finite, roots so small that the fast root of a subnormal v, 0, would not get the same code (below
// 2^-46 of the largest all do: code 1), or a root next to a border between two codes.  The fast root is within 2^-23 of
// the correctly rounded one, its product with the block's factor within 3 last places: eight of 2^19 to either side of a
// border are left to the exact steps (8 blocks of 1,000), so that the codes are theirs in every case.  The largest root
// is the rounded root of the largest v, since rounding keeps the order.
template <class G, class X>
__device__ __forceinline__ bool block8(const Common &c, const At<G, X> &at, const Scalars &s, int o, int lane, const Held8<G, X> &raw)
{
    float x[8], m[8], v[8], r[8];
    const float2 u = raw.u;
    float top_m = 0.f, g[8];
    uint32_t most = 0;  // the largest v's bits (of what is not negative, bits are in order; a NaN's are above all)
    raw.g.unpack(g);
    if (c.grad_scale) {
#pragma unroll
        for (int i = 0; i < 8; i++) g[i] *= s.scale;
    }
    raw.x.unpack(x);
    e4m3_values(raw.m.x, m);
    e4m3_values(raw.m.y, m + 4);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t code = (i < 4 ? raw.v.x : raw.v.y) >> (8 * (i & 3)) & 255u;
        const float gi = g[i], g2 = __fmul_rn(gi, gi), root = __fmul_rn(root_value(code), u.y);
        m[i] = __fadd_rn(__fmul_rn(__fmul_rn(m[i], u.x), c.b1), __fmul_rn(gi, c.o1));
        v[i] = __fadd_rn(__fmul_rn(__fmul_rn(root, root), c.b2), __fmul_rn(g2, c.o2));
        top_m = fmaxf(top_m, fabsf(m[i]));
        most = max(most, __float_as_uint(v[i]));
    }
    top_m = warp_top(top_m);
    most = __reduce_max_sync(0xffffffffu, most);
    const float top_v = __uint_as_float(most);
    if (top_m < SMALLEST) top_m = 0.f;
    const float top_r = __fsqrt_rn(top_v);
    // (a square that is not finite leaves v so)
    if (most >= 0x7f800000u || (top_v > 0.f && top_r < 1.4210855e-14f)) return false;  // (2^-46)
    // the four quotients in four lanes at once: 448 / top, top / 448 and the root's
    const float top = lane & 1 ? top_r : top_m, full = lane & 1 ? 1.9375f : 448.f;
    const float q = top > 0.f ? __fdiv_rn(lane & 2 ? top : full, lane & 2 ? full : top) : 0.f;
    const float im = __shfl_sync(0xffffffffu, q, 0), ir = __shfl_sync(0xffffffffu, q, 1);
    const float2 held = make_float2(__shfl_sync(0xffffffffu, q, 2), __shfl_sync(0xffffffffu, q, 3));
    uint32_t close = ~0u, codes[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        uint32_t code[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int i = 4 * j + e;
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r[i]) : "f"(v[i]));
            const uint32_t b = __float_as_uint(fmaxf(__fmul_rn(r[i], ir), 17.f / 524288.f));  // code 1 at least
            const uint32_t near = b + (0x40000u - (112u << 23));  // its code in the upper bits (no ties here: they are close)
            close = min(close, near * 8192u + (8u << 13));        // how far its lower 19 bits are from -8, as the upper ones
            code[e] = min(near >> 19, __float_as_uint(v[i]));  // (0 for a v of 0, whose root counted as code 1's)
        }
        codes[j] = __byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410);
    }
    if (__any_sync(0xffffffffu, close <= 16u << 13)) return false;
    if (lane == 0) at.scales[o / BLOCK] = held;
#pragma unroll
    for (int j = 0; j < 2; j++) {
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int i = 4 * j + e;
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(r[i], s.root2_rate, s.eps_rate)));
            x[i] = fmaf(x[i], s.shrink, -(m[i] * inv));
            m[i] = __fmul_rn(m[i], im);
        }
    }
    store_eight<X>(at.x + o, x);
    if (X::kBytes == 4 && at.p) {
        if (at.pt == MOE_F32) store_eight<F32>(static_cast<float *>(at.p) + o, x);
        else if (at.pt == MOE_BF16) Bf16::store8(static_cast<uint16_t *>(at.p) + o, x);
        else Fp16::store8(static_cast<uint16_t *>(at.p) + o, x);
    }
    *reinterpret_cast<uint2 *>(at.m + o) = make_uint2(e4m3_codes(m), e4m3_codes(m + 4));
    *reinterpret_cast<uint2 *>(at.v + o) = make_uint2(codes[0], codes[1]);
    return true;
}

template <class F>
__device__ __forceinline__ void on_type(int type, F f)
{
    if (type == MOE_F32) f(F32{});
    else if (type == MOE_BF16) f(Bf16{});
    else f(Fp16{});
}

// A warp's blocks of a chunk, the next one's values on their way.  Returns which of them are left to the exact steps: a
// last short block, values next to a border.
template <class G, class X>
__device__ __forceinline__ uint32_t blocks8(const Common &c, const Tensor &t, const Scalars &s, int64_t base, int n, int lane)
{
    const At<G, X> at(t, base, lane);
    Held8<G, X> cur, nxt;
    uint32_t left = 0;
    if (BLOCK <= n) cur.load(at, 0);
#pragma unroll 1
    for (int o = 0; o < n; o += MIN_CHUNK) {
        if (o + MIN_CHUNK + BLOCK <= n) nxt.load(at, o + MIN_CHUNK);
        if (o + BLOCK > n || !block8<G, X>(c, at, s, o, lane, cur)) left |= 1u << (o / MIN_CHUNK);
        cur = nxt;
    }
    return left;
}

// k8: the launch's tensors have 8-bit states.
template <int N, bool k8>
__global__ void __launch_bounds__(THREADS, 3) step_kernel(const __grid_constant__ Params<N> p)
{
    const Common &c = p.c;
    const int which = find(p, blockIdx.x);
    const Tensor &t = p.t[which];
    float lr = c.lr, rate1 = c.rate1;
    Scalars s;
    s.scale = c.grad_scale ? *c.grad_scale : 1.f;
    s.root2 = c.root2;
    if (c.lr_dev) lr = *c.lr_dev;
    if (c.step_dev) {  // 1 - b^t, without cancellation
        const float n = (float)max(*c.step_dev, (int64_t)1);
        rate1 = 1.f / -expm1f(n * c.log_b1);
        s.root2 = rsqrtf(-expm1f(n * c.log_b2));
    }
    lr *= t.lr_factor;
    s.rate = lr * rate1;
    s.shrink = 1.f - lr * t.decay;
    const bool tiny = s.rate != 0.f && fabsf(s.rate) < 9.0949470e-13f;  // (2^-40)
    s.before = tiny ? 1.f : s.rate;
    s.after = tiny ? s.rate : 1.f;
    s.root2_rate = s.rate == 0.f ? 0.f : s.root2 / s.rate;
    s.eps_rate = s.rate == 0.f ? INFINITY : c.eps / s.rate;
    const int lane = lane_id();
    const int64_t begin = (int64_t)(blockIdx.x - p.first[which]) * c.chunk, end = min(begin + c.chunk, t.n);
    const int64_t first = begin + warp_id() * BLOCK;
    if (k8) {
        uint32_t left = ~0u;
        if (t.vec && first < end && s.fast(c.eps))
            on_type(t.gt, [&](auto g) {
                on_type(t.master ? (int)MOE_F32 : t.pt,
                        [&](auto x) { left = blocks8<decltype(g), decltype(x)>(c, t, s, first, (int)(end - first), lane); });
            });
        for (int64_t base = first; base < end; base += MIN_CHUNK, left >>= 1)
            if (left & 1) block<true, false>(c, t, s, base, lane);
    } else {
        for (int64_t base = first; base < end; base += MIN_CHUNK) {
            if (t.vec) block<false, true>(c, t, s, base, lane);
            else block<false, false>(c, t, s, base, lane);
        }
    }
}

// The states' values: t.master takes m's, t.param v's (fp32, either may be NULL).
template <int N>
__global__ void __launch_bounds__(THREADS, 8) states_kernel(const __grid_constant__ Params<N> p)
{
    const int which = find(p, blockIdx.x);
    const Tensor &t = p.t[which];
    float *mo = t.master, *vo = static_cast<float *>(t.param);
    const int lane = lane_id();
    const int64_t begin = (int64_t)(blockIdx.x - p.first[which]) * p.c.chunk, end = min(begin + p.c.chunk, t.n);
    for (int64_t base = begin + warp_id() * BLOCK; base < end; base += MIN_CHUNK) {
        float2 u = make_float2(0.f, 0.f);
        if (t.scales) u = *reinterpret_cast<const float2 *>(t.scales + base / BLOCK * 2);
        if (t.vec && base + BLOCK <= t.n) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t i = place<true>(base, 4 * j, lane);
                float m[4], v[4];
                if (t.scales) {
                    e4m3_values(*reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(t.m) + i), m);
                    const uint32_t q = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(t.v) + i);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        m[e] = __fmul_rn(m[e], u.x);
                        v[e] = __fmul_rn(root_value(q >> (8 * e) & 255u), u.y);
                        v[e] = __fmul_rn(v[e], v[e]);
                    }
                } else {
                    F32::load4(static_cast<const float *>(t.m) + i, m);
                    F32::load4(static_cast<const float *>(t.v) + i, v);
                }
                if (mo) F32::store4(mo + i, m);
                if (vo) F32::store4(vo + i, v);
            }
            continue;
        }
        uint32_t rm[8], rv[8];
        load8<false>(t.m, base, t.n - base, lane, t.scales ? BYTES : (int)MOE_F32, rm);
        load8<false>(t.v, base, t.n - base, lane, t.scales ? BYTES : (int)MOE_F32, rv);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t e = place<false>(base, i, lane);
            if (e >= t.n) continue;
            float q[4] = {__uint_as_float(rm[i])}, v = __uint_as_float(rv[i]);
            if (t.scales) {
                e4m3_values(rm[i], q);
                q[0] = __fmul_rn(q[0], u.x);
                v = __fmul_rn(root_value(rv[i]), u.y);
                v = __fmul_rn(v, v);
            }
            if (mo) mo[e] = q[0];
            if (vo) vo[e] = v;
        }
    }
}

static moe_status check(const moe_adamw_tensor *t, int n)
{
    MOE_REQUIRE(n >= 0, "n_tensors must not be negative (got %d)", n);
    MOE_REQUIRE(t || n == 0, "tensors must not be NULL");
    for (int i = 0; i < n; i++) {
        const moe_adamw_tensor &a = t[i];
        MOE_REQUIRE(a.n >= 0 && a.n <= (1ll << 40), "tensor %d: n must be in [0, 2^40] (got %lld)", i, (long long)a.n);
        if (a.n == 0) continue;
        MOE_REQUIRE(a.m && a.v, "tensor %d: NULL pointer", i);
        MOE_REQUIRE(aligned_to(a.scales, 8) && (a.scales || (aligned_to(a.m, 4) && aligned_to(a.v, 4))),
                    "tensor %d: scales must be 8-byte aligned, fp32 states aligned to their type", i);
    }
    return MOE_OK;
}

// Fills launches of up to MANY tensors (kind 0 or 1: those without or with scales; -1: all); `one` sets a tensor's outputs and says whether its pointers are aligned for fours.
template <class K, class F>
moe_status launch(const moe_adamw_tensor *tensors, int n, int kind, const Common &c, const char *what, K kernel, F one)
{
    int64_t total = 0;
    for (int i = 0; i < n; i++) total += tensors[i].n;
    // a CTA's values: enough CTAs for eight turns of all SMs, no more than 16,384 a CTA
    const int64_t per = total / ((int64_t)sm_count() * 64);
    int chunk = MIN_CHUNK;
    while (chunk < 16384 && chunk < per) chunk *= 2;
    static_assert(sizeof(Params<MANY>) <= 32764, "a launch's parameters");
    auto run = [&](auto &p, int &i) -> moe_status {
        constexpr int kN = sizeof(p.t) / sizeof(Tensor);
        p.c = c;
        p.c.n = 0;
        p.c.chunk = chunk;
        int64_t chunks = 0;
        for (; i < n && p.c.n < kN; i++) {
            const moe_adamw_tensor &a = tensors[i];
            if (a.n == 0 || (kind >= 0 && kind != (a.scales != nullptr))) continue;
            const int64_t more = (a.n + chunk - 1) / chunk;
            if (more > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "tensor %d is too large (n=%lld)", i, (long long)a.n);
            if (chunks + more > INT32_MAX) break;
            p.first[p.c.n] = (int32_t)chunks;
            Tensor &t = p.t[p.c.n++];
            t = {a.param, a.grad, a.master, a.m, a.v, a.scales, a.n, a.lr_factor, a.weight_decay, (int8_t)a.param_dtype,
                 (int8_t)a.grad_dtype, 0, {}};
            const int states = a.scales ? 4 : 16;
            t.vec = aligned_to(a.m, states) && aligned_to(a.v, states);
            one(i, t);
            chunks += more;
        }
        if (chunks == 0) return MOE_OK;
        kernel(p, (unsigned)chunks);
        return check_launch(what);
    };
    for (int i = 0; i < n;) {
        moe_status st;
        if (n - i <= FEW) {  // (a few tensors' parameters are copied in 1.3 KB)
            Params<FEW> p;
            st = run(p, i);
        } else {
            Params<MANY> p;
            st = run(p, i);
        }
        if (st != MOE_OK) return st;
    }
    return MOE_OK;
}

// Whether two tensors' params overlap (the same tensor named twice): sorted by address, unless they are so already.
struct Range {
    uintptr_t a, b;
};

static moe_status check_overlap(const moe_adamw_tensor *t, int n)
{
    bool ascending = true;
    uintptr_t end = 0;
    for (int i = 0; i < n && ascending; i++) {
        if (t[i].n == 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(t[i].param);
        ascending = a >= end;
        end = a + (size_t)t[i].n * dtype_bytes((moe_dtype)t[i].param_dtype);
    }
    if (ascending) return MOE_OK;
    Range *r = new (std::nothrow) Range[n];
    if (!r) return fail(MOE_ERR_INVALID_ARG, "no host memory to check %d tensors", n);
    int k = 0;
    for (int i = 0; i < n; i++)
        if (t[i].n) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(t[i].param);
            r[k++] = {a, a + (size_t)t[i].n * dtype_bytes((moe_dtype)t[i].param_dtype)};
        }
    std::sort(r, r + k, [](const Range &x, const Range &y) { return x.a < y.a; });
    bool over = false;
    for (int i = 1; i < k; i++) over |= r[i].a < r[i - 1].b;
    delete[] r;
    return over ? fail(MOE_ERR_INVALID_ARG, "two tensors' param overlap") : MOE_OK;
}

}  // namespace aw
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_adamw_step(const moe_adamw_tensor *tensors, int n_tensors, const moe_adamw_options *o,
                                     int32_t *dev_status, moe_stream_t stream)
{
    using namespace aw;
    moe_status st = check(tensors, n_tensors);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(o, "options must not be NULL");
    MOE_REQUIRE(o->beta1 >= 0 && o->beta1 < 1 && o->beta2 >= 0 && o->beta2 < 1, "beta1 and beta2 must be in [0, 1) (got %g, %g)",
                o->beta1, o->beta2);
    MOE_REQUIRE((float)o->eps >= 1.17549435e-38f && (float)o->eps < INFINITY, "eps must be a normal fp32 number above zero (got %g)", o->eps);
    MOE_REQUIRE(o->step_dev || o->step >= 1, "step must be 1 or more (got %lld)", (long long)o->step);
    MOE_REQUIRE(o->lr_dev || (o->lr - o->lr == 0), "lr must be finite (got %g)", o->lr);
    MOE_REQUIRE(aligned_to(o->lr_dev, 4) && aligned_to(o->grad_scale, 4) && aligned_to(o->step_dev, 8) && aligned_to(dev_status, 4),
                "device scalars must be aligned to their types");
    for (int i = 0; i < n_tensors; i++) {
        const moe_adamw_tensor &a = tensors[i];
        if (a.n == 0) continue;
        MOE_REQUIRE(a.param && a.grad, "tensor %d: NULL pointer", i);
        MOE_REQUIRE(dtype_ok((moe_dtype)a.param_dtype) && dtype_ok((moe_dtype)a.grad_dtype),
                    "tensor %d: param_dtype and grad_dtype must be MOE_F32, MOE_BF16 or MOE_F16 (got %d, %d)", i, a.param_dtype,
                    a.grad_dtype);
        MOE_REQUIRE(aligned_to(a.param, dtype_bytes((moe_dtype)a.param_dtype)) && aligned_to(a.grad, dtype_bytes((moe_dtype)a.grad_dtype)) &&
                        aligned_to(a.master, 4),
                    "tensor %d: param, grad and master must be aligned to their types", i);
        MOE_REQUIRE(a.lr_factor - a.lr_factor == 0 && a.weight_decay - a.weight_decay == 0,
                    "tensor %d: lr_factor and weight_decay must be finite (got %g, %g)", i, a.lr_factor, a.weight_decay);
    }
    st = check_overlap(tensors, n_tensors);
    if (st != MOE_OK) return st;
    Common c = {};
    c.b1 = (float)o->beta1, c.o1 = (float)(1.0 - o->beta1), c.b2 = (float)o->beta2, c.o2 = (float)(1.0 - o->beta2);
    c.eps = (float)o->eps, c.lr = (float)o->lr;
    const double t = (double)(o->step_dev ? 1 : o->step), l1 = log(o->beta1), l2 = log(o->beta2);
    c.rate1 = (float)(1.0 / -expm1(t * l1));
    c.root2 = (float)(1.0 / sqrt(-expm1(t * l2)));
    c.log_b1 = (float)l1, c.log_b2 = (float)l2;
    c.lr_dev = o->lr_dev, c.grad_scale = o->grad_scale, c.step_dev = o->step_dev, c.status = dev_status;
    const cudaStream_t s = to_cuda(stream);
    auto one = [&](int i, Tensor &t) {
        const moe_adamw_tensor &a = tensors[i];
        const int n = a.scales ? 8 : 4;  // values that a lane takes at once
        t.vec = aligned_to(a.m, a.scales ? 8 : 16) && aligned_to(a.v, a.scales ? 8 : 16) &&
                aligned_to(a.param, n * dtype_bytes((moe_dtype)a.param_dtype)) &&
                aligned_to(a.grad, n * dtype_bytes((moe_dtype)a.grad_dtype)) && aligned_to(a.master, n * 4);
    };
    bool kinds[2] = {false, false};
    for (int i = 0; i < n_tensors; i++)
        if (tensors[i].n) kinds[tensors[i].scales != nullptr] = true;
    if (kinds[0])
        st = launch(
            tensors, n_tensors, 0, c, "adamw_step", [&](auto &p, unsigned grid) { step_kernel<sizeof(p.t) / sizeof(Tensor), false><<<grid, THREADS, 0, s>>>(p); }, one);
    if (kinds[1] && st == MOE_OK)
        st = launch(
            tensors, n_tensors, 1, c, "adamw_step", [&](auto &p, unsigned grid) { step_kernel<sizeof(p.t) / sizeof(Tensor), true><<<grid, THREADS, 0, s>>>(p); }, one);
    return st;
}

extern "C" moe_status moe_adamw_states(const moe_adamw_tensor *tensors, int n_tensors, float *const *m_values,
                                       float *const *v_values, moe_stream_t stream)
{
    using namespace aw;
    moe_status st = check(tensors, n_tensors);
    if (st != MOE_OK) return st;
    auto out = [&](float *const *a, int i) { return a ? a[i] : nullptr; };
    for (int i = 0; i < n_tensors; i++)
        MOE_REQUIRE(aligned_to(out(m_values, i), 4) && aligned_to(out(v_values, i), 4), "tensor %d: values must be 4-byte aligned", i);
    const cudaStream_t s = to_cuda(stream);
    return launch(
        tensors, n_tensors, -1, Common{}, "adamw_states",
        [&](auto &p, unsigned grid) { states_kernel<<<grid, THREADS, 0, s>>>(p); },
        [&](int i, Tensor &t) {
            t.master = out(m_values, i);
            t.param = out(v_values, i);
            t.vec = t.vec && aligned16(t.master) && aligned16(t.param);
        });
}
