// block_norm.cuh -- what the norm kernels and their gradients share: a row of
// H columns held by a group of threads, its sums, and its way through shared
// memory.
#pragma once

#include "rows.cuh"

namespace moe {

constexpr int kNormMaxH = 16384;   // 512 threads x 32 columns
constexpr int kNormWarpH = 512;    // rows up to here take one warp, four rows a CTA
constexpr int kNormRingBytes = 200 * 1024;

struct NormArgs {
    const void *x, *b, *dy, *du;
    int64_t x_stride, b_stride;
    int T, H;
    const float *w_post, *w_pre, *gate;
    int gate_kind;
    float alpha, eps;
    void *y, *u;  // the gradients dx and db in the backward pass
    float *dgate_token;
    float *part;  // [gridDim.x][2][H]: sums over the CTA's rows
    int stages;   // rows on their way through shared memory per group (0: rows are read in place)
};

// How a group of threads shares a row.  kWarp: a warp per row, four rows a CTA;
// else the CTA.  A thread holds NV groups of eight columns, consecutive when
// kVec (16 or 32 byte accesses), else strided by the group's width.
template <int NV_, bool kVec_, bool kWarp_>
struct Group {
    static constexpr int NV = NV_, N = NV_ * 8;
    static constexpr bool kVec = kVec_, kWarp = kWarp_;
    static constexpr int kThreads = kWarp ? 128 : 512;  // at most
    // registers of the gradient's kernel: 80 leave room for three CTAs of 256 threads
    static constexpr int kBackRegs = kWarp ? 168 : NV == 1 ? 80 : 128;

    __device__ static int width() { return kWarp ? 32 : (int)blockDim.x; }
    __device__ static int rank() { return kWarp ? lane_id() : (int)threadIdx.x; }
    __device__ static int index() { return kWarp ? warp_id() : 0; }
    __device__ static int count() { return kWarp ? (int)blockDim.x / 32 : 1; }
    __device__ static void sync()
    {
        if (kWarp) __syncwarp();
        else __syncthreads();
    }

    // K sums over the group, the same bits in every thread: lanes by a tree,
    // then the warps in order.  `slots`: 32 floats per sum, not those of the
    // sum before (so one barrier per call is enough).
    template <int K>
    __device__ static void sum(float (&v)[K], float (*slots)[32])
    {
#pragma unroll
        for (int k = 0; k < K; k++)
#pragma unroll
            for (int o = 16; o; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if constexpr (!kWarp) {
#pragma unroll
            for (int k = 0; k < K; k++)
                if (lane_id() == 0) slots[k][warp_id()] = v[k];
            __syncthreads();
            const int warps = (int)(blockDim.x >> 5);
#pragma unroll
            for (int k = 0; k < K; k++) v[k] = 0.f;
            for (int i = 0; i < warps; i++)
#pragma unroll
                for (int k = 0; k < K; k++) v[k] += slots[k][i];
        }
    }

    __device__ static int col(int i) { return kVec ? ((i >> 3) * width() + rank()) * 8 + (i & 7) : rank() + i * width(); }

    template <class A>
    __device__ static void load(const typename A::T *p, int H, float (&v)[N])
    {
        if (kVec) {
#pragma unroll
            for (int g = 0; g < NV; g++) {
                float t[8] = {};
                if (col(g * 8) < H) A::load8(p + col(g * 8), t);
#pragma unroll
                for (int i = 0; i < 8; i++) v[g * 8 + i] = t[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = col(i) < H ? A::load(p + col(i)) : 0.f;
        }
    }
    template <class A>
    __device__ static void store(typename A::T *p, int H, const float (&v)[N])
    {
        if (kVec) {
#pragma unroll
            for (int g = 0; g < NV; g++) {
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; i++) t[i] = v[g * 8 + i];
                if (col(g * 8) < H) A::store8(p + col(g * 8), t);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (col(i) < H) A::store(p + col(i), v[i]);
        }
    }
    // w (NULL: ones), times the channel gate if there is one
    __device__ static void weights(const float *w, const float *gate, int H, float (&v)[N])
    {
        if (w) {
            load<F32>(w, H, v);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = 1.f;
        }
        if (gate) {
            float g[N];
            load<F32>(gate, H, g);
#pragma unroll
            for (int i = 0; i < N; i++) v[i] *= g[i];
        }
    }
};

// Bytes that one array's row takes in shared memory: it may begin anywhere in
// its first 16-byte piece.
__host__ __device__ constexpr int norm_slot(int H, int elem) { return ((H * elem + 15) / 16 + 1) * 16; }

// Starts the copy of a row's 16-byte pieces (those that hold any of it; the
// last one only up to the row's end) into shared memory.
template <class A, class G>
__device__ __forceinline__ void norm_fetch(char *dst, const typename A::T *row, int H)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(row), lo = a & ~uintptr_t(15), end = a + (uintptr_t)H * A::kBytes;
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    for (uintptr_t c = lo + G::rank() * 16; c < end; c += G::width() * 16) {
        const int n = end - c < 16 ? (int)(end - c) : 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + (uint32_t)(c - lo)), "l"(c), "r"(n) : "memory");
    }
}

template <class A>
__device__ __forceinline__ const typename A::T *norm_slot_row(const char *slot, const typename A::T *row)
{
    return reinterpret_cast<const typename A::T *>(slot + (reinterpret_cast<uintptr_t>(row) & 15));
}

__device__ __forceinline__ void norm_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits for the oldest of `stages` rows on their way.
__device__ __forceinline__ void norm_wait(int stages)
{
    if (stages > 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

struct NormPlan {
    int threads, nv, grid, stages;
    size_t smem;
    bool vec, warp;
};

NormPlan norm_plan(int T, int H, int res_bytes, int act_bytes, bool backward, bool vec);

moe_status check_norm(const void *x, moe_dtype res, int64_t x_stride, const void *b, moe_dtype act, int64_t b_stride, int T,
                      int H, const float *gate, int gate_kind, float eps);

template <class F>
moe_status with_norm_types(moe_dtype r, moe_dtype a, F f)
{
    if (r == a) return with_dtype(r, [&](auto t) { return f(t, t); });
    return with_dtype(a, [&](auto t) { return f(F32{}, t); });
}

// Calls f(group) with the plan's group type.
template <class F>
moe_status with_norm_group(const NormPlan &q, F f)
{
    if (q.warp) return q.vec ? f(Group<2, true, true>{}) : f(Group<2, false, true>{});
    if (q.nv == 1) return q.vec ? f(Group<1, true, false>{}) : f(Group<1, false, false>{});
    if (q.nv == 2) return q.vec ? f(Group<2, true, false>{}) : f(Group<2, false, false>{});
    return q.vec ? f(Group<4, true, false>{}) : f(Group<4, false, false>{});
}

}  // namespace moe
