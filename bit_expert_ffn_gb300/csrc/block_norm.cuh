// block_norm.cuh -- what the norm kernels and their gradients share: a row of
// H columns held by a group of threads, its sums, and its way through shared
// memory.
#pragma once

#include "rows.cuh"

namespace moe {

constexpr int kNormMaxH = 16384;   // 512 threads x 32 columns
constexpr int kNormWarpH = 512;    // rows up to here take one warp, four rows a CTA
constexpr int kNormRingBytes = 200 * 1024;
constexpr size_t kNormPlainBytes = 40 * 1024;  // more needs the larger limit (48 KB count the kernels' own, too)

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
// else the CTA.  A thread holds 8 NV columns: fours, strided by the group's
// width, when kVec (a warp's access is 256 or 512 bytes in a row; eights gave
// fp32 rows half sectors, 156 against 100 us for the gradient of 16384 x 2048), else twos.
template <int NV_, bool kVec_, bool kWarp_>
struct Group {
    static constexpr int NV = NV_, N = NV_ * 8;
    static constexpr bool kVec = kVec_, kWarp = kWarp_;
    static constexpr int kThreads = kWarp ? 128 : 512;  // at most
    // registers of the gradient's kernel: 80 leave room for three CTAs of 256 threads
    static constexpr int kBackRegs = NV == 1 ? 80 : 128;

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
    // then the warps in fours.  `slots`: 32 floats per sum, not those of the
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
#pragma unroll
            for (int k = 0; k < K; k++) {
                v[k] = 0.f;
#pragma unroll
                for (int i = 0; i < kThreads / 128; i++) {
                    if (i * 128 >= (int)blockDim.x) break;
                    const float4 q = reinterpret_cast<const float4 *>(slots[k])[i];  // zero past the last warp
                    v[k] += (q.x + q.y) + (q.z + q.w);
                }
            }
        }
    }

    // Before the first sum.
    template <int K>
    __device__ static void clear(float (&slots)[K][32])
    {
        if constexpr (!kWarp) {
            for (int i = threadIdx.x; i < K * 32; i += blockDim.x) slots[i / 32][i % 32] = 0.f;
            __syncthreads();
        }
    }

    __device__ static int col(int i)
    {
        return kVec ? ((i >> 2) * width() + rank()) * 4 + (i & 3) : ((i >> 1) * width() + rank()) * 2 + (i & 1);
    }
    // Unaligned rows go by pairs where their length is even.
    template <class A>
    __device__ static bool pairs(const typename A::T *p, int H)
    {
        return H % 2 == 0 && (reinterpret_cast<uintptr_t>(p) & (2 * A::kBytes - 1)) == 0;
    }

    template <class A>
    __device__ static void load(const typename A::T *p, int H, float (&v)[N])
    {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                v[i] = v[i + 1] = v[i + 2] = v[i + 3] = 0.f;
                if (col(i) < H) A::load4(p + col(i), v + i);
            }
        } else if (pairs<A>(p, H)) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float t[2] = {};
                if (col(i) < H) Unit<A, 2>::unpack(Unit<A, 2>::raw(p + col(i)), t);
                v[i] = t[0], v[i + 1] = t[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = col(i) < H ? A::load(p + col(i)) : 0.f;
        }
    }
    template <class A>
    __device__ static void store(typename A::T *p, int H, const float (&v)[N])
    {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                if (col(i) < H) A::store4(p + col(i), v + i);
        } else if (pairs<A>(p, H)) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float t[2] = {v[i], v[i + 1]};
                if (col(i) < H) Unit<A, 2>::store(p + col(i), t);
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

__device__ __forceinline__ void norm_copy16(uint32_t dst, const void *src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Starts the copy of a row into shared memory.  Aligned rows: each thread
// fetches the pieces of its own columns and needs no barrier to read them.  Others: all 16-byte
// pieces that hold any of the row, the last one only up to the row's end.
template <class A, class G>
__device__ __forceinline__ void norm_fetch(uint32_t dst, const typename A::T *row, int H)
{
    if constexpr (G::kVec) {
#pragma unroll
        for (int i = 0; i < G::N; i += 4) {
            const int c = G::col(i);
            if (c >= H) break;
            if (A::kBytes == 4) norm_copy16(dst + c * 4, row + c, 16);
            else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + c * 2), "l"(row + c) : "memory");
        }
    } else {
        const uintptr_t a = reinterpret_cast<uintptr_t>(row), lo = a & ~uintptr_t(15), end = a + (uintptr_t)H * A::kBytes;
        for (uintptr_t c = lo + G::rank() * 16; c < end; c += G::width() * 16)
            norm_copy16(dst + (uint32_t)(c - lo), reinterpret_cast<const void *>(c), end - c < 16 ? (int)(end - c) : 16);
    }
}

// The thread's columns of a row fetched to `slot` (`row`: where it came from).
template <class A, class G>
__device__ __forceinline__ void norm_read(const char *slot, const typename A::T *row, int H, float (&v)[G::N])
{
    if constexpr (G::kVec) {
        G::template load<A>(reinterpret_cast<const typename A::T *>(slot), H, v);
    } else {
        G::template load<A>(reinterpret_cast<const typename A::T *>(slot + (reinterpret_cast<uintptr_t>(row) & 15)), H, v);
    }
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
    if (q.warp && q.nv == 1) return q.vec ? f(Group<1, true, true>{}) : f(Group<1, false, true>{});
    if (q.warp) return q.vec ? f(Group<2, true, true>{}) : f(Group<2, false, true>{});
    if (q.nv == 1) return q.vec ? f(Group<1, true, false>{}) : f(Group<1, false, false>{});
    if (q.nv == 2) return q.vec ? f(Group<2, true, false>{}) : f(Group<2, false, false>{});
    return q.vec ? f(Group<4, true, false>{}) : f(Group<4, false, false>{});
}

}  // namespace moe
