// block_norm.cu -- the norm after a block with its gate and residual scale,
// fused with the norm in front of the next block; and its gradients.
//
//   v = b r1 w_post,  r1 = 1 / sqrt(mean b^2 + eps)
//   y = x + alpha gate v
//   u = y r2 w_pre,   r2 = 1 / sqrt(mean y^2 + eps)
//
// Bound by memory: a row of x and b is read once, y and u are written once.
// One CTA holds a row in registers (8, 16 or 32 columns per thread), so
// nothing is read twice; the means are fp32 sums in a fixed order.
#include "rows.cuh"

namespace moe {

constexpr int kNormMaxH = 16384;  // 512 threads x 32 columns

// Sum over the CTA, the same bits in every thread.  `slot` (32 floats of
// shared memory per call in flight): a caller alternates between two, so one
// barrier per sum is enough.
__device__ __forceinline__ float block_sum(float v, float *slot)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane_id() == 0) slot[warp_id()] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 5); i++) s += slot[i];
    return s;
}

// The columns of one thread: NV groups of eight, consecutive when kVec (16 or
// 32 byte accesses), else strided by the CTA's width.
template <int NV, bool kVec>
struct Cols {
    static constexpr int N = NV * 8;
    __device__ static int col(int i)
    {
        return kVec ? ((i >> 3) * (int)blockDim.x + (int)threadIdx.x) * 8 + (i & 7) : (int)threadIdx.x + i * (int)blockDim.x;
    }
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
    // an fp32 vector, all ones when it is NULL
    __device__ static void load_w(const float *w, int H, float (&v)[N])
    {
        if (w) {
            load<F32>(w, H, v);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = 1.f;
        }
    }
};

struct NormArgs {
    const void *x, *b, *dy, *du;
    int64_t x_stride, b_stride;
    int T, H;
    const float *w_post, *w_pre, *gate;
    int gate_kind;
    float alpha, eps;
    void *y, *u;  // the gradients dx and db in the backward pass
    float *dgate_token;
    float *part;  // [gridDim.x][2][H]: sums of alpha gate' t b r1 and of du y r2 over the CTA's rows
};

template <class R, class A, int NV, bool kVec>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ NormArgs p)
{
    using C = Cols<NV, kVec>;
    constexpr int N = C::N;
    __shared__ float slots[2][32];
    const int H = p.H;
    float gp[N], gn[N];
    C::load_w(p.w_post, H, gp);
    C::load_w(p.w_pre, H, gn);
    if (p.gate_kind == MOE_GATE_CHANNEL) {
        float g[N];
        C::template load<F32>(p.gate, H, g);
#pragma unroll
        for (int i = 0; i < N; i++) gp[i] *= g[i];
    }
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        float x[N], b[N];
        C::template load<A>(static_cast<const typename A::T *>(p.b) + t * p.b_stride, H, b);
        C::template load<R>(static_cast<const typename R::T *>(p.x) + t * p.x_stride, H, x);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) s = fmaf(b[i], b[i], s);
        const float r1 = 1.0f / sqrtf(block_sum(s, slots[0]) / (float)H + p.eps);
        const float f = p.alpha * r1 * (p.gate_kind == MOE_GATE_TOKEN ? p.gate[t] : 1.f);
        s = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) {
            x[i] = fmaf(f * b[i], gp[i], x[i]);
            s = fmaf(x[i], x[i], s);
        }
        const float r2 = 1.0f / sqrtf(block_sum(s, slots[1]) / (float)H + p.eps);
        C::template store<R>(static_cast<typename R::T *>(p.y) + (int64_t)t * H, H, x);
#pragma unroll
        for (int i = 0; i < N; i++) x[i] *= r2 * gn[i];
        C::template store<A>(static_cast<typename A::T *>(p.u) + (int64_t)t * H, H, x);
    }
}

// With d2 = du w_pre:   t  = dy + r2 d2 - y r2^3 mean(d2 y)   (= dx)
// with d1 = alpha gate w_post t:   db = r1 d1 - b r1^3 mean(d1 b)
// y is recomputed from x and b in fp32.  A thread keeps its columns over all
// rows of its CTA, so the weights' gradients are register sums, written once
// per CTA and added up by norm_columns_kernel in CTA order.
template <class R, class A, int NV, bool kVec>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const __grid_constant__ NormArgs p)
{
    using C = Cols<NV, kVec>;
    constexpr int N = C::N;
    __shared__ float slots[4][32];
    const int H = p.H;
    const float inv_h = 1.0f / (float)H;
    float gp[N], gn[N], a1[N] = {}, a2[N] = {};
    C::load_w(p.w_post, H, gp);
    C::load_w(p.w_pre, H, gn);
    if (p.gate_kind == MOE_GATE_CHANNEL) {
        float g[N];
        C::template load<F32>(p.gate, H, g);
#pragma unroll
        for (int i = 0; i < N; i++) gp[i] *= g[i];
    }
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        float y[N], b[N], du[N], dy[N];
        C::template load<A>(static_cast<const typename A::T *>(p.b) + t * p.b_stride, H, b);
        C::template load<R>(static_cast<const typename R::T *>(p.x) + t * p.x_stride, H, y);
        if (p.du) {
            C::template load<A>(static_cast<const typename A::T *>(p.du) + (int64_t)t * H, H, du);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) du[i] = 0.f;
        }
        if (p.dy) {
            C::template load<R>(static_cast<const typename R::T *>(p.dy) + (int64_t)t * H, H, dy);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) dy[i] = 0.f;
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) s = fmaf(b[i], b[i], s);
        const float r1 = 1.0f / sqrtf(block_sum(s, slots[0]) * inv_h + p.eps);
        const float gt = p.gate_kind == MOE_GATE_TOKEN ? p.gate[t] : 1.f;
        const float f = p.alpha * r1 * gt;
        s = 0.f;
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) {
            y[i] = fmaf(f * b[i], gp[i], y[i]);
            s = fmaf(y[i], y[i], s);
            q = fmaf(du[i] * gn[i], y[i], q);
        }
        s = block_sum(s, slots[1]);
        q = block_sum(q, slots[2]);
        const float r2 = 1.0f / sqrtf(s * inv_h + p.eps);
        const float m2 = r2 * r2 * r2 * q * inv_h;
        q = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float n2 = y[i] * r2;
            a2[i] = fmaf(du[i], n2, a2[i]);
            dy[i] = dy[i] + r2 * du[i] * gn[i] - y[i] * m2;
            a1[i] = fmaf(f * dy[i], b[i], a1[i]);
            q = fmaf(dy[i] * gp[i], b[i], q);
        }
        C::template store<R>(static_cast<typename R::T *>(p.y) + (int64_t)t * H, H, dy);
        q = block_sum(q, slots[3]);  // sum of t w_post' b
        const float m1 = p.alpha * gt * r1 * r1 * r1 * q * inv_h;
#pragma unroll
        for (int i = 0; i < N; i++) b[i] = f * gp[i] * dy[i] - b[i] * m1;
        C::template store<A>(static_cast<typename A::T *>(p.u) + (int64_t)t * H, H, b);
        if (p.dgate_token && threadIdx.x == 0) p.dgate_token[t] = p.alpha * r1 * q;
    }
    float *o = p.part + (int64_t)blockIdx.x * 2 * H;
    C::template store<F32>(o, H, a1);
    C::template store<F32>(o + H, H, a2);
}

// Column sums of the CTAs' partial rows, in CTA order: a warp takes 32 columns
// of eight interleaved runs of CTAs (one per warp of the CTA), then the runs.
__global__ void __launch_bounds__(256) norm_columns_kernel(const float *__restrict__ part, int n, int H,
                                                           const float *__restrict__ w_post,
                                                           const float *__restrict__ gate_channel,
                                                           float *__restrict__ dw_post, float *__restrict__ dw_pre,
                                                           float *__restrict__ dgate)
{
    __shared__ float sum[2][8][32];
    const int c = blockIdx.x * 32 + lane_id(), g = warp_id();
    float a = 0.f, b = 0.f;
    if (c < H) {
        for (int i = g; i < n; i += 8) {
            a += part[(int64_t)i * 2 * H + c];
            b += part[((int64_t)i * 2 + 1) * H + c];
        }
    }
    sum[0][g][lane_id()] = a;
    sum[1][g][lane_id()] = b;
    __syncthreads();
    if (g != 0 || c >= H) return;
    a = b = 0.f;
    for (int i = 0; i < 8; i++) {
        a += sum[0][i][lane_id()];
        b += sum[1][i][lane_id()];
    }
    if (dw_post) dw_post[c] = gate_channel ? gate_channel[c] * a : a;
    if (dgate) dgate[c] = w_post ? w_post[c] * a : a;
    if (dw_pre) dw_pre[c] = b;
}

struct NormPlan {
    int threads, nv, grid;
    bool vec;
};

static NormPlan norm_plan(int T, int H, bool vec, int per_sm)
{
    NormPlan q;
    q.vec = vec;
    q.nv = H <= 4096 ? 1 : H <= 8192 ? 2 : 4;  // at most 512 threads
    q.threads = ((H + 8 * q.nv - 1) / (8 * q.nv) + 31) / 32 * 32;
    const int resident = std::max(1, std::min(per_sm, 2048 / q.threads));
    q.grid = (int)std::min<int64_t>(T, (int64_t)sm_count() * resident);
    return q;
}

template <class F>
static moe_status with_norm_types(moe_dtype r, moe_dtype a, F f)
{
    if (r == a) return with_dtype(r, [&](auto t) { return f(t, t); });
    return with_dtype(a, [&](auto t) { return f(F32{}, t); });
}

static moe_status check_norm(const void *x, moe_dtype res, int64_t x_stride, const void *b, moe_dtype act,
                             int64_t b_stride, int T, int H, const float *gate, int gate_kind, float eps)
{
    MOE_REQUIRE(T >= 0 && H >= 1, "T >= 0 and H >= 1 (got T=%d H=%d)", T, H);
    if (H > kNormMaxH) return fail(MOE_ERR_UNSUPPORTED, "H must be at most %d (got %d)", kNormMaxH, H);
    MOE_REQUIRE(dtype_ok(res) && dtype_ok(act) && (res == act || res == MOE_F32),
                "the residual stream is fp32 or of the block's type (got %d, %d)", (int)res, (int)act);
    MOE_REQUIRE(gate_kind == MOE_GATE_NONE || gate_kind == MOE_GATE_TOKEN || gate_kind == MOE_GATE_CHANNEL,
                "gate_kind must be a moe_gate (got %d)", gate_kind);
    MOE_REQUIRE(eps >= 0.f, "eps must be >= 0");
    MOE_REQUIRE(x_stride >= H || x_stride == 0, "x_stride must be 0 or >= H (got %lld)", (long long)x_stride);
    MOE_REQUIRE(b_stride >= H || b_stride == 0, "b_stride must be 0 or >= H (got %lld)", (long long)b_stride);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && b, "NULL pointer");
    MOE_REQUIRE((gate != nullptr) == (gate_kind != MOE_GATE_NONE), "gate must be given exactly when gate_kind is not NONE");
    MOE_REQUIRE(aligned_to(x, dtype_bytes(res)) && aligned_to(b, dtype_bytes(act)) && aligned_to(gate, 4),
                "x, b and gate must be aligned to their types");
    return MOE_OK;
}

constexpr int kNormPerSm = 8, kNormBackPerSm = 3;

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_norm(const void *x, moe_dtype res_dtype, int64_t x_stride, const void *b, moe_dtype dtype,
                                     int64_t b_stride, int T, int H, const float *w_post, const float *w_pre,
                                     const float *gate, moe_gate gate_kind, float alpha, float eps, void *y, void *u,
                                     moe_stream_t stream)
{
    moe_status st = check_norm(x, res_dtype, x_stride, b, dtype, b_stride, T, H, gate, gate_kind, eps);
    if (st != MOE_OK || T == 0) return st;
    MOE_REQUIRE(y && u, "NULL pointer");
    const int rb = dtype_bytes(res_dtype), ab = dtype_bytes(dtype);
    MOE_REQUIRE(aligned_to(y, rb) && aligned_to(u, ab) && aligned_to(w_post, 4) && aligned_to(w_pre, 4),
                "y, u, w_post and w_pre must be aligned to their types");
    const bool vec = H % 8 == 0 && aligned16(x) && aligned16(b) && aligned16(y) && aligned16(u) && aligned16(w_post) &&
                     aligned16(w_pre) && (gate_kind != MOE_GATE_CHANNEL || aligned16(gate)) &&
                     x_stride * rb % 16 == 0 && b_stride * ab % 16 == 0;
    const NormPlan q = norm_plan(T, H, vec, kNormPerSm);
    NormArgs p = {};
    p.x = x, p.b = b, p.x_stride = x_stride, p.b_stride = b_stride, p.T = T, p.H = H, p.w_post = w_post, p.w_pre = w_pre;
    p.gate = gate, p.gate_kind = gate_kind, p.alpha = alpha, p.eps = eps, p.y = y, p.u = u;
    return with_norm_types(res_dtype, dtype, [&](auto r, auto a) {
        using R = decltype(r);
        using A = decltype(a);
        auto fn = q.vec ? (q.nv == 1 ? block_norm_kernel<R, A, 1, true> : q.nv == 2 ? block_norm_kernel<R, A, 2, true> : block_norm_kernel<R, A, 4, true>)
                        : (q.nv == 1 ? block_norm_kernel<R, A, 1, false> : q.nv == 2 ? block_norm_kernel<R, A, 2, false> : block_norm_kernel<R, A, 4, false>);
        fn<<<q.grid, q.threads, 0, to_cuda(stream)>>>(p);
        return check_launch("block_norm");
    });
}

extern "C" moe_status moe_block_norm_backward_workspace_size(int T, int H, moe_gate gate_kind, size_t *bytes)
{
    MOE_REQUIRE(bytes, "bytes is NULL");
    MOE_REQUIRE(T >= 0 && H >= 1, "T >= 0 and H >= 1 (got T=%d H=%d)", T, H);
    if (H > kNormMaxH) return fail(MOE_ERR_UNSUPPORTED, "H must be at most %d (got %d)", kNormMaxH, H);
    MOE_REQUIRE(gate_kind == MOE_GATE_NONE || gate_kind == MOE_GATE_TOKEN || gate_kind == MOE_GATE_CHANNEL,
                "gate_kind must be a moe_gate (got %d)", (int)gate_kind);
    *bytes = (size_t)norm_plan(T, H, true, kNormBackPerSm).grid * 2 * H * sizeof(float);
    return MOE_OK;
}

extern "C" moe_status moe_block_norm_backward(const void *x, moe_dtype res_dtype, int64_t x_stride, const void *b,
                                              moe_dtype dtype, int64_t b_stride, int T, int H, const float *w_post,
                                              const float *w_pre, const float *gate, moe_gate gate_kind, float alpha,
                                              float eps, const void *dy, const void *du, void *dx, void *db,
                                              float *dw_post, float *dw_pre, float *dgate, void *ws, size_t ws_bytes,
                                              moe_stream_t stream)
{
    moe_status st = check_norm(x, res_dtype, x_stride, b, dtype, b_stride, T, H, gate, gate_kind, eps);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(dgate == nullptr || gate_kind != MOE_GATE_NONE, "dgate is given but gate_kind is MOE_GATE_NONE");
    cudaStream_t s = to_cuda(stream);
    if (T == 0) {  // sums over no rows
        if (dw_post) MOE_CUDA_TRY(cudaMemsetAsync(dw_post, 0, sizeof(float) * H, s));
        if (dw_pre) MOE_CUDA_TRY(cudaMemsetAsync(dw_pre, 0, sizeof(float) * H, s));
        if (dgate && gate_kind == MOE_GATE_CHANNEL) MOE_CUDA_TRY(cudaMemsetAsync(dgate, 0, sizeof(float) * H, s));
        return MOE_OK;
    }
    MOE_REQUIRE(dx && db, "NULL pointer");
    const int rb = dtype_bytes(res_dtype), ab = dtype_bytes(dtype);
    MOE_REQUIRE(aligned_to(dy, rb) && aligned_to(dx, rb) && aligned_to(du, ab) && aligned_to(db, ab) &&
                    aligned_to(w_post, 4) && aligned_to(w_pre, 4) && aligned_to(dw_post, 4) && aligned_to(dw_pre, 4) &&
                    aligned_to(dgate, 4),
                "the gradients and weights must be aligned to their types");
    const bool vec = H % 8 == 0 && aligned16(x) && aligned16(b) && aligned16(dy) && aligned16(du) && aligned16(dx) &&
                     aligned16(db) && aligned16(w_post) && aligned16(w_pre) &&
                     (gate_kind != MOE_GATE_CHANNEL || aligned16(gate)) && x_stride * rb % 16 == 0 &&
                     b_stride * ab % 16 == 0;
    const NormPlan q = norm_plan(T, H, vec, kNormBackPerSm);
    const size_t need = (size_t)q.grid * 2 * H * sizeof(float);
    if (!ws || ws_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "block_norm_backward needs %zu bytes (%.2f MiB) of workspace, got %zu", need,
                    mib((double)need), ws ? ws_bytes : (size_t)0);
    MOE_REQUIRE(aligned16(ws), "ws must be 16-byte aligned");
    NormArgs p = {};
    p.x = x, p.b = b, p.x_stride = x_stride, p.b_stride = b_stride, p.T = T, p.H = H, p.w_post = w_post, p.w_pre = w_pre;
    p.gate = gate, p.gate_kind = gate_kind, p.alpha = alpha, p.eps = eps, p.dy = dy, p.du = du, p.y = dx, p.u = db;
    p.dgate_token = gate_kind == MOE_GATE_TOKEN ? dgate : nullptr;
    p.part = static_cast<float *>(ws);
    st = with_norm_types(res_dtype, dtype, [&](auto r, auto a) {
        using R = decltype(r);
        using A = decltype(a);
        auto fn = q.vec ? (q.nv == 1 ? block_norm_backward_kernel<R, A, 1, true> : q.nv == 2 ? block_norm_backward_kernel<R, A, 2, true> : block_norm_backward_kernel<R, A, 4, true>)
                        : (q.nv == 1 ? block_norm_backward_kernel<R, A, 1, false> : q.nv == 2 ? block_norm_backward_kernel<R, A, 2, false> : block_norm_backward_kernel<R, A, 4, false>);
        fn<<<q.grid, q.threads, 0, s>>>(p);
        return check_launch("block_norm_backward");
    });
    if (st != MOE_OK) return st;
    const bool channel = gate_kind == MOE_GATE_CHANNEL;
    if (dw_post || dw_pre || (dgate && channel)) {
        norm_columns_kernel<<<(H + 31) / 32, 256, 0, s>>>(p.part, q.grid, H, w_post, channel ? gate : nullptr, dw_post,
                                                          dw_pre, channel ? dgate : nullptr);
        return check_launch("norm_columns");
    }
    return MOE_OK;
}
