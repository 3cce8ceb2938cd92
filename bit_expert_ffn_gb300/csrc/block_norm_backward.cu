// block_norm_backward.cu -- gradients of the norms around a block.
//
// With d2 = du w_pre:   t  = dy + r2 d2 - y r2^3 mean(d2 y)   (= dx)
// with d1 = alpha gate w_post t:   db = r1 d1 - b r1^3 mean(d1 b)
// dw_pre = sum_t du y r2, dw_post = sum_t alpha gate t b r1, and the gate's from
// the same products.
//
// Bound by memory: four rows in, two out; y and the statistics are recomputed
// from x and b in fp32.  The row is held as in the forward pass, the rows
// ahead come through shared memory.  A thread keeps its columns over all rows
// of its group, so the weights' gradients are register sums, written once per
// CTA and added up by norm_columns_kernel in CTA order (no atomics).  Measured,
// 16,384 x 2048, fp32 stream and bf16 block: 104 us with the column sums (5.8 TB/s).
#include "block_norm.cuh"

namespace moe {

template <class R, class A, class G>
__global__ void __launch_bounds__(G::kThreads) __maxnreg__(G::kBackRegs) block_norm_backward_kernel(const __grid_constant__ NormArgs p)
{
    constexpr int N = G::N;
    constexpr bool kRing = G::NV < 4;
    constexpr bool kKeep = G::NV < 4;  // the weights stay in registers (else they come from L1 for each row)
    extern __shared__ __align__(16) char ring[];
    __shared__ __align__(16) float slots[4][32];
    const int H = p.H, step = gridDim.x * G::count();
    const float inv_h = 1.0f / (float)H;
    const int rs = norm_slot(H, R::kBytes), as = norm_slot(H, A::kBytes), row_bytes = 2 * (rs + as);
    G::clear(slots);
    char *mine = ring + G::index() * p.stages * row_bytes;
    const float *gate_c = p.gate_kind == MOE_GATE_CHANNEL ? p.gate : nullptr;
    auto x_row = [&](int64_t t) { return static_cast<const typename R::T *>(p.x) + t * p.x_stride; };
    auto b_row = [&](int64_t t) { return static_cast<const typename A::T *>(p.b) + t * p.b_stride; };
    auto dy_row = [&](int64_t t) { return static_cast<const typename R::T *>(p.dy) + t * H; };
    auto du_row = [&](int64_t t) { return static_cast<const typename A::T *>(p.du) + t * H; };
    auto fetch = [&](int64_t t, const char *slot) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
        if (t < p.T) {
            norm_fetch<R, G>(to, x_row(t), H);
            norm_fetch<A, G>(to + rs, b_row(t), H);
            if (p.dy) norm_fetch<R, G>(to + rs + as, dy_row(t), H);
            if (p.du) norm_fetch<A, G>(to + 2 * rs + as, du_row(t), H);
        }
        norm_commit();
    };
    const int t0 = blockIdx.x * G::count() + G::index();
    if (kRing)
        for (int s = 0; s < p.stages; s++) fetch((int64_t)t0 + (int64_t)s * step, mine + s * row_bytes);
    float gp[N], gn[N], a1[N] = {}, a2[N] = {};
    if (kKeep) {
        G::weights(p.w_post, gate_c, H, gp);
        G::weights(p.w_pre, nullptr, H, gn);
    }
    int s = 0;
    for (int64_t t = t0; t < p.T; t += step) {
        float y[N], b[N], d[N];  // (du and dy are read again where they are needed: registers are scarcer)
        char *slot = mine + s * row_bytes;
        auto read_du = [&] {
            if (!p.du) {
#pragma unroll
                for (int i = 0; i < N; i++) d[i] = 0.f;
            } else if constexpr (kRing) {
                norm_read<A, G>(slot + 2 * rs + as, du_row(t), H, d);
            } else {
                G::template load<A>(du_row(t), H, d);
            }
        };
        if constexpr (kRing) {
            norm_wait(p.stages);
            if (!G::kVec) G::sync();
            norm_read<A, G>(slot + rs, b_row(t), H, b);
            norm_read<R, G>(slot, x_row(t), H, y);
        } else {
            G::template load<A>(b_row(t), H, b);
            G::template load<R>(x_row(t), H, y);
        }
        float q[1] = {};
#pragma unroll
        for (int i = 0; i < N; i++) q[0] = fmaf(b[i], b[i], q[0]);
        G::sum(q, slots);
        const float r1 = rsqrtf(q[0] * inv_h + p.eps);
        const float gt = p.gate_kind == MOE_GATE_TOKEN ? p.gate[t] : 1.f;
        const float f = p.alpha * r1 * gt;
        if (!kKeep) {
            G::weights(p.w_post, gate_c, H, gp);
            G::weights(p.w_pre, nullptr, H, gn);
        }
        float q2[2] = {};
        read_du();
#pragma unroll
        for (int i = 0; i < N; i++) {
            y[i] = fmaf(f * b[i], gp[i], y[i]);
            q2[0] = fmaf(y[i], y[i], q2[0]);
            q2[1] = fmaf(d[i] * gn[i], y[i], q2[1]);
        }
        G::sum(q2, slots + 1);
        const float r2 = rsqrtf(q2[0] * inv_h + p.eps);
        // (no r cubed, here or below: it leaves fp32's range where rows and gradients do not)
        const float m2 = r2 * (r2 * q2[1] * inv_h);
        q[0] = 0.f;
        read_du();
#pragma unroll
        for (int i = 0; i < N; i++) {
            a2[i] = fmaf(d[i], y[i] * r2, a2[i]);
            y[i] = r2 * (d[i] * gn[i] - y[i] * m2);
        }
        if (p.dy) {
            if constexpr (kRing) norm_read<R, G>(slot + rs + as, dy_row(t), H, d);
            else G::template load<R>(dy_row(t), H, d);
#pragma unroll
            for (int i = 0; i < N; i++) y[i] += d[i];
        }
#pragma unroll
        for (int i = 0; i < N; i++) {  // y holds t now
            a1[i] = fmaf(f * y[i], b[i], a1[i]);
            q[0] = fmaf(y[i] * gp[i], b[i], q[0]);
        }
        G::sum(q, slots + 3);  // sum of t w_post' b
        if (kRing) {  // every thread has read the slot
            if (G::kWarp && !G::kVec) __syncwarp();
            fetch(t + (int64_t)p.stages * step, slot);
            if (++s == p.stages) s = 0;
        }
        G::template store<R>(static_cast<typename R::T *>(p.y) + t * H, H, y);
        const float m1 = f * (r1 * q[0] * inv_h);
#pragma unroll
        for (int i = 0; i < N; i++) b[i] = f * y[i] * gp[i] - b[i] * r1 * m1;
        G::template store<A>(static_cast<typename A::T *>(p.u) + t * H, H, b);
        if (p.dgate_token && G::rank() == 0) p.dgate_token[t] = p.alpha * r1 * q[0];
    }
    float *o = p.part + (int64_t)blockIdx.x * 2 * H;
    if (G::kWarp) {  // the four warps' sums, in order
        __shared__ float acc[G::kWarp ? kNormWarpH : 1];
        for (int k = 0; k < 2; k++) {
            for (int w = 0; w < G::count(); w++) {
                if (w == G::index()) {
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        const int c = G::col(i);
                        if (c < H) acc[c] = (w ? acc[c] : 0.f) + (k ? a2[i] : a1[i]);
                    }
                }
                __syncthreads();
            }
            for (int c = threadIdx.x; c < H; c += blockDim.x) o[k * H + c] = acc[c];
            __syncthreads();
        }
    } else {
        G::template store<F32>(o, H, a1);
        G::template store<F32>(o + H, H, a2);
    }
}

// Column sums of the CTAs' partial rows: a CTA takes 32 columns of one of the
// two, its 32 warps interleaved runs of rows (in order), then the runs in order.
__global__ void __launch_bounds__(1024) norm_columns_kernel(const float *__restrict__ part, int n, int H,
                                                            const float *__restrict__ w_post,
                                                            const float *__restrict__ gate_channel,
                                                            float *__restrict__ dw_post, float *__restrict__ dw_pre,
                                                            float *__restrict__ dgate)
{
    __shared__ float sum[32][33];
    const int c = blockIdx.x * 32 + lane_id(), k = blockIdx.y;
    float a = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int i = warp_id(); i < n; i += 32) a += part[((int64_t)i * 2 + k) * H + c];
    }
    sum[warp_id()][lane_id()] = a;
    __syncthreads();
    if (warp_id() != 0 || c >= H) return;
    a = 0.f;
    for (int i = 0; i < 32; i++) a += sum[i][lane_id()];
    if (k == 1) {
        if (dw_pre) dw_pre[c] = a;
        return;
    }
    if (dw_post) dw_post[c] = gate_channel ? gate_channel[c] * a : a;
    if (dgate) dgate[c] = w_post ? w_post[c] * a : a;
}

// (the workspace's size does not depend on the types: the most that any plan takes)
static int64_t norm_parts(int T, int H)
{
    return norm_plan(T, H, 2, 2, true, true).grid;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_norm_backward_workspace_size(int T, int H, moe_gate gate_kind, size_t *bytes)
{
    MOE_REQUIRE(bytes, "bytes is NULL");
    MOE_REQUIRE(T >= 0 && H >= 1, "T >= 0 and H >= 1 (got T=%d H=%d)", T, H);
    if (H > kNormMaxH) return fail(MOE_ERR_UNSUPPORTED, "H must be at most %d (got %d)", kNormMaxH, H);
    MOE_REQUIRE(gate_kind == MOE_GATE_NONE || gate_kind == MOE_GATE_TOKEN || gate_kind == MOE_GATE_CHANNEL,
                "gate_kind must be a moe_gate (got %d)", (int)gate_kind);
    *bytes = (size_t)norm_parts(T, H) * 2 * H * sizeof(float);
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
    const bool vec = H % 4 == 0 && aligned_to(x, 4 * rb) && aligned_to(b, 4 * ab) && aligned_to(dy, 4 * rb) &&
                     aligned_to(du, 4 * ab) && aligned_to(dx, 4 * rb) && aligned_to(db, 4 * ab) && aligned16(w_post) && aligned16(w_pre) &&
                     (gate_kind != MOE_GATE_CHANNEL || aligned16(gate)) && x_stride % 4 == 0 && b_stride % 4 == 0;
    const NormPlan q = norm_plan(T, H, rb, ab, true, vec);
    const size_t need = (size_t)norm_parts(T, H) * 2 * H * sizeof(float);
    if (!ws || ws_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "block_norm_backward needs %zu bytes (%.2f MiB) of workspace, got %zu", need,
                    mib((double)need), ws ? ws_bytes : (size_t)0);
    MOE_REQUIRE(aligned16(ws), "ws must be 16-byte aligned");
    NormArgs p = {};
    p.x = x, p.b = b, p.x_stride = x_stride, p.b_stride = b_stride, p.T = T, p.H = H, p.w_post = w_post, p.w_pre = w_pre;
    p.gate = gate, p.gate_kind = gate_kind, p.alpha = alpha, p.eps = eps, p.dy = dy, p.du = du, p.y = dx, p.u = db;
    p.dgate_token = gate_kind == MOE_GATE_TOKEN ? dgate : nullptr;
    p.part = static_cast<float *>(ws);
    p.stages = q.stages;
    st = with_norm_types(res_dtype, dtype, [&](auto r, auto a) {
        return with_norm_group(q, [&](auto g) {
            auto fn = block_norm_backward_kernel<decltype(r), decltype(a), decltype(g)>;
            if (q.smem > kNormPlainBytes) MOE_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingBytes));
            fn<<<q.grid, q.threads, q.smem, s>>>(p);
            return check_launch("block_norm_backward");
        });
    });
    if (st != MOE_OK) return st;
    const bool channel = gate_kind == MOE_GATE_CHANNEL;
    if (dw_post || dw_pre || (dgate && channel)) {
        norm_columns_kernel<<<dim3((H + 31) / 32, 2), 1024, 0, s>>>(p.part, q.grid, H, w_post, channel ? gate : nullptr, dw_post,
                                                          dw_pre, channel ? dgate : nullptr);
        return check_launch("norm_columns");
    }
    return MOE_OK;
}
