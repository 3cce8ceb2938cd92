// block_norm.cu -- the norm after a block with its gate and residual scale,
// fused with the norm in front of the next block.
//
//   v = b r1 w_post,  r1 = 1 / sqrt(mean b^2 + eps)
//   y = x + alpha gate v
//   u = y r2 w_pre,   r2 = 1 / sqrt(mean y^2 + eps)
//
// Bound by memory: a row of x and b is read once, y and u are written once.
// A row is held in registers by a warp (H up to 512) or a CTA, so nothing is
// read twice; the means are fp32 sums in a fixed order.  A group works through
// several rows, and the next ones are on their way into shared memory
// (cp.async) while it sums: two sums in turn leave the memory idle otherwise.
// Rows of any alignment come in 16-byte pieces.  Measured, 16,384 x 2048: fp32
// stream and bf16 block 69 us (5.9 TB/s), all bf16 45 us (6.0 TB/s).
#include "block_norm.cuh"

namespace moe {

template <class R, class A, class G>
__global__ void __launch_bounds__(G::kThreads) block_norm_kernel(const __grid_constant__ NormArgs p)
{
    constexpr int N = G::N;
    constexpr bool kRing = G::NV < 4;
    extern __shared__ __align__(16) char ring[];
    __shared__ __align__(16) float slots[2][32];
    const int H = p.H, step = gridDim.x * G::count();
    const float inv_h = 1.0f / (float)H;
    const int xs = norm_slot(H, R::kBytes), row_bytes = xs + norm_slot(H, A::kBytes);
    G::clear(slots);
    char *mine = ring + G::index() * p.stages * row_bytes;
    auto x_row = [&](int64_t t) { return static_cast<const typename R::T *>(p.x) + t * p.x_stride; };
    auto b_row = [&](int64_t t) { return static_cast<const typename A::T *>(p.b) + t * p.b_stride; };
    auto fetch = [&](int64_t t, const char *slot) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
        if (t < p.T) {
            norm_fetch<R, G>(to, x_row(t), H);
            norm_fetch<A, G>(to + xs, b_row(t), H);
        }
        norm_commit();
    };
    const int t0 = blockIdx.x * G::count() + G::index();
    if (kRing)
        for (int s = 0; s < p.stages; s++) fetch((int64_t)t0 + (int64_t)s * step, mine + s * row_bytes);
    float gp[N], gn[N];
    G::weights(p.w_post, p.gate_kind == MOE_GATE_CHANNEL ? p.gate : nullptr, H, gp);
    G::weights(p.w_pre, nullptr, H, gn);
    int s = 0;
    for (int64_t t = t0; t < p.T; t += step) {
        float x[N], b[N];
        char *slot = mine + s * row_bytes;
        if (kRing) {
            norm_wait(p.stages);
            if (!G::kVec) G::sync();
            norm_read<A, G>(slot + xs, b_row(t), H, b);
            norm_read<R, G>(slot, x_row(t), H, x);
        } else {
            G::template load<A>(b_row(t), H, b);
            G::template load<R>(x_row(t), H, x);
        }
        float q[1] = {};
#pragma unroll
        for (int i = 0; i < N; i++) q[0] = fmaf(b[i], b[i], q[0]);
        G::sum(q, slots);
        if (kRing) {  // every thread has read the slot
            if (G::kWarp && !G::kVec) __syncwarp();
            fetch(t + (int64_t)p.stages * step, slot);
            if (++s == p.stages) s = 0;
        }
        const float r1 = rsqrtf(q[0] * inv_h + p.eps);
        const float f = p.alpha * r1 * (p.gate_kind == MOE_GATE_TOKEN ? p.gate[t] : 1.f);
        q[0] = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) {
            x[i] = fmaf(f * b[i], gp[i], x[i]);
            q[0] = fmaf(x[i], x[i], q[0]);
        }
        G::sum(q, slots + 1);
        const float r2 = rsqrtf(q[0] * inv_h + p.eps);
        G::template store<R>(static_cast<typename R::T *>(p.y) + t * H, H, x);
#pragma unroll
        for (int i = 0; i < N; i++) x[i] *= r2 * gn[i];
        G::template store<A>(static_cast<typename A::T *>(p.u) + t * H, H, x);
    }
}

NormPlan norm_plan(int T, int H, int res_bytes, int act_bytes, bool backward, bool vec)
{
    NormPlan q = {};
    q.vec = vec;
    q.warp = H <= kNormWarpH;
    // (16384 x 2048: 68.7 us with 16 columns a thread, 71.1 with eight; the
    // gradient, short of registers, 140 and 102)
    q.nv = q.warp ? (H <= 256 ? 1 : 2) : H <= (backward ? 4096 : 1024) ? 1 : H <= 8192 ? 2 : 4;
    const int groups = q.warp ? 4 : 1;
    q.threads = q.warp ? 128 : ((H + 8 * q.nv - 1) / (8 * q.nv) + 31) / 32 * 32;
    const size_t row = (size_t)(backward ? 2 : 1) * (norm_slot(H, res_bytes) + norm_slot(H, act_bytes)) * groups;
    // two rows ahead where they fit, one else; the widest rows are read in place
    q.stages = q.nv == 4 ? 0 : 2 * row <= kNormRingBytes ? 2 : 1;
    q.smem = row * q.stages;
    // threads that an SM holds at the kernels' registers
    const int per_sm = q.nv > 1 ? 512 : backward ? 768 : 1024;
    int resident = std::max(1, std::min(32, per_sm / q.threads));
    if (q.smem) resident = std::max(1, std::min<int>(resident, (int)((kNormRingBytes + 20 * 1024) / (q.smem + 1024))));
    q.grid = (int)std::min<int64_t>(((int64_t)T + groups - 1) / groups, (int64_t)sm_count() * resident);
    return q;
}

moe_status check_norm(const void *x, moe_dtype res, int64_t x_stride, const void *b, moe_dtype act,
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
    const bool vec = H % 4 == 0 && aligned_to(x, 4 * rb) && aligned_to(b, 4 * ab) && aligned_to(y, 4 * rb) && aligned_to(u, 4 * ab) &&
                     aligned16(w_post) &&
                     aligned16(w_pre) && (gate_kind != MOE_GATE_CHANNEL || aligned16(gate)) &&
                     x_stride % 4 == 0 && b_stride % 4 == 0;
    const NormPlan q = norm_plan(T, H, rb, ab, false, vec);
    NormArgs p = {};
    p.x = x, p.b = b, p.x_stride = x_stride, p.b_stride = b_stride, p.T = T, p.H = H, p.w_post = w_post, p.w_pre = w_pre;
    p.gate = gate, p.gate_kind = gate_kind, p.alpha = alpha, p.eps = eps, p.y = y, p.u = u;
    p.stages = q.stages;
    return with_norm_types(res_dtype, dtype, [&](auto r, auto a) {
        return with_norm_group(q, [&](auto g) {
            auto fn = block_norm_kernel<decltype(r), decltype(a), decltype(g)>;
            if (q.smem > kNormPlainBytes) MOE_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingBytes));
            fn<<<q.grid, q.threads, q.smem, to_cuda(stream)>>>(p);
            return check_launch("block_norm");
        });
    });
}
