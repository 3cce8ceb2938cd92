// router_loss.cu -- moe_router_loss: the balance loss, the squared log-sum loss
// and the counts per expert of a batch of router logits; and their gradient
// together with the routing weights'.
//
//   p = softmax(l_t), n tokens, P_e = sum_t p_te / n, f_e = count_e / (n k)
//   loss0 = E sum_e f_e P_e, loss1 = sum_t lse_t^2 / n
//   dl_te = p_te (g_e - sum p g + z lse_t) + [the weights' part],
//   g_e = dloss0 E count_e / (n^2 k), z = 2 dloss1 / n
//
// A warp takes a row whole into registers (a lane four columns side by side, or
// one where rows are not aligned), two rows in turn, one on its way; the logits are
// read once.  The forward sums over tokens stay in the lanes' registers, then
// go warp by warp, CTA by CTA, in a fixed order: through shared memory, then
// through the cluster's shared memory (few tokens, one launch) or the
// workspace (a second, small launch).  The gradient needs the counts and lse of
// the whole batch, so the logits come a second time.
//
// Memory bounds it.  Measured on one GB300, 32,768 x 512 fp32: the losses 17.4 us
// (67 MB; some 12 of the first kernel, 5 of the second), with the gradient 43.5
// (201 MB, part of the logits still in L2); 32 x 512 5.2 us, one launch (device
// times).  Twelve warps a CTA and two CTAs an SM: with 16 the two rows spill.
#include "cluster.cuh"
#include "router_loss_deal.cuh"
#include "rows.cuh"

namespace moe {
namespace rl {

constexpr int MAX_E = 1024, MAX_K = 16;
constexpr int WARPS = 12, THREADS = WARPS * 32;
constexpr int MAX_CLUSTER = 8;
// Up to this many tokens are one cluster's.  Device times by one cluster and by two launches, us: 384 tokens of 64 columns
// 5.9 and 6.1, of 512 7.5 and 7.8, of 1,024 8.4 and 8.9; 512 tokens 6.6 and 6.2, 8.6 and 7.7, 9.8 and 9.1.
constexpr int CLUSTER_ROWS = 384;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float FUSED = 1e6f;  // below it x log2 e is rounded by at most 1/16

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of the warp's values (not NaN), by one integer reduction: the bits of negative values are turned over.
__device__ __forceinline__ float warp_max(float v)
{
    const int b = __float_as_int(v), m = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
    return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

// The kernels of a call, and of the calls after it, are launched while the one before may still run: nothing before this
// reads what that one writes.
__device__ __forceinline__ void next_launch()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How a lane takes a row: single columns, fours of them (aligned rows), fours of a row that fills the lanes' registers.
enum Mode { ONES, FOURS, FULL };

// A row's columns of a lane: 4 (lane + 32 j) + 0..3, or lane + 32 i.
template <Mode M>
__device__ __forceinline__ int column(int i, int lane)
{
    return M != ONES ? 4 * (lane + 32 * (i >> 2)) + (i & 3) : lane + 32 * i;
}

// The lane's columns of a row; those past E as `fill`.
template <class A, int NV, Mode M>
__device__ __forceinline__ void load_row(const typename A::T *row, int E, int lane, float fill, float (&v)[NV])
{
    if (M != ONES) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            const int c = column<M>(i, lane);
            if (M != FULL) v[i] = v[i + 1] = v[i + 2] = v[i + 3] = fill;
            if (M == FULL || c < E) A::load4(row + c, v + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = column<M>(i, lane);
            v[i] = c < E ? A::load(row + c) : fill;
        }
    }
}

// Words of a CTA's part: E sums of p, E counts, sum of lse^2, tokens; whole 16 bytes where the experts are.
__host__ __device__ constexpr int pitch_of(int E) { return 2 * E + 4; }

struct Params {
    const void *logits;
    int T, E, k;
    const int32_t *ids;
    const uint8_t *keep;
    float *loss, *mean, *lse;
    int32_t *counts;
    float *part;  // the CTAs' parts; NULL: one cluster
    int32_t *status;
};

// Sums over `parts` parts in order, a slice of the experts per CTA of the
// cluster.  get<V>(part, i): words i .. i+V-1 of the part's E sums, E counts,
// sum of lse^2 and tokens.  Groups of threads take every G-th part of V columns.
template <int kThreads, int V, class G>
__device__ __forceinline__ void finish(const Params &p, int parts, G get, float *red, float *slot)
{
    const int C = gridDim.x, r = C > 1 ? (int)cluster_rank() : 0, tid = threadIdx.x;
    const int E = p.E, units = (E + V - 1) / V;
    const int e0 = (int)((int64_t)units * r / C) * V, w = (int)((int64_t)units * (r + 1) / C) - e0 / V;
    const Deal d = deal(w, kThreads, parts, V);
    const int per = d.per, groups = d.groups;
    const int g = per ? tid / per : groups, c0 = per ? tid % per : 0;
    __shared__ float s_n, s_z, s_dot[kThreads / 32];
    __shared__ int s_tok;
    float dot = 0.f;
    for (int c = c0;; c += per) {  // (one round, unless a slice is wider than the CTA)
        float a[V];
        int b[V];
#pragma unroll
        for (int i = 0; i < V; i++) a[i] = 0.f, b[i] = 0;
        if (g < groups && c < w) {
#pragma unroll 8
            for (int i = g; i < parts; i += groups) {
                float x[V], y[V];
                get(i, e0 + c * V, x);
                get(i, E + e0 + c * V, y);
#pragma unroll
                for (int j = 0; j < V; j++) a[j] += x[j], b[j] += __float_as_int(y[j]);
            }
        }
        if (groups > 1) {
#pragma unroll
            for (int j = 0; j < V; j++) {
                red[j * kThreads + tid] = a[j];
                red[(V + j) * kThreads + tid] = __int_as_float(b[j]);
            }
        }
        if (c == c0 && tid >= kThreads - 32) {  // tokens and the squares, by the last warp of every CTA
            int n = 0;
            float z = 0.f;
            for (int i = tid & 31; i < parts; i += 256) {  // eight a lane at once
                float x[8][1], y[8][1];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    x[j][0] = y[j][0] = 0.f;
                    if (i + 32 * j < parts) get(i + 32 * j, 2 * E, x[j]), get(i + 32 * j, 2 * E + 1, y[j]);
                }
#pragma unroll
                for (int j = 0; j < 8; j++) z += x[j][0], n += __float_as_int(y[j][0]);
            }
            z = warp_sum(z);
            n = __reduce_add_sync(0xffffffffu, n);
            if ((tid & 31) == 0) s_tok = n, s_n = n > 0 ? (float)n : 1.f, s_z = z;
        }
        __syncthreads();
        const int values = d.values, turns = d.turns;
        const bool twice = d.twice;
        if (twice) {
            float f = 0.f;
            int k = 0;
            const int o = tid % values, j = o / per, first = tid / values;
            if (first < turns) {
                const float *src = red + j * kThreads + o % per;
#pragma unroll 4
                for (int i = first; i < groups; i += turns) {
                    if (j < V) f += src[i * per];
                    else k += __float_as_int(src[i * per]);
                }
            }
            __syncthreads();
            if (first < turns) red[j * kThreads + first * per + o % per] = j < V ? f : __int_as_float(k);
            __syncthreads();
        }
        if (g == 0 && c < w) {
            if (twice) {
#pragma unroll
                for (int j = 0; j < V; j++) a[j] = red[j * kThreads + tid], b[j] = __float_as_int(red[(V + j) * kThreads + tid]);
            }
            const int sums = twice ? turns : groups;
            for (int i = 1; i < sums; i++) {
#pragma unroll
                for (int j = 0; j < V; j++) {
                    a[j] += red[j * kThreads + tid + i * per];
                    b[j] += __float_as_int(red[(V + j) * kThreads + tid + i * per]);
                }
            }
#pragma unroll
            for (int j = 0; j < V; j++) {
                const float m = a[j] / s_n;
                p.mean[e0 + c * V + j] = m;
                p.counts[e0 + c * V + j] = b[j];
                dot += (float)b[j] * m;
            }
        }
        if (per == 0 || c - c0 + per >= w) break;
        __syncthreads();
    }
    dot = warp_sum(dot);
    if ((tid & 31) == 0) s_dot[tid >> 5] = dot;
    __syncthreads();
    if (tid < 32) {
        dot = warp_sum(tid < kThreads / 32 ? s_dot[tid] : 0.f);
        if (tid == 0) *slot = dot;
    }
    if (C > 1) cluster_sync();
    if (r == 0 && tid == 0) {
        dot = 0.f;
        for (int i = 0; i < C; i++) dot += C > 1 ? __uint_as_float(ld_cluster((uint32_t)__cvta_generic_to_shared(slot), i)) : *slot;
        p.loss[0] = (float)E * (dot / (s_n * (float)p.k));
        p.loss[1] = s_z / s_n;
        p.counts[E] = s_tok;
    }
    if (C > 1) cluster_sync();  // no CTA leaves while another reads its slot
}

template <class A, int NV, Mode M>
__global__ void __launch_bounds__(THREADS, NV <= 16 ? 2 : 1) loss_kernel(const __grid_constant__ Params p)
{
    extern __shared__ float dyn[];  // [WARPS][E] sums of p, [E] sums of the CTA, [E] counts, 2; 2 THREADS words for finish
    const int lane = lane_id(), warp = warp_id(), E = p.E, k = p.k;
    float *rows = dyn, *cta = dyn + WARPS * E;
    int *hist = reinterpret_cast<int *>(cta + E);
    __shared__ float s_z[WARPS], s_slot;
    __shared__ int s_tok[WARPS];
    for (int i = threadIdx.x; i < E; i += THREADS) hist[i] = 0;
    __syncthreads();
    next_launch();

    using T = typename A::T;
    const int step = gridDim.x * WARPS;
    int t = blockIdx.x * WARPS + warp, tokens = 0;
    const T *src = static_cast<const T *>(p.logits) + (int64_t)t * E;
    const int64_t src_step = (int64_t)step * E;
    const int32_t *ids = p.ids + (int64_t)t * k + lane;
    float acc[NV], one[NV], two[NV], z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) acc[i] = 0.f;
    int id1 = 0, id2 = 0;
    bool in1 = true, in2 = true;
    auto fetch = [&](int t, float (&v)[NV], int &id, bool &in) {
        load_row<A, NV, M>(src, E, lane, -INFINITY, v);
        if (lane < k) id = *ids;
        if (p.keep) in = p.keep[t] != 0;
        src += src_step;
        ids += step * k;
    };
    auto row = [&](int t, float (&v)[NV], int id, bool in) {
        float top = v[0];
#pragma unroll
        for (int i = 1; i < NV; i++) top = fmaxf(top, v[i]);
        top = warp_max(top);
        // exponents as products and sums in one; where the product's rounding is no small matter, the difference comes first
        float off = top * LOG2E, s = 0.f;
        if (fabsf(top) < FUSED) {
#pragma unroll
            for (int i = 0; i < NV; i++) v[i] = ex2(fmaf(v[i], LOG2E, -off));
        } else {
            off = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++) v[i] = ex2((v[i] - (top == -INFINITY ? 0.f : top)) * LOG2E);
        }
#pragma unroll
        for (int i = 0; i < NV; i++) s += v[i];
        s = warp_sum(s);
        // (s is NaN when a logit is NaN or +inf, 0 when all are -inf)
        if (in && s != s && lane == 0) set_status(p.status, MOE_ERR_NONFINITE);
        const bool counts = in && s > 0.f;
        // (what the product's rounding left out of the exponents; nothing in the other form)
        const float lse = counts ? top + (logf(s) - (off != 0.f ? fmaf(top, LOG2E, -off) * LN2 : 0.f)) : -INFINITY;
        if (lane == 0) p.lse[t] = lse;
        if (lane < k && (unsigned)id >= (unsigned)E && id != MOE_ID_NOT_LOCAL) set_status(p.status, MOE_ERR_BOUNDS);
        if (counts) {
            const float inv = __fdividef(1.f, s);
#pragma unroll
            for (int i = 0; i < NV; i++) acc[i] = fmaf(v[i], inv, acc[i]);
            z = fmaf(lse, lse, z);
            tokens++;
            if (lane < k && (unsigned)id < (unsigned)E) atomicAdd(&hist[id], 1);
        }
    };
    if (t < p.T) fetch(t, one, id1, in1);
    while (t < p.T) {  // two rows in turn, the other one on its way
        if (p.T - t > step) fetch(t + step, two, id2, in2);
        row(t, one, id1, in1);
        if (p.T - t <= step) break;
        t += step;
        if (p.T - t > step) fetch(t + step, one, id1, in1);
        row(t, two, id2, in2);
        if (p.T - t <= step) break;
        t += step;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = column<M>(i, lane);
        if (M == FULL || c < E) rows[warp * E + c] = acc[i];
    }
    if (lane == 0) s_z[warp] = z, s_tok[warp] = tokens;
    __syncthreads();
    for (int c = threadIdx.x; c < E; c += THREADS) {
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; w++) a += rows[w * E + c];
        cta[c] = a;
    }
    if (threadIdx.x == 0) {
        float a = 0.f;
        int n = 0;
        for (int w = 0; w < WARPS; w++) a += s_z[w], n += s_tok[w];
        cta[2 * E] = a;
        reinterpret_cast<int *>(cta)[2 * E + 1] = n;
    }
    __syncthreads();
    if (p.part) {
        for (int c = threadIdx.x; c < 2 * E + 2; c += THREADS) p.part[(int64_t)blockIdx.x * pitch_of(E) + c] = cta[c];
        return;
    }
    const int C = gridDim.x;
    if (C > 1) cluster_sync();
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(cta);
    finish<THREADS, 1>(p, C, [&](int i, int w, float (&v)[1]) { v[0] = C > 1 ? __uint_as_float(ld_cluster(base + w * 4, i)) : cta[w]; },
                       cta + 2 * E + 2, &s_slot);
}

constexpr int FINISH = 1024;

template <int V>
__global__ void __launch_bounds__(FINISH, 1) finish_kernel(const __grid_constant__ Params p, int parts)
{
    __shared__ float red[2 * V * FINISH], slot;
    next_launch();
    const float *part = p.part;
    const int pitch = pitch_of(p.E);
    finish<FINISH, V>(
        p, parts,
        [&](int i, int w, auto &v) {
            const float *q = part + (int64_t)i * pitch + w;
            if constexpr (sizeof(v) == 16) F32::load4(q, v);
            else v[0] = *q;
        },
        red, &slot);
}

// Four values that this call does not read again.
template <class A>
__device__ __forceinline__ void store4_once(typename A::T *p, const float *v)
{
    if constexpr (A::kBytes == 4) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    } else {
        typename A::T q[4];
        A::store4(q, v);
        __stcs(reinterpret_cast<uint2 *>(p), *reinterpret_cast<const uint2 *>(q));
    }
}

struct GradParams {
    const void *logits;
    void *dlogits;
    int T, E, k;
    const int32_t *ids, *counts;
    const float *lse, *dloss, *w, *dw;
};

template <class A, int NV, Mode M>
__global__ void __launch_bounds__(THREADS, NV <= 16 ? 2 : 1) grad_kernel(const __grid_constant__ GradParams p)
{
    extern __shared__ float dyn[];  // [WARPS][E rounded up to 4]: the weights' part of a warp's row; then g
    const int lane = lane_id(), warp = warp_id(), E = p.E, k = p.k;
    using T = typename A::T;
    float *extra = dyn + warp * ((E + 3) & ~3), *g = dyn + WARPS * ((E + 3) & ~3);
    for (int i = lane; i < E; i += 32) extra[i] = 0.f;
    __syncwarp();
    next_launch();
    const int step = gridDim.x * WARPS;
    int t = blockIdx.x * WARPS + warp;
    const T *src = static_cast<const T *>(p.logits) + (int64_t)t * E;
    T *out = static_cast<T *>(p.dlogits) + (int64_t)t * E;
    const int64_t row_step = (int64_t)step * E;
    int64_t pair = (int64_t)t * k + lane;
    float one[NV], two[NV], zc = 0.f, lse1 = 0.f, lse2 = 0.f, w1 = 0.f, w2 = 0.f, d1 = 0.f, d2 = 0.f;
    int id1 = -1, id2 = -1;
    const bool slot = p.w && lane < k, base = p.dloss != nullptr;
    auto fetch = [&](int t, float (&v)[NV], float &lse, int &id, float &w, float &d) {
        if (base) {
            load_row<A, NV, M>(src, E, lane, -INFINITY, v);
            lse = p.lse[t];
        }
        if (slot) id = p.ids[pair], w = p.w[pair], d = p.dw[pair];
        src += row_step;
        pair += step * k;
    };
    auto each_g = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NV; i += M == ONES ? 1 : 4) {
            const int c = column<M>(i, lane);
            if (M != FULL && c >= E) continue;
            if (M != ONES) {
                const float4 a = *reinterpret_cast<const float4 *>(g + c);
                f(i, a.x), f(i + 1, a.y), f(i + 2, a.z), f(i + 3, a.w);
            } else {
                f(i, g[c]);
            }
        }
    };
    auto row = [&](float (&v)[NV], float lse, int id, float w, float d) {
        if (base && lse - lse == 0.f) {
            // p = 2^(l log2 e - lse log2 e), the last product's rounding put right by a factor of the whole row (where it
            // is no small matter, the difference comes first)
            float nl = -lse * LOG2E, right = 1.f, dot = 0.f;
            if (fabsf(lse) < FUSED) {
                right = ex2(-fmaf(lse, LOG2E, nl));
#pragma unroll
                for (int i = 0; i < NV; i++) v[i] = ex2(fmaf(v[i], LOG2E, nl));
            } else {
#pragma unroll
                for (int i = 0; i < NV; i++) v[i] = ex2((v[i] - lse) * LOG2E);
            }
            each_g([&](int i, float gi) { dot = fmaf(v[i], gi, dot); });
            const float add = right * (zc * lse - right * warp_sum(dot));
            each_g([&](int i, float gi) { v[i] *= fmaf(gi, right, add); });
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++) v[i] = 0.f;
        }
        const bool mine = slot && (unsigned)id < (unsigned)E;
        if (p.w) {
            float u = w * (d - warp_sum(w * d));  // (w = d = 0 in the lanes without a slot)
            // (an expert named twice gets the sum, in the slots' order, at its first slot)
            const uint32_t same = __match_any_sync(0xffffffffu, mine ? id : E + lane);
            const bool first = mine && (same & ((1u << lane) - 1)) == 0;
            if (__any_sync(0xffffffffu, mine && !first)) {
                float total = 0.f;
                for (int j = 0; j < k; j++) {
                    const float o = __shfl_sync(0xffffffffu, u, j);
                    if (same >> j & 1) total += o;
                }
                u = total;
            }
            if (first) extra[id] = u;
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < NV; i += M == ONES ? 1 : 4) {
            const int c = column<M>(i, lane);
            if (M != FULL && c >= E) continue;
            if (M != ONES) {
                if (p.w) {
                    const float4 a = *reinterpret_cast<const float4 *>(extra + c);
                    v[i] += a.x, v[i + 1] += a.y, v[i + 2] += a.z, v[i + 3] += a.w;
                }
                store4_once<A>(out + c, v + i);
            } else {
                A::store(out + c, p.w ? v[i] + extra[c] : v[i]);
            }
        }
        out += row_step;
        __syncwarp();
        if (mine) extra[id] = 0.f;
        __syncwarp();
    };
    if (t < p.T) fetch(t, one, lse1, id1, w1, d1);
    if (base) {
        const float n = (float)max(p.counts[E], 1), c = p.dloss[0] * (float)E / n / (n * (float)k);
        zc = 2.f * p.dloss[1] / n;
        for (int i = threadIdx.x; i < E; i += THREADS) g[i] = c * (float)p.counts[i];
    }
    __syncthreads();
    while (t < p.T) {  // two rows in turn, the other one on its way
        if (p.T - t > step) fetch(t + step, two, lse2, id2, w2, d2);
        row(one, lse1, id1, w1, d1);
        if (p.T - t <= step) break;
        t += step;
        if (p.T - t > step) fetch(t + step, one, lse1, id1, w1, d1);
        row(two, lse2, id2, w2, d2);
        if (p.T - t <= step) break;
        t += step;
    }
}

// CTAs of the large form: two an SM, or one where a row takes a lane's 32 registers.
static int grid_of(int T, int E) { return std::min((T + WARPS - 1) / WARPS, sm_count() * (E <= 512 ? 2 : 1)); }

static size_t loss_smem(int E) { return ((size_t)WARPS * E + 2 * E + 2 + 2 * THREADS) * 4; }
static size_t grad_smem(int E) { return (size_t)(WARPS + 1) * ((E + 3) & ~3) * 4; }

// Calls f with the registers of a row and how they are filled (`fours`: rows are aligned for four columns at once).
template <class F>
moe_status with_row(int E, bool fours, F f)
{
    auto mode = [&](auto nv) {
        if (fours && E == 32 * decltype(nv)::value) return f(nv, std::integral_constant<Mode, FULL>{});
        if (fours) return f(nv, std::integral_constant<Mode, FOURS>{});
        return f(nv, std::integral_constant<Mode, ONES>{});
    };
    if (E <= 128) return mode(std::integral_constant<int, 4>{});
    if (E <= 256) return mode(std::integral_constant<int, 8>{});
    if (E <= 512) return mode(std::integral_constant<int, 16>{});
    return mode(std::integral_constant<int, 32>{});
}

static moe_status check(moe_dtype dtype, int T, int E, int k)
{
    MOE_REQUIRE(dtype_ok(dtype), "dtype must be MOE_F32, MOE_BF16 or MOE_F16 (got %d)", (int)dtype);
    MOE_REQUIRE(E >= 1 && E <= MAX_E, "E must be in [1, %d] (got %d)", MAX_E, E);
    MOE_REQUIRE(k >= 1 && k <= std::min(E, MAX_K), "k must be in [1, min(E, %d)] (got %d)", MAX_K, k);
    MOE_REQUIRE(T >= 0 && (int64_t)T * k < (1ll << 31), "T must be in [0, 2^31 / k) (got %d)", T);
    return MOE_OK;
}

static bool vec_rows(const void *p, moe_dtype t, int E) { return E % 4 == 0 && aligned_to(p, 4 * dtype_bytes(t)); }

}  // namespace rl
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_router_loss_workspace_size(int T, int E, size_t *bytes)
{
    using namespace rl;
    MOE_REQUIRE(bytes, "bytes must not be NULL");
    moe_status st = check(MOE_F32, T, E, 1);
    if (st != MOE_OK) return st;
    *bytes = T <= CLUSTER_ROWS ? 0 : (size_t)grid_of(T, E) * pitch_of(E) * 4;
    return MOE_OK;
}

extern "C" moe_status moe_router_loss(const void *logits, moe_dtype dtype, int T, int E, const int32_t *ids, int k,
                                      const uint8_t *keep, float *loss, int32_t *counts, float *mean_prob, float *lse,
                                      void *ws, size_t ws_bytes, int32_t *dev_status, moe_stream_t stream)
{
    using namespace rl;
    moe_status st = check(dtype, T, E, k);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(loss && counts && mean_prob && (T == 0 || (logits && ids && lse)), "NULL pointer");
    MOE_REQUIRE(aligned_to(logits, dtype_bytes(dtype)) && aligned_to(ids, 4) && aligned_to(loss, 4) && aligned_to(counts, 4) &&
                    aligned_to(mean_prob, 4) && aligned_to(lse, 4) && aligned_to(dev_status, 4),
                "tensors must be aligned to their types");
    size_t need = 0;
    st = moe_router_loss_workspace_size(T, E, &need);
    if (st != MOE_OK) return st;
    if (ws_bytes < need || (need && !ws))
        return fail(MOE_ERR_WORKSPACE, "moe_router_loss needs %zu bytes of workspace (got %zu)", need, ws ? ws_bytes : (size_t)0);
    MOE_REQUIRE(!need || aligned16(ws), "ws must be 16-byte aligned");
    Params p = {logits, T, E, k, ids, keep, loss, mean_prob, lse, counts, need ? static_cast<float *>(ws) : nullptr, dev_status};
    const cudaStream_t s = to_cuda(stream);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int grid = grid_of(T, E);
    if (!need) {  // one cluster: a row or more per warp
        int c = 1;
        while (c < MAX_CLUSTER && c * WARPS < T) c *= 2;
        grid = c;
        at[1].val.clusterDim.x = (unsigned)c;
        cfg.numAttrs = 2;
    }
    cfg.gridDim = dim3((unsigned)grid);
    cfg.dynamicSmemBytes = loss_smem(E);
    st = with_dtype(dtype, [&](auto a) {
        return with_row(E, vec_rows(logits, dtype, E), [&](auto nv, auto mode) {
            auto fn = loss_kernel<decltype(a), decltype(nv)::value, decltype(mode)::value>;
            if (cfg.dynamicSmemBytes > 40 * 1024)  // (with the static part more than the 48 KB of any kernel)
                MOE_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)loss_smem(32 * decltype(nv)::value)));
            MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, fn, p));
            return check_launch("router_loss");
        });
    });
    if (st != MOE_OK || !need) return st;
    int c = 1;
    while (c < MAX_CLUSTER && c * 64 < E) c *= 2;
    at[1].val.clusterDim.x = (unsigned)c;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(FINISH);
    cfg.dynamicSmemBytes = 0;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, E % 4 == 0 ? finish_kernel<4> : finish_kernel<1>, p, grid));
    return check_launch("router_loss_finish");
}

extern "C" moe_status moe_router_loss_backward(const void *logits, moe_dtype dtype, int T, int E, const int32_t *ids, int k,
                                               const int32_t *counts, const float *lse, const float *dloss, const float *w,
                                               const float *dw, void *dlogits, moe_stream_t stream)
{
    using namespace rl;
    moe_status st = check(dtype, T, E, k);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(dlogits && (!dloss || (logits && counts && lse)), "NULL pointer");
    MOE_REQUIRE(!w == !dw && (!w || ids), "w and dw go together, and with ids");
    MOE_REQUIRE(aligned_to(logits, dtype_bytes(dtype)) && aligned_to(dlogits, dtype_bytes(dtype)) && aligned_to(ids, 4) &&
                    aligned_to(counts, 4) && aligned_to(lse, 4) && aligned_to(dloss, 4) && aligned_to(w, 4) && aligned_to(dw, 4),
                "tensors must be aligned to their types");
    GradParams p = {logits, dlogits, T, E, k, ids, counts, lse, dloss, w, dw};
    return with_dtype(dtype, [&](auto a) {
        return with_row(E, vec_rows(logits, dtype, E) && vec_rows(dlogits, dtype, E), [&](auto nv, auto mode) {
            auto fn = grad_kernel<decltype(a), decltype(nv)::value, decltype(mode)::value>;
            if (grad_smem(E) > 40 * 1024)
                MOE_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)grad_smem(32 * decltype(nv)::value)));
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)grid_of(T, E));
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = grad_smem(E);
            cfg.stream = to_cuda(stream);
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, fn, p));
            return check_launch("router_loss_backward");
        });
    });
}
