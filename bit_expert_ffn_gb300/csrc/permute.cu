// permute.cu -- moe_permute: stable counting sort of the T*k (token, slot)
// pairs by expert id.  All integer work, bit-exact and deterministic: counts
// may be gathered with atomics (integer sums do not depend on order), but
// every position comes from ordered scans.
//
// The pages group the tokens of a verify window that share an expert
// ("Strata serves a 125B MoE at 94 tokens/s from a 12 GB card and 64 GB of
// RAM", section "Six billion active parameters per token").
#include "cluster.cuh"
#include "common.cuh"

namespace moe {

constexpr int kPermChunk = 2048;     // pairs per chunk in the multi-CTA path
constexpr int kPlaceWarps = 8;       // warps per chunk in the multi-CTA path
// Up to 128 pairs by counting (10 of them over 512 experts take 1.6 us, a single
// CTA 2.5; 128 take 2.2 and 2.7).  A single CTA up to 1,024, a cluster from
// there: 4,000 pairs over 512 experts take it 5.3 us, a single CTA 8.9; 20,480
// take it 8.3, the three passes 11.9 (40,960: 12.0 and 11.5).  Only the three
// passes need a workspace.
constexpr int kClusterCtas = 8;
constexpr int kPermSmallMax = 1024, kPermClusterMax = 32768;
constexpr int kPermRankMax = 128, kRankThreads = 128;

// Warp-serial stable placement of pairs [f0, f1) starting from per-expert
// cursors `cur` (shared memory).  Lanes take 32 pairs at a time in order.
__device__ void place_pairs(const int32_t *__restrict__ ids, int64_t f0, int64_t f1, int E, int32_t *cur,
                            int32_t *__restrict__ perm, int32_t *__restrict__ inv)
{
    int lane = lane_id();
    unsigned lt = (1u << lane) - 1u;
    // the ids of the next two rounds are on their way
    auto at = [&](int64_t f) { return f < f1 ? ids[f] : -1; };
    int id0 = at(f0 + lane), id1 = at(f0 + 32 + lane);
    for (int64_t base = f0; base < f1; base += 32) {
        int64_t f = base + lane;
        bool in = f < f1;
        const int id = id0;
        id0 = id1;
        id1 = at(f + 64);
        bool valid = in && id >= 0 && id < E;
        int key = valid ? id : (in ? -1 : -2);  // invalid lanes never match a valid id
        unsigned m = __match_any_sync(0xffffffffu, key);
        if (valid) {
            int pos = cur[id] + __popc(m & lt);
            perm[pos] = (int32_t)f;
            inv[f] = pos;
        } else if (in) {
            inv[f] = -1;
        }
        __syncwarp();
        if (valid && (m & lt) == 0) cur[id] += __popc(m);
        __syncwarp();
    }
}

// The warps of a CTA share pairs [f0, f1): warp w takes the w-th run of `seg`
// (a multiple of 32) pairs.  A warp places 32 pairs in some 0.4 us whatever
// it does beside (a chain of dependent steps), so the runs are short: each
// warp first counts its own, and starts from the counts of the warps before.
// hist: [warps][E] int32 in shared memory.
__device__ void count_runs(const int32_t *__restrict__ ids, int64_t f0, int64_t f1, int seg, int E, int warps,
                           int32_t *hist, int32_t *status)
{
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    if (warp_id() < warps) {
        const int64_t a = f0 + (int64_t)warp_id() * seg, b = min(f1, a + seg);
        for (int64_t f = a + lane_id(); f < b; f += 32) {
            const int id = ids[f];
            if (id >= 0 && id < E) atomicAdd(&hist[warp_id() * E + id], 1);
            else if (id != MOE_ID_NOT_LOCAL) set_status(status, MOE_ERR_BOUNDS);
        }
    }
    __syncthreads();
}

// Counts become cursors: expert e's first warp starts at `start`.
__device__ __forceinline__ void runs_to_cursors(int e, int E, int warps, int start, int32_t *hist)
{
    for (int w = 0; w < warps; w++) {
        const int c = hist[w * E + e];
        hist[w * E + e] = start;
        start += c;
    }
}

// Block-wide exclusive scan of one int per thread (blockDim.x <= 1024).
__device__ int block_exclusive_scan(int v, int32_t *warp_tot, int &total)
{
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane_id() >= o) incl += y;
    }
    if (lane_id() == 31) warp_tot[warp_id()] = incl;
    __syncthreads();
    if (warp_id() == 0) {
        int nw = blockDim.x >> 5;
        int wt = lane_id() < nw ? warp_tot[lane_id()] : 0;
        int wi = wt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            int y = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane_id() >= o) wi += y;
        }
        if (lane_id() < nw) warp_tot[lane_id()] = wi - wt;
        if (lane_id() == 31) warp_tot[32] = wi;
    }
    __syncthreads();
    int excl = incl - v + warp_tot[warp_id()];
    total = warp_tot[32];
    __syncthreads();
    return excl;
}

// A few pairs: every expert's offset and every pair's place is a count of the
// keys before its own, id * kPermRankMax + pair, all of them in shared memory.
// The first CTA places the pairs, the others take kRankThreads experts each;
// none waits for another.
__global__ void __launch_bounds__(kRankThreads) permute_rank_kernel(const int32_t *__restrict__ ids, int n, int E,
                                                                    int32_t *__restrict__ offsets, int32_t *__restrict__ perm,
                                                                    int32_t *__restrict__ inv, int32_t *status)
{
    __shared__ __align__(16) int32_t key[kPermRankMax];
    const int tid = threadIdx.x;
    const int id = tid < n ? ids[tid] : MOE_ID_NOT_LOCAL;
    const bool valid = id >= 0 && id < E;
    const int mine = valid ? id * kPermRankMax + tid : INT32_MAX;  // after every expert
    if (!valid && id != MOE_ID_NOT_LOCAL && blockIdx.x == 0) set_status(status, MOE_ERR_BOUNDS);
    if (tid < kPermRankMax) key[tid] = mine;
    const int total = __syncthreads_count(valid);
    auto before = [&](int x) {
        int c = 0;
#pragma unroll 4
        for (int i = 0; i < n; i += 4) {
            const int4 k = *reinterpret_cast<const int4 *>(key + i);
            c += (k.x < x) + (k.y < x) + (k.z < x) + (k.w < x);
        }
        return c;
    };
    if (blockIdx.x > 0) {
        const int e = ((int)blockIdx.x - 1) * kRankThreads + tid;
        if (e <= E) offsets[e] = before(e * kPermRankMax);
    } else if (tid < n) {
        const int pos = valid ? before(mine) : -1;
        inv[tid] = pos;
        if (valid) perm[pos] = tid;
        if (tid >= total) perm[tid] = -1;
    }
}

// Single CTA (1024 threads): count, scan, place.
__global__ void __launch_bounds__(1024) permute_small_kernel(const int32_t *__restrict__ ids, int n, int E, int warps,
                                                             int seg, int32_t *__restrict__ offsets,
                                                             int32_t *__restrict__ perm, int32_t *__restrict__ inv,
                                                             int32_t *status)
{
    extern __shared__ int32_t hist[];
    __shared__ int32_t warp_tot[33];
    int tid = threadIdx.x;
    count_runs(ids, 0, n, seg, E, warps, hist, status);
    int v = 0;
    if (tid < E)
        for (int w = 0; w < warps; w++) v += hist[w * E + tid];
    int total = 0;
    int excl = block_exclusive_scan(v, warp_tot, total);
    if (tid < E) {
        offsets[tid] = excl;
        runs_to_cursors(tid, E, warps, excl, hist);
    }
    if (tid == 0) offsets[E] = total;
    for (int p = total + tid; p < n; p += blockDim.x) perm[p] = -1;
    __syncthreads();
    if (warp_id() < warps) {
        const int64_t f0 = (int64_t)warp_id() * seg;
        place_pairs(ids, f0, min((int64_t)n, f0 + seg), E, hist + warp_id() * E, perm, inv);
    }
}

// One cluster of CTAs, a share of the pairs each (per_cta, a multiple of 32):
// as the single CTA, but an expert's start also counts the CTAs before, whose
// counts are read from their shared memory.
__global__ void __launch_bounds__(1024) permute_cluster_kernel(const int32_t *__restrict__ ids, int n, int E, int per_cta,
                                                               int warps, int seg, int32_t *__restrict__ offsets,
                                                               int32_t *__restrict__ perm, int32_t *__restrict__ inv,
                                                               int32_t *status)
{
    extern __shared__ int32_t hist[];
    __shared__ int32_t mine[1024];
    __shared__ int32_t warp_tot[33];
    const int tid = threadIdx.x, rank = (int)cluster_rank();
    const int64_t f0 = min((int64_t)n, (int64_t)rank * per_cta), f1 = min((int64_t)n, f0 + per_cta);
    count_runs(ids, f0, f1, seg, E, warps, hist, status);
    if (tid < E) {
        int v = 0;
        for (int w = 0; w < warps; w++) v += hist[w * E + tid];
        mine[tid] = v;
    }
    cluster_sync();
    int before = 0, all = 0;
    if (tid < E) {
        const uint32_t a = (uint32_t)__cvta_generic_to_shared(&mine[tid]);
        int v[kClusterCtas];
#pragma unroll
        for (int r = 0; r < kClusterCtas; r++) v[r] = (int)ld_cluster(a, r);
#pragma unroll
        for (int r = 0; r < kClusterCtas; r++) {
            before += r < rank ? v[r] : 0;
            all += v[r];
        }
    }
    int total = 0;
    const int excl = block_exclusive_scan(all, warp_tot, total);
    if (tid < E) {
        if (rank == 0) offsets[tid] = excl;
        runs_to_cursors(tid, E, warps, excl + before, hist);
    }
    if (rank == 0 && tid == 0) offsets[E] = total;
    for (int p = total + rank * (int)blockDim.x + tid; p < n; p += kClusterCtas * (int)blockDim.x) perm[p] = -1;
    __syncthreads();
    if (warp_id() < warps) {
        const int64_t a = f0 + (int64_t)warp_id() * seg;
        place_pairs(ids, a, min(f1, a + seg), E, hist + warp_id() * E, perm, inv);
    }
    cluster_sync();  // no CTA leaves while another reads its counts
}

// Multi-CTA pass 1: per-chunk histograms -> counts[chunk][E].
__global__ void permute_count_kernel(const int32_t *__restrict__ ids, int64_t n, int E, int32_t *__restrict__ counts,
                                     int32_t *status)
{
    __shared__ int32_t h[1024];
    for (int e = threadIdx.x; e < E; e += blockDim.x) h[e] = 0;
    __syncthreads();
    int64_t f0 = (int64_t)blockIdx.x * kPermChunk;
    int64_t f1 = min(n, f0 + kPermChunk);
    for (int64_t f = f0 + threadIdx.x; f < f1; f += blockDim.x) {
        int id = ids[f];
        if (id >= 0 && id < E) atomicAdd(&h[id], 1);
        else if (id != MOE_ID_NOT_LOCAL) set_status(status, MOE_ERR_BOUNDS);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[(int64_t)blockIdx.x * E + e] = h[e];
}

// Multi-CTA pass 2: base[chunk][e] = expert e's pairs in the chunks before.  A CTA
// takes 32 experts, its 32 warps runs of chunks.
__global__ void __launch_bounds__(1024) permute_prefix_kernel(const int32_t *__restrict__ counts, int n_chunks, int E,
                                                              int32_t *__restrict__ base)
{
    __shared__ int32_t sum[32][33];
    const int e = blockIdx.x * 32 + lane_id(), w = warp_id();
    const int run = (n_chunks + 31) / 32, c0 = min(n_chunks, w * run), c1 = min(n_chunks, c0 + run);
    int v = 0;
    if (e < E) {
#pragma unroll 8
        for (int c = c0; c < c1; c++) v += counts[(int64_t)c * E + e];
    }
    sum[w][lane_id()] = v;
    __syncthreads();
    if (e >= E) return;
    int before = 0;
    for (int i = 0; i < w; i++) before += sum[i][lane_id()];
#pragma unroll 8
    for (int c = c0; c < c1; c++) {
        base[(int64_t)c * E + e] = before;
        before += counts[(int64_t)c * E + e];
    }
}

// Multi-CTA pass 3: a CTA of kPlaceWarps warps per chunk places its pairs in
// order.  Each scans the experts' totals (the last chunk's base and count) for
// itself; the first writes the offsets.
__global__ void __launch_bounds__(kPlaceWarps * 32) permute_place_kernel(const int32_t *__restrict__ ids, int64_t n, int E,
                                                                         const int32_t *__restrict__ counts,
                                                                         const int32_t *__restrict__ base,
                                                                         int32_t *__restrict__ offsets,
                                                                         int32_t *__restrict__ perm,
                                                                         int32_t *__restrict__ inv)
{
    __shared__ int32_t hist[kPlaceWarps * 1024];
    __shared__ int32_t warp_tot[33];
    constexpr int seg = kPermChunk / kPlaceWarps, kThreads = kPlaceWarps * 32, kPer = 1024 / kThreads;
    const int64_t f0 = (int64_t)blockIdx.x * kPermChunk, f1 = min(n, f0 + kPermChunk);
    const int64_t last = ((int64_t)gridDim.x - 1) * E;
    int start[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = threadIdx.x * kPer + i;
        start[i] = sum;
        if (e < E) sum += base[last + e] + counts[last + e];
    }
    count_runs(ids, f0, f1, seg, E, kPlaceWarps, hist, nullptr);
    int total = 0;
    const int excl = block_exclusive_scan(sum, warp_tot, total);
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = threadIdx.x * kPer + i;
        if (e >= E) break;
        if (blockIdx.x == 0) offsets[e] = excl + start[i];
        runs_to_cursors(e, E, kPlaceWarps, excl + start[i] + base[(int64_t)blockIdx.x * E + e], hist);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = total;
    for (int64_t p = total + (int64_t)blockIdx.x * kThreads + threadIdx.x; p < n; p += (int64_t)gridDim.x * kThreads) perm[p] = -1;
    __syncthreads();
    const int64_t a = f0 + (int64_t)warp_id() * seg;
    place_pairs(ids, a, min(f1, a + seg), E, hist + warp_id() * E, perm, inv);
}

static int64_t n_chunks_for(int64_t n) { return (n + kPermChunk - 1) / kPermChunk; }

// local[i] = ids[i] - e0 for ids in [e0, e0 + e_count), MOE_ID_NOT_LOCAL otherwise.
__global__ void shard_ids_kernel(const int32_t *__restrict__ ids, int64_t n, int e0, int e_count,
                                 int32_t *__restrict__ local)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int id = ids[i];
        local[i] = (id >= e0 && id - e0 < e_count) ? id - e0 : MOE_ID_NOT_LOCAL;
    }
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_shard_ids(const int32_t *ids, int64_t n, int e0, int e_count, int32_t *local_ids,
                                    moe_stream_t stream)
{
    MOE_REQUIRE(n >= 0, "n must be >= 0");
    MOE_REQUIRE(e0 >= 0 && e_count >= 1 && e_count <= 1024, "e0 >= 0 and 1 <= e_count <= 1024 (got %d, %d)", e0,
                e_count);
    if (n == 0) return MOE_OK;
    MOE_REQUIRE(ids && local_ids, "NULL pointer");
    const int64_t blocks = std::min<int64_t>((n + 255) / 256, (int64_t)sm_count() * 8);
    shard_ids_kernel<<<(unsigned)blocks, 256, 0, to_cuda(stream)>>>(ids, n, e0, e_count, local_ids);
    return check_launch("shard_ids");
}

namespace moe {

// The sort of up to kPermClusterMax pairs: no scratch in global memory.
static moe_status permute_few(const int32_t *ids, int n, int E, int32_t *offsets, int32_t *perm, int32_t *inv_perm,
                              int32_t *dev_status, cudaStream_t s)
{
    if (n <= kPermRankMax) {
        permute_rank_kernel<<<1 + (E + kRankThreads) / kRankThreads, kRankThreads, 0, s>>>(ids, n, E, offsets, perm, inv_perm,
                                                                                         dev_status);
        return check_launch("permute_rank");
    }
    if (n <= kPermSmallMax) {
        // as many runs of 32 or more pairs as 48,000 bytes of counters hold
        const int most = std::min(std::min(32, 12000 / E), (n + 31) / 32);
        const int seg = (n + most * 32 - 1) / (most * 32) * 32;
        const int warps = (n + seg - 1) / seg;
        permute_small_kernel<<<1, 1024, (size_t)warps * E * sizeof(int32_t), s>>>(ids, n, E, warps, seg, offsets, perm, inv_perm,
                                                                                dev_status);
        return check_launch("permute_small");
    }
    const int per_cta = (n + kClusterCtas * 32 - 1) / (kClusterCtas * 32) * 32;
    const int most = std::min(std::min(32, 11000 / E), per_cta / 32);  // runs, in 44,000 bytes of counters
    const int seg = (per_cta + most * 32 - 1) / (most * 32) * 32;
    const int warps = (per_cta + seg - 1) / seg;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kClusterCtas);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = (size_t)warps * E * sizeof(int32_t);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kClusterCtas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, permute_cluster_kernel, ids, n, E, per_cta, warps, seg, offsets, perm, inv_perm,
                                    dev_status));
    return check_launch("permute_cluster");
}

// The sort of any number of pairs, in three passes over counts and base, [chunks][E] each.
static moe_status permute_many(const int32_t *ids, int64_t n, int E, int32_t *counts, int32_t *base, int32_t *offsets,
                               int32_t *perm, int32_t *inv_perm, int32_t *dev_status, cudaStream_t s)
{
    const int64_t c = n_chunks_for(n);
    permute_count_kernel<<<(unsigned)c, 256, 0, s>>>(ids, n, E, counts, dev_status);
    moe_status st = check_launch("permute_count");
    if (st != MOE_OK) return st;
    permute_prefix_kernel<<<(E + 31) / 32, 1024, 0, s>>>(counts, (int)c, E, base);
    st = check_launch("permute_prefix");
    if (st != MOE_OK) return st;
    permute_place_kernel<<<(unsigned)c, kPlaceWarps * 32, 0, s>>>(ids, n, E, counts, base, offsets, perm, inv_perm);
    return check_launch("permute_place");
}

}  // namespace moe

extern "C" moe_status moe_permute_workspace_size(int T, int k, int E, size_t *bytes)
{
    MOE_REQUIRE(bytes, "bytes is NULL");
    MOE_REQUIRE(T >= 0 && k >= 1 && E >= 1 && E <= 1024, "T >= 0, k >= 1, 1 <= E <= 1024");
    int64_t n = (int64_t)T * k;
    if (n <= kPermClusterMax) {
        *bytes = 0;
        return MOE_OK;
    }
    int64_t c = n_chunks_for(n);
    *bytes = 2 * align256((size_t)c * E * sizeof(int32_t));
    return MOE_OK;
}

extern "C" moe_status moe_permute(const int32_t *ids, int T, int k, int E, int32_t *offsets, int32_t *perm,
                                  int32_t *inv_perm, void *ws, size_t ws_bytes, int32_t *dev_status,
                                  moe_stream_t stream)
{
    MOE_REQUIRE(T >= 0 && k >= 1 && k <= 16, "T >= 0 and 1 <= k <= 16 (got T=%d k=%d)", T, k);
    MOE_REQUIRE(E >= 1 && E <= 1024, "E must be in [1, 1024] (got %d)", E);
    MOE_REQUIRE(offsets, "offsets is NULL");
    int64_t n = (int64_t)T * k;
    MOE_REQUIRE(n <= INT32_MAX, "T*k too large");
    cudaStream_t s = to_cuda(stream);
    if (n == 0) {
        MOE_CUDA_TRY(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), s));
        return MOE_OK;
    }
    MOE_REQUIRE(ids && perm && inv_perm, "NULL pointer");
    if (n <= kPermClusterMax) return permute_few(ids, (int)n, E, offsets, perm, inv_perm, dev_status, s);
    size_t part = align256((size_t)n_chunks_for(n) * E * sizeof(int32_t));
    if (!ws || ws_bytes < 2 * part)
        return fail(MOE_ERR_WORKSPACE, "permute needs %zu bytes (%.2f MiB) of workspace, got %zu", 2 * part,
                    mib(2.0 * part), ws ? ws_bytes : (size_t)0);
    int32_t *counts = static_cast<int32_t *>(ws);
    int32_t *base = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + part);
    return permute_many(ids, n, E, counts, base, offsets, perm, inv_perm, dev_status, s);
}

// --------------------------------------------------------------------------
// moe_permute_noalloc: the same sorts, the scratch of the three passes in a fixed
// device array of this library instead of a caller workspace.
// --------------------------------------------------------------------------
#include <cuda.h>

#include <mutex>

namespace moe {

// Per-chunk counts and per-chunk bases, kNoAllocScratchInts int32 each.
constexpr int64_t kNoAllocScratchInts = 32768;  // chunks * E <= 32768 -> 2 x 128 KiB
static __device__ __align__(256) int32_t g_permute_scratch[2 * kNoAllocScratchInts];

// The current CUDA context through the driver's cuCtxGetCurrent, found by
// the runtime's entry-point query (no link against the driver library).
static CUcontext current_context()
{
    using Fn = CUresult (*)(CUcontext *);
    static Fn fn = []() -> Fn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<Fn>(p);
    }();
    CUcontext c = nullptr;
    if (!fn || fn(&c) != CUDA_SUCCESS) return nullptr;
    return c;
}

// Device address of g_permute_scratch on the current device, looked up with
// that device current and cached together with the context it belongs to: a
// new context on the device (after cudaDeviceReset, say, which unloads the
// library's device code) finds the cached context changed and looks the
// address up again.
static moe_status permute_scratch_address(int32_t **out)
{
    static std::mutex mu;
    static int32_t *addr[64] = {nullptr};
    static CUcontext ctx[64] = {nullptr};
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return fail(MOE_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    const CUcontext cur = current_context();  // NULL before the runtime has made one current
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev] || !cur || cur != ctx[dev]) {
        void *p = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&p, g_permute_scratch);  // makes the primary context current
        if (e != cudaSuccess)
            return fail(MOE_ERR_CUDA, "cudaGetSymbolAddress(g_permute_scratch) on device %d: %s", dev,
                        cudaGetErrorString(e));
        addr[dev] = static_cast<int32_t *>(p);
        ctx[dev] = current_context();
    }
    *out = addr[dev];
    return MOE_OK;
}

}  // namespace moe

extern "C" moe_status moe_permute_noalloc(const int32_t *ids, int T, int k, int E, int32_t *offsets, int32_t *perm,
                                          int32_t *inv_perm, int32_t *dev_status, moe_stream_t stream)
{
    MOE_REQUIRE(T >= 0 && k >= 1 && k <= 16, "T >= 0 and 1 <= k <= 16 (got T=%d k=%d)", T, k);
    MOE_REQUIRE(E >= 1 && E <= 1024, "E must be in [1, 1024] (got %d)", E);
    MOE_REQUIRE(offsets, "offsets is NULL");
    int64_t n = (int64_t)T * k;
    int64_t c = n_chunks_for(n);
    if (c * E > kNoAllocScratchInts)
        return fail(MOE_ERR_INVALID_ARG,
                    "moe_permute_noalloc holds at most %lld (chunks x experts) counters in its fixed scratch: "
                    "T*k=%lld pairs form %lld chunks of %d, times E=%d is %lld; use moe_permute with a workspace",
                    (long long)kNoAllocScratchInts, (long long)n, (long long)c, kPermChunk, E, (long long)(c * E));
    cudaStream_t s = to_cuda(stream);
    if (n == 0) {
        MOE_CUDA_TRY(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), s));
        return MOE_OK;
    }
    MOE_REQUIRE(ids && perm && inv_perm, "NULL pointer");
    if (n <= kPermClusterMax) return permute_few(ids, (int)n, E, offsets, perm, inv_perm, dev_status, s);
    int32_t *scratch = nullptr;
    moe_status st = permute_scratch_address(&scratch);
    if (st != MOE_OK) return st;
    // (every cell read is written earlier in the same call)
    return permute_many(ids, n, E, scratch, scratch + kNoAllocScratchInts, offsets, perm, inv_perm, dev_status, s);
}
