/*
 * moe_gb300.h -- C ABI of the GB300 (sm_103a) routed-expert MoE layer with
 * 2-bit / 3-bit block-quantised experts.
 *
 * The layer this library computes, per token x (bf16, hidden size H):
 *   logits = W_router x + b                      (fp32, E experts)
 *   ids, w = top-k of logits, ties to the lower id; w = the kept softmax
 *            probabilities renormalised to sum to 1
 *   out    = S(x) + sum_j w_j * FFN_{ids_j}(x)
 *   FFN_e(x) = Wd_e (silu(Wg_e x) * (Wu_e x)),  silu(g) = g / (1 + e^-g)
 *   S(x)   = the always-on shared expert, the same SwiGLU with bf16 weights.
 * The routed experts are stored in 32-weight blocks along each row's input
 * dimension with one fp16 scale s per block; a 2-bit code c stands for
 * (c - 1.5) s and a 3-bit code for (c - 3.5) s.
 *
 * Where this comes from.  "How Strata runs a 125-billion-parameter model on
 * a single 12 GB to 24 GB graphics card" (introduction and the Step 1
 * byte-census table) and "Strata Open-Source Runtime: Running a 125B-Parameter
 * Qwen3 Model on a 12GB GPU" (section "The Model Itself") describe a router
 * that keeps 10 of 512 experts per layer for every token, an always-on shared
 * expert, 48 layers, and 2-bit ("Q2_0") routed experts of which one token
 * reads 0.66 GB of 34.0 GB; "Strata serves a 125B MoE at 94 tokens/s from a
 * 12 GB card and 64 GB of RAM" (Table 1, "Where the weights live") repeats the
 * census.  The first page, Step 2, sums the finished expert vectors on the
 * GPU.  The pages give no bit layout, activation function, router
 * normalisation or shared-expert precision; the statements above are the
 * readings this library takes.
 *
 * Conventions for every call:
 *  - Status.  Every call returns a moe_status.  Argument errors are found on
 *    the host before anything is launched and leave all buffers untouched.
 *    A non-OK return also sets a thread-local message, moe_last_error(),
 *    that names the argument and, for sizes, the bytes or MiB involved.
 *  - Device-detected errors (bad ids, NaN logits, codes that do not fit,
 *    values outside the range of an fp16 tensor-core operand) are
 *    written into a caller-provided int32 status word in device memory
 *    (dev_status; the first error wins, 0 means OK; it may be NULL, in which
 *    case such errors are not reported).  Read it with moe_check_status().
 *    A kernel that detects such an error skips the offending element and
 *    still writes every output it owns.
 *  - Ownership.  The caller allocates every buffer and passes raw device
 *    pointers (unless a parameter says "host").  The library never allocates
 *    or frees memory and never synchronises a stream, except
 *    moe_check_status(), which synchronises the stream it is given.  Scratch
 *    memory comes from a caller-provided workspace whose size the matching
 *    *_workspace_size() call returns; a smaller workspace returns
 *    MOE_ERR_WORKSPACE with the bytes needed in the message.  One call is the
 *    exception: moe_permute_noalloc keeps its scratch in a fixed array inside
 *    the library (its own comment states the size, limit and sharing).
 *  - Asynchrony.  Work is enqueued on `stream` and returns at once.
 *  - Shapes.  H and I are multiples of 32; 1 <= E <= 1024;
 *    1 <= k <= min(E, 16); T >= 0 (T = 0 is a no-op that returns MOE_OK).
 *  - Types.  bf16 and fp16 values are passed as uint16_t bit patterns.
 *    Row-major everywhere.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The same handle type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st *moe_stream_t;

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1, /* a bad pointer, shape, code or scale           */
    MOE_ERR_UNSUPPORTED = 2, /* a valid request this library does not implement */
    MOE_ERR_WORKSPACE = 3,   /* workspace smaller than *_workspace_size()     */
    MOE_ERR_CUDA = 4,        /* a CUDA runtime call failed                    */
    MOE_ERR_TIMEOUT = 5,     /* a device-side wait ran out of its time limit  */
    MOE_ERR_NONFINITE = 6,   /* a NaN router logit                            */
    MOE_ERR_BOUNDS = 7,      /* an expert id outside [0, E)                   */
    MOE_ERR_RANGE = 8        /* a value outside the finite range of the fp16
                                or e4m3 operands the tensor cores take (see the
                                PREFILL and PREFILL_FP8 paths of
                                moe_expert_forward, moe_decode_forward) */
} moe_status;

typedef enum moe_dtype {
    MOE_F32 = 0,
    MOE_BF16 = 1,
    MOE_F16 = 2 /* the row, 4-bit and norm calls and the training calls after them only */
} moe_dtype;

typedef enum moe_path {
    MOE_PATH_AUTO = 0,        /* DECODE for T <= 8, PREFILL otherwise (never FP8) */
    MOE_PATH_DECODE = 1,      /* dequant-fused GEMVs on CUDA cores, fp32 maths  */
    MOE_PATH_PREFILL = 2,     /* grouped GEMM over the experts' token lists     */
    MOE_PATH_PREFILL_FP8 = 3  /* the same GEMMs on e4m3 operands: an opt-in
                                 approximation, see moe_expert_forward       */
} moe_path;

/* Message for the last non-OK status returned on this thread ("" if none). */
const char *moe_last_error(void);

/* Short name of a status code, e.g. "MOE_ERR_BOUNDS". */
const char *moe_status_name(moe_status s);

/*
 * Synchronise `stream`, read the int32 device status word and return it as a
 * moe_status (setting moe_last_error() when it is not MOE_OK).  If `reset` is
 * non-zero the word is set back to 0 afterwards.
 */
moe_status moe_check_status(int32_t *dev_status, int reset, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Packed block format                                                      */
/* ------------------------------------------------------------------------ */

/*
 * Bytes of one packed [rows][cols] matrix.  cols is a multiple of 32.
 *   code plane:  rows * row_bytes, row_bytes = cols/4 (2-bit) or 3*cols/8
 *                (3-bit);
 *   scale plane: rows * (cols/32) fp16 values = rows * cols/16 bytes.
 * Layout of one packed row of codes:
 *   bytes [0, cols/4):     weight i's two low code bits at bits
 *                          2*(i%4) .. 2*(i%4)+1 of byte i/4;
 *   bytes [cols/4, 3cols/8) (3-bit only): one little-endian 32-bit word per
 *                          32-weight block b, at byte cols/4 + 4b, holding
 *                          the high bit of weight 32b+i at bit
 *                          (i&7) | ((i&8)<<1) | ((i&16)>>1).
 * The scale plane is [rows][cols/32] fp16, block b of row r covering weights
 * 32b .. 32b+31 of that row.  Sizes follow the byte census of the pages (a
 * 2-bit expert with H=2048, I=768 is 1,474,560 bytes; see the Step 1 table of
 * "How Strata runs a 125-billion-parameter model ...").
 */
moe_status moe_packed_size(int bits, int64_t rows, int64_t cols, size_t *code_bytes,
                           size_t *scale_bytes);

/*
 * Pack n_mats matrices of [rows][cols] logical codes (one code per byte,
 * device, 16-byte aligned) and their fp16 scales [rows][cols/32] (device) into
 * the layout of moe_packed_size.  packed_scales may equal scales (in place:
 * no copy).  A code >= 2^bits or a non-finite scale sets *dev_status to
 * MOE_ERR_INVALID_ARG; that block is still written, with the codes' low bits
 * and the scale as given.
 */
moe_status moe_pack_experts(int bits, int64_t n_mats, int64_t rows, int64_t cols,
                            const uint8_t *codes, const uint16_t *scales, uint8_t *packed_codes,
                            uint16_t *packed_scales, int32_t *dev_status, moe_stream_t stream);

/*
 * Inverse of moe_pack_experts for the code plane: packed -> one code per byte
 * (codes [n_mats][rows][cols], device).  The pages store the routed experts
 * at 2 bits per weight and count their bytes ("How Strata runs a
 * 125-billion-parameter model ...", introduction and the Step 1 byte-census
 * table); this call recovers the logical codes from that storage.
 */
moe_status moe_unpack_experts(int bits, int64_t n_mats, int64_t rows, int64_t cols,
                              const uint8_t *packed_codes, uint8_t *codes, moe_stream_t stream);

/*
 * The routed experts of one layer, resident in device memory (structure of
 * arrays; expert e's data starts at e times the per-expert size):
 *   gu_codes  [E][2I rows][row_bytes(H)]   rows 0..I-1 gate, I..2I-1 up
 *   gu_scales [E][2I][H/32] fp16
 *   d_codes   [E][H rows][row_bytes(I)]
 *   d_scales  [E][H][I/32] fp16
 * Every pointer must be 16-byte aligned.
 */
typedef struct moe_expert_arena {
    int32_t bits; /* 2 or 3 */
    int32_t H;
    int32_t I;
    int32_t E;
    const uint8_t *gu_codes;
    const uint16_t *gu_scales;
    const uint8_t *d_codes;
    const uint16_t *d_scales;
} moe_expert_arena;

/* ------------------------------------------------------------------------ */
/* Router                                                                   */
/* ------------------------------------------------------------------------ */

/*
 * logits[t][e] = bias[e] + sum_i W[e][i] * x[t][i] in fp32; then the top-k
 * selection and weights of moe_topk_from_logits.
 *   x_bf16      [T][H] bf16
 *   w_router    [E][H] fp32 (16-byte aligned)
 *   bias        [E] fp32, or NULL for none
 *   logits_out  [T][E] fp32, or NULL (then the workspace holds them)
 *   topk_ids    [T][k] int32,  topk_w [T][k] fp32
 * T <= 8 runs an fp32 GEMV.  Larger T with H a multiple of 64 runs on the
 * tensor cores: W is split into three bf16 pieces (W1 + W2 + W3 carries
 * W's 24 significant bits), every product with the bf16 x is exact and
 * the sums are fp32; other shapes take an fp32 FFMA GEMM.
 * Workspace: moe_router_workspace_size (0 bytes when logits_out is given
 * and T <= 8; the split weights, E * 3H * 2 bytes, for the tensor cores).
 * A wait of the tensor-core kernel that runs out (about 2 s) sets
 * *dev_status = MOE_ERR_TIMEOUT.
 * The pages: the router keeps 10 of 512 experts per token per layer
 * ("Strata Open-Source Runtime ...", section "The Model Itself").
 */
moe_status moe_router_workspace_size(int T, int H, int E, int logits_given, size_t *bytes);
moe_status moe_router_topk(const uint16_t *x_bf16, int T, int H, const float *w_router,
                           const float *bias, int E, int k, float *logits_out, int32_t *topk_ids,
                           float *topk_w, void *ws, size_t ws_bytes, int32_t *dev_status,
                           moe_stream_t stream);

/*
 * Top-k of fp32 logits [T][E]:
 *   ids[t][j]: experts in the order (logit descending, id ascending), compared
 *              as IEEE floats (-0 == +0, so the lower id wins);
 *   w[t][j]  = softmax(logits[t])[ids[t][j]] / sum over the kept ones, which
 *              equals the softmax of the k kept logits; when the largest logit
 *              is infinite the weights are uniform over the kept experts that
 *              hold it (the softmax's limit).
 * A NaN logit sets *dev_status = MOE_ERR_NONFINITE; that token's ids are set
 * to 0..k-1 and its weights to 1/k.
 * The pages: the router keeps the 10 best of 512 experts for each token and
 * layer ("Strata Open-Source Runtime ...", section "The Model Itself"), and
 * ranks 0..9 carry decreasing router weights ("How Strata runs a
 * 125-billion-parameter model ...", Step 2, "Verify-window route tail
 * skip").  This call is the selection step alone, so that a test can feed
 * both this library and a reference the same fp32 logits.
 */
moe_status moe_topk_from_logits(const float *logits, int T, int E, int k, int32_t *ids, float *w,
                                int32_t *dev_status, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Token -> expert permutation                                              */
/* ------------------------------------------------------------------------ */

/*
 * Stable counting sort of the T*k (token, slot) pairs by expert id:
 *   offsets [E+1]: offsets[e] = pairs with id < e, offsets[E] = T*k;
 *   perm    [T*k]: perm[p] = t*k + j of the p-th pair in (expert, t*k+j) order;
 *   inv_perm[T*k]: inv_perm[perm[p]] = p.
 * Bit-exact and deterministic.  An id of MOE_ID_NOT_LOCAL (-1) marks a pair
 * that another expert shard computes (see moe_shard_ids): it is left out
 * without an error.  Any other id outside [0, E) sets *dev_status to
 * MOE_ERR_BOUNDS and is left out the same way.  A left-out pair is not
 * counted in offsets, its inv_perm entry is -1 and perm entries past
 * offsets[E] are -1; moe_expert_forward skips such pairs (they add nothing
 * to their token's output).
 * The pages group the tokens of a verify window that share an expert
 * ("Strata serves a 125B MoE ...", section "Six billion active parameters
 * per token").
 */
moe_status moe_permute_workspace_size(int T, int k, int E, size_t *bytes);

/* The id of a (token, slot) pair whose expert lives on another shard. */
#define MOE_ID_NOT_LOCAL (-1)

/*
 * Expert parallelism: the ids of the shard that holds experts
 * [e0, e0 + e_count) of a layer.  local_ids[i] = ids[i] - e0 for ids in that
 * range, MOE_ID_NOT_LOCAL otherwise (n ids, device).  A shard then runs
 * moe_permute(local_ids, ..., E = e_count) and moe_expert_forward on an arena
 * of its e_count experts with the full routing weights: its output is the sum
 * of its own experts' terms, and the sum of all shards' outputs (plus the
 * shared expert once) is the layer.  The pages run the layer on one GPU;
 * sharding the 512 experts of a layer over several GPUs is this library's
 * extension for GPUs that serve the whole model from memory.
 */
moe_status moe_shard_ids(const int32_t *ids, int64_t n, int e0, int e_count, int32_t *local_ids,
                         moe_stream_t stream);
moe_status moe_permute(const int32_t *ids, int T, int k, int E, int32_t *offsets, int32_t *perm,
                       int32_t *inv_perm, void *ws, size_t ws_bytes, int32_t *dev_status,
                       moe_stream_t stream);

/*
 * moe_permute_noalloc -- the same stable counting sort as moe_permute, for
 * callers that cannot allocate device memory.  (This entry point has no
 * counterpart in the pages: it is a convenience of this library.)  Some
 * callers cannot call cudaMalloc or hand the library a workspace: a plugin
 * whose host framework owns every device allocation and offers no scratch
 * buffer, or a serving loop that must not allocate after start-up because an
 * allocation may synchronise the device or fail under memory pressure.  This
 * call allocates nothing and takes no workspace: its scratch is a fixed array
 * of 2 x 32,768 int32 (256 KiB) inside the library, which every GPU that
 * loads the library holds until the process exits.  (moe_permute itself needs
 * a workspace above 32,768 pairs only; up to there the two are one.)
 *   - Limit: ceil(T*k / 2048) * E <= 32,768 (e.g. T*k <= 65,536 pairs for
 *     E = 1024, <= 131,072 for E = 512); larger requests return
 *     MOE_ERR_INVALID_ARG with the sizes in the message.
 *   - Outputs, errors and ordering are those of moe_permute.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it together with the device's current
 *     context; a call under a new context (after cudaDeviceReset, say) looks
 *     it up again.  Make the first call on a device, and the first after a
 *     reset, before any stream capture.
 *   - Every call of more than 32,768 pairs on a device shares the one array,
 *     and each such call overwrites the cells it reads (nothing needs clearing
 *     between calls); those whose kernels overlap on the GPU (other streams,
 *     other host threads) race on it, so serialise them.
 */
moe_status moe_permute_noalloc(const int32_t *ids, int T, int k, int E, int32_t *offsets,
                               int32_t *perm, int32_t *inv_perm, int32_t *dev_status,
                               moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Routed experts                                                           */
/* ------------------------------------------------------------------------ */

/*
 * out[t] = (accumulate ? out[t] : 0) + sum_{j<k} w[t][j] * FFN_{ids[t][j]}(x[t]),
 * the slot sum taken in slot order.  ids/w/offsets/perm/inv_perm come from
 * moe_router_topk (or the caller) and moe_permute.
 *   out: [T][H], fp32 (MOE_F32) or bf16 (MOE_BF16, round-to-nearest-even of
 *        the fp32 result).
 * DECODE: fp32 dequantisation and accumulation; a token's result does not
 *   depend on which other tokens share the call (bit-identical alone or in a
 *   group).
 * PREFILL: grouped GEMM over the experts' token lists.  With H and I
 *   multiples of 64 (2-bit) or 128 (3-bit) it runs on the tensor cores with
 *   fp16 operands: x converts to fp16 (exact for 2^-14 <= |x| <= 65504,
 *   fewer bits below, none below 2^-25), the weights (c - mid) s round once to
 *   fp16, h = silu(g) u rounds to fp16 between the two projections and each
 *   pair's y = Wd_e h is kept as fp16 until the combine (fp32 accumulation
 *   throughout; relative L2 error about 4e-4 on N(0,1) inputs).  The caller
 *   keeps every one of these inside fp16's finite range: |x|, |h| and |y|
 *   below 65504 and every block scale with |s| * max|c - mid| below 65520
 *   (max|c - mid| = 1.5 for 2 bits, 3.5 for 3 bits).  RMS-normalised inputs
 *   (|x| of order 1) and weight scales of order 0.02 stay far inside.  A value
 *   outside it sets *dev_status = MOE_ERR_RANGE and the affected outputs are
 *   not finite.  Other shapes take an fp32 FFMA form with no such limit.
 * PREFILL_FP8: the PREFILL GEMMs with e4m3 operands (kind::f8f6f4 tensor-core
 *   instructions), an opt-in approximation that AUTO never picks.  The pages
 *   run no 8-bit arithmetic; this scheme is the library's own.  2- and
 *   3-bit arenas with H and I multiples of 128 only; anything else returns
 *   MOE_ERR_UNSUPPORTED.  Every operand is an e4m3 value after a power-of-two
 *   scaling 2^e with e = 7 - floor(log2 m) (clamped to [-64, 64]), m the
 *   largest magnitude it covers: one e per weight row (m = max|c - mid|
 *   times the row's largest |s|), per pair for x, and per pair for h, which
 *   is first rounded to fp16 as in PREFILL; each weight is
 *   e4m3((c - mid) s 2^e), rounded once.  Products accumulate in fp32 and the scalings are undone on
 *   the accumulators; y is kept as fp16 until the combine.  The rounding of
 *   three operands to 3 mantissa bits costs a relative L2 error of about
 *   6e-2 on one expert's output and about 3e-2 on a layer whose bf16 shared
 *   expert is added (H=2048, I=768, N(0,1) inputs), not the 1e-3 of PREFILL.
 *   MOE_ERR_RANGE: a non-finite x or block scale, an |x| above 464 * 2^64, or
 *   an h or y outside fp16's range (as in PREFILL).
 * Workspace: moe_expert_forward_workspace_size for the same arguments.
 * The pages: each token's routed experts run on the GPU and their finished
 * output vectors are summed there, weighted by the router ("How Strata runs
 * a 125-billion-parameter model ...", Step 2, "Dynamic PCIe and CPU
 * co-execution"); long prompts are read in chunks of tokens ("Strata
 * Open-Source Runtime ...", section "Prefill and Long Context"), which the
 * PREFILL path serves as one grouped GEMM per chunk.
 */
moe_status moe_expert_forward_workspace_size(const moe_expert_arena *arena, int T, int k,
                                             moe_path path, size_t *bytes);
moe_status moe_expert_forward(const moe_expert_arena *arena, const uint16_t *x_bf16, int T,
                              const int32_t *ids, const float *w, int k, const int32_t *offsets,
                              const int32_t *perm, const int32_t *inv_perm, void *out,
                              moe_dtype out_dtype, int accumulate, moe_path path, void *ws,
                              size_t ws_bytes, int32_t *dev_status, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Shared expert                                                            */
/* ------------------------------------------------------------------------ */

/*
 * out[t] = (accumulate ? out[t] : 0) + Wd (silu(Wg x[t]) * (Wu x[t])),
 * bf16 weights wg [I][H], wu [I][H], wd [H][I] (I here is the shared
 * expert's width), fp32 accumulation.  T <= 8 runs fp32 GEMVs; larger T
 * with H and I multiples of 64 runs on the tensor cores with exact bf16
 * products, h carried as two bf16 halves (h_hi + h_lo, 16 significant
 * bits) into the down projection; other shapes take an fp32 FFMA GEMM.
 * A wait of the tensor-core kernels that runs out (about 2 s) sets
 * *dev_status = MOE_ERR_TIMEOUT (dev_status may be NULL: then it is not
 * reported).  The pages: one always-on shared expert per layer
 * ("Strata Open-Source Runtime ...", section "The Model Itself").
 * Workspace: moe_shared_expert_workspace_size.
 */
moe_status moe_shared_expert_workspace_size(int H, int I, int T, size_t *bytes);
moe_status moe_shared_expert(const uint16_t *wg, const uint16_t *wu, const uint16_t *wd, int H,
                             int I, const uint16_t *x_bf16, int T, void *out, moe_dtype out_dtype,
                             int accumulate, void *ws, size_t ws_bytes, int32_t *dev_status,
                             moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Fused decode over a stack of layers                                      */
/* ------------------------------------------------------------------------ */

/* The weights of one layer for moe_decode_forward (device pointers). */
typedef struct moe_layer_weights {
    moe_expert_arena experts;      /* routed experts (same shape in every layer) */
    const float *w_router;         /* [E][H] fp32 */
    const float *bias;             /* [E] fp32, or NULL */
    const uint16_t *shared_wg;     /* [shared_I][H] bf16 (ignored if shared_I == 0) */
    const uint16_t *shared_wu;     /* [shared_I][H] bf16 */
    const uint16_t *shared_wd;     /* [H][shared_I] bf16 */
    int32_t shared_I;              /* shared expert width, 0 for none */
} moe_layer_weights;

/*
 * Decode up to 4 tokens through n_layers (<= 64) MoE layers in one
 * persistent cooperative kernel, updating the fp32 residual stream in place:
 *   for each layer l:  u = bf16(x[t] / sqrt(mean(x[t]^2) + rms_eps))
 *                      x[t] += S_l(u) + sum_j w_tj FFN_{l,ids_tj}(u)
 * (rms_eps < 0: u = bf16(x[t]), no normalisation; see moe_rms_norm_bf16)
 * with the routing of moe_router_topk (fp32 logits, ties to the lower id,
 * renormalised softmax weights), exact dequantisation (centred codes c - mid
 * in fp16 on the tensor cores, the block scale applied in fp32) and fp32
 * accumulation.
 *   layers   host array of n_layers descriptors (copied into the launch)
 *   x        [T][H] fp32, device, 16-byte aligned, in/out
 *   ids_out, w_out  [n_layers][T][k] device outputs of the routing, or both NULL
 * A token's result does not depend on the other tokens of the call.  The
 * tensor-core operands are fp16: u must stay below 65520 in magnitude (always
 * so when normalised, |u| <= sqrt(H)) and so must h = silu(g) u; a value
 * outside sets *dev_status = MOE_ERR_RANGE.  Shapes:
 * H a multiple of 256 with at most 16 output rows per SM (H <= 2432 on 152
 * SMs), I a multiple of 128 up to 4096, shared_I a multiple of 64 up to 4096,
 * E <= 1024, k <= 16; MOE_ERR_UNSUPPORTED when the buffers do not fit in
 * shared memory.  The workspace (moe_decode_workspace_size) holds counters and
 * tagged exchange words that the call zeroes on the stream before its launch.
 * Every wait in the kernel gives up after about 2 s and reports
 * MOE_ERR_TIMEOUT through dev_status.  The pages: 48 layers of a
 * router, ten of 512 experts and a shared expert, verify windows of up to
 * four tokens ("Strata serves a 125B MoE ...", section "Six billion active
 * parameters per token").
 */
moe_status moe_decode_workspace_size(int T, int H, int I, int E, int k, int shared_I, size_t *bytes);
moe_status moe_decode_forward(const moe_layer_weights *layers, int n_layers, float *x, int T, int k,
                              float rms_eps, int32_t *ids_out, float *w_out, void *ws, size_t ws_bytes,
                              int32_t *dev_status, moe_stream_t stream);

/*
 * Options of moe_decode_forward_ex (all zero: the exact layer of
 * moe_decode_forward).
 *
 * route_tail_skip (an approximation, off at 0): from this rank on (0-based
 *   slot in the token's top-k order), a (token, slot) pair is left out of the
 *   layer -- its expert's weights are neither fetched nor multiplied -- when
 *   no token of the call keeps that expert at a lower rank and the expert is
 *   not marked hot.  The other pairs keep their weights (no renormalisation),
 *   so a token's output loses the left-out terms w_j FFN_j(u).  The pages
 *   skip, in a verify window of up to four tokens, the experts every token
 *   ranks 7, 8 or 9 of its top-10 (rank threshold 7) unless the expert is in
 *   the fast memory tier, trading a small shift of the output distribution
 *   for fewer expert reads ("How Strata runs a 125-billion-parameter model
 *   ...", Step 2, "Verify-window route tail skip").  Must be in [0, k].
 *   ids_out / w_out still report the router's full selection.
 * hot_experts (device, [n_layers][(E + 31) / 32] uint32 bit masks, bit e of
 *   layer l set for a hot expert, or NULL): the copies of a marked expert's
 *   weights carry an L2 evict-last hint and every other weight copy an
 *   evict-first hint, so that the marked experts stay in the 129 MB L2 from
 *   one decode step to the next -- the on-chip counterpart of the pages'
 *   adaptive expert cache ("How Strata runs ...", Step 1, "Tier 1: GPU VRAM
 *   ... adaptive expert cache"; "Strata serves a 125B MoE ...", "Where the
 *   weights live").  The results are the same bits with or without masks.
 *   The caller chooses the set (for instance from the routing the previous
 *   steps reported through ids_out) and may change it between calls.
 */
typedef struct moe_decode_options {
    int32_t route_tail_skip;
    const uint32_t *hot_experts;
} moe_decode_options;

/*
 * moe_decode_forward with options (opts may be NULL: moe_decode_forward).
 * Every other argument, the shapes, workspace and errors are those of
 * moe_decode_forward.
 */
moe_status moe_decode_forward_ex(const moe_layer_weights *layers, int n_layers, float *x, int T, int k,
                                 float rms_eps, const moe_decode_options *opts, int32_t *ids_out, float *w_out,
                                 void *ws, size_t ws_bytes, int32_t *dev_status, moe_stream_t stream);

/*
 * Self-test of the grid barrier's time limit used by moe_decode_forward: one
 * cooperative launch (one CTA per SM) runs a single barrier whose target is
 * `extra_arrivals` above the number of CTAs.  With extra_arrivals = 0 it
 * completes; otherwise every CTA gives up after timeout_ms, writes
 * MOE_ERR_TIMEOUT to *dev_status and returns, leaving the context usable.
 * ws: 8 bytes (int at ws+4 counts the CTAs that passed the barrier).
 */
moe_status moe_selftest_barrier(unsigned extra_arrivals, int timeout_ms, void *ws, size_t ws_bytes,
                                int32_t *dev_status, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Residual stream helper                                                   */
/* ------------------------------------------------------------------------ */

/* out_bf16[i] = round-to-nearest-even bf16 of in_f32[i], n elements. */
moe_status moe_f32_to_bf16(const float *in_f32, uint16_t *out_bf16, int64_t n, moe_stream_t stream);

/*
 * The input of a stacked layer: out[t] = bf16(x[t] / sqrt(mean(x[t]^2) + eps))
 * for x [T][H] fp32 (a root-mean-square normalisation without a gain).  The
 * pages' layers read a residual stream; a stack of synthetic layers without
 * this normalisation diverges, so the stacked workloads normalise in front
 * of every layer.
 */
moe_status moe_rms_norm_bf16(const float *x, uint16_t *out, int T, int H, float eps, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Rows to their experts and back                                           */
/* ------------------------------------------------------------------------ */

/*
 * The movement of activation rows around a layer's experts, for experts that
 * are not this library's 2-/3-bit ones (moe_expert_forward does it inside),
 * and its gradients.  offsets and inv_perm are moe_permute's: pair (t, j) is
 * row inv_perm[t*k + j] of the T*k sorted rows, or none (-1, a left-out pair).
 * An inv_perm entry outside [0, T*k) counts as left out.  Rows are fp32, bf16
 * or fp16; sums and dot products are fp32 and rounded once; nothing is added
 * with atomics, so the same call gives the same bits.  1 <= k <= 16, any
 * H >= 1 (rows of 16-byte multiples move fastest).  T = 0 is a no-op.
 *
 * moe_dispatch: out[inv_perm[t*k + j]] = x[t]; rows at and past offsets[E] are
 * set to zero.  Row t of x starts at x + t * x_stride elements (x_stride >= H,
 * or 0: the same row for every token).
 * moe_dispatch_backward: dx[t] = sum_j drows[inv_perm[t*k + j]], in slot order.
 */
moe_status moe_dispatch(const void *x, moe_dtype dtype, int64_t x_stride, int T, int H, int k, int E,
                        const int32_t *offsets, const int32_t *inv_perm, void *out, moe_stream_t stream);
moe_status moe_dispatch_backward(const void *drows, moe_dtype dtype, int T, int H, int k,
                                 const int32_t *inv_perm, void *dx, moe_stream_t stream);

/*
 * out[t] = (accumulate ? out[t] : 0) + sum_j w[t][j] * y[inv_perm[t*k + j]],
 * in slot order; a token all of whose pairs are left out gets 0 (or keeps its
 * value).  out_dtype: the rows' type or MOE_F32.
 * moe_combine_backward: dy[inv_perm[t*k + j]] = w[t][j] * dout[t] and
 * dw[t][j] = <dout[t], y[inv_perm[t*k + j]]> (fp32; 0 for a left-out pair);
 * rows of dy at and past offsets[E] are set to zero.  The gradient of an
 * accumulated out is dout itself.
 */
moe_status moe_combine(const void *y, moe_dtype dtype, int T, int H, int k, const float *w,
                       const int32_t *inv_perm, void *out, moe_dtype out_dtype, int accumulate,
                       moe_stream_t stream);
moe_status moe_combine_backward(const void *dout, const void *y, moe_dtype dtype, int T, int H, int k, int E,
                                const int32_t *offsets, const float *w, const int32_t *inv_perm, void *dy,
                                float *dw, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 4-bit floating point matrices (MXFP4)                                    */
/* ------------------------------------------------------------------------ */

/*
 * A matrix [rows][cols], cols a multiple of 32, in the OCP microscaling format
 * MXFP4 (Open Compute Project, "Microscaling Formats (MX) Specification" 1.0):
 *   codes:  [rows][cols/2] bytes, value i of a row in the low (i even) or high
 *           (i odd) half of byte i/2: an e2m1 number, sign at bit 3, magnitude
 *           0, 0.5, 1, 1.5, 2, 3, 4 or 6 for codes 0..7;
 *   scales: [rows][32 * ceil(cols/1024)] bytes, byte b of a row the exponent
 *           (e8m0, 2^(byte - 127), 255 = NaN) of values 32b .. 32b+31; bytes
 *           past cols/32 are 0.
 * codes are 16-byte and scales 32-byte aligned.
 *
 * moe_mx4_quantise: per block of 32, with m its largest magnitude,
 * e = max(floor(log2 m) - 2, -127) and code = e2m1(x 2^-e), to nearest, ties
 * to even, magnitudes above 6 to 6 (the specification's conversion; m = 0
 * gives byte 0).  A block that holds an infinity or a NaN gets the scale NaN
 * and zero codes, and sets *dev_status = MOE_ERR_NONFINITE.  Row r starts at
 * x + r * x_stride elements (x_stride >= cols, or 0).
 * moe_mx4_dequantise: out = code * 2^(byte - 127), exact in fp32 and bf16, one
 * rounding to fp16; NaN for a block of scale NaN.
 */
moe_status moe_mx4_size(int64_t rows, int64_t cols, size_t *code_bytes, size_t *scale_bytes);
moe_status moe_mx4_quantise(const void *x, moe_dtype dtype, int64_t x_stride, int64_t rows, int64_t cols,
                            uint8_t *codes, uint8_t *scales, int32_t *dev_status, moe_stream_t stream);
moe_status moe_mx4_dequantise(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                              void *out, moe_dtype dtype, moe_stream_t stream);

typedef enum moe_mx4_epilogue {
    MOE_MX4_PLAIN = 0, /* out = x W^T, W [E][N][K]                               */
    MOE_MX4_SWIGLU = 1 /* out = silu(x Wg^T) * (x Wu^T), W [E][2N][K]: rows 0..N-1
                          of an expert gate, N..2N-1 up                         */
} moe_mx4_epilogue;

/*
 * Products of quantised rows with their expert's quantised weights, on the
 * tensor cores (products exact, fp32 sums, one rounding to out_dtype):
 *   out[p][n] = sum_k x[p][k] W_e[n][k],  e the group with offsets[e] <= p <
 *   offsets[e+1]
 * x is a [rows][K] and W one [E * N (or 2N)][K] matrix of the format above;
 * offsets [E+1] as moe_permute gives them (or a slice of them: offsets[0] need
 * not be 0), or NULL when E = 1 (all rows).  Rows of no group, before offsets[0]
 * or at and past offsets[E], are set to zero.  out [rows][N], any N >= 1.
 * Offsets that decrease or leave [0, rows] set *dev_status = MOE_ERR_BOUNDS and
 * are clipped, and a group then begins no earlier than the one before it ends;
 * a wait that runs out (about 2 s) sets MOE_ERR_TIMEOUT.  E <= 1024, and at most
 * 2^30 tiles (128 columns, or 64 with SwiGLU, times a tile's rows).
 */
moe_status moe_mx4_matmul(const uint8_t *w_codes, const uint8_t *w_scales, int E, int N, int K,
                          const uint8_t *x_codes, const uint8_t *x_scales, int rows, const int32_t *offsets,
                          void *out, moe_dtype out_dtype, moe_mx4_epilogue epilogue, int32_t *dev_status,
                          moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Norms around a block                                                     */
/* ------------------------------------------------------------------------ */

typedef enum moe_gate {
    MOE_GATE_NONE = 0,
    MOE_GATE_TOKEN = 1,  /* gate [T]: one factor per token    */
    MOE_GATE_CHANNEL = 2 /* gate [H]: one factor per channel  */
} moe_gate;

/*
 * The end of one block and the start of the next, in one pass: with b the
 * block's output and x the residual stream,
 *   v = w_post * b / sqrt(mean(b^2) + eps)
 *   y = x + alpha * gate * v
 *   u = w_pre * y / sqrt(mean(y^2) + eps)
 * The residual stream (x, y) is fp32 or of the type of b and u (fp32, bf16,
 * fp16); w_post, w_pre (NULL: ones) and gate are fp32.  All arithmetic is
 * fp32; u comes from y before its rounding.  y may be x and u may be b (packed
 * rows).  Rows of x and b start every x_stride and b_stride elements (>= H, or
 * 0: the same row for every token).  1 <= H <= 16384; T = 0 is a no-op.
 */
moe_status moe_block_norm(const void *x, moe_dtype res_dtype, int64_t x_stride, const void *b,
                          moe_dtype dtype, int64_t b_stride, int T, int H, const float *w_post,
                          const float *w_pre, const float *gate, moe_gate gate_kind, float alpha, float eps,
                          void *y, void *u, moe_stream_t stream);

/*
 * Gradients of moe_block_norm for dy and du, the gradients of y and u (NULL:
 * zero): dx [T][H] (residual type), db [T][H] (the block's type), and the fp32
 * sums dw_post [H], dw_pre [H] and dgate ([T] or [H] like gate), each of which
 * may be NULL.  dx may be dy and db may be du.  The statistics are recomputed
 * from x and b.  With T = 0 the sums over tokens are set to zero.  Sums over
 * tokens are taken in a fixed order.
 */
moe_status moe_block_norm_backward_workspace_size(int T, int H, moe_gate gate_kind, size_t *bytes);
moe_status moe_block_norm_backward(const void *x, moe_dtype res_dtype, int64_t x_stride, const void *b,
                                   moe_dtype dtype, int64_t b_stride, int T, int H, const float *w_post,
                                   const float *w_pre, const float *gate, moe_gate gate_kind, float alpha,
                                   float eps, const void *dy, const void *du, void *dx, void *db,
                                   float *dw_post, float *dw_pre, float *dgate, void *ws, size_t ws_bytes,
                                   moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* The router's losses                                                      */
/* ------------------------------------------------------------------------ */

/*
 * What a router is trained on beside the model's own loss.  With p the softmax
 * of a token's E logits, n the tokens that count, count[e] their pairs of
 * expert e, f_e = count[e] / (n k) and P_e the mean of p_e over them:
 *   loss[0] = E sum_e f_e P_e                   (1 for an even load)
 *   loss[1] = mean over the tokens of lse^2,    lse = log sum_e exp(logit_e)
 *   counts  [E + 1] int32: count[0 .. E-1], then n
 *   mean_prob [E]: P,   lse [T]: for the gradient
 * A token counts unless keep (bytes [T], NULL: all) is 0 or all its logits are
 * -inf; a single logit of -inf is an expert that cannot be chosen.  A logit of
 * NaN or +inf sets *dev_status = MOE_ERR_NONFINITE and its token does not
 * count.  lse of a token that does not count is -inf.  An id of
 * MOE_ID_NOT_LOCAL counts for no expert, any other outside [0, E) sets
 * MOE_ERR_BOUNDS too.  No token that counts (or T = 0): losses, counts and
 * means are 0.  logits and dlogits are fp32, bf16 or fp16 [T][E], everything
 * is summed in fp32 in a fixed order.  1 <= E <= 1024, 1 <= k <= min(E, 16).
 *
 * moe_router_loss_backward: the logits' gradient, from dloss [2] (device; the
 * gradients of the two losses; NULL: none) and from the gradient dw [T][k] of
 * the routing weights w [T][k], the softmax over the kept logits as
 * moe_router_topk gives it (both NULL: none):
 *   dlogits[t][e] = p_te (g_e - sum_e' p_te' g_e' + 2 dloss[1] lse_t / n)
 *                   + sum over j with ids[t][j] = e of
 *                     w_tj (dw_tj - sum_i w_ti dw_ti)
 * with g_e = dloss[0] E count[e] / (n^2 k); the first part is 0 for a token
 * that does not count, the second goes by w and dw alone.  counts and lse are
 * moe_router_loss's.  dlogits may be logits.
 */
moe_status moe_router_loss_workspace_size(int T, int E, size_t *bytes);
moe_status moe_router_loss(const void *logits, moe_dtype dtype, int T, int E, const int32_t *ids, int k,
                           const uint8_t *keep, float *loss, int32_t *counts, float *mean_prob, float *lse,
                           void *ws, size_t ws_bytes, int32_t *dev_status, moe_stream_t stream);
moe_status moe_router_loss_backward(const void *logits, moe_dtype dtype, int T, int E, const int32_t *ids,
                                    int k, const int32_t *counts, const float *lse, const float *dloss,
                                    const float *w, const float *dw, void *dlogits, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Cross entropy over a vocabulary                                          */
/* ------------------------------------------------------------------------ */

/*
 * The loss at the end of a model, from the hidden states h [T][H] and the
 * head's weights w [V][H] (both bf16 or both fp16), on the tensor cores,
 * without the T x V logits ever being held:
 *   z_t = w h_t,  lse[t] = log sum_v exp(z_tv),  loss[t] = lse[t] - z_t,labels[t]
 * A negative label leaves its token out (loss 0; lse is given all the same);
 * one of V or more does too and sets *dev_status = MOE_ERR_BOUNDS.  Products
 * are exact, sums fp32.  A logit of NaN or +inf (values of h or w that are not
 * finite, sums beyond fp32) makes its token's lse and loss NaN; one of -inf is
 * a probability of zero (as a label's, its loss is infinite).  No status tells
 * of either.  H a multiple of 8, V >= 1; h and w 16-byte aligned.  T = 0 is a
 * no-op.
 *
 * moe_cross_entropy_backward: with dloss [T] and dlse [T] (NULL: zero) the
 * gradients of loss and lse, and d_tv = exp(z_tv - lse[t]) (dloss[t] + dlse[t])
 * - [v = labels[t]] dloss[t] (a token that is left out has dloss = 0),
 *   dh[t] = sum_v d_tv w_v      [T][H], of h's type
 *   dw[v] (+)= sum_t d_tv h_t   [V][H], of h's type or MOE_F32
 * either of which may be NULL.  accumulate adds to dw as it is (MOE_F32 only;
 * one addition per value and call).  The products are computed again, in
 * pieces of the vocabulary: d enters the two gradients rounded to h's type,
 * relative to the largest finite |dloss| or |dlse| of the call, and is held for
 * one piece at a time (at most 256 MiB of the workspace, at least 256 columns
 * of the vocabulary); a product over the whole of T or V is summed in fp32 and
 * rounded once.  A dloss or dlse that is not finite makes its token's dh, and
 * dw, so too, and no other token's dh; so does a lse that is not finite, of a
 * token whose weights are not zero.  A value w[v][j] (or h[t][j]) that is not
 * finite leaves no finite value in column j of dh (or dw): a d of zero times it
 * is NaN.  dh and dw must not overlap h and w.  With T = 0 dw is set to zero
 * unless it is accumulated.
 * A wait that runs out (about 2 s) sets MOE_ERR_TIMEOUT.
 *
 * Both sizes grow with T: a workspace of the largest batch's size is enough
 * for every smaller one of the same H and V.
 */
moe_status moe_cross_entropy_workspace_size(int T, int H, int V, size_t *bytes);
moe_status moe_cross_entropy(const void *h, moe_dtype dtype, int T, int H, const void *w, int V,
                             const int32_t *labels, float *loss, float *lse, void *ws, size_t ws_bytes,
                             int32_t *dev_status, moe_stream_t stream);
moe_status moe_cross_entropy_backward_workspace_size(int T, int H, int V, size_t *bytes);
moe_status moe_cross_entropy_backward(const void *h, moe_dtype dtype, int T, int H, const void *w, int V,
                                      const int32_t *labels, const float *lse, const float *dloss,
                                      const float *dlse, void *dh, void *dw, moe_dtype dw_dtype, int accumulate,
                                      void *ws, size_t ws_bytes, int32_t *dev_status, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* AdamW                                                                    */
/* ------------------------------------------------------------------------ */

/* One tensor of n values (device pointers, aligned to their types; n = 0: nothing is done). */
typedef struct moe_adamw_tensor {
    void *param;        /* in/out, of param_dtype */
    const void *grad;   /* of grad_dtype */
    float *master;      /* in/out: the value in fp32, of which param is the rounding; NULL: param is the value */
    void *m, *v;        /* in/out: fp32 [n], or codes (uint8 [n]) when scales are given */
    float *scales;      /* in/out: [ceil(n / 256)][2], of m and of v's root; NULL: m and v are fp32 */
    int64_t n;
    int32_t param_dtype, grad_dtype; /* moe_dtype: any of the three */
    float lr_factor;    /* the tensor's learning rate is lr * lr_factor */
    float weight_decay;
} moe_adamw_tensor;

typedef struct moe_adamw_options {
    double lr, beta1, beta2, eps;
    int64_t step;              /* 1 for the first step */
    const float *lr_dev;       /* device: the learning rate instead of lr, or NULL */
    const int64_t *step_dev;   /* device: the step instead of `step`, or NULL */
    const float *grad_scale;   /* device: a factor of all gradients (clipping, loss scaling), or NULL: 1 */
} moe_adamw_options;

/*
 * One step of AdamW (I. Loshchilov, F. Hutter, "Decoupled Weight Decay
 * Regularization", 2019) over all tensors, few launches whatever their number:
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   x = x (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in fp32.  tensors is a host array, copied into the launches; lr_dev, step_dev
 * and grad_scale are read on the device, so that a captured step can be
 * replayed with others.  An element whose g or g^2 is not finite is left as it
 * is, m and v too, and sets *dev_status = MOE_ERR_NONFINITE; a grad_scale of
 * NaN or infinity so leaves every tensor as it is.  What a step writes must not
 * overlap anything else of the call; overlapping params are refused.  beta1 and beta2 in [0, 1),
 * eps a normal fp32 number above 0, step >= 1 (a step_dev below 1 counts as 1).
 *
 * States in 8 bits (scales given; all zeros to begin with): a block of 256
 * values shares two fp32 scales.  m is held in e4m3 (to nearest, ties to even)
 * of m * (448 / max|m|), the scale being max|m| / 448.  The root r of v is held
 * in a float without a sign, with 4 exponent and 4 mantissa bits, of
 * r * (1.9375 / max r): code c > 0 stands for (1 + c % 16 / 16) 2^(c / 16 - 15)
 * times the scale, max r / 1.9375 (to nearest, ties to even; what is not zero
 * gets code 1 at least, so that no small v is taken for none); code 0 is zero.
 * A block whose largest m (or r) is below 2^-100 is held as zeros.  m and v are
 * computed in fp32, every operation rounded to nearest in the order written
 * above (no product is fused with a sum), so that the codes do not depend on a
 * machine's or compiler's choices.  x is updated from m and v before they are
 * rounded to 8 bits.  A v that changes by less than half a step of its code
 * (some 3 to 6 percent) keeps it, and the change is lost.  With beta2 up to some
 * 0.97 v is followed all the same.  With 0.999 a v that falls is NOT followed: a
 * step takes a thousandth of it, and where the gradients become ten times
 * smaller the root stays up to ten times, and the steps so much too small, for
 * good (a growing v is followed only from gradients whose squares are 30 to 60
 * times v).  Such a beta2 wants fp32 states.
 *
 * moe_adamw_states: the values that the states stand for, in fp32, tensor i's
 * to m_values[i] and v_values[i] (host arrays of device pointers, NULL entries
 * or arrays are left out): of codes, or copies of fp32 states.
 */
moe_status moe_adamw_step(const moe_adamw_tensor *tensors, int n_tensors, const moe_adamw_options *options,
                          int32_t *dev_status, moe_stream_t stream);
moe_status moe_adamw_states(const moe_adamw_tensor *tensors, int n_tensors, float *const *m_values,
                            float *const *v_values, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
