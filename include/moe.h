/*
 * moe.h -- C ABI of the MI355X (gfx950) routed-expert MoE FFN library, and
 * of the operators that surround the layer in a decode step (4-bit linears
 * with low-rank adapters beside them, norms with the residual's addition, a
 * paged key/value cache, attention over it, rules on logits, token log
 * probabilities).
 *
 * The layer: 256 routed experts, top-6 per token, plus one always-on shared
 * expert (tcti.cn post on DeepSeek-V4-Flash on 4x RTX 2080 Ti, section
 * "DeepSeek-V4-Flash的可能性"; ai-muninn.com "[洋垃圾跑大模型 #3]", section
 * "目標不是「載得進去」...").  Expert weights are FP4 E2M1 with one UE8M0
 * scale per 32 inputs, or FP8 E4M3 with one fp32 scale per 128x128 block;
 * activations are FP8 E4M3 with one fp32 scale (amax/448) per 128.  The
 * pages name the operators this ABI exposes: act_quant feeding the low-bit
 * linears, fp4_gemm (FP8-quantised activation x FP4 packed weight) and
 * fp8_gemm (tcti.cn post, section "补齐软件栈缺失"); the router picks the
 * token's experts first (dpshk.com article on deepseek-v4-flash-0731-in-c,
 * section "核心实现一"); each expert is read once for all of its tokens
 * (same article, "核心实现三"); dequantisation happens inside the product,
 * gate and up share one quantised input, and workspaces are allocated once
 * and reused (same article, "核心实现四").
 *
 * Conventions for every call:
 *  - Every buffer is a DEVICE pointer owned by the caller.  The library never
 *    allocates, frees or synchronises inside these calls (the debug helpers
 *    at the end are the only exceptions and say so).
 *  - Arguments are validated on the host first; on any error nothing is
 *    enqueued and a negative MOE_E* status is returned.  Otherwise the work
 *    is enqueued on `stream` (a hipStream_t passed as void*; NULL = the
 *    default stream) and MOE_OK is returned.  MOE_ELAUNCH means the HIP
 *    launch itself failed (the HIP error is cleared).
 *  - All device pointers must be 16-byte aligned (MOE_EALIGN otherwise);
 *    `ws` must be 256-byte aligned.
 *  - bf16 values are passed as their uint16_t bit patterns.
 *  - Expert ids outside [0, E) found on the device are skipped (their rows
 *    produce zero contribution) and set bit MOE_STATUS_BAD_EXPERT_ID in the
 *    workspace status word; no memory is accessed out of bounds.
 *  - Calls are reentrant for distinct workspaces; two calls in flight on the
 *    same workspace race.
 *  - Limits: 1 <= E <= 256, 1 <= k <= min(E, 16), H and I multiples of 128,
 *    128 <= H <= 8192, 128 <= I <= 8192, 0 <= T <= 262144 (MOE_ENOTSUP
 *    beyond the size limits, MOE_EINVAL for malformed values).  The device must be a
 *    gfx950 (MOE_ENOTSUP otherwise).
 *  - T = 0 (rows = 0 for act_quant_fp8) is an empty batch: the other
 *    arguments are checked as usual, then MOE_OK is returned with nothing
 *    read, written or enqueued (no device is needed for that answer).
 */
#ifndef BEF_MOE_H
#define BEF_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MOE_OK = 0,
  MOE_EINVAL = -1,     /* null pointer, bad size, unknown dtype            */
  MOE_ENOTSUP = -2,    /* not a gfx950 device, unknown format, size limit   */
  MOE_EALIGN = -3,     /* pointer not 16-byte (ws: 256-byte) aligned        */
  MOE_EWORKSPACE = -4, /* workspace smaller than moe_workspace_bytes()      */
  MOE_ELAUNCH = -5     /* a HIP launch failed                               */
};

/* Weight formats. */
enum {
  MOE_W_FP4_E2M1_UE8M0_K32 = 1, /* E2M1 codes 2/byte (element 2j in bits 0-3),
                                   one UE8M0 byte per 32 inputs               */
  MOE_W_FP8_E4M3_F32_B128 = 2,  /* E4M3 codes, one fp32 per 128x128 block     */
  MOE_W_INT4_BF16_GROUP = 3     /* (w4_linear only) unsigned 4-bit codes, 2/byte
                                   as above, one bf16 scale and an optional u8
                                   zero point per group of inputs             */
};

/* Activation / output dtypes (MOE_DT_FP8_E4M3, MOE_DT_FP4_E2M1: key/value
 * caches only). */
enum { MOE_DT_BF16 = 1, MOE_DT_F32 = 2, MOE_DT_FP8_E4M3 = 3, MOE_DT_FP4_E2M1 = 4 };

/* Device status word bits (see moe_device_status).  MOE_STATUS_SYNC_TIMEOUT:
 * on the small-T router or the one-token path, a block waiting for the
 * values of other blocks gave up after its bounded wait; the results of that
 * call are invalid, and the workspace must go through moe_workspace_init
 * again before its next use (a late value could outlive the clean-up). */
enum { MOE_STATUS_BAD_EXPERT_ID = 1u, MOE_STATUS_SYNC_TIMEOUT = 2u };

/* Bits that the decode-step operators OR into the caller's `status` word (a
 * device uint32_t, 4-byte aligned, cleared by the caller; NULL: not reported). */
enum { MOE_STATUS_BAD_PAGE = 4u, MOE_STATUS_BAD_TOKEN = 8u, MOE_STATUS_BAD_INDEX = 16u };

/* Stacked expert weights, expert-major; slot E (the last) is the shared
 * expert, which must have the same intermediate size as the routed ones.
 * Matrices are [out][in] row-major.
 *   FP4: gate_q/up_q [E+1][I][H/2] u8, gate_s/up_s [E+1][I][H/32] u8,
 *        down_q [E+1][H][I/2] u8,     down_s [E+1][H][I/32] u8.
 *   FP8: gate_q/up_q [E+1][I][H] u8,   gate_s/up_s [E+1][I/128][H/128] f32,
 *        down_q [E+1][H][I] u8,       down_s [E+1][H/128][I/128] f32.
 * The descriptor itself is host memory, read during the call only. */
typedef struct moe_weights {
  int32_t format;    /* MOE_W_*                      */
  int32_t n_experts; /* E, routed experts            */
  int32_t hidden;    /* H                            */
  int32_t inter;     /* I, expert intermediate size  */
  const void* gate_q;
  const void* gate_s;
  const void* up_q;
  const void* up_s;
  const void* down_q;
  const void* down_s;
} moe_weights;

/* Bytes of workspace needed by any call below for up to `max_tokens` tokens
 * at top-k `top_k` (router partials, quantised activations, routing tables,
 * intermediate h, y rows, status word).  0 if the arguments are invalid or
 * max_tokens < 1.
 * Allocate once, call moe_workspace_init once, then reuse for every call
 * (dpshk.com article, section "核心实现四": workspaces preallocated). */
size_t moe_workspace_bytes(const moe_weights* w, int32_t max_tokens, int32_t top_k);

/* Enqueue a zero-fill of the workspace's control block (about 1.3 MB: the
 * status word and the slots through which blocks of one launch hand each
 * other router partials and h values without device-scope fences; a slot
 * holds a valid mark with its value, and the block that consumes it clears
 * it, so the slots must start zeroed).  Call once after allocating a
 * workspace, before its first use (and again after MOE_STATUS_SYNC_TIMEOUT);
 * the kernels keep the control block consistent from then on. */
int moe_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* S1+S2, the router (dpshk.com article, section "核心实现一"; top-6 of 256:
 * ai-muninn.com "[洋垃圾跑大模型 #3]").
 *   x        [T][H] bf16 activations
 *   w_router [H][E] bf16
 *   topk_ids [T][k] int32 out: experts ordered by (logit desc, id asc)
 *   topk_w   [T][k] f32 out: sigmoid(logit) renormalised over the k chosen
 * Logits are fp32 sums of the exact bf16 x bf16 products in a fixed order
 * for a given T: below 256 tokens, 64-wide chunk partials (chains of fused
 * multiply-adds in ascending h from +0), sums of 4 consecutive chunks in
 * ascending order, those group sums in ascending order; from 256 tokens on,
 * sums over 512-row groups formed on the matrix cores (bf16 MFMA, fp32
 * accumulation in the hardware's order), added in ascending group order.
 * The ids are deterministic.  They are the
 * exact top-k of these logits; logits summed in any other order differ by
 * rounding only, so another order can rank two experts differently only
 * where their logits lie within rounding distance of each other.
 * ws: workspace of at least moe_workspace_bytes(.., T, k). */
int moe_route(const uint16_t* x, const uint16_t* w_router, int32_t T, int32_t H, int32_t E,
              int32_t k, int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes,
              void* stream);

/* S3, act_quant (tcti.cn post, section "补齐软件栈缺失"): per row and per
 * 128 columns, s = amax/448 (fp32, IEEE division) and
 * q = E4M3(x / s) rounded to nearest even, saturating at +-448, sign kept;
 * an all-zero block gives s = 0 and q = 0.
 *   x      [rows][cols] bf16 (x_dtype MOE_DT_BF16) or f32 (MOE_DT_F32)
 *   q      [rows][cols] u8 E4M3 codes out
 *   scales [rows][cols/128] f32 out
 * cols must be a multiple of 128; rows >= 0. */
int act_quant_fp8(const void* x, int32_t x_dtype, int64_t rows, int32_t cols, uint8_t* q,
                  float* scales, void* stream);

/* S4, permute (dpshk.com article, section "核心实现三": each expert read
 * once for all of its tokens): a stable counting sort of the T*k
 * (token, slot) pairs by expert, tokens ascending within an expert, then
 * the shared-expert group (index E) holding tokens 0..T-1.
 *   offsets   [E+2] out: group g is rows offsets[g] .. offsets[g+1]-1
 *   row_token [T*k+T] out: token of each row
 *   row_of    [T][k+1] out: row of (t, slot j); row_of[t][k] = shared row;
 *             -1 for a pair whose id is outside [0, E)
 * Rows that a dropped pair would have used are never written. */
int moe_permute(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E, int32_t* offsets,
                int32_t* row_token, int32_t* row_of, void* ws, size_t ws_bytes, void* stream);

/* S5+S6, the experts (tcti.cn post, section "补齐软件栈缺失": fp4_gemm and
 * fp8_gemm; dpshk.com article, section "核心实现四": dequantise inside the
 * product, gate and up share one quantised input).  For every row r of
 * group g (expert g, or the shared expert for g = E) and its token t:
 *   g = W_gate[g] . deq(xq[t]),  u = W_up[g] . deq(xq[t])   (fp32 accumulate)
 *   h = silu(g) * u, requantised to E4M3 per 128 exactly as act_quant_fp8
 *   y_rows[r] = W_down[g] . deq(hq)
 *   xq [T][H] u8, xs [T][H/128] f32 (act_quant_fp8 of x)
 *   offsets, row_token as produced by moe_permute
 *   y_rows [T*k+T][H] f32 out (rows of dropped pairs are left untouched)
 * A few tokens -- 1 <= T <= 4 with k+1 <= 8, T*(k+1) <= 32, H <= 8192 and
 * I <= 4096, either weight format -- run the VALU GEMV kernels (weights
 * streamed from HBM into registers, no matrix-core tile to fill); any other
 * shape runs the MFMA grouped GEMM kernels. */
int moe_expert_ffn(const moe_weights* w, const uint8_t* xq, const float* xs, int32_t T, int32_t k,
                   const int32_t* offsets, const int32_t* row_token, float* y_rows, void* ws,
                   size_t ws_bytes, void* stream);

/* S5 alone: gate + up + SwiGLU for every row, h requantised to E4M3 per 128
 * and kept in `ws` for moe_expert_down (same kernels moe_expert_ffn runs
 * first; arguments as moe_expert_ffn). */
int moe_expert_gate_up(const moe_weights* w, const uint8_t* xq, const float* xs, int32_t T,
                       int32_t k, const int32_t* offsets, const int32_t* row_token, void* ws,
                       size_t ws_bytes, void* stream);

/* S6 alone (+ S7): the down projection of the h that moe_expert_gate_up left
 * in `ws` (same T, k, offsets), into y_rows [T*k+T][H] f32.  When `out` is
 * set the combine (S7) follows, using row_of and topk_w: on the VALU GEMV
 * path (see moe_expert_ffn) it is fused into the down kernel and y_rows may
 * be NULL; on the MFMA path y_rows is required and a combine kernel runs. */
int moe_expert_down(const moe_weights* w, int32_t T, int32_t k, const int32_t* offsets,
                    const int32_t* row_of, const float* topk_w, float* y_rows, void* out,
                    int32_t out_dtype, void* ws, size_t ws_bytes, void* stream);

/* S7, combine: the always-on shared expert's output plus the token's routed
 * experts' outputs weighted by their gate weights (tcti.cn post, section
 * "DeepSeek-V4-Flash的可能性": top-6 routed experts beside one shared
 * expert; the rows come back from the expert-major order of the batch,
 * dpshk.com article, section "核心实现三"):
 *   out[t] = y_rows[row_of[t][k]] + sum_{j<k} topk_w[t][j] * y_rows[row_of[t][j]]
 * in fp32 in that order (rows of -1 contribute 0), written as bf16 (nearest
 * even) or f32.
 *   y_rows [rows][H] f32, row_of [T][k+1] int32, topk_w [T][k] f32
 *   out [T][H] (out_dtype MOE_DT_BF16 or MOE_DT_F32)
 * Limits as for every call: 1 <= k <= 16, 0 <= T <= 262144, H a multiple of
 * 128 up to 8192. */
int moe_combine(const float* y_rows, const int32_t* row_of, const float* topk_w, int32_t T,
                int32_t k, int32_t H, void* out, int32_t out_dtype, void* stream);

/* The whole layer, S1..S7, on x [T][H] bf16 -> out [T][H] (bf16 or f32).
 * routing_ids/routing_w [T][k] (both NULL, or both set) inject routing
 * (e.g. a drawn routing, or a speculative-verification batch whose routing
 * is known, dpshk.com article section "核心实现三"); when NULL the router
 * runs on x. */
int dsv4_moe_forward(const moe_weights* w, const uint16_t* w_router, const uint16_t* x, int32_t T,
                     int32_t k, const int32_t* routing_ids, const float* routing_w, void* out,
                     int32_t out_dtype, void* ws, size_t ws_bytes, void* stream);

/* The whole layer as dsv4_moe_forward, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): no workspace argument, no allocation of
 * any kind.  The workspace is a file-scope device array of the library,
 * MOE_NOALLOC_SCRATCH_BYTES bytes on each GPU it runs on, held until the
 * process ends; its device address is looked up on the first call on a
 * device (that device current), and its control block is then cleared by a
 * fill kernel enqueued on `stream`.  A call whose workspace need
 * (moe_workspace_bytes(w, T, k)) exceeds the array returns MOE_ENOTSUP with
 * nothing enqueued -- about 100 tokens at hidden 4096, intermediate 2048,
 * top-6.  Every call on one GPU shares that array: two calls in flight at
 * once on one GPU (different streams, or different threads) race and give
 * wrong results.  Results equal dsv4_moe_forward's bit for bit (same
 * kernels).  Its status word cannot be read (moe_device_status needs a
 * workspace); bad expert ids are still skipped. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
int dsv4_moe_forward_noalloc(const moe_weights* w, const uint16_t* w_router, const uint16_t* x,
                             int32_t T, int32_t k, const int32_t* routing_ids,
                             const float* routing_w, void* out, int32_t out_dtype, void* stream);

/* ---- Host-resident experts ------------------------------------------------
 * For layers whose routed experts do not all fit in HBM, the pages keep the
 * routed experts in host memory and move each to the GPU when a token needs
 * it, computing on arrival, with a per-layer LRU cache of experts on the GPU
 * and double-buffered copies (dpshk.com article, sections "核心实现一" and
 * "核心实现二"; tcti.cn post, section "DeepSeek-V4-Flash的可能性": routed
 * experts in host memory).  Here: one layer's cache is n_slots expert slots
 * in HBM plus one slot for the shared expert; a call routes on the GPU,
 * reads the ids back (it synchronises `stream` once for that), keeps hits in
 * their slots, copies each miss into a free or least-recently-used slot on
 * `copy_stream`, runs the experts already resident at once and the copied
 * ones when `copies_done` (recorded after the last copy) has fired, then
 * combines.  Expert math and the combine order are those of
 * dsv4_moe_forward.
 *
 * The cache state lives in caller-owned HOST memory:
 *   n_experts = E of the layer, n_slots = slots in HBM (1..E),
 *   slot_of [E] (slot of expert e or -1), expert_of [n_slots] (-1 if free),
 *   last_use [n_slots] (call count of last use), initially all -1 / -1 / 0,
 *   calls = 0, shared_resident = 0 (the first call copies the shared
 *   expert into slot n_slots, where it stays); hits, misses, bytes_copied
 *   count distinct experts per call and bytes sent to the GPU. */
typedef struct moe_expert_cache {
  int32_t n_experts;
  int32_t n_slots;
  int32_t* slot_of;
  int32_t* expert_of;
  uint64_t* last_use;
  uint64_t calls;
  int32_t shared_resident;
  int32_t pad_;
  uint64_t hits, misses, bytes_copied;
} moe_expert_cache;

/* Workspace bytes (device) of moe_forward_host_experts for up to max_tokens
 * tokens of the layer `host_w` (0 on invalid arguments). */
size_t moe_host_experts_workspace_bytes(const moe_weights* host_w, int32_t max_tokens,
                                        int32_t top_k);

/* Pinned host scratch bytes of moe_forward_host_experts (ids read back, slot
 * ids and group masks staged for upload). */
size_t moe_host_experts_scratch_bytes(int32_t n_experts, int32_t max_tokens, int32_t top_k);

/* The whole layer with routed experts in host memory (see above).
 *   host_w: the layer's E+1 experts in HOST memory (pinned for asynchronous
 *           copies), layout as moe_weights;
 *   slot_w: the cache's slots in DEVICE memory, n_experts = n_slots: slot s
 *           of each array holds one expert, slot n_slots the shared expert;
 *   w_router [H][E], x [T][H] bf16 on the device; out [T][H] bf16 or f32;
 *   ws: device workspace of moe_host_experts_workspace_bytes (moe_workspace_init
 *       once), host_scratch: pinned host memory of
 *       moe_host_experts_scratch_bytes;
 *   copies_done: a hipEvent_t (void*) the call records on copy_stream;
 *   stream: compute stream; copy_stream: host-to-device copies.
 * Requires every expert of a call to fit at once: T*k <= n_slots unless
 * n_slots = E (MOE_ENOTSUP otherwise).  Synchronises `stream` once (the ids
 * must reach the host to choose the copies); returns with the copies and the
 * layer enqueued.  Reentrant only for distinct caches, slots, workspaces and
 * streams. */
int moe_forward_host_experts(const moe_weights* host_w, const moe_weights* slot_w,
                             moe_expert_cache* cache, const uint16_t* w_router, const uint16_t* x,
                             int32_t T, int32_t k, void* out, int32_t out_dtype, void* ws,
                             size_t ws_bytes, void* host_scratch, size_t host_scratch_bytes,
                             void* copies_done, void* stream, void* copy_stream);

/* ---- Operators of the decode step around the layer --------------------------
 * The conventions at the top hold: device pointers, host-checked arguments,
 * nothing allocated or synchronised, the work enqueued on `stream`, calls
 * capturable in a HIP graph.  Workspaces need no initialisation.  Where a limit
 * is not stated otherwise, 0 <= T <= 262144 tokens, T = 0 an empty batch.
 * Strides are in elements.  Index arrays (tokens, positions, pages) need 4-byte
 * alignment, everything else 16 bytes. */

/* 4-bit weights of a linear, [n_out][n_in] row-major, two codes per byte
 * (element 2j in bits 0-3), n_in a multiple of 32.
 *   MOE_W_FP4_E2M1_UE8M0_K32: group 32, scale u8 [n_out][n_in/32] UE8M0 (255 is
 *     NaN), zero NULL; w = e2m1(code) * 2^(scale - 127)
 *   MOE_W_INT4_BF16_GROUP: group 32, 64 or 128, G = ceil(n_in / group), scale
 *     bf16 [n_out][G], zero u8 [n_out][G] or NULL (8 everywhere);
 *     w = scale * (code - zero)
 * The descriptor is host memory, read during the call only. */
typedef struct w4_weights {
  int32_t format;
  int32_t n_out;
  int32_t n_in;
  int32_t group;
  const void* q;
  const void* scale;
  const void* zero;
} w4_weights;

/* y[t][n] = sum_k x[t][k] w[n][k]: the projections around the expert layer for
 * a few tokens (any T is valid; tuned up to 64).  Codes and activations
 * enter the products unrounded, sums are fp32, y is rounded once.  (INT4 sums
 * code x and x apart, so an infinite activation gives NaN in its token.)
 *   x [T][n_in] bf16, rows x_stride apart (a multiple of 8, >= n_in)
 *   y [T][n_out] bf16 or f32 (y_dtype), rows y_stride >= n_out apart
 * n_out and n_in up to 2^20 (MOE_ENOTSUP beyond). */
int w4_linear(const w4_weights* w, const uint16_t* x, int64_t x_stride, int32_t T, void* y,
              int64_t y_stride, int32_t y_dtype, void* stream);

/* Low-rank adapters of one linear, n_adapters of them stacked:
 *   a [n_adapters][max_rank][n_in] bf16, b [n_adapters][n_out][max_rank] bf16
 *   rank [n_adapters] int32 (device), 0 to max_rank, or NULL (all max_rank): what a
 *     and b hold past an adapter's rank is not used
 *   scale [n_adapters] f32 (device) or NULL (1)
 * max_rank and n_in are multiples of 8, max_rank up to 128, n_in and n_out up to
 * 2^20, n_adapters up to 65536 (MOE_ENOTSUP beyond).  The descriptor is host memory,
 * read during the call only. */
typedef struct lora_weights {
  int32_t n_adapters;
  int32_t max_rank;
  int32_t n_in;
  int32_t n_out;
  const void* a;
  const void* b;
  const int32_t* rank;
  const float* scale;
} lora_weights;

/* Workspace bytes of lora_linear for up to T tokens (0 on invalid arguments). */
size_t lora_workspace_bytes(const lora_weights* w, int32_t T);

/* y[t] = base[t] + scale_i b_i (a_i x[t]) with i = adapter_of[t]: the adapters of many
 * requests beside a projection that they share (base: what w4_linear or another
 * product left).  a_i x is kept in fp32, both products accumulate in fp32, y is
 * rounded once.  An infinite element of b gives its infinity or NaN, by the number
 * of tokens and the bits of a_i x (which meets b_i in three bf16 parts that add up
 * to it; a part of 0 gives NaN).
 *   x [T][n_in] bf16, rows x_stride apart (a multiple of 8, >= n_in)
 *   adapter_of [T] int32; negative: none (y = base).  An index >= n_adapters is none
 *     too and sets MOE_STATUS_BAD_INDEX.  Tokens of one adapter need not be
 *     neighbours; runs of 16 or more of them read its weights less often.
 *   base [T][n_out], rows base_stride apart, of y's type; NULL: zeros.  base may be y,
 *     with y's stride; otherwise they must not overlap
 *   y [T][n_out] bf16 or f32 (y_dtype), rows y_stride >= n_out apart */
int lora_linear(const lora_weights* w, const uint16_t* x, int64_t x_stride, int32_t T,
                const int32_t* adapter_of, const void* base, int64_t base_stride, void* y,
                int64_t y_stride, int32_t y_dtype, uint32_t* status, void* ws, size_t ws_bytes,
                void* stream);

/* The residual's addition and the root-mean-square norm, with the quantisation that
 * the experts and the FP8 linears take:
 *   r = x + residual, rounded to the residual's type (what res_out holds; without a
 *       residual r = x),  y = r / sqrt(mean(r^2) + eps) * weight  in fp32
 *   x [T][H] bf16, rows x_stride apart (a multiple of 8)
 *   residual [T][H] bf16 or f32 (res_dtype), rows res_stride apart (a multiple of 8),
 *     or NULL (res_out then NULL too)
 *   weight [H] bf16 or NULL (1); eps >= 2^-100
 *   res_out [T][H] of res_dtype, rows res_stride apart, or NULL; may be `residual`
 *   y [T][H] bf16, contiguous, or NULL
 *   q [T][H] u8 and scales [T][H/128] f32, contiguous: y quantised from fp32 by the
 *     rule of act_quant_fp8 (not from the rounded y; NaN and infinities as
 *     kv_append_rope has them in an E4M3 cache), or both NULL; H then a multiple
 *     of 128
 * One of y and q at least.  H is a multiple of 8 up to 16384.  Outputs overlap no input
 * but as stated.  Sums of squares past fp32's range are formed again in units of a
 * power of two; a row with a NaN or an infinity follows the formula. */
int add_rmsnorm(const uint16_t* x, int64_t x_stride, const void* residual, int32_t res_dtype,
                int64_t res_stride, int32_t T, int32_t H, const uint16_t* weight, float eps,
                void* res_out, uint16_t* y, uint8_t* q, float* scales, void* stream);

/* A paged key/value cache.  k and v are [n_pages][n_kv_heads][page_size]
 * [head_dim], bf16, E4M3 or E2M1 (two codes per byte, element 2j in bits 0-3).  An E4M3
 * cache has one fp32 scale per row in k_scale and v_scale, [n_pages][n_kv_heads]
 * [page_size]; an E2M1 cache one UE8M0 byte per 32 columns, [n_pages][n_kv_heads]
 * [page_size][head_dim/32], whose bytes above 252 stand for 32 NaN; NULL for bf16.
 * page_size is a power of two, 16 to 1024; head_dim 64, 128 or 256; n_kv_heads
 * <= 1024.  The descriptor is host memory, read during the call only. */
typedef struct kv_cache {
  int32_t dtype;
  int32_t n_pages;
  int32_t page_size;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t pad_;
  void* k;
  void* v;
  float* k_scale; /* E2M1: its uint8_t, as this pointer */
  float* v_scale;
} kv_cache;

/* How pairs are laid out in a rotated head of rope_dim elements: element i
 * with i + rope_dim/2, or 2i with 2i + 1. */
enum { MOE_ROPE_HALF = 1, MOE_ROPE_PAIRS = 2 };

/* Rotates q and k by their tokens' positions and appends k and v to the cache.
 * Token t is key number pos[t] of sequence seq_of[t]: its slot is
 * pos % page_size of page page_table[seq][pos / page_size].  A pair (a, b) of
 * the first rope_dim elements of a head becomes (a c - b s, b c + a s) in fp32,
 * each operation rounded, with c = rope[pos][i], s = rope[pos][rope_dim/2 + i];
 * the other elements and v are taken as they are.  Cache rows are bf16 (nearest
 * even), or E4M3 by the rule of act_quant_fp8 over the whole head row, where a NaN
 * becomes E4M3's NaN and leaves the row's other values as they are; an infinity
 * leaves the row no finite value (scale inf).  In an E2M1 cache each 32 columns have
 * the smallest power of two that brings their largest to 6 at most (2^-127 at least,
 * 2^125 at most, where larger values become 6), and codes are rounded to nearest
 * even; a NaN or an infinity makes the 32 columns NaN (byte 255).
 *   q [T][n_q_heads][head_dim] bf16, token rows q_stride apart; n_q_heads = 0
 *     (q, q_out NULL): keys and values only
 *   k, v [T][n_kv_heads][head_dim] bf16, token rows k_stride, v_stride apart
 *     (multiples of 8; a fused projection's output can be passed in place)
 *   rope [rope_rows][rope_dim] f32: cosines, then sines; rope_dim a multiple of
 *     16 up to head_dim, or 0 (no rotation, rope NULL)
 *   seq_of, pos [T] int32; page_table [n_seqs][table_cols] int32
 *   q_out [T][n_q_heads][head_dim] bf16, contiguous; must not overlap an input
 * A negative seq_of or pos is padding: nothing is written for the token.  So is
 * a token whose sequence, position or page is out of range, which also sets
 * MOE_STATUS_BAD_PAGE.  Two tokens of one call for the same slot race. */
int kv_append_rope(const kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                   const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                   int32_t T, const float* rope, int32_t rope_rows, int32_t rope_dim,
                   int32_t rope_style, const int32_t* seq_of, const int32_t* pos,
                   const int32_t* page_table, int32_t n_seqs, int32_t table_cols, uint16_t* q_out,
                   uint32_t* status, void* stream);

/* Workspace bytes of attn_shared_prefix with these arguments (0 if they are
 * invalid). */
size_t attn_workspace_bytes(const kv_cache* cache, int32_t n_seqs, int32_t q_len,
                            int32_t n_q_heads, int32_t prefix_len, int32_t max_keys);

/* Attention over the cache for a batch whose sequences share their first
 * prefix_len keys, which are read once for the whole batch.  Query token
 * t = b * q_len + i of sequence b sees the keys 0 .. pos[t] of its sequence:
 * those below prefix_len in the pages prefix_pages [ceil(prefix_len /
 * page_size)], the others in page_table[b] (indexed from key 0, as kv_append_rope
 * does; its entries below prefix_len / page_size are not read).  prefix_len
 * may end inside a page, and may be 0.
 *   q [n_seqs * q_len][n_q_heads][head_dim] bf16, token rows q_stride apart (a
 *     multiple of 8); n_q_heads a multiple of n_kv_heads, head h reading kv head
 *     h / (n_q_heads / n_kv_heads)
 *   pos [n_seqs * q_len] int32; negative: the token sees no key (padding)
 *   max_keys: an upper bound of pos + 1 (prefix_len <= max_keys <=
 *     table_cols * page_size); keys from max_keys on are not seen and a token
 *     that would see one sets MOE_STATUS_BAD_PAGE
 *   scale: positive; o = sum_j softmax_j(scale q.k_j) v_j
 *   out [n_seqs * q_len][n_q_heads][head_dim] bf16
 *   lse [n_seqs * q_len][n_q_heads] f32 or NULL: log sum_j exp(scale q.k_j)
 * A row that sees no key, or none with a score above -inf, gives out 0 and lse
 * -inf; one with a NaN score (in q, or in K at a key it sees) gives NaN.  What the
 * cache holds at keys that a row does not see (NaN included) does not enter it.  A
 * page number outside the cache hides its keys and sets MOE_STATUS_BAD_PAGE.
 * Scores and sums are fp32.  K and V of an E2M1 cache become bf16 exactly.  For the
 * product with V a key's weight is rounded to bf16; in an E4M3 cache the weight times
 * the key's V scale to fp16, by 2^-11 of itself or by 2^-29 of the row's largest if
 * that is more (V scales up to 2^80 apart).
 * Sums are formed of weights up to 8 and divided at the end: |v| times 8 times the
 * keys has to stay within fp32's range.
 * n_seqs * q_len <= 262144, n_q_heads <= 1024, n_seqs * q_len * n_q_heads < 2^24
 * and max_keys <= 2^28. */
int attn_shared_prefix(const kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t n_seqs,
                       int32_t q_len, int32_t n_q_heads, const int32_t* pos,
                       const int32_t* prefix_pages, int32_t prefix_len, const int32_t* page_table,
                       int32_t table_cols, int32_t max_keys, float scale, uint16_t* out,
                       float* lse, uint32_t* status, void* ws, size_t ws_bytes, void* stream);

/* Rules on the logits of T rows; what is NULL (n_bias 0) is left out.
 *   history [n_seqs][>= max_history] int32, rows history_stride apart: token ids; row
 *     t's text is the first n_tokens[t] of row seq_of[t] (NULL: row t; negative: no
 *     text), and its first n_prompt[t] (NULL: 0) were given, the others
 *     generated.  n_tokens is at most max_history (a longer text is cut, and sets
 *     MOE_STATUS_BAD_INDEX, as does a seq_of >= n_seqs, which has no text).
 *     Negative ids are padding; so is an id >= V, which sets MOE_STATUS_BAD_TOKEN.
 *   repetition [T]: ids of the text: z > 0 ? z / repetition : z * repetition
 *   presence, frequency [T]: ids generated c > 0 times: z - (presence + frequency c)
 *   bias_ids [T][n_bias] int32, bias [T][n_bias] f32: added to z.  Of several entries of
 *     one id the last counts; negative ids are no entry; so is an id >= V, which
 *     sets MOE_STATUS_BAD_TOKEN
 *   mask [n_masks] rows of ceil(V/32) words, mask_stride words apart: bit v % 32 of word
 *     v / 32 allows id v; row t has mask mask_of[t] (NULL: mask t; negative: all
 *     are allowed; so for a number >= n_masks, which sets MOE_STATUS_BAD_INDEX)
 * The rule pointers are device memory, 4-byte aligned; the struct is host memory,
 * read during the call only.  max_history < 2^20, n_bias <= 2047 (MOE_ENOTSUP beyond). */
typedef struct logits_rules {
  const int32_t* history;
  int64_t history_stride;
  int32_t max_history;
  int32_t n_seqs;
  const int32_t* seq_of;
  const int32_t* n_tokens;
  const int32_t* n_prompt;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* mask;
  int64_t mask_stride;
  const int32_t* mask_of;
  int32_t n_masks;
  int32_t n_bias;
} logits_rules;

/* out[t] = the logits z[t] under the rules, in this order: bias, repetition, presence
 * and frequency, mask (-inf where an id is not allowed, whatever z is there).
 * In fp32, rounded once.  A mask may leave a row nothing: it is then -inf
 * throughout.
 *   z [T][V] bf16 or f32, rows z_stride >= V apart
 *   out [T][V] bf16 or f32, rows out_stride >= V apart; may be z, with z's type and
 *     stride (logits that no rule touches are then not written); otherwise they
 *     must not overlap
 * z and out need the alignment of their elements only.  1 <= V <= 2^24. */
int logits_adjust(const logits_rules* rules, const void* z, int32_t z_dtype, int64_t z_stride,
                  int32_t T, int32_t V, void* out, int32_t out_dtype, int64_t out_stride,
                  uint32_t* status, void* stream);

/* Workspace bytes of token_logprobs for up to T rows (0 on invalid arguments). */
size_t token_logprobs_workspace_bytes(int32_t T, int32_t V, int32_t n_top);

/* Log probabilities under softmax(z[t]) of the given tokens, the entropy of the
 * distribution, and the n_top best alternatives by (z descending, id ascending,
 * NaN last).
 *   z [T][V] bf16 or f32, rows row_stride >= V apart (any alignment of the rows)
 *   tokens [T] int32 and logprob [T] f32, or both NULL; an id outside [0, V) is
 *     no token: logprob 0 (an id >= V also sets MOE_STATUS_BAD_TOKEN)
 *   entropy [T] f32 (nats) or NULL
 *   top_ids [T][n_top] int32, top_logprobs [T][n_top] f32, 0 <= n_top <=
 *     min(64, V) (both may be NULL when n_top = 0)
 * A logit of -inf has probability 0.  A row of nothing else gives log
 * probabilities of -inf and entropy 0; a row with +inf or NaN gives NaN.
 * 1 <= V <= 2^24. */
int token_logprobs(const void* z, int32_t z_dtype, int64_t row_stride, int32_t T, int32_t V,
                   const int32_t* tokens, int32_t n_top, float* logprob, float* entropy,
                   int32_t* top_ids, float* top_logprobs, uint32_t* status, void* ws,
                   size_t ws_bytes, void* stream);

/* A static string naming a status code. */
const char* moe_status_string(int status);

/* DEBUG/TESTS ONLY -- synchronises `stream`.  Reads the workspace status
 * word into *status (MOE_STATUS_* bits) and clears it when `clear` != 0. */
int moe_device_status(void* ws, void* stream, uint32_t* status, int clear);

/* DEBUG/TESTS ONLY -- device pointers to the intermediate activations that
 * the last moe_expert_ffn / dsv4_moe_forward call with the same (w, T, k)
 * left in `ws`: h [T*k+T][I] f32 (VALU path only, else NULL), and
 * hq [T*k+T][I] u8 with hs [T*k+T][I/128] f32 (both paths).  T >= 1 (an
 * empty batch leaves none: MOE_EINVAL). */
int moe_debug_intermediates(const moe_weights* w, int32_t T, int32_t k, void* ws,
                            size_t ws_bytes, float** h, uint8_t** hq, float** hs);

/* DEBUG/TESTS ONLY -- while set, every MFMA grouped-GEMM gate+up launch of
 * a call with (T*k+T)*I <= n_floats also stores its fp32 h (SwiGLU output,
 * before requantisation) into h [T*k+T][I] (device memory owned by the
 * caller, 16-byte aligned); the VALU path keeps its h in the workspace (see
 * moe_debug_intermediates).  NULL and 0 clear it.  Process-wide and not
 * thread-safe.  MOE_EINVAL if exactly one of h, n_floats is zero. */
int moe_debug_store_h(float* h, size_t n_floats);

/* DEBUG/TESTS ONLY -- device pointers to the expert ids [T][k] int32 and
 * weights [T][k] f32 that the router of the last dsv4_moe_forward call with
 * the same (w, T, k) and no injected routing left in `ws`.  T >= 1. */
int moe_debug_routing(const moe_weights* w, int32_t T, int32_t k, void* ws, size_t ws_bytes,
                      int32_t** ids, float** topk_w);

/* Kernels that moe_debug_time_kernel can time: the gate+up and the down
 * kernels of the VALU path (GEMV) and of the grouped GEMM, and the fused
 * one-token expert kernel (gate+up, down and combine in one launch). */
enum {
  MOE_KERNEL_GEMV_GATE_UP = 1,
  MOE_KERNEL_GEMM_GATE_UP = 2,
  MOE_KERNEL_GEMV_DOWN = 3,
  MOE_KERNEL_GEMM_DOWN = 4,
  MOE_KERNEL_DECODE_FFN = 5
};

/* DEBUG/BENCHMARK ONLY -- the one-token path of dsv4_moe_forward with the
 * router on the device and FP4 weights: `fused` = 1 runs the routed experts'
 * gate+up, the down projection of all k + 1 experts and the combine as one
 * persistent kernel wherever it fits (T = 1, k + 1 <= 8, inter <= 2048,
 * hidden <= 4096 and a multiple of 16 with hidden / 16 <= the device's
 * compute units), 0 (the default: measured faster) the separate gate+up and
 * down+combine kernels.  Both give bit-identical outputs.  The fused kernel runs one block per compute unit
 * and its blocks wait on each other's results (bounded waits): it expects
 * the device to itself for its duration; when other work holds compute
 * units, the waits may run out, which sets MOE_STATUS_SYNC_TIMEOUT.
 * Process-wide and not thread-safe; MOE_EINVAL for other values. */
int moe_debug_set_decode_fused(int32_t fused);

/* DEBUG/BENCHMARK ONLY -- kernel timing.  While set, every launch of kernel
 * `which` (MOE_KERNEL_*) records `start_event` and `stop_event` (hipEvent_t
 * passed as void*) at that kernel's own begin and end, as part of its
 * dispatch (hipExtLaunchKernelGGL), so their elapsed time is the kernel's
 * duration without queueing gaps.  Two NULL events clear it.  Process-wide
 * and not thread-safe.  MOE_EINVAL for an unknown kernel. */
int moe_debug_time_kernel(int32_t which, void* start_event, void* stop_event);

/* DEBUG/BENCHMARK ONLY -- enqueue a plain streaming read of `bytes` (a
 * multiple of 16) at `src` by `blocks` blocks of 512 threads (16-byte
 * loads, four in flight per lane): the practical HBM read ceiling the
 * kernels are measured against.  `sink` (4 bytes of device memory) is
 * written only if the XOR of the data read equals an arbitrary constant. */
int moe_debug_stream_read(const void* src, size_t bytes, uint32_t* sink, int32_t blocks,
                          void* stream);

#ifdef __cplusplus
}
#endif
#endif /* BEF_MOE_H */
