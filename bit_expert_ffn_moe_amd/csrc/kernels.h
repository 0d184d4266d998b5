// kernels.h -- launchers of the gfx950 kernels (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace bef {

constexpr int kRouteSmallT = 4;           // router: per-chunk blocks + last-block top-k
constexpr int kRouteMaxGroups = 32;       // router: 256-row groups, H <= 8192
constexpr int kRouteSplitT = 256;         // router: experts also split in quarters below this T
constexpr int kRouteMfmaRows = 512;       // router from kRouteSplitT tokens: rows per group sum
constexpr int kPermuteSmallPairs = 2048;  // permute: single block up to this many pairs
constexpr int kPermuteTokBlock = 256;     // permute: tokens per block above that
constexpr int kGemvMaxRows = 8;           // VALU GEMV path: rows (k + 1) per token
constexpr int kGemvMaxT = 4;              // VALU GEMV path: at most this many tokens
constexpr int kHSlotRowsHost = 32;        // VALU GEMV path: rows T*(k+1) (h exchange slots)
constexpr uint32_t MOE_STATUS_BAD_EXPERT_ID_DEV = 1u;

// Optional start/stop events of one kernel's launches (debug timing; set by
// moe_debug_time_kernel, index MOE_KERNEL_*).
struct KernelTimer {
  hipEvent_t start, stop;
};
extern KernelTimer g_kernel_timer[6];

struct GemvArgs {
  const uint8_t *gq, *gs, *uq, *us, *dq, *ds;
  const uint8_t* xq;
  const float* xs;
  const int4* active;      // set: {group, first row, end row} per slot
  const int32_t *offsets, *row_token, *row_of;
  const float* topk_w;
  int E, H, I, k, n_slots;
  float* h;
  float* y_rows;
  void* out;
  int out_bf16;
  uint8_t* hq_ws;
  float* hs_ws;
  uint64_t* h_slots;    // tagged slots of the h exchange (zero between launches)
  uint32_t* status;
  int n_rows;           // down with an active list: T*k + T rows, the last T the shared ones
  int fmt;              // 1: FP4 weights, 2: FP8
  int T;                // tokens
  const uint8_t* group_mask;  // [E+1] or null: groups with 0 are skipped (no active list)
};

struct GemmArgs {
  int fmt;
  const uint8_t *gq, *uq, *dq;
  const void *gs, *us, *ds;
  const uint8_t* xq;
  const float* xs;
  const int32_t *offsets, *row_token;
  int T, k, E, H, I;
  uint8_t* hq;
  float* hs;
  float* y_rows;
  float* h_dbg;   // debug: fp32 h [T*k+T][I] of the gate+up kernels when set
  const uint8_t* group_mask;  // [E+1] or null: groups with 0 are skipped
};

// The one-token fused expert kernel (decode.hip): 16 output rows per block
// (one block per CU), 12 waves, at most 8 h rows (k + 1).
constexpr int kDecRowsPerBlock = 16;
constexpr int kDecWaves = 12;
constexpr int kDecMaxRows = 8;
struct DecodeArgs {
  const uint8_t *gq, *gs, *uq, *us, *dq, *ds;  // FP4 weights [E+1][...]
  const uint8_t* xq;          // the token's E4M3 codes [H] and scales [H/128]
  const float* xs;
  const int4* active;         // routed slots {group, row, row + 1} (rows 0 .. k-1)
  const int32_t* row_of;      // [k+1]: h row of rank j, then the shared row
  const float* topk_w;        // [k]
  int E, H, I, k;
  float* h;                   // [k+1][I] fp32 h (inspection)
  uint8_t* hq;                // [k+1][I] requantised h (row k: the shared expert's, read)
  float* hs;                  // [k+1][I/128]
  uint64_t* dec_h;            // WsCtl::dec_h, dec_c, dec_epoch, dec_done
  uint64_t* dec_c;
  uint32_t* epoch;
  uint32_t* done;
  uint32_t* cnt;              // [8][16] published gate+up units per 128-block
  uint32_t* status;
  void* out;                  // [H] f32 or bf16
  int out_bf16;
};
bool decode_ffn_fits(int fmt, int T, int k, int H, int I);
hipError_t launch_decode_ffn(const DecodeArgs& a, hipStream_t st);

// Debug sink of the grouped GEMM's fp32 h (moe_debug_store_h).
struct HSink {
  float* h;
  size_t n;
};
extern HSink g_h_sink;

// Small-T front of the layer: router (+ act_quant of x when xq is set,
// + permutation tables when offsets is set).
struct WsCtl;
struct FrontArgs {
  const uint16_t* x;
  const uint16_t* wr;
  int T, H, E, k;
  uint64_t* slots;        // [H/256][T][E] tagged group sums (zero between launches)
  int32_t* ids;
  float* w;
  uint8_t* xq;
  float* xs;
  int32_t *offsets, *row_token, *row_of;
  int4* active;           // routed groups {group, first row, end row}, -1 padded
  int n_active_slots;
  // shared expert's gate+up rows run in the same kernel when sh_h is set
  // (fmt 1: FP4 weights, 2: FP8)
  const uint8_t *sh_gq, *sh_gs, *sh_uq, *sh_us;
  int fmt;
  int I;
  float* sh_h;
  uint8_t* sh_hq;         // requantised h (rows of the shared expert)
  float* sh_hs;
  uint64_t* h_slots;
  uint32_t* status;
};
void set_route_sync(FrontArgs& a, WsCtl* ctl);
hipError_t launch_route_front(const FrontArgs& a, hipStream_t st);

hipError_t launch_act_quant(const void* x, bool bf16, int64_t rows, int32_t cols, uint8_t* q,
                            float* s, hipStream_t st);
// T > kRouteSmallT needs gsum: (H/256) * T * E floats of workspace (group sums;
// from kRouteSplitT tokens on, H/kRouteMfmaRows of them are used), and from
// kRouteSplitT tokens on wrT: E * H bf16 (the router matrix transposed).
// xq/xs set: the act_quant of x runs in the same launch (T > kRouteSmallT) or
// in the front kernel (T <= kRouteSmallT).
hipError_t launch_route(const uint16_t* x, const uint16_t* wr, int T, int H, int E, int k,
                        int32_t* ids, float* w, WsCtl* ctl, float* gsum, uint16_t* wrT,
                        hipStream_t st, uint8_t* xq = nullptr, float* xs = nullptr);
hipError_t launch_permute(const int32_t* ids, int T, int k, int E, int32_t* offsets,
                          int32_t* row_token, int32_t* row_of, int32_t* cnt,
                          uint32_t* status, hipStream_t st);
hipError_t launch_combine(const float* y, const int32_t* row_of, const float* topk_w, int T, int k,
                          int H, void* out, bool bf16, hipStream_t st);
hipError_t launch_gemv_gate_up(const GemvArgs& a, hipStream_t st);
hipError_t launch_gemv_down(const GemvArgs& a, bool combine, hipStream_t st);
hipError_t launch_gemm_gate_up(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_down(const GemmArgs& a, hipStream_t st);
hipError_t launch_zero_words(uint32_t* p, int n, hipStream_t st);

// ---- host helpers shared by the entry points (moe_api.hip) ----
int check_device();               // MOE_OK on a gfx950, else MOE_ENOTSUP
int launch_status(hipError_t e);  // MOE_ELAUNCH (error cleared) unless success

// ---- the operators around the layer (argument checks in ops_api.hip) ----

// 4-bit linear (w4.hip).
struct W4Args {
  const uint8_t* q;        // [N][K/2]
  const void* scale;       // FP4: u8 [N][K/32]; INT4: bf16 [N][n_groups]
  const uint8_t* zero;     // INT4: [N][n_groups] or null (8)
  const uint16_t* x;
  void* y;
  int64_t x_stride, y_stride;
  int T, N, K, n_groups, group_shift;
  bool int4, y_bf16;
};
hipError_t launch_w4(const W4Args& a, hipStream_t st);

// Low-rank adapters beside a linear (lora.hip).
struct LoraArgs {
  const uint16_t *a, *b;   // [n][R][K], [n][N][R]
  const int32_t* rank;     // or null (R)
  const float* scale;      // or null (1)
  const uint16_t* x;
  const int32_t* of;
  const void* base;        // or null
  void* y;
  float* h;                // [parts][T][R] partial sums of a x
  uint16_t* op;            // many tokens: [T][3][R] their sum times the scale, in three parts
  uint32_t* status;
  int64_t x_stride, base_stride, y_stride;
  int T, K, N, R, n;
  int parts, part_cols;    // parts of the columns of x
  int h_slots, h_groups;   // set by the launcher
  bool y_bf16, in_place;
  bool many;               // tokens enough that a tile's adapters are taken in turn
};
hipError_t launch_lora(const LoraArgs& a, hipStream_t st);

// Residual's addition and root-mean-square norm (norm.hip).
struct NormArgs {
  const uint16_t* x;
  const void* res;         // null: none
  void* res_out;
  const uint16_t* w;       // null: 1
  uint16_t* y;
  uint8_t* q;
  float* qs;
  int64_t x_stride, res_stride;
  float eps;
  int T, H;
  bool res_f32;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);

// Rules on logits (logits.hip).
struct LogitsArgs {
  const void* z;
  void* out;
  int64_t z_stride, out_stride;
  int T, V;
  const int32_t *history, *seq_of, *n_tokens, *n_prompt;
  int64_t history_stride;
  int max_history, n_seqs;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_ids;
  const float* bias;
  int n_bias, n_masks;
  const uint32_t* mask;
  int64_t mask_stride;
  const int32_t* mask_of;
  uint32_t* status;
  bool z_bf16, out_bf16, in_place;
};
hipError_t launch_logits(const LogitsArgs& a, hipStream_t st);

// What a key/value cache holds: bf16, E4M3 with a scale a row, E2M1 with a scale per 32
// columns.
constexpr int kKvBf16 = 0, kKvE4M3 = 1, kKvE2M1 = 2;

// Paged cache append with rotation (kv.hip).
struct KvAppendArgs {
  void *kc, *vc, *ks, *vs;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride;
  const float* rope;
  const int32_t *seq_of, *pos, *table;
  uint32_t* status;
  int T, Hq, Hkv, D, R, rope_rows, n_seqs, table_cols, n_pages, page_shift;
  int iters;               // set by the launcher: head groups per block
  int kv;                  // kKv*
  bool pairs;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st);

// Token log probabilities (logprobs.hip): W waves of kLogprobChunk elements a row.
constexpr int kLogprobChunk = 2048;
struct LogprobArgs {
  const void* z;
  int64_t row_stride;
  int T, V, W, n_top;
  bool by_row;                  // one block per row: no partials
  const int32_t* tokens;
  float *logprob, *entropy, *top_logprobs;
  int32_t* top_ids;
  uint32_t* status;
  float *pm, *pl, *ps;          // [T][W] partials
  unsigned long long* pk;       // [T][n_top][W] candidate keys
};
hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t st);

// Shared-prefix attention (attn.hip).
constexpr int kAttnTile = 3;
struct AttnArgs {
  const void *k, *v, *ks, *vs;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t *pos, *prefix_pages, *table;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  float* po;                    // [part][n_tok][Hq][D] unnormalised sums
  float2* pml;                  // [part][n_tok][Hq] maximum (log2 units), weight
  float scale_log2;             // scale * log2(e)
  int B, Q, n_tok, Hq, Hkv, G, D;
  int table_cols, n_pages, page_shift, prefix_len, max_keys;
  int kv;                       // kKv*
  // split of the prefix's items and of the sequences' own: kind (1, 2: blocks of
  // 16 x kind rows, keys straight to registers; kAttnTile: of 256 rows, 128 at 256
  // columns, keys through LDS), row blocks, keys per part, parts
  int prefix_kind, prefix_blocks, prefix_chunk, n_prefix_parts;
  int own_kind, own_blocks, own_chunk, n_own_parts;
};
hipError_t launch_attn(const AttnArgs& a, hipStream_t st);

}  // namespace bef
