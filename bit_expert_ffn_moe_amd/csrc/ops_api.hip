// ops_api.hip -- host side of the decode-step operators declared in
// include/moe.h: argument checks, workspace layout and how long axes are split.
// Nothing here allocates, frees or synchronises; every entry point checks
// all its arguments before it enqueues anything.
#include <math.h>
#include <string.h>

#include "kernels.h"
#include "moe.h"

using namespace bef;
namespace {

constexpr int kMaxT = 1 << 18;

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
int ceil_div(int a, int b) { return (int)(((int64_t)a + b - 1) / b); }

int check_cache(const kv_cache* c) {
  if (!c || !c->k || !c->v) return MOE_EINVAL;
  if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_FP8_E4M3) return MOE_EINVAL;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->page_size < 1) return MOE_EINVAL;
  if (c->page_size & (c->page_size - 1)) return MOE_EINVAL;
  if (c->page_size < 16 || c->page_size > 1024 || c->n_kv_heads > 1024) return MOE_ENOTSUP;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ENOTSUP;
  const bool fp8 = c->dtype == MOE_DT_FP8_E4M3;
  if (fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr)) return MOE_EINVAL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16))
    return MOE_EALIGN;
  return MOE_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// A row of n elements per token, rows `stride` apart.
int check_rows(int64_t stride, int64_t n) {
  return stride < n || stride % 8 != 0 || stride > ((int64_t)1 << 40) ? MOE_EINVAL : MOE_OK;
}

}  // namespace

// ---- attention: how the work is split ---------------------------------------
namespace {

// How `rows` query rows of a kv head are taken (see AttnArgs).  Measured at 128
// columns over 8192 shared keys: blocks of 16 rows up to 64 (32 rows: 16.0 us, 18.9 in
// blocks of 32), of 32 rows up to 128 (128 rows: 23.7 us, 29.0 in blocks of 16, whose
// repeated reads of K and V L2 then bounds), keys through LDS above (512 rows over
// 32768 keys: 114 us, 189 in blocks of 32).
void split_rows(int rows, int D, int* kind, int* blocks) {
  if (rows <= 128) {
    *kind = rows <= 64 || D == 256 ? 1 : 2;
    *blocks = ceil_div(rows, 16 * *kind);
  } else {
    *kind = kAttnTile;
    *blocks = ceil_div(rows, D == 256 ? 128 : 256);
  }
}

// Keys per part (a multiple of 128) and parts, for about `want` blocks.  A part has
// 256 keys at least (its sums are written and read again), or 128 where the chip
// would not even get a block per CU.
void split_keys(int keys, int kind, int base_blocks, int want, int* chunk, int* parts) {
  *chunk = 128, *parts = 0;
  if (keys <= 0) return;
  if (base_blocks < 1) base_blocks = 1;
  const int least =
      kind != kAttnTile && keys <= 4096 && (int64_t)base_blocks * ceil_div(keys, 256) < 256 ? 128 : 256;
  const int most = ceil_div(keys, least);
  int p = want / base_blocks;
  p = p < 1 ? 1 : p > most ? most : p;
  *chunk = ceil_div(ceil_div(keys, p), 128) * 128;
  *parts = ceil_div(keys, *chunk);
}

// Everything that follows from the shapes; MOE_OK or why not.
int attn_plan(const kv_cache* c, int n_seqs, int q_len, int n_q_heads, int prefix_len,
              int max_keys, AttnArgs* a) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (n_seqs < 0 || q_len < 1 || n_q_heads < 1 || n_q_heads % c->n_kv_heads) return MOE_EINVAL;
  if (prefix_len < 0 || max_keys < 1 || prefix_len > max_keys) return MOE_EINVAL;
  if (n_q_heads > 1024 || (int64_t)n_seqs * q_len > kMaxT ||
      (int64_t)n_seqs * q_len * n_q_heads >= (1 << 24) || max_keys > (1 << 28))
    return MOE_ENOTSUP;
  // (a launch has at most a block of 256 threads per row, or about `want` below: with 2^24
  // rows that would be more threads than a grid holds)
  memset(a, 0, sizeof *a);
  a->B = n_seqs, a->Q = q_len, a->n_tok = n_seqs * q_len;
  a->Hq = n_q_heads, a->Hkv = c->n_kv_heads, a->G = n_q_heads / c->n_kv_heads, a->D = c->head_dim;
  a->n_pages = c->n_pages, a->page_shift = log2_of(c->page_size);
  a->prefix_len = prefix_len, a->max_keys = max_keys;
  a->fp8 = c->dtype == MOE_DT_FP8_E4M3;
  split_rows(a->n_tok * a->G, a->D, &a->prefix_kind, &a->prefix_blocks);
  split_rows(q_len * a->G, a->D, &a->own_kind, &a->own_blocks);
  const int base_p = a->Hkv * a->prefix_blocks;
  // blocks wanted: a prefix one per CU, all together four per CU (half of each at
  // 256 columns, whose blocks take twice the registers)
  const int want_p = a->D == 256 ? 128 : 256, want = 4 * want_p;
  split_keys(prefix_len, a->prefix_kind, base_p,
             a->prefix_kind == kAttnTile ? 256 : want_p, &a->prefix_chunk, &a->n_prefix_parts);
  const int taken = a->prefix_kind != kAttnTile && a->own_kind != kAttnTile
                        ? base_p * a->n_prefix_parts
                        : 0;
  split_keys(max_keys > prefix_len ? max_keys - (prefix_len & ~31) : 0, a->own_kind,
             a->B * a->Hkv * a->own_blocks, want - taken < want_p ? want_p : want - taken,
             &a->own_chunk, &a->n_own_parts);
  return MOE_OK;
}

size_t attn_ml_bytes(const AttnArgs& a) {
  return up256((size_t)(a.n_prefix_parts + a.n_own_parts) * a.n_tok * a.Hq * 8);
}
size_t attn_bytes(const AttnArgs& a) {
  return attn_ml_bytes(a) +
         up256((size_t)(a.n_prefix_parts + a.n_own_parts) * a.n_tok * a.Hq * a.D * 4);
}

// rows from which a block walks each row (rows of 50021 bf16 with their best: 256 rows 14.2
// us so, 13.2 with a wave per chunk and a join; 512 rows 17.8 either way; 768 rows 21.3 and
// 22.1)
constexpr int kLogprobRows = 512;

struct LogprobLayout {
  int W;
  bool by_row;
  size_t pm, pl, ps, pk, total;
};

// The largest offset of a row's first element in its 16-byte word is 7
// elements (bf16): W covers V + 7.
LogprobLayout logprob_layout(int T, int V, int n_top) {
  LogprobLayout L;
  L.W = ceil_div(V + 7, kLogprobChunk);
  // two rows per CU keep a block per row busy; without partials nothing is needed, but
  // a workspace has a size
  L.by_row = T >= kLogprobRows;
  const size_t n = L.by_row ? 1 : (size_t)T * L.W;
  L.pm = 0;
  L.pl = L.pm + up256(n * 4);
  L.ps = L.pl + up256(n * 4);
  L.pk = L.ps + up256(n * 4);
  L.total = L.pk + up256(n * n_top * 8);
  return L;
}

int check_logprobs(int T, int V, int n_top) {
  if (T < 0 || V < 1 || n_top < 0 || n_top > V) return MOE_EINVAL;
  if (T > kMaxT || V > (1 << 24) || n_top > 64) return MOE_ENOTSUP;
  return MOE_OK;
}

}  // namespace

extern "C" {

int w4_linear(const w4_weights* w, const uint16_t* x, int64_t x_stride, int32_t T, void* y,
              int64_t y_stride, int32_t y_dtype, void* stream) {
  if (!w || !w->q || !w->scale || !x || !y) return MOE_EINVAL;
  const bool int4 = w->format == MOE_W_INT4_BF16_GROUP;
  if (!int4 && w->format != MOE_W_FP4_E2M1_UE8M0_K32) return MOE_ENOTSUP;
  if (y_dtype != MOE_DT_BF16 && y_dtype != MOE_DT_F32) return MOE_EINVAL;
  if (T < 0 || w->n_out < 1 || w->n_in < 32 || w->n_in % 32) return MOE_EINVAL;
  if (int4 ? w->group != 32 && w->group != 64 && w->group != 128
           : w->group != 32 || w->zero != nullptr)
    return MOE_EINVAL;
  if (check_rows(x_stride, w->n_in) || y_stride < w->n_out || y_stride > ((int64_t)1 << 40))
    return MOE_EINVAL;
  if (T > kMaxT || w->n_out > (1 << 20) || w->n_in > (1 << 20)) return MOE_ENOTSUP;
  if (!aligned(w->q, 16) || !aligned(w->scale, 16) || !aligned(w->zero, 16) || !aligned(x, 16) ||
      !aligned(y, 16))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  int rc = check_device();
  if (rc) return rc;
  W4Args a;
  memset(&a, 0, sizeof a);
  a.q = (const uint8_t*)w->q, a.scale = w->scale, a.zero = (const uint8_t*)w->zero;
  a.x = x, a.y = y, a.x_stride = x_stride, a.y_stride = y_stride;
  a.T = T, a.N = w->n_out, a.K = w->n_in;
  a.n_groups = ceil_div(w->n_in, w->group), a.group_shift = log2_of(w->group);
  a.int4 = int4, a.y_bf16 = y_dtype == MOE_DT_BF16;
  return launch_status(launch_w4(a, (hipStream_t)stream));
}

int kv_append_rope(const kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                   const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                   int32_t T, const float* rope, int32_t rope_rows, int32_t rope_dim,
                   int32_t rope_style, const int32_t* seq_of, const int32_t* pos,
                   const int32_t* page_table, int32_t n_seqs, int32_t table_cols, uint16_t* q_out,
                   uint32_t* status, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (!k || !v || !seq_of || !pos || !page_table) return MOE_EINVAL;
  if (T < 0 || n_q_heads < 0 || n_seqs < 1 || table_cols < 1) return MOE_EINVAL;
  if ((n_q_heads > 0) != (q != nullptr) || (n_q_heads > 0) != (q_out != nullptr))
    return MOE_EINVAL;
  if (rope_dim < 0 || rope_dim > cache->head_dim || rope_dim % 16) return MOE_EINVAL;
  if (rope_dim ? !rope || rope_rows < 1 || (rope_style != MOE_ROPE_HALF &&
                                            rope_style != MOE_ROPE_PAIRS)
               : rope != nullptr)
    return MOE_EINVAL;
  const int64_t D = cache->head_dim;
  if (n_q_heads && check_rows(q_stride, n_q_heads * D)) return MOE_EINVAL;
  if (check_rows(k_stride, cache->n_kv_heads * D) || check_rows(v_stride, cache->n_kv_heads * D))
    return MOE_EINVAL;
  if (T > kMaxT || n_q_heads > 1024) return MOE_ENOTSUP;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(rope, 16) || !aligned(seq_of, 4) || !aligned(pos, 4) || !aligned(page_table, 4) ||
      !aligned(status, 4))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  rc = check_device();
  if (rc) return rc;
  KvAppendArgs a;
  memset(&a, 0, sizeof a);
  a.kc = cache->k, a.vc = cache->v, a.ks = cache->k_scale, a.vs = cache->v_scale;
  a.q = q, a.k = k, a.v = v, a.q_out = q_out;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.rope = rope, a.seq_of = seq_of, a.pos = pos, a.table = page_table, a.status = status;
  a.T = T, a.Hq = n_q_heads, a.Hkv = cache->n_kv_heads, a.D = cache->head_dim, a.R = rope_dim;
  a.rope_rows = rope_rows, a.n_seqs = n_seqs, a.table_cols = table_cols;
  a.n_pages = cache->n_pages, a.page_shift = log2_of(cache->page_size);
  a.fp8 = cache->dtype == MOE_DT_FP8_E4M3, a.pairs = rope_style == MOE_ROPE_PAIRS;
  return launch_status(launch_kv_append(a, (hipStream_t)stream));
}

size_t attn_workspace_bytes(const kv_cache* cache, int32_t n_seqs, int32_t q_len,
                            int32_t n_q_heads, int32_t prefix_len, int32_t max_keys) {
  AttnArgs a;
  if (n_seqs < 1 || attn_plan(cache, n_seqs, q_len, n_q_heads, prefix_len, max_keys, &a)) return 0;
  return attn_bytes(a);
}

int attn_shared_prefix(const kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t n_seqs,
                       int32_t q_len, int32_t n_q_heads, const int32_t* pos,
                       const int32_t* prefix_pages, int32_t prefix_len, const int32_t* page_table,
                       int32_t table_cols, int32_t max_keys, float scale, uint16_t* out,
                       float* lse, uint32_t* status, void* ws, size_t ws_bytes, void* stream) {
  AttnArgs a;
  int rc = attn_plan(cache, n_seqs, q_len, n_q_heads, prefix_len, max_keys, &a);
  if (rc) return rc;
  if (!q || !pos || !out) return MOE_EINVAL;
  if (prefix_len > 0 && !prefix_pages) return MOE_EINVAL;
  if (max_keys > prefix_len &&
      (!page_table || table_cols < 1 || (int64_t)table_cols * cache->page_size < max_keys))
    return MOE_EINVAL;
  if (check_rows(q_stride, (int64_t)n_q_heads * cache->head_dim)) return MOE_EINVAL;
  if (!(scale > 0.0f) || !isfinite(scale)) return MOE_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 16) || !aligned(pos, 4) ||
      !aligned(prefix_pages, 4) || !aligned(page_table, 4) || !aligned(status, 4))
    return MOE_EALIGN;
  if (n_seqs == 0) return MOE_OK;
  if (!ws) return MOE_EINVAL;
  if (!aligned(ws, 256)) return MOE_EALIGN;
  if (ws_bytes < attn_bytes(a)) return MOE_EWORKSPACE;
  rc = check_device();
  if (rc) return rc;
  a.k = cache->k, a.v = cache->v, a.ks = cache->k_scale, a.vs = cache->v_scale;
  a.q = q, a.q_stride = q_stride, a.pos = pos, a.prefix_pages = prefix_pages;
  a.table = page_table, a.table_cols = table_cols;
  a.out = out, a.lse = lse, a.status = status;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.pml = (float2*)ws;
  a.po = (float*)((uint8_t*)ws + attn_ml_bytes(a));
  return launch_status(launch_attn(a, (hipStream_t)stream));
}

size_t token_logprobs_workspace_bytes(int32_t T, int32_t V, int32_t n_top) {
  if (T < 1 || check_logprobs(T, V, n_top)) return 0;
  return logprob_layout(T, V, n_top).total;
}

int token_logprobs(const void* z, int32_t z_dtype, int64_t row_stride, int32_t T, int32_t V,
                   const int32_t* tokens, int32_t n_top, float* logprob, float* entropy,
                   int32_t* top_ids, float* top_logprobs, uint32_t* status, void* ws,
                   size_t ws_bytes, void* stream) {
  if (!z || (z_dtype != MOE_DT_BF16 && z_dtype != MOE_DT_F32)) return MOE_EINVAL;
  int rc = check_logprobs(T, V, n_top);
  if (rc) return rc;
  if (row_stride < V || row_stride > ((int64_t)1 << 40)) return MOE_EINVAL;
  if ((tokens != nullptr) != (logprob != nullptr)) return MOE_EINVAL;
  if (n_top > 0 && (!top_ids || !top_logprobs)) return MOE_EINVAL;
  if (!aligned(z, 16) || !aligned(logprob, 16) || !aligned(entropy, 16) || !aligned(top_ids, 4) ||
      !aligned(top_logprobs, 16) || !aligned(tokens, 4) || !aligned(status, 4))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const LogprobLayout L = logprob_layout(T, V, n_top);
  if (!ws) return MOE_EINVAL;
  if (!aligned(ws, 256)) return MOE_EALIGN;
  if (ws_bytes < L.total) return MOE_EWORKSPACE;
  rc = check_device();
  if (rc) return rc;
  LogprobArgs a;
  memset(&a, 0, sizeof a);
  a.z = z, a.row_stride = row_stride, a.T = T, a.V = V, a.W = L.W, a.n_top = n_top;
  a.by_row = L.by_row;
  a.tokens = tokens, a.logprob = logprob, a.entropy = entropy;
  a.top_ids = top_ids, a.top_logprobs = top_logprobs, a.status = status;
  uint8_t* p = (uint8_t*)ws;
  a.pm = (float*)(p + L.pm), a.pl = (float*)(p + L.pl), a.ps = (float*)(p + L.ps);
  a.pk = (unsigned long long*)(p + L.pk);
  return launch_status(launch_logprobs(a, z_dtype == MOE_DT_BF16, (hipStream_t)stream));
}

}  // extern "C"
