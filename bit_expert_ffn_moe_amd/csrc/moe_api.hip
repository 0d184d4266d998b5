// moe_api.hip -- host side of the C ABI declared in include/moe.h:
// argument validation, workspace carving and launch sequencing.  Nothing here
// allocates, frees or synchronises (except the two debug helpers, which say
// so); every entry point validates first and enqueues only on success.
#include <string.h>

#include <atomic>
#include <mutex>

#include "common.h"
#include "kernels.h"
#include "moe.h"

namespace bef {

KernelTimer g_kernel_timer[6];
// the one-token FP4 path: the fused expert kernel where it fits when set
// (measured slower than the separate kernels: off by default)
std::atomic<int> g_decode_fused{0};
HSink g_h_sink;

__global__ void zero_words_kernel(uint32_t* p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0u;
}

hipError_t launch_zero_words(uint32_t* p, int n, hipStream_t st) {
  zero_words_kernel<<<(n + 255) / 256, 256, 0, st>>>(p, n);
  return hipGetLastError();
}

// A plain streaming read (the practical HBM ceiling the kernels are compared
// with): 16-byte loads, four independent ones in flight per lane, grid-stride
// over n16 16-byte words; the XOR of everything read decides a store that
// never happens in practice, so the loads cannot be dropped.
__global__ __launch_bounds__(512) void stream_read_kernel(const uint4* __restrict__ p, size_t n16,
                                                          uint32_t* sink) {
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  uint32_t acc = 0;
  for (; i + 3 * stride < n16; i += 4 * stride) {
    const uint4 a = p[i], b = p[i + stride], c = p[i + 2 * stride], d = p[i + 3 * stride];
    acc ^= a.x ^ a.y ^ a.z ^ a.w ^ b.x ^ b.y ^ b.z ^ b.w ^ c.x ^ c.y ^ c.z ^ c.w ^ d.x ^ d.y ^
           d.z ^ d.w;
  }
  for (; i < n16; i += stride) {
    const uint4 a = p[i];
    acc ^= a.x ^ a.y ^ a.z ^ a.w;
  }
  if (acc == 0x9E3779B9u) sink[0] = acc;
}

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kCtlBytes = sizeof(WsCtl);
static_assert(sizeof(WsCtl) % 256 == 0, "control block");

size_t up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Workspace layout for one call shape.  Sections are carved in this order so
// that the standalone calls, which know fewer sizes, agree with the whole-
// layer call: control | permute scratch (T, E) | router partials (T, H, E) |
// everything else (needs the weights' shapes).
struct Layout {
  size_t ctl, cnt, gsum, wrT, ids, w, xq, xs, offsets, row_token, row_of, active, h, hq, hs,
      y, total;
  size_t end_permute, end_route, end_ffn;
};

// The VALU GEMV path (weights streamed once per token row from registers,
// no MFMA tile to fill) for a few tokens; the grouped GEMM otherwise.  The
// crossover in T per format is the measured one (small-batch sweep of the
// benchmark at hidden 4096, intermediate 2048, 256 experts top-6).
constexpr int kGemvCrossT[3] = {0, 4, 4};  // by format: FP4, FP8

bool gemv_path(int fmt, int T, int k, int H, int I) {
  return T >= 1 && T <= kGemvMaxT && T <= kGemvCrossT[fmt == MOE_W_FP8_E4M3_F32_B128 ? 2 : 1] &&
         k + 1 <= kGemvMaxRows && T * (k + 1) <= kHSlotRowsHost && H <= 8192 && I <= 4096;
}

Layout layout_for(int E, int H, int I, int T, int k, bool with_h) {
  Layout L;
  const size_t R = (size_t)T * k + T;
  const size_t nblk = ((size_t)T + kPermuteTokBlock - 1) / kPermuteTokBlock;
  size_t o = 0;
  L.ctl = o;
  o += up(kCtlBytes);
  L.cnt = o;
  o += up(nblk * E * 4);
  L.end_permute = o;
  // router group sums for T > kRouteSmallT: [ceil(H/256)][T][E] f32
  L.gsum = o;
  if (T > kRouteSmallT) o += up((size_t)((H / 64 + 3) / 4) * T * E * 4);
  // the router matrix transposed, [E][H] bf16, from kRouteSplitT tokens on
  L.wrT = o;
  if (T >= kRouteSplitT) o += up((size_t)E * H * 2);
  L.end_route = o;
  L.ids = o;
  o += up((size_t)T * k * 4);
  L.w = o;
  o += up((size_t)T * k * 4);
  L.xq = o;
  o += up((size_t)T * H);
  L.xs = o;
  o += up((size_t)T * (H / 128) * 4);
  L.offsets = o;
  o += up((size_t)(E + 2) * 4);
  L.row_token = o;
  o += up(R * 4);
  L.row_of = o;
  o += up((size_t)T * (k + 1) * 4);
  L.active = o;
  o += up((size_t)(E + 1) * 16);
  L.h = o;
  if (with_h) o += up(R * I * 4);
  L.hq = o;
  o += up(R * I);
  L.hs = o;
  o += up(R * (I / 128) * 4);
  L.end_ffn = o;
  L.y = o;
  o += up(R * H * 4);
  L.total = o;
  return L;
}

Layout layout_w(const moe_weights* w, int T, int k) {
  return layout_for(w->n_experts, w->hidden, w->inter, T, k,
                    gemv_path(w->format, T, k, w->hidden, w->inter));
}

// One-time check per device that it is a gfx950 (the only global state).
std::atomic<int> g_arch_ok[64];

}  // namespace

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return MOE_ENOTSUP;
  }
  if (dev < 64) {
    int v = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (v == 1) return MOE_OK;
    if (v == 2) return MOE_ENOTSUP;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ENOTSUP;
  }
  const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < 64) g_arch_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? MOE_OK : MOE_ENOTSUP;
}

int launch_status(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ELAUNCH;
  }
  return MOE_OK;
}

namespace {

// T = 0 is an empty batch: valid, and the entry points return MOE_OK after
// checking their other arguments, reading, writing and launching nothing.
// At most 2^18 tokens per call: the kernels address a token's row of x or xq
// (T x H bytes, H <= 8192) with 32-bit offsets.
constexpr int kMaxTokens = 1 << 18;

int check_tk(int T, int k, int E) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_EINVAL;
  if (E > 256 || k > 16 || T > kMaxTokens) return MOE_ENOTSUP;
  return MOE_OK;
}

int check_hidden(int H) {
  if (H < 128 || H % 128 != 0) return H > 0 && H % 128 == 0 ? MOE_ENOTSUP : MOE_EINVAL;
  if (H > 8192) return MOE_ENOTSUP;
  return MOE_OK;
}

int check_weights(const moe_weights* w) {
  if (!w) return MOE_EINVAL;
  if (w->format != MOE_W_FP4_E2M1_UE8M0_K32 && w->format != MOE_W_FP8_E4M3_F32_B128)
    return MOE_ENOTSUP;
  if (w->n_experts < 1) return MOE_EINVAL;
  if (w->n_experts > 256) return MOE_ENOTSUP;
  int rc = check_hidden(w->hidden);
  if (rc) return rc;
  rc = check_hidden(w->inter);
  if (rc) return rc;
  const void* ps[6] = {w->gate_q, w->gate_s, w->up_q, w->up_s, w->down_q, w->down_s};
  for (const void* p : ps)
    if (!p) return MOE_EINVAL;
  for (const void* p : ps)
    if (!aligned16(p)) return MOE_EALIGN;
  return MOE_OK;
}

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return MOE_EINVAL;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_EALIGN;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  return MOE_OK;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(ws) + off);
}

// ---- enqueue helpers (arguments already validated) -----------------------

GemvArgs gemv_args(const moe_weights* w, int T, int k, const Layout& L, void* ws) {
  GemvArgs a;
  memset(&a, 0, sizeof a);
  a.gq = (const uint8_t*)w->gate_q;
  a.gs = (const uint8_t*)w->gate_s;
  a.uq = (const uint8_t*)w->up_q;
  a.us = (const uint8_t*)w->up_s;
  a.dq = (const uint8_t*)w->down_q;
  a.ds = (const uint8_t*)w->down_s;
  a.E = w->n_experts, a.H = w->hidden, a.I = w->inter, a.k = k;
  a.fmt = w->format, a.T = T;
  a.n_slots = (T * k < w->n_experts ? T * k : w->n_experts) + 1;
  a.h = at<float>(ws, L.h);
  a.hq_ws = at<uint8_t>(ws, L.hq);
  a.hs_ws = at<float>(ws, L.hs);
  a.h_slots = at<WsCtl>(ws, L.ctl)->h_slots;
  a.status = &at<WsCtl>(ws, L.ctl)->status;
  return a;
}

GemmArgs gemm_args(const moe_weights* w, int T, int k, const Layout& L, void* ws) {
  GemmArgs g;
  memset(&g, 0, sizeof g);
  g.fmt = w->format;
  g.gq = (const uint8_t*)w->gate_q;
  g.uq = (const uint8_t*)w->up_q;
  g.dq = (const uint8_t*)w->down_q;
  g.gs = w->gate_s;
  g.us = w->up_s;
  g.ds = w->down_s;
  g.T = T, g.k = k, g.E = w->n_experts, g.H = w->hidden, g.I = w->inter;
  g.hq = at<uint8_t>(ws, L.hq);
  g.hs = at<float>(ws, L.hs);
  const size_t R = (size_t)T * k + T;
  if (g_h_sink.h && g_h_sink.n >= R * (size_t)w->inter) g.h_dbg = g_h_sink.h;
  return g;
}

// S5: gate + up + SwiGLU (+ requantised h in ws).
int enqueue_gate_up(const moe_weights* w, const uint8_t* xq, const float* xs, int T, int k,
                    const int32_t* offsets, const int32_t* row_token, const Layout& L, void* ws,
                    hipStream_t st, const uint8_t* mask = nullptr) {
  if (gemv_path(w->format, T, k, w->hidden, w->inter)) {
    GemvArgs a = gemv_args(w, T, k, L, ws);
    a.xq = xq, a.xs = xs, a.offsets = offsets, a.row_token = row_token;
    a.group_mask = mask;
    return launch_status(launch_gemv_gate_up(a, st));
  }
  GemmArgs g = gemm_args(w, T, k, L, ws);
  g.xq = xq, g.xs = xs, g.offsets = offsets, g.row_token = row_token;
  g.group_mask = mask;
  return launch_status(launch_gemm_gate_up(g, st));
}

// S6 (+ S7 when out is set): down projection of the h left in ws.
int enqueue_down(const moe_weights* w, int T, int k, const int32_t* offsets,
                 const int32_t* row_of, const float* topk_w, float* y_rows, void* out,
                 int out_dtype, const Layout& L, void* ws, hipStream_t st,
                 const uint8_t* mask = nullptr) {
  if (gemv_path(w->format, T, k, w->hidden, w->inter)) {
    GemvArgs a = gemv_args(w, T, k, L, ws);
    a.offsets = offsets, a.row_of = row_of, a.topk_w = topk_w;
    a.y_rows = y_rows, a.out = out, a.out_bf16 = out_dtype == MOE_DT_BF16;
    a.group_mask = mask;
    return launch_status(launch_gemv_down(a, out != nullptr, st));
  }
  GemmArgs g = gemm_args(w, T, k, L, ws);
  g.offsets = offsets, g.y_rows = y_rows;
  g.group_mask = mask;
  int rc = launch_status(launch_gemm_down(g, st));
  if (rc || !out) return rc;
  return launch_status(launch_combine(y_rows, row_of, topk_w, T, k, w->hidden, out,
                                      out_dtype == MOE_DT_BF16, st));
}

}  // namespace
}  // namespace bef

using namespace bef;

extern "C" {

size_t moe_workspace_bytes(const moe_weights* w, int32_t max_tokens, int32_t top_k) {
  if (check_weights(w) != MOE_OK || max_tokens < 1) return 0;
  if (check_tk(max_tokens, top_k, w->n_experts) != MOE_OK) return 0;
  size_t a = layout_w(w, max_tokens, top_k).total;
  size_t b = layout_w(w, 1, top_k).total;
  return a > b ? a : b;
}

int moe_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  int rc = check_ws(ws, ws_bytes, kCtlBytes);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  return launch_status(launch_zero_words((uint32_t*)ws, (int)(kCtlBytes / 4), (hipStream_t)stream));
}

int moe_route(const uint16_t* x, const uint16_t* w_router, int32_t T, int32_t H, int32_t E,
              int32_t k, int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes,
              void* stream) {
  if (!x || !w_router || !topk_ids || !topk_w) return MOE_EINVAL;
  int rc = check_tk(T, k, E);
  if (rc) return rc;
  rc = check_hidden(H);
  if (rc) return rc;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(topk_ids) || !aligned16(topk_w))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const Layout L = layout_for(E, H, 128, T, k, false);
  rc = check_ws(ws, ws_bytes, L.end_route);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  WsCtl* ctl = at<WsCtl>(ws, L.ctl);
  return launch_status(
      launch_route(x, w_router, T, H, E, k, topk_ids, topk_w, ctl, at<float>(ws, L.gsum),
                   at<uint16_t>(ws, L.wrT), (hipStream_t)stream));
}

int act_quant_fp8(const void* x, int32_t x_dtype, int64_t rows, int32_t cols, uint8_t* q,
                  float* scales, void* stream) {
  if (!x || !q || !scales) return MOE_EINVAL;
  if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F32) return MOE_EINVAL;
  if (rows < 0 || cols < 128 || cols % 128 != 0) return MOE_EINVAL;
  if (rows * (int64_t)(cols / 128) * 16 > (int64_t)0x7fffffff * 256) return MOE_ENOTSUP;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales)) return MOE_EALIGN;
  if (rows == 0) return MOE_OK;
  int rc = check_device();
  if (rc) return rc;
  return launch_status(
      launch_act_quant(x, x_dtype == MOE_DT_BF16, rows, cols, q, scales, (hipStream_t)stream));
}

int moe_permute(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E, int32_t* offsets,
                int32_t* row_token, int32_t* row_of, void* ws, size_t ws_bytes, void* stream) {
  if (!topk_ids || !offsets || !row_token || !row_of) return MOE_EINVAL;
  int rc = check_tk(T, k, E);
  if (rc) return rc;
  if (!aligned16(topk_ids) || !aligned16(offsets) || !aligned16(row_token) || !aligned16(row_of))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const Layout L = layout_for(E, 128, 128, T, k, false);
  rc = check_ws(ws, ws_bytes, L.end_permute);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  WsCtl* ctl = at<WsCtl>(ws, L.ctl);
  return launch_status(launch_permute(topk_ids, T, k, E, offsets, row_token, row_of,
                                      at<int32_t>(ws, L.cnt), &ctl->status,
                                      (hipStream_t)stream));
}

int moe_expert_ffn(const moe_weights* w, const uint8_t* xq, const float* xs, int32_t T, int32_t k,
                   const int32_t* offsets, const int32_t* row_token, float* y_rows, void* ws,
                   size_t ws_bytes, void* stream) {
  int rc = check_weights(w);
  if (rc) return rc;
  if (!xq || !xs || !offsets || !row_token || !y_rows) return MOE_EINVAL;
  rc = check_tk(T, k, w->n_experts);
  if (rc) return rc;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(offsets) || !aligned16(row_token) ||
      !aligned16(y_rows))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const Layout L = layout_w(w, T, k);
  rc = check_ws(ws, ws_bytes, L.end_ffn);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  rc = enqueue_gate_up(w, xq, xs, T, k, offsets, row_token, L, ws, (hipStream_t)stream);
  if (rc) return rc;
  return enqueue_down(w, T, k, offsets, nullptr, nullptr, y_rows, nullptr, 0, L, ws,
                      (hipStream_t)stream);
}

int moe_expert_gate_up(const moe_weights* w, const uint8_t* xq, const float* xs, int32_t T,
                       int32_t k, const int32_t* offsets, const int32_t* row_token, void* ws,
                       size_t ws_bytes, void* stream) {
  int rc = check_weights(w);
  if (rc) return rc;
  if (!xq || !xs || !offsets || !row_token) return MOE_EINVAL;
  rc = check_tk(T, k, w->n_experts);
  if (rc) return rc;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(offsets) || !aligned16(row_token))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const Layout L = layout_w(w, T, k);
  rc = check_ws(ws, ws_bytes, L.end_ffn);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  return enqueue_gate_up(w, xq, xs, T, k, offsets, row_token, L, ws, (hipStream_t)stream);
}

int moe_expert_down(const moe_weights* w, int32_t T, int32_t k, const int32_t* offsets,
                    const int32_t* row_of, const float* topk_w, float* y_rows, void* out,
                    int32_t out_dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_weights(w);
  if (rc) return rc;
  if (!offsets) return MOE_EINVAL;
  rc = check_tk(T, k, w->n_experts);
  if (rc) return rc;
  const bool gv = gemv_path(w->format, T, k, w->hidden, w->inter);
  if (out) {
    if (!row_of || !topk_w) return MOE_EINVAL;
    if (out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F32) return MOE_EINVAL;
    if (!aligned16(out) || !aligned16(row_of) || !aligned16(topk_w)) return MOE_EALIGN;
  }
  if (!y_rows && !(gv && out)) return MOE_EINVAL;
  if (!aligned16(offsets) || (y_rows && !aligned16(y_rows))) return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const Layout L = layout_w(w, T, k);
  rc = check_ws(ws, ws_bytes, L.end_ffn);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  return enqueue_down(w, T, k, offsets, row_of, topk_w, y_rows, out, out_dtype, L, ws,
                      (hipStream_t)stream);
}

int moe_combine(const float* y_rows, const int32_t* row_of, const float* topk_w, int32_t T,
                int32_t k, int32_t H, void* out, int32_t out_dtype, void* stream) {
  if (!y_rows || !row_of || !topk_w || !out) return MOE_EINVAL;
  if (T < 0 || k < 1) return MOE_EINVAL;
  if (k > 16 || T > kMaxTokens) return MOE_ENOTSUP;
  int rc = check_hidden(H);
  if (rc) return rc;
  if (out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F32) return MOE_EINVAL;
  if (!aligned16(y_rows) || !aligned16(row_of) || !aligned16(topk_w) || !aligned16(out))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  rc = check_device();
  if (rc) return rc;
  return launch_status(
      launch_combine(y_rows, row_of, topk_w, T, k, H, out, out_dtype == MOE_DT_BF16,
                     (hipStream_t)stream));
}

}  // extern "C"

namespace bef {
namespace {

// Arguments of the whole-layer call other than the workspace.
int check_forward_args(const moe_weights* w, const uint16_t* w_router, const uint16_t* x,
                       int32_t T, int32_t k, const int32_t* routing_ids, const float* routing_w,
                       const void* out, int32_t out_dtype) {
  int rc = check_weights(w);
  if (rc) return rc;
  if (!x || !out) return MOE_EINVAL;
  if ((routing_ids == nullptr) != (routing_w == nullptr)) return MOE_EINVAL;
  if (!routing_ids && !w_router) return MOE_EINVAL;
  if (out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F32) return MOE_EINVAL;
  rc = check_tk(T, k, w->n_experts);
  if (rc) return rc;
  if (!aligned16(x) || !aligned16(out) || (w_router && !aligned16(w_router)) ||
      (routing_ids && (!aligned16(routing_ids) || !aligned16(routing_w))))
    return MOE_EALIGN;
  return MOE_OK;
}

// The whole layer, arguments already checked, T >= 1, ws large enough.
int enqueue_forward(const moe_weights* w, const uint16_t* w_router, const uint16_t* x, int32_t T,
                    int32_t k, const int32_t* routing_ids, const float* routing_w, void* out,
                    int32_t out_dtype, void* ws, hipStream_t st) {
  int rc = MOE_OK;
  const Layout L = layout_w(w, T, k);
  const int E = w->n_experts, H = w->hidden;
  WsCtl* ctl = at<WsCtl>(ws, L.ctl);
  const int32_t* ids = routing_ids;
  const float* tw = routing_w;
  uint8_t* xq = at<uint8_t>(ws, L.xq);
  float* xs = at<float>(ws, L.xs);
  int32_t* offsets = at<int32_t>(ws, L.offsets);
  int32_t* row_token = at<int32_t>(ws, L.row_token);
  int32_t* row_of = at<int32_t>(ws, L.row_of);
  if (!ids && T <= kRouteSmallT) {
    FrontArgs fa = {};
    fa.x = x, fa.wr = w_router, fa.T = T, fa.H = H, fa.E = E, fa.k = k;
    set_route_sync(fa, ctl);
    fa.ids = at<int32_t>(ws, L.ids), fa.w = at<float>(ws, L.w);
    fa.offsets = offsets, fa.row_token = row_token, fa.row_of = row_of;
    if (gemv_path(w->format, T, k, H, w->inter)) {
      // decided before anything is enqueued: the fused expert kernel's shape
      // conditions (it refuses nothing that passes them)
      const bool fused =
          g_decode_fused.load() && decode_ffn_fits(w->format, T, k, H, w->inter);
      // one token on the VALU path: the front kernel also quantises x, runs
      // the shared expert's gate+up (its waves quantise x themselves, same
      // rule) and lists the routed groups for the gate+up kernel
      fa.fmt = w->format;
      fa.sh_gq = (const uint8_t*)w->gate_q;  // the kernel reads group E (the shared expert)
      fa.sh_uq = (const uint8_t*)w->up_q;
      fa.sh_gs = (const uint8_t*)w->gate_s;
      fa.sh_us = (const uint8_t*)w->up_s;
      fa.I = w->inter;
      fa.sh_h = at<float>(ws, L.h);
      fa.sh_hq = at<uint8_t>(ws, L.hq);
      fa.sh_hs = at<float>(ws, L.hs);
      fa.h_slots = ctl->h_slots;
      fa.active = at<int4>(ws, L.active);
      fa.n_active_slots = (T * k < E ? T * k : E);
      fa.xq = xq, fa.xs = xs;  // act_quant blocks run in the same kernel
      rc = launch_status(launch_route_front(fa, st));
      if (rc) return rc;
      GemvArgs a = gemv_args(w, T, k, L, ws);
      a.xq = xq, a.xs = xs, a.offsets = offsets, a.row_token = row_token;
      a.active = at<int4>(ws, L.active);
      a.n_slots = fa.n_active_slots;
      if (fused) {
        // routed gate+up, down of all k + 1 rows and the combine, one launch
        DecodeArgs d;
        memset(&d, 0, sizeof d);
        d.gq = a.gq, d.gs = a.gs, d.uq = a.uq, d.us = a.us, d.dq = a.dq, d.ds = a.ds;
        d.xq = xq, d.xs = xs, d.active = a.active, d.row_of = row_of, d.topk_w = fa.w;
        d.E = E, d.H = H, d.I = w->inter, d.k = k;
        d.h = a.h, d.hq = a.hq_ws, d.hs = a.hs_ws;
        d.dec_h = ctl->dec_h, d.dec_c = ctl->dec_c;
        d.epoch = &ctl->dec_epoch, d.done = &ctl->dec_done, d.status = &ctl->status;
        d.cnt = ctl->dec_cnt;
        d.out = out, d.out_bf16 = out_dtype == MOE_DT_BF16;
        return launch_status(launch_decode_ffn(d, st));
      }
      rc = launch_status(launch_gemv_gate_up(a, st));
      if (rc) return rc;
      // down + combine, the rows' groups from the same active list
      a.row_of = row_of, a.topk_w = fa.w, a.n_rows = T * k + T;
      a.out = out, a.out_bf16 = out_dtype == MOE_DT_BF16;
      return launch_status(launch_gemv_down(a, true, st));
    }
    // router + act_quant + permute in one kernel
    fa.xq = xq, fa.xs = xs;
    rc = launch_status(launch_route_front(fa, st));
    if (rc) return rc;
    rc = enqueue_gate_up(w, xq, xs, T, k, offsets, row_token, L, ws, st);
    if (rc) return rc;
    return enqueue_down(w, T, k, offsets, row_of, fa.w, at<float>(ws, L.y), out, out_dtype, L,
                        ws, st);
  }
  if (!ids) {
    // router, with the act_quant of x in the same launch
    int32_t* ids_ws = at<int32_t>(ws, L.ids);
    float* w_ws = at<float>(ws, L.w);
    rc = launch_status(launch_route(x, w_router, T, H, E, k, ids_ws, w_ws, ctl,
                                    at<float>(ws, L.gsum), at<uint16_t>(ws, L.wrT), st, xq, xs));
    if (rc) return rc;
    ids = ids_ws;
    tw = w_ws;
  } else {
    rc = launch_status(launch_act_quant(x, true, T, H, xq, xs, st));
    if (rc) return rc;
  }
  rc = launch_status(launch_permute(ids, T, k, E, offsets, row_token, row_of,
                                    at<int32_t>(ws, L.cnt), &ctl->status, st));
  if (rc) return rc;
  rc = enqueue_gate_up(w, xq, xs, T, k, offsets, row_token, L, ws, st);
  if (rc) return rc;
  return enqueue_down(w, T, k, offsets, row_of, tw, at<float>(ws, L.y), out, out_dtype, L, ws,
                      st);
}

// ---- the allocation-free forward: a file-scope device array as workspace --

// At most this much workspace per call: the one-token and small-batch
// shapes (at hidden 4096, intermediate 2048, top-6, about 100 tokens).
constexpr size_t kStaticScratchBytes = (size_t)16 << 20;
static_assert(kStaticScratchBytes == MOE_NOALLOC_SCRATCH_BYTES, "moe.h limit");

// In host code `scratch` names a host-side stand-in, not the device array:
// its device address on each GPU comes from hipGetSymbolAddress, once per
// device, and only that address is ever handed to a kernel.
__device__ __align__(256) uint8_t scratch[kStaticScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_dev[64];

// Device address of this device's `scratch`, looked up (with the device
// current) on its first use, when its control block is also cleared by a
// fill kernel on `st` (the kernels keep it zero from then on).
int static_scratch(void** ptr, hipStream_t st) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
    (void)hipGetLastError();
    return MOE_ENOTSUP;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_dev[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) {
      (void)hipGetLastError();
      return MOE_ELAUNCH;
    }
    int rc = launch_status(launch_zero_words((uint32_t*)p, (int)(kCtlBytes / 4), st));
    if (rc) return rc;
    g_scratch_dev[dev] = p;
  }
  *ptr = g_scratch_dev[dev];
  return MOE_OK;
}

// ---- host-resident experts: an LRU cache of expert slots in HBM ----------

// Bytes of one expert's matrix (codes, scales) in either format.
struct MatBytes {
  size_t gq, gs, dq, ds;
};
MatBytes mat_bytes(const moe_weights* w) {
  const size_t H = (size_t)w->hidden, I = (size_t)w->inter;
  if (w->format == MOE_W_FP4_E2M1_UE8M0_K32) return {I * H / 2, I * H / 32, H * I / 2, H * I / 32};
  return {I * H, (I / 128) * (H / 128) * 4, H * I, (H / 128) * (I / 128) * 4};
}

// The call's own layout: sized for the routed-expert count E of the router
// (the slot space has at most E groups), plus its slot ids and group masks.
struct HostLayout {
  Layout L;
  size_t slot_ids, masks, total;
};
HostLayout host_layout(const moe_weights* host_w, int T, int k) {
  HostLayout h;
  const int E = host_w->n_experts;
  h.L = layout_for(E, host_w->hidden, host_w->inter, T, k,
                   gemv_path(host_w->format, T, k, host_w->hidden, host_w->inter));
  h.slot_ids = h.L.total;
  h.masks = h.slot_ids + up((size_t)T * k * 4);
  h.total = h.masks + up((size_t)2 * (E + 1));
  return h;
}
// Pinned host scratch: ids read back [T][k], slot ids [T][k], masks [2][E+1].
size_t host_scratch_need(int E, int T, int k) {
  return up((size_t)T * k * 4) * 2 + up((size_t)2 * (E + 1));
}

// Enqueue the copy of expert e's six arrays (host_w) into slot s (slot_w).
int copy_expert(const moe_weights* host_w, const moe_weights* slot_w, int e, int s,
                hipStream_t cs, uint64_t* bytes) {
  const MatBytes b = mat_bytes(host_w);
  const void* src[6] = {host_w->gate_q, host_w->gate_s, host_w->up_q,
                        host_w->up_s,   host_w->down_q, host_w->down_s};
  const void* dst[6] = {slot_w->gate_q, slot_w->gate_s, slot_w->up_q,
                        slot_w->up_s,   slot_w->down_q, slot_w->down_s};
  const size_t n[6] = {b.gq, b.gs, b.gq, b.gs, b.dq, b.ds};
  for (int i = 0; i < 6; ++i) {
    if (hipMemcpyAsync((uint8_t*)dst[i] + (size_t)s * n[i],
                       (const uint8_t*)src[i] + (size_t)e * n[i], n[i], hipMemcpyHostToDevice,
                       cs) != hipSuccess) {
      (void)hipGetLastError();
      return MOE_ELAUNCH;
    }
    *bytes += n[i];
  }
  return MOE_OK;
}

}  // namespace
}  // namespace bef

extern "C" {

int dsv4_moe_forward(const moe_weights* w, const uint16_t* w_router, const uint16_t* x, int32_t T,
                     int32_t k, const int32_t* routing_ids, const float* routing_w, void* out,
                     int32_t out_dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_forward_args(w, w_router, x, T, k, routing_ids, routing_w, out, out_dtype);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  rc = check_ws(ws, ws_bytes, layout_w(w, T, k).total);
  if (rc) return rc;
  rc = check_device();
  if (rc) return rc;
  return enqueue_forward(w, w_router, x, T, k, routing_ids, routing_w, out, out_dtype, ws,
                         (hipStream_t)stream);
}

int dsv4_moe_forward_noalloc(const moe_weights* w, const uint16_t* w_router, const uint16_t* x,
                             int32_t T, int32_t k, const int32_t* routing_ids,
                             const float* routing_w, void* out, int32_t out_dtype, void* stream) {
  int rc = check_forward_args(w, w_router, x, T, k, routing_ids, routing_w, out, out_dtype);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (layout_w(w, T, k).total > kStaticScratchBytes) return MOE_ENOTSUP;
  rc = check_device();
  if (rc) return rc;
  void* ws = nullptr;
  rc = static_scratch(&ws, (hipStream_t)stream);
  if (rc) return rc;
  return enqueue_forward(w, w_router, x, T, k, routing_ids, routing_w, out, out_dtype, ws,
                         (hipStream_t)stream);
}

size_t moe_host_experts_workspace_bytes(const moe_weights* host_w, int32_t max_tokens,
                                        int32_t top_k) {
  if (check_weights(host_w) != MOE_OK || max_tokens < 1) return 0;
  if (check_tk(max_tokens, top_k, host_w->n_experts) != MOE_OK) return 0;
  size_t a = host_layout(host_w, max_tokens, top_k).total;
  size_t b = host_layout(host_w, 1, top_k).total;
  return a > b ? a : b;
}

size_t moe_host_experts_scratch_bytes(int32_t n_experts, int32_t max_tokens, int32_t top_k) {
  if (n_experts < 1 || max_tokens < 1 || top_k < 1) return 0;
  return host_scratch_need(n_experts, max_tokens, top_k);
}

int moe_forward_host_experts(const moe_weights* host_w, const moe_weights* slot_w,
                             moe_expert_cache* cache, const uint16_t* w_router, const uint16_t* x,
                             int32_t T, int32_t k, void* out, int32_t out_dtype, void* ws,
                             size_t ws_bytes, void* host_scratch, size_t host_scratch_bytes,
                             void* copies_done, void* stream, void* copy_stream) {
  int rc = check_weights(host_w);
  if (rc) return rc;
  rc = check_weights(slot_w);
  if (rc) return rc;
  if (!cache || !cache->slot_of || !cache->expert_of || !cache->last_use || !w_router || !x ||
      !out || !host_scratch || !copies_done)
    return MOE_EINVAL;
  const int E = host_w->n_experts, NS = cache->n_slots;
  if (host_w->format != slot_w->format || host_w->hidden != slot_w->hidden ||
      host_w->inter != slot_w->inter || cache->n_experts != E || slot_w->n_experts != NS ||
      NS < 1 || NS > E)
    return MOE_EINVAL;
  if (out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F32) return MOE_EINVAL;
  rc = check_tk(T, k, E);
  if (rc) return rc;
  if ((int64_t)T * k > NS && NS < E) return MOE_ENOTSUP;  // every expert of a call fits at once
  if (!aligned16(x) || !aligned16(out) || !aligned16(w_router) || !aligned16(host_scratch))
    return MOE_EALIGN;
  if (T == 0) return MOE_OK;
  const HostLayout HL = host_layout(host_w, T, k);
  const Layout& L = HL.L;
  rc = check_ws(ws, ws_bytes, HL.total);
  if (rc) return rc;
  if (host_scratch_bytes < host_scratch_need(E, T, k)) return MOE_EWORKSPACE;
  rc = check_device();
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream, cs = (hipStream_t)copy_stream;
  const int H = host_w->hidden;
  WsCtl* ctl = at<WsCtl>(ws, L.ctl);
  int32_t* ids_dev = at<int32_t>(ws, L.ids);
  float* tw_dev = at<float>(ws, L.w);
  uint8_t* xq = at<uint8_t>(ws, L.xq);
  float* xs = at<float>(ws, L.xs);
  // 1. the router (with the act_quant of x) on the GPU; the ids to the host
  rc = launch_status(launch_route(x, w_router, T, H, E, k, ids_dev, tw_dev, ctl,
                                  at<float>(ws, L.gsum), at<uint16_t>(ws, L.wrT), st, xq, xs));
  if (rc) return rc;
  int32_t* h_ids = (int32_t*)host_scratch;
  int32_t* h_slot_ids = (int32_t*)((uint8_t*)host_scratch + up((size_t)T * k * 4));
  uint8_t* h_masks = (uint8_t*)host_scratch + 2 * up((size_t)T * k * 4);
  if (hipMemcpyAsync(h_ids, ids_dev, (size_t)T * k * 4, hipMemcpyDeviceToHost, st) !=
          hipSuccess ||
      hipStreamSynchronize(st) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ELAUNCH;
  }
  // 2. the cache: hits keep their slots; each miss takes a free slot or the
  // least recently used slot no expert of this call needs, and its weights
  // go over on the copy stream
  const uint64_t now = ++cache->calls;
  uint8_t* mask_a = h_masks;          // groups computed at once: hits + shared
  uint8_t* mask_b = h_masks + E + 1;  // groups computed on arrival: misses
  memset(h_masks, 0, (size_t)2 * (E + 1));
  for (int i = 0; i < T * k; ++i) {
    const int e = h_ids[i];
    if (e < 0 || e >= E) continue;
    const int sl = cache->slot_of[e];
    if (sl >= 0 && cache->last_use[sl] != now) {
      cache->last_use[sl] = now;
      mask_a[sl] = 1;
      cache->hits++;
    }
  }
  int n_miss = 0;
  if (!cache->shared_resident) {
    rc = copy_expert(host_w, slot_w, E, NS, cs, &cache->bytes_copied);
    if (rc) return rc;
    cache->shared_resident = 1;
    mask_b[NS] = 1;
    ++n_miss;
  } else {
    mask_a[NS] = 1;
  }
  for (int i = 0; i < T * k; ++i) {
    const int e = h_ids[i];
    if (e < 0 || e >= E || cache->slot_of[e] >= 0) continue;
    int victim = -1;
    for (int sl = 0; sl < NS; ++sl) {
      if (cache->last_use[sl] == now) continue;
      if (victim < 0 || cache->last_use[sl] < cache->last_use[victim]) victim = sl;
    }
    if (victim < 0) return MOE_ENOTSUP;  // unreachable: NS >= distinct experts of the call
    if (cache->expert_of[victim] >= 0) cache->slot_of[cache->expert_of[victim]] = -1;
    cache->expert_of[victim] = e;
    cache->slot_of[e] = victim;
    cache->last_use[victim] = now;
    rc = copy_expert(host_w, slot_w, e, victim, cs, &cache->bytes_copied);
    if (rc) return rc;
    mask_b[victim] = 1;
    cache->misses++;
    ++n_miss;
  }
  if (n_miss && hipEventRecord((hipEvent_t)copies_done, cs) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ELAUNCH;
  }
  // 3. slot ids and masks to the device
  for (int i = 0; i < T * k; ++i) {
    const int e = h_ids[i];
    h_slot_ids[i] = (e >= 0 && e < E) ? cache->slot_of[e] : -1;
  }
  int32_t* slot_ids = at<int32_t>(ws, HL.slot_ids);
  uint8_t* masks = at<uint8_t>(ws, HL.masks);
  if (hipMemcpyAsync(slot_ids, h_slot_ids, (size_t)T * k * 4, hipMemcpyHostToDevice, st) !=
          hipSuccess ||
      hipMemcpyAsync(masks, h_masks, (size_t)2 * (E + 1), hipMemcpyHostToDevice, st) !=
          hipSuccess) {
    (void)hipGetLastError();
    return MOE_ELAUNCH;
  }
  // 4. the experts in slot space: resident groups now, the copied ones on
  // arrival, then the combine
  int32_t* offsets = at<int32_t>(ws, L.offsets);
  int32_t* row_token = at<int32_t>(ws, L.row_token);
  int32_t* row_of = at<int32_t>(ws, L.row_of);
  float* y = at<float>(ws, L.y);
  rc = launch_status(launch_permute(slot_ids, T, k, NS, offsets, row_token, row_of,
                                    at<int32_t>(ws, L.cnt), &ctl->status, st));
  if (rc) return rc;
  rc = enqueue_gate_up(slot_w, xq, xs, T, k, offsets, row_token, L, ws, st, masks);
  if (rc) return rc;
  rc = enqueue_down(slot_w, T, k, offsets, nullptr, nullptr, y, nullptr, 0, L, ws, st, masks);
  if (rc) return rc;
  if (n_miss) {
    if (hipStreamWaitEvent(st, (hipEvent_t)copies_done, 0) != hipSuccess) {
      (void)hipGetLastError();
      return MOE_ELAUNCH;
    }
    rc = enqueue_gate_up(slot_w, xq, xs, T, k, offsets, row_token, L, ws, st, masks + E + 1);
    if (rc) return rc;
    rc = enqueue_down(slot_w, T, k, offsets, nullptr, nullptr, y, nullptr, 0, L, ws, st,
                      masks + E + 1);
    if (rc) return rc;
  }
  return launch_status(
      launch_combine(y, row_of, tw_dev, T, k, H, out, out_dtype == MOE_DT_BF16, st));
}

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_EINVAL: return "invalid argument";
    case MOE_ENOTSUP: return "not supported (device, format or size limit)";
    case MOE_EALIGN: return "misaligned pointer";
    case MOE_EWORKSPACE: return "workspace too small";
    case MOE_ELAUNCH: return "kernel launch failed";
    default: return "unknown status";
  }
}

int moe_device_status(void* ws, void* stream, uint32_t* status, int clear) {
  if (!ws || !status) return MOE_EINVAL;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_EALIGN;
  int rc = check_device();
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  if (hipMemcpyAsync(status, ws, sizeof(uint32_t), hipMemcpyDeviceToHost, st) != hipSuccess ||
      hipStreamSynchronize(st) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ELAUNCH;
  }
  if (clear) {
    rc = launch_status(launch_zero_words((uint32_t*)ws, 1, st));
    if (rc) return rc;
    if (hipStreamSynchronize(st) != hipSuccess) {
      (void)hipGetLastError();
      return MOE_ELAUNCH;
    }
  }
  return MOE_OK;
}

int moe_debug_stream_read(const void* src, size_t bytes, uint32_t* sink, int32_t blocks,
                          void* stream) {
  if (!src || !sink || bytes < 16 || bytes % 16 != 0 || blocks < 1 || blocks > (1 << 20))
    return MOE_EINVAL;
  if (!aligned16(src)) return MOE_EALIGN;
  int rc = check_device();
  if (rc) return rc;
  stream_read_kernel<<<blocks, 512, 0, (hipStream_t)stream>>>((const uint4*)src, bytes / 16,
                                                               sink);
  return launch_status(hipGetLastError());
}

int moe_debug_set_decode_fused(int32_t fused) {
  if (fused != 0 && fused != 1) return MOE_EINVAL;
  g_decode_fused.store(fused);
  return MOE_OK;
}

int moe_debug_time_kernel(int32_t which, void* start_event, void* stop_event) {
  if (which < MOE_KERNEL_GEMV_GATE_UP || which > MOE_KERNEL_DECODE_FFN) return MOE_EINVAL;
  if ((start_event == nullptr) != (stop_event == nullptr)) return MOE_EINVAL;
  g_kernel_timer[which].start = (hipEvent_t)start_event;
  g_kernel_timer[which].stop = (hipEvent_t)stop_event;
  return MOE_OK;
}

int moe_debug_intermediates(const moe_weights* w, int32_t T, int32_t k, void* ws,
                            size_t ws_bytes, float** h, uint8_t** hq, float** hs) {
  int rc = check_weights(w);
  if (rc) return rc;
  rc = check_tk(T, k, w->n_experts);
  if (rc) return rc;
  if (T == 0) return MOE_EINVAL;  // an empty batch leaves no intermediates
  const Layout L = layout_w(w, T, k);
  rc = check_ws(ws, ws_bytes, L.end_ffn);
  if (rc) return rc;
  const bool gv = gemv_path(w->format, T, k, w->hidden, w->inter);
  if (h) *h = gv ? at<float>(ws, L.h) : nullptr;
  if (hq) *hq = at<uint8_t>(ws, L.hq);
  if (hs) *hs = at<float>(ws, L.hs);
  return MOE_OK;
}

int moe_debug_store_h(float* h, size_t n_floats) {
  if ((h == nullptr) != (n_floats == 0)) return MOE_EINVAL;
  if (h && !aligned16(h)) return MOE_EALIGN;
  g_h_sink.h = h;
  g_h_sink.n = n_floats;
  return MOE_OK;
}

int moe_debug_routing(const moe_weights* w, int32_t T, int32_t k, void* ws, size_t ws_bytes,
                      int32_t** ids, float** topk_w) {
  int rc = check_weights(w);
  if (rc) return rc;
  rc = check_tk(T, k, w->n_experts);
  if (rc) return rc;
  if (T == 0) return MOE_EINVAL;  // an empty batch routes nothing
  const Layout L = layout_w(w, T, k);
  rc = check_ws(ws, ws_bytes, L.total);
  if (rc) return rc;
  if (ids) *ids = at<int32_t>(ws, L.ids);
  if (topk_w) *topk_w = at<float>(ws, L.w);
  return MOE_OK;
}

}  // extern "C"
