// kv.hip -- appending keys and values to a paged cache, with the rotary
// position rotation of q and k on the way.
//
// A pair (a, b) of a head becomes (a c - b s, b c + a s) with the cosine and
// sine of the token's position from the caller's fp32 table; both products
// and the sum are rounded separately (no fused multiply-add), so the result is
// the fp32 evaluation of the formula as written, bit for bit, whatever the
// head layout.  K (rotated) and V go to the token's slot as bf16 (nearest
// even), or as E4M3 codes with one fp32 scale amax/448 per (token, head) by
// the act_quant rule.
//
// HBM-bound elementwise work.  One lane owns 8 consecutive elements of a head
// (16 bytes of bf16), D/8 lanes a head, so the pair partner of the "half"
// style is one more 16-byte load of the same row (an L1 hit) and a row's
// amax is a reduction inside an aligned lane group.  A lane keeps its
// table entries in registers for all the heads it takes.
//
// Bound by HBM where tokens are many: FP8 cache, 48 heads of 128, 8192 tokens,
// 187 MB read and written in 39.0 us, the rate of a plain copy of that size.
// A few tokens cost a launch and the latency of three dependent loads (3.4 us).
#include "common.h"
#include "kernels.h"

namespace bef {

namespace {

// The rotated pair, each operation rounded on its own (the empty asm keeps the
// products as values of their own: this library is compiled with fused
// multiply-adds allowed everywhere).
__device__ __forceinline__ void rotate(float a, float b, float c, float s, float& ra, float& rb) {
  float ac = a * c, bs = b * s, bc = b * c, as = a * s;
  asm("" : "+v"(ac), "+v"(bs), "+v"(bc), "+v"(as));
  ra = ac - bs;
  rb = bc + as;
}

__device__ __forceinline__ void unpack8(const uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 0x7f, E4M3's NaN, in the byte of each of four values that is NaN.
__device__ __forceinline__ uint32_t nan_bytes(const float* v) {
  return (v[0] != v[0] ? 0x7fu : 0u) | (v[1] != v[1] ? 0x7f00u : 0u) |
         (v[2] != v[2] ? 0x7f0000u : 0u) | (v[3] != v[3] ? 0x7f000000u : 0u);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                    f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
}

}  // namespace

// grid: (tokens, head groups).  LPH lanes per head (D/8); a block of 256 takes
// 256/LPH heads at a time, `iters` times.
template <int LPH, bool FP8, bool PAIRS>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a) {
  constexpr int D = LPH * 8, HPB = 256 / LPH;
  const int t = blockIdx.x;
  const int c = threadIdx.x % LPH, hs = threadIdx.x / LPH;
  const int seq = a.seq_of[t], pos = a.pos[t];
  if (seq < 0 || pos < 0) return;  // padding
  const int pi = pos >> a.page_shift;
  int page = -1;
  if (seq < a.n_seqs && pi < a.table_cols && (a.R == 0 || pos < a.rope_rows))
    page = a.table[(size_t)seq * a.table_cols + pi];
  if (page < 0 || page >= a.n_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && a.status) set_status(a.status, MOE_STATUS_BAD_PAGE);
    return;
  }
  const int slot = pos & ((1 << a.page_shift) - 1);
  // this lane's cosines and sines: pair i of the head uses table entries i and
  // R/2 + i.  Half style: elements 8c.. pair with 8c +- R/2 (R/2 a multiple
  // of 8); pairs style: elements 8c.. are pairs 4c..4c+3.
  const bool rot = 8 * c < a.R;
  const int half = a.R >> 1;
  const bool upper = !PAIRS && 8 * c >= half;
  constexpr int NC = PAIRS ? 4 : 8;
  float cs[NC], sn[NC];
  if (rot) {
    const float* row = a.rope + (size_t)pos * a.R + (PAIRS ? 4 * c : upper ? 8 * c - half : 8 * c);
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(row + i);
      const float4 y = *reinterpret_cast<const float4*>(row + half + i);
      cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
      sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
    }
  }
  const int nh = a.Hq + 2 * a.Hkv;
  for (int it = 0; it < a.iters; ++it) {
    const int h = (blockIdx.y * a.iters + it) * HPB + hs;
    if (h >= nh) return;
    const int kvh = h - a.Hq;  // >= 0: k heads, then v heads
    const bool is_v = kvh >= a.Hkv;
    const uint16_t* src = kvh < 0 ? a.q + (size_t)t * a.q_stride + (size_t)h * D
                          : is_v  ? a.v + (size_t)t * a.v_stride + (size_t)(kvh - a.Hkv) * D
                                  : a.k + (size_t)t * a.k_stride + (size_t)kvh * D;
    uint4 raw = *reinterpret_cast<const uint4*>(src + 8 * c);
    float v[8];
    unpack8(raw, v);
    if (rot && !is_v) {
      if (PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float ra, rb;
          rotate(v[2 * i], v[2 * i + 1], cs[i % NC], sn[i % NC], ra, rb);
          v[2 * i] = ra, v[2 * i + 1] = rb;
        }
      } else {
        float w[8];
        unpack8(*reinterpret_cast<const uint4*>(src + (upper ? 8 * c - half : 8 * c + half)), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float ra, rb;
          rotate(upper ? w[i] : v[i], upper ? v[i] : w[i], cs[i % NC], sn[i % NC], ra, rb);
          v[i] = upper ? rb : ra;
        }
      }
    }
    if (kvh < 0) {
      *reinterpret_cast<uint4*>(a.q_out + ((size_t)t * a.Hq + h) * D + 8 * c) = pack8(v);
      continue;
    }
    const size_t row = (((size_t)page * a.Hkv + (is_v ? kvh - a.Hkv : kvh)) << a.page_shift) + slot;
    uint8_t* dst = (uint8_t*)(is_v ? a.vc : a.kc);
    if (!FP8) {
      *reinterpret_cast<uint4*>(dst + (row * D + 8 * c) * 2) = pack8(v);
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
      amax = group_max<LPH>(amax);
      const float sc = amax / 448.0f;
      uint2 q = make_uint2(0, 0);
      if (amax != 0.0f) {
        q.x = e4m3_pack4(v[0] / sc, v[1] / sc, v[2] / sc, v[3] / sc);
        q.y = e4m3_pack4(v[4] / sc, v[5] / sc, v[6] / sc, v[7] / sc);
      }
      // a NaN keeps its place (the maximum and the conversion's clamp pass over it)
      const uint2 nan = make_uint2(nan_bytes(v), nan_bytes(v + 4));
      if (__ballot((nan.x | nan.y) != 0))
        q = make_uint2((q.x & ~(nan.x << 1)) | nan.x, (q.y & ~(nan.y << 1)) | nan.y);
      *reinterpret_cast<uint2*>(dst + row * D + 8 * c) = q;
      if (c == 0) (is_v ? a.vs : a.ks)[row] = sc;
    }
  }
}

namespace {

template <int LPH, bool FP8>
void launch_style(const KvAppendArgs& a, dim3 grid, hipStream_t st) {
  if (a.pairs)
    kv_append_kernel<LPH, FP8, true><<<grid, 256, 0, st>>>(a);
  else
    kv_append_kernel<LPH, FP8, false><<<grid, 256, 0, st>>>(a);
}

template <int LPH>
void launch_dim(KvAppendArgs a, hipStream_t st) {
  constexpr int HPB = 256 / LPH;
  const int groups = (a.Hq + 2 * a.Hkv + HPB - 1) / HPB;
  // Many tokens: a block takes all heads of one, its table entries read once (4096
  // tokens, 48 bf16 heads of 128: 18.4 us, 20.4 with a block per 16 heads).  Fewer:
  // a block per 256/LPH heads, or too few blocks wait on memory (512 tokens: 5.2 us,
  // 5.4 the other way; 32 tokens: 3.4 and 4.3).
  a.iters = a.T >= 1024 ? groups : 1;
  const dim3 grid(a.T, (groups + a.iters - 1) / a.iters);
  if (a.fp8)
    launch_style<LPH, true>(a, grid, st);
  else
    launch_style<LPH, false>(a, grid, st);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st) {
  if (a.D == 64)
    launch_dim<8>(a, st);
  else if (a.D == 128)
    launch_dim<16>(a, st);
  else
    launch_dim<32>(a, st);
  return hipGetLastError();
}

}  // namespace bef
