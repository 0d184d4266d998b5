// kv.hip -- appending keys and values to a paged cache, with the rotary
// position rotation of q and k on the way.
//
// A pair (a, b) of a head becomes (a c - b s, b c + a s) with the cosine and
// sine of the token's position from the caller's fp32 table; both products
// and the sum are rounded separately (no fused multiply-add), so the result is
// the fp32 evaluation of the formula as written, bit for bit, whatever the
// head layout.  K (rotated) and V go to the token's slot as bf16 (nearest
// even), as E4M3 codes with one fp32 scale amax/448 per (token, head) by
// the act_quant rule, or as E2M1 codes with a power of two per 32 columns.
//
// HBM-bound elementwise work.  One lane owns 8 consecutive elements of a head
// (16 bytes of bf16), D/8 lanes a head, so the pair partner of the "half"
// style is one more 16-byte load of the same row (an L1 hit) and a row's
// amax is a reduction inside an aligned lane group.  A lane keeps its
// table entries in registers for all the heads it takes.
//
// Bound by HBM where tokens are many: FP8 cache, 48 heads of 128, 8192 tokens,
// 187 MB read and written in 39.0 us, the rate of a plain copy of that size; 4-bit cache, 177
// MB in 37.6 us; bf16, 201 MB in 42.8.  A few tokens cost a launch and the latency of three
// dependent loads (3.4 us).
#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace bef {

namespace {

// E2M1 codes (nearest even) of a lane's 8 values and the UE8M0 byte of the 32 columns that
// it shares with the other three lanes of its quad: the smallest power of two that
// brings their largest to 6 at most, so that no value is off by more than half the
// step between its neighbours (with the power below, 6 to 8 times it would all become
// 6).  Bytes end at 252: 6 times the next power is past bf16.  A NaN or an infinity
// leaves the group no value: byte 255.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], uint32_t& sb) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    amax = fmaxf(amax, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : INFINITY);
  const uint32_t top = __float_as_uint(group_max<4>(amax));
  const int e = max(0, min((int)(top >> 23) - 2 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0), 252));
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    u[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[i], 127 - e), -6.0f, 6.0f);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, u[0], u[1], 1.0f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, u[2], u[3], 1.0f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, u[4], u[5], 1.0f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, u[6], u[7], 1.0f, 3);
  const bool none = top == 0x7f800000u;
  sb = none ? 255u : (uint32_t)e;
  return none ? 0u : q;
}

// The rotated pair, each operation rounded on its own (the empty asm keeps the
// products as values of their own: this library is compiled with fused
// multiply-adds allowed everywhere).
__device__ __forceinline__ void rotate(float a, float b, float c, float s, float& ra, float& rb) {
  float ac = a * c, bs = b * s, bc = b * c, as = a * s;
  asm("" : "+v"(ac), "+v"(bs), "+v"(bc), "+v"(as));
  ra = ac - bs;
  rb = bc + as;
}

}  // namespace

// grid: (tokens, head groups).  LPH lanes per head (D/8); a block of 256 takes
// 256/LPH heads at a time, `iters` times.
template <int LPH, int KV, bool PAIRS>
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
    if constexpr (KV == kKvBf16) {
      *reinterpret_cast<uint4*>(dst + (row * D + 8 * c) * 2) = pack8(v);
    } else if constexpr (KV == kKvE4M3) {
      float sc;
      const uint2 q = e4m3x8<LPH>(v, sc);
      *reinterpret_cast<uint2*>(dst + row * D + 8 * c) = q;
      if (c == 0) ((float*)(is_v ? a.vs : a.ks))[row] = sc;
    } else {
      uint32_t sb;
      const uint32_t q = e2m1x8(v, sb);
      *reinterpret_cast<uint32_t*>(dst + row * (D / 2) + 4 * c) = q;
      if ((c & 3) == 0) ((uint8_t*)(is_v ? a.vs : a.ks))[row * (D / 32) + (c >> 2)] = (uint8_t)sb;
    }
  }
}

namespace {

template <int LPH, int KV>
void launch_style(const KvAppendArgs& a, dim3 grid, hipStream_t st) {
  if (a.pairs)
    kv_append_kernel<LPH, KV, true><<<grid, 256, 0, st>>>(a);
  else
    kv_append_kernel<LPH, KV, false><<<grid, 256, 0, st>>>(a);
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
  if (a.kv == kKvE2M1)
    launch_style<LPH, kKvE2M1>(a, grid, st);
  else if (a.kv == kKvE4M3)
    launch_style<LPH, kKvE4M3>(a, grid, st);
  else
    launch_style<LPH, kKvBf16>(a, grid, st);
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
