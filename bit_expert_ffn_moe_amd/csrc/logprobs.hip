// logprobs.hip -- log probabilities of given tokens, the entropy of their
// distributions and the n best alternatives, from rows of logits z:
//   M = max z,  l = sum e^(z-M),  logprob(i) = (z_i - M) - log l,
//   H = log l - sum (z-M) e^(z-M) / l,  best n by (z descending, id ascending).
//
// One pass over the logits.  A wave takes 2048 consecutive elements into
// registers (32 a lane), forms its own maximum and sums there, and selects its
// n best: its lanes' best elements are sorted across the wave, which bounds the
// n-th best from below; lanes whose next element still beats that bound
// offer it, until none does.  Partials (m, l, sum, n keys) go to the
// workspace; a second kernel joins a row's waves.  HBM-bound when there are many
// rows, latency-bound for one.
//
// A candidate is one 64-bit key: the logit's order in the high word (a
// monotone map of fp32 to unsigned, NaN 1 and below every number, 0 for places
// outside the row, -0 = +0), the complement of
// the id in the low word; keys are distinct and a larger key ranks
// first, so ties go to the lower id and the result depends on no order of
// execution.
#include "common.h"
#include "kernels.h"

namespace bef {

namespace {

typedef unsigned long long u64;
constexpr int kPerLane = kLogprobChunk / 64;

__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  if (z != z) return 1u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  if (u == 1u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ u64 shfl_xor64(u64 v, int m) {
  const uint32_t lo = __shfl_xor((uint32_t)v, m), hi = __shfl_xor((uint32_t)(v >> 32), m);
  return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 lane64(u64 v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, l);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), l);
  return (u64)hi << 32 | lo;
}

// Bitonic sort over the wave, largest key in lane 0.
__device__ __forceinline__ u64 wave_sort(u64 v, int lane) {
#pragma unroll
  for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const u64 o = shfl_xor64(v, j);
      const bool keep_max = ((lane & j) == 0) == ((lane & k) == 0);
      v = (v > o) == keep_max ? v : o;
    }
  return v;
}

// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ u64 wave_merge(u64 a, u64 b, int lane) {
  const u64 r = shfl_xor64(b, 63);
  u64 v = a > r ? a : r;
#pragma unroll
  for (int j = 32; j > 0; j >>= 1) {
    const u64 o = shfl_xor64(v, j);
    v = (v > o) == ((lane & j) == 0) ? v : o;
  }
  return v;
}

template <bool BF16>
__device__ __forceinline__ float load_z(const void* row, int64_t i) {
  if (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[i]);
  return reinterpret_cast<const float*>(row)[i];
}

}  // namespace

// grid (T, ceil(W / 4)): wave = one chunk of one row.
template <bool BF16>
__global__ __launch_bounds__(256) void logprob_chunk_kernel(LogprobArgs a) {
  constexpr int VE = BF16 ? 8 : 4, NV = kPerLane / VE, ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x, w = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (w >= a.W) return;
  const uint8_t* row = (const uint8_t*)a.z + (size_t)t * a.row_stride * ES;
  // 16-byte words from the row's address rounded down; the elements before the
  // row's first and after its last are not read
  const int off = (int)((uintptr_t)row & 15) / ES;
  const uint8_t* base = row - off * ES;
  float z[kPerLane];
  const int e0 = w * kLogprobChunk + lane * VE;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = e0 + v * 64 * VE;
    if (e >= off && e + VE <= off + a.V) {
      const uint4 r = *reinterpret_cast<const uint4*>(base + (size_t)e * ES);
      const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (BF16) {
          z[v * VE + 2 * i] = __uint_as_float(x[i] << 16);
          z[v * VE + 2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        } else {
          z[v * VE + i] = __uint_as_float(x[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        z[v * VE + i] = (e + i >= off && e + i < off + a.V) ? load_z<BF16>(base, e + i) : -INFINITY;
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) m = fmaxf(m, z[i]);
  m = wave_max(m);
  const float mu = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, s = 0.0f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const float d = z[i] - mu, e = __expf(d);
    l += e;
    s = fmaf(fmaxf(d, -1e30f), e, s);  // -inf contributes 0; NaN stays in e
  }
  l = wave_sum_dpp(l);
  s = wave_sum_dpp(s);
  const size_t part = (size_t)t * a.W + w;
  if (lane == 0) {
    a.pm[part] = m;
    a.pl[part] = l;
    a.ps[part] = s;
  }
  if (a.n_top == 0) return;

  uint32_t key[kPerLane];
  const bool full = w * kLogprobChunk >= off && (w + 1) * kLogprobChunk <= off + a.V;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    key[i] = order_of(z[i]);
    const int e = e0 + (i / VE) * 64 * VE + i % VE;
    if (!full && (e < off || e >= off + a.V)) key[i] = 0u;
  }
  // key64 of this lane's element i; elements outside the row rank last
  auto whole = [&](uint32_t k, int i) -> u64 {
    const int e = e0 + (i / VE) * 64 * VE + i % VE;
    if (e < off || e >= off + a.V) return 0;
    return (u64)k << 32 | (0xffffffffu - (uint32_t)(e - off));
  };
  uint32_t ck = 0;
  int ci = kPerLane - 1;
#pragma unroll
  for (int i = kPerLane - 1; i >= 0; --i)
    if (key[i] >= ck) ck = key[i], ci = i;
  u64 cur = whole(ck, ci);
  u64 top = wave_sort(cur, lane);
  u64 thr = lane64(top, a.n_top - 1);
  while (true) {
    // this lane's next element after (ck, ci); none if the last fell short
    uint32_t nk = 1;  // 0: outside the row
    int ni = -1;
    if (cur >= thr && cur != 0) {
#pragma unroll
      for (int i = kPerLane - 1; i >= 0; --i)
        if ((key[i] < ck || (key[i] == ck && i > ci)) && key[i] >= nk) nk = key[i], ni = i;
    }
    cur = ni >= 0 ? whole(nk, ni) : 0;
    ck = nk, ci = ni;
    if (cur <= thr) cur = 0;
    if (!__ballot(cur != 0)) break;
    top = wave_merge(top, wave_sort(cur, lane), lane);
    thr = lane64(top, a.n_top - 1);
  }
  // rank-major, so that the join sees every wave's best first
  if (lane < a.n_top) a.pk[((size_t)t * a.n_top + lane) * a.W + w] = top;
}

// One block per row: joins the waves' sums and candidates.
template <bool BF16>
__global__ __launch_bounds__(256) void logprob_join_kernel(LogprobArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  __shared__ float sm[4], sl[4], ss[4];
  __shared__ u64 st[4][64];
  const size_t p0 = (size_t)t * a.W;
  float M = -INFINITY;
  for (int i = threadIdx.x; i < a.W; i += 256) M = fmaxf(M, a.pm[p0 + i]);
  M = wave_max(M);
  if (lane == 0) sm[wv] = M;
  __syncthreads();
  M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float l = 0.0f, s = 0.0f;
  for (int i = threadIdx.x; i < a.W; i += 256) {
    const float m = a.pm[p0 + i], li = a.pl[p0 + i];
    if (m == -INFINITY) {
      l += li;  // 0, or NaN where the wave held nothing but NaN and -inf
      continue;
    }
    const float d = m - M, e = __expf(d);
    l = fmaf(e, li, l);
    s = fmaf(e, fmaf(d, li, a.ps[p0 + i]), s);
  }
  l = wave_sum_dpp(l);
  s = wave_sum_dpp(s);
  if (lane == 0) sl[wv] = l, ss[wv] = s;
  u64 top = 0;
  if (a.n_top) {
    const int total = a.n_top * a.W;
    const u64* pk = a.pk + (size_t)t * total;
    u64 thr = 0;
    for (int b = wv * 64; b < total; b += 256) {
      u64 c = b + lane < total ? pk[b + lane] : 0;
      if (c <= thr) c = 0;
      if (!__ballot(c != 0)) continue;
      top = wave_merge(top, wave_sort(c, lane), lane);
      thr = lane64(top, a.n_top - 1);
    }
    st[wv][lane] = top;
  }
  __syncthreads();
  if (wv) return;
  l = sl[0] + sl[1] + sl[2] + sl[3];
  s = ss[0] + ss[1] + ss[2] + ss[3];
  const bool empty = M == -INFINITY && l == 0.0f;  // every logit is -inf
  const float ll = logf(l);
  if (lane == 0) {
    if (a.entropy) a.entropy[t] = empty ? 0.0f : ll - s / l;
    if (a.tokens) {
      const int tok = a.tokens[t];
      float lp = 0.0f;
      if (tok >= 0 && tok < a.V) {
        const float z = load_z<BF16>(
            (const uint8_t*)a.z + (size_t)t * a.row_stride * (BF16 ? 2 : 4), tok);
        lp = empty ? -INFINITY : (z - M) - ll;
      } else if (tok >= a.V && a.status) {
        set_status(a.status, MOE_STATUS_BAD_TOKEN);
      }
      a.logprob[t] = lp;
    }
  }
  if (a.n_top == 0) return;
#pragma unroll
  for (int k = 1; k < 4; ++k) top = wave_merge(top, st[k][lane], lane);
  if (lane < a.n_top) {
    const float z = order_value((uint32_t)(top >> 32));
    a.top_ids[(size_t)t * a.n_top + lane] = (int32_t)(0xffffffffu - (uint32_t)top);
    a.top_logprobs[(size_t)t * a.n_top + lane] = empty ? -INFINITY : (z - M) - ll;
  }
}

hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t st) {
  const dim3 grid(a.T, (a.W + 3) / 4);
  if (bf16) {
    logprob_chunk_kernel<true><<<grid, 256, 0, st>>>(a);
    logprob_join_kernel<true><<<a.T, 256, 0, st>>>(a);
  } else {
    logprob_chunk_kernel<false><<<grid, 256, 0, st>>>(a);
    logprob_join_kernel<false><<<a.T, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace bef
