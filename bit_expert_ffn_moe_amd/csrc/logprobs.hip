// logprobs.hip -- log probabilities of given tokens, the entropy of their
// distributions and the n best alternatives, from rows of logits z:
//   M = max z,  l = sum e^(z-M),  logprob(i) = (z_i - M) - log l,
//   H = log l - sum (z-M) e^(z-M) / l,  best n by (z descending, id ascending).
//
// One pass over the logits.  A wave takes 2048 consecutive elements into
// registers (32 a lane) and forms its maximum and sums there.  Its n best: the
// n-th largest of the lanes' maxima bounds the n-th best from below, so the
// few elements that reach it are collected and sorted across the wave.
//   Few rows: a wave per 2048 elements leaves (m, l, sum, n keys) in the workspace
// and a second kernel joins a row's waves: latency-bound.
//   Many rows: a block of four waves walks a row, each wave keeping its statistics and
// its n best so far (later elements then mostly fall short of its n-th best), and
// joins them itself: bound by HBM and, closely, by the vector unit (an
// exponential and ten more operations an element).
// Measured: one row of 131072 fp32 with its 20 best 12.8 us, 32 rows of bf16 with 5
// 14.8 us (two launches and their latencies); 4096 rows of 50021 bf16, 410 MB, 82 to 86
// us (4.8 to 5.0 TB/s).
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

// The value of lane l ^ J: DPP inside rows of 16 (4 as mirror of 8, then of 4), row
// swaps across them.
template <int J>
__device__ __forceinline__ uint32_t exch(uint32_t v) {
  if constexpr (J == 1) {
    return dpp_row<0xB1>((int)v);
  } else if constexpr (J == 2) {
    return dpp_row<0x4E>((int)v);
  } else if constexpr (J == 4) {
    return dpp_row<0x1B>(dpp_row<0x141>((int)v));
  } else if constexpr (J == 8) {
    return dpp_row<0x128>((int)v);  // row_ror:8
  } else if constexpr (J == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? r[0] : r[1];
  }
}
template <int J>
__device__ __forceinline__ u64 exch(u64 v) {
  return (u64)exch<J>((uint32_t)(v >> 32)) << 32 | exch<J>((uint32_t)v);
}
__device__ __forceinline__ u64 lane64(u64 v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, l);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), l);
  return (u64)hi << 32 | lo;
}

// One step of a bitonic network over the wave: pairs (l, l ^ J), the larger to
// the lane where `first` says so.
template <int J, class T>
__device__ __forceinline__ T step(T v, bool first) {
  const T o = exch<J>(v);
  return (v > o) == first ? v : o;
}
// Sorts runs of K, falling where lane & K is 0 (everywhere for K = 64).
template <int K, int J, class T>
__device__ __forceinline__ T clean(T v, int lane) {
  v = step<J>(v, ((lane & J) == 0) == ((lane & K) == 0));
  if constexpr (J > 1) v = clean<K, J / 2>(v, lane);
  return v;
}
// Bitonic sort over the wave, largest in lane 0 (unsigned values).
template <int K = 2, class T>
__device__ __forceinline__ T wave_sort(T v, int lane) {
  v = clean<K, K / 2>(v, lane);
  if constexpr (K < 64) v = wave_sort<2 * K>(v, lane);
  return v;
}

__device__ __forceinline__ u64 larger(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ u64 wave_largest(u64 v) {
  v = larger(v, exch<1>(v));
  v = larger(v, exch<2>(v));
  v = larger(v, exch<4>(v));
  v = larger(v, exch<8>(v));
  v = larger(v, exch<16>(v));
  return larger(v, exch<32>(v));
}

// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ u64 wave_merge(u64 a, u64 b, int lane) {
  // b turned round: lane l ^ 63
  u64 r = exch<32>(exch<16>(b));
  r = (u64)(uint32_t)dpp_row<0x140>((int)(r >> 32)) << 32 | (uint32_t)dpp_row<0x140>((int)r);
  return clean<64, 32>(a > r ? a : r, lane);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// (a - b) log2 e, not below -1e30: sums may be multiplied by it where their weight 2^it
// is 0 (a and b of the type's lowest and highest values are 2^129 apart).
__device__ __forceinline__ float log2_ratio(float a, float b) {
  return fmaxf((a - b) * kLog2e, -1e30f);
}

__device__ __forceinline__ float max_of(const float (&z)[kPerLane]) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < kPerLane; ++i) m = fmaxf(m, z[i]);
  return m;
}

// Adds a part (m, l, s) to sums relative to M >= m.
__device__ __forceinline__ void add_part(float m, float li, float si, float M, float& l,
                                         float& s) {
  if (m == -INFINITY) {
    l += li;  // 0, or NaN where the part held nothing but NaN and -inf
    return;
  }
  const float d = log2_ratio(m, M), f = __builtin_amdgcn_exp2f(d);
  l = fmaf(f, li, l);
  s = fmaf(f, fmaf(d, li, si), s);
}

template <bool BF16>
__device__ __forceinline__ float load_z(const void* row, int64_t i) {
  if (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[i]);
  return reinterpret_cast<const float*>(row)[i];
}

}  // namespace

namespace {

// A row as aligned 16-byte words: `base` is its address rounded down, `off`
// its first element's place there.  Nothing before the row's first element or
// after its last is read.
struct Row {
  const uint8_t* base;
  int off, end;  // elements [off, end)
};
template <bool BF16>
__device__ __forceinline__ Row row_of(const LogprobArgs& a, int t) {
  constexpr int ES = BF16 ? 2 : 4;
  const uint8_t* row = (const uint8_t*)a.z + (size_t)t * a.row_stride * ES;
  Row r;
  r.off = (int)((uintptr_t)row & 15) / ES;
  r.base = row - r.off * ES;
  r.end = r.off + a.V;
  return r;
}

// Place of element i of this lane in chunk w.
template <bool BF16>
__device__ __forceinline__ int place(int w, int lane, int i) {
  constexpr int VE = BF16 ? 8 : 4;
  return w * kLogprobChunk + ((i / VE) * 64 + lane) * VE + i % VE;
}

// Chunk w's raw words (whole ones; others are read element by element in unpack).
constexpr int kMaxWords = kPerLane / 4;
template <bool BF16>
__device__ __forceinline__ void load_chunk(const Row& r, int w, int lane,
                                           uint4 (&raw)[kMaxWords]) {
  constexpr int VE = BF16 ? 8 : 4, ES = BF16 ? 2 : 4;
#pragma unroll
  for (int v = 0; v < kPerLane / VE; ++v) {
    const int e = place<BF16>(w, lane, v * VE);
    if (e >= r.off && e + VE <= r.end)
      raw[v] = *reinterpret_cast<const uint4*>(r.base + (size_t)e * ES);
  }
}
// ... as fp32, -inf outside the row.
template <bool BF16>
__device__ __forceinline__ void unpack_chunk(const Row& r, int w, int lane,
                                             const uint4 (&raw)[kMaxWords],
                                             float (&z)[kPerLane]) {
  constexpr int VE = BF16 ? 8 : 4;
#pragma unroll
  for (int v = 0; v < kPerLane / VE; ++v) {
    const uint32_t x[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
#pragma unroll
    for (int i = 0; i < VE; ++i)
      z[v * VE + i] = BF16 ? __uint_as_float((i & 1) ? x[i / 2] & 0xffff0000u : x[i / 2] << 16)
                           : __uint_as_float(x[i % 4]);
  }
  if (w * kLogprobChunk < r.off || (w + 1) * kLogprobChunk > r.end) {
#pragma unroll
    for (int v = 0; v < kPerLane / VE; ++v) {
      const int e = place<BF16>(w, lane, v * VE);
      if (!(e >= r.off && e + VE <= r.end)) {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          z[v * VE + i] = e + i >= r.off && e + i < r.end ? load_z<BF16>(r.base, e + i) : -INFINITY;
      }
    }
  }
}

// Running statistics of a lane: maximum m (of the wave), l = sum 2^t and
// s = sum t 2^t with t = (z - m) log2 e; t of -inf counts as -1e30 in s, where its
// weight is 0.  A NaN or +inf makes l NaN.
struct Stats {
  float m, l, s;
};
// l and s of a chunk, t_of giving each element's t (two sums each: shorter chains).
template <class F>
__device__ __forceinline__ void chunk_sums(const float (&z)[kPerLane], F&& t_of, float& l,
                                           float& s) {
  float l0 = 0.0f, l1 = 0.0f, s0 = 0.0f, s1 = 0.0f;
#pragma unroll
  for (int i = 0; i < kPerLane; i += 2) {
    const float t0 = t_of(z[i]), t1 = t_of(z[i + 1]);
    const float e0 = __builtin_amdgcn_exp2f(t0), e1 = __builtin_amdgcn_exp2f(t1);
    l0 += e0, l1 += e1;
    s0 = fmaf(fmaxf(t0, -1e30f), e0, s0), s1 = fmaf(fmaxf(t1, -1e30f), e1, s1);
  }
  l = l0 + l1, s = s0 + s1;
}
__device__ __forceinline__ void add_chunk(const float (&z)[kPerLane], float lane_max, Stats& st) {
  const float m = fmaxf(st.m, wave_max(lane_max));
  if (m > st.m) {
    if (st.m != -INFINITY) {
      const float d = log2_ratio(st.m, m), f = __builtin_amdgcn_exp2f(d);
      st.s = f * fmaf(d, st.l, st.s);
      st.l *= f;
    }
    st.m = m;
  }
  float l, s;
  if (fabsf(m) <= 65536.0f) {
    // One operation an element: t + d = z log2 e + c with c = -m log2 e rounded, so every
    // term carries 2^d, d the rounding error of c (2^-8 at most here), which is taken
    // out of the chunk's sums.
    const float c = -m * kLog2e, d = fmaf(m, kLog2e, c), g = __builtin_amdgcn_exp2f(-d);
    chunk_sums(z, [&](float v) { return fmaf(v, kLog2e, c); }, l, s);
    st.l = fmaf(g, l, st.l);
    st.s = fmaf(g, fmaf(-d, l, s), st.s);
  } else {
    // m log2 e may overflow and d be anything: subtracted first
    const float r = m == -INFINITY ? 0.0f : m;
    chunk_sums(z, [&](float v) { return (v - r) * kLog2e; }, l, s);
    st.l += l;
    st.s += s;
  }
}

// The wave's n best so far: sorted keys, the n-th (0: fewer than n yet).
struct Best {
  u64 top, thr;
};

// Any chunk, NaN and -inf included: each lane offers its elements best first, all
// lanes' next ones sorted and merged at a time, until none beats the n-th best.
template <bool BF16>
__device__ __forceinline__ void select_any(const Row& r, int w, int lane, int n,
                                           const float (&z)[kPerLane], Best& b) {
  uint32_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = place<BF16>(w, lane, i);
    key[i] = e >= r.off && e < r.end ? order_of(z[i]) : 0u;
  }
  uint32_t ck = 0xffffffffu;  // the lane's last offer
  int ci = kPerLane;
  bool going = true;
  while (true) {
    uint32_t nk = 1;  // 0: outside the row
    int ni = -1;
    if (going) {
#pragma unroll
      for (int i = kPerLane - 1; i >= 0; --i)
        if ((key[i] < ck || (key[i] == ck && i > ci)) && key[i] >= nk) nk = key[i], ni = i;
    }
    u64 cur = 0;
    if (ni >= 0) cur = (u64)nk << 32 | (0xffffffffu - (uint32_t)(place<BF16>(w, lane, ni) - r.off));
    if (cur <= b.thr) cur = 0;
    going = cur != 0;
    ck = nk, ci = ni;
    if (!__ballot(going)) break;
    b.top = wave_merge(b.top, wave_sort(cur, lane), lane);
    b.thr = lane64(b.top, n - 1);
  }
}

// Adds chunk w (its values z, their lane maximum) to the n best.  cand: this wave's
// room for kCand keys in LDS.
constexpr int kCand = 256;
template <bool BF16>
__device__ __forceinline__ void select_chunk(const Row& r, int w, int lane, int n, bool nan,
                                             const float (&z)[kPerLane], float lane_max, Best& b,
                                             u64* cand) {
  constexpr int VE = BF16 ? 8 : 4;
  const bool have = b.thr != 0;
  // elements of a later chunk have higher ids: they must exceed the n-th best
  const float least = have ? order_value((uint32_t)(b.thr >> 32)) : -INFINITY;
  nan |= least != least;
  if (!nan && have && !__ballot(lane_max > least)) return;
  if (n == 1 && !nan) {
    // the maximum and its first place
    const float best = wave_max(lane_max);
    if (best != -INFINITY) {
      int at = kPerLane;
#pragma unroll
      for (int i = kPerLane - 1; i >= 0; --i)
        if (z[i] == best) at = i;
      const int id = wave_min_all(
          at < kPerLane ? place<BF16>(w, lane, 0) + (at / VE) * 64 * VE + at % VE - r.off
                        : 0x7fffffff);
      b.thr = (u64)order_of(best) << 32 | (0xffffffffu - (uint32_t)id);
      b.top = lane == 0 ? b.thr : 0;
      return;
    }
  }
  float tau = least;
  if (!nan && !have)
    tau = order_value(__builtin_amdgcn_readlane(wave_sort(order_of(lane_max), lane), n - 1));
  if (nan || tau == -INFINITY) {
    select_any<BF16>(r, w, lane, n, z, b);
    return;
  }
  uint32_t mask = 0;  // bit 31 - i: element i is a candidate
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) mask = 2 * mask + ((have ? z[i] > tau : z[i] >= tau) ? 1u : 0u);
  const int count = (int)wave_sum_dpp((float)__popc(mask));
  if (count > kCand) {  // ties in their hundreds
    select_any<BF16>(r, w, lane, n, z, b);
    return;
  }
  int at = 0;
  while (true) {
    const u64 some = __ballot(mask != 0);
    if (!some) break;
    if (mask) {
      const int i = __clz(mask);
      mask &= ~(0x80000000u >> i);
      const int e = place<BF16>(w, lane, i);
      const int p = at + __popcll(some & (((u64)1 << lane) - 1));
      cand[p] = (u64)order_of(load_z<BF16>(r.base, e)) << 32 | (0xffffffffu - (uint32_t)(e - r.off));
    }
    at += __popcll(some);
  }
  __builtin_amdgcn_wave_barrier();
  for (int i = 0; i < count; i += 64) {
    u64 c = i + lane < count ? cand[i + lane] : 0;
    if (c <= b.thr) c = 0;
    if (!__ballot(c != 0)) continue;
    b.top = wave_merge(b.top, wave_sort(c, lane), lane);
    b.thr = lane64(b.top, n - 1);
  }
  __builtin_amdgcn_wave_barrier();
}

// Stats and n best of the waves of a block, joined: wave 0 returns the row's (all lanes).
// NW waves, `top` valid where n > 0.
template <int NW>
__device__ __forceinline__ void join_waves(Stats& st, u64& top, int n, int lane, int wv,
                                           float* sm, u64 (*sk)[64]) {
  st.l = wave_sum_dpp(st.l);
  st.s = wave_sum_dpp(st.s);
  if constexpr (NW == 1) return;
  if (lane == 0) sm[wv] = st.m, sm[NW + wv] = st.l, sm[2 * NW + wv] = st.s;
  if (n) sk[wv][lane] = top;
  __syncthreads();
  if (n) {
#pragma unroll
    for (int half = NW / 2; half > 0; half >>= 1) {
      if (wv < half) {
        top = wave_merge(top, sk[wv + half][lane], lane);
        sk[wv][lane] = top;
      }
      __syncthreads();
    }
  }
  if (wv) return;
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < NW; ++i) M = fmaxf(M, sm[i]);
  float l = 0.0f, s = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) add_part(sm[i], sm[NW + i], sm[2 * NW + i], M, l, s);
  st.m = M, st.l = l, st.s = s;
}

// The row's outputs from its joined statistics (one wave).
template <bool BF16>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int t, int lane, const Stats& st,
                                          u64 top) {
  const bool empty = st.m == -INFINITY && st.l == 0.0f;  // every logit is -inf
  // the largest term is 1, whatever the sum's rounding: no log probability above 0
  const float l = st.l < 1.0f ? 1.0f : st.l, ll = logf(l);
  if (lane == 0) {
    if (a.entropy) a.entropy[t] = empty ? 0.0f : ll - st.s / l * kLn2;
    if (a.tokens) {
      const int tok = a.tokens[t];
      float lp = 0.0f;
      if (tok >= 0 && tok < a.V) {
        const float z = load_z<BF16>(
            (const uint8_t*)a.z + (size_t)t * a.row_stride * (BF16 ? 2 : 4), tok);
        lp = empty ? -INFINITY : (z - st.m) - ll;
      } else if (tok >= a.V && a.status) {
        set_status(a.status, MOE_STATUS_BAD_TOKEN);
      }
      a.logprob[t] = lp;
    }
  }
  if (lane < a.n_top) {
    const float z = order_value((uint32_t)(top >> 32));
    a.top_ids[(size_t)t * a.n_top + lane] = (int32_t)(0xffffffffu - (uint32_t)top);
    a.top_logprobs[(size_t)t * a.n_top + lane] = empty ? -INFINITY : (z - st.m) - ll;
  }
}

}  // namespace

// grid (T, ceil(W / waves of a block)): a wave takes one chunk of one row.
template <bool BF16>
__global__ __launch_bounds__(256) void logprob_chunk_kernel(LogprobArgs a) {
  __shared__ u64 cand[4][kCand];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x, w = blockIdx.y * (blockDim.x >> 6) + wv;
  if (w >= a.W) return;
  const Row r = row_of<BF16>(a, t);
  uint4 raw[kMaxWords];
  float z[kPerLane];
  load_chunk<BF16>(r, w, lane, raw);
  unpack_chunk<BF16>(r, w, lane, raw, z);
  const float lane_max = max_of(z);
  Stats st = {-INFINITY, 0.0f, 0.0f};
  add_chunk(z, lane_max, st);
  const float l = wave_sum_dpp(st.l), s = wave_sum_dpp(st.s);
  const size_t part = (size_t)t * a.W + w;
  if (lane == 0) a.pm[part] = st.m, a.pl[part] = l, a.ps[part] = s;
  if (a.n_top == 0) return;
  Best b = {0, 0};
  select_chunk<BF16>(r, w, lane, a.n_top, !(l < INFINITY), z, lane_max, b, cand[wv]);
  // rank-major, so that the join sees every wave's best first
  if (lane < a.n_top) a.pk[((size_t)t * a.n_top + lane) * a.W + w] = b.top;
}

// One block of NW waves per row: joins its chunks' sums and candidates.
template <bool BF16, int NW>
__global__ __launch_bounds__(64 * NW) void logprob_join_kernel(LogprobArgs a) {
  __shared__ float sm[3 * NW];
  __shared__ u64 sk[NW][64];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const size_t p0 = (size_t)t * a.W;
  Stats st = {-INFINITY, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < a.W; i += 64 * NW) st.m = fmaxf(st.m, a.pm[p0 + i]);
  st.m = wave_max(st.m);
  for (int i = threadIdx.x; i < a.W; i += 64 * NW)
    add_part(a.pm[p0 + i], a.pl[p0 + i], a.ps[p0 + i], st.m, st.l, st.s);
  Best b = {0, 0};
  const int total = a.n_top * a.W;
  const u64* pk = a.pk + (size_t)t * total;
  if (a.n_top == 1) {
    for (int i = threadIdx.x; i < total; i += 64 * NW) b.top = b.top > pk[i] ? b.top : pk[i];
    b.top = wave_largest(b.top);
    if (lane) b.top = 0;
  } else if (a.n_top) {
    for (int i = wv * 64; i < total; i += 64 * NW) {
      u64 c = i + lane < total ? pk[i + lane] : 0;
      if (c <= b.thr) c = 0;
      if (!__ballot(c != 0)) continue;
      b.top = wave_merge(b.top, wave_sort(c, lane), lane);
      b.thr = lane64(b.top, a.n_top - 1);
    }
  }
  join_waves<NW>(st, b.top, a.n_top, lane, wv, sm, sk);
  if (wv == 0) write_row<BF16>(a, t, lane, st, b.top);
}

// One block per row, its four waves walking the chunks.
template <bool BF16>
__global__ __launch_bounds__(256) void logprob_row_kernel(LogprobArgs a) {
  __shared__ u64 cand[4][kCand];
  __shared__ float sm[12];
  __shared__ u64 sk[4][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x;
  const Row r = row_of<BF16>(a, t);
  Stats st = {-INFINITY, 0.0f, 0.0f};
  Best b = {0, 0};
  uint4 raw[kMaxWords];
  if (wv < a.W) load_chunk<BF16>(r, wv, lane, raw);
  for (int w = wv; w < a.W; w += 4) {
    float z[kPerLane];
    unpack_chunk<BF16>(r, w, lane, raw, z);
    if (w + 4 < a.W) load_chunk<BF16>(r, w + 4, lane, raw);
    const float lane_max = max_of(z);
    add_chunk(z, lane_max, st);
    if (a.n_top)
      select_chunk<BF16>(r, w, lane, a.n_top, __ballot(!(st.l < INFINITY)) != 0, z, lane_max, b,
                         cand[wv]);
  }
  join_waves<4>(st, b.top, a.n_top, lane, wv, sm, sk);
  if (wv == 0) write_row<BF16>(a, t, lane, st, b.top);
}

namespace {

template <bool BF16>
void launch_type(const LogprobArgs& a, hipStream_t st) {
  if (a.by_row) {
    logprob_row_kernel<BF16><<<a.T, 256, 0, st>>>(a);
    return;
  }
  // a wave per block while that does not fill the chip: each then has a CU's loads
  if ((int64_t)a.T * a.W <= 1024)
    logprob_chunk_kernel<BF16><<<dim3(a.T, a.W), 64, 0, st>>>(a);
  else
    logprob_chunk_kernel<BF16><<<dim3(a.T, (a.W + 3) / 4), 256, 0, st>>>(a);
  if (a.W * (a.n_top ? a.n_top : 1) <= 256)
    logprob_join_kernel<BF16, 1><<<a.T, 64, 0, st>>>(a);
  else
    logprob_join_kernel<BF16, 16><<<a.T, 1024, 0, st>>>(a);
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t st) {
  if (bf16)
    launch_type<true>(a, st);
  else
    launch_type<false>(a, st);
  return hipGetLastError();
}

}  // namespace bef
