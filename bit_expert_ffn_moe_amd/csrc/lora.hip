// lora.hip -- low-rank adapters of many requests beside a projection that they share:
//   y[t] = base[t] + s_i B_i (A_i x[t]),  i = adapter_of[t].
//
// Two kernels (one for a few tokens of small adapters: lora_one_kernel): h = A_i x in parts of
// the columns of x (fp32, in the workspace), then y = base + s_i B_i h, where the parts are
// added up.  Both take tiles of 16 tokens with
// v_mfma_f32_16x16x32_bf16, the adapter's weights as the first operand (lane: row l%16, 8
// consecutive k from 8 (l/16)) and the tokens as the columns of the second, so a token's
// results are a column of its own.  A tile's different adapters are multiplied in turn
// with all 16 tokens, and each token keeps its own adapter's column: nothing has to be
// sorted, weights of adapters that no token of the tile has are not read, and what one
// adapter or one token holds (NaN, infinities) does not reach another's column.
//
// x, A and B meet the matrix cores as they are, in bf16; h, which is fp32, as three bf16
// parts that add up to it exactly (8 bits each, cut off), along the k axis where the
// rank leaves room: a rank of 8 takes one instruction, 16 two, 32 three.
//
// 4096 tokens of 6 adapters in runs, 4096 x 4096, rank 32, 104 MB and 2.1 GFLOP (HBM alone: 20
// us): 39.9 us, of which h takes 14.9 (x read once, 35 MB; every block reads its adapters' A
// from L2, as many bytes as x), its operands 4.6 and y 20.2 (70 MB; every block of 64 x 64
// outputs reads its part of B and its tokens' operands from L2; the vector unit is busy 56%
// with that and base + d).  Outputs of 128 or 256 columns a block halve or quarter the
// operands' reads but leave fewer waves a SIMD: 46 and 57 us.  32 tokens of 24 adapters, ranks
// up to 64, 4096 x 6144, are a read of their weights (18.7 MB: 3.3 us): h 6.0, y 8.5, each a
// launch and three dependent trips to memory (numbers, rank and weights, result).
#include <string.h>

#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace bef {

namespace {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f_t mfma(const uint4 a, const uint4 b, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a),
                                                 __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// The adapter of token t0 + l%16: -1 none, -2 no token.
__device__ __forceinline__ int adapter_at(const LoraArgs& a, int t0, int c, bool& bad) {
  if (t0 + c >= a.T) return -2;
  const int i = a.of[t0 + c];
  bad = i >= a.n;
  return i < 0 || i >= a.n ? -1 : i;
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int i) {
  return a.rank ? max(0, min(a.rank[i], a.R)) : a.R;
}

constexpr int kWaves = 8;  // of the first kernel

}  // namespace

// h: grid (parts, tiles of 16 TT tokens, slots x groups of 32 ranks).  A wave takes 32 S
// columns at a time, of which x stays in registers for all the adapters that the block
// takes: those of its tile are dealt out over the slots, their ranks over the groups (many
// tokens: one slot, one group).
template <int S, int TT>
__global__ __launch_bounds__(64 * kWaves) void lora_h_kernel(LoraArgs a) {
  constexpr int NT = 16 * TT;
  __shared__ v4f_t red[kWaves][2][TT][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * NT;
  const int slots = a.h_slots, first_slot = blockIdx.z % slots, group = blockIdx.z / slots;
  bool bad = false;
  const int id = adapter_at(a, t0, lane & (NT - 1), bad);
  const int k_lo = blockIdx.x * a.part_cols, k_hi = min(a.K, k_lo + a.part_cols);
  const int passes = (k_hi - k_lo + 256 * S - 1) / (256 * S);
  uint4 x[TT][S];
  // (columns past the end: 0 on both sides; with slots, of the block's tokens alone)
  auto column = [&](int p, int s) { return k_lo + ((p * kWaves + wv) * S + s) * 32 + 8 * g; };
  auto load_x = [&](int p, uint32_t of) {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint16_t* xr = a.x + (size_t)min(t0 + 16 * j + c, a.T - 1) * a.x_stride;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int k = column(p, s);
        x[j][s] = make_uint4(0, 0, 0, 0);
        if (k < k_hi && (of >> (16 * j + c) & 1u)) x[j][s] = *reinterpret_cast<const uint4*>(xr + k);
      }
    }
  };
  if (passes == 1 && slots == 1) load_x(0, 0xffffffffu);
  if (a.status && bad && blockIdx.x == 0 && blockIdx.z == 0 && wv == 0)
    set_status(a.status, MOE_STATUS_BAD_INDEX);

  const uint32_t all = NT == 32 ? 0xffffffffu : 0xffffu;
  uint32_t left = (uint32_t)__ballot(id >= 0) & all;
  for (int slot = 0; left; ++slot) {
    const int i = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t mine = (uint32_t)__ballot(id == i) & all;
    left &= ~mine;
    if (slot % slots != first_slot) continue;
    const int rank = rank_of(a, i);
    const uint16_t* wa = a.a + (size_t)i * a.R * a.K;
    for (int r0 = 32 * group; r0 < a.R; r0 += 32 * a.h_groups) {  // two tiles of 16 ranks
      v4f_t acc[2][TT];
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[rt][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < (r0 && r0 >= rank ? 0 : passes); ++p) {
        if (passes > 1 || (slots > 1 && r0 == 32 * group)) load_x(p, slots > 1 ? mine : 0xffffffffu);
        // Both tiles' weights on their way together (the first ranks' do not wait for the rank's
        // number)
        uint4 w[2][S];
        const bool two = r0 + 16 < rank;
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          if (rt && !two) break;
          const uint16_t* row = wa + (size_t)min(r0 + 16 * rt + c, a.R - 1) * a.K;
#pragma unroll
          for (int s = 0; s < S; ++s) {
            const int k = column(p, s);
            w[rt][s] = make_uint4(0, 0, 0, 0);
            if (k < k_hi) w[rt][s] = *reinterpret_cast<const uint4*>(row + k);
          }
        }
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          if (rt && !two) break;
#pragma unroll
          for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int s = 0; s < S; ++s) acc[rt][j] = mfma(w[rt][s], x[j][s], acc[rt][j]);
        }
      }
      // the waves' sums, four consecutive ranks of a token a thread
      __syncthreads();
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int j = 0; j < TT; ++j) red[wv][rt][j][lane] = acc[rt][j];
      __syncthreads();
      const int rt = wv & 1, j = wv >> 1, tok = 16 * j + c, r = r0 + 16 * rt + 4 * g;
      if (j < TT && (mine >> tok & 1u) && r < a.R) {
        v4f_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += red[w][rt][j][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e >= rank) v[e] = 0.0f;
        *reinterpret_cast<v4f_t*>(a.h + ((size_t)blockIdx.x * a.T + t0 + tok) * a.R + r) = v;
      }
    }
  }
}

namespace {

// Three bf16 whose sum is v (an infinity or NaN in the first alone).
__device__ __forceinline__ void cut3(float v, uint32_t (&p)[3]) {
  p[0] = __float_as_uint(v) & 0xffff0000u;
  float d = v - __uint_as_float(p[0]);
  d = d != d ? 0.0f : d;
  p[1] = __float_as_uint(d) & 0xffff0000u;
  p[2] = __float_as_uint(d - __uint_as_float(p[1])) & 0xffff0000u;
}

// Four consecutive outputs at element `at`, which has their alignment only, as words: two of
// bf16 pairs or four of fp32.
template <bool BF16>
struct Four {
  uint32_t w[BF16 ? 2 : 4];
};
template <bool BF16>
__device__ __forceinline__ Four<BF16> load4(const void* p, size_t at) {
  Four<BF16> f;
  memcpy(f.w, (const uint8_t*)p + at * (BF16 ? 2 : 4), sizeof f.w);
  return f;
}
// y = base + d at four outputs
template <bool BF16>
__device__ __forceinline__ void store4(void* p, size_t at, const Four<BF16>& base, float d0, float d1,
                                       float d2, float d3) {
  Four<BF16> o;
  if constexpr (BF16) {
    o.w[0] = f32x2_to_bf16x2(bf16_to_f32(base.w[0] & 0xffffu) + d0,
                             __uint_as_float(base.w[0] & 0xffff0000u) + d1);
    o.w[1] = f32x2_to_bf16x2(bf16_to_f32(base.w[1] & 0xffffu) + d2,
                             __uint_as_float(base.w[1] & 0xffff0000u) + d3);
  } else {
    o.w[0] = __float_as_uint(__uint_as_float(base.w[0]) + d0);
    o.w[1] = __float_as_uint(__uint_as_float(base.w[1]) + d1);
    o.w[2] = __float_as_uint(__uint_as_float(base.w[2]) + d2);
    o.w[3] = __float_as_uint(__uint_as_float(base.w[3]) + d3);
  }
  memcpy((uint8_t*)p + at * (BF16 ? 2 : 4), o.w, sizeof o.w);
}
// the same where fewer than four are left
template <bool BF16>
__device__ __forceinline__ void store_some(const LoraArgs& a, int t, int n, const float (&d)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (n + k >= a.N) break;
    const size_t at = (size_t)t * a.y_stride + n + k, ab = (size_t)t * a.base_stride + n + k;
    float v = d[k];
    if (a.base) v += BF16 ? bf16_to_f32(((const uint16_t*)a.base)[ab]) : ((const float*)a.base)[ab];
    if (BF16)
      ((uint16_t*)a.y)[at] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
    else
      ((float*)a.y)[at] = v;
  }
}

// The first operand of the second product: h of token t (a row per lane, l%16) at the ranks
// of lane group g, parts added up in order, times the adapter's scale, cut in three along
// the k axis.  MODE: how many times 8 ranks the k axis holds before it starts over with the
// next part: 1, 2 or 4 (NB blocks of 32 ranks).
template <int MODE, int NB>
struct Rows {
  static constexpr int NP = MODE == 1 ? 1 : MODE == 2 ? 2 : 3;  // products per block of ranks
  uint4 op[NB][NP];
  __device__ __forceinline__ void load(const LoraArgs& a, int t, int g, bool mine, float sc) {
    const int ro = 8 * (g & (MODE - 1));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 32 * b + ro;
      float h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = 0.0f;
      if (mine && r < a.R)
        for (int p0 = 0; p0 < a.parts; p0 += 4) {
          float4 u[4], v[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float* hp = a.h + ((size_t)min(p0 + p, a.parts - 1) * a.T + t) * a.R + r;
            u[p] = *reinterpret_cast<const float4*>(hp), v[p] = *reinterpret_cast<const float4*>(hp + 4);
          }
#pragma unroll
          for (int p = 0; p < 4; ++p)
            if (p0 + p < a.parts) {
              h[0] += u[p].x, h[1] += u[p].y, h[2] += u[p].z, h[3] += u[p].w;
              h[4] += v[p].x, h[5] += v[p].y, h[6] += v[p].z, h[7] += v[p].w;
            }
        }
      uint32_t p[3][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t q[3];
        cut3(h[e] * sc, q);
        p[0][e] = q[0], p[1][e] = q[1], p[2][e] = q[2];
      }
      auto pack = [&](int k) {
        return make_uint4(p[k][0] >> 16 | p[k][1], p[k][2] >> 16 | p[k][3],
                          p[k][4] >> 16 | p[k][5], p[k][6] >> 16 | p[k][7]);
      };
      const uint4 zero = make_uint4(0, 0, 0, 0), p0 = pack(0), p1 = pack(1), p2 = pack(2);
      if constexpr (MODE == 1) {
        op[b][0] = g == 0 ? p0 : g == 1 ? p1 : g == 2 ? p2 : zero;
      } else if constexpr (MODE == 2) {
        op[b][0] = g < 2 ? p0 : p1;
        op[b][1] = g < 2 ? p2 : zero;
      } else {
        op[b][0] = p0, op[b][1] = p1, op[b][2] = p2;
      }
    }
  }
  // The same from a.op, where lora_op_kernel left the three parts of a token one behind the
  // other: along the k axis as well.
  __device__ __forceinline__ void load_ready(const LoraArgs& a, int t, int g) {
    const uint4* p = reinterpret_cast<const uint4*>(a.op) + (size_t)t * 3 * (a.R >> 3);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int pieces = a.R >> 3;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (MODE == 1) {
        op[b][0] = g < 3 ? p[g] : zero;
      } else if constexpr (MODE == 2) {
        op[b][0] = p[g];
        op[b][1] = g < 2 ? p[4 + g] : zero;
      } else {
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          op[b][q] = p[q * pieces + min(4 * b + g, pieces - 1)];
          if (4 * b + g >= pieces) op[b][q] = zero;
        }
      }
    }
  }
  // d[k] += products with w(b, k), the weights of output k; those past the rank may be anything
  template <class W>
  __device__ __forceinline__ void multiply(int g, int rank, W&& w, v4f_t (&d)[4]) const {
    const int ro = 8 * (g & (MODE - 1));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (32 * b >= rank) break;
      const int r = 32 * b + ro;
      uint32_t keep[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        keep[e] = (r + 2 * e < rank ? 0xffffu : 0u) | (r + 2 * e + 1 < rank ? 0xffff0000u : 0u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 x = w(b, k);
        x.x &= keep[0], x.y &= keep[1], x.z &= keep[2], x.w &= keep[3];
#pragma unroll
        for (int p = NP - 1; p >= 0; --p) d[k] = mfma(op[b][p], x, d[k]);
      }
    }
  }
};

}  // namespace

// The operands of many tokens, formed once: four ranks of a token a thread.
__global__ __launch_bounds__(256) void lora_op_kernel(LoraArgs a) {
  const int per = a.R >> 2;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(at / per), r = 4 * (int)(at % per);
  if (t >= a.T) return;
  const int id = a.of[t];
  if (id < 0 || id >= a.n) return;  // (its row of the products is not looked at)
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < a.parts; ++p) {
    const float4 u = *reinterpret_cast<const float4*>(a.h + ((size_t)p * a.T + t) * a.R + r);
    h[0] += u.x, h[1] += u.y, h[2] += u.z, h[3] += u.w;
  }
  const float sc = a.scale ? a.scale[id] : 1.0f;
  uint32_t q[4][3];
#pragma unroll
  for (int e = 0; e < 4; ++e) cut3(h[e] * sc, q[e]);
#pragma unroll
  for (int p = 0; p < 3; ++p)
    *reinterpret_cast<uint2*>(a.op + ((size_t)t * 3 + p) * a.R + r) =
        make_uint2(q[0][p] >> 16 | q[1][p], q[2][p] >> 16 | q[3][p]);
}

// y, few tokens: grid (64 outputs a wave, tiles of 16 tokens, slots).  Tokens are the rows of
// the result, output n0 + 4 (l%16) + k the column of product k: a lane ends with four
// consecutive outputs of tokens 4 (l/16) .. + 3, 16 lanes with 64 consecutive ones.
template <int MODE, int NB, bool BF16>
__global__ __launch_bounds__(256) void lora_y_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16, n0 = (blockIdx.x * 4 + wv) * 64, n = n0 + 4 * c;
  if (n0 >= a.N) return;
  bool bad;
  const int id = adapter_at(a, t0, c, bad);
  uint32_t left = (uint32_t)__ballot(id >= (a.in_place ? 0 : -1)) & 0xffffu;
  for (int slot = 0; left; ++slot) {
    const int i = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t ours = (uint32_t)__ballot(id == i) & 0xffffu;
    left &= ~ours;
    if (slot % (int)gridDim.z != (int)blockIdx.z) continue;
    Four<BF16> base[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      memset(&base[e], 0, sizeof base[e]);
      if (a.base && (ours >> (4 * g + e) & 1u) && n + 4 <= a.N)
        base[e] = load4<BF16>(a.base, (size_t)(t0 + 4 * g + e) * a.base_stride + n);
    }
    v4f_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = v4f_t{0.f, 0.f, 0.f, 0.f};
    if (i >= 0) {
      const uint16_t* wb = a.b + (size_t)i * a.N * a.R;
      const int ro = 8 * (g & (MODE - 1));
      uint4 w[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[b][k] = *reinterpret_cast<const uint4*>(wb + (size_t)min(n + k, a.N - 1) * a.R +
                                                    min(32 * b + ro, a.R - 8));
      const int rank = rank_of(a, i);
      Rows<MODE, NB> rows;
      rows.load(a, min(t0 + c, a.T - 1), g, id == i, a.scale ? a.scale[i] : 1.0f);
      rows.multiply(g, rank, [&](int b, int k) { return w[b][k]; }, d);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!(ours >> (4 * g + e) & 1u)) continue;
      const int t = t0 + 4 * g + e;
      if (n + 4 <= a.N) {
        store4<BF16>(a.y, (size_t)t * a.y_stride + n, base[e], d[0][e], d[1][e], d[2][e], d[3][e]);
      } else {
        const float v[4] = {d[0][e], d[1][e], d[2][e], d[3][e]};
        store_some<BF16>(a, t, n, v);
      }
    }
  }
}

// y, many tokens: grid (64 outputs, 64 tokens).  A wave takes 16 of the tokens; the
// adapter's weights of these outputs, which lie together in memory, come through LDS for all
// of them, their 16-byte pieces permuted by row so that the 16 lanes of a group, four
// rows apart, meet distinct banks.  What does not wait for the adapter's number (base, h) is
// loaded first, the next adapter's weights under this one's products.
//
// Five waves a SIMD suit one block of ranks (96 registers).  Two and four blocks of ranks, up to 64
// and 128, need more and keep 84 and 368 or 400 bytes a lane in scratch: 4096 tokens, 4096 x 4096,
// bf16, rank 32: 20.2 us, 64: 39.8, 128: 142.  Ranks up to 16 read their zeros through 32 bytes of it:
// rank 8 14.6, rank 16 15.8.
template <int MODE, int NB, bool BF16>
__global__ __launch_bounds__(256, 5) void lora_y_many_kernel(LoraArgs a) {
  constexpr int PR = 4 * NB;                  // pieces of a row in LDS (R / 8 of them are there)
  __shared__ uint4 lw[64 * PR];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int tb = blockIdx.y * 64, t0 = tb + 16 * wv;
  const int n0 = blockIdx.x * 64;
  bool bad;
  const int id = adapter_at(a, tb, lane, bad);  // of the block's token l
  // four outputs of four tokens; those past the last token stand in as the last
  Four<BF16> base[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    memset(&base[e], 0, sizeof base[e]);
    if (a.base && n0 + 64 <= a.N)
      base[e] = load4<BF16>(a.base, (size_t)min(t0 + 4 * g + e, a.T - 1) * a.base_stride + n0 + 4 * c);
  }
  Rows<MODE, NB> rows;
  rows.load_ready(a, min(t0 + c, a.T - 1), g);

  auto place = [](int row, int piece) { return (row * PR + piece) ^ ((row >> 2) & 15); };
  const int pieces = a.R >> 3;                // of a row in memory
  const int ro = g & (MODE - 1);
  uint4 wreg[NB];
  auto load_w = [&](int i) {
    const uint4* wb = reinterpret_cast<const uint4*>(a.b) + (size_t)i * a.N * pieces;
    const size_t from = (size_t)n0 * pieces, last = (size_t)a.N * pieces - 1;
#pragma unroll
    for (int l = 0; l < NB; ++l) {
      const size_t at = from + min(l * 256 + (int)threadIdx.x, 64 * pieces - 1);
      wreg[l] = wb[at < last ? at : last];
    }
  };
  uint64_t left = __ballot(id >= (a.in_place ? 0 : -1));
  int i = left ? __builtin_amdgcn_readlane(id, __builtin_ctzll(left)) : -1;
  if (i >= 0) load_w(i);
  while (left) {
    const uint64_t all = __ballot(id == i);
    const uint32_t ours = (uint32_t)(all >> (16 * wv)) & 0xffffu;
    left &= ~all;
    const int next = left ? __builtin_amdgcn_readlane(id, __builtin_ctzll(left)) : -1;
    if (i >= 0) {
      __syncthreads();  // (the adapter before is done with LDS)
#pragma unroll
      for (int l = 0; l < NB; ++l) {
        const int j = l * 256 + threadIdx.x;
        if (j < 64 * pieces) lw[place(j / pieces, j % pieces)] = wreg[l];
      }
      __syncthreads();
    }
    if (next >= 0) load_w(next);
    const int rank = i >= 0 ? rank_of(a, i) : 0;
    if (ours) {
      const int n = n0 + 4 * c;
      v4f_t d[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = v4f_t{0.f, 0.f, 0.f, 0.f};
      rows.multiply(g, rank, [&](int b, int k) {
        return lw[place(4 * c + k, min(4 * b + ro, pieces - 1))];
      }, d);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(ours >> (4 * g + e) & 1u)) continue;
        const int t = t0 + 4 * g + e;
        if (n0 + 64 <= a.N) {
          store4<BF16>(a.y, (size_t)t * a.y_stride + n, base[e], d[0][e], d[1][e], d[2][e], d[3][e]);
        } else {
          const float v[4] = {d[0][e], d[1][e], d[2][e], d[3][e]};
          store_some<BF16>(a, t, n, v);
        }
      }
    }
    i = next;
  }
}

// A few tokens of small adapters, in one launch: grid (512 outputs, tokens).  Every block forms
// its token's h again on the vector unit, 4096 columns of all ranks on their way at once, a wave
// 1 KB of a row of A at a time (as a matrix operand, 16 rows of 64 bytes at a time, A of
// 131 KB took 2.5 us more); rows of B and base arrive meanwhile, and an output is a
// thread's dot product with h.  P: pieces of 8 ranks.
template <int P, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void lora_one_kernel(LoraArgs a) {
  __shared__ float red[kWaves][8 * P];
  __shared__ float hs[8 * P];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t = blockIdx.y, n = blockIdx.x * 64 * kWaves + threadIdx.x;
  const int i = a.of[t];
  if (i >= a.n && a.status && blockIdx.x == 0 && threadIdx.x == 0)
    set_status(a.status, MOE_STATUS_BAD_INDEX);
  const bool has = i >= 0 && i < a.n;
  if (!has && a.in_place) return;
  const size_t at = (size_t)t * a.y_stride + n;
  float y = 0.0f;
  if (a.base && n < a.N) {
    const size_t ab = (size_t)t * a.base_stride + n;
    y = BF16 ? bf16_to_f32(((const uint16_t*)a.base)[ab]) : ((const float*)a.base)[ab];
  }
  if (has) {
    const uint4* wb = reinterpret_cast<const uint4*>(a.b) + ((size_t)i * a.N + min(n, a.N - 1)) * (a.R >> 3);
    uint4 b[P];
#pragma unroll
    for (int p = 0; p < P; ++p) b[p] = wb[min(p, (a.R >> 3) - 1)];
    const int rank = rank_of(a, i);
    const uint16_t* xr = a.x + (size_t)t * a.x_stride;
    const uint16_t* wa = a.a + (size_t)i * a.R * a.K;
    float h[8 * P];
#pragma unroll
    for (int r = 0; r < 8 * P; ++r) h[r] = 0.0f;
    for (int k = 8 * threadIdx.x; k < a.K; k += 512 * kWaves) {
      const uint4 xw = *reinterpret_cast<const uint4*>(xr + k);
      uint4 w[8 * P];
#pragma unroll
      for (int r = 0; r < 8 * P; ++r)
        w[r] = *reinterpret_cast<const uint4*>(wa + (size_t)min(r, a.R - 1) * a.K + k);
      float xf[8];
      unpack8(xw, xf);
#pragma unroll
      for (int r = 0; r < 8 * P; ++r) {
        float wf[8];
        unpack8(w[r], wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[r] = fmaf(wf[e], xf[e], h[r]);
      }
    }
    // halves, then quarters of the wave exchange two ranks' sums and keep one each
#pragma unroll
    for (int r = 0; r < 4 * P; ++r) {
      const auto z = __builtin_amdgcn_permlane32_swap(__float_as_uint(h[r]),
                                                      __float_as_uint(h[r + 4 * P]), false, false);
      h[r] = __uint_as_float(z[0]) + __uint_as_float(z[1]);
    }
#pragma unroll
    for (int r = 0; r < 2 * P; ++r) {
      const auto z = __builtin_amdgcn_permlane16_swap(__float_as_uint(h[r]),
                                                      __float_as_uint(h[r + 2 * P]), false, false);
      h[r] = __uint_as_float(z[0]) + __uint_as_float(z[1]);
    }
    // lane group g has ranks r + 2 P (g & 1) + 4 P (g >> 1)
#pragma unroll
    for (int r = 0; r < 2 * P; ++r) {
      float v = h[r];
#pragma unroll
      for (int o = 1; o < 16; o *= 2) v += __shfl_xor(v, o, 16);
      if (c == 0) red[wv][r + 2 * P * (g & 1) + 4 * P * (g >> 1)] = v;
    }
    __syncthreads();
    if (threadIdx.x < 8 * P) {
      float v = 0.0f;
#pragma unroll
      for (int u = 0; u < kWaves; ++u) v += red[u][threadIdx.x];
      hs[threadIdx.x] = v * (a.scale ? a.scale[i] : 1.0f);
    }
    __syncthreads();
    float d = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t u[4] = {b[p].x, b[p].y, b[p].z, b[p].w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * p + e < rank)
          d = fmaf(hs[8 * p + e], e & 1 ? __uint_as_float(u[e / 2] & 0xffff0000u)
                                        : bf16_to_f32(u[e / 2] & 0xffffu), d);
    }
    y += d;
  }
  if (n >= a.N) return;
  if (BF16)
    ((uint16_t*)a.y)[at] = (uint16_t)f32x2_to_bf16x2(y, 0.0f);
  else
    ((float*)a.y)[at] = y;
}

namespace {

int clamp_to(int64_t v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : (int)v; }

template <int MODE, int NB>
void launch_y(const LoraArgs& a, int slots, hipStream_t st) {
  if (a.many) {
    const dim3 grid((a.N + 63) / 64, (a.T + 63) / 64);
    if (a.y_bf16)
      lora_y_many_kernel<MODE, NB, true><<<grid, 256, 0, st>>>(a);
    else
      lora_y_many_kernel<MODE, NB, false><<<grid, 256, 0, st>>>(a);
  } else {
    const dim3 grid((a.N + 255) / 256, (a.T + 15) / 16, slots);
    if (a.y_bf16)
      lora_y_kernel<MODE, NB, true><<<grid, 256, 0, st>>>(a);
    else
      lora_y_kernel<MODE, NB, false><<<grid, 256, 0, st>>>(a);
  }
}

template <int P>
void launch_one(const LoraArgs& a, hipStream_t st) {
  const dim3 grid((a.N + 64 * kWaves - 1) / (64 * kWaves), a.T);
  if (a.y_bf16)
    lora_one_kernel<P, true><<<grid, 64 * kWaves, 0, st>>>(a);
  else
    lora_one_kernel<P, false><<<grid, 64 * kWaves, 0, st>>>(a);
}

}  // namespace

hipError_t launch_lora(const LoraArgs& args, hipStream_t st) {
  LoraArgs a = args;
  // One launch where a block's A comes faster than a second launch and there is a CU for every
  // block.  4096 x 4096, rank 16, graph replays: 1 token 4.9 us so, 7.3 in two launches, 16 tokens
  // 5.1 and 8.8, 32 (256 blocks) 7.9 and 9.0, 64 9.3 and 9.6.  14336 x 4096, rank 16, 32 tokens:
  // 12.3 and 12.6, 64 tokens 20.2 and 15.6.  Past rank 16, whose sums take twice the registers,
  // the blocks read 2^24 elements of A at most between them: 4096 x 4096, rank 32: 8 tokens 7.7
  // and 9.1, 16 (2^24) 9.6 and 9.7, 24 11.9 and 10.2, 64 17.5 and 10.1; rank 24: 16 tokens 8.9 and
  // 9.2, 24 (1.1 x 2^24) 10.6 and 9.6; 2048 x 2048, rank 32, 64 tokens (2^24) 8.7 and 10.0, 128 14.1
  // and 10.2; 8192 x 8192, rank 32, 1 token 9.3 and 8.9.
  const int64_t blocks = (int64_t)a.T * ((a.N + 64 * kWaves - 1) / (64 * kWaves));
  const int64_t of_a = (int64_t)a.R * a.K;
  if (blocks <= 256 && (a.R <= 16 ? of_a <= 1 << 18
                                  : a.R <= 32 && of_a <= 1 << 17 && blocks * of_a <= 1 << 24)) {
    if (a.R <= 8)
      launch_one<1>(a, st);
    else if (a.R <= 16)
      launch_one<2>(a, st);
    else
      launch_one<4>(a, st);
    return hipGetLastError();
  }
  const int most = a.T < 16 ? a.T : 16, different = most < a.n ? most : a.n;
  if (a.many) {
    a.h_slots = a.h_groups = 1;
    lora_h_kernel<4, 2><<<dim3(a.parts, (a.T + 31) / 32), 64 * kWaves, 0, st>>>(a);
    lora_op_kernel<<<(unsigned)(((int64_t)a.T * (a.R / 4) + 255) / 256), 256, 0, st>>>(a);
  } else {
    const int tiles = (a.T + 15) / 16;
    a.h_slots = different, a.h_groups = (a.R + 31) / 32;
    lora_h_kernel<4, 1><<<dim3(a.parts, tiles, a.h_slots * a.h_groups), 64 * kWaves, 0, st>>>(a);
  }
  const int slots = clamp_to(different + (a.in_place ? 0 : 1), 1, most);
  if (a.R <= 8)
    launch_y<1, 1>(a, slots, st);
  else if (a.R <= 16)
    launch_y<2, 1>(a, slots, st);
  else if (a.R <= 32)
    launch_y<4, 1>(a, slots, st);
  else if (a.R <= 64)
    launch_y<4, 2>(a, slots, st);
  else
    launch_y<4, 4>(a, slots, st);
  return hipGetLastError();
}

}  // namespace bef
