// lora.hip -- low-rank adapters of many requests beside a projection that they share:
//   y[t] = base[t] + s_i B_i (A_i x[t]),  i = adapter_of[t].
//
// Two kernels: h = A_i x in parts of the columns of x (fp32, in the workspace), then y =
// base + s_i B_i h, where the parts are added up.  Both take tiles of 16 tokens with
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
#include <string.h>

#include "common.h"
#include "kernels.h"

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

// h: grid (parts, tiles of 16 tokens, slots).  A wave takes 32 S columns at a time, of
// which x stays in registers for all the tile's adapters and their ranks; adapters of the
// tile are dealt out over the slots.
template <int S>
__global__ __launch_bounds__(64 * kWaves) void lora_h_kernel(LoraArgs a) {
  __shared__ float red[kWaves][4][4][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16;
  bool bad = false;
  const int id = adapter_at(a, t0, c, bad);
  if (a.status && bad && blockIdx.x == 0 && blockIdx.z == 0 && wv == 0)
    set_status(a.status, MOE_STATUS_BAD_INDEX);
  const int k_lo = blockIdx.x * a.part_cols, k_hi = min(a.K, k_lo + a.part_cols);
  const int passes = (k_hi - k_lo + 256 * S - 1) / (256 * S);
  const uint16_t* xr = a.x + (size_t)min(t0 + c, a.T - 1) * a.x_stride;
  uint4 x[S];
  // (columns past the end: 0 on both sides)
  auto column = [&](int p, int s) { return k_lo + ((p * kWaves + wv) * S + s) * 32 + 8 * g; };
  auto load_x = [&](int p) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = column(p, s);
      x[s] = *reinterpret_cast<const uint4*>(xr + min(k, a.K - 8));
      if (k >= k_hi) x[s] = make_uint4(0, 0, 0, 0);
    }
  };
  if (passes == 1) load_x(0);

  uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
  for (int slot = 0; left; ++slot) {
    const int i = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t mine = (uint32_t)__ballot(id == i) & 0xffffu;
    left &= ~mine;
    if (slot % (int)gridDim.z != (int)blockIdx.z) continue;
    const int rank = rank_of(a, i);
    const uint16_t* wa = a.a + (size_t)i * a.R * a.K;
    for (int r0 = 0; r0 < a.R; r0 += 64) {  // four tiles of 16 ranks
      v4f_t acc[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) acc[rt] = v4f_t{0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < passes; ++p) {
        if (passes > 1) load_x(p);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
          if (r0 + 16 * rt < rank) {
            const uint16_t* row = wa + (size_t)min(r0 + 16 * rt + c, rank - 1) * a.K;
            uint4 w[S];
#pragma unroll
            for (int s = 0; s < S; ++s) {
              const int k = column(p, s);
              w[s] = *reinterpret_cast<const uint4*>(row + min(k, a.K - 8));
              if (k >= k_hi) w[s] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int s = 0; s < S; ++s) acc[rt] = mfma(w[s], x[s], acc[rt]);
          }
      }
      // the waves' sums, four consecutive ranks of a token a thread
      __syncthreads();
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
        if (r0 + 16 * rt < rank)
#pragma unroll
          for (int e = 0; e < 4; ++e) red[wv][rt][e][lane] = acc[rt][e];
      __syncthreads();
      const int tok = threadIdx.x >> 4, rt = (threadIdx.x >> 2) & 3, q = threadIdx.x & 3;
      const int r = r0 + 16 * rt + 4 * q;
      if (threadIdx.x < 256 && (mine >> tok & 1u) && r < a.R) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < rank)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v[e] += red[w][rt][e][16 * q + tok];
        *reinterpret_cast<float4*>(a.h + ((size_t)blockIdx.x * a.T + t0 + tok) * a.R + r) =
            make_float4(v[0], v[1], v[2], v[3]);
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

template <bool BF16>
__device__ __forceinline__ void load16(const void* p, size_t at, float (&v)[16]) {
  if constexpr (BF16) {
    uint32_t w[8];
    memcpy(w, (const uint16_t*)p + at, sizeof w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_to_f32(w[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    memcpy(v, (const float*)p + at, sizeof v);
  }
}

}  // namespace

// y: grid (64 outputs a wave, tiles of 16 tokens, slots).  MODE: how many times 8 ranks the
// k axis holds before it starts over with the next part of h: 1, 2 or 4 (NB blocks of 32
// ranks).  Row m of product i is output n0 + 16 (m / 4) + 4 i + m % 4, so that a lane ends
// with 16 consecutive outputs of its token.
template <int MODE, int NB, bool BF16>
__global__ __launch_bounds__(256) void lora_y_kernel(LoraArgs a) {
  constexpr int NP = MODE == 1 ? 1 : MODE == 2 ? 2 : 3;  // products per block of ranks
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16, n0 = (blockIdx.x * 4 + wv) * 64;
  if (n0 >= a.N) return;
  bool bad;
  const int id = adapter_at(a, t0, c, bad);
  const int t = min(t0 + c, a.T - 1);
  // this lane's outputs n.. n + 15
  const int n = n0 + 16 * g;
  const bool whole = n + 16 <= a.N;
  float v0[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v0[j] = 0.0f;
  if (a.base) {
    const size_t at = (size_t)t * a.base_stride + n;
    if (whole) {
      load16<BF16>(a.base, at, v0);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (n + j < a.N)
          v0[j] = BF16 ? bf16_to_f32(((const uint16_t*)a.base)[at + j])
                       : ((const float*)a.base)[at + j];
    }
  }
  // h of this lane's token at its ranks, parts added up in order
  const int ro = 8 * (g & (MODE - 1));
  float h[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) h[b][e] = 0.0f;
  if (id >= 0)
    for (int p = 0; p < a.parts; ++p) {
      const float* hp = a.h + ((size_t)p * a.T + t) * a.R;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int r = 32 * b + ro;
        if (r < a.R) {
          const float4 u = *reinterpret_cast<const float4*>(hp + r);
          const float4 v = *reinterpret_cast<const float4*>(hp + r + 4);
          h[b][0] += u.x, h[b][1] += u.y, h[b][2] += u.z, h[b][3] += u.w;
          h[b][4] += v.x, h[b][5] += v.y, h[b][6] += v.z, h[b][7] += v.w;
        }
      }
    }
  const float sc = id >= 0 && a.scale ? a.scale[id] : 1.0f;
  uint4 op[NB][NP];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t p[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t q[3];
      cut3(h[b][e] * sc, q);
      p[0][e] = q[0], p[1][e] = q[1], p[2][e] = q[2];
    }
    auto pack = [&](int k) {
      return make_uint4(p[k][0] >> 16 | p[k][1], p[k][2] >> 16 | p[k][3], p[k][4] >> 16 | p[k][5],
                        p[k][6] >> 16 | p[k][7]);
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

  auto finish = [&](const v4f_t (&d)[4]) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = v0[j] + d[j >> 2][j & 3];
    const size_t at = (size_t)t * a.y_stride + n;
    if (whole) {
      if constexpr (BF16) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = f32x2_to_bf16x2(v[2 * j], v[2 * j + 1]);
        memcpy((uint16_t*)a.y + at, w, sizeof w);
      } else {
        memcpy((float*)a.y + at, v, sizeof v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (n + j < a.N) {
          if (BF16)
            ((uint16_t*)a.y)[at + j] = (uint16_t)f32x2_to_bf16x2(v[j], 0.0f);
          else
            ((float*)a.y)[at + j] = v[j];
        }
    }
  };

  uint32_t left = (uint32_t)__ballot(id >= (a.in_place ? 0 : -1)) & 0xffffu;
  for (int slot = 0; left; ++slot) {
    const int i = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(id == i);
    if (slot % (int)gridDim.z != (int)blockIdx.z) continue;
    v4f_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = v4f_t{0.f, 0.f, 0.f, 0.f};
    if (i >= 0) {
      const int rank = rank_of(a, i);
      const uint16_t* wb = a.b + (size_t)i * a.N * a.R;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (32 * b >= rank) break;
        const int r = 32 * b + ro;
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = min(n0 + 16 * (c >> 2) + 4 * k + (c & 3), a.N - 1);
          w[k] = *reinterpret_cast<const uint4*>(wb + (size_t)row * a.R + min(r, a.R - 8));
        }
        // weights past the rank may be anything
        uint32_t keep[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          keep[e] = (r + 2 * e < rank ? 0xffffu : 0u) | (r + 2 * e + 1 < rank ? 0xffff0000u : 0u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k].x &= keep[0], w[k].y &= keep[1], w[k].z &= keep[2], w[k].w &= keep[3];
#pragma unroll
          for (int p = NP - 1; p >= 0; --p) d[k] = mfma(w[k], op[b][p], d[k]);
        }
      }
    }
    if (id == i) finish(d);
  }
}

namespace {

int clamp_to(int64_t v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : (int)v; }

template <int MODE, int NB>
void launch_y(const LoraArgs& a, dim3 grid, hipStream_t st) {
  if (a.y_bf16)
    lora_y_kernel<MODE, NB, true><<<grid, 256, 0, st>>>(a);
  else
    lora_y_kernel<MODE, NB, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, hipStream_t st) {
  const int tiles = (a.T + 15) / 16, most = min(min(a.T, 16), a.n);
  const dim3 gh(a.parts, tiles, clamp_to(1024 / ((int64_t)a.parts * tiles), 1, most));
  if (a.steps == 1)
    lora_h_kernel<1><<<gh, 64 * kWaves, 0, st>>>(a);
  else if (a.steps == 2)
    lora_h_kernel<2><<<gh, 64 * kWaves, 0, st>>>(a);
  else if (a.steps == 4)
    lora_h_kernel<4><<<gh, 64 * kWaves, 0, st>>>(a);
  else
    lora_h_kernel<8><<<gh, 64 * kWaves, 0, st>>>(a);
  const int nb = (a.N + 255) / 256;
  const dim3 gy(nb, tiles, clamp_to(2048 / ((int64_t)nb * tiles), 1, min(most + 1, 16)));
  if (a.R <= 8)
    launch_y<1, 1>(a, gy, st);
  else if (a.R <= 16)
    launch_y<2, 1>(a, gy, st);
  else if (a.R <= 32)
    launch_y<4, 1>(a, gy, st);
  else if (a.R <= 64)
    launch_y<4, 2>(a, gy, st);
  else
    launch_y<4, 4>(a, gy, st);
  return hipGetLastError();
}

}  // namespace bef
