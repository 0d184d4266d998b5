// w4.hip -- y[t][n] = sum_k x[t][k] w[n][k] with 4-bit weights and group
// scales, for few tokens: the projections around the expert layer.
//
// Codes become bf16 exactly and meet the bf16 activations in instructions
// that accumulate in fp32 (v_dot2_f32_bf16, bf16 MFMA), so no weight and no
// activation is rounded; group scales are applied to fp32 sums, except
// where a power-of-two scale goes exactly into the conversion:
//   FP4   w = e2m1(code) 2^(b-127): v_cvt_scalef32_pk_bf16_fp4;
//   INT4  w = s (code - z): a byte holding a code 0..15 IS the E4M3 value
//         code 2^-9 (subnormals 0..7, then the first binade 8..15, one
//         spacing), so v_cvt_scalef32_pk_bf16_fp8 with scale 2^9 converts
//         two codes; sum s (code - z) x = s (sum code x - z sum x).
//
// A lane owns a chunk of 32 weights (one 16-byte load), within one
// scale group in both formats.
//
// Bound by the weights' bytes where there are many: 131072 x 4096 FP4, 285 MB, in
// 47 us for one token and 66 us for 32 tokens (4.3 TB/s).  Small products are bound
// by latency: 4096 x 4096 FP4, one token, 3.9 us, where reading 9 MB takes 3.4.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace bef {

namespace {

typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t as_u32(bf2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float dot2bf(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2_t, a),
                                         __builtin_bit_cast(bf2_t, b), c, false);
}

// 2^(b-127) as the conversions take it (only the exponent field counts; 255
// is NaN in both readings).
__device__ __forceinline__ float ue8m0_operand(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : b << 23);
}

// Eight codes of one dword -> four bf16 pairs.  FP4: element pairs (0,1),
// (2,3), (4,5), (6,7).  INT4: (0,2), (4,6), (1,3), (5,7); pair_order puts
// activations into the same order.
template <bool INT4>
__device__ __forceinline__ void codes8(uint32_t w, float scale, uint32_t (&p)[4]) {
  if constexpr (!INT4) {
    p[0] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    p[1] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    p[2] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    p[3] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  } else {
    const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
    p[0] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
    p[1] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
    p[2] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
    p[3] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  }
}

template <bool INT4>
__device__ __forceinline__ uint4 pair_order(const uint4 x) {
  if constexpr (!INT4) return x;
  return make_uint4(__builtin_amdgcn_perm(x.y, x.x, 0x05040100u),   // (0, 2)
                    __builtin_amdgcn_perm(x.w, x.z, 0x05040100u),   // (4, 6)
                    __builtin_amdgcn_perm(x.y, x.x, 0x07060302u),   // (1, 3)
                    __builtin_amdgcn_perm(x.w, x.z, 0x07060302u));  // (5, 7)
}

__device__ __forceinline__ void store_y(const W4Args& a, int t, int n, float v) {
  if (a.y_bf16)
    reinterpret_cast<uint16_t*>(a.y)[(size_t)t * a.y_stride + n] =
        (uint16_t)f32x2_to_bf16x2(v, 0.0f);
  else
    reinterpret_cast<float*>(a.y)[(size_t)t * a.y_stride + n] = v;
}

// The values of the first N = 1, 2 or 4 lane groups in every lane, in group order.
template <int N>
__device__ __forceinline__ void spread(float v, float* r) {
  const uint32_t u = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  if constexpr (N == 1) {
    r[0] = v;  // every group has it
  } else if constexpr (N == 2) {
    const auto lo = __builtin_amdgcn_permlane16_swap(b[0], b[0], false, false);
    r[0] = __uint_as_float(lo[0]), r[1] = __uint_as_float(lo[1]);
  } else {
    const auto lo = __builtin_amdgcn_permlane16_swap(b[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(b[1], b[1], false, false);
    r[0] = __uint_as_float(lo[0]), r[1] = __uint_as_float(lo[1]);
    r[2] = __uint_as_float(hi[0]), r[3] = __uint_as_float(hi[1]);
  }
}

// Dword i of lane group g <-> dword g of lane group i.
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
  const auto s0 = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  const auto s1 = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  const auto s2 = __builtin_amdgcn_permlane16_swap(s0[0], s1[0], false, false);
  const auto s3 = __builtin_amdgcn_permlane16_swap(s0[1], s1[1], false, false);
  d[0] = s2[0], d[1] = s2[1], d[2] = s3[0], d[3] = s3[1];
}

// Workgroup barrier after this wave's LDS accesses; global loads stay in
// flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace

// ---- a token or a few: one wave per R rows on the vector unit --------------
// Lane l owns chunk l + 64 i of every row; R rows' loads of a pass are in
// flight together; T tokens' sums per row.
template <bool INT4, int TT, int R>
__global__ __launch_bounds__(256) void w4_gemv_kernel(W4Args a) {
  const int lane = threadIdx.x & 63;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * R;
  if (n0 >= a.N) return;
  const int nch = a.K >> 5;
  const int gsh = a.group_shift - 5;  // chunks per group, log2
  float acc[R][TT] = {};
  for (int c0 = 0; c0 < nch; c0 += 64) {
    // chunks past the end are clamped into the row and meet activations of 0
    const bool in = c0 + lane < nch;
    const int ch = in ? c0 + lane : nch - 1;
    uint4 w[R];
    uint32_t sc[R], zp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const size_t n = min(n0 + r, a.N - 1);
      w[r] = *reinterpret_cast<const uint4*>(a.q + n * (a.K >> 1) + 16 * ch);
      if constexpr (INT4) {
        const size_t at = n * a.n_groups + (ch >> gsh);
        sc[r] = reinterpret_cast<const uint16_t*>(a.scale)[at];
        zp[r] = a.zero ? a.zero[at] : 8u;
      } else {
        sc[r] = reinterpret_cast<const uint8_t*>(a.scale)[n * nch + ch];
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint16_t* xr = a.x + (size_t)min(t, a.T - 1) * a.x_stride + 32 * ch;
      uint4 x[4];
      float xsum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = *reinterpret_cast<const uint4*>(xr + 8 * i);
        if (!in) x[i] = make_uint4(0, 0, 0, 0);
        x[i] = pair_order<INT4>(x[i]);
        if constexpr (INT4) {
          constexpr uint32_t one = 0x3f803f80u;
          xsum = dot2bf(x[i].x, one, xsum);
          xsum = dot2bf(x[i].y, one, xsum);
          xsum = dot2bf(x[i].z, one, xsum);
          xsum = dot2bf(x[i].w, one, xsum);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t ww[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
        float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[4];
          codes8<INT4>(ww[i], 1.0f, p);
          d0 = dot2bf(p[0], x[i].x, d0);
          d1 = dot2bf(p[1], x[i].y, d1);
          d0 = dot2bf(p[2], x[i].z, d0);
          d1 = dot2bf(p[3], x[i].w, d1);
        }
        float d = d0 + d1;
        if constexpr (INT4) {
          d = fmaf(-(float)zp[r], xsum, d);
          acc[r][t] = fmaf(bf16_to_f32(sc[r]), d, acc[r][t]);
        } else {
          acc[r][t] += sc[r] == 255u ? __uint_as_float(0x7fc00000u) : scale_ue8m0(d, sc[r]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float s = wave_sum_dpp(acc[r][t]);
      if (lane == r * TT + t && n0 + r < a.N && t < a.T) store_y(a, t, n0 + r, s);
    }
}

// ---- more tokens: matrix cores ---------------------------------------------
// A block (8 waves) walks over tiles of 16 rows for TT x 16 tokens.  K is dealt
// out over the waves, S steps of 128 each (and passes of 8 S steps where K is
// longer): a wave keeps the activations of its steps in registers for all of
// its tiles, so the loop streams weights only, straight from memory into
// registers, the next tile's while this one multiplies.  The eight partial
// sums of a tile meet in LDS.
//
// v_mfma_f32_16x16x32_bf16 with the tokens as A (lane: token l%16) and the
// weights as B (lane: row l%16): a lane's scales are its own row's, and a
// result has 16 consecutive outputs of a token in 16 lanes.  In a step, lane
// group g = l/16 loads chunk 4 q + g of its row (64 consecutive bytes a row).
//   FP4: product i of the step takes dword i of every group, so its 32 columns
//   are codes 8i.. of four chunks, each converted with its own scale.
//   INT4: dwords are transposed over the groups first (dword i of group g <->
//   dword g of group i, four swaps), so that product i holds chunk 4 q + i
//   alone: products of one scale group add up in the matrix core, then
//   acc += s (sum code x) - (s z) (sum x), with the sums of x in LDS.
constexpr int kW4Waves = 8;
constexpr int kW4PassTiles = 16;  // tiles whose sums are kept over the passes

// DEPTH tiles of weights are in flight per wave (8 KB per tile and wave at
// K = 4096).  A step's scales are fetched once for the four lane groups: group
// g loads the words of entry 4 r + g of the pass's list (FP4: the four scale
// bytes of a step; INT4: a scale and a zero point), row swaps hand them round.
// WHOLE: K is a multiple of 128, so every step is whole (one lane offset for all
// weight loads; FP4: a step's four scale bytes are one aligned dword);
// otherwise chunks are clamped into the row one by one.
// MANY: a block has 2 DEPTH tiles or more, see the loop over them (as a variant of its
// own, because its code makes short calls longer: 4096 x 4096 FP4, 4 tokens, 6.2 us
// without it, 6.4 with; 32768 rows, 32 tokens, 26.4 us without it, 25.1 with).
template <bool INT4, int S, int TT, int NG, int DEPTH, bool WHOLE, bool MANY>
__global__ __launch_bounds__(64 * kW4Waves, kW4Waves / 4) void w4_mfma_kernel(W4Args a) {
  constexpr int NW = kW4Waves;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16 * TT;
  const int nch = a.K >> 5, nq = (nch + 3) >> 2;
  const int passes = (nq + NW * S - 1) / (NW * S);
  const int tiles = (a.N + 15) >> 4;
  // neighbouring tiles on one XCD (blocks are dealt out over the eight in turn, the
  // first gridDim.x % 8 of them getting one more): a line of y, four tiles of a token, is
  // put together in one L2 (129280 rows, 253 blocks, FP4, 8 tokens: 54.9 us, 56.9 with
  // tiles in block order)
  const int xcd = blockIdx.x & 7;
  const int first = xcd * (int)(gridDim.x >> 3) + min(xcd, (int)(gridDim.x & 7)) +
                    (int)(blockIdx.x >> 3);
  const int mine = first < tiles ? (tiles - first + gridDim.x - 1) / gridDim.x : 0;
  __shared__ float red[2][NW][TT * 4][64];
  __shared__ float keep[kW4PassTiles][TT * 256];
  __shared__ v4f_t xsum[INT4 ? NW : 1][S][NG][4 * TT];

  // NG scale groups in a step: 4, 2, 1 for groups of 32, 64, 128
  constexpr int NE = INT4 ? S * NG : S;                   // entries of a pass
  constexpr int NR = INT4 || WHOLE ? (NE + 3) / 4 : S;    // words per lane
  constexpr int NWO = WHOLE ? 1 : S;
  // (without zero points, bytes of the scales are loaded in their place, from lines
  // that are fetched anyway: no load is conditional)
  const uint8_t* zero = a.zero ? a.zero : reinterpret_cast<const uint8_t*>(a.scale);
  const int zsh = a.zero ? 0 : 1;
  struct Tile {
    u4_t w[S];
    // (as loaded: widened at once, they would be waited for at once)
    std::conditional_t<INT4, uint16_t, uint32_t> sc[NR];
    uint8_t zp[INT4 ? NR : 1];
  };
  // first row of this block's tile `it`: the last tile of the matrix ends at its
  // last row (rows it shares with the one before are computed twice, alike);
  // fewer than 16 rows: lanes past the last repeat it
  const int cr = min(c, a.N - 1);
  auto first_row = [&](int it) {
    return max(0, min((int)(first + it * gridDim.x) * 16, a.N - 16));
  };
  const int group_tiles = passes == 1 ? mine : kW4PassTiles;
  int buf = 0;
  for (int it0 = 0; it0 < mine; it0 += group_tiles) {
    const int n_it = min(group_tiles, mine - it0);
    for (int p = 0; p < passes; ++p) {
      // the wave's steps q0 .. q0 + S - 1; past the end of K it repeats the last
      // ones (loads stay inside the row) against activations of 0
      const int q1 = (p * NW + wv) * S, q0 = min(q1, nq - S);
      // lane offsets from the tile's first row: the same for every tile
      uint32_t wo[WHOLE ? 1 : S], so[NR];
      if constexpr (WHOLE) {
        wo[0] = (uint32_t)cr * (a.K >> 1) + 64 * q0 + 16 * g;
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i)
          wo[i] = (uint32_t)cr * (a.K >> 1) + 16 * min(4 * (q0 + i) + g, nch - 1);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if constexpr (INT4)
          so[r] = (uint32_t)cr * a.n_groups + min(NG * q0 + min(4 * r + g, NE - 1), a.n_groups - 1);
        else if constexpr (WHOLE)
          so[r] = 4 * ((uint32_t)cr * nq + q0 + min(4 * r + g, NE - 1));
        else
          so[r] = (uint32_t)cr * nch + min(4 * (q0 + r) + g, nch - 1);
      }
      auto load_tile = [&](int it, Tile& t) {
        const size_t n0 = first_row(it0 + it);
        const uint8_t* wb = a.q + n0 * (a.K >> 1);
        // (lane offsets made opaque: tile base in scalar registers + one 32-bit
        // offset, instead of a 64-bit address per load kept over the loop)
        uint32_t ow[NWO], os[NR];
#pragma unroll
        for (int i = 0; i < NWO; ++i) {
          ow[i] = wo[i];
          asm volatile("" : "+v"(ow[i]));
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          os[r] = so[r];
          asm volatile("" : "+v"(os[r]));
        }
#pragma unroll
        for (int i = 0; i < S; ++i)
          t.w[i] = *reinterpret_cast<const u4_t*>(wb + ow[i % NWO] + (WHOLE ? 64 * i : 0));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if constexpr (INT4) {
            const uint8_t* sb = reinterpret_cast<const uint8_t*>(a.scale) + n0 * a.n_groups * 2;
            t.sc[r] = *reinterpret_cast<const uint16_t*>(sb + 2 * os[r]);
            t.zp[r] = (zero + (n0 * a.n_groups << zsh))[os[r] << zsh];
          } else if constexpr (WHOLE) {
            const uint8_t* sb = reinterpret_cast<const uint8_t*>(a.scale) + n0 * nch;
            t.sc[r] = *reinterpret_cast<const uint32_t*>(sb + os[r]);
          } else {
            t.sc[r] = (reinterpret_cast<const uint8_t*>(a.scale) + n0 * nch)[os[r]];
          }
        }
      };
      Tile ring[DEPTH];
#pragma unroll
      for (int d = 0; d < DEPTH; ++d)
        if (d < n_it) load_tile(d, ring[d]);
      uint4 x[S][4][TT];
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ch = 4 * (q0 + i) + (INT4 ? j : g);
          const int k = 32 * min(ch, nch - 1) + 8 * (INT4 ? g : j);
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const int tok = min(t0 + 16 * t + c, a.T - 1);
            uint4 v = *reinterpret_cast<const uint4*>(a.x + (size_t)tok * a.x_stride + k);
            if (ch >= nch || q0 + i < q1) v = make_uint4(0, 0, 0, 0);
            x[i][j][t] = pair_order<INT4>(v);
          }
        }
      if constexpr (INT4) {
        // sums of x by group: the product with ones, every column alike
        uint32_t one[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        const v4f_t z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S; ++i) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
              v4f_t d = z;
#pragma unroll
              for (int j = n * 4 / NG; j < (n + 1) * 4 / NG; ++j)
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, x[i][j][t]),
                                                            __builtin_bit_cast(bf8_t, one), d, 0, 0,
                                                            0);
              if (c == 0) xsum[wv][i][n][4 * t + g] = d;
            }
        }
      }
      // joins the partial sums of the pass's tile `it` in the half just written.
      // te: token tile and element, at most TT x 4 / NW (rounded up) a wave
      constexpr int NTE = (4 * TT + NW - 1) / NW;
      auto read_partials = [&](float (&rv)[NTE][NW]) {
#pragma unroll
        for (int i = 0; i < NTE; ++i)
          if (wv + NW * i < 4 * TT)
#pragma unroll
            for (int w = 0; w < NW; ++w) rv[i][w] = red[buf ^ 1][w][wv + NW * i][lane];
      };
      auto join = [&](int it, const float (&rv)[NTE][NW]) {
#pragma unroll
        for (int i = 0; i < NTE; ++i) {
          const int te = wv + NW * i;
          if (te >= 4 * TT) break;
          const int slot = 64 * te + lane;
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < NW; ++w) v += rv[i][w];
          if (p) v += keep[it % kW4PassTiles][slot];
          if (p + 1 < passes) {
            keep[it % kW4PassTiles][slot] = v;
          } else {
            const int tok = t0 + 16 * (te >> 2) + 4 * g + (te & 3);
            const int n = first_row(it0 + it) + c;
            if (tok < a.T && n < a.N) store_y(a, tok, n, v);
          }
        }
      };
      int pending = -1;  // tile whose partial sums wait in LDS
      float rv[NTE][NW];
      auto step = [&](auto more, int it, Tile& cur) {
        constexpr bool MORE = decltype(more)::value;
        // the last tile's partial sums arrive while this one multiplies
        if (pending >= 0) read_partials(rv);
        // an offset the compiler cannot see through, or it keeps all the sums
        // of x in registers over the tiles (and spills)
        int xo = g;
        asm volatile("" : "+v"(xo));
        // FP4: the pass's scales, in every lane group
        float gs[INT4 ? 4 : S < 4 ? 4 : S], gz[4];
        if constexpr (!INT4 && WHOLE) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            spread<(NE < 4 ? NE : 4)>(__uint_as_float(cur.sc[r]), &gs[4 * r]);
#pragma unroll
          for (int i = 0; i < S; ++i)
            gs[i] = ue8m0_operand((__float_as_uint(gs[i]) >> (8 * g)) & 255u);
        } else if constexpr (!INT4) {
#pragma unroll
          for (int i = 0; i < S; ++i) gs[i] = ue8m0_operand(cur.sc[i]);
        }
        // FP4: 6 x 2^126 and more is past bf16.  A row with such a scale is converted at a
        // quarter and its sums, of this lane's row alone, are multiplied by 4 again.
        bool large = false;
        float back = 1.0f;
        if constexpr (!INT4) {
          float top = gs[0];
#pragma unroll
          for (int i = 1; i < S; ++i) top = fmaxf(top, gs[i]);
          large = __ballot(top >= 0x1p126f) != 0;
          if (large) {
            top = fmaxf(top, xchg16(top));  // over the row's lane groups
            top = fmaxf(top, xchg32(top));
            if (top >= 0x1p126f) {
              back = 4.0f;
#pragma unroll
              for (int i = 0; i < S; ++i) gs[i] *= 0.25f;
            }
          }
        }
        v4f_t acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = v4f_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if constexpr (!INT4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t pr[4];
              codes8<false>(cur.w[i][j], gs[i], pr);
#pragma unroll
              for (int t = 0; t < TT; ++t)
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf8_t, x[i][j][t]), __builtin_bit_cast(bf8_t, pr), acc[t],
                    0, 0, 0);
            }
          } else {
            // steps in order: without this their operands are formed at once and
            // spill
            __builtin_amdgcn_sched_barrier(0);
            constexpr int per = 4 / NG;  // steps per word
            if (i % per == 0) {
              const float sc = bf16_to_f32(cur.sc[i / per]);
              spread<(NE < 4 ? NE : 4)>(sc, gs);
              const float z = a.zero ? (float)cur.zp[i / per] : 8.0f;
              spread<(NE < 4 ? NE : 4)>(sc * z, gz);  // exact: 8 x 8 bits
            }
            uint32_t w[4] = {cur.w[i][0], cur.w[i][1], cur.w[i][2], cur.w[i][3]};
            transpose4(w);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              v4f_t dd[TT];
#pragma unroll
              for (int t = 0; t < TT; ++t) dd[t] = v4f_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = n * 4 / NG; j < (n + 1) * 4 / NG; ++j) {
                uint32_t pr[4];
                codes8<true>(w[j], 1.0f, pr);
#pragma unroll
                for (int t = 0; t < TT; ++t)
                  dd[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                      __builtin_bit_cast(bf8_t, x[i][j][t]), __builtin_bit_cast(bf8_t, pr), dd[t],
                      0, 0, 0);
              }
#pragma unroll
              for (int t = 0; t < TT; ++t) {
                const v4f_t xs = xsum[wv][i][n][4 * t + xo];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  acc[t][e] = fmaf(gs[(NG * i + n) % 4], dd[t][e],
                                   fmaf(-gz[(NG * i + n) % 4], xs[e], acc[t][e]));
                // (here, not sunk to the end with every dd and xs kept)
                asm volatile("" : "+v"(acc[t]));
              }
            }
          }
        }
        if (MORE || it + DEPTH < n_it) load_tile(it + DEPTH, cur);
        if (large) {
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[t] *= back;
        }
        if (pending >= 0) join(pending, rv);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) red[buf][wv][4 * t + e][lane] = acc[t][e];
        lds_barrier();
        pending = it;
        // the other half is written next: its readers are past this barrier
        buf ^= 1;
      };
      int itd = 0;
      // While every tile has a successor to load, no load is conditional, so the waits
      // leave the younger tiles' loads in flight (131072 rows, INT4, 16 tokens: 59.6 us;
      // with conditional loads each tile waits for all: 70.4).  What came before, the
      // activations, is waited for here, or it would be at every tile.
      if (MANY && 2 * DEPTH <= n_it) {
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        do {
#pragma unroll
          for (int d = 0; d < DEPTH; ++d) step(std::true_type{}, itd + d, ring[d]);
          itd += DEPTH;
        } while (itd + 2 * DEPTH <= n_it);
      }
      for (; itd < n_it; itd += DEPTH)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          if (itd + d >= n_it) break;
          step(std::false_type{}, itd + d, ring[d]);
        }
      if (pending >= 0) {
        read_partials(rv);
        join(pending, rv);
      }
    }
  }
}

namespace {

template <bool INT4, int S, int TT, int NG, int DEPTH>
void launch_tiles(const W4Args& a, hipStream_t st) {
  // One block per CU walks its tiles: its waves hold the activations once.  With few
  // tiles a block, as many blocks as share them evenly: fewer read the activations (6144
  // rows, FP4, 64 tokens: 23.3 us with 192 blocks of two tiles, 25.1 with 256), unless
  // too few CUs would be left (4352 rows of 2048, 4 tokens: 5.5 us with 136, 5.3 with 256).
  const int tiles = (a.N + 15) / 16, rounds = (tiles + 255) / 256;
  const int even = (tiles + rounds - 1) / rounds;
  const dim3 grid(tiles <= 256 ? tiles : even >= 160 ? even : 256,
                  (a.T + 16 * TT - 1) / (16 * TT));
  const bool whole = a.K % 128 == 0, many = tiles >= 2 * DEPTH * 256;
  if (whole && many)
    w4_mfma_kernel<INT4, S, TT, NG, DEPTH, true, true><<<grid, 64 * kW4Waves, 0, st>>>(a);
  else if (whole)
    w4_mfma_kernel<INT4, S, TT, NG, DEPTH, true, false><<<grid, 64 * kW4Waves, 0, st>>>(a);
  else if (many)
    w4_mfma_kernel<INT4, S, TT, NG, DEPTH, false, true><<<grid, 64 * kW4Waves, 0, st>>>(a);
  else
    w4_mfma_kernel<INT4, S, TT, NG, DEPTH, false, false><<<grid, 64 * kW4Waves, 0, st>>>(a);
}

template <bool INT4, int TT, int NG>
void launch_steps(const W4Args& a, hipStream_t st) {
  // steps a wave keeps: the fewest of 1, 2, 4 that hold K in one pass (two for
  // many scales and two token tiles, whose registers four would not fit)
  constexpr int MOST = TT == 4 || (INT4 && TT == 2 && NG == 4) ? 2 : 4;
  if (a.K <= 1024)
    launch_tiles<INT4, 1, TT, NG, TT == 4 ? 3 : 4>(a, st);
  else if (a.K <= 2048)
    launch_tiles<INT4, 2, TT, NG, TT == 4 ? 3 : 4>(a, st);
  else
    launch_tiles<INT4, MOST, TT, NG, TT == 1 ? 4 : 3>(a, st);
}

template <bool INT4, int NG>
void launch_groups(const W4Args& a, hipStream_t st) {
  // One token on the vector unit: 2 rows a wave, 4 from 16384 rows on, where
  // there are waves enough (131072 x 4096 FP4: 50.0 us with 2, 47.1 with 4;
  // 4096 x 4096: 4.15 with 2, 4.73 with 4).  Two tokens too while rows are few
  // (4096 x 4096 FP4: 5.1 us, 5.7 on the matrix cores; 131072 rows: 60.3 and 48.4).
  if (a.T == 1 && a.N >= 16384) {
    w4_gemv_kernel<INT4, 1, 4><<<(a.N + 15) / 16, 256, 0, st>>>(a);
  } else if (a.T == 1) {
    w4_gemv_kernel<INT4, 1, 2><<<(a.N + 7) / 8, 256, 0, st>>>(a);
  } else if (a.T == 2 && a.N < 16384) {
    w4_gemv_kernel<INT4, 2, 2><<<(a.N + 7) / 8, 256, 0, st>>>(a);
  } else if (a.T <= 16) {
    launch_steps<INT4, 1, NG>(a, st);
  } else if (a.T <= 32) {
    launch_steps<INT4, 2, NG>(a, st);
  } else {
    launch_steps<INT4, 4, NG>(a, st);
  }
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t st) {
  if (!a.int4)
    launch_groups<false, 1>(a, st);
  else if (a.group_shift == 5)
    launch_groups<true, 4>(a, st);
  else if (a.group_shift == 6)
    launch_groups<true, 2>(a, st);
  else
    launch_groups<true, 1>(a, st);
  return hipGetLastError();
}

}  // namespace bef
