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

}  // namespace

// ---- a token or a few: one wave per R rows on the vector unit --------------
// Lane l owns chunk l + 64 i of every row; R rows' loads of a pass are in
// flight together; T tokens' sums per row, one butterfly at the end.
template <bool INT4, int TT, int R>
__global__ __launch_bounds__(256) void w4_gemv_kernel(W4Args a) {
  const int lane = threadIdx.x & 63;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * R;
  if (n0 >= a.N) return;
  const int nch = a.K >> 5;
  const int gsh = a.group_shift - 5;  // chunks per group, log2
  float acc[R][TT] = {};
  for (int c0 = 0; c0 < nch; c0 += 64) {
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
// Block: RT x 16 rows and TT x 16 tokens, the K range dealt out over 4 waves.
// v_mfma_f32_16x16x32_bf16 with the weights as A (lane: row l%16) and the
// tokens as B (lane: token l%16); lane group g = l/16 owns chunk 8i + 2g + j
// of its row (j = 0, 1), so two 16-byte loads of the four groups are 128
// consecutive bytes of a row.
template <bool INT4, int RT, int TT>
__global__ __launch_bounds__(256) void w4_mfma_kernel(W4Args a) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * TT;
  const int nch = a.K >> 5;
  const int gsh = a.group_shift - 5;
  const int steps = (nch + 7) >> 3;
  v4f_t acc[RT][TT] = {};
  const uint8_t* wrow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wrow[r] = a.q + (size_t)min(n0 + 16 * r + c, a.N - 1) * (a.K >> 1);
  const uint16_t* xrow[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xrow[t] = a.x + (size_t)min(t0 + 16 * t + c, a.T - 1) * a.x_stride;

  for (int s = wv; s < steps; s += 4) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int cg = 8 * s + 2 * g + j;
      const bool in = cg < nch;
      const int ch = in ? cg : nch - 1;
      u4_t w[RT];
      float ws[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        w[r] = *reinterpret_cast<const u4_t*>(wrow[r] + 16 * ch);
        if constexpr (!INT4)
          ws[r] = ue8m0_operand(reinterpret_cast<const uint8_t*>(
              a.scale)[(size_t)min(n0 + 16 * r + c, a.N - 1) * nch + ch]);
      }
      if constexpr (!INT4) {
        uint4 x[TT][4];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[t][i] = *reinterpret_cast<const uint4*>(xrow[t] + 32 * ch + 8 * i);
            if (!in) x[t][i] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t p[4];
            codes8<false>(w[r][i], ws[r], p);
            const bf8_t wa = __builtin_bit_cast(bf8_t, p);
#pragma unroll
            for (int t = 0; t < TT; ++t)
              acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  wa, __builtin_bit_cast(bf8_t, x[t][i]), acc[r][t], 0, 0, 0);
          }
      } else {
        // dwords of the four groups transposed (dword i of group g <-> dword
        // g of group i): product i then holds 32 codes of the one chunk
        // 8s + 2i + j, whose scale applies to its fp32 sums
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          auto s0 = __builtin_amdgcn_permlane32_swap(w[r][0], w[r][2], false, false);
          auto s1 = __builtin_amdgcn_permlane32_swap(w[r][1], w[r][3], false, false);
          auto s2 = __builtin_amdgcn_permlane16_swap(s0[0], s1[0], false, false);
          auto s3 = __builtin_amdgcn_permlane16_swap(s0[1], s1[1], false, false);
          w[r][0] = s2[0], w[r][1] = s2[1], w[r][2] = s3[0], w[r][3] = s3[1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cc = 8 * s + 2 * i + j;  // wave-uniform
          if (cc >= nch) break;
          uint4 x[TT];
          v4f_t xs[TT];
          uint32_t one[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            x[t] = pair_order<true>(*reinterpret_cast<const uint4*>(xrow[t] + 32 * cc + 8 * g));
            const v4f_t z = {0.f, 0.f, 0.f, 0.f};
            xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf8_t, one), __builtin_bit_cast(bf8_t, x[t]), z, 0, 0, 0);
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            uint32_t p[4];
            codes8<true>(w[r][i], 1.0f, p);
            float sc[4], sz[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const size_t at =
                  (size_t)min(n0 + 16 * r + 4 * g + e, a.N - 1) * a.n_groups + (cc >> gsh);
              sc[e] = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.scale)[at]);
              sz[e] = -sc[e] * (a.zero ? (float)a.zero[at] : 8.0f);  // exact: 8 x 8 bits
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
              const v4f_t z = {0.f, 0.f, 0.f, 0.f};
              const v4f_t d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf8_t, p), __builtin_bit_cast(bf8_t, x[t]), z, 0, 0, 0);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[r][t][e] = fmaf(sc[e], d[e], fmaf(sz[e], xs[t][0], acc[r][t][e]));
            }
          }
        }
      }
    }
  }
  // the four waves' sums joined in wave order
  __shared__ v4f_t red[3][RT * TT][64];
  if (wv) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) red[wv - 1][r * TT + t][lane] = acc[r][t];
  }
  __syncthreads();
  if (wv) return;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      v4f_t v = acc[r][t];
#pragma unroll
      for (int k = 0; k < 3; ++k) v += red[k][r * TT + t][lane];
      const int tok = t0 + 16 * t + c, n = n0 + 16 * r + 4 * g;
      if (tok < a.T) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) store_y(a, tok, n + e, v[e]);
      }
    }
}

namespace {

template <bool INT4>
void launch_fmt(const W4Args& a, hipStream_t st) {
  if (a.T <= 2) {
    constexpr int R = 4;
    const int grid = (a.N + 4 * R - 1) / (4 * R);
    if (a.T == 1)
      w4_gemv_kernel<INT4, 1, R><<<grid, 256, 0, st>>>(a);
    else
      w4_gemv_kernel<INT4, 2, R><<<grid, 256, 0, st>>>(a);
  } else if (a.T <= 16) {
    w4_mfma_kernel<INT4, 1, 1><<<dim3((a.N + 15) / 16, 1), 256, 0, st>>>(a);
  } else {
    w4_mfma_kernel<INT4, 2, 2><<<dim3((a.N + 31) / 32, (a.T + 31) / 32), 256, 0, st>>>(a);
  }
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t st) {
  if (a.int4)
    launch_fmt<true>(a, st);
  else
    launch_fmt<false>(a, st);
  return hipGetLastError();
}

}  // namespace bef
