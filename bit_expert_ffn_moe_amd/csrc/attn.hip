// attn.hip -- attention of a batch over a paged cache whose first prefix_len
// keys are shared by every sequence:
//   o = sum_j softmax_j(scale q.k_j) v_j   over the keys j <= pos of the query.
//
// A work item is one kv head, a set of query rows (token x query head of the
// kv head's group) and a range of keys: prefix items take rows of the whole
// batch, so the prefix is read once for all of them; the other items take
// one sequence's rows over its own pages.  Every item leaves an unnormalised
// sum with its maximum and weight in the workspace and a second kernel joins
// a row's items, so long axes are split over the chip.
//
// A wave multiplies 32 keys at a time with v_mfma_f32_16x16x32_bf16, scores
// transposed: S^T = K Q^T has a query per lane column (query l%16) and the
// keys {4g..4g+3, 16+4g..16+4g+3} of the tile in lane group g = l/16.  These
// eight probabilities, rounded to bf16, are directly the B operand of
// O^T = V^T P^T when the key slots of the V operand are numbered the same way;
// softmax statistics are per lane column and need two row swaps.  The A
// operand of V^T wants 8 keys per lane at one column: a lane loads 16 bytes (8
// columns) of each of its 8 keys, coalesced, and packs them with byte
// permutes -- no LDS and no transposed copy of the cache.
//
// Scores, statistics and sums are fp32.  P is rounded to bf16 (2^-9 relative
// per key, the price of the matrix cores with bf16 V); the weights summed are
// the unrounded ones.
#include "common.h"
#include "kernels.h"

namespace bef {

namespace {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4f_t mfma(const uint4 a, const uint4 b, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a),
                                                 __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// four E4M3 codes -> two dwords of bf16 pairs (exact)
__device__ __forceinline__ uint32_t fp8_lo(uint32_t v) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
}
__device__ __forceinline__ uint32_t fp8_hi(uint32_t v) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
}
__device__ __forceinline__ uint4 fp8x8(uint32_t a, uint32_t b) {
  return make_uint4(fp8_lo(a), fp8_hi(a), fp8_lo(b), fp8_hi(b));
}

// W consecutive dwords (1, 2, 4 or 8) at an address aligned to min(4 W, 16).
template <int W>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&d)[W]) {
  if constexpr (W == 1) {
    d[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    d[0] = x.x, d[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + 4 * i);
      d[i] = x.x, d[i + 1] = x.y, d[i + 2] = x.z, d[i + 3] = x.w;
    }
  }
}

__device__ __forceinline__ float quad_max(float v) {  // over the 4 lane groups
  v = fmaxf(v, xchg16(v));
  return fmaxf(v, xchg32(v));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += xchg16(v);
  return v + xchg32(v);
}

// keys the item reads: [lo, hi) of one page list
struct Range {
  const int32_t* pages;
  int lo, hi;
};

}  // namespace

// Query rows per item and the limits of a row.
__device__ __forceinline__ int row_limit(const AttnArgs& a, int t) {
  const int p = a.pos[t];
  return p < 0 ? 0 : min(p + 1, a.max_keys);
}

// One block (4 waves): RT x 16 rows from row r0 of `rows` (row r is token
// t0 + r / G, query head h G + r % G) over the keys [lo, hi); 32-key tiles are
// dealt out over the waves and joined in LDS at the end.
template <int D, bool FP8, int RT>
__device__ __forceinline__ void attn_item(const AttnArgs& a, int h, int t0, int r0, int rows,
                                          const Range& rg, int part, float* lds) {
  constexpr int NS = D / 32;        // 32-column steps of the score product
  constexpr int VD = D / 16;        // columns per lane of V and O
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int page_size = 1 << a.page_shift;

  // this lane's query of each row tile, its operand and its limit
  uint4 q[RT][NS];
  int lim[RT], tok[RT], head[RT];
  int maxlim = 0, minlim = 0x7fffffff;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + c;
    const int rr = min(r, rows - 1);
    tok[rt] = t0 + rr / a.G;
    head[rt] = h * a.G + rr % a.G;
    lim[rt] = r < rows ? row_limit(a, tok[rt]) : 0;
    if (lim[rt] > 0) {
      maxlim = max(maxlim, lim[rt]);
      minlim = min(minlim, lim[rt]);
    }
    // column order of the score product: bf16 K, step s of group g holds
    // columns 32 s + 8 g; FP8 K, steps 2u and 2u+1 the halves of the 16 codes
    // from 64 u + 16 g
    const uint16_t* qr = a.q + (size_t)tok[rt] * a.q_stride + (size_t)head[rt] * D;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      q[rt][s] = *reinterpret_cast<const uint4*>(
          qr + (FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g));
  }
  maxlim = wave_max_all(maxlim);
  minlim = wave_min_all(minlim);
  const int hi = min(rg.hi, maxlim);

  v4f_t o[RT][VD];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY, l[rt] = 0.0f;
#pragma unroll
    for (int j = 0; j < VD; ++j) o[rt][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
  }

  const int first = (rg.lo & ~31) + 32 * wv;
  for (int j0 = first; j0 < hi; j0 += 128) {
    // the pages of the two 16-key halves (the second may lie past the last key)
    const uint8_t *kb[2], *vb[2];
    const float *ksb[2], *vsb[2];
    bool bad[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int ju = max(rg.lo, min(j0 + 16 * u, hi - 1));
      int pg = __builtin_amdgcn_readfirstlane(rg.pages[ju >> a.page_shift]);
      bad[u] = pg < 0 || pg >= a.n_pages;
      pg = bad[u] ? 0 : pg;
      const int slot = (j0 + 16 * u) & (page_size - 1);
      const size_t row = ((size_t)pg * a.Hkv + h) * page_size + slot;
      kb[u] = (const uint8_t*)a.k + row * D * (FP8 ? 1 : 2);
      vb[u] = (const uint8_t*)a.v + row * D * (FP8 ? 1 : 2);
      ksb[u] = a.ks + row, vsb[u] = a.vs + row;
    }
    if ((bad[0] || bad[1]) && lane == 0 && a.status) set_status(a.status, MOE_STATUS_BAD_PAGE);

    // K operand and V rows
    uint4 kf[2][NS];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if constexpr (FP8) {
#pragma unroll
        for (int s = 0; s < NS; s += 2) {
          const uint4 x = *reinterpret_cast<const uint4*>(kb[u] + c * D + 32 * s + 16 * g);
          kf[u][s] = fp8x8(x.x, x.y);
          kf[u][s + 1] = fp8x8(x.z, x.w);
        }
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s)
          kf[u][s] = *reinterpret_cast<const uint4*>(kb[u] + (c * D + 32 * s + 8 * g) * 2);
      }
    constexpr int VW = FP8 ? VD / 4 : VD / 2;  // dwords per key of this lane's V columns
    uint32_t vr[8][VW];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      load_dwords(vb[e >> 2] + ((4 * g + (e & 3)) * D + VD * c) * (FP8 ? 1 : 2), vr[e]);
    }
    float kscale[8], vscale[8];
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 x = *reinterpret_cast<const float4*>(ksb[u] + 4 * g);
        const float4 y = *reinterpret_cast<const float4*>(vsb[u] + 4 * g);
        kscale[4 * u] = x.x, kscale[4 * u + 1] = x.y, kscale[4 * u + 2] = x.z, kscale[4 * u + 3] = x.w;
        vscale[4 * u] = y.x, vscale[4 * u + 1] = y.y, vscale[4 * u + 2] = y.z, vscale[4 * u + 3] = y.w;
      }
    }
    // a tile that is not wholly inside every row's keys is masked; V rows no
    // row of the item sees are cleared, as they may hold anything
    const bool edge = j0 < rg.lo || j0 + 32 > min(hi, minlim) || bad[0] || bad[1];
    bool leak = false;  // a non-finite V that some row of the item must not see
    if (edge) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + 16 * (e >> 2) + 4 * g + (e & 3);
        const bool keep = j >= rg.lo && j < hi && !bad[e >> 2];
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          vr[e][i] = keep ? vr[e][i] : 0u;
          if (FP8) {
            const uint32_t x = vr[e][i] & 0x7f7f7f7fu;
            leak |= ((x + 0x01010101u) & 0x80808080u) != 0;
          } else {
            leak |= (vr[e][i] & 0x7f80u) == 0x7f80u || (vr[e][i] & 0x7f800000u) == 0x7f800000u;
          }
        }
        if (FP8) {
          vscale[e] = keep ? vscale[e] : 0.0f;
          leak |= !(fabsf(vscale[e]) < INFINITY);
        }
      }
      leak = __ballot(leak) != 0;
    }

    // scores and probabilities
    uint4 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      v4f_t s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        s0 = mfma(kf[0][s], q[rt][s], s0);
        s1 = mfma(kf[1][s], q[rt][s], s1);
      }
      float x[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= FP8 ? a.scale_log2 * kscale[e] : a.scale_log2;
        if (edge) {
          const int j = j0 + 16 * (e >> 2) + 4 * g + (e & 3);
          if (j < rg.lo || j >= lim[rt] || j >= hi || bad[e >> 2]) x[e] = -INFINITY;
        }
      }
      float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                       fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      mx = quad_max(fmaxf(mx, m[rt]));
      if (__ballot(mx > m[rt])) {
        const float f = m[rt] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[rt] - mx);
        l[rt] *= f;
#pragma unroll
        for (int j = 0; j < VD; ++j) o[rt][j] *= f;
        m[rt] = mx;
      }
      const float mu = m[rt] == -INFINITY ? 0.0f : m[rt];
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = __builtin_amdgcn_exp2f(x[e] - mu);
        l[rt] += w[e];
        if (FP8) w[e] = edge && x[e] == -INFINITY ? 0.0f : w[e] * vscale[e];
      }
      p[rt] = make_uint4(f32x2_to_bf16x2(w[0], w[1]), f32x2_to_bf16x2(w[2], w[3]),
                         f32x2_to_bf16x2(w[4], w[5]), f32x2_to_bf16x2(w[6], w[7]));
    }

    // O^T += V^T P^T, column set j of the lanes
    auto v_operand = [&](int j) -> uint4 {
      uint32_t d[4];
      if constexpr (FP8) {
        // byte j%4 of keys 0..3 and 4..7
        const uint32_t sel = 0x0c0c0400u + 0x0101u * (j & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two =
              __builtin_amdgcn_perm(vr[2 * i + 1][j / 4], vr[2 * i][j / 4], sel);
          d[i] = fp8_lo(two);
        }
      } else {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = __builtin_amdgcn_perm(vr[2 * i + 1][j / 2], vr[2 * i][j / 2], sel);
      }
      return make_uint4(d[0], d[1], d[2], d[3]);
    };
    if (!leak) {
#pragma unroll
      for (int j = 0; j < VD; ++j) {
        const uint4 vf = v_operand(j);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[rt][j] = mfma(vf, p[rt], o[rt][j]);
      }
    } else {
      // 0 x inf is NaN: rows with different limits one limit at a time, the
      // values past it cleared
      int done = -1;
      while (true) {
        int next = 0x7fffffff;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (lim[rt] > done) next = min(next, lim[rt]);
        next = wave_min_all(next);
        if (next == 0x7fffffff) break;
        done = next;
        uint32_t keep[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          keep[e] = j0 + 16 * (e >> 2) + 4 * g + (e & 3) < done ? 0xffffffffu : 0u;
#pragma unroll
        for (int j = 0; j < VD; ++j) {
          uint4 vf = v_operand(j);
          vf.x &= (keep[0] & 0xffffu) | (keep[1] & 0xffff0000u);
          vf.y &= (keep[2] & 0xffffu) | (keep[3] & 0xffff0000u);
          vf.z &= (keep[4] & 0xffffu) | (keep[5] & 0xffff0000u);
          vf.w &= (keep[6] & 0xffffu) | (keep[7] & 0xffff0000u);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const v4f_t n = mfma(vf, p[rt], o[rt][j]);
            if (lim[rt] == done) o[rt][j] = n;
          }
        }
      }
    }
  }

  // the four waves' sums joined: two rounds through LDS
  float* lml = lds;                        // [4][RT][64][2]: m, l (l summed over the groups)
  float* lo = lds + 4 * RT * 64 * 2;       // [2][RT * VD * 4][64]
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = quad_sum(l[rt]);
    lml[((wv * RT + rt) * 64 + lane) * 2] = m[rt];
    lml[((wv * RT + rt) * 64 + lane) * 2 + 1] = l[rt];
  }
  __syncthreads();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, lml[((w * RT + rt) * 64 + lane) * 2]);
    float L = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float mw = lml[((w * RT + rt) * 64 + lane) * 2];
      if (mw != -INFINITY)
        L += lml[((w * RT + rt) * 64 + lane) * 2 + 1] * __builtin_amdgcn_exp2f(mw - M);
    }
    const float f = m[rt] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[rt] - M);
#pragma unroll
    for (int j = 0; j < VD; ++j) o[rt][j] *= f;
    m[rt] = M, l[rt] = L;
  }
#pragma unroll
  for (int half = 2; half > 0; half >>= 1) {
    if (wv >= half && wv < 2 * half) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < VD; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            lo[(((wv - half) * RT * VD + rt * VD + j) * 4 + r) * 64 + lane] = o[rt][j][r];
    }
    __syncthreads();
    if (wv < half) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < VD; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            o[rt][j][r] += lo[((wv * RT * VD + rt * VD + j) * 4 + r) * 64 + lane];
    }
    __syncthreads();
  }
  if (wv) return;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (r0 + 16 * rt + c >= rows) continue;
    const size_t row = ((size_t)part * a.n_tok + tok[rt]) * a.Hq + head[rt];
    const bool none = lim[rt] == 0;
    if (g == 0) a.pml[row] = make_float2(none ? -INFINITY : m[rt], none ? 0.0f : l[rt]);
    float* dst = a.po + row * D + VD * 4 * g;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < VD; j += 4)
        *reinterpret_cast<float4*>(dst + VD * r + j) =
            make_float4(o[rt][j][r], o[rt][j + 1][r], o[rt][j + 2][r], o[rt][j + 3][r]);
  }
}

// Number of a sequence's own parts in use: its longest row's keys past the
// prefix in chunks.
__device__ __forceinline__ int own_parts(const AttnArgs& a, int lim) {
  const int lo = a.prefix_len & ~31;
  return lim > a.prefix_len ? (lim - lo + a.own_chunk - 1) / a.own_chunk : 0;
}

// Prefix items first (they are the long ones), then the sequences' own.
template <int D, bool FP8, int RTP, int RTS>
__global__ __launch_bounds__(256) void attn_part_kernel(AttnArgs a) {
  constexpr int RT = RTP > RTS ? RTP : RTS;
  __shared__ float lds[4 * RT * 64 * 2 + 2 * RT * (D / 16) * 4 * 64];
  int item = blockIdx.x;
  const int rows_p = a.n_tok * a.G, rows_s = a.Q * a.G;
  const int np = a.n_prefix_parts * a.Hkv * a.prefix_blocks;
  if (item < np) {
    const int rb = item % a.prefix_blocks;
    item /= a.prefix_blocks;
    const int h = item % a.Hkv, part = item / a.Hkv;
    const Range rg = {a.prefix_pages, part * a.prefix_chunk,
                      min((part + 1) * a.prefix_chunk, a.prefix_len)};
    attn_item<D, FP8, RTP>(a, h, 0, rb * 16 * RTP, rows_p, rg, part, lds);
  } else {
    item -= np;
    const int rb = item % a.own_blocks;
    item /= a.own_blocks;
    const int h = item % a.Hkv;
    item /= a.Hkv;
    const int b = item % a.B, part = item / a.B;
    int lim = 0;
    for (int i = 0; i < a.Q; ++i) lim = max(lim, row_limit(a, b * a.Q + i));
    if (part >= own_parts(a, lim)) return;
    const int base = (a.prefix_len & ~31) + part * a.own_chunk;
    const Range rg = {a.table + (size_t)b * a.table_cols, max(base, a.prefix_len),
                      min(base + a.own_chunk, a.max_keys)};
    attn_item<D, FP8, RTS>(a, h, b * a.Q, rb * 16 * RTS, rows_s, rg, a.n_prefix_parts + part, lds);
  }
}

// One lane group of D/4 lanes per output row: the row's parts weighted by
// 2^(m - M) and normalised.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int LPR = D / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (row >= (int64_t)a.n_tok * a.Hq) return;
  const int t = (int)(row / a.Hq), d = 4 * (threadIdx.x % LPR);
  const int b = t / a.Q;
  int lim = 0;
  for (int i = 0; i < a.Q; ++i) lim = max(lim, row_limit(a, b * a.Q + i));
  const int parts = a.n_prefix_parts + own_parts(a, lim);
  const size_t stride = (size_t)a.n_tok * a.Hq;
  float M = -INFINITY;
  for (int p = 0; p < parts; ++p) M = fmaxf(M, a.pml[p * stride + row].x);
  float L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < parts; ++p) {
    const float2 ml = a.pml[p * stride + row];
    if (ml.x == -INFINITY) continue;
    const float f = __builtin_amdgcn_exp2f(ml.x - M);
    const float4 v = *reinterpret_cast<const float4*>(a.po + (p * stride + row) * D + d);
    L = fmaf(f, ml.y, L);
    o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
  }
  const bool none = M == -INFINITY;
  if (!none) o.x /= L, o.y /= L, o.z /= L, o.w /= L;
  *reinterpret_cast<uint2*>(a.out + row * D + d) =
      make_uint2(f32x2_to_bf16x2(o.x, o.y), f32x2_to_bf16x2(o.z, o.w));
  if (a.lse && d == 0) a.lse[row] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  if (a.status && d == 0 && a.pos[t] >= a.max_keys) set_status(a.status, MOE_STATUS_BAD_PAGE);
}

namespace {

template <int D, bool FP8, int RTP>
void launch_rows(const AttnArgs& a, int grid, hipStream_t st) {
  if (a.own_rt == 1)
    attn_part_kernel<D, FP8, RTP, 1><<<grid, 256, 0, st>>>(a);
  else
    attn_part_kernel<D, FP8, RTP, 2><<<grid, 256, 0, st>>>(a);
}

template <int D, bool FP8>
void launch_dim(const AttnArgs& a, int grid, hipStream_t st) {
  if (a.prefix_rt == 1)
    launch_rows<D, FP8, 1>(a, grid, st);
  else
    launch_rows<D, FP8, 2>(a, grid, st);
}

template <int D>
void launch_all(const AttnArgs& a, hipStream_t st) {
  const int grid = a.n_prefix_parts * a.Hkv * a.prefix_blocks +
                   a.n_own_parts * a.B * a.Hkv * a.own_blocks;
  if (grid > 0) {
    if (a.fp8)
      launch_dim<D, true>(a, grid, st);
    else
      launch_dim<D, false>(a, grid, st);
  }
  constexpr int RPB = 256 / (D / 4);
  const int64_t rows = (int64_t)a.n_tok * a.Hq;
  attn_join_kernel<D><<<(unsigned)((rows + RPB - 1) / RPB), 256, 0, st>>>(a);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t st) {
  if (a.D == 64)
    launch_all<64>(a, st);
  else if (a.D == 128)
    launch_all<128>(a, st);
  else
    launch_all<256>(a, st);
  return hipGetLastError();
}

}  // namespace bef
