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
// Scores, statistics and sums are fp32.  P is rounded for the matrix cores: to bf16 beside
// bf16 V, each weight by 2^-8 of itself at most; the weights summed are the unrounded ones.
// Beside E4M3 V a weight is P times the key's V scale, no value of which is exact, and is
// rounded to fp16: by 2^-11 of itself, or by 2^-29 of the row's largest weight where
// that is more.  fp16 holds 2^40 in all, so a row's weights are formed against its own
// largest P v_scale (raise_max's reference): a scale far from the others', of a key that the
// row does not see or gives no weight, takes nothing from the weights beside it.
//
// Measured at 128 columns, bf16, 32 sequences of 8 kv heads and 4 query heads each:
// 8192 shared keys and up to 2048 of their own, 161 MB, in 47 us and 5 for the join (3.1
// TB/s in all: the shared keys are read by four blocks of rows, from L2 but for the
// first).  16 sequences of 4 tokens, 8 kv heads of 8 query heads each, 32768 shared
// E4M3 keys and up to 1024 of their own, 70 GFLOP: 133 us.
//
// E2M1 keys and values are widened to bf16 on the way to the matrix cores, by the codes' own
// scale (v_cvt_scalef32_pk_bf16_fp4, four for 8 codes), which is exact: what follows is bf16
// attention over what the cache holds.  A lane's 8 V codes come as a dword, and their permutes
// are those of bf16.  Two tiles of 16 bytes less a lane hide less latency, so the next tile's
// codes are loaded before this tile's products: without a branch and in the order in which they
// are wanted, so that a wait for one leaves the later ones on their way.  Bound by vector
// instructions (widening, softmax) and those waits, not by bytes: 8 sequences of 8 kv heads
// and 8 query heads each over up to 65536 keys of 128 columns, 241 MB, in 59 us (4.1 TB/s;
// issue 46% busy) and 5 for the join; 32 sequences, 4 query heads each, behind 8192 shared
// keys, up to 2048 of their own, 43 MB, in 21.5 us (59%) and 4.  In the first more or fewer
// parts took 69 to 114 us, a third tile in flight 70 to 102 (the loop's code then no longer fits
// the instruction cache beside the rest), one wave more a SIMD 164 (registers spilled).  The
// weights are rounded to bf16, as beside bf16 V, because V's scales reach over bf16's exponents
// and a weight would need one per 32 columns to be fp16 instead: outputs of these two cases are
// 0.0019 and 0.0020 off in the 2-norm, with weights of 32 bits 0.0017, which is their own rounding.
// At 256 columns 32 sequences of 8 kv heads, 4 query heads each, behind 8192 and 2048 keys take
// 75.7 us and 5.3; 16 registers spill there.
#include <type_traits>

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

// The scale operand of UE8M0 byte b (only the exponent field counts): 2^(b - 127), or NaN
// above 252, where 6 times it is past bf16.
__device__ __forceinline__ float fp4_scale(uint32_t b) {
  return __uint_as_float(b > 252u ? 0x7fc00000u : b << 23);
}
// eight E2M1 codes -> four dwords of bf16 pairs (exact: two significant bits)
__device__ __forceinline__ uint4 fp4x8(uint32_t v, float sc) {
  return make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, sc, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, sc, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, sc, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, sc, 3)));
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
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t w = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += xchg16(v);
  return v + xchg32(v);
}

// two fp32 -> two fp16, nearest even
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const h2_t v = {(_Float16)lo, (_Float16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// V^T P^T: bf16, or fp16 for an FP8 cache (E4M3 values are fp16 values, and P
// then keeps 11 bits)
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
template <bool F16>
__device__ __forceinline__ v4f_t mfma_pv(const uint4 a, const uint4 b, v4f_t c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a),
                                                  __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
  else
    return mfma(a, b, c);
}

template <bool F16>
__device__ __forceinline__ uint4 pack_p(const float (&w)[8]) {
  if constexpr (F16)
    return make_uint4(pack_f16(w[0], w[1]), pack_f16(w[2], w[3]), pack_f16(w[4], w[5]),
                      pack_f16(w[6], w[7]));
  else
    return make_uint4(f32x2_to_bf16x2(w[0], w[1]), f32x2_to_bf16x2(w[2], w[3]),
                      f32x2_to_bf16x2(w[4], w[5]), f32x2_to_bf16x2(w[6], w[7]));
}

// page lists are read through the scalar cache (nothing writes them here)
typedef __attribute__((address_space(4))) const int32_t const_i32;

// keys the item reads: [lo, hi) of one page list
struct Range {
  const int32_t* pages;
  int lo, hi;
};

}  // namespace

// The keys a token sees.
__device__ __forceinline__ int row_limit(const AttnArgs& a, int t) {
  const int p = a.pos[t];
  return p < 0 ? 0 : min(p, a.max_keys - 1) + 1;
}

// V scales of an E4M3 cache are multiplied in units of 2^-12 `bound`, a power of two taken
// once, 4 to 8 times the first scales' largest.
__device__ __forceinline__ float scale_bound(float first) {
  const float b = 8.0f * __uint_as_float(__float_as_uint(first) & 0x7f800000u);
  return __builtin_amdgcn_fmed3f(b, 0x1p-40f, 0x1p40f);
}
// Finite scales stay finite (times a weight of 0 they must be 0).
__device__ __forceinline__ float scale_units(float v, float per) {
  const float u = v * per;
  return fabsf(v) < INFINITY ? __builtin_amdgcn_fmed3f(u, -0x1.fffffep127f, 0x1.fffffep127f) : u;
}
// log2 of a scale in those units against bound, within what leaves the sum of
// 2^(score - reference) in fp32's range: scales of 2^-90 to 2^115 times bound.
__device__ __forceinline__ float scale_log2_of(float u) {
  return __builtin_amdgcn_fmed3f(__builtin_amdgcn_logf(fabsf(u)) - 12.0f, -90.0f, 115.0f);
}
// Scales near enough to bound that a weight may be bounded by P alone.
__device__ __forceinline__ bool scale_far(float lo, float hi, float bound) {
  return !(hi <= bound && lo >= bound * 0x1p-8f);
}
// Brings l to [1, 2) and m along, by the power of two 2^-k (exactly: k is whole).  References
// that follow V scales say nothing of a part's weight; joined parts have to compare.
__device__ __forceinline__ int unit_weight(float& m, float& l) {
  const int e = (int)(__float_as_uint(l) >> 23) - 127;
  const int k = l > 0.0f && l < INFINITY ? e : 0;
  l = __builtin_amdgcn_ldexpf(l, -k);
  m += (float)k;
  return k;
}

__device__ __forceinline__ float max8(const float (&x)[8]) {
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
               fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}
__device__ __forceinline__ float min8(const float (&x)[8]) {
  return fminf(fminf(fminf(x[0], x[1]), fminf(x[2], x[3])),
               fminf(fminf(x[4], x[5]), fminf(x[6], x[7])));
}

// The running maximum m of a lane column (log2 units), given this tile's largest
// scores: P = 2^(score - m).  m is raised where a score passes it by more than
// 3, so P is at most 8 and the sums are rescaled a few times, not at every
// tile that holds a new maximum (most of the first dozens); a key that stands
// out by more than that has P = 1 exactly.  With an E4M3 cache m is the reference of the
// weights P v_scale: mx then is the largest score plus the log2 of its key's scale (or a
// bound of it), and P = 2^(score - m) may be far from 1.
template <class F>
__device__ __forceinline__ void raise_max(float mx, float& m, F&& rescale) {
  if (__ballot(mx > m + 3.0f)) {
    const float mn = quad_max(fmaxf(mx, m));
    rescale(mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn));
    m = mn;
  }
}

// The maximum that a part's weight l goes with.  -inf says that the part holds no key (l is
// then 0) and leaves it out; a row whose scores are all NaN has no maximum either but
// an l of NaN, which has to reach the row's sum: beside any finite maximum it does.
__device__ __forceinline__ float part_max(float m, float l) {
  return m == -INFINITY && l != 0.0f ? 0.0f : m;
}

// Whether key j of the range [lo, hi) lies in a page outside the cache.
__device__ __forceinline__ bool bad_key(const AttnArgs& a, const int32_t* pages, int j, int lo,
                                        int hi) {
  const int pg = pages[max(lo, min(j, hi - 1)) >> a.page_shift];
  return pg < 0 || pg >= a.n_pages;
}
// One block (4 waves) over the keys of rg for RT x 16 rows, r0.. of `rows` (row r
// is token t0 + r / G, query head h G + r % G): 32-key tiles are dealt out over
// the waves, whose sums are joined in LDS at the end.
//
// A tile's K is dead once the scores are formed and its V once they are
// multiplied, so the next tile's are loaded into the same registers right
// then: a load has the rest of a tile's work to arrive in.
template <int D, int KV, int RT>
__device__ __forceinline__ void attn_item(const AttnArgs& a, int h, int t0, int r0, int rows,
                                          const Range& rg, int part, float* lds) {
  constexpr int NS = D / 32;        // 32-column steps of the score product
  constexpr int VD = D / 16;        // columns per lane of V and O
  constexpr bool FP8 = KV == kKvE4M3, FP4 = KV == kKvE2M1;
  constexpr int RB = FP4 ? D / 2 : FP8 ? D : 2 * D;  // bytes of a cache row
  constexpr int NK = FP8 ? NS / 2 : NS;      // 16-byte K loads per 16 keys (bf16, E4M3)
  constexpr int VW = VD * (FP8 ? 1 : 2) / 4; // dwords per key of this lane's V columns (E2M1: as bf16)
  constexpr int SB = D / 32;                 // E2M1: scale bytes of a row
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int slots = (1 << a.page_shift) - 1;

  // this lane's query of each row tile, its operand and its limit.  Column order of
  // the score product: bf16 K, step s of group g holds columns 32 s + 8 g; FP8 K,
  // steps 2u and 2u+1 the halves of the 16 codes from 64 u + 16 g; E2M1 K, columns 8 s
  // of the g-th quarter of the row
  auto row_of = [&](int rt, int& tok, int& head) {
    const int rr = min(r0 + 16 * rt + c, rows - 1);
    tok = t0 + rr / a.G;
    head = h * a.G + rr % a.G;
    return r0 + 16 * rt + c < rows;
  };
  uint4 q[RT][NS];
  int lim[RT], maxlim = 0, minlim = 0x7fffffff;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    int tok, head;
    const bool in = row_of(rt, tok, head);
    lim[rt] = in ? row_limit(a, tok) : 0;
    maxlim = max(maxlim, lim[rt]);
    minlim = min(minlim, lim[rt] > 0 ? lim[rt] : 0x7fffffff);
    const uint16_t* qr = a.q + (size_t)tok * a.q_stride + (size_t)head * D;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      q[rt][s] = *reinterpret_cast<const uint4*>(
          qr + (FP4 ? D / 4 * g + 8 * s : FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g));
  }
  maxlim = __builtin_amdgcn_readfirstlane(wave_max_all(maxlim));
  minlim = __builtin_amdgcn_readfirstlane(wave_min_all(minlim));
  const int lo = rg.lo, hi = min(rg.hi, maxlim);

  v4f_t o[RT][VD];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY, l[rt] = 0.0f;
#pragma unroll
    for (int j = 0; j < VD; ++j) o[rt][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
  }
  // FP8: o is in units of 2^-12 bound (0: not yet known), of which a scale of 1 is `per`
  float bound = 0.0f, per = 1.0f;

  // the 16-key halves' first cache rows (the second half may lie past the last
  // key: any row of a valid page serves), through the scalar cache
  struct Rows {
    size_t row[2];
    bool bad[2];
  };
  const const_i32* pages = (const const_i32*)rg.pages;
  auto rows_at = [&](int j0) {
    Rows r;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int ju = max(lo, min(j0 + 16 * u, hi - 1));
      const int pg = pages[ju >> a.page_shift];
      r.bad[u] = pg < 0 || pg >= a.n_pages;
      r.row[u] = (((size_t)(r.bad[u] ? 0 : pg) * a.Hkv + h) << a.page_shift) +
                 ((j0 + 16 * u) & slots);
    }
    return r;
  };
  const uint32_t ko = c * RB + (FP4 ? D / 8 : 16) * g, vo = 4 * g * RB + RB / 16 * c;
  uint4 kr[2][NK];
  float4 ks4[2], vs4[2];
  uint32_t vr[8][VW];
  // E2M1: a quarter of a K row with its scale bytes (one, or two at 256 columns; at 64
  // two groups share one); a lane's V columns of 8 keys as loaded, and the scale bytes of
  // all columns of these keys
  constexpr int KW = D / 32, VSW = D / 32;
  struct Raw {
    uint32_t kq[2][KW], ksb[2], vq[8][D == 256 ? 2 : 1], vsb[2][VSW];
  };
  auto load_k4 = [&](const Rows& r, Raw& raw) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_dwords((const uint8_t*)a.k + r.row[u] * RB + ko, raw.kq[u]);
      const uint8_t* sb = (const uint8_t*)a.ks + r.row[u] * SB;
      if constexpr (D == 256)
        raw.ksb[u] = *reinterpret_cast<const uint16_t*>(sb + c * SB + 2 * g);
      else
        raw.ksb[u] = sb[c * SB + (D == 64 ? g >> 1 : g)];
    }
  };
  auto load_v4 = [&](const Rows& r, Raw& raw) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* vb = (const uint8_t*)a.v + r.row[e >> 2] * RB + vo + (e & 3) * RB;
      if constexpr (D == 64)
        raw.vq[e][0] = *reinterpret_cast<const uint16_t*>(vb);
      else
        load_dwords(vb, raw.vq[e]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      load_dwords((const uint8_t*)a.vs + (r.row[u] + 4 * g) * SB, raw.vsb[u]);
  };
  auto load_k = [&](const Rows& r) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* kb = (const uint8_t*)a.k + r.row[u] * RB;
#pragma unroll
      for (int s = 0; s < NK; ++s) kr[u][s] = *reinterpret_cast<const uint4*>(kb + ko + 64 * s);
      if constexpr (FP8) {
        ks4[u] = *reinterpret_cast<const float4*>((const float*)a.ks + r.row[u] + 4 * g);
        vs4[u] = *reinterpret_cast<const float4*>((const float*)a.vs + r.row[u] + 4 * g);
      }
    }
  };
  auto load_v = [&](const Rows& r) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      load_dwords((const uint8_t*)a.v + r.row[e >> 2] * RB + vo + (e & 3) * RB, vr[e]);
  };
  // E2M1 V as bf16, from here on as if loaded so
  auto widen_v = [&](const Raw& raw) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // byte VD c / 32 of the row's scale bytes, which are half a dword, one or two
      const uint32_t w = D == 64    ? raw.vsb[e >> 2][(e & 3) >> 1] >> 16 * (e & 1)
                         : D == 128 ? raw.vsb[e >> 2][e & 3]
                         : c < 8    ? raw.vsb[e >> 2][(2 * (e & 3)) % VSW]
                                    : raw.vsb[e >> 2][(2 * (e & 3) + 1) % VSW];
      const float sc = fp4_scale(w >> 8 * (VD * c / 32 & 3) & 0xffu);
      if constexpr (D == 64) {
        const uint4 x = fp4x8(raw.vq[e][0], sc);
        vr[e][0] = x.x, vr[e][1 % VW] = x.y;
      } else {
#pragma unroll
        for (int i = 0; i < VW; i += 4) {
          const uint4 x = fp4x8(raw.vq[e][i / 4], sc);
          vr[e][i] = x.x, vr[e][(i + 1) % VW] = x.y, vr[e][(i + 2) % VW] = x.z,
          vr[e][(i + 3) % VW] = x.w;
        }
      }
    }
  };

  // V rows that no row of the item sees may hold anything: cleared.  A
  // non-finite V that only some rows see must not meet the others' P = 0 (0 x inf
  // is NaN): true where the tile has one.
  auto leaks = [&](int j0, const Rows& cur) -> bool {
    bool leak = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + 16 * (e >> 2) + 4 * g + (e & 3);
      const bool keep = j >= lo && j < hi && !cur.bad[e >> 2];
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        vr[e][i] = keep ? vr[e][i] : 0u;
        if (FP8)
          leak |= (((vr[e][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
        else
          leak |= (vr[e][i] & 0x7f80u) == 0x7f80u || (vr[e][i] & 0x7f800000u) == 0x7f800000u;
      }
      if constexpr (FP8) {
        const float4 v = vs4[e >> 2];
        const float x = (e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w;
        leak |= keep && !(fabsf(x) < INFINITY);
      }
    }
    return __ballot(leak) != 0;
  };

  // One tile, its K and V loaded (or on their way): SLOW, one limit at a time.
  // `after_k` and `after_v` run when K and V are dead.  False: nothing was done,
  // the tile needs SLOW (E2M1: and the next tile's loads are the caller's).
  auto tile = [&](auto slow, int j0, const Rows& cur, const Raw& raw, auto&& after_k,
                  auto&& after_v) -> bool {
    constexpr bool SLOW = decltype(slow)::value;
    const bool bad = cur.bad[0] || cur.bad[1];
    if (bad && lane == 0 && a.status) set_status(a.status, MOE_STATUS_BAD_PAGE);
    // a tile that is not wholly inside every row's keys is masked
    const bool edge = SLOW || j0 < lo || j0 + 32 > min(hi, minlim) || bad;
    auto key_of = [&](int e) { return j0 + 16 * (e >> 2) + 4 * g + (e & 3); };
    auto inside = [&](int e) { return key_of(e) >= lo && key_of(e) < hi && !cur.bad[e >> 2]; };

    // (E2M1: the wait for V is here only where it has to be looked at; SLOW: widened and
    // cleared before)
    if constexpr (FP4 && !SLOW)
      if (edge) widen_v(raw);
    if (!SLOW && edge && leaks(j0, cur)) {
      if constexpr (!FP4) {
        after_k();
        after_v();
      }
      return false;
    }

    // scores
    float x[RT][8];
    {
      uint4 kf[2][NS];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          if constexpr (FP4) {
            const uint32_t b = D == 256 ? raw.ksb[u] >> 8 * (s >> 2) & 0xffu : raw.ksb[u];
            kf[u][s] = fp4x8(raw.kq[u][s], fp4_scale(b));
          } else if constexpr (FP8) {
            const uint4 k = kr[u][s / 2];
            kf[u][s] = (s & 1) ? fp8x8(k.z, k.w) : fp8x8(k.x, k.y);
          } else {
            kf[u][s] = kr[u][s];
          }
        }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        v4f_t s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          s0 = mfma(kf[0][s], q[rt][s], s0);
          s1 = mfma(kf[1][s], q[rt][s], s1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[rt][e] = s0[e], x[rt][4 + e] = s1[e];
      }
    }
    float vscale[8];
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float kk[4] = {ks4[u].x, ks4[u].y, ks4[u].z, ks4[u].w};
        const float vv[4] = {vs4[u].x, vs4[u].y, vs4[u].z, vs4[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) x[rt][4 * u + e] *= kk[e];
          vscale[4 * u + e] = vv[e];
        }
      }
    }
    after_k();

    float lg[8];       // far: log2 of the keys' V scales
    bool far = false;  // (the same in every lane)
    if constexpr (FP8) {
      float mag[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (edge && !inside(e)) vscale[e] = 0.0f;
        mag[e] = fabsf(vscale[e]);
      }
      if (bound == 0.0f) {
        float f = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f = fmaxf(f, mag[e] < INFINITY ? mag[e] : 0.0f);
        f = quad_max(f);
        if (__ballot(f > 0.0f)) bound = scale_bound(f), per = 0x1p12f / bound;
      }
      far = edge || __ballot(scale_far(min8(mag), max8(mag), bound)) != 0;
      if (!far) {
#pragma unroll
        for (int e = 0; e < 8; ++e) vscale[e] *= per;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          vscale[e] = scale_units(vscale[e], per);
          lg[e] = scale_log2_of(vscale[e]);
        }
      }
    }

    // probabilities
    uint4 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (edge) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!inside(e) || key_of(e) >= lim[rt]) x[rt][e] = -INFINITY;
      }
      float mx;
      if (FP8 && far) {
        mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fmaf(x[rt][e], a.scale_log2, lg[e]));
      } else {
        mx = max8(x[rt]) * a.scale_log2;
      }
      raise_max(mx, m[rt], [&](float f) {
        l[rt] *= f;
#pragma unroll
        for (int j = 0; j < VD; ++j) o[rt][j] *= f;
      });
      const float mu = m[rt] == -INFINITY ? 0.0f : m[rt];
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = __builtin_amdgcn_exp2f(fmaf(x[rt][e], a.scale_log2, -mu));
        l[rt] += w[e];
        // (0 x a non-finite scale: only in tiles set aside)
        if (FP8) w[e] = SLOW && x[rt][e] == -INFINITY ? 0.0f : w[e] * vscale[e];
      }
      p[rt] = pack_p<FP8>(w);
    }

    if constexpr (FP4 && !SLOW) {
      if (!edge) widen_v(raw);
      after_v();
    }
    // O^T += V^T P^T, column set j of the lanes
    auto v_operand = [&](int j) -> uint4 {
      uint32_t d[4];
      if constexpr (FP8) {
        // byte j%4 of two keys, then both converted
        const uint32_t sel = 0x0c0c0400u + 0x0101u * (j & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = __builtin_bit_cast(
              uint32_t,
              e4m3x2_lo(__builtin_amdgcn_perm(vr[2 * i + 1][j / 4], vr[2 * i][j / 4], sel)));
      } else {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = __builtin_amdgcn_perm(vr[2 * i + 1][j / 2], vr[2 * i][j / 2], sel);
      }
      return make_uint4(d[0], d[1], d[2], d[3]);
    };
    if constexpr (!SLOW) {
#pragma unroll
      for (int j = 0; j < VD; ++j) {
        const uint4 vf = v_operand(j);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[rt][j] = mfma_pv<FP8>(vf, p[rt], o[rt][j]);
      }
    } else {
      for (int done = -1;;) {
        int next = 0x7fffffff;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (lim[rt] > done) next = min(next, lim[rt]);
        next = wave_min_all(next);
        if (next == 0x7fffffff) break;
        done = next;
#pragma unroll
        for (int j = 0; j < VD; ++j) {
          const uint4 v = v_operand(j);
          uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d[i] &= (key_of(2 * i) < done ? 0xffffu : 0u) |
                    (key_of(2 * i + 1) < done ? 0xffff0000u : 0u);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const v4f_t n = mfma_pv<FP8>(make_uint4(d[0], d[1], d[2], d[3]), p[rt], o[rt][j]);
            if (lim[rt] == done) o[rt][j] = n;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if (!FP4) after_v();
    return true;
  };

  const int step = 128, first = (lo & ~31) + 32 * wv;
  bool leaked = false;
  Raw ring;
  if constexpr (FP4) {
    // (no branch guards a load, so that a wait leaves the younger in flight; past the last
    // key any row serves)
    if (first < hi) {
      Rows cur = rows_at(first);
      load_k4(cur, ring);
      __builtin_amdgcn_sched_barrier(0);  // (in the order of the loop, or its waits count wrong)
      load_v4(cur, ring);
#pragma unroll 1
      for (int j0 = first; j0 < hi; j0 += step) {
        const Rows nxt = rows_at(j0 + step);
        if (!tile(std::false_type{}, j0, cur, ring, [&] { load_k4(nxt, ring); },
                  [&] { load_v4(nxt, ring); })) {
          // (in the tile these loads would be waited for by the code behind it)
          leaked = true;
          load_k4(nxt, ring);
          __builtin_amdgcn_sched_barrier(0);
          load_v4(nxt, ring);
        }
        cur = nxt;
      }
    }
  } else {
    Rows cur{}, nxt{};
    if (first < hi) {
      cur = rows_at(first);
      load_k(cur);
      load_v(cur);
    }
    for (int j0 = first; j0 < hi; j0 += step) {
      const bool more = j0 + step < hi;
      if (more) nxt = rows_at(j0 + step);
      leaked |= !tile(std::false_type{}, j0, cur, ring, [&] { if (more) load_k(nxt); },
                      [&] { if (more) load_v(nxt); });
      cur = nxt;
    }
  }
  // tiles set aside: found again among the ones at an edge
  if (leaked) {
    for (int j0 = first; j0 < hi; j0 += step) {
      const Rows cur = rows_at(j0);
      if (!(j0 < lo || j0 + 32 > min(hi, minlim) || cur.bad[0] || cur.bad[1])) continue;
      if constexpr (FP4) {
        load_k4(cur, ring);
        load_v4(cur, ring);
        widen_v(ring);
      } else {
        load_k(cur);
        load_v(cur);
      }
      if (leaks(j0, cur)) tile(std::true_type{}, j0, cur, ring, [] {}, [] {});
    }
  }

  // the waves' sums joined through LDS, in halves, a row tile at a time
  float2* lml = reinterpret_cast<float2*>(lds);  // [wave][64]: m, l
  float* lo_ = lds + 4 * 64 * 2;                 // [2][VD * 4][64]
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float mw = m[rt], lw = quad_sum(l[rt]);
    const int k = FP8 ? unit_weight(mw, lw) : 0;
    mw = part_max(mw, lw);
    lml[wv * 64 + lane] = make_float2(mw, lw);
    __syncthreads();
    float M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, lml[w * 64 + lane].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 ml = lml[w * 64 + lane];
      if (ml.x != -INFINITY) L += ml.y * __builtin_amdgcn_exp2f(ml.x - M);
    }
    const float f = (FP8 ? 0x1p-12f * bound : 1.0f) *
                    (mw == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mw - M));
#pragma unroll
    for (int j = 0; j < VD; ++j) {
      o[rt][j] *= f;
      if constexpr (FP8)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[rt][j][r] = __builtin_amdgcn_ldexpf(o[rt][j][r], -k);
    }
#pragma unroll
    for (int half = 2; half > 0; half >>= 1) {
      float* mine = lo_ + (wv % half) * (VD * 4 * 64) + lane;
      if (wv >= half && wv < 2 * half) {
#pragma unroll
        for (int j = 0; j < VD; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) mine[(j * 4 + r) * 64] = o[rt][j][r];
      }
      __syncthreads();
      if (wv < half) {
#pragma unroll
        for (int j = 0; j < VD; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[rt][j][r] += mine[(j * 4 + r) * 64];
      }
      __syncthreads();
    }
    int tok, head;
    if (wv || !row_of(rt, tok, head)) continue;
    const size_t row = ((size_t)part * a.n_tok + tok) * a.Hq + head;
    if (g == 0) a.pml[row] = make_float2(lim[rt] ? M : -INFINITY, lim[rt] ? L : 0.0f);
    float* dst = a.po + row * D + VD * 4 * g;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < VD; j += 4)
        *reinterpret_cast<float4*>(dst + VD * r + j) =
            make_float4(o[rt][j][r], o[rt][j + 1][r], o[rt][j + 2][r], o[rt][j + 3][r]);
  }
}

// The keys that the longest-sighted of sequence b's tokens sees (wave-uniform).
__device__ __forceinline__ int seq_limit(const AttnArgs& a, int b) {
  int lim = 0;
  for (int i = threadIdx.x & 63; i < a.Q; i += 64) lim = max(lim, row_limit(a, b * a.Q + i));
  return __builtin_amdgcn_readfirstlane(wave_max_all(lim));
}

// Number of a sequence's own parts in use: its longest row's keys past the
// prefix in chunks.
__device__ __forceinline__ int own_parts(const AttnArgs& a, int lim) {
  const int lo = a.prefix_len & ~31;
  return lim > a.prefix_len ? (lim - lo + a.own_chunk - 1) / a.own_chunk : 0;
}

// An item of the grid: a range of keys for one kv head and a block of rows.
struct Item {
  Range rg;
  int h, t0, rows, rb, part;
};

// The first `np` items are the prefix's, the others the sequences' own; false
// if the sequence ends before the part.
__device__ __forceinline__ bool item_of(const AttnArgs& a, int item, int np, Item& it) {
  if (item < np) {
    // a prefix part's row blocks on one XCD (block ids alike modulo 8), whose L2
    // then holds the keys they share
    const int pairs = np / a.prefix_blocks;
    int pair, rb;
    if (pairs % 8 == 0) {
      const int q = item >> 3;
      rb = q % a.prefix_blocks;
      pair = (q / a.prefix_blocks) * 8 + (item & 7);
    } else {
      rb = item % a.prefix_blocks;
      pair = item / a.prefix_blocks;
    }
    it.rb = rb, it.h = pair % a.Hkv, it.part = pair / a.Hkv;
    it.t0 = 0, it.rows = a.n_tok * a.G;
    it.rg = {a.prefix_pages, it.part * a.prefix_chunk,
             min((it.part + 1) * a.prefix_chunk, a.prefix_len)};
    return true;
  }
  item -= np;
  it.rb = item % a.own_blocks;
  item /= a.own_blocks;
  it.h = item % a.Hkv;
  item /= a.Hkv;
  const int b = item % a.B, part = item / a.B;
  if (part >= own_parts(a, seq_limit(a, b))) return false;
  const int base = (a.prefix_len & ~31) + part * a.own_chunk;
  it.t0 = b * a.Q, it.rows = a.Q * a.G, it.part = a.n_prefix_parts + part;
  it.rg = {a.table + (size_t)b * a.table_cols, max(base, a.prefix_len),
           min(base + a.own_chunk, a.max_keys)};
  return true;
}

// RTP, RTS: row tiles of a block of the prefix's and of the sequences' own items.
template <int D, int KV, int RTP, int RTS>
__global__ __launch_bounds__(256, D < 256 && RTP == 1 ? 3 : 2) void attn_part_kernel(AttnArgs a,
                                                                                    int np) {
  __shared__ __align__(8) float lds[4 * 64 * 2 + 2 * (D / 16) * 4 * 64];
  Item it;
  if (!item_of(a, blockIdx.x, np, it)) return;
  if (RTP == RTS || (int)blockIdx.x < np)
    attn_item<D, KV, RTP>(a, it.h, it.t0, it.rb * 16 * RTP, it.rows, it.rg, it.part, lds);
  else
    attn_item<D, KV, RTS>(a, it.h, it.t0, it.rb * 16 * RTS, it.rows, it.rg, it.part, lds);
}

// ---- many rows: keys staged in LDS for eight waves of rows -------------------
// A block takes 8 x RT x 16 rows; tiles of 64 keys go through LDS, loaded into
// registers while the tile before multiplies.  K lands as rows of bf16, V
// transposed (a row per column, the eight key slots of a lane group together:
// one 16-byte read is an operand), each with its 16-byte chunks permuted by row
// so that reads of 16 rows meet distinct banks.  An FP8 cache is converted
// here, once for all the waves.
//
// Bound by the vector unit (a score costs an exponential and six more operations, with
// an FP8 cache's two scales) and the matrix cores in turn: 512 rows of 8 kv heads
// over 32768 keys, 69 GFLOP, 114 us bf16 with the join, 113 us FP8 without it, the
// matrix cores busy for 27% of that; 1024 rows of 8 kv heads over 32768 E2M1 keys, 138 GFLOP, 198
// us without it.  (Forming the scores of the next 32 keys
// under the exponentials of these takes the registers that hide LDS and loads: 170
// us bf16.)
template <int D, int KV, int RT>
__global__ __launch_bounds__(512, 2) void attn_tile_kernel(AttnArgs a, int np) {
  constexpr int NS = D / 32, VD = D / 16;
  constexpr bool FP8 = KV == kKvE4M3, FP4 = KV == kKvE2M1;
  constexpr int RB = FP4 ? D / 2 : FP8 ? D : 2 * D;  // bytes of a cache row
  constexpr int KC = RB / 16;                     // 16-byte pieces of a K row
  constexpr int SB = D / 32;                      // E2M1: scale bytes of a row, one per piece
  constexpr int VRW = FP4 ? 1 : FP8 ? 2 : 4;      // dwords of a V unit's key
  constexpr int NKL = 64 * KC / 512 ? 64 * KC / 512 : 1;   // K pieces per thread
  constexpr int CH = D / 8;                       // 16-byte chunks of an LDS K row
  __shared__ uint4 lk[2][64][CH];
  __shared__ uint4 lv[2][D][8];                   // [column][8 chunks of 8 key slots]
  // FP8: K scales; V scales in units of 2^-12 lbound
  __shared__ float lks[2][64], lvs[2][64], lbound;
  // marks by buffer: the tile (its first key) that holds a non-finite V, a bad page, V
  // scales far from lbound; whether a wave has set a group aside
  __shared__ int lleak[2], lbad[2], lfar[2], lslow;
  Item itm;
  if (!item_of(a, blockIdx.x, np, itm)) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int h = itm.h, rows = itm.rows;
  const int rblk = itm.rb * 128 * RT, r0 = rblk + wv * 16 * RT;

  uint4 q[RT][NS];
  int lim[RT];
  int minlim = 0x7fffffff, maxlim = 0;
  auto row_of = [&](int rt, int& tok, int& head) {
    const int rr = min(r0 + 16 * rt + c, rows - 1);
    tok = itm.t0 + rr / a.G;
    head = h * a.G + rr % a.G;
    return r0 + 16 * rt + c < rows;
  };
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    int tok, head;
    const bool in = row_of(rt, tok, head);
    lim[rt] = in ? row_limit(a, tok) : 0;
    if (lim[rt] > 0) minlim = min(minlim, lim[rt]);
    const uint16_t* qr = a.q + (size_t)tok * a.q_stride + (size_t)head * D;
#pragma unroll
    for (int s = 0; s < NS; ++s) q[rt][s] = *reinterpret_cast<const uint4*>(qr + 32 * s + 8 * g);
  }
  minlim = __builtin_amdgcn_readfirstlane(wave_min_all(minlim));
  // keys any row of the block sees (every wave walks the same tiles)
  for (int r = rblk + lane; r < min(rows, rblk + 128 * RT); r += 64)
    maxlim = max(maxlim, row_limit(a, itm.t0 + r / a.G));
  maxlim = __builtin_amdgcn_readfirstlane(wave_max_all(maxlim));
  const int lo = itm.rg.lo, hi = min(itm.rg.hi, maxlim);

  v4f_t o[RT][VD];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY, l[rt] = 0.0f;
#pragma unroll
    for (int j = 0; j < VD; ++j) o[rt][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
  }
  float bound = 0.0f, per = 1.0f;  // as in attn_item (wave 1's, which stages the scales)

  // this thread's pieces of a tile: K piece i is 16 bytes of key kkey + i x
  // (keys per round); V unit i is columns 8 vcol.. of keys 2 vkp, 2 vkp + 1
  constexpr int KPR = 512 / KC;     // keys per round of K loads
  const int kkey = tid / KC, kpc = tid % KC;
  constexpr int VU = D / 8 < 64 ? D / 8 : 64;
  const int vcol = tid % VU, vkp0 = tid / VU;    // 512 / VU key pairs per round
  constexpr int VPR = 512 / VU;
  constexpr int NV = 32 / VPR ? 32 / VPR : 1;
  static_assert(NV * VPR >= 32, "V rounds");
  uint4 kreg[NKL];
  uint32_t vreg[NV][2][VRW];
  uint8_t ksb[NKL], vsb[NV][2];  // E2M1: their scales
  float sreg = 0.0f;
  const int32_t* pages = itm.rg.pages;
  // the pages of this thread's pieces, fetched a tile ahead of them (a V unit's
  // two keys share one)
  int pgk[NKL], pgv[NV], pgs = 0;
  auto page_of = [&](int j) { return pages[max(lo, min(j, hi - 1)) >> a.page_shift]; };
  auto load_pages = [&](int j0) {
#pragma unroll
    for (int i = 0; i < NKL; ++i) pgk[i] = page_of(j0 + kkey + KPR * i);
#pragma unroll
    for (int i = 0; i < NV; ++i) pgv[i] = page_of(j0 + 2 * (vkp0 + VPR * i));
    if (FP8) pgs = page_of(j0 + (tid & 63));
  };
  bool badp = false;
  // cache row of key j in page pg (any valid row where j is outside [lo, hi))
  auto row_at = [&](int j, int pg, bool& ok) {
    const bool bad = pg < 0 || pg >= a.n_pages;
    if (bad && a.status) set_status(a.status, MOE_STATUS_BAD_PAGE);
    badp |= bad;
    ok = j >= lo && j < hi && !bad;
    return (((size_t)(bad ? 0 : pg) * a.Hkv + h) << a.page_shift) +
           (j & ((1 << a.page_shift) - 1));
  };
  uint32_t okbits = 0;  // of the loaded tile: K piece / V key / scale in range
  auto load_tile = [&](int j0) {
    okbits = 0;
    badp = false;
#pragma unroll
    for (int i = 0; i < NKL; ++i)
      if (64 * KC >= 512 || tid < 64 * KC) {
        bool ok;
        const size_t row = row_at(j0 + kkey + KPR * i, pgk[i], ok);
        kreg[i] = *reinterpret_cast<const uint4*>((const uint8_t*)a.k + row * RB + 16 * kpc);
        if constexpr (FP4) ksb[i] = ((const uint8_t*)a.ks)[row * SB + kpc];
      }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (VPR <= 32 || vkp0 < 32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          bool ok;
          const size_t row = row_at(j0 + 2 * (vkp0 + VPR * i) + k, pgv[i], ok);
          load_dwords((const uint8_t*)a.v + row * RB + 4 * VRW * vcol, vreg[i][k]);
          if constexpr (FP4) vsb[i][k] = ((const uint8_t*)a.vs)[row * SB + (vcol >> 2)];
          okbits |= ok ? 1u << (2 * i + k) : 0u;
        }
      }
    if (FP8 && tid < 128) {
      bool ok;
      const size_t row = row_at(j0 + (tid & 63), pgs, ok);
      sreg = ((const float*)(tid < 64 ? a.ks : a.vs))[row];
      okbits |= ok ? 0x80000000u : 0u;
    }
  };
  auto swz_k = [](int r, int ch) { return ch ^ (CH >= 16 ? r & 15 : (r >> 1) & 7); };
  auto swz_v = [](int d, int ch) { return ch ^ (((d >> 1) ^ (d >> 4)) & 7); };
  auto store_tile = [&](int buf, int j0) {
#pragma unroll
    for (int i = 0; i < NKL; ++i)
      if (64 * KC >= 512 || tid < 64 * KC) {
        const int r = kkey + KPR * i;
        const uint4 x = kreg[i];
        if constexpr (FP4) {
          const float sc = fp4_scale(ksb[i]);
          lk[buf][r][swz_k(r, 4 * kpc)] = fp4x8(x.x, sc);
          lk[buf][r][swz_k(r, 4 * kpc + 1)] = fp4x8(x.y, sc);
          lk[buf][r][swz_k(r, 4 * kpc + 2)] = fp4x8(x.z, sc);
          lk[buf][r][swz_k(r, 4 * kpc + 3)] = fp4x8(x.w, sc);
        } else if constexpr (FP8) {
          lk[buf][r][swz_k(r, 2 * kpc)] = fp8x8(x.x, x.y);
          lk[buf][r][swz_k(r, 2 * kpc + 1)] = fp8x8(x.z, x.w);
        } else {
          lk[buf][r][swz_k(r, kpc)] = x;
        }
      }
    bool leak = false;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (VPR <= 32 || vkp0 < 32) {
        const int kp = vkp0 + VPR * i;
        constexpr int W = FP8 ? 2 : 4;
        uint32_t vx[2][W];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (FP4) {
            const uint4 x = fp4x8(vreg[i][k][0], fp4_scale(vsb[i][k]));
            vx[k][0] = x.x, vx[k][1] = x.y, vx[k][2 % W] = x.z, vx[k][3 % W] = x.w;
          } else {
#pragma unroll
            for (int w = 0; w < W; ++w) vx[k][w] = vreg[i][k][w % VRW];
          }
        }
        // rows outside the item's keys may hold anything: cleared
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (!(okbits >> (2 * i + k) & 1u))
#pragma unroll
            for (int w = 0; w < W; ++w) vx[k][w] = 0u;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const uint32_t x = vx[k][w];
            if (FP8)
              leak |= (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
            else
              leak |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
          }
        // key slot of key 2 kp: {4g.., 16 + 4g..} of each 32 together
        const int k32 = (2 * kp) & 31;
        const int slot = ((2 * kp) & 32) + 8 * ((k32 & 15) >> 2) + (k32 & 3) + (k32 & 16 ? 4 : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t two;
          if constexpr (FP8)
            two = __builtin_bit_cast(
                uint32_t, e4m3x2_lo(__builtin_amdgcn_perm(vx[1][e / 4], vx[0][e / 4],
                                                          0x0c0c0400u + 0x0101u * (e & 3))));
          else
            two = __builtin_amdgcn_perm(vx[1][e / 2 % W], vx[0][e / 2 % W],
                                        (e & 1) ? 0x07060302u : 0x05040100u);
          const int d = 8 * vcol + e;
          reinterpret_cast<uint32_t*>(&lv[buf][d][swz_v(d, slot >> 3)])[(slot & 7) >> 1] = two;
        }
      }
    if (FP8 && wv == 0) lks[buf][lane] = sreg;
    if (FP8 && wv == 1) {
      const float v = okbits >> 31 ? sreg : 0.0f;
      const bool finite = fabsf(v) < INFINITY;
      leak |= !finite;
      if (bound == 0.0f) {
        const float first = wave_max(finite ? fabsf(v) : 0.0f);
        if (first > 0.0f) bound = scale_bound(first), per = 0x1p12f / bound;
        if (lane == 0) lbound = bound;
      }
      if (__ballot(okbits >> 31 && scale_far(fabsf(v), fabsf(v), bound)) && lane == 0)
        lfar[buf] = j0;
      lvs[buf][lane] = scale_units(v, per);
    }
    if (leak) lleak[buf] = j0;
    if (badp) lbad[buf] = j0;
  };

  // The tiles in turn.  SLOW: only the groups set aside by the first walk (false:
  // sets them aside, and says so): keys that only some of the wave's rows see, one of
  // them with a non-finite V, which must not meet the other rows' P = 0 (0 x inf is
  // NaN).
  auto walk = [&](auto slow) -> bool {
    constexpr bool SLOW = decltype(slow)::value;
    bool aside = false;
    int buf = 0, j0 = lo & ~31;
    if (j0 < hi) {
      load_pages(j0);
      load_tile(j0);
      load_pages(j0 + 64);
    }
    for (; j0 < hi; j0 += 64, buf ^= 1) {
      store_tile(buf, j0);
      __syncthreads();
      if (j0 + 64 < hi) {
        load_tile(j0 + 64);
        load_pages(j0 + 128);
      }
      const bool any_leak = lleak[buf] == j0, any_bad = lbad[buf] == j0;
      const bool any_far = FP8 && __builtin_amdgcn_readfirstlane(lfar[buf]) == j0;
      // Where registers allow, the scores of both halves first: their products run
      // under the first half's softmax (128 columns and two row tiles: one half at a time,
      // 131 us instead of 147 for 512 rows of a kv head over 32768 keys)
      constexpr int BOTH = RT == 1 || D == 64 ? 2 : 1;
#pragma unroll 1
      for (int kh = 0; kh < 2; kh += BOTH) {
        float x[BOTH][RT][8];
#pragma unroll
        for (int kb = 0; kb < BOTH; ++kb) {
          const int kt = kh + kb;
          v4f_t s0[RT], s1[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s0[rt] = s1[rt] = v4f_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const int ra = 32 * kt + c, rb = ra + 16;
            const uint4 k0 = lk[buf][ra][swz_k(ra, 4 * s + g)];
            const uint4 k1 = lk[buf][rb][swz_k(rb, 4 * s + g)];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              s0[rt] = mfma(k0, q[rt][s], s0[rt]);
              s1[rt] = mfma(k1, q[rt][s], s1[rt]);
            }
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[kb][rt][e] = s0[rt][e], x[kb][rt][4 + e] = s1[rt][e];
        }
#pragma unroll
        for (int kb = 0; kb < BOTH; ++kb) {
          const int kt = kh + kb;
          const int jk = j0 + 32 * kt;
          auto key_of = [&](int e) { return jk + 16 * (e >> 2) + 4 * g + (e & 3); };
          const bool edge = jk < lo || jk + 32 > min(hi, minlim) || any_bad;
          if (SLOW != (edge && any_leak)) {
            aside = true;
            continue;
          }
          float vscale[8];
          if constexpr (FP8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int at = 32 * kt + 16 * u + 4 * g;
              const float4 kk = *reinterpret_cast<const float4*>(&lks[buf][at]);
              const float4 vv = *reinterpret_cast<const float4*>(&lvs[buf][at]);
              const float k4[4] = {kk.x, kk.y, kk.z, kk.w}, v4[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[kb][rt][4 * u + e] *= k4[e];
                vscale[4 * u + e] = v4[e];
              }
            }
          }
          auto v_operand = [&](int j) {
            const int d = 16 * j + c;
            return lv[buf][d][swz_v(d, 4 * kt + g)];
          };
          // the first V operands arrive under the softmax
          constexpr int VPF = 4;
          uint4 va[VPF];
#pragma unroll
          for (int j = 0; j < VPF; ++j) va[j] = v_operand(j);
          uint4 p[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float mx;
            if (edge || any_far) {
              mx = -INFINITY;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if (edge && (key_of(e) < lo || key_of(e) >= min(hi, lim[rt]) ||
                             (any_bad && bad_key(a, pages, key_of(e), lo, hi))))
                  x[kb][rt][e] = -INFINITY;
                mx = fmaxf(mx, fmaf(x[kb][rt][e], a.scale_log2,
                                    FP8 ? scale_log2_of(vscale[e]) : 0.0f));
              }
            } else {
              mx = max8(x[kb][rt]) * a.scale_log2;
            }
            raise_max(mx, m[rt], [&](float f) {
              l[rt] *= f;
#pragma unroll
              for (int j = 0; j < VD; ++j) o[rt][j] *= f;
            });
            const float mu = m[rt] == -INFINITY ? 0.0f : m[rt];
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              w[e] = __builtin_amdgcn_exp2f(fmaf(x[kb][rt][e], a.scale_log2, -mu));
              l[rt] += w[e];
              // (0 x a non-finite scale: only in groups set aside)
              if (FP8) w[e] = SLOW && x[kb][rt][e] == -INFINITY ? 0.0f : w[e] * vscale[e];
            }
            p[rt] = pack_p<FP8>(w);
          }
          if constexpr (!SLOW) {
#pragma unroll
            for (int j = 0; j < VD; ++j) {
              const uint4 vf = j < VPF ? va[j % VPF] : v_operand(j);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) o[rt][j] = mfma_pv<FP8>(vf, p[rt], o[rt][j]);
            }
          } else {
            // one limit at a time, the values past it cleared
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
              for (int e = 0; e < 8; ++e) keep[e] = key_of(e) < done ? 0xffffffffu : 0u;
#pragma unroll
              for (int j = 0; j < VD; ++j) {
                uint4 vf = v_operand(j);
                vf.x &= (keep[0] & 0xffffu) | (keep[1] & 0xffff0000u);
                vf.y &= (keep[2] & 0xffffu) | (keep[3] & 0xffff0000u);
                vf.z &= (keep[4] & 0xffffu) | (keep[5] & 0xffff0000u);
                vf.w &= (keep[6] & 0xffffu) | (keep[7] & 0xffff0000u);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                  const v4f_t n = mfma_pv<FP8>(vf, p[rt], o[rt][j]);
                  if (lim[rt] == done) o[rt][j] = n;
                }
                __builtin_amdgcn_sched_barrier(0);
              }
            }
          }
        }
      }
    }
    return aside;
  };
  if (tid < 2) lleak[tid] = lbad[tid] = lfar[tid] = -1;
  if (tid == 2) lslow = 0, lbound = 0.0f;
  __syncthreads();
  if (walk(std::false_type{})) lslow = 1;
  __syncthreads();
  if (lslow) walk(std::true_type{});
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    int tok, head;
    float lsum = quad_sum(l[rt]), mr = m[rt];
    const int k = FP8 ? unit_weight(mr, lsum) : 0;
    if (!row_of(rt, tok, head)) continue;
    const size_t row = ((size_t)itm.part * a.n_tok + tok) * a.Hq + head;
    const bool none = lim[rt] == 0;
    if (g == 0)
      a.pml[row] = make_float2(none ? -INFINITY : part_max(mr, lsum), none ? 0.0f : lsum);
    float* dst = a.po + row * D + 4 * g;
    const float f = FP8 ? 0x1p-12f * lbound : 1.0f;
#pragma unroll
    for (int j = 0; j < VD; ++j) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[r] = FP8 ? __builtin_amdgcn_ldexpf(o[rt][j][r] * f, -k) : o[rt][j][r];
      *reinterpret_cast<float4*>(dst + 16 * j) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Joins a row's parts, weighted by 2^(m - M), and normalises.  D/4 lanes hold a
// row's columns; 4 such groups a row take its parts in turn, U loads at a time: 4
// where that takes all in one round (16 parts), 8 beyond (4 sequences of 560 keys, the
// whole call: 8.8 us, 9.1 with 8; one of 8192 keys: 11.0, 11.5 with 4).
constexpr int kJoinGroups = 4;
template <int D, int U>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int LPR = D / 4, RPB = 256 / (LPR * kJoinGroups);
  __shared__ float4 so[RPB][kJoinGroups][LPR];
  __shared__ float2 sml[RPB][kJoinGroups];
  const int ln = threadIdx.x % LPR, pg = threadIdx.x / LPR % kJoinGroups,
            rl = threadIdx.x / (LPR * kJoinGroups);
  const int64_t nrows = (int64_t)a.n_tok * a.Hq;
  const int64_t row_ = (int64_t)blockIdx.x * RPB + rl;
  const int64_t row = row_ < nrows ? row_ : nrows - 1;
  const int t = (int)(row / a.Hq), b = t / a.Q;
  const int parts = a.n_prefix_parts + own_parts(a, seq_limit(a, b));  // (a wave has one row)
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = pg; p0 < parts; p0 += kJoinGroups * U) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const size_t at = (size_t)min(p0 + kJoinGroups * i, parts - 1) * nrows + row;
      ml[i] = a.pml[at];
      v[i] = *reinterpret_cast<const float4*>(a.po + at * D + 4 * ln);
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (p0 + kJoinGroups * i >= parts) ml[i].x = -INFINITY;
      mn = fmaxf(mn, ml[i].x);
    }
    if (mn == -INFINITY) continue;
    const float f0 = __builtin_amdgcn_exp2f(M - mn);
    M = mn;
    L *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (ml[i].x != -INFINITY) {  // (a part without keys may hold anything)
        const float f = __builtin_amdgcn_exp2f(ml[i].x - M);
        L = fmaf(f, ml[i].y, L);
        o.x = fmaf(f, v[i].x, o.x), o.y = fmaf(f, v[i].y, o.y);
        o.z = fmaf(f, v[i].z, o.z), o.w = fmaf(f, v[i].w, o.w);
      }
  }
  so[rl][pg][ln] = o;
  if (ln == 0) sml[rl][pg] = make_float2(M, L);
  __syncthreads();
  if (pg || row_ >= nrows) return;
  for (int k = 0; k < kJoinGroups; ++k) M = fmaxf(M, sml[rl][k].x);
  L = 0.0f, o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < kJoinGroups; ++k) {
    if (sml[rl][k].x == -INFINITY) continue;
    const float f = __builtin_amdgcn_exp2f(sml[rl][k].x - M);
    const float4 v = so[rl][k][ln];
    L = fmaf(f, sml[rl][k].y, L);
    o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
  }
  const bool none = M == -INFINITY;
  if (!none) o.x /= L, o.y /= L, o.z /= L, o.w /= L;
  *reinterpret_cast<uint2*>(a.out + row * D + 4 * ln) =
      make_uint2(f32x2_to_bf16x2(o.x, o.y), f32x2_to_bf16x2(o.z, o.w));
  if (a.lse && ln == 0) a.lse[row] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  if (a.status && ln == 0 && a.pos[t] >= a.max_keys) set_status(a.status, MOE_STATUS_BAD_PAGE);
}

namespace {

// Items whose blocks take few rows (AttnArgs kinds 1, 2), both sorts in one launch.
template <int D, int KV>
void launch_few(const AttnArgs& a, int np, int no, hipStream_t st) {
  const bool p2 = np && a.prefix_kind == 2, s2 = no && a.own_kind == 2;
  if constexpr (D < 256) {
    if (p2 && !s2 && no) {
      attn_part_kernel<D, KV, 2, 1><<<np + no, 256, 0, st>>>(a, np);
      return;
    }
    if (p2 || s2) {  // (where both are there, the prefix's blocks are no smaller: attn_plan)
      attn_part_kernel<D, KV, 2, 2><<<np + no, 256, 0, st>>>(a, np);
      return;
    }
  }
  attn_part_kernel<D, KV, 1, 1><<<np + no, 256, 0, st>>>(a, np);
}

template <int D, int KV>
void launch_dim(const AttnArgs& a, hipStream_t st) {
  const int np = a.n_prefix_parts * a.Hkv * a.prefix_blocks;
  const int no = a.n_own_parts * a.B * a.Hkv * a.own_blocks;
  constexpr int RT = D == 256 ? 1 : 2;
  const int tp = a.prefix_kind == kAttnTile ? np : 0, ts = a.own_kind == kAttnTile ? no : 0;
  if (tp + ts) attn_tile_kernel<D, KV, RT><<<tp + ts, 512, 0, st>>>(a, tp);
  if (np + no > tp + ts) launch_few<D, KV>(a, np - tp, no - ts, st);
}

template <int D>
void launch_all(const AttnArgs& a, hipStream_t st) {
  if (a.kv == kKvE2M1)
    launch_dim<D, kKvE2M1>(a, st);
  else if (a.kv == kKvE4M3)
    launch_dim<D, kKvE4M3>(a, st);
  else
    launch_dim<D, kKvBf16>(a, st);
  constexpr int RPB = 256 / (D / 4 * kJoinGroups);
  const int64_t rows = (int64_t)a.n_tok * a.Hq;
  const unsigned blocks = (unsigned)((rows + RPB - 1) / RPB);
  if (a.n_prefix_parts + a.n_own_parts <= 4 * kJoinGroups)
    attn_join_kernel<D, 4><<<blocks, 256, 0, st>>>(a);
  else
    attn_join_kernel<D, 8><<<blocks, 256, 0, st>>>(a);
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
