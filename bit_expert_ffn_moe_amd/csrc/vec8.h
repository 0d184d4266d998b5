// vec8.h -- a lane's 8 consecutive elements: bf16 words to fp32 and back, and their E4M3
// codes under one scale for a group of lanes.
#pragma once
#include "common.h"

namespace bef {

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

// E4M3 codes of the 8 values of a lane, with one scale amax/448 for the aligned group of
// G lanes (in every lane of it), by the rule of act_quant_fp8; a NaN keeps its place (the
// maximum and the conversion's clamp pass over it) and leaves the other values as they are.
template <int G>
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float& sc) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = group_max<G>(amax);
  sc = amax / 448.0f;
  uint2 q = make_uint2(0, 0);
  if (amax != 0.0f) {
    q.x = e4m3_pack4(v[0] / sc, v[1] / sc, v[2] / sc, v[3] / sc);
    q.y = e4m3_pack4(v[4] / sc, v[5] / sc, v[6] / sc, v[7] / sc);
  }
  const uint2 nan = make_uint2(nan_bytes(v), nan_bytes(v + 4));
  if (__ballot((nan.x | nan.y) != 0))
    q = make_uint2((q.x & ~(nan.x << 1)) | nan.x, (q.y & ~(nan.y << 1)) | nan.y);
  return q;
}

}  // namespace bef
