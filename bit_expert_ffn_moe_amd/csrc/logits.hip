// logits.hip -- rules on logits: out = z + bias, then z > 0 ? z / p : z p for ids of the
// text, z - (presence + frequency c) for ids generated c times, -inf where the row's
// mask does not allow the id.
//
// A block owns C ids of a row.  Its share of the rules is gathered in LDS first, a word an
// id: the number of the id's last bias entry + 1 (bits 21..31), whether the id was given in
// the text (bit 20), how often it was generated (bits 0..19).  The gathering is whole numbers
// (atomic maximum, or, add in LDS), so its order does not show; every block of a row
// reads the row's text (from L2), so there is one launch and no workspace.  Then the
// logits stream through once.
#include <string.h>

#include "common.h"
#include "kernels.h"

namespace bef {

namespace {

constexpr int kGiven = 1 << 20, kCount = kGiven - 1, kBiasShift = 21;

// E elements at p, which has their own alignment only
template <bool BF16, int E>
__device__ __forceinline__ void load_z(const void* p, size_t at, float (&v)[E]) {
  if constexpr (BF16) {
    uint32_t w[E / 2];
    memcpy(w, (const uint16_t*)p + at, sizeof w);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      v[2 * i] = bf16_to_f32(w[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    memcpy(v, (const float*)p + at, sizeof v);
  }
}
template <bool BF16, int E>
__device__ __forceinline__ void store_z(void* p, size_t at, const float (&v)[E]) {
  if constexpr (BF16) {
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    memcpy((uint16_t*)p + at, w, sizeof w);
  } else {
    memcpy((float*)p + at, v, sizeof v);
  }
}
template <bool BF16>
__device__ __forceinline__ float load_1(const void* p, size_t at) {
  return BF16 ? bf16_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at];
}
template <bool BF16>
__device__ __forceinline__ void store_1(void* p, size_t at, float v) {
  if (BF16)
    ((uint16_t*)p)[at] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
  else
    ((float*)p)[at] = v;
}

struct Row {
  float rep, pres, freq;
  const float* bias;
};

// the rules of word w on a logit
__device__ __forceinline__ float ruled(float z, uint32_t w, const Row& r) {
  if (w >> kBiasShift) z += r.bias[(w >> kBiasShift) - 1];
  const uint32_t c = w & kCount;
  if (w & (kGiven | kCount)) z = z > 0.0f ? z / r.rep : z * r.rep;
  if (c) z -= r.pres + r.freq * (float)c;
  return z;
}

}  // namespace

// grid: (chunks of C ids, rows or some of them)
template <int C, bool ZB, bool OB, bool IN_PLACE>
__global__ __launch_bounds__(256) void logits_kernel(LogitsArgs a) {
  constexpr int E = 8, NV = C / (256 * E);
  __shared__ __align__(16) uint32_t word[C];
  const int v0 = blockIdx.x * C, n = min(C, a.V - v0);
  const int tid = threadIdx.x;
  const bool any = a.history || a.n_bias;
  for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
    if (any) {
      __syncthreads();
      for (int i = 4 * tid; i < C; i += 1024)
        *reinterpret_cast<uint4*>(word + i) = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    bool bad_id = false, bad_index = false;
    if (a.n_bias) {
      for (int i = tid; i < a.n_bias; i += 256) {
        const int id = a.bias_ids[(size_t)t * a.n_bias + i];
        bad_id |= id >= a.V;
        if (id >= v0 && id - v0 < n) atomicMax(word + (id - v0), (uint32_t)(i + 1) << kBiasShift);
      }
      __syncthreads();
    }
    if (a.history) {
      const int seq = a.seq_of ? a.seq_of[t] : t;
      const int total = a.n_tokens[t], given = a.n_prompt ? a.n_prompt[t] : 0;
      const bool has = seq >= 0 && seq < a.n_seqs;
      bad_index = seq >= a.n_seqs || (has && total > a.max_history);
      const int len = has ? min(total, a.max_history) : 0;
      const int32_t* ids = a.history + (size_t)(has ? seq : 0) * a.history_stride;
      for (int i = tid; i < len; i += 256) {
        const int id = ids[i];
        bad_id |= id >= a.V;
        if (id >= v0 && id - v0 < n) {
          if (i < given)
            atomicOr(word + (id - v0), (uint32_t)kGiven);
          else
            atomicAdd(word + (id - v0), 1u);
        }
      }
      __syncthreads();
    }
    int m = -1;
    if (a.mask) {
      m = a.mask_of ? a.mask_of[t] : t;
      if (m >= a.n_masks) bad_index = true, m = -1;
    }
    if (a.status && blockIdx.x == 0) {
      if (bad_id) set_status(a.status, MOE_STATUS_BAD_TOKEN);
      if (bad_index && tid == 0) set_status(a.status, MOE_STATUS_BAD_INDEX);
    }
    const uint32_t* mask = m < 0 ? nullptr : a.mask + (size_t)m * a.mask_stride;
    Row r;
    r.rep = a.repetition ? a.repetition[t] : 1.0f;
    r.pres = a.presence ? a.presence[t] : 0.0f;
    r.freq = a.frequency ? a.frequency[t] : 0.0f;
    r.bias = a.bias + (size_t)t * a.n_bias;
    const size_t zr = (size_t)t * a.z_stride + v0, outr = (size_t)t * a.out_stride + v0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * 256 + tid) * E;
      if (i >= n) break;
      uint32_t w[E], touched = 0;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const uint4 u = any ? *reinterpret_cast<const uint4*>(word + i + e) : make_uint4(0, 0, 0, 0);
        w[e] = u.x, w[e + 1] = u.y, w[e + 2] = u.z, w[e + 3] = u.w;
        touched |= u.x | u.y | u.z | u.w;
      }
      const uint32_t allowed = mask ? mask[(v0 + i) >> 5] >> ((v0 + i) & 31) & 0xffu : 0xffu;
      if (IN_PLACE && !touched && allowed == 0xffu) continue;
      if (i + E <= n) {
        float z[E];
        load_z<ZB, E>(a.z, zr + i, z);
        if (touched) {
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = w[e] ? ruled(z[e], w[e], r) : z[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = allowed >> e & 1u ? z[e] : -INFINITY;
        store_z<OB, E>(a.out, outr + i, z);
      } else {
        #pragma unroll
        for (int e = 0; e < E; ++e) {
          if (i + e >= n) break;
          float z = load_1<ZB>(a.z, zr + i + e);
          if (w[e]) z = ruled(z, w[e], r);
          if (IN_PLACE && !w[e] && (allowed >> e & 1u)) continue;
          store_1<OB>(a.out, outr + i + e, allowed >> e & 1u ? z : -INFINITY);
        }
      }
    }
  }
}

namespace {

template <int C>
void launch_c(const LogitsArgs& a, hipStream_t st) {
  const dim3 grid((a.V + C - 1) / C, a.T < 32768 ? a.T : 32768);
  if (a.z_bf16) {
    if (a.in_place)
      logits_kernel<C, true, true, true><<<grid, 256, 0, st>>>(a);
    else if (a.out_bf16)
      logits_kernel<C, true, true, false><<<grid, 256, 0, st>>>(a);
    else
      logits_kernel<C, true, false, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (a.in_place)
      logits_kernel<C, false, false, true><<<grid, 256, 0, st>>>(a);
    else if (a.out_bf16)
      logits_kernel<C, false, true, false><<<grid, 256, 0, st>>>(a);
    else
      logits_kernel<C, false, false, false><<<grid, 256, 0, st>>>(a);
  }
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, hipStream_t st) {
  if ((int64_t)a.T * a.V <= (1 << 19))
    launch_c<2048>(a, st);
  else
    launch_c<8192>(a, st);
  return hipGetLastError();
}

}  // namespace bef
