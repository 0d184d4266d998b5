// logits.hip -- rules on logits: out = z + bias, then z > 0 ? z / p : z p for ids of the
// text, z - (presence + frequency c) for ids generated c times, -inf where the row's
// mask does not allow the id.
//
// A block owns C ids of a row.  Its share of the rules is gathered in LDS, a word an id: the
// number of the id's last bias entry + 1 (bits 21..31), whether the id was given in the text
// (bit 20), how often it was generated (bits 0..19).  The gathering is whole numbers (atomic
// maximum, or, add in LDS), so its order does not show; every block of a row reads the row's
// text (from L2), so there is one launch and no workspace.  Whoever finds a word empty puts
// its id on a list.  The logits stream past, under the mask alone; then the list's are
// written again, under their rules.
//
// 256 rows of 131072 fp32 logits with all the rules, 4096 ids of text and 100 biases a row, 274 MB:
// 68.7 us.  The logits alone take 50 (the rate of a large copy), the mask 2 more, the biases 5, a
// text 14, most of them for the second look at each id that it holds: 4 bytes read and written at
// random cost a line each.  The rules applied as the logits pass, which then have to wait for the
// text, took 95; blocks of 256 threads and counts in bytes or bits of LDS 70 to 92.  Few
// rows: a launch and three dependent trips to memory, text, LDS, logit (4.3 us).
#include <string.h>

#include "common.h"
#include "kernels.h"

namespace bef {

namespace {

constexpr int kGiven = 1 << 20, kCount = kGiven - 1, kBiasShift = 21;
constexpr int kThreads = 512;

// E logits as loaded from a place with their alignment only, and their values
template <bool BF16, int E>
struct Logits {
  uint32_t w[E / (BF16 ? 2 : 1)];
  __device__ __forceinline__ void load(const void* p, size_t at) {
    memcpy(w, (const uint8_t*)p + at * (BF16 ? 2 : 4), sizeof w);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF16)
      return i & 1 ? __uint_as_float(w[i / 2] & 0xffff0000u) : bf16_to_f32(w[i / 2] & 0xffffu);
    else
      return __uint_as_float(w[i]);
  }
};
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

// grid: (chunks of C ids, rows or some of them).  What can be read at once is: the logits,
// the mask and the text's first kThreads x 8 ids are on their way while LDS is cleared.
template <int C, bool ZB, bool OB, bool IN_PLACE>
__global__ __launch_bounds__(kThreads, 6) void logits_kernel(LogitsArgs a) {
  constexpr int E = ZB ? 8 : 4, STEP = kThreads * E, NV = C / STEP ? C / STEP : 1;
  constexpr uint32_t ALL = (1u << E) - 1;
  __shared__ __align__(16) uint32_t word[C];
  __shared__ uint16_t list[C];
  __shared__ int listed;
  const int tid = threadIdx.x;
  const bool any = a.history || a.n_bias;
  for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
    // rows start at different chunks: blocks of one chunk, some of which hold most of every
    // text, would otherwise meet on one XCD where the chunks' number is a multiple of 8
    const int v0 = (int)((blockIdx.x + t) % gridDim.x) * C, n = min(C, a.V - v0);
    const size_t zr = (size_t)t * a.z_stride + v0, outr = (size_t)t * a.out_stride + v0;
    bool bad_id = false, bad_index = false;
    int m = -1;
    if (a.mask) {
      m = a.mask_of ? a.mask_of[t] : t;
      if (m >= a.n_masks) bad_index = true, m = -1;
    }
    const uint32_t* mask = m < 0 ? nullptr : a.mask + (size_t)m * a.mask_stride + (v0 >> 5);
    Logits<ZB, E> z[NV];
    uint32_t ok[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * STEP + tid * E;
      if (!IN_PLACE && i + E <= n) z[k].load(a.z, zr + i);
      ok[k] = mask && i < n ? mask[i >> 5] : 0xffffffffu;
    }
    // the row's text
    int len = 0, given = 0;
    const int32_t* ids = a.history;
    if (a.history) {
      const int seq = a.seq_of ? a.seq_of[t] : t, total = a.n_tokens[t];
      given = a.n_prompt ? a.n_prompt[t] : 0;
      const bool has = seq >= 0 && seq < a.n_seqs;
      bad_index |= seq >= a.n_seqs || (has && total > a.max_history);
      len = has ? min(total, a.max_history) : 0;
      ids += (size_t)(has ? seq : 0) * a.history_stride;
    }
    int q[8];
    auto load_ids = [&](int from) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = from + k * kThreads + tid;
        q[k] = i < len ? ids[i] : -1;
      }
    };
    auto mine = [&](int id) { return id >= v0 && id - v0 < n; };
    load_ids(0);
    const int32_t* bias_ids = a.bias_ids + (size_t)t * a.n_bias;

    if (any) {
#pragma unroll
      for (int i = 4 * tid; i < C; i += 4 * kThreads)
        *reinterpret_cast<uint4*>(word + i) = make_uint4(0, 0, 0, 0);
      if (tid == 0) listed = 0;
      __syncthreads();
      auto met = [&](int at, uint32_t before) {
        if (before == 0) list[atomicAdd(&listed, 1)] = (uint16_t)at;
      };
      if (a.n_bias) {
        for (int i = tid; i < a.n_bias; i += kThreads) {
          const int id = bias_ids[i];
          bad_id |= id >= a.V;
          if (mine(id)) met(id - v0, atomicMax(word + (id - v0), (uint32_t)(i + 1) << kBiasShift));
        }
        __syncthreads();
      }
#pragma unroll 1
      for (int from = 0; from < len; from += 8 * kThreads) {
        if (from) load_ids(from);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          bad_id |= q[k] >= a.V;
          if (!mine(q[k])) continue;
          uint32_t* w = word + (q[k] - v0);
          met(q[k] - v0, from + k * kThreads + tid < given ? atomicOr(w, (uint32_t)kGiven)
                                                            : atomicAdd(w, 1u));
        }
      }
    }
    if (a.status && v0 == 0) {
      if (bad_id) set_status(a.status, MOE_STATUS_BAD_TOKEN);
      if (bad_index && tid == 0) set_status(a.status, MOE_STATUS_BAD_INDEX);
    }

#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = k * STEP + tid * E;
      if (i >= n) break;
      const uint32_t o = ok[k] >> (i & 31) & ALL;
      if (IN_PLACE && o == ALL) continue;
      if (i + E <= n && (!IN_PLACE || o == 0)) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = !IN_PLACE && (o >> e & 1u) ? z[k][e] : -INFINITY;
        store_z<OB, E>(a.out, outr + i, v);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool allow = o >> e & 1u;
          if (i + e < n && !(IN_PLACE && allow))
            store_1<OB>(a.out, outr + i + e, allow ? load_1<ZB>(a.z, zr + i + e) : -INFINITY);
        }
      }
    }
    if (!any) continue;
    // the gathered words are whole, and what this block wrote lies before what follows
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    Row r;
    r.rep = a.repetition ? a.repetition[t] : 1.0f;
    r.pres = a.presence ? a.presence[t] : 0.0f;
    r.freq = a.frequency ? a.frequency[t] : 0.0f;
    r.bias = a.bias + (size_t)t * a.n_bias;
    for (int j = tid; j < listed; j += kThreads) {
      const int i = list[j];
      if (mask && !(mask[i >> 5] >> (i & 31) & 1u)) continue;
      store_1<OB>(a.out, outr + i, ruled(load_1<ZB>(a.z, zr + i), word[i], r));
    }
    __syncthreads();  // (before the next row clears the words)
  }
}

namespace {

template <int C>
void launch_c(const LogitsArgs& a, hipStream_t st) {
  const dim3 grid((a.V + C - 1) / C, a.T < 32768 ? a.T : 32768);
  if (a.z_bf16) {
    if (a.in_place)
      logits_kernel<C, true, true, true><<<grid, kThreads, 0, st>>>(a);
    else if (a.out_bf16)
      logits_kernel<C, true, true, false><<<grid, kThreads, 0, st>>>(a);
    else
      logits_kernel<C, true, false, false><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (a.in_place)
      logits_kernel<C, false, false, true><<<grid, kThreads, 0, st>>>(a);
    else if (a.out_bf16)
      logits_kernel<C, false, true, false><<<grid, kThreads, 0, st>>>(a);
    else
      logits_kernel<C, false, false, false><<<grid, kThreads, 0, st>>>(a);
  }
}

}  // namespace

// Chunks of 2048 ids spread few logits over more of the chip (fp32, texts of 2000 tokens,
// 131072 ids: 1 row 4.3 us, 5.2 in chunks of 8192; 8 rows 6.1 and 6.7; 16 rows of 32000: 5.4 and
// 6.8); with many, every chunk reads its row's text again (16 rows 10.7 and 8.8; 64 rows of 32000:
// 11.2 and 9.4).  Chunks of 4096 and of 16384 ids take longer than both with 256 rows.
hipError_t launch_logits(const LogitsArgs& a, hipStream_t st) {
  if ((int64_t)a.T * a.V <= (1 << 20))
    launch_c<2048>(a, st);
  else
    launch_c<8192>(a, st);
  return hipGetLastError();
}

}  // namespace bef
