// norm.hip -- the residual's addition and the root-mean-square norm, with an E4M3 output
// for the experts and the FP8 linears:
//   r = x + residual (stored in the residual's type; the norm is of what is stored),
//   y = r / sqrt(mean(r^2) + eps) w,  q = E4M3(y / s), s = amax/448 per 128 columns.
//
// One pass: a block owns a row, which stays in its registers (fp32) between the sum of
// squares and the outputs.  y is quantised from fp32, so a code is off by one
// rounding; r is rounded first because the next block reads the stored stream.
//
// A sum of squares past fp32's range (|r| from 2^57 on at 16384 columns) is formed again
// in units of the row's largest power of two; small squares need no such care, since eps
// >= 2^-100 is far above what underflow loses.
//
// Bound by HBM where tokens are many: 8192 of 4096 columns with residual, E4M3 and scales, 302
// MB read and written in 56.3 us, 5.4 TB/s, what a copy of that size takes.  A few tokens
// cost a launch, one trip to memory and one through LDS (2.6 us at 4096 columns, which is less
// than the caller's thread takes to launch it).
#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace bef {

namespace {

// Sum over the block, in every thread.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* tmp) {
  v = wave_sum_dpp(v);
  if constexpr (THREADS == 64) return v;
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) s += tmp[i];
  return s;
}

}  // namespace

// NV x 8 elements a thread: chunk i of thread t is elements 8 (i THREADS + t)...
template <int THREADS, int NV, bool QUANT>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a) {
  __shared__ float tmp[THREADS / 64], tmp2[THREADS / 64], tmp3[THREADS / 64];
  const size_t t = blockIdx.x;
  const int nch = a.H >> 3;
  const uint16_t* xr = a.x + t * a.x_stride;
  uint4 xv[NV], wv[NV], rv[NV][2];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = min(i * THREADS + (int)threadIdx.x, nch - 1);
    xv[i] = *reinterpret_cast<const uint4*>(xr + 8 * c);
    rv[i][0] = rv[i][1] = make_uint4(0, 0, 0, 0);
    if (a.res) {
      if (a.res_f32) {
        const uint4* p = reinterpret_cast<const uint4*>((const float*)a.res + t * a.res_stride + 8 * c);
        rv[i][0] = p[0], rv[i][1] = p[1];
      } else {
        rv[i][0] = *reinterpret_cast<const uint4*>((const uint16_t*)a.res + t * a.res_stride + 8 * c);
      }
    }
    wv[i] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    if (a.w) wv[i] = *reinterpret_cast<const uint4*>(a.w + 8 * c);
  }
  float r[NV][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * THREADS + threadIdx.x;
    unpack8(xv[i], r[i]);
    if (a.res) {
      float b[8];
      if (a.res_f32) {
        const uint32_t u[8] = {rv[i][0].x, rv[i][0].y, rv[i][0].z, rv[i][0].w,
                               rv[i][1].x, rv[i][1].y, rv[i][1].z, rv[i][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] += __uint_as_float(u[e]);
        if (a.res_out && c < nch) {
          float4* o = reinterpret_cast<float4*>((float*)a.res_out + t * a.res_stride + 8 * c);
          o[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
          o[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        }
      } else {
        unpack8(rv[i][0], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] += b[e];
        const uint4 p = pack8(r[i]);
        if (a.res_out && c < nch)
          *reinterpret_cast<uint4*>((uint16_t*)a.res_out + t * a.res_stride + 8 * c) = p;
        unpack8(p, r[i]);
      }
    }
    if (c >= nch)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(r[i][e], r[i][e], ss);
  }
  ss = block_sum<THREADS>(ss, tmp);
  float eps = a.eps;
  if (ss == INFINITY) {  // (the same in every thread)
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(r[i][e]));
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) tmp2[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) m = fmaxf(m, tmp2[i]);
    if (m < INFINITY) {  // r and sqrt(eps) in units of 2^k
      const int k = (int)(__float_as_uint(m) >> 23) - 127;
      eps = ldexpf(eps, -2 * k);
      ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          r[i][e] = ldexpf(r[i][e], -k);
          ss = fmaf(r[i][e], r[i][e], ss);
        }
      ss = block_sum<THREADS>(ss, tmp3);
    }
  }
  const float rs = 1.0f / sqrtf(ss / (float)a.H + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * THREADS + threadIdx.x;
    float y[8], w[8];
    unpack8(wv[i], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = r[i][e] * rs * w[e];
    if (a.y && c < nch) *reinterpret_cast<uint4*>(a.y + t * a.H + 8 * c) = pack8(y);
    if constexpr (QUANT) {  // (16 lanes a group of 128 columns)
      float sc;
      const uint2 q = e4m3x8<16>(y, sc);
      if (c < nch) {
        *reinterpret_cast<uint2*>(a.q + t * a.H + 8 * c) = q;
        if ((threadIdx.x & 15) == 0) a.qs[t * (a.H >> 7) + (c >> 4)] = sc;
      }
    }
  }
}

namespace {

template <int THREADS, int NV>
void launch_nv(const NormArgs& a, hipStream_t st) {
  if (a.q)
    norm_kernel<THREADS, NV, true><<<a.T, THREADS, 0, st>>>(a);
  else
    norm_kernel<THREADS, NV, false><<<a.T, THREADS, 0, st>>>(a);
}

}  // namespace

// A row's time is the latency of its loads and of the block's sum, so a thread has one chunk
// of 8 where a block can have that many threads (1024 columns, 64 rows: 2.7 us so, 3.3 with
// two; 2048: 2.7 and 3.5; 4096: 3.1 and 3.6; 8192: 4.6 and 4.7, 5.5 with four).  Thousands
// of rows of up to 4096 columns stream faster from smaller blocks (4096 rows of 4096: 28.0 us
// with two chunks a thread, 29.3 with one; 2048 rows 16.4 and 15.9).
hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  const int nch = a.H >> 3;
  if (nch <= 64)
    launch_nv<64, 1>(a, st);
  else if (nch <= 128)
    launch_nv<128, 1>(a, st);
  else if (nch <= 256)
    launch_nv<256, 1>(a, st);
  else if (nch <= 512 && a.T > 2048)
    launch_nv<256, 2>(a, st);
  else if (nch <= 512)
    launch_nv<512, 1>(a, st);
  else if (nch <= 1024)
    launch_nv<1024, 1>(a, st);
  else
    launch_nv<1024, 2>(a, st);
  return hipGetLastError();
}

}  // namespace bef
