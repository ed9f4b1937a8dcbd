// spec_train_device.h -- device helpers of the operators that stream logit rows in segments.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spec_device.h"
#include "spec_train.h"

namespace specv {

constexpr int kTrPer = kTrSeg / kThreads;   // 32 logits per thread

template <int DT>
struct TrEl {
  static constexpr int n = DT == kDtBF16 ? 8 : 4;   // logits of a 16-byte vector
};

// 16 bytes from and to any address (rows of an odd vocabulary start off the 16-byte grid): the
// hardware takes unaligned vectors whole, and a wave's 64 of them are contiguous all the same.
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 ld16_any(const void* p) {
  const u32x4_any w = __builtin_nontemporal_load((const u32x4_any*)p);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool PAST>   // PAST: not to be read again soon
__device__ __forceinline__ void st16_any(void* p, uint4 x) {
  const u32x4_any w = {x.x, x.y, x.z, x.w};
  if constexpr (PAST) __builtin_nontemporal_store(w, (u32x4_any*)p);
  else *(u32x4_any*)p = w;
}

// This thread's 32 logits of the n logits at p: 16-byte vectors dealt round-robin over the
// threads; what lies past n reads as -inf.  All vectors go out together (those past n read the
// segment's first one), the one vector that n may cut is read again by element.
template <int DT>
__device__ __forceinline__ void tr_load(const void* p, int n, float (&v)[kTrPer]) {
  constexpr int kEl = TrEl<DT>::n, kSz = 16 / kEl;
  const int t0 = kEl * (int)threadIdx.x;
  uint4 x[kTrPer / kEl];
  if (n >= kEl) {   // uniform
#pragma unroll
    for (int q = 0; q < kTrPer / kEl; ++q) {
      const int e0 = t0 + kEl * kThreads * q;
      x[q] = ld16_any((const char*)p + (e0 + kEl <= n ? e0 : 0) * kSz);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kTrPer / kEl; ++q) x[q] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int q = 0; q < kTrPer / kEl; ++q) {
    if constexpr (DT == kDtBF16) {
      v[8 * q + 0] = bf16_lo(x[q].x); v[8 * q + 1] = bf16_hi(x[q].x); v[8 * q + 2] = bf16_lo(x[q].y); v[8 * q + 3] = bf16_hi(x[q].y);
      v[8 * q + 4] = bf16_lo(x[q].z); v[8 * q + 5] = bf16_hi(x[q].z); v[8 * q + 6] = bf16_lo(x[q].w); v[8 * q + 7] = bf16_hi(x[q].w);
    } else {
      v[4 * q + 0] = __uint_as_float(x[q].x); v[4 * q + 1] = __uint_as_float(x[q].y);
      v[4 * q + 2] = __uint_as_float(x[q].z); v[4 * q + 3] = __uint_as_float(x[q].w);
    }
  }
  if (n < kTrSeg)   // uniform
#pragma unroll
    for (int q = 0; q < kTrPer / kEl; ++q) {
      const int e0 = t0 + kEl * kThreads * q;
      if (e0 + kEl > n)
#pragma unroll
        for (int e = 0; e < kEl; ++e) {
          v[kEl * q + e] = -INFINITY;
          if (e0 < n && e0 + e < n) v[kEl * q + e] = logit_at<DT>(p, e0 + e);
        }
    }
}

// sum of 2^((v - m) c) over this thread's logits, m their wave's maximum: v c - fl(m c) in one fma
// (an operation a logit less than a difference and a product), whose terms share the rounding of
// m c, an exact fma of its own, taken off the sum.  For large m c, where that rounding has no bound
// that an exponential bears, the difference comes first.  m = +inf gives NaN; with m = -inf the
// sum is 0, or NaN where fmaxf has passed over one.
__device__ __forceinline__ float tr_sum_exp(const float (&v)[kTrPer], float m, float c) {
  float s = 0.f;
  if (m > -INFINITY) {
    float p[4] = {0.f, 0.f, 0.f, 0.f};   // (no exponential's result is needed by the next instruction)
    const float mc = m * c;
    if (__builtin_expect(fabsf(mc) < 0x1p20f, 1)) {   // uniform; the rounding is below 2^-4
#pragma unroll
      for (int j = 0; j < kTrPer; j += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) p[q] += __builtin_amdgcn_exp2f(fmaf(v[j + q], c, -mc));
      s = ((p[0] + p[1]) + (p[2] + p[3])) * __builtin_amdgcn_exp2f(-fmaf(m, c, -mc));
    } else {
#pragma unroll
      for (int j = 0; j < kTrPer; j += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) p[q] += __builtin_amdgcn_exp2f((v[j + q] - m) * c);
      s = (p[0] + p[1]) + (p[2] + p[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kTrPer; ++j)
      if (v[j] != v[j]) s = v[j];
  }
  return s;
}

// The workgroup's sum of n parts, relative to their maximum m (-inf: 0, or NaN), in fp64.
__device__ __forceinline__ double tr_total(const MaxSum* ms, int n, float c, float& m, float* redf, double* redd) {
  m = -INFINITY;
  for (int i = threadIdx.x; i < n; i += kThreads) m = fmaxf(m, ms[i].m);
  m = block_max(m, redf);
  double z = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const MaxSum p = ms[i];
    z += p.m > -INFINITY ? (double)p.s * exp2_split(((double)p.m - (double)m) * (double)c) : (double)p.s;
  }
  return block_sum_d(z, redd);
}
// ln sum e^(l / T) of a row from its parts; NaN for one with a NaN or +inf, or no finite logit.
__device__ __forceinline__ double tr_log_z(const MaxSum* ms, int n, float c, double inv_t, float& m, float* redf,
                                           double* redd) {
  const double z = tr_total(ms, n, c, m, redf, redd);
  if (!(z > 0.0)) return __longlong_as_double(0x7ff8000000000000ll);
  return (double)m * inv_t + log2_split(z) * 0.6931471805599453;
}

}  // namespace specv
