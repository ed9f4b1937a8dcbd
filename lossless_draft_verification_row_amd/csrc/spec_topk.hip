// spec_topk.hip -- the k largest logits of each row, with the row's log Z.
//
//   k_tk_seg    one workgroup per 8192 logits of a row, all in registers: the segment's maximum
//               and sum of exponentials, and every logit that can be among the row's k largest
//   k_tk_merge  one workgroup per row: the segments' candidates -> the k largest, in order
//
// A logit's 64-bit key holds its order key (a larger logit, a larger key; -0 counts as +0) above
// the complement of its index, so that keys are distinct and equal logits rank by index.  The
// k-th largest of a segment's 256 per-thread maxima (of each thread's two largest for k > 128) is
// no larger than the segment's k-th largest logit, so what reaches it holds the segment's k
// largest; for a row without order that is a few more than k.  Where more than `cap` reach it
// (ties, an ordered row) the exact k-th key is found by bisection over its bits.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spec_device.h"
#include "spec_train.h"

namespace specv {

constexpr int kPer = kTrSeg / kThreads;   // 32 logits per thread

__device__ __forceinline__ uint32_t tk_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);   // -0 -> +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float tk_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // tk_key(-inf)

// Index of register j of this thread: 16-byte vectors dealt round-robin over the threads.
template <int DT>
__device__ __forceinline__ int tk_index(int j) {
  constexpr int kEl = DT == kDtBF16 ? 8 : 4;
  return kEl * ((int)threadIdx.x + kThreads * (j / kEl)) + j % kEl;
}
template <int DT, bool VEC>
__device__ __forceinline__ void tk_load(const void* row, int V, int base, float (&v)[kPer]) {
  constexpr int kEl = DT == kDtBF16 ? 8 : 4;
#pragma unroll
  for (int q = 0; q < kPer / kEl; ++q) {
    const int e0 = base + tk_index<DT>(q * kEl);
    if (VEC && e0 + kEl <= V) {
      const uint4 x = ld_nt16((const char*)row + (int64_t)e0 * (16 / kEl));
      if constexpr (DT == kDtBF16) {
        v[8 * q + 0] = bf16_lo(x.x); v[8 * q + 1] = bf16_hi(x.x); v[8 * q + 2] = bf16_lo(x.y); v[8 * q + 3] = bf16_hi(x.y);
        v[8 * q + 4] = bf16_lo(x.z); v[8 * q + 5] = bf16_hi(x.z); v[8 * q + 6] = bf16_lo(x.w); v[8 * q + 7] = bf16_hi(x.w);
      } else {
        v[4 * q + 0] = __uint_as_float(x.x); v[4 * q + 1] = __uint_as_float(x.y);
        v[4 * q + 2] = __uint_as_float(x.z); v[4 * q + 3] = __uint_as_float(x.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kEl; ++e) v[kEl * q + e] = e0 + e < V ? logit_at<DT>(row, e0 + e) : -INFINITY;
    }
  }
}

// The K-th largest of the workgroup's 256 (NM = 1) or 512 (NM = 2) values x, by counting the
// larger ones (ties by place); 1 <= K <= 256.
template <typename T, int NM>
__device__ __forceinline__ T kth_of_maxima(const T (&x)[NM], int K, T* lds, T* res) {
#pragma unroll
  for (int n = 0; n < NM; ++n) lds[NM * threadIdx.x + n] = x[n];
  __syncthreads();
  int rank[NM];
#pragma unroll
  for (int n = 0; n < NM; ++n) rank[n] = 0;
  for (int i = 0; i < NM * kThreads; ++i) {
    const T o = lds[i];
#pragma unroll
    for (int n = 0; n < NM; ++n) rank[n] += o > x[n] || (o == x[n] && i < (int)(NM * threadIdx.x + n)) ? 1 : 0;
  }
#pragma unroll
  for (int n = 0; n < NM; ++n)
    if (rank[n] == K - 1) *res = x[n];
  __syncthreads();
  return *res;
}
__device__ __forceinline__ int block_sum_i(int v, int* red) {
  v = wave_sum_i(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  int r = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) r += red[i];
  __syncthreads();
  return r;
}

template <int DT, bool VEC, int NM>
__global__ __launch_bounds__(kThreads) void k_tk_seg(TopkArgs a) {
  __shared__ uint32_t mx[NM * kThreads];
  __shared__ uint32_t res;
  __shared__ int red[2 * kWaves];
  __shared__ int count;
  __shared__ float redf[2 * kWaves];
  const int seg = blockIdx.x % a.n_seg, r = blockIdx.x / a.n_seg, base = seg * kTrSeg;
  const void* row = row_ptr<DT>(a.logits, a.ld, r);
  float v[kPer];
  tk_load<DT, VEC>(row, a.V, base, v);
  if (threadIdx.x == 0) count = 0;
  float m1 = -INFINITY, m2 = -INFINITY;
  int bad = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    bad |= !(v[j] < INFINITY) ? 1 : 0;
    if constexpr (NM == 2) m2 = fmaxf(m2, fminf(m1, v[j]));
    m1 = fmaxf(m1, v[j]);
  }
  const float m = block_max(m1, redf);
  float s = 0.f;
  if (m > -INFINITY) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += __builtin_amdgcn_exp2f((v[j] - m) * a.c);
  }
  bad = block_or(bad, red);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) redf[threadIdx.x >> 6] = s;
  const int64_t slot = (int64_t)r * a.n_seg + seg;
  if (bad) {   // uniform
    if (threadIdx.x == 0) a.n_cand[slot] = -1;
    return;
  }
  uint32_t x[NM];
  x[0] = tk_key(m1);
  if constexpr (NM == 2) x[1] = tk_key(m2);
  uint32_t thr = kth_of_maxima<uint32_t, NM>(x, a.K, mx, &res);
  if (threadIdx.x == 0) a.ms[slot] = MaxSum{m, (redf[0] + redf[1]) + (redf[2] + redf[3])};
  if (thr <= kKeyNegInf) thr = kKeyNegInf + 1;   // a logit of -inf is no candidate
  int n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) n += tk_key(v[j]) >= thr ? 1 : 0;
  const int total = block_sum_i(n, red);
  int last = INT_MAX;   // of the keys equal to thr, those up to this index
  if (total > a.cap) {
    // exactly the K largest: the K-th largest key, then the index of its last one
    uint32_t lo = thr, hi = 0xffffffffu;   // count(>= lo) >= K
    while (lo < hi) {
      const uint32_t mid = lo + (uint32_t)(((uint64_t)hi - lo + 1) / 2);
      n = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) n += tk_key(v[j]) >= mid ? 1 : 0;
      if (block_sum_i(n, red) >= a.K) lo = mid;
      else hi = mid - 1;
    }
    thr = lo;
    n = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) n += tk_key(v[j]) > thr ? 1 : 0;
    const int ties = a.K - block_sum_i(n, red);   // >= 1
    int il = 0, ih = kTrSeg - 1;
    while (il < ih) {
      const int mid = (il + ih) / 2;
      n = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) n += tk_key(v[j]) == thr && tk_index<DT>(j) <= mid ? 1 : 0;
      if (block_sum_i(n, red) >= ties) ih = mid;
      else il = mid + 1;
    }
    last = il;
  }
  uint64_t* out = a.cand + slot * a.cap;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t k = tk_key(v[j]);
    if (k > thr || (k == thr && tk_index<DT>(j) <= last)) {
      const int i = atomicAdd(&count, 1);
      out[i] = ((uint64_t)k << 32) | (uint32_t)~(base + tk_index<DT>(j));
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.n_cand[slot] = count;
}

constexpr int kMergeCap = 1024;   // candidates that are ranked against each other

template <int NM>
__global__ __launch_bounds__(kThreads) void k_tk_merge(TopkArgs a) {
  __shared__ uint64_t key[kMergeCap];
  __shared__ uint64_t res;
  __shared__ int red[2 * kWaves];
  __shared__ float redf[2 * kWaves];
  __shared__ double redd[kWaves];
  __shared__ int count;
  const int r = blockIdx.x, t = threadIdx.x;
  const MaxSum* ms = a.ms + (int64_t)r * a.n_seg;
  const int32_t* nc = a.n_cand + (int64_t)r * a.n_seg;
  const uint64_t* cand = a.cand + (int64_t)r * a.n_seg * a.cap;
  int32_t* oi = a.index + (int64_t)r * a.K;
  float* ol = a.logit + (int64_t)r * a.K;
  const float nan = __int_as_float(0x7fc00000);
  if (t == 0) count = 0;
  int bad = 0;
  float m = -INFINITY;
  for (int i = t; i < a.n_seg; i += kThreads) {
    if (nc[i] < 0) bad = 1;
    else m = fmaxf(m, ms[i].m);
  }
  bad = block_or(bad, red);
  m = block_max(m, redf);
  if (bad || m == -INFINITY) {   // NaN or +inf, or no finite logit
    for (int j = t; j < a.K; j += kThreads) {
      oi[j] = -1;
      ol[j] = nan;
    }
    if (t == 0 && a.log_z) a.log_z[r] = nan;
    return;
  }
  double z = 0.0;
  for (int i = t; i < a.n_seg; i += kThreads)
    if (ms[i].m > -INFINITY) z += (double)ms[i].s * (double)__builtin_amdgcn_exp2f((ms[i].m - m) * a.c);
  z = block_sum_d(z, redd);
  if (t == 0 && a.log_z) a.log_z[r] = (float)((double)m * a.inv_t + log2_split(z) * 0.6931471805599453);

  // the largest candidates of each thread, and from them a bound that the K largest reach
  uint64_t x[NM];
#pragma unroll
  for (int n = 0; n < NM; ++n) x[n] = 0;
  int total = 0;
  const int n_all = a.n_seg * a.cap;
  for (int i = t; i < n_all; i += kThreads)
    if (i % a.cap < nc[i / a.cap]) {
      const uint64_t k = cand[i];
      ++total;
      if constexpr (NM == 2) {
        if (k > x[0]) { x[1] = x[0]; x[0] = k; }
        else if (k > x[1]) x[1] = k;
      } else {
        x[0] = k > x[0] ? k : x[0];
      }
    }
  total = block_sum_i(total, red);
  uint64_t thr = 1;
  if (total > kMergeCap) {
    thr = kth_of_maxima<uint64_t, NM>(x, a.K, key, &res);
    if (thr == 0) thr = 1;
    int n = 0;
    for (int i = t; i < n_all; i += kThreads) n += i % a.cap < nc[i / a.cap] && cand[i] >= thr ? 1 : 0;
    if (block_sum_i(n, red) > kMergeCap) {
      uint64_t lo = thr, hi = ~0ull;   // count(>= lo) >= K: the keys are distinct
      while (lo < hi) {
        const uint64_t mid = lo + (hi - lo) / 2 + 1;
        n = 0;
        for (int i = t; i < n_all; i += kThreads) n += i % a.cap < nc[i / a.cap] && cand[i] >= mid ? 1 : 0;
        if (block_sum_i(n, red) >= a.K) lo = mid;
        else hi = mid - 1;
      }
      thr = lo;
    }
    __syncthreads();
  }
  for (int i = t; i < n_all; i += kThreads)
    if (i % a.cap < nc[i / a.cap] && cand[i] >= thr) key[atomicAdd(&count, 1)] = cand[i];
  __syncthreads();
  const int n = count;
  for (int i = t; i < n; i += kThreads) {
    const uint64_t k = key[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += key[j] > k ? 1 : 0;
    if (rank < a.K) {
      oi[rank] = (int32_t)~(uint32_t)k;
      ol[rank] = tk_value((uint32_t)(k >> 32));
    }
  }
  for (int j = n + t; j < a.K; j += kThreads) {   // fewer finite logits than K
    oi[j] = -1;
    ol[j] = -INFINITY;
  }
}

namespace {
template <int DT, bool VEC, int NM>
void row_topk(const TopkArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_tk_seg<DT, VEC, NM>), dim3((unsigned)(a.R * a.n_seg)), dim3(kThreads), 0, st, a);
  hipLaunchKernelGGL((k_tk_merge<NM>), dim3((unsigned)a.R), dim3(kThreads), 0, st, a);
}
template <int DT, bool VEC>
void row_topk_k(const TopkArgs& a, hipStream_t st) {
  if (a.K > 128) row_topk<DT, VEC, 2>(a, st);
  else row_topk<DT, VEC, 1>(a, st);
}
}  // namespace

hipError_t launch_row_topk(const TopkArgs& a, int dt, int vec, hipStream_t st) {
  if (dt == kDtBF16) vec ? row_topk_k<kDtBF16, true>(a, st) : row_topk_k<kDtBF16, false>(a, st);
  else vec ? row_topk_k<kDtF32, true>(a, st) : row_topk_k<kDtF32, false>(a, st);
  return hipGetLastError();
}

}  // namespace specv
