// spec_distill.hip -- distillation of logit rows from a teacher's top logits, with its gradient.
//
//   q = softmax(s / T) of a student row s; the teacher's list holds tokens x_j with logits t_j.
//   Without the teacher's log Z the list is the teacher:  p_j = softmax(t / T)_j,  rho = 0.
//   With it:  p_j = e^(t_j / T - log Z),  rho = max(0, 1 - sum_j p_j)  is the mass off the list.
//   L = sum_j p_j (ln p_j - ln q_(x_j)) + rho (ln rho - ln q_rho),  q_rho = sum off the list of q
//   dL/ds_v = (M q_v - sum of p_j with x_j = v) / T on the list, (M - rho / q_rho) q_v / T off it,
//   M = sum_j p_j + rho.
// Off the list the gradient is one factor per row times 2^((s_v - m) log2(e) / T), m the largest
// logit off the list, so that a small q_rho neither underflows nor cancels.  The logits off the
// list are summed without those on it (never as a difference of sums).
//
//   k_td_stats  one workgroup per 8192 logits of a row: maximum and sum of exponentials off the list
//   k_td_loss   one workgroup per row: those and the list -> loss, log Z, the gradient's factors
//   k_td_grad   one workgroup per 8192 logits of a row: the gradient
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spec_device.h"
#include "spec_train.h"
#include "spec_train_device.h"

namespace specv {

constexpr int kTdPer = kTrSeg / kThreads;   // 32 logits per thread
constexpr int64_t kTdPast = 1 << 27;        // bytes
constexpr double kTdTailMin = 0x1p-20;      // mass off the list that counts: below it is the
                                            // rounding of an fp32 log Z

// Index within the segment of register j of this thread (tr_load's order).
template <int DT>
__device__ __forceinline__ int td_index(int j) {
  constexpr int kEl = TrEl<DT>::n;
  return kEl * ((int)threadIdx.x + kThreads * (j / kEl)) + j % kEl;
}
__device__ __forceinline__ uint32_t td_pack(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
template <int DT>
__device__ __forceinline__ void td_put(void* row, int i, float x) {
  if constexpr (DT == kDtBF16) ((__bf16*)row)[i] = (__bf16)x;
  else ((float*)row)[i] = x;
}
// The first n of a segment's logits to p, in tr_load's order.
template <int DT, bool PAST>
__device__ __forceinline__ void td_store(void* p, int n, const float (&v)[kTdPer]) {
  constexpr int kEl = TrEl<DT>::n;
#pragma unroll
  for (int q = 0; q < kTdPer / kEl; ++q) {
    const int e0 = td_index<DT>(q * kEl);
    if (e0 + kEl <= n) {
      uint4 x;
      if constexpr (DT == kDtBF16)
        x = make_uint4(td_pack(v[8 * q], v[8 * q + 1]), td_pack(v[8 * q + 2], v[8 * q + 3]),
                       td_pack(v[8 * q + 4], v[8 * q + 5]), td_pack(v[8 * q + 6], v[8 * q + 7]));
      else
        x = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                       __float_as_uint(v[4 * q + 3]));
      st16_any<PAST>((char*)p + (int64_t)e0 * (16 / kEl), x);
    } else {
#pragma unroll
      for (int e = 0; e < kEl; ++e)
        if (e0 + e < n) td_put<DT>(p, e0 + e, v[kEl * q + e]);
    }
  }
}

// Entry j of row r's list: its token, or -1 for one that does not count (a token outside the
// vocabulary, a logit of -inf).
__device__ __forceinline__ int td_token(const DistillArgs& a, int64_t r, int j, float& t) {
  if (j >= a.K) return -1;
  const int x = a.index[r * a.K + j];
  t = a.teacher[r * a.K + j];
  return x >= 0 && x < a.V && t != -INFINITY ? x : -1;
}

// Bound by the read: 2048 bf16 rows of 151,936 (622 MB) in 100 us, 6.2 TB/s; 448 rows in 26 us,
// 5.2 TB/s.  8192 logits are 16 or 32 KB, all of whose loads are in flight before the first is used;
// the list goes into a bit per logit in LDS meanwhile.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_td_stats(DistillArgs a) {
  __shared__ uint32_t listed[kTrSeg / 32];   // a bit per logit of the segment
  const int seg = blockIdx.x % a.n_seg, r = blockIdx.x / a.n_seg, base = seg * a.seg, t = threadIdx.x;
  constexpr int kEl = TrEl<DT>::n;
  float v[kTdPer];
  tr_load<DT>((const char*)row_ptr<DT>(a.logits, a.ld, r) + (int64_t)base * (16 / kEl), min(a.seg, a.V - base), v);
  listed[t] = 0;
  __syncthreads();
  float tl;
  const int x = td_token(a, r, t, tl) - base;
  if (x >= 0 && x < a.seg) atomicOr(&listed[x >> 5], 1u << (x & 31));
  __syncthreads();
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < kTdPer / kEl; ++q) {
    const int i = td_index<DT>(q * kEl);
    const uint32_t b = listed[i >> 5] >> (i & 31) & ((1u << kEl) - 1);
    if (b)
#pragma unroll
      for (int e = 0; e < kEl; ++e)
        if (b & (1u << e)) v[kEl * q + e] = -INFINITY;
#pragma unroll
    for (int e = 0; e < kEl; ++e) m = fmaxf(m, v[kEl * q + e]);
  }
  m = wave_max(m);
  const float s = wave_sum(tr_sum_exp(v, m, a.c));
  if ((t & 63) == 0) a.ms[((int64_t)r * a.n_seg + seg) * kWaves + (t >> 6)] = MaxSum{m, s};
}

// One workgroup per row.  Its time is a chain of latencies, so everything it reads goes out first and
// the reductions go in three rounds: 5.4 us for 7 rows, 6.2 us for
// 448, 18.7 us for 2048.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_td_loss(DistillArgs a) {
  __shared__ alignas(16) int lx[kTrMaxK];
  __shared__ double lp[kTrMaxK];
  __shared__ float rm[kWaves][3];
  __shared__ int any[kWaves], twice[kWaves];
  __shared__ double rs[kWaves][3], rt[kWaves];
  const int r = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const MaxSum* ms = a.ms + (int64_t)r * a.n_seg * kWaves;
  const int n_ms = a.n_seg * kWaves;
  MaxSum part = {-INFINITY, 0.f};
  if (t < n_ms) part = ms[t];
  const float lz_t = a.teacher_log_z ? a.teacher_log_z[r] : 0.f;
  const float weight = a.row_weight ? a.row_weight[r] : 1.f;
  float tl = -INFINITY;
  const int x = td_token(a, r, t, tl);
  lx[t] = x;
  const float l = x >= 0 ? logit_at<DT>(row_ptr<DT>(a.logits, a.ld, r), x) : -INFINITY;

  // maxima: off the list, on it, the teacher's
  float m_out = part.m, m_in = l, tm = x >= 0 ? tl : -INFINITY;
  for (int i = t + kThreads; i < n_ms; i += kThreads) m_out = fmaxf(m_out, ms[i].m);
  m_out = wave_max(m_out);
  m_in = wave_max(m_in);
  tm = wave_max(tm);
  const int any_w = __any(x >= 0) ? 1 : 0;
  if (lane == 0) {
    rm[wave][0] = m_out;
    rm[wave][1] = m_in;
    rm[wave][2] = tm;
    any[wave] = any_w;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    m_out = fmaxf(m_out, rm[w][0]);
    m_in = fmaxf(m_in, rm[w][1]);
    tm = fmaxf(tm, rm[w][2]);
  }
  const bool some = any[0] | any[1] | any[2] | any[3];
  const float m = fmaxf(m_out, m_in);
  bool first = x >= 0;   // the same token twice is one place of the row
  for (int j0 = 0; j0 < a.K; j0 += 8) {
    int e[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = lx[j0 + q];   // (-1 past the list)
#pragma unroll
    for (int q = 0; q < 8; ++q) first = first && !(e[q] == x && j0 + q < t);
  }

  // sums: off the list relative to m_out, on it relative to m, the teacher's masses
  const auto term_of = [&](const MaxSum& p) {
    return p.m > -INFINITY ? (double)p.s * exp2_split(((double)p.m - (double)m_out) * (double)a.c) : (double)p.s;
  };
  double z_out = t < n_ms ? term_of(part) : 0.0;
  for (int i = t + kThreads; i < n_ms; i += kThreads) z_out += term_of(ms[i]);
  const double e_l = x >= 0 ? exp2_split(((double)l - (double)m) * (double)a.c) : 0.0;
  const double at = x >= 0 ? (a.teacher_log_z ? (double)tl * a.inv_t - (double)lz_t : ((double)tl - (double)tm) * a.inv_t) : 0.0;
  double p = x >= 0 ? exp(at) : 0.0;
  double s_in = wave_sum_d(first ? e_l : 0.0), s_p = wave_sum_d(p);
  z_out = wave_sum_d(z_out);
  if (lane == 0) {
    rs[wave][0] = z_out;
    rs[wave][1] = s_in;
    rs[wave][2] = s_p;
  }
  const int twice_w = __any(x >= 0 && !first) ? 1 : 0;
  __syncthreads();
  z_out = (rs[0][0] + rs[1][0]) + (rs[2][0] + rs[3][0]);
  s_in = (rs[0][1] + rs[1][1]) + (rs[2][1] + rs[3][1]);
  s_p = (rs[0][2] + rs[1][2]) + (rs[2][2] + rs[3][2]);
  const double f_out = m_out > -INFINITY ? exp2_split(((double)m_out - (double)m) * (double)a.c) : 0.0;
  double z = s_in + (m_out > -INFINITY ? z_out * f_out : z_out);
  if (!(m > -INFINITY)) z = __longlong_as_double(0x7ff8000000000000ll);   // no finite logit
  const double lz = (double)m * a.inv_t + log(z);
  double ln_p = at, sum_p = s_p, rho = 0.0;
  if (a.teacher_log_z) {
    rho = 1.0 - s_p;
    if (rho <= kTdTailMin) rho = 0.0;
  } else if (some) {   // the list is the teacher
    ln_p = at - log(s_p);
    p /= s_p;
    sum_p = s_p == s_p ? 1.0 : s_p;
  }
  lp[t] = p;
  double term = p > 0.0 ? p * (ln_p - ((double)l * a.inv_t - lz)) : p;   // p is 0, or NaN
  term = wave_sum_d(term);
  if (lane == 0) {
    rt[wave] = term;
    twice[wave] = twice_w;
  }
  __syncthreads();
  double loss = (rt[0] + rt[1]) + (rt[2] + rt[3]);
  if (rho > 0.0) loss += rho * (log(rho) - (z_out > 0.0 ? (double)m_out * a.inv_t + log(z_out) - lz : -INFINITY));
  if (z != z) loss = z;
  if (t == 0) {
    a.loss[r] = some ? (float)loss : 0.f;
    if (a.log_z) a.log_z[r] = (float)lz;
  }
  if (!a.d_logits) return;
  const double scale = (double)weight * a.inv_t, mass = sum_p + rho;
  if (t == 0) {
    DistillRow o;
    o.m = m_out > -INFINITY ? m_out : 0.f;   // nothing off the list: its -inf logits give 0, not NaN
    o.f = (float)(scale * (mass * f_out / z - (rho > 0.0 && z_out > 0.0 ? rho / z_out : 0.0)));
    o.zero = !some || scale == 0.0 ? 1 : 0;
    o.pad = 0;
    a.rows[r] = o;
  }
  if (x >= 0) {
    double ps = p;
    if (twice[0] | twice[1] | twice[2] | twice[3]) {   // a token stands in the list twice
      ps = 0.0;
      for (int j = 0; j < a.K; ++j) ps += lx[j] == x ? lp[j] : 0.0;
    }
    a.d_list[(int64_t)r * a.K + t] = (float)(scale * (mass * e_l / z - ps));
  }
}

// Bound by memory: 2048 bf16 rows of 151,936 are read and written (1.24 GB) in 189 to 193 us, 6.5
// TB/s; a copy of that size reaches 5.2 to 5.6.  Reading a row a second time is the price of log Z:
// one workgroup that keeps to one row and finds it in the caches was no faster (351 us, when the three
// kernels took 350), nor were groups of rows (128 to 1024: 510 to 348 us), or the rows in reverse with
// the first read kept (367 us, when they took 347).
template <int DT, bool PAST>
__global__ __launch_bounds__(kThreads) void k_td_grad(DistillArgs a) {
  const int seg = blockIdx.x % a.n_seg, r = blockIdx.x / a.n_seg, base = seg * a.seg, n = min(a.seg, a.V - base);
  constexpr int kSz = 16 / TrEl<DT>::n;   // bytes of a logit
  void* out = (char*)const_cast<void*>(row_ptr<DT>(a.d_logits, a.d_ld, r)) + (int64_t)base * kSz;
  const DistillRow row = a.rows[r];
  float v[kTdPer];
  if (row.zero) {
#pragma unroll
    for (int j = 0; j < kTdPer; ++j) v[j] = 0.f;
    td_store<DT, PAST>(out, n, v);
    return;
  }
  tr_load<DT>((const char*)row_ptr<DT>(a.logits, a.ld, r) + (int64_t)base * kSz, n, v);
#pragma unroll
  for (int j = 0; j < kTdPer; ++j) v[j] = __builtin_amdgcn_exp2f((v[j] - row.m) * a.c) * row.f;
  td_store<DT, PAST>(out, n, v);
  wait_vmem();       // the list's tokens are written over what this stored
  __syncthreads();
  float tl;
  const int x = td_token(a, r, threadIdx.x, tl) - base;
  if (x >= 0 && x < a.seg) td_put<DT>(out, x, a.d_list[(int64_t)r * a.K + threadIdx.x]);
}

namespace {
template <int DT>
void topk_distill(const DistillArgs& a, hipStream_t st) {
  const dim3 segs((unsigned)(a.R * a.n_seg)), block(kThreads);
  hipLaunchKernelGGL((k_td_stats<DT>), segs, block, 0, st, a);
  hipLaunchKernelGGL((k_td_loss<DT>), dim3((unsigned)a.R), block, 0, st, a);
  if (!a.d_logits) return;
  // A gradient that is a good part of the memory-side cache (256 MB) or more goes past it: 2048 rows of
  // 151,936 in bf16 312 us (343 by way of it), 512 rows (156 MB) 88 (92), 2048 rows of 32,000 (131 MB)
  // 85 (90).  A smaller one stays where its reader finds it: 256 rows of 151,936 (78 MB) 50 us (51 past
  // it), 512 fp32 rows of 32,000 (66 MB) 43 (45).
  if (a.R * (int64_t)a.V * (16 / TrEl<DT>::n) > kTdPast) hipLaunchKernelGGL((k_td_grad<DT, true>), segs, block, 0, st, a);
  else hipLaunchKernelGGL((k_td_grad<DT, false>), segs, block, 0, st, a);
}
}  // namespace

hipError_t launch_topk_distill(const DistillArgs& a, int dt, hipStream_t st) {
  dt == kDtBF16 ? topk_distill<kDtBF16>(a, st) : topk_distill<kDtF32>(a, st);
  return hipGetLastError();
}

}  // namespace specv
