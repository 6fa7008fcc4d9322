// k_prefill.cuh -- causal attention of ragged prompts over expanded keys and values.
#pragma once
#include <math_constants.h>

#include "umma.cuh"

namespace s4r {

struct PrefillAttend {
  int32_t batch, hq, hkv, dim, rope, vdim, causal, max_q;
  int64_t total_q, total_k;
  float scale;
  const bf16 *q, *k, *v, *k_rope;
  int64_t k_ts, v_ts, k_rope_ts;
  const int32_t *cu_q, *cu_k;
  bf16 *out;
  float *lse;
};

// Rows of sequence b (false, and the library-wide status set, if its offsets
// are not within the tensors).
struct PrefillSeq {
  int64_t q0, k0;
  int32_t nq, nk;
};
__device__ __forceinline__ bool prefill_seq(const PrefillAttend &p, int b, PrefillSeq &s) {
  const int32_t q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
  s.q0 = q0;
  s.k0 = k0;
  s.nq = q1 - q0;
  s.nk = k1 - k0;
  return q0 >= 0 && q1 >= q0 && q1 <= p.total_q && k0 >= 0 && k1 >= k0 && k1 <= p.total_k;
}

// One warp a (query, head): keys one after another with a running maximum and sum.
__global__ void __launch_bounds__(256) prefill_attend_simt(const PrefillAttend p) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
  const int32_t i = (int32_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  PrefillSeq s;
  if (!prefill_seq(p, b, s)) {
    set_status(&g_device_status, kDevStatusCheck);
    return;
  }
  if (s.nq > p.max_q) set_status(&g_device_status, kDevStatusCheck);
  if (i >= smin(s.nq, p.max_q)) return;
  const int32_t g = h / (p.hq / p.hkv);
  const bf16 *q = p.q + ((s.q0 + i) * p.hq + h) * (int64_t)(p.dim + p.rope);
  float qv[4], qr[2], acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qv[j] = lane + 32 * j < p.dim ? to_f(q[lane + 32 * j]) : 0.0f;
    acc[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) qr[j] = lane + 32 * j < p.rope ? to_f(q[p.dim + lane + 32 * j]) : 0.0f;
  const int64_t sees = p.causal ? (int64_t)s.nk - s.nq + i + 1 : s.nk;
  float m = -CUDART_INF_F, l = 0.0f;
  for (int64_t j = 0; j < sees; ++j) {
    const int64_t row = s.k0 + j;
    float z = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < p.dim) z = fmaf(qv[c], to_f(p.k[row * p.k_ts + (int64_t)g * p.dim + lane + 32 * c]), z);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (lane + 32 * c < p.rope) z = fmaf(qr[c], to_f(p.k_rope[row * p.k_rope_ts + lane + 32 * c]), z);
    z = warp_sum(z) * p.scale;
    const float top = fmaxf(m, z);
    const float f = m == -CUDART_INF_F ? 0.0f : expf(m - top);
    const float e = expf(z - top);
    l = l * f + e;
    m = top;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < p.vdim) acc[c] = acc[c] * f + e * to_f(p.v[row * p.v_ts + (int64_t)g * p.vdim + lane + 32 * c]);
  }
  bf16 *o = p.out + ((s.q0 + i) * p.hq + h) * (int64_t)p.vdim;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.vdim) o[lane + 32 * c] = from_f<bf16>(sees > 0 ? acc[c] / l : 0.0f);
  if (lane == 0 && p.lse) p.lse[(s.q0 + i) * p.hq + h] = sees > 0 ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace s4r
