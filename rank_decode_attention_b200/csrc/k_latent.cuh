// k_latent.cuh -- attention over the rows of a paged latent cache.
#pragma once
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "common.cuh"
#include "k_page.cuh"

namespace s4r {

struct LatentAttend {
  int32_t batch, n_query, n_heads, width, rank, page_size, page_shift, max_pages;
  int64_t n_pages;
  float scale, cache_scale;
  const bf16 *q;
  const unsigned char *cache;
  const int32_t *block_table, *lengths;
  bf16 *out;
  float *lse;
  uint32_t *status;
};

constexpr int kLaCols = (S4R_MAX_LATENT_WIDTH + 31) / 32;

// Column `col` of a cached row.
template <bool FP4>
__device__ __forceinline__ float latent_value(const LatentAttend &p, int64_t page, int32_t row, int32_t col) {
  const unsigned char *base = p.cache + page * latent_page_bytes(FP4, p.page_size, p.width);
  if constexpr (!FP4) {
    return to_f(reinterpret_cast<const bf16 *>(base)[(int64_t)row * p.width + col]);
  } else {
    const unsigned char c = base[(int64_t)row * (p.width / 2) + col / 2];
    const unsigned char s = base[(int64_t)p.page_size * (p.width / 2) + (int64_t)row * (p.width / 16) + col / 16];
    const float v = __half2float(__half(__nv_cvt_fp4_to_halfraw((__nv_fp4_storage_t)((col & 1) ? c >> 4 : c & 15), __NV_E2M1)));
    return v * __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3))) * p.cache_scale;
  }
}

// One warp a (request, query token, head): rows one after another with a
// running maximum and sum.
template <bool FP4>
__global__ void __launch_bounds__(256) latent_attend_simt(const LatentAttend p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)p.batch * p.n_query * p.n_heads) return;
  const int32_t t = (int32_t)(w / p.n_heads % p.n_query), b = (int32_t)(w / p.n_heads / p.n_query);
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  int64_t len = p.lengths[b];
  if (len < 0 || len > cap) {
    set_status(p.status, kDevStatusCheck);
    len = len < 0 ? 0 : cap;
  }
  const int64_t sees = len - p.n_query + 1 + t;
  float q[kLaCols], acc[kLaCols];
#pragma unroll
  for (int i = 0; i < kLaCols; ++i) {
    const int col = lane + 32 * i;
    q[i] = col < p.width ? to_f(p.q[w * p.width + col]) : 0.0f;
    acc[i] = 0.0f;
  }
  float m = -CUDART_INF_F, l = 0.0f;
  for (int64_t i = 0; i < sees; ++i) {
    const int32_t page = p.block_table[(int64_t)b * p.max_pages + (i >> p.page_shift)];
    const bool ok = page >= 0 && page < p.n_pages;
    if (!ok) set_status(p.status, kDevStatusCheck);
    float x[kLaCols], z = 0.0f;
#pragma unroll
    for (int j = 0; j < kLaCols; ++j) {
      const int col = lane + 32 * j;
      x[j] = ok && col < p.width ? latent_value<FP4>(p, page, (int32_t)(i & (p.page_size - 1)), col) : 0.0f;
      z = fmaf(q[j], x[j], z);
    }
    z = warp_sum(z) * p.scale;
    const float top = fmaxf(m, z);
    const float f = m == -CUDART_INF_F ? 0.0f : expf(m - top);
    const float e = expf(z - top);
    l = l * f + e;
    m = top;
#pragma unroll
    for (int j = 0; j < kLaCols; ++j) acc[j] = acc[j] * f + e * x[j];
  }
#pragma unroll
  for (int i = 0; i < kLaCols; ++i) {
    const int col = lane + 32 * i;
    if (col < p.rank) p.out[w * p.rank + col] = from_f<bf16>(sees > 0 ? acc[i] / l : 0.0f);
  }
  if (lane == 0 && p.lse) p.lse[w] = sees > 0 ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace s4r
