// k_latent_project.cuh -- per-head products between head space and latent space.
#pragma once
#include "common.cuh"

namespace s4r {

struct LatentProject {
  int64_t n_tokens;
  int32_t n_heads, head_dim, rank, to_latent;
  const bf16 *x, *basis;
  bf16 *out;
  int64_t x_ts, x_hs, out_ts, out_hs;
};

// One thread an output value.
__global__ void __launch_bounds__(256) latent_project_simt(const LatentProject p) {
  const int32_t nk = p.to_latent ? p.head_dim : p.rank, no = p.to_latent ? p.rank : p.head_dim;
  const int64_t n = p.n_tokens * p.n_heads * no;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int32_t j = (int32_t)(i % no), h = (int32_t)(i / no % p.n_heads);
    const int64_t t = i / no / p.n_heads;
    const bf16 *x = p.x + t * p.x_ts + h * p.x_hs;
    const bf16 *b = p.basis + (int64_t)h * p.head_dim * p.rank + (p.to_latent ? j : (int64_t)j * p.rank);
    const int32_t step = p.to_latent ? p.rank : 1;
    float a = 0.0f;
    for (int32_t k = 0; k < nk; ++k) a = fmaf(to_f(x[k]), to_f(b[(int64_t)k * step]), a);
    p.out[t * p.out_ts + h * p.out_hs + j] = from_f<bf16>(a);
  }
}

}  // namespace s4r
