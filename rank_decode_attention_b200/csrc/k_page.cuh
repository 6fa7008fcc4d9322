// k_page.cuh -- the paged latent cache: block tables and slot maps of a step
// (page_plan_kernel, page_commit_kernel) and the rows' way into the pages
// (latent_write_bf16, latent_write_fp4).
#pragma once
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "common.cuh"

namespace s4r {

// ------------------------------------------------------------------ page plan
//
// The plan needs two prefix sums over the requests (new tokens, new pages);
// everything else follows from them per token and per page.  Each CTA takes
// both sums of the whole batch by itself (at most S4R_MAX_REQUESTS requests,
// a few microseconds out of L2), keeps them in shared memory and then serves
// its share of the tokens and of the new pages, each found by binary search.
// So no CTA waits for another one, and one request with all the tokens is
// spread as well as many with one.  Latency is most of it: 5.6 us on the device
// for 256 requests with a token each (one CTA), 10.8 us for 1001 requests with 600
// thousand tokens (a CTA on each of 148 multiprocessors and the commit kernel;
// the 10 MB written would take 1.5 us).
struct PagePlan {
  int32_t batch, page_size, page_shift, max_pages, free_capacity;
  int64_t max_tokens;
  const int32_t *lengths, *new_tokens, *free_pages, *free_count;
  int32_t *block_table, *lengths_out, *free_count_out, *cu_tokens;
  int64_t *slots;
  int32_t *positions, *requests;
  uint32_t *status;
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanPerThread = S4R_MAX_REQUESTS / kPlanThreads;
// A token a thread: more CTAs cost less than a longer loop, the commit kernel
// included (1100 tokens 6.2 us against 6.8 with 4096 tokens a CTA, 6400 tokens 5.8
// against 8.4, 32000 tokens 5.9 against 7.6).
constexpr int kPlanTokensPerCta = kPlanThreads;
inline size_t plan_smem_bytes(int batch) { return 2 * sizeof(int32_t) * (size_t)(batch + 1); }

// Whether a request's counts are legal and its rows fit its table row.
__host__ __device__ inline bool plan_fits(int32_t old, int32_t add, int32_t max_pages, int32_t page_size) {
  return old >= 0 && add >= 0 && (int64_t)old + add <= (int64_t)max_pages * page_size;
}
// Pages a request needs beyond those it has.
__host__ __device__ inline int32_t plan_need(int32_t old, int32_t add, int32_t max_pages, int page_shift) {
  const int32_t ps = 1 << page_shift;
  if (!plan_fits(old, add, max_pages, ps)) return 0;
  return (int32_t)((((int64_t)old + add + ps - 1) >> page_shift) - (((int64_t)old + ps - 1) >> page_shift));
}
// Whether a request is served, by its counts, the running demand up to it and the
// free pages.  The need is worked out where the demand does not fit (per token it
// took 0.3 us of 600 thousand tokens' 10.9): the demand says nothing about it,
// since neighbours are equal where it is held at its largest value.
__host__ __device__ inline bool plan_served(int32_t old, int32_t add, int32_t max_pages, int page_shift, uint32_t demand,
                                            int32_t free_pages) {
  return plan_fits(old, add, max_pages, 1 << page_shift) &&
         (demand <= (uint32_t)free_pages || plan_need(old, add, max_pages, page_shift) == 0);
}
// What a sum is held at: tokens fit their 32-bit offsets; pages stay above any
// count of free ones.
__host__ __device__ inline int32_t plan_hold_tokens(long long x) { return (int32_t)smin<long long>(x, INT32_MAX); }
__host__ __device__ inline uint32_t plan_hold_pages(long long x) { return (uint32_t)smin<long long>(x, UINT32_MAX); }
// Largest i in [0, n] with a[i] <= x, for ascending a and a[0] <= x: the last
// of several equal entries, so that empty requests own nothing.
template <typename T> __host__ __device__ inline int plan_find(const T *a, int n, T x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Exclusive prefix sums of tokens and pages over the batch, batch + 1 entries
// each, 64-bit inside.
__device__ inline void plan_scan(const PagePlan &p, int32_t *s_tok, uint32_t *s_pg) {
  __shared__ long long w_tok[32], w_pg[32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;   // <= kPlanPerThread
  const int b0 = t * per;
  int32_t tok[kPlanPerThread], pg[kPlanPerThread];
  long long st = 0, sp = 0;
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    tok[i] = pg[i] = 0;
    if (i < per && b0 + i < p.batch) {
      const int32_t old = p.lengths[b0 + i], add = p.new_tokens[b0 + i];
      tok[i] = add > 0 ? add : 0;
      pg[i] = plan_need(old, add, p.max_pages, p.page_shift);
    }
    st += tok[i];
    sp += pg[i];
  }
  long long it = st, ip = sp;   // inclusive over the warp, then over the block
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      it += a;
      ip += b;
    }
  }
  if (lane == 31) {
    w_tok[warp] = it;
    w_pg[warp] = ip;
  }
  __syncthreads();
  if (warp == 0) {
    long long a = w_tok[lane], b = w_pg[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += x;
        b += y;
      }
    }
    w_tok[lane] = a;
    w_pg[lane] = b;
  }
  __syncthreads();
  long long et = it - st + (warp ? w_tok[warp - 1] : 0), ep = ip - sp + (warp ? w_pg[warp - 1] : 0);
  if (t == 0) {
    s_tok[0] = 0;
    s_pg[0] = 0u;
  }
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    if (i < per && b0 + i < p.batch) {
      et += tok[i];
      ep += pg[i];
      s_tok[b0 + i + 1] = plan_hold_tokens(et);
      s_pg[b0 + i + 1] = plan_hold_pages(ep);
    }
  }
  __syncthreads();
}

// Pages the free list holds (clamped to its capacity).
__device__ __forceinline__ int32_t plan_free(const PagePlan &p, bool report) {
  const int32_t f = *p.free_count;
  const int32_t c = smin(smax(f, 0), p.free_capacity);
  if (report && c != f) set_status(p.status, kDevStatusCheck);
  return c;
}

// The per-request results: lengths_out, free_count_out.  They may overwrite
// the inputs, so every read of those is behind the caller's barrier.
__device__ inline void plan_commit(const PagePlan &p, const uint32_t *s_pg, int32_t free_pages, int32_t taken) {
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = threadIdx.x * per;
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    const int b = b0 + i;
    if (i < per && b < p.batch) {
      const int32_t old = p.lengths[b], add = p.new_tokens[b];
      const bool served = plan_served(old, add, p.max_pages, p.page_shift, s_pg[b + 1], free_pages);
      if (!served) set_status(p.status, kDevStatusCheck);
      p.lengths_out[b] = served ? old + add : old;
    }
  }
  if (threadIdx.x == 0) *p.free_count_out = free_pages - taken;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlan p) {
  extern __shared__ int32_t plan_smem[];
  int32_t *s_tok = plan_smem;
  uint32_t *s_pg = reinterpret_cast<uint32_t *>(plan_smem + p.batch + 1);
  if (gridDim.x > 1) pdl_trigger();   // the commit kernel may take its sums; it waits for this grid before it writes
  plan_scan(p, s_tok, s_pg);
  const int32_t total = s_tok[p.batch];
  const int32_t free_pages = plan_free(p, blockIdx.x == 0);
  // Requests are served as long as the running demand fits, so what they take
  // is the largest running demand that does.
  const int32_t taken = (int32_t)s_pg[plan_find(s_pg, p.batch, (uint32_t)free_pages)];
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= p.batch; i += kPlanThreads) p.cu_tokens[i] = s_tok[i];
    if (threadIdx.x == 0 && total > p.max_tokens) set_status(p.status, kDevStatusCheck);
  }
  const int64_t step = (int64_t)gridDim.x * kPlanThreads, first = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  // New table entries.  They are never read here: the tokens below take the
  // ids of new pages from the free list.
  for (int64_t j = first; j < taken; j += step) {
    const int b = plan_find(s_pg, p.batch, (uint32_t)j);
    const int32_t have = (int32_t)(((int64_t)p.lengths[b] + p.page_size - 1) >> p.page_shift);
    p.block_table[(int64_t)b * p.max_pages + have + (j - s_pg[b])] = p.free_pages[free_pages - 1 - j];
  }
  for (int64_t t = first; t < p.max_tokens; t += step) {
    int64_t slot = -1;
    int32_t pos = -1, req = -1;
    if (t < total) {
      req = plan_find(s_tok, p.batch, (int32_t)t);
      const int32_t old = p.lengths[req], add = p.new_tokens[req];
      pos = (int32_t)(old + (t - s_tok[req]));
      const uint32_t d0 = s_pg[req], d1 = s_pg[req + 1];
      if (plan_served(old, add, p.max_pages, p.page_shift, d1, free_pages)) {
        const int32_t have = (int32_t)(((int64_t)old + p.page_size - 1) >> p.page_shift), at = pos >> p.page_shift;
        const int32_t page = at < have ? p.block_table[(int64_t)req * p.max_pages + at]
                                       : p.free_pages[free_pages - 1 - ((int32_t)d0 + at - have)];
        slot = (int64_t)page * p.page_size + (pos & (p.page_size - 1));
      }
    }
    p.slots[t] = slot;
    if (p.positions) p.positions[t] = pos;
    if (p.requests) p.requests[t] = req;
  }
  if (gridDim.x == 1) {
    __syncthreads();
    plan_commit(p, s_pg, free_pages, taken);
  }
}

// With several CTAs the per-request results, which may overwrite the inputs,
// wait for all of them in a launch of their own.
__global__ void __launch_bounds__(kPlanThreads) page_commit_kernel(const PagePlan p) {
  extern __shared__ int32_t plan_smem[];
  int32_t *s_tok = plan_smem;
  uint32_t *s_pg = reinterpret_cast<uint32_t *>(plan_smem + p.batch + 1);
  plan_scan(p, s_tok, s_pg);
  const int32_t free_pages = plan_free(p, false);
  const int32_t taken = (int32_t)s_pg[plan_find(s_pg, p.batch, (uint32_t)free_pages)];
  __syncthreads();
  pdl_wait();
  plan_commit(p, s_pg, free_pages, taken);
}

// --------------------------------------------------------------- latent write

struct LatentWrite {
  int64_t n_tokens, n_rows, latents_ld;
  int32_t width, page_size, page_shift;
  float cache_scale;
  const bf16 *latents;
  const int64_t *slots;
  unsigned char *cache;
  bf16 *stored;
  uint32_t *status;
};

// Bytes of a page.
__host__ __device__ inline int64_t latent_page_bytes(bool fp4, int32_t page_size, int32_t width) {
  return fp4 ? (int64_t)page_size * width * 9 / 16 : (int64_t)page_size * width * 2;
}

// A CTA takes kWriteTokens rows; within them every thread a piece at a time,
// found with a 32-bit division.
constexpr int kWriteTokens = 8, kWriteThreads = 256;

// One thread a 16-byte piece of a row.
__global__ void __launch_bounds__(kWriteThreads) latent_write_bf16(const LatentWrite p) {
  const uint32_t per = (uint32_t)p.width / 8;
  const int64_t t0 = (int64_t)blockIdx.x * kWriteTokens;
  const uint32_t n = (uint32_t)smin<int64_t>(kWriteTokens, p.n_tokens - t0) * per;
  for (uint32_t i = threadIdx.x; i < n; i += kWriteThreads) {
    const uint32_t r = i / per, c = i - r * per;
    const int64_t t = t0 + r, slot = p.slots[t];
    if (slot < 0) continue;
    if (slot >= p.n_rows) {
      if (c == 0) set_status(p.status, kDevStatusCheck);
      continue;
    }
    const uint4 v = *reinterpret_cast<const uint4 *>(p.latents + t * p.latents_ld + c * 8);
    *reinterpret_cast<uint4 *>(p.cache + (slot * p.width + c * 8) * 2) = v;
  }
}

// One thread a group of 16 columns: 32 bytes in, 8 bytes of codes and one
// scale byte out.  The codes follow from the definition bit by bit.  ONE
// (cache_scale 1): the quotients need no division.  x has 8 significant bits
// and the scale 4, so x / scale is either exactly a border between two codes
// (at most 3 bits) or a part in 2^15 away from every border; the product with
// the rounded reciprocal is within 2^-22 of it, and rounded to 20 bits it is on
// the border, or on the same side of it, as the quotient is.  (32765 rows of 576
// columns, the same ones each time: 21.4 us with divisions, 16 x 9 instructions a
// group, now 17.7 us; with inputs changing 22.5 us, 3.8 TB/s.)
template <bool ONE>
__global__ void __launch_bounds__(kWriteThreads) latent_write_fp4(const LatentWrite p) {
  const uint32_t per = (uint32_t)p.width / 16;
  const int64_t t0 = (int64_t)blockIdx.x * kWriteTokens;
  const uint32_t n = (uint32_t)smin<int64_t>(kWriteTokens, p.n_tokens - t0) * per;
  const int64_t page_bytes = latent_page_bytes(true, p.page_size, p.width);
  for (uint32_t i = threadIdx.x; i < n; i += kWriteThreads) {
    const uint32_t r = i / per, g = i - r * per;
    const int64_t t = t0 + r, slot = p.slots[t];
    const bool bad = slot >= p.n_rows;
    if (bad && g == 0) set_status(p.status, kDevStatusCheck);
    if ((slot < 0 || bad) && !p.stored) continue;
    float x[16];
    load16(p.latents + t * p.latents_ld + g * 16, x);
    load16(p.latents + t * p.latents_ld + g * 16 + 8, x + 8);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (!ONE) x[j] = __fdiv_rn(x[j], p.cache_scale);
      top = fmaxf(top, fabsf(x[j]));
    }
    const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(fminf(__fdiv_rn(top, 6.0f), 448.0f), __NV_SATFINITE, __NV_E4M3);
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
    uint32_t code[2] = {0u, 0u};
    if (s > 0.0f) {
      const float inv = __frcp_rn(s);
      auto quotient = [&](float v) {
        if (!ONE) return __fdiv_rn(v, s);
        const float q = v * inv;
        // infinities and NaN have no bits to round
        return fabsf(q) < CUDART_INF_F ? __uint_as_float((__float_as_uint(q) + 8u) & ~15u) : q;
      };
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_fp4x2_storage_t c =
            __nv_cvt_float2_to_fp4x2(make_float2(quotient(x[2 * j]), quotient(x[2 * j + 1])), __NV_E2M1, cudaRoundNearest);
        code[j >> 2] |= (uint32_t)c << (8 * (j & 3));
      }
    }
    if (slot >= 0 && !bad) {
      const int64_t page = slot >> p.page_shift;
      const int32_t row = (int32_t)(slot & (p.page_size - 1));
      unsigned char *base = p.cache + page * page_bytes;
      *reinterpret_cast<uint2 *>(base + (int64_t)row * (p.width / 2) + g * 8) = make_uint2(code[0], code[1]);
      base[(int64_t)p.page_size * (p.width / 2) + (int64_t)row * per + g] = s8;
    }
    if (p.stored) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(code[j >> 2] >> (8 * (j & 3))), __NV_E2M1));
        const float2 f = __half22float2(h);
        const float m = ONE ? 1.0f : p.cache_scale;
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s * m, f.y * s * m);
        w[j] = (uint32_t)__bfloat16_as_ushort(b.x) | ((uint32_t)__bfloat16_as_ushort(b.y) << 16);
      }
      uint4 *dst = reinterpret_cast<uint4 *>(p.stored + t * p.width + g * 16);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace s4r
