// k_latent.cuh -- attention over the rows of a paged latent cache, absorbed
// form: z_i = scale q . row_i, out = sum_i softmax(z)_i row_i[0 .. rank-1] for
// every query row (query token, head) of a request.
//
// One row of the cache serves every head, so a tile of cached rows is read
// once and used for up to 64 query rows.  At 64 query rows of width 576 a
// token costs 1152 bytes and 139 kFLOP: both HBM and the tensor cores are
// within a factor of two of their limits, and few query rows leave the kernel
// to HBM alone.
//
// latent_attend_kernel: a persistent grid, one CTA per SM.  The work is the
// stream of 64-token tiles of all (request, block of NB query rows) units, cut
// into equal consecutive ranges, so ragged batches and single long requests
// load every SM alike; a unit that crosses a border leaves partial sums, which
// latent_combine_kernel joins (no CTA waits for another one).
//
// Both products are computed transposed, tokens on M: S^T = K Q^T (M = 64
// tokens, N = NB) and O^T = V^T P^T (M = 128 latent columns, N = NB).  So few
// heads shrink N instead of wasting rows of M, and K and V are the same bytes
// in shared memory: K-major for the first product, M-major for the second.
// O^T stays in TMEM for a whole unit (4 blocks of 128 columns x NB).
//
// Roles:
//   warp 0     one thread copies tiles with TMA: 128 columns x 64 tokens a
//              ring slot, one box a page and 64 columns; and the unit's
//              queries;
//   warp 1     one thread issues tcgen05.mma: S^T of tile i + 1, as far as the
//              ring holds it, before O^T of tile i, so the softmax of one tile
//              runs beside the products of another; slots are released column
//              block by column block;
//   warps 2-5  softmax: probabilities against a reference maximum that moves
//              only when a logit exceeds it by more than 2^8 (then O^T is
//              rescaled in TMEM), sums in fp32, P^T into shared memory; at the
//              end of a unit they write the result or the partial sums.
//   warps 6-13 (4-bit cache) turn codes into fp16 ring slots: e2m1 * e4m3 has
//              6 significant bits, so fp16 holds the stored values exactly.
//              Queries become fp16 too, scaled by a power of two per row, exact
//              over 29 binades below the row's largest value.
// Probabilities are rounded to bf16 (4-bit cache: fp16) for the second
// product; the sum that divides it is not.
//
// Every wait is bounded (umma.cuh); a wait that gives up sets the status word
// and ends its role, and every other role then runs out too.
#pragma once
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "k_page.cuh"
#include "umma.cuh"

namespace s4r {

constexpr int kLaTile = 64;                  // tokens a tile
constexpr int kLaSlot = kLaTile * 128 * 2;   // bytes of a ring slot: 64 tokens x 128 columns
constexpr int kLaMaxSlots = 12;
constexpr int kLaMaxPairs = (S4R_MAX_LATENT_WIDTH + 127) / 128;
constexpr int kLaSmemBudget = 227 * 1024;
constexpr int kLaDequantWarps = 8;
constexpr int kLaRawStages = 2;
constexpr float kLaLift = 8.0f;              // how far (in powers of two) a logit may exceed the reference

struct LatentAttend {
  int32_t batch, n_query, n_heads, width, rank, page_size, page_shift, max_pages;
  int64_t n_pages;
  float scale, cache_scale;
  const bf16 *q;
  const unsigned char *cache;
  const int32_t *block_table, *lengths;
  bf16 *out;
  float *lse;
  // plan
  int32_t rows, row_blocks, n_ctas, slots;   // query rows a request, blocks of NB of them, grid, ring slots
  // workspace
  uint32_t *status;
  int32_t *flags;                            // [batch * row_blocks] recompute the unit (see latent_combine_kernel)
  float2 *ml;                                // [2 * n_ctas][NB] reference maximum and sum of a partial
  float *part;                               // [2 * n_ctas][NB][rank] unscaled partial results
};

// Query rows a block of the kernel takes, and how many blocks a request has.
__host__ __device__ inline int la_block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct LaLayout {
  int q, p, raw, ring, control, total, slots;
};
constexpr int kLaControlBytes = 4096;
__host__ __device__ inline int la_raw_bytes(int width) { return (kLaTile * width * 9 / 16 + 127) / 128 * 128; }
__host__ __device__ inline LaLayout la_layout(int nb, int width, bool fp4) {
  LaLayout l;
  const int chunks = (width + 63) / 64;
  int off = 0;
  l.q = off;
  off += chunks * nb * 128;
  off = (off + 1023) & ~1023;
  l.p = off;
  off += 2 * kLaTile * 128;
  l.ring = off;
  const int tail = (fp4 ? kLaRawStages * la_raw_bytes(width) : 0) + kLaControlBytes + 1024;
  l.slots = smin((kLaSmemBudget - off - tail) / kLaSlot, kLaMaxSlots);
  off += l.slots * kLaSlot;
  l.raw = off;
  off += fp4 ? kLaRawStages * la_raw_bytes(width) : 0;
  l.control = off;
  off += kLaControlBytes;
  l.total = off + 1024;   // aligning the start
  return l;
}

struct LaControl {
  uint64_t full[kLaMaxSlots], empty[kLaMaxSlots];
  uint64_t raw_full[kLaRawStages], raw_empty[kLaRawStages];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, q_empty, o_free;
  uint32_t tmem_base;
  int fail;   // a wait of the softmax warps gave up
  int first_b, first_off, n_tiles;   // start of this CTA's range and its length
  int qexp[2][64];                   // 4-bit cache: queries are scaled by 2^qexp (segments alternate)
  alignas(8) float wmax[4][64];
  float fac[64];
};
static_assert(sizeof(LaControl) <= kLaControlBytes, "control block");

// Length of a request within what its table row can name.
__device__ __forceinline__ int32_t la_length(const LatentAttend &p, int b) {
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  const int32_t n = p.lengths[b];
  return n < 0 ? 0 : (int32_t)smin<int64_t>(n, cap);
}
__device__ __forceinline__ int32_t la_tiles(int32_t len) { return (len + kLaTile - 1) / kLaTile; }

// Tiles of all units of the batch, those of requests before `upto` (both
// block-wide results in every thread).  scratch: blockDim.x / 32 pairs.
__device__ inline void la_count(const LatentAttend &p, int upto, long long *scratch, long long &total, long long &before) {
  long long t = 0, f = 0;
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const long long n = (long long)la_tiles(la_length(p, b)) * p.row_blocks;
    t += n;
    if (b < upto) f += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t += __shfl_xor_sync(0xffffffffu, t, o);
    f += __shfl_xor_sync(0xffffffffu, f, o);
  }
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    scratch[2 * warp] = t;
    scratch[2 * warp + 1] = f;
  }
  __syncthreads();
  total = before = 0;
  for (int w = 0; w < nw; ++w) {
    total += scratch[2 * w];
    before += scratch[2 * w + 1];
  }
  __syncthreads();
}
// Tiles a CTA takes of `total`.
__host__ __device__ inline long long la_share(long long total, int n_ctas) { return (total + n_ctas - 1) / n_ctas; }

// The segments of a CTA: consecutive tiles of one unit.
struct LaSegment {
  int b, rb, tile, n, unit_tiles, len, index;
};
struct LaWalk {
  int b, off, left, index;
  __device__ __forceinline__ LaWalk(const LaControl *c) : b(c->first_b), off(c->first_off), left(c->n_tiles), index(-1) {}
  __device__ __forceinline__ bool next(const LatentAttend &p, LaSegment &s) {
    if (left <= 0) return false;
    int len, nt;
    while (true) {   // requests without rows have no tiles
      len = la_length(p, b);
      nt = la_tiles(len);
      if (off < nt * p.row_blocks) break;
      off = 0;
      ++b;
    }
    s.b = b;
    s.rb = off / nt;
    s.tile = off - s.rb * nt;
    s.n = smin(nt - s.tile, left);
    s.unit_tiles = nt;
    s.len = len;
    s.index = ++index;
    left -= s.n;
    off += s.n;
    return true;
  }
};

// tcgen05.ld of 16 lanes x 8 N columns: thread t gets, for each group j of 8
// columns, lane t / 4 and columns 8 j + 2 (t % 4) + {0, 1} in r[4j], r[4j+1],
// and lane t / 4 + 8 of the same columns in r[4j+2], r[4j+3].
template <int N>
__device__ __forceinline__ void tmem_ld16x256(uint32_t taddr, uint32_t (&r)[4 * N]) {
  if constexpr (N == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else if constexpr (N == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    static_assert(N == 8, "groups of 8 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  }
}
// 32 lanes x 16 columns (tmem_ld32 and tmem_st32 for half the columns).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Barrier of the 128 softmax threads, and the same with an "any" of a flag.
__device__ __forceinline__ void la_bar() {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool la_bar_any(bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// 3-D tiled load: columns, row in the page, page.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// kind::f16 with fp16 operands instead of bf16 ones.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn_major, int b_mn_major) {
  return idesc_bf16_f32(M, N, a_mn_major, b_mn_major) & ~((7u << 7) | (7u << 10));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return (uint32_t)__bfloat16_as_ushort(h.x) | ((uint32_t)__bfloat16_as_ushort(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return (uint32_t)__half_as_ushort(__low2half(h)) | ((uint32_t)__half_as_ushort(__high2half(h)) << 16);
}

// Whether any of eight 16-bit floats is infinite or NaN (all exponent bits set).
template <bool FP4>
__device__ __forceinline__ bool la_not_finite(const uint4 &v) {
  const uint32_t e = FP4 ? 0x7c00u : 0x7f80u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (w[i] & e) == e || ((w[i] >> 16) & e) == e;
  return bad;
}

template <int NB, bool FP4>
__global__ void __launch_bounds__(192 + (FP4 ? kLaDequantWarps * 32 : 0), 1)
latent_attend_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_q,
                     const LatentAttend p) {
  extern __shared__ __align__(1024) unsigned char la_smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(la_smem_raw) + 1023) & ~uintptr_t(1023));
  const LaLayout ly = la_layout(NB, p.width, FP4);
  LaControl *ctl = reinterpret_cast<LaControl *>(smem + ly.control);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (p.width + 63) / 64, pairs = (chunks + 1) / 2, vblocks = (p.rank + 127) / 128;
  const int n_slots = p.slots;
  constexpr int kStatCols = 4 * NB;   // S^T behind the four blocks of O^T

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_slots; ++s) {
      mbar_init(&ctl->full[s], FP4 ? kLaDequantWarps : 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < kLaRawStages; ++s) {
      mbar_init(&ctl->raw_full[s], 1);
      mbar_init(&ctl->raw_empty[s], kLaDequantWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->pv_done[i], 1);
    }
    mbar_init(&ctl->q_full, FP4 ? kLaDequantWarps : 1);
    mbar_init(&ctl->q_empty, 1);
    mbar_init(&ctl->o_free, 4);
    mbar_fence_init();
    ctl->fail = 0;
    ctl->first_b = 0;
    ctl->first_off = 0;
    ctl->n_tiles = 0;
  }
  if (warp == 0) tmem_alloc(&ctl->tmem_base, 512);
  // This CTA's range of the tile stream: every thread sums a consecutive run
  // of requests, and the one whose run holds the start walks to it.
  {
    long long *scratch = reinterpret_cast<long long *>(ctl->wmax);   // per warp, before it is in use
    const int per = (p.batch + blockDim.x - 1) / blockDim.x;
    const int b0 = threadIdx.x * per, b1 = smin(b0 + per, p.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int32_t n = p.lengths[b];
      if (blockIdx.x == 0 && (n < 0 || n > (int64_t)p.max_pages * p.page_size)) set_status(p.status, kDevStatusCheck);
      mine += (long long)la_tiles(la_length(p, b)) * p.row_blocks;
    }
    long long before = mine, total = 0;   // inclusive over the warp first
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) scratch[warp] = before;
    __syncthreads();
    before -= mine;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
      const long long v = scratch[w];
      if (w < warp) before += v;
      total += v;
    }
    const long long share = la_share(total, p.n_ctas), start = share * blockIdx.x;
    if (start < total && start >= before && start < before + mine) {
      long long at = before;
      int b = b0;
      while (true) {
        const long long n = (long long)la_tiles(la_length(p, b)) * p.row_blocks;
        if (start < at + n) break;
        at += n;
        ++b;
      }
      ctl->first_b = b;
      ctl->first_off = (int)(start - at);
      ctl->n_tiles = (int)smin<long long>(share, total - start);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // the combine kernel may set itself up
  const uint32_t tmem = ctl->tmem_base;
  unsigned char *ring = smem + ly.ring;

  if (threadIdx.x == 0) {
    // ------------------------------------------------------------ producer
    LaWalk walk(ctl);
    LaSegment s;
    uint32_t slot = 0, raw = 0;
    bool ok = true;
    const int box = smin(p.page_size, kLaTile);
    while (ok && walk.next(p, s)) {
      if constexpr (!FP4) {
        if (s.index > 0) ok = mbar_wait(&ctl->q_empty, (uint32_t)(s.index - 1) & 1, p.status);
        if (!ok) break;
        mbar_arrive_expect_tx(&ctl->q_full, (uint32_t)(chunks * NB * 128));
        for (int c = 0; c < chunks; ++c)
          tma_load_2d(smem + ly.q + c * NB * 128, &map_q, &ctl->q_full, c * 64, s.b * p.rows + s.rb * NB);
      }
      const int32_t *table = p.block_table + (int64_t)s.b * p.max_pages;
      int32_t id[4], next_id[4];
      // pages of tile j: those that hold tokens below the length
      auto look = [&](int j, int32_t (&to)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t tok = (int64_t)j * kLaTile + i * box;
          to[i] = (i * box < kLaTile && tok < s.len) ? table[tok >> p.page_shift] : 0;
        }
      };
      look(s.tile, next_id);
      for (int j = s.tile; j < s.tile + s.n && ok; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = next_id[i];
        if (j + 1 < s.tile + s.n) look(j + 1, next_id);
        int boxes = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i * box < kLaTile && j * kLaTile + i * box < s.len) {
            boxes = i + 1;
            if (id[i] < 0 || id[i] >= p.n_pages) set_status(p.status, kDevStatusCheck);
          }
        const int row = (j * kLaTile) & (p.page_size - 1);
        if constexpr (FP4) {
          const int st = (int)(raw % kLaRawStages);
          if (raw >= kLaRawStages) ok = mbar_wait(&ctl->raw_empty[st], ((raw / kLaRawStages) - 1) & 1, p.status);
          if (!ok) break;
          unsigned char *dst = smem + ly.raw + st * la_raw_bytes(p.width);
          const int64_t page_bytes = latent_page_bytes(true, p.page_size, p.width);
          const uint32_t cb = (uint32_t)(box * (p.width / 2)), sb = (uint32_t)(box * (p.width / 16));
          uint32_t bytes = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < boxes && id[i] >= 0 && id[i] < p.n_pages) bytes += cb + sb;
          mbar_arrive_expect_tx(&ctl->raw_full[st], bytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < boxes && id[i] >= 0 && id[i] < p.n_pages) {
              const unsigned char *page = p.cache + id[i] * page_bytes;
              bulk_load(dst + i * cb, page + (int64_t)row * (p.width / 2), cb, &ctl->raw_full[st]);
              bulk_load(dst + kLaTile * (p.width / 2) + i * sb,
                        page + (int64_t)p.page_size * (p.width / 2) + (int64_t)row * (p.width / 16), sb,
                        &ctl->raw_full[st]);
            }
          ++raw;
        } else {
          for (int k = 0; k < pairs && ok; ++k, ++slot) {
            const int pr = pairs - 1 - k, st = (int)(slot % n_slots);
            if (slot >= (uint32_t)n_slots) ok = mbar_wait(&ctl->empty[st], ((slot / n_slots) - 1) & 1, p.status);
            if (!ok) break;
            const int halves = smin(2, chunks - 2 * pr);
            unsigned char *dst = ring + st * kLaSlot;
            mbar_arrive_expect_tx(&ctl->full[st], (uint32_t)(halves * boxes * box * 128));
            for (int h = 0; h < halves; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < boxes)
                  tma_load_3d(dst + h * (kLaTile * 128) + i * box * 128, &map_kv, &ctl->full[st], (2 * pr + h) * 64, row, id[i]);
          }
        }
      }
    }
    if (!ok) {   // let the copies in flight land before the CTA ends
      if constexpr (!FP4)
        for (uint32_t n = slot > (uint32_t)n_slots ? slot - n_slots : 0; n < slot; ++n)
          mbar_wait(&ctl->full[n % n_slots], (n / n_slots) & 1, p.status);
      else
        for (uint32_t n = raw > kLaRawStages ? raw - kLaRawStages : 0; n < raw; ++n)
          mbar_wait(&ctl->raw_full[n % kLaRawStages], (n / kLaRawStages) & 1, p.status);
    }
  } else if (threadIdx.x == 32) {
    // ---------------------------------------------------------- MMA issuer
    LaWalk walk(ctl);
    LaSegment s;
    bool ok = true;
    const uint32_t id_s = FP4 ? idesc_f16_f32(64, NB, 0, 0) : idesc_bf16_f32(64, NB, 0, 0);
    const uint32_t id_o = FP4 ? idesc_f16_f32(128, NB, 1, 1) : idesc_bf16_f32(128, NB, 1, 1);
    uint32_t slot = 0, n = 0;   // ring slots and tiles so far
    // the tile whose second product is still to be issued
    bool due = false, due_first = false;
    uint32_t due_slot = 0;
    int due_index = 0;
    auto second = [&]() {   // O^T += V^T P^T of tile n - 1
      const uint32_t t = n - 1, buf = t & 1;
      if (!mbar_wait(&ctl->p_full[buf], (t >> 1) & 1, p.status)) return false;
      if (due_first && due_index > 0 && !mbar_wait(&ctl->o_free, (uint32_t)(due_index - 1) & 1, p.status)) return false;
      tc_fence_after();
      const uint32_t p_base = smem_u32(smem + ly.p + buf * (kLaTile * 128));
      for (int k = pairs - vblocks; k < pairs; ++k) {
        const int vb = pairs - 1 - k;
        const int st = (int)((due_slot + k) % n_slots);
        const uint32_t a_base = smem_u32(ring + st * kLaSlot);
#pragma unroll
        for (int ks = 0; ks < kLaTile / 16; ++ks)
          umma_f16(tmem + vb * NB, sdesc_sw128(a_base + ks * 2048, kLaTile * 128, 1024),
                   sdesc_sw128(p_base + ks * 2048, kLaTile * 128, 1024), id_o, (due_first && ks == 0) ? 0u : 1u);
        umma_commit(&ctl->empty[st]);
      }
      umma_commit(&ctl->pv_done[buf]);
      return true;
    };
    while (ok && walk.next(p, s)) {
      // between units the queries change: finish the last one while they load
      if (due) ok = second();
      due = false;
      if (ok) ok = mbar_wait(&ctl->q_full, (uint32_t)s.index & 1, p.status);
      for (int j = 0; j < s.n && ok; ++j) {
        const uint32_t d = tmem + kStatCols + (n & 1) * NB;
        const uint32_t my_slot = slot;
        for (int k = 0; k < pairs && ok; ++k, ++slot) {
          const int pr = pairs - 1 - k, st = (int)(slot % n_slots);
          // a slot that the tile before still holds comes free with its second product
          if (due && slot >= (uint32_t)n_slots && slot - n_slots >= due_slot + (uint32_t)(pairs - vblocks)) {
            ok = second();
            due = false;
          }
          if (ok) ok = mbar_wait(&ctl->full[st], (slot / n_slots) & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          const int halves = smin(2, chunks - 2 * pr);
          for (int h = 0; h < halves; ++h) {
            const uint32_t a_base = smem_u32(ring + st * kLaSlot + h * (kLaTile * 128));
            const uint32_t b_base = smem_u32(smem + ly.q + (2 * pr + h) * NB * 128);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_f16(d, sdesc_sw128(a_base + ks * 32, 16, 1024), sdesc_sw128(b_base + ks * 32, 16, 1024), id_s,
                       (k | h | ks) ? 1u : 0u);
          }
          if (pr >= vblocks) umma_commit(&ctl->empty[st]);   // columns that are not values: done with
        }
        if (!ok) break;
        umma_commit(&ctl->s_full[n & 1]);
        if (j == s.n - 1) umma_commit(&ctl->q_empty);
        if (due) ok = second();
        due = true;
        due_first = j == 0;
        due_slot = my_slot;
        due_index = s.index;
        ++n;
      }
    }
    if (ok && due) second();
  } else if (warp >= 2 && warp < 6) {
    // ------------------------------------------------------------- softmax
    const int quad = warp & 3;
    const int tid = threadIdx.x - 64;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const float to2 = p.scale * 1.4426950408889634f * (FP4 ? p.cache_scale : 1.0f);
    // requests without rows
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x)
      if (la_length(p, b) == 0) {
        for (int64_t i = tid; i < (int64_t)p.rows * p.rank; i += 128) p.out[(int64_t)b * p.rows * p.rank + i] = from_f<bf16>(0.0f);
        if (p.lse)
          for (int i = tid; i < p.rows; i += 128) p.lse[(int64_t)b * p.rows + i] = -CUDART_INF_F;
        if (p.n_query > 1)
          for (int i = tid; i < p.row_blocks; i += 128) p.flags[b * p.row_blocks + i] = 0;
      }
    LaWalk walk(ctl);
    LaSegment s;
    uint32_t n = 0, slot = 0;
    bool ok = true;
    constexpr int R = NB / 4;   // query rows a thread sees: 8 (i / 2) + 2 (lane % 4) + i % 2
    while (ok && walk.next(p, s)) {
      float m[R], l[R], mul[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.0f;
        mul[i] = to2;
      }
      const int all_see = s.len - p.n_query + 1;   // tokens that every query row sees
      bool poison = false;
      for (int j = s.tile; j < s.tile + s.n; ++j, ++n) {
        const uint32_t buf = n & 1;
        if (!mbar_wait(&ctl->s_full[buf], (n >> 1) & 1, p.status)) ctl->fail = 1;
        __syncwarp();
        tc_fence_after();
        uint32_t v[2 * R];
        tmem_ld16x256<NB / 8>(tmem + lanes + kStatCols + buf * NB, v);
        tmem_wait_ld();
        if constexpr (FP4) {
          if (j == s.tile) {
            if (!mbar_wait(&ctl->q_full, (uint32_t)s.index & 1, p.status)) ctl->fail = 1;
#pragma unroll
            for (int i = 0; i < R; ++i)
              mul[i] = to2 * exp2f((float)-ctl->qexp[s.index & 1][8 * (i >> 1) + 2 * (lane & 3) + (i & 1)]);
          }
        }
        const int tok = j * kLaTile + quad * 16 + (lane >> 2);
        float y0[R], y1[R];   // tokens tok and tok + 8
        bool over = false;
        const bool edge = (j + 1) * kLaTile > all_see;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          y0[i] = __uint_as_float(v[4 * (i >> 1) + (i & 1)]) * mul[i];
          y1[i] = __uint_as_float(v[4 * (i >> 1) + 2 + (i & 1)]) * mul[i];
          if (edge) {
            const int row = s.rb * NB + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
            const int sees = p.n_query == 1 ? all_see : all_see + smin(row, p.rows - 1) / p.n_heads;
            if (tok >= sees) y0[i] = -CUDART_INF_F;
            if (tok + 8 >= sees) y1[i] = -CUDART_INF_F;
          }
          over |= fmaxf(y0[i], y1[i]) > m[i] + kLaLift;
        }
        over = la_bar_any(over);
        if (ctl->fail) {
          ok = false;
          break;
        }
        if (edge) {
          // Rows behind the length hold anything: their probabilities are 0,
          // and so must they be.  Rows that some query rows see and others do
          // not must be finite, or the unit is computed again by the combine
          // kernel.
          const int valid = smin(s.len - j * kLaTile, kLaTile), shared_rows = smax(all_see - j * kLaTile, 0);
          for (int k = pairs - vblocks; k < pairs; ++k) {
            const uint32_t sl = slot + k;
            if (!mbar_wait(&ctl->full[sl % n_slots], (sl / n_slots) & 1, p.status)) ctl->fail = 1;
            unsigned char *base = ring + (sl % n_slots) * kLaSlot;
            const int halves = smin(2, chunks - 2 * (pairs - 1 - k));
            for (int h = 0; h < halves; ++h) {
              unsigned char *half = base + h * (kLaTile * 128);
              for (int i = valid * 8 + tid; i < kLaTile * 8; i += 128)
                *reinterpret_cast<uint4 *>(half + i * 16) = make_uint4(0u, 0u, 0u, 0u);
              if (p.n_query > 1)
                for (int i = shared_rows * 8 + tid; i < valid * 8; i += 128)
                  poison |= la_not_finite<FP4>(*reinterpret_cast<const uint4 *>(half + i * 16));
            }
          }
        }
        slot += pairs;
        if (over) {
          // New reference: the largest logit of each query row so far.
#pragma unroll
          for (int i = 0; i < R; ++i) {
            float t = fmaxf(y0[i], y1[i]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            if (lane < 4) ctl->wmax[quad][8 * (i >> 1) + 2 * lane + (i & 1)] = t;
          }
          la_bar();
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int row = 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
            float t = m[i];
#pragma unroll
            for (int w = 0; w < 4; ++w) t = fmaxf(t, ctl->wmax[w][row]);
            const float f = t == m[i] ? 1.0f : exp2f(m[i] - t);   // from -inf: 0
            m[i] = t;
            l[i] *= f;
            if (quad == 0 && lane < 4) ctl->fac[row] = f;
          }
          la_bar();
          if (j > s.tile) {
            if (!mbar_wait(&ctl->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, p.status)) ctl->fail = 1;
            __syncwarp();
            tc_fence_after();
            for (int c = 0; c < vblocks * NB; c += 16) {
              uint32_t w[16];
              tmem_ld16(tmem + lanes + c, w);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * ctl->fac[(c + i) % NB]);
              tmem_st16(tmem + lanes + c, w);
            }
            tmem_wait_st();
          }
        }
        // P^T: token lines of NB query rows, swizzled; free once the products
        // of tile n - 2 are done.
        if (n >= 2 && !mbar_wait(&ctl->pv_done[buf], ((n - 2) >> 1) & 1, p.status)) ctl->fail = 1;
        unsigned char *pb = smem + ly.p + buf * (kLaTile * 128);
        const int t0 = quad * 16 + (lane >> 2);
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float a = m[i] == -CUDART_INF_F ? 0.0f : m[i], b = m[i + 1] == -CUDART_INF_F ? 0.0f : m[i + 1];
          const float p00 = ex2_approx(y0[i] - a), p01 = ex2_approx(y0[i + 1] - b);
          const float p10 = ex2_approx(y1[i] - a), p11 = ex2_approx(y1[i + 1] - b);
          l[i] += p00 + p10;
          l[i + 1] += p01 + p11;
          const uint32_t at = (uint32_t)((((i >> 1) ^ (t0 & 7)) << 4) + (lane & 3) * 4);
          *reinterpret_cast<uint32_t *>(pb + t0 * 128 + at) = FP4 ? pack_half(p00, p01) : pack_bf16(p00, p01);
          *reinterpret_cast<uint32_t *>(pb + (t0 + 8) * 128 + at) = FP4 ? pack_half(p10, p11) : pack_bf16(p10, p11);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[buf]);
      }
      if (!ok) break;
      // End of the segment: sums over the tokens, then the result.
      la_bar();   // wmax is free
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if (lane < 4) ctl->wmax[quad][8 * (i >> 1) + 2 * lane + (i & 1)] = l[i];
      }
      const bool whole = s.n == s.unit_tiles;
      const int part = 2 * (int)blockIdx.x + (s.index > 0 ? 1 : 0);
      const int rows = smin(NB, p.rows - s.rb * NB);
      const int64_t row0 = (int64_t)s.b * p.rows + s.rb * NB;
      la_bar();
      if (quad == 0 && lane < 4) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int row = 8 * (i >> 1) + 2 * lane + (i & 1);
          const float sum = (ctl->wmax[0][row] + ctl->wmax[1][row]) + (ctl->wmax[2][row] + ctl->wmax[3][row]);
          if (whole) {
            ctl->fac[row] = sum > 0.0f || sum != sum ? (FP4 ? p.cache_scale : 1.0f) / sum : 0.0f;
            if (p.lse && row < rows)
              p.lse[row0 + row] = m[i] == -CUDART_INF_F && !(sum != sum) ? -CUDART_INF_F : (m[i] + log2f(sum)) * 0.6931471805599453f;
          } else if (row < rows) {
            p.ml[(int64_t)part * NB + row] = make_float2(m[i], sum);
          }
        }
      }
      if (p.n_query > 1 && s.tile + s.n == s.unit_tiles) {
        const bool any = la_bar_any(poison);
        if (tid == 0) p.flags[s.b * p.row_blocks + s.rb] = any ? 1 : 0;
      } else {
        la_bar();
      }
      if (!mbar_wait(&ctl->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, p.status)) ctl->fail = 1;
      __syncwarp();
      tc_fence_after();
      for (int vb = 0; vb < vblocks; ++vb) {
        const int col = vb * 128 + quad * 32 + lane;
        for (int c = 0; c < NB; c += 16) {
          uint32_t w[16];
          __syncwarp();
          tmem_ld16(tmem + lanes + vb * NB + c, w);
          tmem_wait_ld();
          if (col < p.rank) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int row = c + i;
              if (row < rows) {
                if (whole) {
                  const float f = ctl->fac[row];
                  p.out[(row0 + row) * p.rank + col] = from_f<bf16>(f == 0.0f ? 0.0f : __uint_as_float(w[i]) * f);
                } else {
                  p.part[((int64_t)part * NB + row) * p.rank + col] = __uint_as_float(w[i]);
                }
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_free);
    }
  } else if (FP4 && warp >= 6) {
    // -------------------------------------------------------- 4-bit to fp16
    const int tid = threadIdx.x - 192, dw = warp - 6;
    LaWalk walk(ctl);
    LaSegment s;
    uint32_t slot = 0, raw = 0;
    bool ok = true;
    while (ok && walk.next(p, s)) {
      // queries: one warp a row, scaled so that the largest value lies in [2^14, 2^15)
      if (s.index > 0 && !mbar_wait(&ctl->q_empty, (uint32_t)(s.index - 1) & 1, p.status)) break;
      for (int row = dw; row < NB; row += kLaDequantWarps) {
        const bool live = s.rb * NB + row < p.rows;
        const bf16 *src = p.q + ((int64_t)s.b * p.rows + s.rb * NB + row) * p.width;
        float x[2 * ((S4R_MAX_LATENT_WIDTH + 63) / 64)];
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < (S4R_MAX_LATENT_WIDTH + 63) / 64; ++c) {
          const int col = c * 64 + 2 * lane;
          x[2 * c] = x[2 * c + 1] = 0.0f;
          if (live && col < p.width) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(src + col);
            x[2 * c] = __uint_as_float(w << 16);
            x[2 * c + 1] = __uint_as_float(w & 0xffff0000u);
          }
          top = fmaxf(top, fmaxf(fabsf(x[2 * c]), fabsf(x[2 * c + 1])));
        }
        top = warp_max(top);
        const int e = top > 0.0f && top < CUDART_INF_F ? 14 - ilogbf(top) : 0;
        if (lane == 0) ctl->qexp[s.index & 1][row] = e;
        const float f = ldexpf(1.0f, e / 2), g = ldexpf(1.0f, e - e / 2);   // 2^e may leave fp32's range
#pragma unroll
        for (int c = 0; c < (S4R_MAX_LATENT_WIDTH + 63) / 64; ++c)
          if (c < chunks)
            *reinterpret_cast<uint32_t *>(smem + ly.q + c * NB * 128 + sw128_offset(row, 2 * lane)) =
                pack_half(x[2 * c] * f * g, x[2 * c + 1] * f * g);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full);
      const int tok = tid & 63, quarter = tid >> 6;
      for (int j = 0; j < s.n && ok; ++j, ++raw) {
        const int st = (int)(raw % kLaRawStages);
        ok = mbar_wait(&ctl->raw_full[st], (raw / kLaRawStages) & 1, p.status);
        const unsigned char *src = smem + ly.raw + st * la_raw_bytes(p.width);
        for (int k = 0; k < pairs && ok; ++k, ++slot) {
          const int pr = pairs - 1 - k, sl = (int)(slot % n_slots);
          if (slot >= (uint32_t)n_slots) ok = mbar_wait(&ctl->empty[sl], ((slot / n_slots) - 1) & 1, p.status);
          if (!ok) break;
          const int col = pr * 128 + quarter * 32;
          unsigned char *line = ring + sl * kLaSlot + (quarter >> 1) * (kLaTile * 128) + tok * 128;
          uint4 code = make_uint4(0u, 0u, 0u, 0u);
          __half2 sc[2] = {__half2half2(__ushort_as_half(0)), __half2half2(__ushort_as_half(0))};
          if (col < p.width) {
            code = *reinterpret_cast<const uint4 *>(src + tok * (p.width / 2) + col / 2);
            const unsigned short two =
                *reinterpret_cast<const unsigned short *>(src + kLaTile * (p.width / 2) + tok * (p.width / 16) + col / 16);
            const __half2 both = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
            sc[0] = __half2half2(__low2half(both));
            sc[1] = __half2half2(__high2half(both));
          }
          const uint32_t w[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const __half2 h = __hmul2(
                  __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w[i] >> (8 * b)), __NV_E2M1)), sc[i >> 1]);
              o[b] = (uint32_t)__half_as_ushort(__low2half(h)) | ((uint32_t)__half_as_ushort(__high2half(h)) << 16);
            }
            *reinterpret_cast<uint4 *>(line + ((((quarter & 1) * 4 + i) ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->full[sl]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->raw_empty[st]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

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

// Joins the partial sums of one query row, 128 columns a CTA:
//   out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k, m = max_k m_k.
// Units that one CTA computed whole are skipped.  A unit whose flag is set
// (rows that only some of its query rows see hold infinities or NaN, which a
// probability of 0 would not hide from the others in a matrix product) is
// computed again here, row by row over the rows it sees: rare, and slow.
constexpr int kLcThreads = 128;
template <int NB, bool FP4>
__global__ void __launch_bounds__(kLcThreads) latent_combine_kernel(const LatentAttend p) {
  __shared__ long long scratch[2 * kLcThreads / 32];
  __shared__ float sm[kLcThreads / 32], sl[kLcThreads / 32], sacc[kLcThreads / 32][kLcThreads];
  const int row = blockIdx.x % p.rows, b = blockIdx.x / p.rows, rb = row / NB;
  const int col = blockIdx.y * 128 + threadIdx.x;
  const int64_t at = (int64_t)b * p.rows + row;
  pdl_wait();
  const int len = la_length(p, b), nt = la_tiles(len);
  if (nt == 0) return;
  if (p.n_query > 1 && p.flags[b * p.row_blocks + rb]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sees = len - p.n_query + 1 + row / p.n_heads;
    float m = -CUDART_INF_F, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = warp; i < sees; i += kLcThreads / 32) {
      const int32_t page = p.block_table[(int64_t)b * p.max_pages + (i >> p.page_shift)];
      if (page < 0 || page >= p.n_pages) continue;   // reported by the main kernel
      const int32_t r = i & (p.page_size - 1);
      float z = 0.0f;
      for (int c = lane; c < p.width; c += 32) z = fmaf(to_f(p.q[at * p.width + c]), latent_value<FP4>(p, page, r, c), z);
      z = warp_sum(z) * p.scale;
      const float top = fmaxf(m, z);
      const float f = m == -CUDART_INF_F ? 0.0f : expf(m - top), e = expf(z - top);
      l = l * f + e;
      m = top;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = blockIdx.y * 128 + k * 32 + lane;
        if (c < p.rank) acc[k] = acc[k] * f + e * latent_value<FP4>(p, page, r, c);
      }
    }
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sacc[warp][k * 32 + lane] = acc[k];
    __syncthreads();
    float top = -CUDART_INF_F, sum = 0.0f, o = 0.0f;
    for (int w = 0; w < kLcThreads / 32; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < kLcThreads / 32; ++w) {
      const float f = sl[w] == 0.0f ? 0.0f : expf(sm[w] - top);
      if (sl[w] != 0.0f) {
        sum += f * sl[w];
        o += f * sacc[w][threadIdx.x];
      }
    }
    if (col < p.rank) p.out[at * p.rank + col] = from_f<bf16>(sees > 0 ? o / sum : 0.0f);
    if (p.lse && blockIdx.y == 0 && threadIdx.x == 0) p.lse[at] = sees > 0 ? top + logf(sum) : -CUDART_INF_F;
    return;
  }
  long long total, before;
  la_count(p, b, scratch, total, before);
  const long long share = la_share(total, p.n_ctas);
  const long long first = before + (long long)rb * nt, last = first + nt - 1;
  const int c0 = (int)(first / share), c1 = (int)(last / share);
  if (c0 == c1) return;
  const int r = row - rb * NB;
  float top = -CUDART_INF_F;
  for (int c = c0; c <= c1; ++c) top = fmaxf(top, p.ml[(int64_t)(2 * c + (first > c * share ? 1 : 0)) * NB + r].x);
  float sum = 0.0f, o = 0.0f;
  for (int c = c0; c <= c1; ++c) {
    const int64_t k = (int64_t)(2 * c + (first > c * share ? 1 : 0)) * NB + r;
    const float2 ml = p.ml[k];
    if (ml.x == -CUDART_INF_F && ml.y == 0.0f) continue;   // this part saw nothing
    const float f = exp2f(ml.x - top);
    sum = fmaf(f, ml.y, sum);
    if (col < p.rank) o = fmaf(f, p.part[k * p.rank + col], o);
  }
  const bool none = top == -CUDART_INF_F && sum == 0.0f;
  if (col < p.rank) p.out[at * p.rank + col] = from_f<bf16>(none ? 0.0f : o * (p.cache_scale / sum));
  if (p.lse && blockIdx.y == 0 && threadIdx.x == 0)
    p.lse[at] = none ? -CUDART_INF_F : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace s4r
