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
// stream of 64-token tiles of all requests, cut into equal consecutive ranges,
// so ragged batches and single long requests load every SM alike; a request
// that crosses a border leaves partial sums, which latent_combine_kernel joins
// (no CTA waits for another one).  With more than NB query rows a request, a
// range belongs to as many CTAs as there are blocks of NB rows: they read the
// same tiles at the same time, so L2 serves all but one.
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
//   warp 1     one thread issues tcgen05.mma: O^T of tile i as soon as its
//              probabilities are there, until then S^T of tile i + 1 as far as
//              the ring holds it, so the softmax of one tile runs beside the
//              products of another; slots are released column block by column
//              block;
//   warps 2-9  softmax: probabilities against a reference maximum that moves
//              only when a logit exceeds it by more than 2^8 (then O^T is
//              rescaled in TMEM), sums in fp32, P^T into shared memory; at the
//              end of a unit they write the result or the partial sums.
//   warps 10-17 (4-bit cache) turn codes into fp16 ring slots: e2m1 * e4m3 has
//              6 significant bits, so fp16 holds the stored values exactly.
//              Queries become fp16 too, scaled by a power of two per row, exact
//              over 29 binades below the row's largest value.
// Probabilities are rounded to bf16 (4-bit cache: fp16, in its upper range) for
// the second product; the sum that divides it is not.
//
// Measured (width 576, rank 512): a CTA takes a tile in 1.64 us with 16 heads
// (together 6.65 TB/s, the rate of a copy) and 1.9 us with 64; from 4-bit rows in
// 2.0, 2.1 and 2.4 us with 16, 32 and 64.  What paces those is not known: the
// products' own rates make it 0.8 us and the passage through shared memory 0.5,
// slots handed on without conversion took 2.1 us, a ring of 6 slots instead of 9
// 2% more (both 16 heads).  Whole calls through the binding, inputs changing: 32
// ragged requests of 8250 rows on average, 64 heads 88 us; 8 requests of 32K, 128
// heads, two query tokens 230 us; 4-bit, 5 requests up to 128K, 20 heads 96 us;
// one request of 8K, 16 heads 15.5 us, of which 12 are one tile's chain of
// latencies and the rest the join of 128 parts.
//
// Every wait is bounded (umma.cuh); a wait that gives up sets the status word
// and ends its role, and every other role then runs out too.  The producer and
// the issuer end only when what they issued has ended.
#pragma once
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include <type_traits>

#include "k_page.cuh"
#include "umma.cuh"

namespace s4r {

constexpr int kLaTile = 64;                  // tokens a tile
constexpr int kLaSlot = kLaTile * 128 * 2;   // bytes of a ring slot: 64 tokens x 128 columns
constexpr int kLaMaxSlots = 12;
constexpr int kLaSmemBudget = 227 * 1024;
constexpr int kLaSoftmaxWarps = 8;           // two groups of 4, half of the query rows each
constexpr int kLaDequantWarps = 8;           // groups of kLaDequantGroup take turns at the ring slots
constexpr int kLaDequantGroup = 2;
constexpr int kLaRawStages = 2;
// How far (in powers of two) the largest logit lies above the reference when the
// reference moves, and how far a later one may come to lie.  fp16 probabilities
// (4-bit cache) start at 2^7 and end at 2^15, half of fp16's range: so they keep
// 11 bits down to 2^-21 of the largest one and are off by at most 2^-32 of it
// below that (2^-25, half of fp16's smallest step).  bf16 has fp32's range.
template <bool FP4> struct LaRange {
  static constexpr float kHead = FP4 ? 7.0f : 0.0f, kLift = kHead + 8.0f;
};

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
  int32_t rows, row_blocks, n_groups, slots; // query rows a request, blocks of NB of them, ranges of tiles, ring slots
  // workspace
  uint32_t *status;
  // first row with a value that some query rows must not see (see latent_combine_kernel), INT32_MAX for none, as each
  // softmax group found it: of a unit that one CTA computes whole, of a part
  int2 *unit_poison, *part_poison;           // [batch * row_blocks], [2 * CTAs]
  int2 *units;                               // [batch * row_blocks] first part, and how many (1: computed whole)
  float2 *ml;                                // [2 * CTAs][NB] reference maximum and sum of a partial
  float *part;                               // [2 * CTAs][NB][rank] unscaled partial results
};

// Query rows a block of the kernel takes: the least that hold a request's (a tile
// costs 1.64 us with 16, 1.70 with 32, 1.90 with 64), at most 64, which TMEM and
// shared memory hold next to a tile of 576 columns.
__host__ __device__ inline int la_block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

__host__ __device__ constexpr int la_threads(bool fp4) { return 64 + 32 * (kLaSoftmaxWarps + (fp4 ? kLaDequantWarps : 0)); }

struct LaLayout {
  int q, p, raw, ring, control, total, slots;
};
constexpr int kLaControlBytes = 2048;
__host__ __device__ inline int la_raw_bytes(int width) { return (kLaTile * width * 9 / 16 + 127) / 128 * 128; }
__host__ __device__ inline LaLayout la_layout(int nb, int width, bool fp4) {
  LaLayout l;
  const int chunks = (width + 63) / 64;
  int off = 0;
  l.q = off;
  off += chunks * nb * 128;
  off = (off + 1023) & ~1023;
  l.p = off;
  off += kLaTile * 128;
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
  uint64_t s_full[2], p_full, pv_done;
  uint64_t q_full[2], q_empty, o_free, drained;
  uint64_t never;                    // no one arrives (s4r_debug_waits)
  uint32_t tmem_base;
  int first_b, first_off, n_tiles;   // start of this CTA's range and its length
  int share;                         // tiles of a full range
  int poison[kLaSoftmaxWarps];
  int16_t qexp[2][64];               // 4-bit cache: queries are scaled by 2^qexp (segments alternate)
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

// Tiles of a range, of `total`.
__host__ __device__ inline long long la_share(long long total, int n_groups) { return (total + n_groups - 1) / n_groups; }

// The slots of the partial sums of a unit: its parts, from the record (first
// slot, count) of the CTA with its first tile.  Part 0 lies in the slot of the
// record, the others in the first slot of the CTAs behind it, row_blocks apart.
__host__ __device__ inline int la_part_slot(int first, int i, int row_blocks) {
  return i == 0 ? first : 2 * (first / 2 + i * row_blocks);
}
// Whether a record names slots that exist.  After a wait that gave up it may be
// what the memory held before the call.
__host__ __device__ inline bool la_parts_ok(int first, int count, int n_groups, int row_blocks) {
  const uint32_t ctas = (uint32_t)(n_groups * row_blocks), more = (uint32_t)count - 1u;
  return (more < (uint32_t)n_groups) & ((uint32_t)first < 2u * ctas) & ((uint32_t)first / 2u + more * (uint32_t)row_blocks < ctas);
}

// A place in a ring of n slots and the parity of its turn (no divisions: the
// single-warp roles are bound by the instructions they issue).
struct LaRing {
  int st = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void step(int n) {
    if (++st == n) {
      st = 0;
      ++turn;
    }
  }
};

// The queries of segment `index` arrive on barrier la_query_bar of two, in the
// phase of parity la_query_parity.  The softmax warps wait for them too, and may
// be a segment late (they store the end of a unit, or zeros for empty requests,
// while the products of the next segment run): the queries of segment index + 1
// may then be complete already.  On one barrier their phase would hide the one
// waited for; on two by turns the phase that could hide it is that of segment
// index + 2, whose queries wait for products that need these warps.
__host__ __device__ inline int la_query_bar(int index) { return index & 1; }
__host__ __device__ inline uint32_t la_query_parity(int index) { return (uint32_t)(index >> 1) & 1u; }

// The segments of a CTA: consecutive tiles of one request.
struct LaSegment {
  int b, tile, n, unit_tiles, len, index;
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
      if (off < nt) break;
      off = 0;
      ++b;
    }
    s.b = b;
    s.tile = off;
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
  if constexpr (N == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else if constexpr (N == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else {
    static_assert(N == 4, "groups of 8 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}
// 32 lanes x 8 columns (tmem_ld32 and tmem_st32 for a quarter of the columns).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Barrier of a group of 128 softmax threads, and the same with an "any" of a flag.
__device__ __forceinline__ void la_bar(int id) {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool la_bar_any(int id, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return (uint32_t)__half_as_ushort(__low2half(h)) | ((uint32_t)__half_as_ushort(__high2half(h)) << 16);
}

// Eight 4-bit codes (even columns in the low bits of their bytes) times a
// scale given twice: four pairs of fp16.  (Putting the codes' bits in fp16's
// place with shifts and byte permutes took 6% more time for the whole kernel
// than the conversion instruction.)
__device__ __forceinline__ void codes_to_half(uint32_t codes, uint32_t scale2, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 h0, h1, h2, h3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 h0, b0;\n\tcvt.rn.f16x2.e2m1x2 h1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 h2, b2;\n\tcvt.rn.f16x2.e2m1x2 h3, b3;\n\t"
      "mul.rn.f16x2 %0, h0, %5;\n\tmul.rn.f16x2 %1, h1, %5;\n\t"
      "mul.rn.f16x2 %2, h2, %5;\n\tmul.rn.f16x2 %3, h3, %5;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(codes), "r"(scale2));
}
// Two e4m3 scales, each as a pair of equal fp16.
__device__ __forceinline__ void scales_to_half(unsigned short two, uint32_t (&o)[2]) {
  asm("{\n\t.reg .b32 h;\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %2;\n\tmov.b32 {a, b}, h;\n\t"
      "mov.b32 %0, {a, a};\n\tmov.b32 %1, {b, b};\n\t}"
      : "=r"(o[0]), "=r"(o[1])
      : "h"(two));
}

template <int NB, bool FP4>
__global__ void __launch_bounds__(la_threads(FP4), 1)
latent_attend_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_q,
                     const LatentAttend p) {
  extern __shared__ __align__(1024) unsigned char la_smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(la_smem_raw) + 1023) & ~uintptr_t(1023));
  const LaLayout ly = la_layout(NB, p.width, FP4);
  LaControl *ctl = reinterpret_cast<LaControl *>(smem + ly.control);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int chunks = (p.width + 63) / 64, pairs = (chunks + 1) / 2, vblocks = (p.rank + 127) / 128;
  const int n_slots = p.slots, rb = blockIdx.x % p.row_blocks;   // this CTA's block of query rows
  const long long limit = wait_limit();
  const bool unreachable = wait_unreachable();
  constexpr int kStatCols = 4 * NB;   // S^T behind the four blocks of O^T

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_slots; ++s) {
      mbar_init(&ctl->full[s], FP4 ? kLaDequantGroup : 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < kLaRawStages; ++s) {
      mbar_init(&ctl->raw_full[s], 1);
      mbar_init(&ctl->raw_empty[s], kLaDequantWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->s_full[i], 1);
    mbar_init(&ctl->p_full, kLaSoftmaxWarps);
    mbar_init(&ctl->pv_done, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->q_full[i], FP4 ? kLaDequantWarps : 1);
    mbar_init(&ctl->q_empty, 1);
    mbar_init(&ctl->drained, 1);
    mbar_init(&ctl->never, 1);
    mbar_init(&ctl->o_free, kLaSoftmaxWarps);
    mbar_fence_init();
    ctl->first_b = 0;
    ctl->first_off = 0;
    ctl->n_tiles = 0;
  }
  if (warp == 0) tmem_alloc(&ctl->tmem_base, 512);
  pdl_wait();   // nothing before this touches memory that another kernel writes
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
      mine += la_tiles(la_length(p, b));
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
    const long long share = la_share(total, p.n_groups), start = share * (blockIdx.x / p.row_blocks);
    if (start < total && start >= before && start < before + mine) {
      long long at = before;
      int b = b0;
      while (true) {
        const long long n = la_tiles(la_length(p, b));
        if (start < at + n) break;
        at += n;
        ++b;
      }
      ctl->first_b = b;
      ctl->first_off = (int)(start - at);
      ctl->n_tiles = (int)smin<long long>(share, total - start);
      ctl->share = (int)share;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // the combine kernel may set itself up
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  unsigned char *ring = smem + ly.ring;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The whole warp in step, as in the MMA issuer below: its lanes read 32
    // boxes' page ids at a time, one lane issues.
    LaWalk walk(ctl);
    LaSegment s;
    LaRing slot, raw;
    int asked = -1;   // the last segment whose queries were copied
    bool ok = true;
    const uint32_t leader = elect_one();
    const int box = smin(p.page_size, kLaTile), box_shift = smin(p.page_shift, 6), per_tile = kLaTile >> box_shift;
    const int64_t page_bytes = latent_page_bytes(true, p.page_size, p.width);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __shfl_sync(0xffffffffu, (int)mbar_wait_within(bar, parity & 1, limit, p.status), 0) != 0;
    };
    while (ok && __shfl_sync(0xffffffffu, (int)walk.next(p, s), 0)) {
      s.b = __shfl_sync(0xffffffffu, s.b, 0);
      s.tile = __shfl_sync(0xffffffffu, s.tile, 0);
      s.n = __shfl_sync(0xffffffffu, s.n, 0);
      s.len = __shfl_sync(0xffffffffu, s.len, 0);
      s.index = __shfl_sync(0xffffffffu, s.index, 0);
      // ids of the boxes from `first` on; a box behind the length has none
      const int32_t *table = p.block_table + (int64_t)s.b * p.max_pages;
      auto look = [&](int first) {
        const int64_t tok = ((int64_t)first + lane) << box_shift;
        int32_t id = 0;
        if (tok < s.len) {
          id = table[tok >> p.page_shift];
          if (id < 0 || id >= p.n_pages) {
            set_status(p.status, kDevStatusCheck);
            id = -1;
          }
        }
        return id;
      };
      int next = s.tile * per_tile, left = 0;   // the box after those in `ids`; how many of `ids` are left
      int32_t ids = 0, more = look(next);
      if constexpr (!FP4) {
        if (s.index > 0) ok = wait(&ctl->q_empty, (uint32_t)(s.index - 1));
        if (!ok) break;
        uint64_t *q_full = &ctl->q_full[la_query_bar(s.index)];
        asked = s.index;
        mbar_expect_if(leader, q_full, (uint32_t)(chunks * NB * 128));
        for (int c = 0; c < chunks; ++c)
          tma_load_2d_if(leader, smem + ly.q + c * NB * 128, &map_q, q_full, c * 64, s.b * p.rows + rb * NB);
      }
      for (int j = s.tile; j < s.tile + s.n && ok; ++j) {
        if (left == 0) {   // 32 is a multiple of a tile's boxes
          ids = more;
          next += 32;
          left = 32;
          more = look(next);
        }
        const int at = 32 - left;
        left -= per_tile;
        const int boxes = smin(per_tile, (s.len - j * kLaTile + box - 1) >> box_shift);
        const int row = (j * kLaTile) & (p.page_size - 1);
        if constexpr (FP4) {
          const int st = raw.st;
          if (raw.turn > 0) ok = wait(&ctl->raw_empty[st], raw.turn - 1);
          if (!ok) break;
          unsigned char *dst = smem + ly.raw + st * la_raw_bytes(p.width);
          const uint32_t cb = (uint32_t)(box * (p.width / 2)), sb = (uint32_t)(box * (p.width / 16));
          const uint32_t known = __ballot_sync(0xffffffffu, ids >= 0) >> at;
          mbar_expect_if(leader, &ctl->raw_full[st], (cb + sb) * __popc(known & ((1u << boxes) - 1u)));
          for (int i = 0; i < boxes; ++i) {
            const int32_t id = __shfl_sync(0xffffffffu, ids, at + i);
            const unsigned char *page = p.cache + id * page_bytes;
            const uint32_t on = leader && id >= 0;
            bulk_load_if(on, dst + i * cb, page + (int64_t)row * (p.width / 2), cb, &ctl->raw_full[st]);
            bulk_load_if(on, dst + kLaTile * (p.width / 2) + i * sb,
                         page + (int64_t)p.page_size * (p.width / 2) + (int64_t)row * (p.width / 16), sb, &ctl->raw_full[st]);
          }
          raw.step(kLaRawStages);
        } else {
          for (int pr = pairs - 1; pr >= 0 && ok; --pr, slot.step(n_slots)) {
            if (slot.turn > 0) ok = wait(&ctl->empty[slot.st], slot.turn - 1);
            if (!ok) break;
            const int halves = smin(2, chunks - 2 * pr);
            unsigned char *dst = ring + slot.st * kLaSlot;
            mbar_expect_if(leader, &ctl->full[slot.st], (uint32_t)(halves * boxes) << (7 + box_shift));
            for (int i = 0; i < boxes; ++i) {
              // an unknown page is read as page -1: the copy fills in zeros
              const int32_t id = __shfl_sync(0xffffffffu, ids, at + i);
              tma_load_3d_if(leader, dst + (i << (7 + box_shift)), &map_kv, &ctl->full[slot.st], 2 * pr * 64, row, id);
              if (halves > 1)
                tma_load_3d_if(leader, dst + kLaTile * 128 + (i << (7 + box_shift)), &map_kv, &ctl->full[slot.st],
                               (2 * pr + 1) * 64, row, id);
            }
          }
        }
      }
    }
    // Shared memory goes with the CTA: let the copies in flight land, whichever
    // role gave up.
    auto land = [&](uint64_t *bar, uint32_t parity) { mbar_wait_within(bar, parity & 1, kWaitCycles, p.status); };
    if constexpr (!FP4) {
      if (asked >= 0) land(&ctl->q_full[la_query_bar(asked)], la_query_parity(asked));
      for (int i = 0; i < n_slots; ++i)
        if (slot.turn > 0 || i < slot.st) land(&ctl->full[i], slot.turn - (i < slot.st ? 0 : 1));
    } else {
      for (int i = 0; i < kLaRawStages; ++i)
        if (raw.turn > 0 || i < raw.st) land(&ctl->raw_full[i], raw.turn - (i < raw.st ? 0 : 1));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks along and one lane issues under a predicate.  What
    // steers it is broadcast from lane 0, so that the compiler sees uniform
    // control flow and keeps descriptors in uniform registers: moving them
    // there for every instruction took 70 cycles each, twice the 33 to 49 of
    // the products themselves.
    LaWalk walk(ctl);
    LaSegment s;
    bool ok = true;
    const uint32_t leader = elect_one();
    const uint32_t id_s = FP4 ? idesc_f16_f32(64, NB, 0, 0) : idesc_bf16_f32(64, NB, 0, 0);
    const uint32_t id_o = FP4 ? idesc_f16_f32(128, NB, 1, 1) : idesc_bf16_f32(128, NB, 1, 1);
    // descriptors of slot 0, of the queries' columns 0 and of P^T; the others are offsets (in 16 bytes) away
    const uint64_t k_desc = sdesc_sw128(smem_u32(ring), 16, 1024), q_desc = sdesc_sw128(smem_u32(smem + ly.q), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(ring), kLaTile * 128, 1024);
    const uint64_t p_desc = sdesc_sw128(smem_u32(smem + ly.p), kLaTile * 128, 1024);
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __shfl_sync(0xffffffffu, (int)mbar_wait_within(bar, parity & 1, limit, p.status), 0) != 0; };
    auto ready = [&](uint64_t *bar, uint32_t parity) { return __shfl_sync(0xffffffffu, (int)mbar_test(bar, parity & 1), 0) != 0; };
    uint64_t *const p_full = unreachable ? &ctl->never : &ctl->p_full;
    LaRing slot;
    uint32_t n = 0;                      // tiles so far
    bool due = false, due_first = false; // the tile before waits for its second product; it is its unit's first
    LaRing due_slot;                     // its first slot of values
    int due_index = 0;
    auto second = [&]() {   // O^T += V^T P^T of tile n - 1
      if (!wait(p_full, n - 1)) return false;
      if (due_first && due_index > 0 && !wait(&ctl->o_free, (uint32_t)(due_index - 1))) return false;
      tc_fence_after();
      for (int vb = vblocks - 1; vb >= 0; --vb, due_slot.step(n_slots)) {
        const uint64_t a = v_desc + (uint32_t)__shfl_sync(0xffffffffu, due_slot.st, 0) * (kLaSlot >> 4);
#pragma unroll
        for (int ks = 0; ks < kLaTile / 16; ++ks)
          umma_f16_if(leader, tmem + vb * NB, a + ks * (2048 >> 4), p_desc + ks * (2048 >> 4), id_o, ks > 0 || !due_first);
        umma_commit_if(leader, &ctl->empty[due_slot.st]);
      }
      umma_commit_if(leader, &ctl->pv_done);
      return true;
    };
    while (ok && __shfl_sync(0xffffffffu, (int)walk.next(p, s), 0)) {
      s.n = __shfl_sync(0xffffffffu, s.n, 0);
      s.index = __shfl_sync(0xffffffffu, s.index, 0);
      // between units the queries change: finish the last one while they load
      if (due) ok = second();
      due = false;
      if (ok) ok = wait(&ctl->q_full[la_query_bar(s.index)], la_query_parity(s.index));
      for (int j = 0; j < s.n && ok; ++j) {
        const uint32_t d = tmem + kStatCols + (n & 1) * NB;
        LaRing first = slot;
        for (int k = pairs - 1; k >= 0 && ok; --k, slot.step(n_slots)) {
          // The second product of the tile before goes first once its
          // probabilities are there (its slots are then free early), or if
          // this slot comes free only with it.
          if (due && (ready(p_full, n - 1) ||
                      (slot.turn > 0 && (slot.turn - 1 > due_slot.turn || (slot.turn - 1 == due_slot.turn && slot.st >= due_slot.st))))) {
            ok = second();
            due = false;
          }
          if (ok) ok = wait(&ctl->full[slot.st], slot.turn);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = k_desc + (uint32_t)__shfl_sync(0xffffffffu, slot.st, 0) * (kLaSlot >> 4), b = q_desc + (uint32_t)k * (2 * NB * 128 >> 4);
          umma_f16_if(leader, d, a, b, id_s, k < pairs - 1);
#pragma unroll
          for (int ks = 1; ks < 4; ++ks) umma_f16_if(leader, d, a + ks * 2, b + ks * 2, id_s, true);
          if (2 * k + 1 < chunks)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_f16_if(leader, d, a + (kLaTile * 128 >> 4) + ks * 2, b + (NB * 128 >> 4) + ks * 2, id_s, true);
          if (k >= vblocks) {   // columns that are not values: done with
            umma_commit_if(leader, &ctl->empty[slot.st]);
            first = slot;
            first.step(n_slots);
          }
        }
        if (!ok) break;
        umma_commit_if(leader, &ctl->s_full[n & 1]);
        if (j == s.n - 1) umma_commit_if(leader, &ctl->q_empty);
        if (due) ok = second();
        due = true;
        due_first = j == 0;
        due_slot = first;
        due_index = s.index;
        ++n;
      }
    }
    if (ok && due) ok = second();
    // TMEM and shared memory go with the CTA: let the products in flight end,
    // whichever role gave up.
    umma_commit_if(leader, &ctl->drained);
    mbar_wait_within(&ctl->drained, 0, kWaitCycles, p.status);
    __syncwarp();
  } else if (warp < 2 + kLaSoftmaxWarps) {
    // ------------------------------------------------------------- softmax
    // Two groups of four warps, each with half of the query rows and all tokens;
    // nothing passes between them but their arrivals.
    const int quad = warp & 3, grp = (warp - 2) >> 2, bar = 1 + grp, r0 = grp * (NB / 2);
    const int tid = threadIdx.x - 64 - 128 * grp;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const float to2 = p.scale * 1.4426950408889634f * (FP4 ? p.cache_scale : 1.0f);
    // requests without rows
    for (int b = blockIdx.x; b < p.batch && grp == 0; b += gridDim.x)
      if (la_length(p, b) == 0) {
        for (int64_t i = tid; i < (int64_t)p.rows * p.rank; i += 128) p.out[(int64_t)b * p.rows * p.rank + i] = from_f<bf16>(0.0f);
        if (p.lse)
          for (int i = tid; i < p.rows; i += 128) p.lse[(int64_t)b * p.rows + i] = -CUDART_INF_F;
        for (int i = tid; i < p.row_blocks; i += 128) {
          p.unit_poison[b * p.row_blocks + i] = make_int2(INT32_MAX, INT32_MAX);
          p.units[b * p.row_blocks + i] = make_int2(0, 1);
        }
      }
    LaWalk walk(ctl);
    LaSegment s;
    uint32_t n = 0;
    LaRing slot;
    bool ok = true, bad = false;   // bad: a wait of this thread gave up
    constexpr int R = NB / 8;   // query rows a thread sees: r0 + 8 (i / 2) + 2 (lane % 4) + i % 2
    while (ok && walk.next(p, s)) {
      float m[R], l[R], mul[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.0f;
        mul[i] = to2;
      }
      const int all_see = s.len - p.n_query + 1;   // tokens that every query row sees
      int poison = INT32_MAX;
      for (int j = s.tile; j < s.tile + s.n; ++j, ++n) {
        const uint32_t buf = n & 1;
        if (!mbar_wait_within(&ctl->s_full[buf], (n >> 1) & 1, limit, p.status)) bad = true;
        __syncwarp();
        tc_fence_after();
        uint32_t v[2 * R];
        tmem_ld16x256<NB / 16>(tmem + lanes + kStatCols + buf * NB + r0, v);
        tmem_wait_ld();
        if constexpr (FP4) {
          if (j == s.tile) {
            if (!mbar_wait_within(&ctl->q_full[la_query_bar(s.index)], la_query_parity(s.index), limit, p.status)) bad = true;
#pragma unroll
            for (int i = 0; i < R; ++i)
              mul[i] = to2 * exp2f((float)-ctl->qexp[s.index & 1][r0 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1)]);
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
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            int sees = all_see;
            if (p.n_query > 1) sees += smin(rb * NB + r0 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1), p.rows - 1) / p.n_heads;
            if (tok >= sees) y0[i] = -CUDART_INF_F;
            if (tok + 8 >= sees) y1[i] = -CUDART_INF_F;
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) over |= fmaxf(y0[i], y1[i]) > m[i] + LaRange<FP4>::kLift;
        // A wait that gave up in one thread ends the group as a whole: the second
        // vote tells it from a moved maximum, so that all threads agree.
        over = la_bar_any(bar, over || bad);
        if (over && la_bar_any(bar, bad)) {
          ok = false;
          break;
        }
        if (edge) {
          // Rows behind the length hold anything: their probabilities are 0,
          // and so must they be.  Rows that some query rows see and others do
          // not must be finite, too: what is not becomes 0, and the query rows
          // that see it are computed again by the combine kernel.
          const int valid = smin(s.len - j * kLaTile, kLaTile), shared_rows = smax(all_see - j * kLaTile, 0);
          LaRing at = slot;
          for (int k = 0; k < pairs; ++k, at.step(n_slots)) {
            if (k < pairs - vblocks) continue;
            if (!mbar_wait_within(&ctl->full[at.st], at.turn & 1, limit, p.status)) bad = true;
            unsigned char *base = ring + at.st * kLaSlot;
            const int halves = smin(2, chunks - 2 * (pairs - 1 - k));
            for (int h = 0; h < halves; ++h) {
              unsigned char *half = base + h * (kLaTile * 128);
              if (h == grp || halves == 1)   // a single half by both
                for (int i = valid * 8 + tid; i < kLaTile * 8; i += 128)
                  *reinterpret_cast<uint4 *>(half + i * 16) = make_uint4(0u, 0u, 0u, 0u);
              if (p.n_query > 1 && (h == grp || halves == 1))
                for (int i = shared_rows * 8 + tid; i < valid * 8; i += 128)
                  if (clear_not_finite<FP4 ? 0x7c00u : 0x7f80u>(*reinterpret_cast<uint4 *>(half + i * 16)))
                    poison = smin(poison, j * kLaTile + (i >> 3));
            }
          }
        }
        slot.st += pairs;   // pairs <= n_slots
        if (slot.st >= n_slots) {
          slot.st -= n_slots;
          ++slot.turn;
        }
        if (over) {
          // New reference: the largest logit of each query row so far, less kHead.
#pragma unroll
          for (int i = 0; i < R; ++i) {
            float t = fmaxf(y0[i], y1[i]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            if (lane < 4) ctl->wmax[quad][r0 + 8 * (i >> 1) + 2 * lane + (i & 1)] = t;
          }
          la_bar(bar);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int row = r0 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
            float t = m[i];
#pragma unroll
            for (int w = 0; w < 4; ++w) t = fmaxf(t, ctl->wmax[w][row] - LaRange<FP4>::kHead);
            const float f = t == m[i] ? 1.0f : exp2f(m[i] - t);   // from -inf: 0
            m[i] = t;
            l[i] *= f;
            if (quad == 0 && lane < 4) ctl->fac[row] = f;
          }
          la_bar(bar);
          if (j > s.tile) {
            if (!mbar_wait_within(&ctl->pv_done, (n - 1) & 1, limit, p.status)) bad = true;
            __syncwarp();
            tc_fence_after();
            for (int c = r0; c < r0 + NB / 2; c += 8) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = ctl->fac[c + i];
              for (int vb = 0; vb < vblocks; ++vb) {
                uint32_t w[8];
                tmem_ld8(tmem + lanes + vb * NB + c, w);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f[i]);
                tmem_st8(tmem + lanes + vb * NB + c, w);
              }
            }
            tmem_wait_st();
          }
        }
        // P^T: token lines of NB query rows, swizzled; free once the products
        // of tile n - 1 are done.
        if (n >= 1 && !mbar_wait_within(&ctl->pv_done, (n - 1) & 1, limit, p.status)) bad = true;
        unsigned char *pb = smem + ly.p;
        const int t0 = quad * 16 + (lane >> 2);
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float a = m[i] == -CUDART_INF_F ? 0.0f : m[i], b = m[i + 1] == -CUDART_INF_F ? 0.0f : m[i + 1];
          const float p00 = ex2_approx(y0[i] - a), p01 = ex2_approx(y0[i + 1] - b);
          const float p10 = ex2_approx(y1[i] - a), p11 = ex2_approx(y1[i + 1] - b);
          l[i] += p00 + p10;
          l[i + 1] += p01 + p11;
          const uint32_t at = (uint32_t)((((r0 / 8 + (i >> 1)) ^ (t0 & 7)) << 4) + (lane & 3) * 4);
          *reinterpret_cast<uint32_t *>(pb + t0 * 128 + at) = FP4 ? pack_half(p00, p01) : pack_bf16(p00, p01);
          *reinterpret_cast<uint32_t *>(pb + (t0 + 8) * 128 + at) = FP4 ? pack_half(p10, p11) : pack_bf16(p10, p11);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full);
      }
      if (!ok) break;
      // End of the segment: sums over the tokens (a thread a row), then the
      // result.
      la_bar(bar);   // wmax is free
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        const int row = r0 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
        if (lane < 4) {
          ctl->wmax[quad][row] = l[i];
          if (quad == 0) ctl->fac[row] = m[i];
        }
      }
      const bool whole = s.n == s.unit_tiles;
      const int part = 2 * (int)blockIdx.x + (s.index > 0 ? 1 : 0);
      const int rows = smin(NB, p.rows - rb * NB);
      const int64_t row0 = (int64_t)s.b * p.rows + rb * NB;
      la_bar(bar);
      if (tid < NB / 2) {
        const int row = r0 + tid;
        const float sum = (ctl->wmax[0][row] + ctl->wmax[1][row]) + (ctl->wmax[2][row] + ctl->wmax[3][row]);
        const float top = ctl->fac[row];
        if (whole) {
          ctl->fac[row] = sum > 0.0f || sum != sum ? (FP4 ? p.cache_scale : 1.0f) / sum : 0.0f;
          if (p.lse && row < rows)
            p.lse[row0 + row] = top == -CUDART_INF_F && !(sum != sum) ? -CUDART_INF_F : (top + log2f(sum)) * 0.6931471805599453f;
        } else if (row < rows) {
          p.ml[(int64_t)part * NB + row] = make_float2(top, sum);
        }
      }
      // The CTA with a unit's first tile says which parts there will be: its
      // own one (the second if it began with another request) and the first
      // one of each CTA behind it that has the same query rows.
      if (s.tile == 0 && tid == 0 && grp == 0) {
        const int rest = s.unit_tiles - s.n, share = ctl->share;
        p.units[s.b * p.row_blocks + rb] = make_int2(part, 1 + (rest + share - 1) / share);
      }
      if (p.n_query > 1) {
        // each group has looked at one half of the columns
        poison = __reduce_min_sync(0xffffffffu, poison);
        if (lane == 0) ctl->poison[warp - 2] = poison;
      }
      la_bar(bar);
      if (p.n_query > 1 && tid == 0) {
        const int *of = ctl->poison + 4 * grp;
        int2 *to = whole ? p.unit_poison + s.b * p.row_blocks + rb : p.part_poison + part;
        (grp ? to->y : to->x) = smin(smin(of[0], of[1]), smin(of[2], of[3]));
      }
      if (!mbar_wait_within(&ctl->pv_done, (n - 1) & 1, limit, p.status)) bad = true;
      __syncwarp();
      tc_fence_after();
      if (whole) {
        float f[NB / 2];   // of this group's rows
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) f[i] = ctl->fac[r0 + i];
        bool none = false;   // a row without any weight is 0, whatever its values are
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) none |= f[i] == 0.0f;
        const bool up1 = lane & 1, up2 = lane & 2, up4 = lane & 4;
        bf16 *out = p.out + (row0 + r0 + (lane & 7)) * p.rank + quad * 32 + (lane & 24);
        for (int vb = 0; vb < vblocks; ++vb, out += 128) {
          uint32_t w[NB / 16][8];
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NB / 16; ++c) tmem_ld8(tmem + lanes + vb * NB + r0 + 8 * c, w[c]);
          tmem_wait_ld();
          if (none) {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i)
              if (f[i] == 0.0f) w[i / 8][i % 8] = 0u;
          }
          const bool in = vb * 128 + quad * 32 + (lane & 24) < p.rank;
#pragma unroll
          for (int c = 0; c < NB / 16; ++c) {
            // Eight columns of one row a lane, by exchanges with the lanes 1, 2
            // and 4 away: a 16-byte store.
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t t = pack_bf16(__uint_as_float(w[c][2 * i]) * f[8 * c + 2 * i],
                                           __uint_as_float(w[c][2 * i + 1]) * f[8 * c + 2 * i + 1]);
              const uint32_t x = __shfl_xor_sync(0xffffffffu, t, 1);
              q[i] = up1 ? __byte_perm(x, t, 0x7632) : __byte_perm(t, x, 0x5410);   // row 2 i + lane % 2
            }
            const uint32_t xa = __shfl_xor_sync(0xffffffffu, up2 ? q[0] : q[1], 2), xb = __shfl_xor_sync(0xffffffffu, up2 ? q[2] : q[3], 2);
            const uint32_t a0 = up2 ? xa : q[0], a1 = up2 ? q[1] : xa, b0 = up2 ? xb : q[2], b1 = up2 ? q[3] : xb;
            const uint32_t x0 = __shfl_xor_sync(0xffffffffu, up4 ? a0 : b0, 4), x1 = __shfl_xor_sync(0xffffffffu, up4 ? a1 : b1, 4);
            if (in && r0 + 8 * c + (lane & 7) < rows)
              *reinterpret_cast<uint4 *>(out + (int64_t)8 * c * p.rank) = up4 ? make_uint4(x0, x1, b0, b1) : make_uint4(a0, a1, x0, x1);
          }
        }
      } else {
        float *pt = p.part + ((int64_t)part * NB + r0) * p.rank + quad * 32 + lane;
        for (int vb = 0; vb < vblocks; ++vb, pt += 128) {
          uint32_t w[NB / 16][8];
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NB / 16; ++c) tmem_ld8(tmem + lanes + vb * NB + r0 + 8 * c, w[c]);
          tmem_wait_ld();
          const int live = vb * 128 + quad * 32 + lane < p.rank ? rows - r0 : 0;
          float *at = pt;
#pragma unroll
          for (int i = 0; i < NB / 2; ++i, at += p.rank)
            if (i < live) *at = __uint_as_float(w[i / 8][i % 8]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_free);
    }
  } else if (FP4) {
    // -------------------------------------------------------- 4-bit to fp16
    const int dw = warp - 2 - kLaSoftmaxWarps, my = dw / kLaDequantGroup;
    LaWalk walk(ctl);
    LaSegment s;
    constexpr int kGroups = kLaDequantWarps / kLaDequantGroup;
    LaRing slot, raw;
    int turn = 0;   // the group whose slot is next
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_within(bar, parity & 1, limit, p.status)) != 0; };
    while (ok && walk.next(p, s)) {
      // queries: one warp a row, scaled so that the largest value lies in [2^14, 2^15)
      if (s.index > 0 && !wait(&ctl->q_empty, (uint32_t)(s.index - 1))) break;
      for (int row = dw; row < NB; row += kLaDequantWarps) {
        const bool live = rb * NB + row < p.rows;
        const bf16 *src = p.q + ((int64_t)s.b * p.rows + rb * NB + row) * p.width;
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
        if (lane == 0) ctl->qexp[s.index & 1][row] = (int16_t)e;
        const float f = ldexpf(1.0f, e / 2), g = ldexpf(1.0f, e - e / 2);   // 2^e may leave fp32's range
#pragma unroll
        for (int c = 0; c < (S4R_MAX_LATENT_WIDTH + 63) / 64; ++c)
          if (c < chunks)
            *reinterpret_cast<uint32_t *>(smem + ly.q + c * NB * 128 + sw128_offset(row, 2 * lane)) =
                pack_half(x[2 * c] * f * g, x[2 * c + 1] * f * g);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[la_query_bar(s.index)]);
      // Ring slots: a group of two warps takes every fourth, a thread one token
      // of it, 128 columns.
      const int tok = (dw % kLaDequantGroup) * 32 + lane;
      for (int j = 0; j < s.n && ok; ++j, raw.step(kLaRawStages)) {
        const int st = raw.st;
        ok = wait(&ctl->raw_full[st], raw.turn);
        const unsigned char *src = smem + ly.raw + st * la_raw_bytes(p.width);
        for (int pr = pairs - 1; pr >= 0 && ok; --pr, slot.step(n_slots), turn = (turn + 1) % kGroups) {
          if (turn != my) continue;
          const int sl = slot.st;
          const unsigned char *codes = src + tok * (p.width / 2) + pr * 64;
          const unsigned char *scales = src + kLaTile * (p.width / 2) + tok * (p.width / 16) + pr * 8;
          uint4 code[4];
          unsigned short two[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const bool in = pr * 128 + c * 32 < p.width;   // columns behind the row are zeros
            code[c] = in ? *reinterpret_cast<const uint4 *>(codes + c * 16) : make_uint4(0u, 0u, 0u, 0u);
            two[c] = in ? *reinterpret_cast<const unsigned short *>(scales + c * 2) : (unsigned short)0;
          }
          if (slot.turn > 0) ok = wait(&ctl->empty[sl], slot.turn - 1);
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            unsigned char *line = ring + sl * kLaSlot + (c >> 1) * (kLaTile * 128) + tok * 128;
            uint32_t sc[2];
            scales_to_half(two[c], sc);
            const uint32_t w[4] = {code[c].x, code[c].y, code[c].z, code[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t o[4];
              codes_to_half(w[i], sc[i >> 1], o);
              *reinterpret_cast<uint4 *>(line + ((((c & 1) * 4 + i) ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->full[sl]);
        }
        __syncwarp();
        if (!ok) break;   // the copies into this stage may still be under way: it is not free
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

// Joins the partial sums of one query row (and of `cols` columns, a multiple
// of 128 that is less than the rank when there are few rows), a CTA each:
//   out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k, m = max_k m_k.
// Units that one CTA computed whole are skipped.  Query rows that see an
// infinity or a NaN which other rows of the request must not see (the products
// took it as 0) are computed again here, row by row over the cache: rare, and
// slow.
constexpr int kLcThreads = 128;
template <int NB, bool FP4>
__global__ void __launch_bounds__(kLcThreads) latent_combine_kernel(const LatentAttend p, const int cols) {
  __shared__ __align__(16) float sm[kLcThreads / 32], sl[kLcThreads / 32], sacc[kLcThreads / 32][S4R_MAX_LATENT_RANK], f_s[kLcThreads];
  __shared__ int first_bad[kLcThreads / 32];
  const int row = blockIdx.x % p.rows, b = blockIdx.x / p.rows, rb = row / NB;
  const int64_t at = (int64_t)b * p.rows + row;
  pdl_wait();
  const int unit = b * p.row_blocks + rb;
  int2 parts = p.units[unit];
  if (!la_parts_ok(parts.x, parts.y, p.n_groups, p.row_blocks)) parts.y = 1;   // a wait gave up, and the status says so
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int W = kLcThreads / 32, kCols = S4R_MAX_LATENT_RANK / 32;
  const int sees = la_length(p, b) - p.n_query + 1 + row / p.n_heads;
  int poison = INT32_MAX;
  if (p.n_query > 1) {
    for (int i = threadIdx.x; i < parts.y; i += kLcThreads) {
      const int2 x = parts.y == 1 ? p.unit_poison[unit] : p.part_poison[la_part_slot(parts.x, i, p.row_blocks)];
      poison = smin(poison, smin(x.x, x.y));
    }
    poison = __reduce_min_sync(0xffffffffu, poison);
    if (lane == 0) first_bad[warp] = poison;
    __syncthreads();
    poison = smin(smin(first_bad[0], first_bad[1]), smin(first_bad[2], first_bad[3]));
  }
  if (sees > poison) {
    if (blockIdx.y > 0) return;
    float m = -CUDART_INF_F, l = 0.0f, acc[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] = 0.0f;
    for (int i = warp; i < sees; i += W) {
      const int32_t page = p.block_table[(int64_t)b * p.max_pages + (i >> p.page_shift)];
      if (page < 0 || page >= p.n_pages) continue;   // reported by the main kernel
      const int32_t r = i & (p.page_size - 1);
      float z = 0.0f;
      for (int c = lane; c < p.width; c += 32) z = fmaf(to_f(p.q[at * p.width + c]), latent_value<FP4>(p, page, r, c), z);
      z = warp_sum(z) * p.scale;
      // logits of -infinity weigh nothing, also while there is no other one
      const float top = fmaxf(m, z);
      const float f = m == -CUDART_INF_F ? 0.0f : expf(m - top), e = expf(z - (top == -CUDART_INF_F ? 0.0f : top));
      l = l * f + e;
      m = top;
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        const int c = k * 32 + lane;
        if (c < p.rank) acc[k] = acc[k] * f + e * latent_value<FP4>(p, page, r, c);
      }
    }
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k) sacc[warp][k * 32 + lane] = acc[k];
    __syncthreads();
    float top = -CUDART_INF_F, sum = 0.0f, f[W];
    for (int w = 0; w < W; ++w) top = fmaxf(top, sm[w]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f[w] = sm[w] == -CUDART_INF_F ? 0.0f : expf(sm[w] - top);
      sum += f[w] * sl[w];   // a NaN in a warp's sum stays one
    }
    for (int c = threadIdx.x; c < p.rank; c += kLcThreads) {
      float o = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) o += f[w] * sacc[w][c];
      p.out[at * p.rank + c] = from_f<bf16>(sum == 0.0f ? 0.0f : o / sum);
    }
    if (p.lse && threadIdx.x == 0) p.lse[at] = top + logf(sum);   // no weight at all: -infinity
    return;
  }
  if (parts.y <= 1) return;
  // Statistics first, a thread a part; then the warps share out the parts, a
  // lane adding up 4 neighbouring columns of every 128.
  const int r = row - rb * NB;
  auto slot_of = [&](int i) { return (int64_t)la_part_slot(parts.x, i, p.row_blocks) * NB + r; };
  float top = -CUDART_INF_F;
  for (int i = threadIdx.x; i < parts.y; i += kLcThreads) top = fmaxf(top, p.ml[slot_of(i)].x);
  top = warp_max(top);
  if (lane == 0) sm[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) top = fmaxf(top, sm[w]);
  float sum = 0.0f;
  float4 o[S4R_MAX_LATENT_RANK / 128];
#pragma unroll
  for (int k = 0; k < S4R_MAX_LATENT_RANK / 128; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int col0 = blockIdx.y * cols + 4 * lane, col1 = smin((int)(blockIdx.y + 1) * cols, p.rank);
  for (int base = 0; base < parts.y; base += kLcThreads) {
    const int m = smin(parts.y - base, kLcThreads);
    float f = 0.0f, part_sum = 0.0f;
    if ((int)threadIdx.x < m) {
      const float2 ml = p.ml[slot_of(base + threadIdx.x)];
      // No part weighs less than the least positive value: what is not finite in
      // its sums is not in the row either.  (That also is the weight where no
      // part has a reference, exp2 of NaN.)
      f = fmaxf(exp2f(ml.x - top), __uint_as_float(1u));
      part_sum = f * ml.y;
    }
    part_sum = warp_sum(part_sum);
    __syncthreads();
    f_s[threadIdx.x] = f;
    if (lane == 0) sl[warp] = part_sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) sum += sl[w];
    // Eight loads under way at a time, without a condition between them: of
    // eight parts where there are many parts and few columns, else of two
    // parts with up to four columns each.
    auto batch = [&](int i0, auto parts_, auto ks_) {
      constexpr int N = decltype(parts_)::value, K = decltype(ks_)::value;
      float4 x[N][K];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float *src = p.part + slot_of(base + smin(i0 + n * W, m - 1)) * p.rank;
#pragma unroll
        for (int k = 0; k < K; ++k) x[n][k] = *reinterpret_cast<const float4 *>(src + smin(col0 + 128 * k, p.rank - 4));
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float w = i0 + n * W < m ? f_s[i0 + n * W] : 0.0f;
        if (w != 0.0f) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            o[k].x = fmaf(w, x[n][k].x, o[k].x);
            o[k].y = fmaf(w, x[n][k].y, o[k].y);
            o[k].z = fmaf(w, x[n][k].z, o[k].z);
            o[k].w = fmaf(w, x[n][k].w, o[k].w);
          }
        }
      }
    };
    using std::integral_constant;
    if (cols == 128)
      for (int i = warp; i < m; i += 8 * W) batch(i, integral_constant<int, 8>{}, integral_constant<int, 1>{});
    else
      for (int i = warp; i < m; i += 2 * W)
        batch(i, integral_constant<int, 2>{}, integral_constant<int, S4R_MAX_LATENT_RANK / 128>{});
  }
#pragma unroll
  for (int k = 0; k < S4R_MAX_LATENT_RANK / 128; ++k)
    *reinterpret_cast<float4 *>(&sacc[warp][128 * k + 4 * lane]) = o[k];
  __syncthreads();
  const bool none = top == -CUDART_INF_F && sum == 0.0f;
  const float f = none ? 0.0f : p.cache_scale / sum;
  const int at_col = 4 * threadIdx.x, col = blockIdx.y * cols + at_col;
  if (col < col1) {
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!none)
      for (int w = 0; w < W; ++w) {
        const float4 x = *reinterpret_cast<const float4 *>(&sacc[w][at_col]);
        t.x += x.x;
        t.y += x.y;
        t.z += x.z;
        t.w += x.w;
      }
    *reinterpret_cast<uint2 *>(p.out + at * p.rank + col) = make_uint2(pack_bf16(t.x * f, t.y * f), pack_bf16(t.z * f, t.w * f));
  }
  if (p.lse && threadIdx.x == 0 && blockIdx.y == 0)
    p.lse[at] = none ? -CUDART_INF_F : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace s4r
