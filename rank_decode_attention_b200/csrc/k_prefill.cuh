// k_prefill.cuh -- attention of ragged prompts over expanded keys and values.
//
// S = scale (q . k + q_rope . k_rope), P = softmax(S) with a causal limit a
// row, O = P V: bound by the tensor cores (320 multiply-adds a query, key and
// head at 128 + 64 | 128, and one exponential).
//
// A CTA takes 256 queries of one head as two tiles of 128 and walks along the
// keys in tiles of 128.  While the softmax of one query tile runs, the tensor
// cores work for the other one.  TMEM holds S and O of both tiles (4 x 128
// columns); P, in bf16, replaces the S it comes from and is the first operand
// of the second product straight from TMEM, so shared memory holds queries,
// keys and values only.
//   warp 0     loads with TMA: the queries once, then K and V in 128 x 64
//              chunks through a ring;
//   warp 1     issues tcgen05.mma;
//   warps 2-9  softmax, a thread a query: the reference maximum moves only when
//              a logit exceeds it by more than 2^8 (then the thread rescales its
//              row of O), so no thread waits for another one.
//   warps 10, 11  look after chunks of V that not every query may see whole: they
//              clear the rows behind the end of the sequence, and infinities
//              and NaN in rows on the diagonal (a probability of 0 would not
//              hide them from the rows that must not see them); rows that do see
//              one are computed again one by one at the end.
// CTAs start with the queries that see most keys, all heads of them, so that
// the short ones fill up the end.  Every wait is bounded (umma.cuh); after one
// that gave up every role runs out, the producer and the issuer when what they
// issued has ended.
//
// Measured through the binding, inputs changing: one prompt of 8192, 16 heads,
// 128 + 64 | 128: 360 us, 0.95 PFLOP/s (303 us before the power cap settles); six
// prompts of 33 to 2900 behind a prefix of 517, 32 over 8 heads, 128 | 128: 400
// us, 0.59 PFLOP/s (385 before).  A step of 256 queries x 128 keys takes some 4400 cycles,
// of which the products need 2600, the exponentials of both tiles 2048 of the
// special-function unit, and about 900 are waits for K and V (a ring of 8 chunks
// beside 96 KB of queries).  Exponentials by polynomial on the multiply-add
// units were slower at every share tried (1/8: +1%, 1/4: +6%, 1/2: +11%), and so
// were heads in groups of 8, 4 and 2 for the sake of L2 (0 to +20%).
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

constexpr int kPfTile = 128;                     // queries a tile, keys a tile
constexpr int kPfChunk = kPfTile * 128;          // bytes of 128 rows x 64 columns
constexpr int kPfThreads = 384;
constexpr int kPfMaxSlots = 12;
constexpr int kPfControlBytes = 1024;
constexpr float kPfLift = 8.0f;

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

// Chunks of a key (and query) row, of a value row, and ring slots that fit.
__host__ __device__ inline int pf_key_chunks(int dim, int rope) { return (dim + 63) / 64 + (rope + 63) / 64; }
__host__ __device__ constexpr int pf_slots(int key_chunks) {
  return (227 * 1024 - 1024 - kPfControlBytes - 2 * key_chunks * kPfChunk) / kPfChunk < kPfMaxSlots
             ? (227 * 1024 - 1024 - kPfControlBytes - 2 * key_chunks * kPfChunk) / kPfChunk
             : kPfMaxSlots;
}
__host__ inline size_t pf_smem_bytes(int key_chunks) {
  return (size_t)(2 * key_chunks + pf_slots(key_chunks)) * kPfChunk + kPfControlBytes + 1024;
}

struct PfControl {
  uint64_t full[kPfMaxSlots], empty[kPfMaxSlots];
  uint64_t landed[kPfMaxSlots];   // a chunk of V that is looked after first
  uint64_t q_full, drained;
  uint64_t never;                 // no one arrives (s4r_debug_waits)
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint32_t tmem_base;
  int poison;   // first key whose values some rows must not see
};
static_assert(sizeof(PfControl) <= kPfControlBytes, "control block");

struct PfRing {
  int st = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void step(int n) {
    if (++st == n) {
      st = 0;
      ++turn;
    }
  }
};

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16, under a predicate.
__device__ __forceinline__ void umma_f16_ts_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(on)
      : "memory");
}

// One query row by one warp, keys one after another: the rows of a CTA that
// met infinities where only some of its rows may see them.
__device__ __noinline__ void prefill_row(const PrefillAttend &p, const PrefillSeq &s, int i, int h) {
  const int lane = threadIdx.x & 31;
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
    // logits of -infinity weigh nothing, also while there is no other one
    const float f = m == -CUDART_INF_F ? 0.0f : expf(m - top);
    const float e = expf(z - (top == -CUDART_INF_F ? 0.0f : top));
    l = l * f + e;
    m = top;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < p.vdim) acc[c] = acc[c] * f + e * to_f(p.v[row * p.v_ts + (int64_t)g * p.vdim + lane + 32 * c]);
  }
  bf16 *o = p.out + ((s.q0 + i) * p.hq + h) * (int64_t)p.vdim;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.vdim) o[lane + 32 * c] = from_f<bf16>(l == 0.0f ? 0.0f : acc[c] / l);
  if (lane == 0 && p.lse) p.lse[(s.q0 + i) * p.hq + h] = m + logf(l);   // no weight at all: -infinity
}

// KC, VC: 64-column chunks of a key (rotary part included) and of a value; as
// constants, since the issuing warp is bound by the instructions around its
// products (one prompt of 8192 and 16 heads took 393 us with them as variables,
// 368 us as constants).
template <int KC, int VC>
__global__ void __launch_bounds__(kPfThreads, 1)
prefill_attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_qr,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_kr,
                      const __grid_constant__ CUtensorMap map_v, const PrefillAttend p) {
  extern __shared__ __align__(1024) unsigned char pf_smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(pf_smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kc = KC, vc = VC, n_slots = pf_slots(KC);
  const int nope = (p.dim + 63) / 64;
  unsigned char *ring = smem + 2 * kc * kPfChunk;
  PfControl *ctl = reinterpret_cast<PfControl *>(ring + n_slots * kPfChunk);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int h = blockIdx.x, b = blockIdx.y, q0 = (int)(gridDim.z - 1 - blockIdx.z) * 2 * kPfTile;
  const int g = h / (p.hq / p.hkv);
  PrefillSeq s;
  if (!prefill_seq(p, b, s)) {   // the same in every thread
    if (threadIdx.x == 0) set_status(&g_device_status, kDevStatusCheck);
    return;
  }
  if (s.nq > p.max_q && threadIdx.x == 0) set_status(&g_device_status, kDevStatusCheck);
  const int rows = smin(s.nq, p.max_q);   // rows to compute
  if (q0 >= rows) return;
  // Key tiles of each query tile: up to what its last row sees.
  int n_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = smin(q0 + (t + 1) * kPfTile, rows) - 1;
    const int64_t sees = last < q0 + t * kPfTile ? 0 : p.causal ? smin<int64_t>((int64_t)s.nk - s.nq + last + 1, s.nk) : s.nk;
    // broadcast, for the compiler to see that it is uniform
    n_t[t] = __shfl_sync(0xffffffffu, sees > 0 ? (int)((sees + kPfTile - 1) / kPfTile) : 0, 0);
  }
  const int n_all = smax(n_t[0], n_t[1]);
  const long long limit = wait_limit();
  const bool unreachable = wait_unreachable();

  if (threadIdx.x == 0) {
    for (int i = 0; i < n_slots; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
      mbar_init(&ctl->landed[i], 1);
    }
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->drained, 1);
    mbar_init(&ctl->never, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ctl->s_full[t], 1);
      mbar_init(&ctl->p_full[t], 4);
      mbar_init(&ctl->pv_done[t], 1);
    }
    mbar_fence_init();
    ctl->poison = INT32_MAX;
  }
  if (warp == 0) tmem_alloc(&ctl->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return __shfl_sync(0xffffffffu, (int)mbar_wait_within(bar, parity & 1, limit, nullptr), 0) != 0;
  };

  // Rows of V in key tile j that exist and that every query of the CTA sees.
  auto live_rows = [&](int j) { return smin(s.nk - j * kPfTile, kPfTile); };
  auto common_rows = [&](int j) {
    const int64_t n = p.causal ? (int64_t)s.nk - s.nq + q0 + 1 - (int64_t)j * kPfTile : kPfTile;
    return (int)smax<int64_t>(0, smin<int64_t>(n, kPfTile));
  };
  auto touched = [&](int j) { return __shfl_sync(0xffffffffu, (int)(smin(live_rows(j), common_rows(j)) < kPfTile), 0) != 0; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t leader = elect_one();
    bool ok = n_all > 0;
    PfRing slot;
    // by slot: whether its last copy arrives on `landed`, and how many did, modulo 2
    uint32_t on_landed = 0, landed = 0;
    if (ok) {
      mbar_expect_if(leader, &ctl->q_full, (uint32_t)(2 * kc) * kPfChunk);
      for (int t = 0; t < 2; ++t)
        for (int c = 0; c < kc; ++c) {
          const int row = (int)s.q0 + q0 + t * kPfTile;
          unsigned char *dst = smem + (t * kc + c) * kPfChunk;
          if (c < nope) tma_load_3d_if(leader, dst, &map_q, &ctl->q_full, c * 64, h, row);
          else tma_load_3d_if(leader, dst, &map_qr, &ctl->q_full, (c - nope) * 64, h, row);
        }
    }
    for (int j = 0; j < n_all && ok; ++j) {
      const int row = (int)s.k0 + j * kPfTile;
      for (int c = 0; c < kc && ok; ++c, slot.step(n_slots)) {
        if (slot.turn > 0) ok = wait(&ctl->empty[slot.st], slot.turn - 1);
        if (!ok) break;
        on_landed &= ~(1u << slot.st);
        mbar_expect_if(leader, &ctl->full[slot.st], kPfChunk);
        if (c < nope) tma_load_3d_if(leader, ring + slot.st * kPfChunk, &map_k, &ctl->full[slot.st], c * 64, g, row);
        else tma_load_3d_if(leader, ring + slot.st * kPfChunk, &map_kr, &ctl->full[slot.st], (c - nope) * 64, 0, row);
      }
      if (ok && vc == 2 && slot.st == n_slots - 1) {   // the two chunks of V lie side by side: skip the last slot
        if (slot.turn > 0) ok = wait(&ctl->empty[slot.st], slot.turn - 1);
        if (!ok) break;
        on_landed &= ~(1u << slot.st);
        if (leader) mbar_arrive(&ctl->full[slot.st]);
        slot.step(n_slots);
      }
      const bool touch = touched(j);
      for (int c = 0; c < vc && ok; ++c, slot.step(n_slots)) {
        if (slot.turn > 0) ok = wait(&ctl->empty[slot.st], slot.turn - 1);
        if (!ok) break;
        uint64_t *bar = touch ? &ctl->landed[slot.st] : &ctl->full[slot.st];
        on_landed = (on_landed & ~(1u << slot.st)) | ((uint32_t)touch << slot.st);
        landed ^= (uint32_t)touch << slot.st;
        mbar_expect_if(leader, bar, kPfChunk);
        tma_load_3d_if(leader, ring + slot.st * kPfChunk, &map_v, bar, c * 64, g, row);
      }
    }
    // Shared memory goes with the CTA: let the copies in flight land, whichever
    // role gave up.
    auto land = [&](uint64_t *bar, uint32_t parity) { mbar_wait_within(bar, parity & 1, kWaitCycles, nullptr); };
    if (n_all > 0) {
      land(&ctl->q_full, 0);
      for (int i = 0; i < n_slots; ++i) {
        if (on_landed >> i & 1) land(&ctl->landed[i], (landed >> i) + 1);
        else if (slot.turn > 0 || i < slot.st) land(&ctl->full[i], slot.turn - (i < slot.st ? 0 : 1));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t leader = elect_one();
    const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0), id_o = idesc_bf16_f32(128, 64 * vc, 0, 1);
    const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 16, 1024), k_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(ring), kPfChunk, 1024);
    bool ok = true;   // after a wait that gave up nothing more is issued: a slot whose copy is under way must not be released
    uint64_t *const p_full = unreachable ? &ctl->never : ctl->p_full;   // then of tile 0 alone
    auto until = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = wait(bar, parity);
      tc_fence_after();
    };
    PfRing kp, vp;   // first slots of the key tile and of the value tile in turn
    // S of query tile t and the key tile at kp; the slots are free after the last query tile
    auto scores = [&](int t, bool first, bool last) {
      PfRing at = kp;
      const uint32_t d = tmem + t * 128;
      for (int c = 0; c < kc; ++c, at.step(n_slots)) {
        if (first) until(&ctl->full[at.st], at.turn);
        if (!ok) return;
        const uint64_t a = q_desc + (uint32_t)(t * kc + c) * (kPfChunk >> 4), k = k_desc + (uint32_t)at.st * (kPfChunk >> 4);
        umma_f16_if(leader, d, a, k, id_s, c > 0);
#pragma unroll
        for (int ks = 1; ks < 4; ++ks) umma_f16_if(leader, d, a + ks * 2, k + ks * 2, id_s, true);
        if (last) umma_commit_if(leader, &ctl->empty[at.st]);
      }
      umma_commit_if(leader, &ctl->s_full[t]);
    };
    auto values = [&](int t, int j, bool first, bool last) {
      until(p_full + (unreachable ? 0 : t), (uint32_t)j);
      if (first)
        for (int c = 0; c < vc; ++c) until(&ctl->full[vp.st + c], vp.turn);
      if (!ok) return;
      const uint64_t v = v_desc + (uint32_t)vp.st * (kPfChunk >> 4);
      const uint32_t d = tmem + 256 + t * 128, a = tmem + t * 128;
      umma_f16_ts_if(leader, d, a, v, id_o, j > 0);
#pragma unroll
      for (int ks = 1; ks < kPfTile / 16; ++ks) umma_f16_ts_if(leader, d, a + ks * 8, v + ks * (2048 >> 4), id_o, true);
      if (last)
        for (int c = 0; c < vc; ++c) umma_commit_if(leader, &ctl->empty[vp.st + c]);
      umma_commit_if(leader, &ctl->pv_done[t]);
    };
    // One copy of each product's code for both tiles: what the issuing warp
    // runs has to stay in the instruction cache beside the softmax.
    const int n0 = n_t[0], n1 = n_t[1];
    if (n_all > 0) until(&ctl->q_full, 0);
#pragma unroll 1
    for (int j = -1; j < n_all && ok; ++j) {
      if (j >= 0) {
        // the value tile lies behind the key tile at kp, the next key tile behind that
        vp = kp;
        for (int c = 0; c < kc; ++c) vp.step(n_slots);
        if (vc == 2 && vp.st == n_slots - 1) {
          until(&ctl->full[vp.st], vp.turn);
          if (!ok) break;
          umma_commit_if(leader, &ctl->empty[vp.st]);
          vp.step(n_slots);
        }
        kp = vp;
        for (int c = 0; c < vc; ++c) kp.step(n_slots);
      }
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int mine = t ? n1 : n0, other = t ? n0 : n1;
        // the first tile to use a slot waits for it, the last one releases it
        if (j >= 0 && j < mine) values(t, j, t == 0 || j >= other, t == 1 || j >= other);
        if (j + 1 < mine) scores(t, t == 0 || j + 1 >= other, t == 1 || j + 1 >= other);
      }
    }
    // TMEM and shared memory go with the CTA: let the products in flight end,
    // whichever role gave up.
    umma_commit_if(leader, &ctl->drained);
    mbar_wait_within(&ctl->drained, 0, kWaitCycles, nullptr);
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------------ chunks of V seen in part
    const int c = warp - 10;
    PfRing slot;
    uint32_t seen = 0;   // a slot's uses of this kind, modulo 2: the parity of its barrier
    bool ok = c < vc;
    for (int j = 0; j < n_all && ok; ++j) {
      for (int k = 0; k < kc; ++k) slot.step(n_slots);
      if (vc == 2 && slot.st == n_slots - 1) slot.step(n_slots);
      if (touched(j)) {
        const int at = slot.st + c;
        ok = wait(&ctl->landed[at], seen >> at);
        if (!ok) break;
        seen ^= 1u << at;
        int bad = INT32_MAX;
        const int live = live_rows(j);
        uint4 *chunk = reinterpret_cast<uint4 *>(ring + at * kPfChunk);
#pragma unroll 8
        for (int i = common_rows(j) * 8 + lane; i < live * 8; i += 32) {
          uint4 v = chunk[i];
          if (clear_not_finite<0x7f80u>(v)) {
            chunk[i] = v;
            bad = smin(bad, j * kPfTile + (i >> 3));
          }
        }
        for (int i = live * 8 + lane; i < kPfTile * 8; i += 32) chunk[i] = make_uint4(0u, 0u, 0u, 0u);
        if (bad != INT32_MAX) atomicMin(&ctl->poison, bad);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[at]);
      }
      for (int k = 0; k < vc; ++k) slot.step(n_slots);
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int t = (warp - 2) >> 2, quad = warp & 3;
    const int i = q0 + t * kPfTile + quad * 32 + lane;   // the thread's query
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * 128;
    const int64_t last64 = p.causal ? smin<int64_t>((int64_t)s.nk - s.nq + i, s.nk - 1) : s.nk - 1;
    const int last = (int)smax<int64_t>(last64, -1);     // the last key it sees
    // A scale that is not positive is applied to the logits beforehand.
    const bool odd = !(p.scale > 0.0f);
    const float to2 = p.scale == 0.0f ? 1.0f : fabsf(p.scale) * 1.4426950408889634f, first = p.scale == 0.0f ? 0.0f : -1.0f;
    float m = -CUDART_INF_F, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n_t[t]; ++j) {
      ok = wait(&ctl->s_full[t], (uint32_t)j);
      if (!ok) break;
      tc_fence_after();
      const int left = last - j * kPfTile;   // columns up to this one are seen
      const bool cut = __any_sync(0xffffffffu, left < kPfTile - 1);
      auto fix = [&](uint32_t (&x)[32], int c0) {
        if (odd) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * first);
        }
        if (cut) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c > left) x[c] = 0xff800000u;
        }
      };
      uint32_t v0[32], v1[32];
      uint64_t sum[4] = {0u, 0u, 0u, 0u};   // pairs of fp32
      const uint64_t to2_2 = pair_f32(to2, to2);
      bool done = false;
      if constexpr (KC == 3) {
        // The usual tile, seen whole and after the first: once over the row,
        // the probabilities kept in registers until it is clear that no logit
        // exceeds the reference too far; else the way below, from the same S.
        // With keys of three chunks the softmax is what the products wait for,
        // and this saves 5% (8192 queries of 16 heads: 304 against 319 us);
        // with fewer chunks the exponentials of the two tiles meet at the
        // special-function unit, and it costs 5% (323 against 304 us).
        if (j > 0 && !cut && !odd && __all_sync(0xffffffffu, m > -CUDART_INF_F)) {
          uint32_t w[64];
          float above[2] = {-CUDART_INF_F, -CUDART_INF_F};
          const uint64_t ref_2 = pair_f32(-m, -m);
          auto part = [&](const uint32_t (&x)[32], uint32_t *to) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float a, e;
              unpair_f32(fma_f32x2(pair_f32(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), to2_2, ref_2), a, e);
              above[k & 1] = fmaxf(fmaxf(above[k & 1], a), e);
              a = ex2_approx(a);
              e = ex2_approx(e);
              sum[k & 1] = add_f32x2(sum[k & 1], pair_f32(a, e));
              to[k] = pack_bf16(a, e);
            }
          };
          tmem_ld32(s_at, v0);
          tmem_wait_ld();
          tmem_ld32(s_at + 32, v1);
          part(v0, w);
          tmem_wait_ld();
          tmem_ld32(s_at + 64, v0);
          part(v1, w + 16);
          tmem_wait_ld();
          tmem_ld32(s_at + 96, v1);
          part(v0, w + 32);
          tmem_wait_ld();
          part(v1, w + 48);
          if (__any_sync(0xffffffffu, fmaxf(above[0], above[1]) > kPfLift)) {
            sum[0] = sum[1] = 0u;
          } else {
            tmem_st32(s_at, reinterpret_cast<uint32_t(&)[32]>(w[0]));
            tmem_st32(s_at + 32, reinterpret_cast<uint32_t(&)[32]>(w[32]));
            done = true;
          }
        }
      }
      if (!done) {
        // Twice over the row, 64 columns at a time in a loop: once for the
        // maximum, once for the probabilities (P overwrites only what has been
        // read).  Unrolled over all 128 columns both times the code falls out
        // of the instruction cache, and the issuing warp waits for its own.
        float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
        tmem_ld32(s_at, v0);
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          tmem_wait_ld();
          tmem_ld32(s_at + c + 32, v1);
          fix(v0, c);
#pragma unroll
          for (int k = 0; k < 32; k += 2) top[(k >> 1) & 3] = fmaxf(fmaxf(top[(k >> 1) & 3], __uint_as_float(v0[k])), __uint_as_float(v0[k + 1]));
          tmem_wait_ld();
          tmem_ld32(s_at + ((c + 64) & 127), v0);   // at the end the first columns, for the second time
          fix(v1, c + 32);
#pragma unroll
          for (int k = 0; k < 32; k += 2) top[(k >> 1) & 3] = fmaxf(fmaxf(top[(k >> 1) & 3], __uint_as_float(v1[k])), __uint_as_float(v1[k + 1]));
        }
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float y = most * to2;
        if (__any_sync(0xffffffffu, y > m + kPfLift)) {
          const float mn = fmaxf(m, y), f = mn == m ? 1.0f : exp2f(m - mn);
          m = mn;
          l *= f;
          if (j > 0) {
            ok = wait(&ctl->pv_done[t], (uint32_t)(j - 1));
            if (!ok) break;
            tc_fence_after();
            tmem_wait_ld();
#pragma unroll 1
            for (int c = 0; c < 64 * vc; c += 32) {
              tmem_ld32(o_at + c, v1);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) v1[k] = __float_as_uint(__uint_as_float(v1[k]) * f);
              tmem_st32(o_at + c, v1);
            }
          }
        }
        const float ref = m == -CUDART_INF_F ? 0.0f : m;
        const uint64_t ref_2 = pair_f32(-ref, -ref);
        auto exps = [&](const uint32_t (&x)[32], int c) {   // P of columns c .. c + 31
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a, e;
            unpair_f32(fma_f32x2(pair_f32(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), to2_2, ref_2), a, e);
            a = ex2_approx(a);
            e = ex2_approx(e);
            sum[k & 3] = add_f32x2(sum[k & 3], pair_f32(a, e));
            w[k] = pack_bf16(a, e);
          }
          tmem_st16(s_at + c / 2, w);
        };
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          tmem_wait_ld();
          tmem_ld32(s_at + c + 32, v1);
          fix(v0, c);
          exps(v0, c);
          tmem_wait_ld();
          if (c == 0) tmem_ld32(s_at + 64, v0);
          fix(v1, c + 32);
          exps(v1, c + 32);
        }
      }
      {
        float a, e;
        unpair_f32(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), a, e);
        l += a + e;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[t]);
    }
    tmem_wait_ld();   // a wait that gave up may have left a load under way
    if (ok && n_t[t] > 0) ok = wait(&ctl->pv_done[t], (uint32_t)(n_t[t] - 1));
    tc_fence_after();
    if (ok) {
      const int64_t at = (s.q0 + i) * p.hq + h;
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;   // a row that sees no key: 0
      bf16 *o = p.out + at * p.vdim;
      for (int c = 0; c < 64 * vc; c += 32) {
        uint32_t w[32];
        if (n_t[t] > 0) {
          tmem_ld32(o_at + c, w);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) w[k] = 0u;
        }
        if (i < rows) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + 8 * k < p.vdim) {
              uint32_t r[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                r[x] = inv == 0.0f ? 0u : pack_bf16(__uint_as_float(w[8 * k + 2 * x]) * inv, __uint_as_float(w[8 * k + 2 * x + 1]) * inv);
              *reinterpret_cast<uint4 *>(o + c + 8 * k) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        __syncwarp();
      }
      if (i < rows && p.lse) p.lse[at] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
  // Rows that see an infinity which others must not see are written once more:
  // behind the barrier, which orders both writes and the note of the first key.
  const int poison = ctl->poison;
  if (poison != INT32_MAX)
    for (int r = warp; r < 2 * kPfTile; r += kPfThreads / 32)
      if (q0 + r < rows && (int64_t)s.nk - s.nq + q0 + r >= poison) prefill_row(p, s, q0 + r, h);
}

}  // namespace s4r
