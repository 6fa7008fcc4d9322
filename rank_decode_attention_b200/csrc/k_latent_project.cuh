// k_latent_project.cuh -- per-head products between head space and latent
// space on the tensor cores: out[t][h] = x[t][h] . B_h (absorbing queries) or
// x[t][h] . B_h^T (expanding latents), bf16 in, fp32 sums, bf16 out.
//
// A GEMM for each head with the same small weights for all tokens.  Few tokens
// read the weights once (HBM-bound, 17 MB at 128 heads x 128 x 512); many
// tokens with one latent for all heads are one GEMM over all heads' columns,
// whose operands stay in L2 and whose output is most of the traffic.
//
// Persistent, tokens on M: a tile is 128 tokens x NT output columns in groups
// of 64 (of one head; of neighbouring heads when they share x).  Warp 0 loads
// 64-deep K-blocks with TMA into a ring, warp 1 issues tcgen05.mma (M = 128,
// N = NT) into one of two accumulators, warps 2-5 round a finished accumulator
// to bf16 into swizzled shared memory and store it with TMA (32 tokens x 64
// columns a copy; rows and columns outside the tensor are clipped), while the
// next tile is being multiplied.  Every wait is bounded (umma.cuh); after one
// that gave up every role runs out, the producer and the issuer when what they
// issued has ended.  The weights are K-major when latents are
// expanded and N-major when queries are absorbed; the descriptors say which.
//
// Measured: 64 tokens, 128 heads, 128 -> 512: 6.9 us on the device (3.9 TB/s);
// 8190 tokens with one latent for 32 heads, 512 -> 128: 39 us through the binding
// with inputs changing, 0.88 PFLOP/s (32.4 us in a graph over three input sets,
// 1.06), bound by the 384 KB of operands that a 128 x 256 tile takes from L2 (10
// to 12 TB/s together).
#pragma once
#include "umma.cuh"

namespace s4r {

struct LatentProject {
  int32_t n_tokens, n_heads, n_in, to_latent, shared_x;
  int32_t head_groups;    // 64-column groups of a head's output
  int32_t n_tiles;        // tiles of NT columns over all heads
  int32_t m_tiles;        // tiles of 128 tokens
};

constexpr int kLpThreads = 192;
constexpr int kLpRing = 192 * 1024;
constexpr int kLpStage = 4 * 2 * 32 * 128;   // per epilogue warp two 32 x 64 staging tiles
template <int NT> struct LpCfg {
  static constexpr int kStageBytes = 16384 + NT * 128;
  static constexpr int kStages = kLpRing / kStageBytes;
  static constexpr int kGroups = NT / 64;
};
constexpr int kLpSmem = kLpRing + kLpStage + 1024 + 512;

template <int NT>
__global__ void __launch_bounds__(kLpThreads, 1)
latent_project_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_o, const LatentProject p) {
  using C = LpCfg<NT>;
  extern __shared__ __align__(1024) unsigned char lp_smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(lp_smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *staging = smem + kLpRing;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + kLpStage);
  uint64_t *empty = full + C::kStages, *acc_full = empty + C::kStages, *acc_empty = acc_full + 2;
  uint64_t *drained = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const long long limit = wait_limit();
  const bool unreachable = wait_unreachable();
  const int nk = (p.n_in + 63) / 64;
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  const int head_tiles = (p.head_groups + C::kGroups - 1) / C::kGroups;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(drained, 1);
    mbar_fence_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_b);
    tma_prefetch_desc(&map_o);
  }
  if (warp == 0) tmem_alloc(tmem_slot, 2 * NT);
  pdl_wait();   // nothing before this touches memory that another kernel writes
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // Tile t: 128 tokens from m0, `n` column groups from group `g` of head `h` on.
  struct Tile {
    int m0, h, g, n;
  };
  auto tile_of = [&](int64_t t) {
    Tile r;
    const int mt = (int)(t / p.n_tiles), nt = (int)(t - (int64_t)mt * p.n_tiles);
    r.m0 = mt * 128;
    if (p.shared_x) {
      const int first = nt * C::kGroups;
      r.h = first / p.head_groups;
      r.g = first - r.h * p.head_groups;
      r.n = smin(C::kGroups, p.n_heads * p.head_groups - first);
    } else {
      r.h = nt / head_tiles;
      r.g = (nt - r.h * head_tiles) * C::kGroups;
      r.n = smin(C::kGroups, p.head_groups - r.g);
    }
    return r;
  };
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return __shfl_sync(0xffffffffu, (int)mbar_wait_within(bar, parity & 1, limit, nullptr), 0) != 0;
  };

  if (warp == 0) {
    const uint32_t leader = elect_one();
    bool ok = true;
    int st = 0;
    uint32_t turn = 0;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile r = tile_of(t);
      for (int kb = 0; kb < nk && ok; ++kb) {
        if (turn > 0) ok = wait(&empty[st], turn - 1);
        if (!ok) break;
        unsigned char *a = smem + st * C::kStageBytes;
        mbar_expect_if(leader, &full[st], 16384u + (uint32_t)r.n * 8192u);
        tma_load_3d_if(leader, a, &map_x, &full[st], kb * 64, p.shared_x ? 0 : r.h, r.m0);
        int h = r.h, g = r.g;
        for (int i = 0; i < r.n; ++i) {
          tma_load_3d_if(leader, a + 16384 + i * 8192, &map_b, &full[st], p.to_latent ? g * 64 : kb * 64,
                         p.to_latent ? kb * 64 : g * 64, h);
          if (++g == p.head_groups) {
            g = 0;
            ++h;
          }
        }
        if (++st == C::kStages) {
          st = 0;
          ++turn;
        }
      }
    }
    // Shared memory goes with the CTA: let the copies in flight land, whichever
    // role gave up.
    for (int i = 0; i < C::kStages; ++i)
      if (turn > 0 || i < st) mbar_wait_within(&full[i], (turn - (i < st ? 0 : 1)) & 1, kWaitCycles, nullptr);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t leader = elect_one();
    bool ok = true;
    int st = 0;
    uint32_t turn = 0, n = 0;
    const uint64_t a_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
    // N-major: 64-column groups 8 KB apart, a step of 16 rows is 2 KB; K-major:
    // rows of 128 bytes, a step of 16 columns is 32 bytes.
    const uint64_t b_desc = p.to_latent ? sdesc_sw128(smem_u32(smem) + 16384, 8192, 1024) : sdesc_sw128(smem_u32(smem) + 16384, 16, 1024);
    const uint32_t b_step = p.to_latent ? 2048 >> 4 : 2;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++n) {
      const Tile r = tile_of(t);
      const uint32_t acc = n & 1, id = idesc_bf16_f32(128, 64 * r.n, 0, p.to_latent ? 1 : 0), d = tmem + acc * NT;
      if (n >= 2) ok = wait(&acc_empty[acc], (n >> 1) - 1);
      for (int kb = 0; kb < nk && ok; ++kb) {
        ok = wait(&full[st], turn);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = a_desc + (uint32_t)st * (C::kStageBytes >> 4), b = b_desc + (uint32_t)st * (C::kStageBytes >> 4);
        umma_f16_if(leader, d, a, b, id, kb > 0);
#pragma unroll
        for (int ks = 1; ks < 4; ++ks) umma_f16_if(leader, d, a + ks * 2, b + ks * b_step, id, true);
        umma_commit_if(leader, &empty[st]);
        if (++st == C::kStages) {
          st = 0;
          ++turn;
        }
      }
      if (ok && !unreachable) umma_commit_if(leader, &acc_full[acc]);
    }
    // TMEM and shared memory go with the CTA: let the products in flight end,
    // whichever role gave up.
    umma_commit_if(leader, drained);
    mbar_wait_within(drained, 0, kWaitCycles, nullptr);
    __syncwarp();
  } else {
    const int quad = warp & 3;
    unsigned char *mine = staging + (warp - 2) * 2 * 4096;
    bool ok = true;
    uint32_t n = 0, copies = 0;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++n) {
      const Tile r = tile_of(t);
      const uint32_t acc = n & 1;
      ok = wait(&acc_full[acc], n >> 1);
      if (!ok) break;
      tc_fence_after();
      const int row0 = r.m0 + quad * 32;
      int h = r.h, g = r.g;
      for (int i = 0; i < r.n; ++i, ++copies) {
        unsigned char *buf = mine + (copies & 1) * 4096;
        if (lane == 0) bulk_wait_read<1>();   // the copy from this buffer two groups ago has read it
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[32];
          tmem_ld32(tmem + acc * NT + ((uint32_t)(quad * 32) << 16) + i * 64 + half * 32, v);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pack_bf16(__uint_as_float(v[8 * c + 2 * k]), __uint_as_float(v[8 * c + 2 * k + 1]));
            *reinterpret_cast<uint4 *>(buf + lane * 128 + (((half * 4 + c) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (row0 < p.n_tokens) tma_store_3d(&map_o, buf, g * 64, h, row0);
          bulk_commit();
        }
        if (++g == p.head_groups) {
          g = 0;
          ++h;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
    }
    if (lane == 0) bulk_wait_read<0>();   // shared memory goes with the CTA
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 2 * NT);
}

}  // namespace s4r
