// api_latent.cuh -- entry points of the paged latent cache and of prefill
// attention: argument checks and launches (included by s4r_api.cu, whose
// helpers it uses).
#pragma once

namespace {

inline bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
inline int log2_of(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}
// A grid of `want` CTAs, within what a launch takes.
inline unsigned grid_of(int64_t want, int64_t most) { return (unsigned)smax<int64_t>(1, smin<int64_t>(want, most)); }

// Launch a kernel whose set-up may overlap the end of the kernel before it (it
// calls pdl_wait before it touches global memory).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int block, size_t smem, cudaStream_t st, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

s4r_status page_size_ok(int32_t page_size) {
  if (page_size <= 0) return S4R_ERR_INVALID_ARG;
  return pow2(page_size) && page_size >= 16 && page_size <= S4R_MAX_PAGE_SIZE ? S4R_OK : S4R_ERR_UNSUPPORTED;
}

// Shape of a latent cache: type, width, page size, page count.
s4r_status cache_shape_ok(s4r_dtype dt, int32_t width, int32_t page_size, int64_t n_pages, float cache_scale) {
  if (dt != S4R_F32 && dt != S4R_BF16 && dt != S4R_FP4) return S4R_ERR_INVALID_ARG;
  if (width <= 0 || n_pages < 0) return S4R_ERR_INVALID_ARG;
  const s4r_status rc = page_size_ok(page_size);
  if (rc != S4R_OK) return rc;
  if (dt == S4R_F32 || width > S4R_MAX_LATENT_WIDTH || width % (dt == S4R_FP4 ? 32 : 8) || n_pages > INT32_MAX)
    return S4R_ERR_UNSUPPORTED;
  if (dt == S4R_FP4 && !(cache_scale > 0.0f && cache_scale <= 3.4e38f)) return S4R_ERR_INVALID_ARG;
  return S4R_OK;
}

s4r_status latent_attend_shape(const s4r_latent_attend_args *a) {
  if (!a) return S4R_ERR_INVALID_ARG;
  const s4r_status rc = cache_shape_ok(a->cache_dtype, a->width, a->page_size, a->n_pages, a->cache_scale);
  if (rc != S4R_OK) return rc;
  if (a->batch < 0 || a->n_query <= 0 || a->n_heads <= 0 || a->rank <= 0 || a->rank > a->width || a->max_pages <= 0 ||
      !std::isfinite(a->scale))
    return S4R_ERR_INVALID_ARG;
  if (a->rank % 8 || a->rank > S4R_MAX_LATENT_RANK || a->batch > S4R_MAX_REQUESTS ||
      (int64_t)a->n_query * a->n_heads > INT32_MAX / S4R_MAX_LATENT_WIDTH ||
      (int64_t)a->n_query * a->n_heads * a->batch > INT32_MAX || (int64_t)a->n_query * a->n_heads > 65536 ||
      (int64_t)a->max_pages * a->page_size > INT32_MAX - kLaTile)
    return S4R_ERR_UNSUPPORTED;
  return S4R_OK;
}

// Blocks of query rows, grid and workspace of a latent attention call.
struct LatentPlan {
  int nb, row_blocks, n_groups;   // the grid: row_blocks CTAs for each of n_groups ranges of tiles
  size_t unit_poison, part_poison, units, ml, part, total;
};
LatentPlan latent_plan(const s4r_latent_attend_args *a) {
  LatentPlan l;
  const int64_t rows = (int64_t)a->n_query * a->n_heads;
  l.row_blocks = (int)ceil_div(rows, 64);
  l.nb = la_block_rows(rows);
  const int64_t tiles = (int64_t)a->batch * ceil_div((int64_t)a->max_pages * a->page_size, kLaTile);
  l.n_groups = (int)smax<int64_t>(1, smin<int64_t>(tiles, sm_count() / l.row_blocks));
  const size_t n_ctas = (size_t)l.n_groups * l.row_blocks;
  size_t off = kAlign;   // status word
  l.unit_poison = off;
  off += round_up(sizeof(int2) * (size_t)a->batch * l.row_blocks);
  l.part_poison = off;
  off += round_up(sizeof(int2) * 2 * n_ctas);
  l.units = off;
  off += round_up(sizeof(int2) * (size_t)a->batch * l.row_blocks);
  l.ml = off;
  off += round_up(sizeof(float2) * 2 * n_ctas * l.nb);
  l.part = off;
  off += round_up(sizeof(float) * 2 * n_ctas * l.nb * a->rank);
  l.total = off;
  return l;
}

// bf16 tensor map of up to three dimensions (innermost first), 128-byte swizzle.
bool make_tmap_bf16_nd(CUtensorMap *map, const void *ptr, int n, const uint64_t *dims, const uint64_t *stride_bytes,
                       const uint32_t *box) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], es[3] = {1, 1, 1};
  for (int i = 0; i < n; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i + 1 < n) st[i] = stride_bytes[i];
  }
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)n, const_cast<void *>(ptr), d, st, b, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NB, bool FP4>
s4r_status latent_attend_launch(const LatentAttend &p, cudaStream_t st) {
  CUtensorMap kv{}, q{};
  if (!FP4) {
    const uint64_t row = (uint64_t)p.width * 2;
    const uint64_t kd[3] = {(uint64_t)p.width, (uint64_t)p.page_size, (uint64_t)p.n_pages};
    const uint64_t ks[2] = {row, row * p.page_size};
    const uint32_t kb[3] = {64, (uint32_t)smin(p.page_size, kLaTile), 1};
    const uint64_t qd[2] = {(uint64_t)p.width, (uint64_t)p.batch * p.rows};
    const uint32_t qb[2] = {64, (uint32_t)NB};
    if (!make_tmap_bf16_nd(&kv, p.cache, 3, kd, ks, kb) || !make_tmap_bf16_nd(&q, p.q, 2, qd, &row, qb)) {
      snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed for the latent cache or the queries");
      return S4R_ERR_CUDA;
    }
  }
  const size_t smem = (size_t)la_layout(NB, p.width, FP4).total;
  cudaError_t err = ensure_smem<latent_attend_kernel<NB, FP4>>(smem);
  if (err != cudaSuccess) return fail("latent_attend_kernel (shared memory)", err);
  err = launch_after(latent_attend_kernel<NB, FP4>, (unsigned)(p.n_groups * p.row_blocks), la_threads(FP4), smem, st, kv, q, p);
  if (err != cudaSuccess) return fail("latent_attend_kernel", err);
  cudaLaunchConfig_t cfg = {};
  // Few rows with many parts each: their columns go to CTAs of their own (16
  // rows of 128 parts: the whole call 15.6 us against 18.9; 256 rows: the same;
  // 512 rows 29.3 against 25.2, so there a CTA takes a whole row).
  const int64_t out_rows = (int64_t)p.batch * p.rows;
  const int cols = out_rows < 2 * sm_count() ? 128 : (int)ceil_div(p.rank, 128) * 128;
  cfg.gridDim = dim3((unsigned)out_rows, (unsigned)ceil_div(p.rank, cols));
  cfg.blockDim = dim3(kLcThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, latent_combine_kernel<NB, FP4>, p, cols);
  return err == cudaSuccess ? S4R_OK : fail("latent_combine_kernel", err);
}

// Column tiles of a projection with NT columns a tile, and what the longest
// CTA then computes.
struct LpTiles {
  int32_t n_tiles;
  int64_t cost;
};
template <int NT>
LpTiles lp_tiles(const LatentProject &p) {
  constexpr int kGroups = NT / 64;
  LpTiles t;
  t.n_tiles = (int32_t)(p.shared_x ? ceil_div((int64_t)p.n_heads * p.head_groups, kGroups)
                                   : p.n_heads * ceil_div(p.head_groups, kGroups));
  const int widest = smin(kGroups, p.shared_x ? p.n_heads * p.head_groups : p.head_groups);
  t.cost = ceil_div((int64_t)t.n_tiles * p.m_tiles, sm_count()) * (widest + 1);   // a tile's start and end count as a group
  return t;
}

template <int NT>
s4r_status latent_project_launch(const CUtensorMap &mx, const CUtensorMap &mb, const CUtensorMap &mo, LatentProject p,
                                 int32_t n_tiles, cudaStream_t st) {
  p.n_tiles = n_tiles;
  const cudaError_t err = ensure_smem<latent_project_kernel<NT>>(kLpSmem);
  if (err != cudaSuccess) return fail("latent_project_kernel (shared memory)", err);
  const unsigned grid = grid_of((int64_t)n_tiles * p.m_tiles, sm_count());
  const cudaError_t rc = launch_after(latent_project_kernel<NT>, grid, kLpThreads, kLpSmem, st, mx, mb, mo, p);
  return rc == cudaSuccess ? S4R_OK : fail("latent_project_kernel", rc);
}

template <int KC, int VC>
s4r_status prefill_launch(const CUtensorMap &mq, const CUtensorMap &mqr, const CUtensorMap &mk, const CUtensorMap &mkr,
                          const CUtensorMap &mv, const PrefillAttend &p, cudaStream_t st) {
  const size_t smem = pf_smem_bytes(KC);
  const cudaError_t err = ensure_smem<prefill_attend_kernel<KC, VC>>(smem);
  if (err != cudaSuccess) return fail("prefill_attend_kernel (shared memory)", err);
  // at least one block a sequence, which reports what max_q leaves out
  const dim3 grid((unsigned)p.hq, (unsigned)p.batch, grid_of(ceil_div(p.max_q, 2 * kPfTile), 65535));
  prefill_attend_kernel<KC, VC><<<grid, kPfThreads, smem, st>>>(mq, mqr, mk, mkr, mv, p);
  return check_launch("prefill_attend_kernel");
}

}  // namespace

extern "C" {

s4r_status s4r_page_plan(const s4r_page_plan_args *a, void *stream) {
  if (!a) return S4R_ERR_INVALID_ARG;
  if (a->batch < 0 || a->max_pages <= 0 || a->free_capacity < 0 || a->max_tokens < 0) return S4R_ERR_INVALID_ARG;
  const s4r_status rc = page_size_ok(a->page_size);
  if (rc != S4R_OK) return rc;
  if (a->batch > S4R_MAX_REQUESTS || a->max_tokens > INT32_MAX || (int64_t)a->max_pages * a->page_size > INT32_MAX)
    return S4R_ERR_UNSUPPORTED;
  const void *must[] = {a->free_count, a->free_count_out, a->cu_tokens};
  for (const void *p : must)
    if (!p || !aligned16(p)) return S4R_ERR_INVALID_ARG;
  const void *per_request[] = {a->lengths, a->new_tokens, a->block_table, a->lengths_out};
  for (const void *p : per_request)
    if ((a->batch > 0 && !p) || !aligned16(p)) return S4R_ERR_INVALID_ARG;
  if ((a->free_capacity > 0 && !a->free_pages) || !aligned16(a->free_pages)) return S4R_ERR_INVALID_ARG;
  if ((a->max_tokens > 0 && !a->slots) || !aligned16(a->slots)) return S4R_ERR_INVALID_ARG;
  const void *optional[] = {a->positions, a->requests, a->status_workspace};
  for (const void *p : optional)
    if (!aligned16(p)) return S4R_ERR_INVALID_ARG;
  PagePlan p{a->batch, a->page_size, log2_of(a->page_size), a->max_pages, a->free_capacity, a->max_tokens,
             a->lengths, a->new_tokens, a->free_pages, a->free_count, a->block_table, a->lengths_out,
             a->free_count_out, a->cu_tokens, a->slots, a->positions, a->requests,
             static_cast<uint32_t *>(a->status_workspace)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t smem = plan_smem_bytes(a->batch);
  if (ensure_smem<page_plan_kernel>(smem) != cudaSuccess || ensure_smem<page_commit_kernel>(smem) != cudaSuccess)
    return fail("page_plan_kernel (shared memory)", cudaGetLastError());
  const unsigned grid = grid_of(ceil_div(a->max_tokens, kPlanTokensPerCta), sm_count());
  page_plan_kernel<<<grid, kPlanThreads, smem, st>>>(p);
  if (grid > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, page_commit_kernel, p);
    if (err != cudaSuccess) return fail("page_commit_kernel", err);
  }
  return check_launch("page_plan_kernel");
}

s4r_status s4r_latent_write(const s4r_latent_write_args *a, void *stream) {
  if (!a) return S4R_ERR_INVALID_ARG;
  const s4r_status rc = cache_shape_ok(a->cache_dtype, a->width, a->page_size, a->n_pages, a->cache_scale);
  if (rc != S4R_OK) return rc;
  if (a->n_tokens < 0 || a->latents_ld < a->width) return S4R_ERR_INVALID_ARG;
  if (a->n_tokens > INT32_MAX) return S4R_ERR_UNSUPPORTED;
  if (a->n_tokens == 0) return S4R_OK;
  if (!a->latents || !a->slots || (a->n_pages > 0 && !a->cache)) return S4R_ERR_INVALID_ARG;
  const void *all[] = {a->latents, a->slots, a->cache, a->stored, a->status_workspace};
  for (const void *p : all)
    if (!aligned16(p)) return S4R_ERR_INVALID_ARG;
  if (a->latents_ld % 8 || (a->stored && a->cache_dtype != S4R_FP4)) return S4R_ERR_INVALID_ARG;
  LatentWrite p{a->n_tokens, a->n_pages * a->page_size, a->latents_ld, a->width, a->page_size, log2_of(a->page_size),
                a->cache_scale, static_cast<const bf16 *>(a->latents), a->slots, static_cast<unsigned char *>(a->cache),
                static_cast<bf16 *>(a->stored), static_cast<uint32_t *>(a->status_workspace)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)ceil_div(a->n_tokens, kWriteTokens);
  if (a->cache_dtype == S4R_BF16) latent_write_bf16<<<grid, kWriteThreads, 0, st>>>(p);
  else if (a->cache_scale == 1.0f) latent_write_fp4<true><<<grid, kWriteThreads, 0, st>>>(p);
  else latent_write_fp4<false><<<grid, kWriteThreads, 0, st>>>(p);
  return check_launch("latent_write");
}

size_t s4r_latent_attend_workspace_bytes(const s4r_latent_attend_args *a) {
  return latent_attend_shape(a) == S4R_OK ? latent_plan(a).total : 0;
}

s4r_status s4r_latent_attend(const s4r_latent_attend_args *a, void *stream) {
  const s4r_status rc = latent_attend_shape(a);
  if (rc != S4R_OK) return rc;
  if (a->batch == 0) return S4R_OK;
  const void *must[] = {a->q, a->block_table, a->lengths, a->out};
  for (const void *p : must)
    if (!p || !aligned16(p)) return S4R_ERR_INVALID_ARG;
  if (a->n_pages < 1 || !a->cache || !aligned16(a->cache) || !aligned16(a->lse)) return S4R_ERR_INVALID_ARG;
  const LatentPlan l = latent_plan(a);
  if (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < l.total) return S4R_ERR_WORKSPACE;
  const bool fp4 = a->cache_dtype == S4R_FP4;
  unsigned char *ws = static_cast<unsigned char *>(a->workspace);
  LatentAttend p{};
  p.batch = a->batch;
  p.n_query = a->n_query;
  p.n_heads = a->n_heads;
  p.width = a->width;
  p.rank = a->rank;
  p.page_size = a->page_size;
  p.page_shift = log2_of(a->page_size);
  p.max_pages = a->max_pages;
  p.n_pages = a->n_pages;
  p.scale = a->scale;
  p.cache_scale = fp4 ? a->cache_scale : 1.0f;
  p.q = static_cast<const bf16 *>(a->q);
  p.cache = static_cast<const unsigned char *>(a->cache);
  p.block_table = a->block_table;
  p.lengths = a->lengths;
  p.out = static_cast<bf16 *>(a->out);
  p.lse = a->lse;
  p.rows = a->n_query * a->n_heads;
  p.row_blocks = l.row_blocks;
  p.n_groups = l.n_groups;
  p.slots = la_layout(l.nb, a->width, fp4).slots;
  p.status = reinterpret_cast<uint32_t *>(ws);
  p.unit_poison = reinterpret_cast<int2 *>(ws + l.unit_poison);
  p.part_poison = reinterpret_cast<int2 *>(ws + l.part_poison);
  p.units = reinterpret_cast<int2 *>(ws + l.units);
  p.ml = reinterpret_cast<float2 *>(ws + l.ml);
  p.part = reinterpret_cast<float *>(ws + l.part);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fp4)
    return l.nb == 16   ? latent_attend_launch<16, true>(p, st)
           : l.nb == 32 ? latent_attend_launch<32, true>(p, st)
                        : latent_attend_launch<64, true>(p, st);
  return l.nb == 16   ? latent_attend_launch<16, false>(p, st)
         : l.nb == 32 ? latent_attend_launch<32, false>(p, st)
                      : latent_attend_launch<64, false>(p, st);
}

s4r_status s4r_latent_project(const s4r_latent_project_args *a, void *stream) {
  if (!a) return S4R_ERR_INVALID_ARG;
  if (a->n_tokens < 0 || a->n_heads <= 0 || a->head_dim <= 0 || a->rank <= 0) return S4R_ERR_INVALID_ARG;
  if (a->head_dim % 8 || a->rank % 8 || a->head_dim > S4R_MAX_HEAD_DIM || a->rank > S4R_MAX_LATENT_RANK ||
      a->n_tokens > INT32_MAX - 128 || a->n_heads > 65535)   // token coordinates of the last tile stay in 32 bits
    return S4R_ERR_UNSUPPORTED;
  if (a->n_tokens == 0) return S4R_OK;
  const int64_t n_in = a->to_latent ? a->head_dim : a->rank, n_out = a->to_latent ? a->rank : a->head_dim;
  if (!a->x || !a->basis || !a->out || !aligned16(a->x) || !aligned16(a->basis) || !aligned16(a->out))
    return S4R_ERR_INVALID_ARG;
  if (a->x_ts % 8 || a->x_hs % 8 || a->out_ts % 8 || a->out_hs % 8) return S4R_ERR_INVALID_ARG;
  // Either stride may be the outer one; an input may repeat its row for every
  // head, an output row may not touch another.
  auto apart = [&](int64_t ts, int64_t hs, int64_t n) {
    const bool one_t = a->n_tokens == 1, one_h = a->n_heads == 1;
    if ((!one_t && ts < n) || (!one_h && hs < n)) return false;
    if (one_t || one_h) return true;
    return ts >= hs * (a->n_heads - 1) + n || hs >= ts * (a->n_tokens - 1) + n;
  };
  if (a->x_ts < 0 || a->x_hs < 0 || a->out_ts < 0 || a->out_hs < 0) return S4R_ERR_INVALID_ARG;
  if ((a->n_tokens > 1 && a->x_ts < n_in) || (a->x_hs != 0 && a->x_hs < n_in) || !apart(a->out_ts, a->out_hs, n_out))
    return S4R_ERR_INVALID_ARG;
  const bool shared = a->x_hs == 0 && a->n_heads > 1;
  LatentProject p{};
  p.n_tokens = (int32_t)a->n_tokens;
  p.n_heads = a->n_heads;
  p.n_in = (int32_t)n_in;
  p.to_latent = a->to_latent ? 1 : 0;
  p.shared_x = shared ? 1 : 0;
  p.head_groups = (int32_t)ceil_div(n_out, 64);
  p.m_tiles = (int32_t)ceil_div(a->n_tokens, 128);
  // A dimension of one row needs no stride of the caller's.
  const uint64_t xs[2] = {shared || a->n_heads == 1 ? (uint64_t)n_in * 2 : (uint64_t)a->x_hs * 2,
                          a->n_tokens == 1 ? (uint64_t)n_in * 2 : (uint64_t)a->x_ts * 2};
  const uint64_t xd[3] = {(uint64_t)n_in, shared ? 1u : (uint64_t)a->n_heads, (uint64_t)a->n_tokens};
  const uint32_t xb[3] = {64, 1, 128};
  const uint64_t bs[2] = {(uint64_t)a->rank * 2, (uint64_t)a->rank * a->head_dim * 2};
  const uint64_t bd[3] = {(uint64_t)a->rank, (uint64_t)a->head_dim, (uint64_t)a->n_heads};
  const uint32_t bb[3] = {64, 64, 1};
  const uint64_t os[2] = {a->n_heads == 1 ? (uint64_t)n_out * 2 : (uint64_t)a->out_hs * 2,
                          a->n_tokens == 1 ? (uint64_t)n_out * 2 : (uint64_t)a->out_ts * 2};
  const uint64_t od[3] = {(uint64_t)n_out, (uint64_t)a->n_heads, (uint64_t)a->n_tokens};
  const uint32_t ob[3] = {64, 1, 32};
  CUtensorMap mx, mb, mo;
  if (!make_tmap_bf16_nd(&mx, a->x, 3, xd, xs, xb) || !make_tmap_bf16_nd(&mb, a->basis, 3, bd, bs, bb) ||
      !make_tmap_bf16_nd(&mo, a->out, 3, od, os, ob)) {
    snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed for s4r_latent_project");
    return S4R_ERR_CUDA;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const LpTiles t256 = lp_tiles<256>(p), t128 = lp_tiles<128>(p), t64 = lp_tiles<64>(p);
  // The widest tile unless a narrower one ends earlier (rounds of the grid x
  // column groups and one more): a call with few tokens has only its heads'
  // columns to spread.  Measured with 64 | 128 | 256 columns, 128 x 512 a head:
  // one token, 16 heads 4.1 | 4.5 | 5.0 us; 64 tokens, 128 heads 8.0 | 7.4 | 7.0;
  // 3000 tokens, 32 heads 33 | 26 | 25.
  if (t256.cost <= t128.cost && t256.cost <= t64.cost) return latent_project_launch<256>(mx, mb, mo, p, t256.n_tiles, st);
  if (t128.cost <= t64.cost) return latent_project_launch<128>(mx, mb, mo, p, t128.n_tiles, st);
  return latent_project_launch<64>(mx, mb, mo, p, t64.n_tiles, st);
}

s4r_status s4r_prefill_attend(const s4r_prefill_attend_args *a, void *stream) {
  if (!a) return S4R_ERR_INVALID_ARG;
  if (a->batch < 0 || a->n_heads_q <= 0 || a->n_heads_kv <= 0 || a->head_dim <= 0 || a->rope_dim < 0 ||
      a->value_dim <= 0 || a->max_q < 0 || a->total_q < 0 || a->total_k < 0 || !std::isfinite(a->scale) ||
      a->n_heads_q % a->n_heads_kv)
    return S4R_ERR_INVALID_ARG;
  if (a->head_dim % 8 || a->rope_dim % 8 || a->value_dim % 8 || a->head_dim > 128 || a->value_dim > 128 ||
      a->rope_dim > 64 || a->batch > 65535 || a->n_heads_q > 65535 || a->max_q > 65535 * 2 * kPfTile || a->total_q > INT32_MAX - 2 * kPfTile ||
      a->total_k > INT32_MAX - 2 * kPfTile)
    return S4R_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->total_q == 0) return S4R_OK;
  const void *must[] = {a->q, a->cu_q, a->cu_k, a->out};
  for (const void *p : must)
    if (!p || !aligned16(p)) return S4R_ERR_INVALID_ARG;
  const bool keys = a->total_k > 0;
  if ((keys && (!a->k || !a->v || (a->rope_dim > 0 && !a->k_rope))) || !aligned16(a->k) || !aligned16(a->v) ||
      !aligned16(a->k_rope) || !aligned16(a->lse))
    return S4R_ERR_INVALID_ARG;
  if (a->k_ts % 8 || a->v_ts % 8 || a->k_rope_ts % 8) return S4R_ERR_INVALID_ARG;
  if (keys && (a->k_ts < (int64_t)a->n_heads_kv * a->head_dim || a->v_ts < (int64_t)a->n_heads_kv * a->value_dim ||
               (a->rope_dim > 0 && a->k_rope_ts < a->rope_dim)))
    return S4R_ERR_INVALID_ARG;
  PrefillAttend p{a->batch, a->n_heads_q, a->n_heads_kv, a->head_dim, a->rope_dim, a->value_dim, a->causal, a->max_q,
                  a->total_q, a->total_k, a->scale, static_cast<const bf16 *>(a->q), static_cast<const bf16 *>(a->k),
                  static_cast<const bf16 *>(a->v), static_cast<const bf16 *>(a->k_rope), a->k_ts, a->v_ts, a->k_rope_ts,
                  a->cu_q, a->cu_k, static_cast<bf16 *>(a->out), a->lse};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int chunks = pf_key_chunks(a->head_dim, a->rope_dim);
  // Tensors without rows, or without a rotary part, are never loaded.
  const bf16 *k = keys ? p.k : p.q, *v = keys ? p.v : p.q, *kr = keys && a->rope_dim > 0 ? p.k_rope : p.q;
  const uint64_t nk = keys ? (uint64_t)a->total_k : 1, q_row = (uint64_t)(a->head_dim + a->rope_dim) * 2;
  auto map3 = [](CUtensorMap *m, const bf16 *ptr, int64_t n, int64_t heads, uint64_t rows, uint64_t head_bytes, uint64_t row_bytes) {
    const uint64_t d[3] = {(uint64_t)n, (uint64_t)heads, rows}, st[2] = {head_bytes, row_bytes};
    const uint32_t box[3] = {64, 1, kPfTile};
    return make_tmap_bf16_nd(m, ptr, 3, d, st, box);
  };
  CUtensorMap mq, mqr, mk, mkr, mv;
  const int64_t rd = a->rope_dim > 0 ? a->rope_dim : 8;
  if (!map3(&mq, p.q, a->head_dim, a->n_heads_q, a->total_q, q_row, q_row * a->n_heads_q) ||
      !map3(&mqr, a->rope_dim > 0 ? p.q + a->head_dim : p.q, rd, a->n_heads_q, a->total_q, q_row, q_row * a->n_heads_q) ||
      !map3(&mk, k, a->head_dim, keys ? a->n_heads_kv : 1, nk, (uint64_t)a->head_dim * 2, keys ? (uint64_t)a->k_ts * 2 : 16) ||
      !map3(&mkr, kr, rd, 1, keys && a->rope_dim > 0 ? nk : 1, 16, keys && a->rope_dim > 0 ? (uint64_t)a->k_rope_ts * 2 : 16) ||
      !map3(&mv, v, a->value_dim, keys ? a->n_heads_kv : 1, nk, (uint64_t)a->value_dim * 2, keys ? (uint64_t)a->v_ts * 2 : 16)) {
    snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed for s4r_prefill_attend");
    return S4R_ERR_CUDA;
  }
  const int vc = (int)ceil_div(a->value_dim, 64);
  auto launch = [&](auto kc_, auto vc_) { return prefill_launch<decltype(kc_)::value, decltype(vc_)::value>(mq, mqr, mk, mkr, mv, p, st); };
  using std::integral_constant;
  auto with_values = [&](auto kc_) {
    return vc == 1 ? launch(kc_, integral_constant<int, 1>{}) : launch(kc_, integral_constant<int, 2>{});
  };
  return chunks == 1   ? with_values(integral_constant<int, 1>{})
         : chunks == 2 ? with_values(integral_constant<int, 2>{})
                       : with_values(integral_constant<int, 3>{});
}

}  // extern "C"
