/*
 * s4r.h -- C ABI of libs4r: S4R compressed-KV decode on NVIDIA B200 (sm_100a).
 *
 * The operations are those of "S^4R: Selective Sampling, Subspaces, and
 * Sparse Reconstruction for Compressed Long-Context KV Caching"
 * (arXiv 2608.00528), as its review page on pith.science states them:
 *   - every non-sink token is stored as rank-r coefficients c = s . B
 *     ("What carries the argument", Eq. 3);
 *   - a decode step projects a sliding window of queries into the key basis,
 *     scores every cached key coefficient in latent space with a softmax
 *     (major comment 2, §3.2.2, Eqs. 8-10), keeps the local window plus the
 *     top-k earlier positions (Eqs. 13-15), rebuilds only those rows from
 *     their coefficients and runs exact attention together with the
 *     uncompressed sink tokens (Eqs. 16-18).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers unless a comment says "host".
 *     Every device pointer must be 16-byte aligned.
 *   - The caller owns every buffer.  The library allocates no device memory,
 *     keeps no per-call state between calls and may be called from several
 *     host threads on different streams (each call with its own workspace).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls only enqueue work; none synchronises, except
 *     s4r_read_device_status.
 *   - The kernels of consecutive decode calls on one stream overlap their
 *     start-up (programmatic dependent launch): a call's first kernel may
 *     begin, and read the call's inputs (queries, coefficient caches, bases,
 *     sinks, lengths), while the previous decode call's last kernel is still
 *     running; it touches the workspace and the outputs only after that
 *     kernel has completed.  So the inputs of a call must be complete when
 *     it is enqueued: written by earlier calls or copies, or by kernels that
 *     do not release their dependents early.
 *   - Argument errors are detected on the host before anything is enqueued
 *     and returned as S4R_ERR_INVALID_ARG / S4R_ERR_UNSUPPORTED /
 *     S4R_ERR_WORKSPACE.  A failed launch returns S4R_ERR_CUDA.  Conditions
 *     only the device can see (a full cache on append, a length beyond the
 *     cache capacity, a bounded wait that gave up) set a sticky status word
 *     in the workspace, which s4r_read_device_status returns; the kernels
 *     then skip the offending work instead of touching memory out of bounds.
 *
 * Layouts (row-major, innermost index last).  D' = n_heads_kv * head_dim,
 * G = n_heads_q / n_heads_kv; query head h belongs to kv group g = h / G and
 * uses columns g*head_dim .. (g+1)*head_dim-1 of D'.  Coefficient row i of a
 * problem stores absolute token position n_sink + i; the first n_sink tokens
 * are the uncompressed sinks.
 */
#ifndef S4R_H
#define S4R_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  S4R_OK = 0,
  S4R_ERR_INVALID_ARG = 1,  /* null / misaligned pointer, inconsistent shape */
  S4R_ERR_UNSUPPORTED = 2,  /* valid request outside the supported range */
  S4R_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed */
  S4R_ERR_TIMEOUT = 4,      /* device status: a bounded device-side wait gave up */
  S4R_ERR_DEVICE = 5,       /* device status: a device-side check failed */
  S4R_ERR_WORKSPACE = 6     /* workspace pointer null or smaller than required */
} s4r_status;

/* S4R_FP4 is a storage type of the paged latent cache only (see
 * s4r_latent_write); every other tensor is S4R_F32 or S4R_BF16. */
typedef enum { S4R_F32 = 0, S4R_BF16 = 1, S4R_FP4 = 2 } s4r_dtype;

/* How the query window forms scoring rows (Eqs. 8-10).
 * CONCAT (default): W*G rows; row (w, j) concatenates query head g*G + j of
 *   every kv group g into one D'-vector, projected with the whole key basis.
 * PER_HEAD: W*H_q rows; row (w, h) projects query head h with the head_dim
 *   rows of the key basis that belong to its kv group. */
typedef enum { S4R_ROWS_CONCAT = 0, S4R_ROWS_PER_HEAD = 1 } s4r_row_mode;

/* Pooling of the candidate scores before selection (pool_kernel = odd kappa
 * > 1; "free parameters": kernel 7, from SnapKV).  Stride 1, same padding,
 * over the candidates only; neighbours outside the candidates are left out.
 * MAX: the largest neighbour score.  AVG: the mean of the in-range
 * neighbour scores (their sum in fp32, in position order, divided by their
 * count). */
typedef enum { S4R_POOL_MAX = 0, S4R_POOL_AVG = 1 } s4r_pool_mode;

/* Supported range (S4R_ERR_UNSUPPORTED outside it). */
#define S4R_MAX_D_MODEL 1024    /* D' */
#define S4R_MAX_RANK 256        /* rank_k, rank_v; multiples of 8 */
#define S4R_MAX_HEAD_DIM 256    /* multiple of 8 */
#define S4R_MAX_SCORE_ROWS 512  /* W*G (CONCAT) or W*H_q (PER_HEAD) */
#define S4R_MAX_POOL_KERNEL 63  /* odd */
#define S4R_MAX_GROUP 8         /* G = n_heads_q / n_heads_kv */
#define S4R_MAX_SINKS 16        /* n_sink */
#define S4R_MAX_SELECTED 8192   /* top_k + local_window */
#define S4R_MAX_BASIS_SAMPLE 1048576  /* n_sample T' of s4r_build_basis */
#define S4R_MAX_REQUESTS 8192   /* batch of s4r_page_plan and s4r_latent_attend */
#define S4R_MAX_LATENT_WIDTH 576  /* values a token of a latent cache (rank + rotary part) */
#define S4R_MAX_LATENT_RANK 512 /* leading values of a latent row that form the attended value */
#define S4R_MAX_PAGE_SIZE 1024  /* tokens a page: a power of two from 16 */

/* ------------------------------------------------------------------ encode */

/* Encode token states into coefficients, C = S . B ("What carries the
 * argument", Eq. 3): coeffs[t][j] = sum_d states[t][d] * basis[d][j].
 *   states  [n_tokens][d_model], row stride states_ld elements (>= d_model)
 *   basis   [d_model][rank], contiguous
 *   coeffs  [n_tokens][rank], row stride coeffs_ld elements (>= rank)
 * All three have type `dtype`; accumulation is fp32 and the result is
 * rounded to `dtype` (round to nearest even).  n_tokens == 0 is a no-op.
 * Strides must keep every row 16-byte aligned. */
s4r_status s4r_encode(const void *states, int64_t n_tokens, int64_t states_ld,
                      const void *basis, int32_t d_model, int32_t rank,
                      void *coeffs, int64_t coeffs_ld, s4r_dtype dtype, void *stream);

/* Encode two token sets against their own bases in one launch: the K and V
 * halves of a prompt (Eq. 3, "What carries the argument"), for p = 0, 1:
 *   coeffs_p[t][j] = sum_d states_p[t][d] * basis_p[d][j],  t < n_tokens.
 * Each (states_p, basis_p, coeffs_p) follows the layout, type, rounding and
 * alignment rules of s4r_encode; both share n_tokens, the strides, d_model
 * and rank.  The result equals two s4r_encode calls (the tensor-core path
 * runs both in one persistent grid, so the second problem's tiles fill the
 * SMs the first leaves idle).  Inputs and outputs stay owned by the caller. */
s4r_status s4r_encode2(const void *states0, const void *states1, int64_t n_tokens, int64_t states_ld,
                       const void *basis0, const void *basis1, int32_t d_model, int32_t rank,
                       void *coeffs0, void *coeffs1, int64_t coeffs_ld, s4r_dtype dtype, void *stream);

/* Append one new token per problem to the coefficient caches (Eq. 3 applied
 * to the token a decode step adds).  For each problem b, with n = lengths[b]
 * read on the device:
 *   coeff_k[b][n] = state_k[b] . basis_k[b],  coeff_v[b][n] = state_v[b] . basis_v[b],
 *   then lengths[b] = n + 1.
 * If n >= cache_rows the problem is skipped and the device status
 * (S4R_ERR_DEVICE) is set in `status_workspace` (may be NULL: skip only). */
typedef struct {
  int32_t batch, d_model, rank_k, rank_v;
  s4r_dtype dtype;
  int64_t cache_rows;                 /* row capacity of each problem's caches */
  const void *state_k, *state_v;      /* [batch][d_model] */
  const void *basis_k, *basis_v;      /* [batch][d_model][rank] */
  void *coeff_k, *coeff_v;            /* [batch][cache_rows][rank] */
  int32_t *lengths;                   /* [batch] device, read and incremented */
  void *status_workspace;             /* a decode workspace (its status word), or NULL */
} s4r_append_args;

s4r_status s4r_append(const s4r_append_args *args, void *stream);

/* ------------------------------------------------------------------ bases */

/* Build the low-rank bases at prefill ("What carries the argument" and the
 * Referee Report's summary, Eqs. 1-2; "Core claim" for the sample): for each
 * problem, the top-r right singular vectors of a sampled, token-wise
 * normalised set of its non-sink states.  With L = lengths[p] (read on the
 * device) and n = min(n_sample, L - n_sink) sample rows:
 *   - the last (7n + 5) div 10 rows L-1, L-2, ... (0.7 n rounded half up)
 *     and n_u = n - that many rows s + floor(j * span / n_u), j < n_u,
 *     spread over the older non-sink rows (span = L - s - recent rows);
 *   - every sampled row scaled to unit Euclidean norm (zero rows stay zero);
 *   - basis column k = right singular vector of the k-th largest singular
 *     value sigma[k], signed so that its largest-magnitude entry (lowest
 *     index on ties) is positive.
 * Arithmetic is fp64 throughout (the Gram matrix of the smaller side of the
 * sample and its eigenvectors by parallel cyclic Jacobi rotations); the
 * library owns no memory, so the caller passes a workspace of
 * s4r_basis_workspace_bytes() bytes whose first word is the sticky device
 * status (zero it once with s4r_workspace_init; read it with
 * s4r_read_device_status).  The status is set (S4R_ERR_DEVICE) when a
 * length lies outside [0, state_rows], when a sample has fewer than r rows
 * or rank below r (a kept sigma^2 at or below 1e-13 of the largest), or when
 * the rotations do not settle within 30 sweeps; S4R_ERR_TIMEOUT when a
 * grid-wide wait gave up.  The outputs of such a problem are then not a
 * basis. */
typedef struct {
  int32_t n_problems;     /* independent (sequence, layer, K or V) problems */
  int32_t d_model;        /* D' (<= S4R_MAX_D_MODEL) */
  int32_t rank;           /* r (<= min(n_sample, D', S4R_MAX_RANK)) */
  int32_t n_sink;         /* s: leading rows never sampled */
  int32_t n_sample;       /* T' (<= S4R_MAX_BASIS_SAMPLE) */
  s4r_dtype dtype;        /* type of states and basis_out */
  int64_t state_rows;     /* rows per problem in states (>= every length) */
  const int32_t *lengths; /* [n_problems] prompt length L of each problem */
  const void *states;     /* [n_problems][state_rows][D'] token states */
  void *basis_out;        /* [n_problems][D'][r] in dtype (fp64 -> fp32 -> dtype,
                             nearest even), or NULL */
  double *basis_f64;      /* [n_problems][D'][r] fp64, or NULL (not both NULL) */
  double *sigma;          /* [n_problems][r] singular values, or NULL */
  void *workspace;        /* s4r_basis_workspace_bytes(args) bytes */
  size_t workspace_bytes;
} s4r_basis_args;

/* Workspace bytes for these arguments (0 if they are invalid). */
size_t s4r_basis_workspace_bytes(const s4r_basis_args *args);

/* Enqueue the basis build (six kernels, one of them a cooperative launch).
 * Host-side argument errors: S4R_ERR_INVALID_ARG (null or misaligned
 * pointers, rank above n_sample or D'), S4R_ERR_UNSUPPORTED (sizes above the
 * limits), S4R_ERR_WORKSPACE. */
s4r_status s4r_build_basis(const s4r_basis_args *args, void *stream);

/* ------------------------------------------------------------------ decode */

typedef struct {
  int32_t batch;                      /* independent (sequence, layer) problems */
  int32_t n_heads_q, n_heads_kv, head_dim;
  int32_t rank_k, rank_v;
  int32_t n_sink;                     /* s: uncompressed sink tokens per problem */
  int32_t local_window;               /* w: newest coefficient rows always kept */
  int32_t top_k;                      /* k: global positions chosen before the window */
  int32_t query_window;               /* W: query rows scored per step */
  int32_t pool_kernel;                /* 1 = off; odd kappa = pool candidate scores */
  int32_t pool_mode;                  /* s4r_pool_mode (read when pool_kernel > 1) */
  int32_t row_mode;                   /* s4r_row_mode */
  s4r_dtype dtype;                    /* storage type of q, coefficients, bases, sinks */
  int64_t cache_rows;                 /* row capacity (stride) of the coefficient caches */
  const int32_t *lengths;             /* [batch] device: L_c, coefficient rows in use */
  const void *q;                      /* [batch][W][H_q][head_dim]; slot W-1 = current query */
  const void *coeff_k, *coeff_v;      /* [batch][cache_rows][rank_k | rank_v] */
  const void *basis_k, *basis_v;      /* [batch][D'][rank_k | rank_v] */
  const void *sink_k, *sink_v;        /* [batch][n_sink][D'] */
  float *out;                         /* [batch][H_q][head_dim] attention output */
  int32_t *idx;                       /* [batch][top_k] chosen absolute positions,
                                         ascending, -1 padded (window not listed) */
  float *scores;                      /* optional [batch][cache_rows] latent scores, or NULL */
  void *workspace;                    /* device scratch, see s4r_decode_workspace_bytes */
  size_t workspace_bytes;
  void *profile_events[2];            /* optional cudaEvent_t pair (or NULL): recorded on
                                         `stream` right before and right after the
                                         latent-scoring kernels, for timing them; under
                                         stream capture they become external event
                                         record nodes of the graph */
} s4r_decode_args;

/* Bytes of device workspace s4r_decode_step needs for these arguments (only
 * the shape fields are read).  Returns 0 if the shape is invalid. */
size_t s4r_decode_workspace_bytes(const s4r_decode_args *args);

/* Number of kernel launches one s4r_decode_step with these arguments
 * enqueues (0 if the shape is invalid). */
int32_t s4r_decode_kernel_launches(const s4r_decode_args *args);

/* Prepare a freshly allocated workspace: zeroes all of it (status word,
 * counters and accumulators that the kernels reuse and leave zeroed after
 * each call).  Call once per workspace allocation, before its first use. */
s4r_status s4r_workspace_init(void *workspace, size_t workspace_bytes, void *stream);

/* One decode step for every problem of the batch:
 *   1. C_Q = Q' . B^K for the query window (rows per row_mode);
 *   2. Z = C_Q . C_K^T / sqrt(rank_k), softmax of every row over the L_c
 *      coefficient rows, score[i] = sum of the rows' probabilities (Eqs. 8-10);
 *   3. idx = the top_k rows among 0 .. L_c-w-1 by score (pooled by
 *      pool_mode when pool_kernel > 1), equal scores -> lower position
 *      (Eqs. 13-15);
 *   4. for every query head h, exact attention of q[W-1][h] over the sinks,
 *      the chosen rows and the last w rows, with keys c_K . B^K^T and values
 *      c_V . B^V^T restricted to the head's kv group, logits scaled by
 *      1/sqrt(head_dim) (Eqs. 16-18).  Rebuilt rows are kept in fp32.
 * Arithmetic is fp32 whatever the storage type. */
s4r_status s4r_decode_step(const s4r_decode_args *args, void *stream);

/* ------------------------------------------------- decode without alloc */

/* Library extension: the S4R paper has no counterpart to this entry point.
 *
 * The same decode step as s4r_decode_step, for callers that cannot allocate
 * or own device memory for a workspace (a host program that manages no
 * device memory, or an engine that has handed all free HBM to its cache pool
 * and may not allocate while serving).  Instead of args->workspace (ignored,
 * may be NULL) it uses a scratch array of S4R_NOALLOC_SCRATCH_BYTES compiled
 * into the library, one per device.  It allocates nothing.
 *   - Shapes whose s4r_decode_workspace_bytes exceeds
 *     S4R_NOALLOC_SCRATCH_BYTES are rejected with S4R_ERR_UNSUPPORTED before
 *     anything is enqueued; s4r_last_error names both sizes.
 *   - The first call on a device (current device at call time) looks up the
 *     array and zeroes it synchronously; make that first call before any
 *     stream capture or other work that must not be synchronised.
 *   - Every call on a device shares the one array.  Calls that may overlap
 *     in time (other streams or host threads) race on it and give wrong
 *     results; order them on one stream or synchronise between them.
 *   - Device-side conditions (a bounded wait that gave up, a bad length) go
 *     to the library-wide status of the device: read them with
 *     s4r_read_device_status(NULL, stream). */
#define S4R_NOALLOC_SCRATCH_BYTES (4u << 20)
s4r_status s4r_decode_step_noalloc(const s4r_decode_args *args, void *stream);

/* ----------------------------------------------------------- reconstruct */

/* Rebuild selected rows from coefficients, out[e][d] = sum_j coeffs[rows[e]][j]
 * * basis[d][j] (Eq. 16).  coeffs [n_rows_total][rank] and basis
 * [d_model][rank] have type `dtype`; rows [n] device int32 row numbers (a
 * row < 0 or >= n_rows_total yields a zero output row); out [n][d_model]
 * fp32. */
s4r_status s4r_reconstruct(const void *coeffs, int64_t n_rows_total, const void *basis,
                           int32_t d_model, int32_t rank, const int32_t *rows, int64_t n,
                           float *out, s4r_dtype dtype, void *stream);

/* ------------------------------------------------- paged latent attention */

/* Library extension: attention over EVERY token of a cache that keeps one
 * latent vector a token, shared by all heads (next to s4r_decode_step, which
 * attends over a chosen few of its coefficient rows).  With basis_k, basis_v
 * [n_heads*head_dim][rank] (the layout of the decode bases, one group of rows
 * a head) and latents c [rank], optionally followed by a rotary key part
 * k_r [rope] that needs no basis:
 *   key_h = (basis_k[h] . c, k_r),  value_h = basis_v[h] . c.
 * Expanded form (prompts): keys and values are expanded with
 * s4r_latent_project and attended with s4r_prefill_attend.  Absorbed form
 * (decode): since q_h . (basis_k[h] c) = (q_h . basis_k[h]) . c, the queries
 * are projected into latent space (s4r_latent_project), s4r_latent_attend
 * attends over the cached latents themselves, and s4r_latent_project expands
 * the attended latents with basis_v.
 *
 * The cache is paged: pages of page_size token rows; request b's position p
 * is row p % page_size of page block_table[b][p / page_size], and
 * slot = page * page_size + row names a row of the whole cache.
 * s4r_page_plan hands out pages and computes slots, s4r_latent_write stores
 * rows.  Unlike a decode call's first kernel, the kernels of this section read
 * no input before the work enqueued ahead of them has completed.
 *
 * A page of a S4R_BF16 cache is [page_size][width].  A page of a S4R_FP4
 * cache is page_size * width * 9 / 16 bytes: the codes [page_size][width/2]
 * (two 4-bit values a byte, the even column in the low bits), then the scales
 * [page_size][width/16] (one e4m3 scale for 16 columns).  Column j of a row
 * stands for e2m1(code_j) * scale_{j/16} * cache_scale, e2m1 having the
 * magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit. */

/* Block tables and slot maps of a step, from request lengths, on the device.
 * Request b holds old = lengths[b] tokens and gets new = new_tokens[b] more;
 * have = ceil(old / page_size) pages are listed in its row of block_table.
 * With need_b = ceil((old + new) / page_size) - have and D_b the sum of
 * need_0 .. need_b, request b is SERVED if old, new >= 0, old + new <=
 * max_pages * page_size and (need_b == 0 or D_b <= free); a request that fails
 * the first two counts has need_b = 0.  Pages leave the free list from its
 * end, in request order: entry have + i of a served request becomes
 * free_pages[free - 1 - (D_b - need_b + i)].  Entries before `have` and behind
 * the new ones are left as they are.
 *   lengths_out[b]    = old + new of a served request, else old
 *   free_count_out[0] = free - (pages handed out)
 *   cu_tokens[b]      = new_0 + .. + new_{b-1} (negative counts as 0), b <= batch
 * and for token t of the flat batch (the j-th new token of request b, t =
 * cu_tokens[b] + j, whether b is served or not):
 *   slots[t]     = block_table[b][p / page_size] * page_size + p % page_size,
 *                  p = old + j; -1 if b is not served
 *   positions[t] = p, requests[t] = b
 * Entries of the three from cu_tokens[batch] to max_tokens - 1 become -1, so
 * a captured call with a fixed max_tokens serves any step.
 * lengths_out may be `lengths` and free_count_out may be `free_count` (the
 * state of a serving loop, updated in place); no other buffers may overlap.
 * Device status (S4R_ERR_DEVICE, in status_workspace if given): a request is
 * not served, the new tokens do not fit max_tokens (the rest is not
 * written), or free_count lies outside [0, free_capacity] (it is clamped). */
typedef struct {
  int32_t batch;                /* <= S4R_MAX_REQUESTS */
  int32_t page_size, max_pages; /* block_table row length */
  int32_t free_capacity;        /* entries of free_pages */
  int64_t max_tokens;           /* entries of slots, positions, requests */
  const int32_t *lengths;       /* [batch] tokens held before the step */
  const int32_t *new_tokens;    /* [batch] */
  int32_t *block_table;         /* [batch][max_pages] */
  const int32_t *free_pages;    /* [free_capacity] ids of free pages, the next one last */
  const int32_t *free_count;    /* [1] how many of them are free */
  int32_t *lengths_out;         /* [batch] */
  int32_t *free_count_out;      /* [1] */
  int32_t *cu_tokens;           /* [batch + 1] */
  int64_t *slots;               /* [max_tokens] */
  int32_t *positions;           /* [max_tokens], or NULL */
  int32_t *requests;            /* [max_tokens], or NULL */
  void *status_workspace;       /* a workspace (its status word), or NULL */
} s4r_page_plan_args;

s4r_status s4r_page_plan(const s4r_page_plan_args *args, void *stream);

/* Store latent rows in a paged cache: row slots[t] = latents[t].  A slot of
 * -1 (any negative one) is skipped; a slot of n_pages * page_size or above is
 * skipped and sets the device status (S4R_ERR_DEVICE).  Slots must differ
 * from one another: what a row named twice holds afterwards is not defined.
 * S4R_BF16: the values as they are.  S4R_FP4, for each 16 columns, with
 * fp32 arithmetic and x = latent / cache_scale:
 *   scale = e4m3(min(max|x| / 6, 448)), code = e2m1(x / scale), both to
 *   nearest, ties to even, |x / scale| > 6 to 6; a scale of 0 has codes 0.
 * Infinities therefore become +-6 * scale, NaN becomes 6 * scale.  `stored`
 * (optional, S4R_FP4) gets the values that the cache now stands for, rounded
 * to bf16 (exact when cache_scale is a power of two), skipped rows included. */
typedef struct {
  int64_t n_tokens;
  int32_t width;             /* multiple of 8 (S4R_BF16) or 32 (S4R_FP4) */
  int32_t page_size;
  int64_t n_pages;
  s4r_dtype cache_dtype;     /* S4R_BF16 or S4R_FP4 */
  float cache_scale;         /* S4R_FP4: > 0; ignored for S4R_BF16 */
  const void *latents;       /* [n_tokens][width] bf16 */
  int64_t latents_ld;        /* row stride in elements, a multiple of 8 */
  const int64_t *slots;      /* [n_tokens] */
  void *cache;               /* [n_pages] pages */
  void *stored;              /* [n_tokens][width] bf16 contiguous, or NULL */
  void *status_workspace;    /* a workspace (its status word), or NULL */
} s4r_latent_write_args;

s4r_status s4r_latent_write(const s4r_latent_write_args *args, void *stream);

/* Attention over the cached latents (absorbed form).  Request b holds
 * lengths[b] rows; its n_query query tokens are the last of them, so query
 * token t sees rows 0 .. lengths[b] - n_query + t.  For every head h
 *   z_i = scale * q[b][t][h] . row_i,  p = softmax(z),
 *   out[b][t][h] = sum_i p_i row_i[0 .. rank-1],  lse[b][t][h] = log sum_i e^{z_i}.
 * A query token that sees no row, or none whose logit is above -infinity, gets
 * out = 0, lse = -infinity.  What lies in rows that a query does not see (NaN
 * and infinities included) has no influence.  fp32 statistics and
 * accumulation; probabilities are rounded to 16 bits (bf16 next to bf16 rows,
 * fp16 next to 4-bit ones: those below 2^-21 of the largest one to 2^-32 of it)
 * for the value product only.
 * Device status (S4R_ERR_DEVICE): a length outside [0, max_pages *
 * page_size] (clamped), a page id outside [0, n_pages) among a request's
 * pages (not read); S4R_ERR_TIMEOUT as elsewhere.  The outputs
 * of such a request are not defined.
 * Workspace: s4r_latent_attend_workspace_bytes(args) bytes, prepared once
 * with s4r_workspace_init; calls that may overlap in time need their own. */
typedef struct {
  int32_t batch;             /* <= S4R_MAX_REQUESTS */
  int32_t n_query;           /* query tokens a request (1: plain decode) */
  int32_t n_heads;           /* n_query * n_heads <= 65536 */
  int32_t width;             /* values a cache row: rank + rotary part; multiple of 8 (S4R_FP4: 32) */
  int32_t rank;              /* leading values that are attended; multiple of 8, <= width */
  int32_t page_size;
  int32_t max_pages;         /* max_pages * page_size < 2^31 - 64 */
  s4r_dtype cache_dtype;     /* S4R_BF16 or S4R_FP4 */
  int64_t n_pages;           /* >= 1 */
  float scale;               /* of the logits */
  float cache_scale;         /* S4R_FP4: > 0; ignored for S4R_BF16 */
  const void *q;             /* [batch][n_query][n_heads][width] bf16 */
  const void *cache;         /* [n_pages] pages */
  const int32_t *block_table;/* [batch][max_pages] */
  const int32_t *lengths;    /* [batch] */
  void *out;                 /* [batch][n_query][n_heads][rank] bf16 */
  float *lse;                /* [batch][n_query][n_heads], or NULL */
  void *workspace;
  size_t workspace_bytes;
} s4r_latent_attend_args;

/* Workspace bytes for these arguments on the current device (only the shape
 * fields are read; 0 if they are invalid). */
size_t s4r_latent_attend_workspace_bytes(const s4r_latent_attend_args *args);
s4r_status s4r_latent_attend(const s4r_latent_attend_args *args, void *stream);

/* Per-head products between head space and latent space, bf16 with fp32
 * accumulation, rounded once (nearest even).  With B_h = rows h*head_dim ..
 * (h+1)*head_dim-1 of basis:
 *   to_latent != 0: out[t][h][j] = sum_d x[t][h][d] B_h[d][j]   (absorb queries)
 *   to_latent == 0: out[t][h][d] = sum_j x[t][h][j] B_h[d][j]   (expand latents)
 * x_hs == 0 lets all heads share one x row a token (expanding keys or values
 * from a token's latent).  Strides are in elements, multiples of 8; out rows
 * must not overlap one another or the inputs.  Device status: only
 * S4R_ERR_TIMEOUT, in the library-wide word (s4r_read_device_status(NULL, .)). */
typedef struct {
  int64_t n_tokens;
  int32_t n_heads, head_dim, rank;  /* multiples of 8; head_dim <= S4R_MAX_HEAD_DIM, rank <= S4R_MAX_LATENT_RANK */
  int32_t to_latent;
  const void *x;
  int64_t x_ts, x_hs;               /* token and head strides of x */
  const void *basis;                /* [n_heads*head_dim][rank] */
  void *out;
  int64_t out_ts, out_hs;           /* token and head strides of out */
} s4r_latent_project_args;

s4r_status s4r_latent_project(const s4r_latent_project_args *args, void *stream);

/* Attention of ragged prompts over expanded keys and values (bf16).  Sequence
 * b has query rows cu_q[b] .. cu_q[b+1]-1 and key rows cu_k[b] .. cu_k[b+1]-1;
 * with nq and nk of them, query i sees keys 0 .. nk - nq + i if causal (the
 * queries are the last tokens; a query with nk - nq + i < 0 sees none), else
 * all.  Query head h uses kv head h / (n_heads_q / n_heads_kv):
 *   z = scale * (q[:head_dim] . k + q[head_dim:] . k_rope),
 *   out = softmax(z) . v, lse = log sum e^z
 * k_rope is one row a key token for all heads (rope_dim == 0: none).  A query
 * that sees no key, or none whose logit is above -infinity, gets out = 0, lse =
 * -infinity.  fp32 statistics and accumulation, probabilities rounded to bf16
 * for the value product only.
 * Rows of out and lse outside every sequence are left as they are.
 * max_q must be at least the longest query count; it only sizes the launch.
 * Device status (the library-wide word, s4r_read_device_status(NULL, .)):
 * offsets that decrease or leave [0, total] (the sequence is skipped), a
 * sequence longer than max_q (its rows from max_q on are not computed);
 * S4R_ERR_TIMEOUT as elsewhere. */
typedef struct {
  int32_t batch;                         /* <= 65535 */
  int32_t n_heads_q, n_heads_kv;
  int32_t head_dim, rope_dim, value_dim; /* multiples of 8; head_dim, value_dim <= 128, rope_dim <= 64 */
  int32_t causal;
  int32_t max_q;
  int64_t total_q, total_k;              /* rows of q and out; of k, v and k_rope */
  float scale;
  const void *q;                         /* [total_q][n_heads_q][head_dim + rope_dim] */
  const void *k;                         /* [total_k][n_heads_kv][head_dim] */
  const void *v;                         /* [total_k][n_heads_kv][value_dim] */
  const void *k_rope;                    /* [total_k][rope_dim], or NULL */
  int64_t k_ts, v_ts, k_rope_ts;         /* token strides in elements, multiples of 8 */
  const int32_t *cu_q, *cu_k;            /* [batch + 1] device */
  void *out;                             /* [total_q][n_heads_q][value_dim] bf16 */
  float *lse;                            /* [total_q][n_heads_q], or NULL */
} s4r_prefill_attend_args;

s4r_status s4r_prefill_attend(const s4r_prefill_attend_args *args, void *stream);

/* ------------------------------------------------------------------ status */

/* Synchronise `stream`, then return the sticky device status of `workspace`
 * (S4R_OK, S4R_ERR_TIMEOUT or S4R_ERR_DEVICE); S4R_ERR_CUDA if the
 * synchronisation itself failed.  workspace == NULL reads the library-wide
 * status of the current device, which the kernels that take no workspace
 * (encode, reconstruct) report to. */
s4r_status s4r_read_device_status(const void *workspace, void *stream);

/* Reset the device status word of `workspace` (stream-ordered), or the
 * library-wide word of the current device when workspace == NULL (this
 * form synchronises `stream`). */
s4r_status s4r_clear_device_status(void *workspace, void *stream);

/* Testing hook for the device-side bounded waits; the S4R paper has no
 * counterpart.  Every spin-wait of the kernels (mbarrier waits, grid-wide
 * barriers) gives up after a limit, sets S4R_ERR_TIMEOUT in the device
 * status and lets the kernel finish without it (the call's results are then
 * not defined, but nothing hangs and the context stays usable).  This call
 * sets, for the current device:
 *   - limit_cycles: the limit in SM clock cycles (<= 0: the default, about
 *     2 s);
 *   - unreachable_barrier: when non-zero, the grid-wide barrier of the
 *     latent-scoring kernel waits for one arrival more than its grid has, the
 *     second products of s4r_latent_attend and s4r_prefill_attend for
 *     probabilities, and the results of s4r_latent_project for accumulators
 *     that never come, so they always run out after the limit.
 * It synchronises the device (cudaMemcpyToSymbol); do not call it while
 * other work of this library runs.  S4R_ERR_CUDA if the copy fails. */
s4r_status s4r_debug_waits(int64_t limit_cycles, int32_t unreachable_barrier);

/* Static description of a status code. */
const char *s4r_status_string(s4r_status status);

/* Human-readable description of the last S4R_ERR_CUDA returned on the
 * calling host thread (which step failed and the CUDA error name); "" if
 * none.  The string stays valid until the next failing call on the thread. */
const char *s4r_last_error(void);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int32_t s4r_version(void);

#ifdef __cplusplus
}
#endif
#endif /* S4R_H */
