/*
 * ctr.h -- C-ABI of libctr, the GB300 (sm_103a) CTR sparse-embedding path.
 *
 * The path: batch ID dedup -> pooled embedding-bag gather -> pairwise dot
 * interaction -> interaction backward -> per-unique-row gradient reduce and
 * SGD row update.  Every step runs in this library's CUDA kernels.
 *
 * Conventions shared by every call
 * --------------------------------
 * Memory.   Every pointer is DEVICE memory owned by the caller unless its
 *           comment says "host".  The library never allocates: scratch space
 *           comes from the caller's workspace `ws` (size from the matching
 *           *_workspace_size call, 256-byte aligned).
 * Streams.  Calls enqueue work on `stream` (a cudaStream_t; NULL = the legacy
 *           default stream) and return without synchronising, except
 *           ctr_check_status.
 * Errors.   Host-side validation returns a negative ctr_status before any
 *           launch.  Conditions only the device can see (an ID outside its
 *           table, offsets that are not monotone) set a sticky error word in the
 *           first 256 bytes of `ws`; ctr_check_status reports and clears it.
 *           The kernels never trap: a bad ID is skipped (treated as a zero
 *           row) and flagged.  A CUDA launch error maps to CTR_ERR_CUDA.
 * Bags.     Bags are CSR and field-major: bag (f, b) holds
 *           indices[offsets[f*B + b] .. offsets[f*B + b + 1]), f < num_fields,
 *           b < batch.  Each occurrence counts (a count matrix, not a 0/1 one).
 * Tables.   Several tables live in one buffer [total_rows, d]; table t owns
 *           global rows row_base[t] .. row_base[t+1]-1, and field f reads table
 *           bag_to_table[f].  Rows are contiguous, d elements each.
 * Determinism.  For a given input every output is bit-identical run to run:
 *           no float atomics, fixed reduction orders.
 */
#ifndef CTR_H
#define CTR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* ctr_stream_t; /* identical to cudaStream_t */

typedef enum {
  CTR_OK = 0,
  CTR_ERR_INVALID_ARG = -1,        /* null pointer, bad size, bad enum */
  CTR_ERR_UNSUPPORTED = -2,        /* valid but outside what the kernels cover */
  CTR_ERR_WORKSPACE = -3,          /* ws missing, misaligned or too small */
  CTR_ERR_INDEX_OUT_OF_RANGE = -4, /* device: an ID outside its table */
  CTR_ERR_CUDA = -5,               /* a CUDA runtime call or launch failed */
  CTR_ERR_TIMEOUT = -6,            /* device: a bounded wait ran out */
  CTR_ERR_NOT_IMPLEMENTED = -7,
  CTR_ERR_BAD_OFFSETS = -8,        /* device: offsets not monotone or not ending at n_ids */
  CTR_ERR_BAD_VALUE = -9           /* device: a NaN or +inf where a number is needed */
} ctr_status;

typedef enum { CTR_F32 = 0, CTR_BF16 = 1 } ctr_dtype;
typedef enum { CTR_POOL_SUM = 0, CTR_POOL_MEAN = 1 } ctr_pool;

/* Limits of the host-side per-field and per-table arrays. */
#define CTR_MAX_FIELDS 512
#define CTR_MAX_TABLES 512

/* Human-readable name of a ctr_status value (static string). */
const char* ctr_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int ctr_version(void);

/* Zero the sticky error word at the head of `ws` (async on `stream`).
 * Call once on a fresh workspace before its first use. */
int ctr_status_reset(void* ws, ctr_stream_t stream);

/* Synchronise `stream`, read the sticky error word of `ws`, clear it, and
 * return CTR_OK or the first device-side error recorded since the last reset. */
int ctr_check_status(void* ws, ctr_stream_t stream);

/* Per-kernel timing hook (diagnostics).  After this call, every launch of the
 * named kernel records `before_event` on the launching stream just before the
 * launch and `after_event` just after it (cudaEvent_t handles owned by the
 * caller; both NULL turns the hook off).  Kernels:
 *   CTR_KERNEL_GATHER            the pooled-gather kernel of ctr_embedding_bag_fwd
 *   CTR_KERNEL_BWD_TILES         the short-run tile kernel of ctr_embedding_bag_bwd_update
 *   CTR_KERNEL_BWD_PIECES        its long-run piece kernel
 *   CTR_KERNEL_SORT              all radix passes of ctr_dedup (first to last)
 *   CTR_KERNEL_INTERACTION       the kernel of ctr_dot_interaction
 *   CTR_KERNEL_INTERACTION_BWD   the kernel of ctr_dot_interaction_bwd
 *   CTR_KERNEL_GATHER_ROWS       the kernel of ctr_gather_rows
 * The setting is process-wide and not synchronised with calls running on
 * other host threads. */
typedef enum {
  CTR_KERNEL_GATHER = 1,
  CTR_KERNEL_BWD_TILES = 2,
  CTR_KERNEL_BWD_PIECES = 3,
  CTR_KERNEL_SORT = 4,
  CTR_KERNEL_INTERACTION = 5,
  CTR_KERNEL_INTERACTION_BWD = 6,
  CTR_KERNEL_GATHER_ROWS = 7
} ctr_kernel;
#define CTR_KERNEL_COUNT 8
int ctr_set_timing_events(int kernel, void* before_event, void* after_event);

/* Number of kernel launches this library has issued in this process, on all
 * devices and streams, since it was loaded (diagnostics: the difference across
 * a region counts the library's launches in it).  Host-side atomic counter;
 * never fails. */
uint64_t ctr_launch_count(void);

/* Gather variant of ctr_embedding_bag_fwd for fp32 tables with d = 128 and no
 * FM output: on != 0 selects the TMA row gather (cp.async.bulk.tensor with
 * tile::gather4 into a shared-memory ring), 0 (the default) the register-window
 * gather, which measured faster on GB300.  Both sum each bag in index order.
 * Process-wide; returns the previous setting. */
int ctr_set_tma_gather(int on);

/* Diagnostics: the wall-clock limit (nanoseconds, default 1e9) of each wait of
 * a ctr_dedup radix pass on a predecessor tile's counts.  A wait that runs out
 * records CTR_ERR_TIMEOUT in the workspace (read by ctr_check_status), the
 * pass keeps every write inside its buffers, and the call's outputs are then
 * meaningless.  A short limit makes ordinary waits run out: it exists to test
 * that path.  Process-wide, read at each launch; returns the previous limit. */
uint64_t ctr_set_wait_limit_ns(uint64_t ns);

/* Short-run pass of the row update for fp32 rows under plain SGD (no
 * optimizer state, no stochastic rounding) of d = 128, or of d <= 64 with d a
 * multiple of 4: mode 2 processes the short runs in slices of at most 64
 * columns (two for d = 128, one for d <= 64), two occurrences per warp step,
 * so the pooled-gradient rows of one table take half the L2 space at d = 128
 * and narrow rows keep twice the lanes busy; mode 1 never does; 0 (the
 * default) does for d <= 64 always, and for d = 128 when one table's
 * pooled-gradient rows (batch x 512 bytes) exceed 32 MB.  Every mode gives a
 * deterministic result within the same summation bound (each run's sum order
 * is fixed; the sliced pass adds the run's even and odd positions separately,
 * then the two partials).  Process-wide; returns the previous mode (a mode
 * outside 0..2 selects 0). */
int ctr_set_tile_slices(int mode);

/* ------------------------------------------------------------------------ */
/* Input generation (not part of the method)                                 */
/* ------------------------------------------------------------------------ */
/* Fill rows [row0, row0 + rows) of a table buffer with the counter-based
 * generator.  `table` points at global row row0; element (r, c) gets the value
 * of global element index (row0 + r) * d + c:
 *   gen_kind 0 (uniform, fp32 tables): h = splitmix64(seed ^ idx);
 *       v = (float)((int)(h >> 40) - 2^23) * scale
 *   gen_kind 1 (normal4, bf16 tables): Irwin-Hall sum of four 22-bit fields of
 *       splitmix64(seed ^ 2 idx) and splitmix64(seed ^ (2 idx + 1)), minus
 *       2^23 - 2, times scale, rounded to bf16 (nearest even).
 * splitmix64 is the output function of Steele, Lea and Flood (OOPSLA 2014). */
int ctr_fill_table(void* table, ctr_dtype dtype, int64_t rows, int32_t d, int64_t row0, int gen_kind,
                   uint64_t seed, float scale, ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* a1. Dedup: the virtual sparse feature                                     */
/* ------------------------------------------------------------------------ */
/* Source: "How TensorNet Supercharges Sparse Feature Training on TensorFlow",
 * Core Optimizations, embedding_lookup: collect the batch's IDs, sort them and
 * assign each distinct ID a continuous index; the batch-sized embedding matrix
 * has one row per distinct ID (its capacity is the batch's ID count).
 *
 * Keys are global rows k_i = row_base[bag_to_table[f]] + ids[i] (so equal IDs
 * of different tables stay apart, and per-table dedup falls out of one sort).
 * Requires total_rows = row_base[num_tables] <= 2^32 and n_ids < 2^31.
 *
 * Inputs
 *   ids            int64 [n_ids]        table-local IDs, field-major CSR
 *   offsets        int64 [F*B + 1]      offsets[0] = 0, offsets[F*B] = n_ids
 *   bag_to_table   host int32 [F]       table of each field
 *   row_base       host int64 [T + 1]   first global row of each table
 *   n_ids          host                 number of IDs (the caller sizes buffers by it)
 * Outputs (capacity n_ids each; a NULL int32 output is skipped)
 *   unique_rows    int64 [n_ids]        distinct keys, ascending; first n_unique valid
 *   n_unique       int64 [1]            number of distinct keys (device scalar)
 *   inverse        int32 [n_ids]        rank of key i in unique_rows (the virtual sparse feature)
 *   sorted_pos     int32 [n_ids]        stable sort permutation: position of the s-th key
 *   sorted_bag     int32 [n_ids]        bag (f*B + b) of sorted_pos[s]
 *   run_offsets    int32 [n_ids + 1]    run of unique u is sorted slots run_offsets[u] ..
 *                                       run_offsets[u+1]-1; run_offsets[n_unique] = n_ids
 *   unique_offsets int64 [T + 1]        uniques of table t are unique_rows[unique_offsets[t] ..
 *                                       unique_offsets[t+1]); unique_offsets[T] = n_unique
 * sorted_pos is the costliest output: when it is NULL (and total_rows <= 64 *
 * n_ids, when the ranks come from a presence bitmap over the table rows) the
 * sort carries bags instead of positions and writes sorted_bag directly.
 * Device errors: CTR_ERR_INDEX_OUT_OF_RANGE (an ID outside its table; its key
 * is then replaced by the last row of its table), CTR_ERR_BAD_OFFSETS,
 * CTR_ERR_TIMEOUT (a radix pass waited over 1 s on an earlier tile).
 * Workspace: ctr_dedup_workspace_size(n_ids, F, B, total_rows) bytes; it
 * grows with total_rows / 8 on the bitmap path. */
size_t ctr_dedup_workspace_size(int64_t n_ids, int32_t num_fields, int32_t batch, int64_t total_rows);
int ctr_dedup(const int64_t* ids, const int64_t* offsets, int32_t num_fields, int32_t batch,
              const int32_t* bag_to_table, const int64_t* row_base, int32_t num_tables, int64_t n_ids,
              int64_t* unique_rows, int64_t* n_unique, int32_t* inverse, int32_t* sorted_pos, int32_t* sorted_bag,
              int32_t* run_offsets, int64_t* unique_offsets, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* The same dedup in two parts, so a caller can schedule the other work of a
 * step between them.  CTR_DEDUP_PREPARE launches everything before the radix
 * passes (the keys, and on the presence-bitmap path the bitmap, unique_rows,
 * n_unique, unique_offsets and inverse); CTR_DEDUP_SORT launches the radix
 * passes and what follows them (sorted_pos, sorted_bag, run_offsets, and on
 * the path that sorts the rows themselves the unique outputs too).
 * CTR_DEDUP_ALL = both = ctr_dedup.  A SORT call must follow the PREPARE call
 * in stream order (or behind an event), with the same arguments and the same
 * workspace, which carries the state between them; outputs a part does not
 * write are undefined until the other part has run.  Errors as ctr_dedup;
 * CTR_ERR_INVALID_ARG for a phase mask outside 1..3. */
#define CTR_DEDUP_PREPARE 1
#define CTR_DEDUP_SORT 2
#define CTR_DEDUP_ALL 3
int ctr_dedup_phases(const int64_t* ids, const int64_t* offsets, int32_t num_fields, int32_t batch,
                     const int32_t* bag_to_table, const int64_t* row_base, int32_t num_tables, int64_t n_ids,
                     int64_t* unique_rows, int64_t* n_unique, int32_t* inverse, int32_t* sorted_pos,
                     int32_t* sorted_bag, int32_t* run_offsets, int64_t* unique_offsets, int32_t phases, void* ws,
                     size_t ws_bytes, ctr_stream_t stream);

/* TensorNet's batch-sized matrix (same passage): U[u] = table[unique_rows[u]]
 * for u < *n_unique.  capacity (host) bounds n_unique; rows of U at or beyond
 * n_unique are left untouched.  U is [capacity, d] of the table's dtype. */
int ctr_gather_rows(const void* table, ctr_dtype dtype, int32_t d, int64_t total_rows, const int64_t* unique_rows,
                    const int64_t* n_unique, int64_t capacity, void* U, void* ws, size_t ws_bytes,
                    ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* a2. Pooled embedding-bag forward                                          */
/* ------------------------------------------------------------------------ */
/* Source: "DHEN" notes, section 2.1 (each categorical term has a trainable
 * d-vector) and section 3.1, Solution 2 (sum the active embeddings); "Meta
 * DLRM", section 02 (categorical features go through embeddings).
 *
 *   out(b, f) = sum_{i in bag(f,b)} table[row_i]          (CTR_POOL_SUM)
 *             = that sum / len(bag)   (0 for an empty bag)  (CTR_POOL_MEAN)
 * accumulated in fp32, rounded once to out_dtype.
 * Row selection: if bag_to_table != NULL, indices are table-local int64 IDs and
 * row_i = row_base[bag_to_table[f]] + ids[i] (host arrays as in ctr_dedup);
 * if bag_to_table == NULL, indices are rows of `table` directly (e.g. the
 * int32 inverse map into the unique-row matrix U), num_tables ignored.
 * indices_are_int32 selects int32 or int64 indices; n_indices (host) is the
 * length of `indices` (a bag reaching past it is skipped and flagged).
 * out(b, f) is the d-vector at out + b*out_stride_b + f*out_stride_f
 * (element strides; e.g. the pooled slots of an interaction input [B, F+1, d]
 * are out = X + d, out_stride_b = (F+1)*d, out_stride_f = d).
 * table dtype CTR_F32 or CTR_BF16; out_dtype CTR_F32, or CTR_BF16 (bf16 tables).
 * Device errors: CTR_ERR_INDEX_OUT_OF_RANGE (row skipped), CTR_ERR_BAD_OFFSETS
 * (bag skipped, written as zeros).
 * Workspace: ctr_embedding_bag_workspace_size() bytes (the error word). */
size_t ctr_embedding_bag_workspace_size(void);
int ctr_embedding_bag_fwd(const void* table, ctr_dtype dtype, int32_t d, int64_t total_rows, const void* indices,
                          int indices_are_int32, int64_t n_indices, const int64_t* offsets, int32_t num_fields, int32_t batch,
                          const int32_t* bag_to_table, const int64_t* row_base, int32_t num_tables, ctr_pool pool,
                          void* out, ctr_dtype out_dtype, int64_t out_stride_b, int64_t out_stride_f, void* ws,
                          size_t ws_bytes, ctr_stream_t stream);

/* The same pooled gather, also writing the factorization-machine second-order
 * term of each bag ("DHEN" notes, section 3.1, Solution 2: the sum over pairs
 * of active features of <v_i, v_j> equals 1/2 (|sum v|^2 - sum |v|^2), one
 * pass over the rows):
 *   fm_out[f*B + b] = 1/2 ( |sum_{i in bag} row_i|^2 - sum_{i in bag} |row_i|^2 )
 * over the bag's occurrences (a repeated ID is a repeated feature), from the
 * raw sum whatever the pooling mode; 0 for bags with fewer than two IDs.
 * fp32 accumulation and arithmetic (the difference of the two terms loses
 * relative accuracy when they nearly cancel, as the identity's own form does).
 * fm_out: fp32 [F*B] device, required.  Supported for rows that are a whole
 * number of 16-byte chunks; CTR_ERR_UNSUPPORTED otherwise. */
int ctr_embedding_bag_fwd_fm(const void* table, ctr_dtype dtype, int32_t d, int64_t total_rows, const void* indices,
                             int indices_are_int32, int64_t n_indices, const int64_t* offsets, int32_t num_fields,
                             int32_t batch, const int32_t* bag_to_table, const int64_t* row_base, int32_t num_tables,
                             ctr_pool pool, void* out, ctr_dtype out_dtype, int64_t out_stride_b,
                             int64_t out_stride_f, float* fm_out, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* a3. Pairwise dot interaction                                              */
/* Workspace of both interaction calls: ctr_interaction_workspace_size()     */
/* bytes (the error word; the tensor-core kernel records CTR_ERR_TIMEOUT    */
/* there if one of its bounded waits runs out).                              */
/* ------------------------------------------------------------------------ */
/* Source: "Meta DLRM", section 02 (the interaction is the dot product between
 * every pair of embedding vectors and the processed dense features, cross terms
 * only); "DHEN" notes, section 3.1, Eq. (3) (pairwise inner products
 * concatenated with the dense features).
 *
 * X [batch, n, d], slot 0 = the dense vector, slots 1..n-1 = pooled embeddings.
 *   out[b] = [ X[b,0,:] | Z ],  Z[i(i-1)/2 + j] = <X[b,i,:], X[b,j,:]>,
 *            1 <= i < n, 0 <= j < i   (strict lower triangle, row by row)
 * out is [batch, d + n(n-1)/2] of the input dtype.  fp32: CUDA-core FMA.
 * bf16: tcgen05 tensor cores (fp32 accumulate in TMEM, bf16 output) when
 * n <= 32 and d is a multiple of 64 up to 256; other shapes use a CUDA-core
 * kernel with fp32 accumulation.  The fast kernels need X and out 16-byte
 * aligned; other pointers take the generic kernel. */
size_t ctr_interaction_workspace_size(void);
int ctr_dot_interaction(const void* X, ctr_dtype dtype, int32_t batch, int32_t n, int32_t d, void* out, void* ws,
                        size_t ws_bytes, ctr_stream_t stream);

/* Derivative of ctr_dot_interaction (fp32), not on the pages:
 *   dX[b,i,:] = sum_{j != i} dZ(i,j) X[b,j,:]  (+ dout[b, 0:d] for i = 0)
 * with dZ(i,j) = dout[b, d + hi(hi-1)/2 + lo], hi = max(i,j), lo = min(i,j).
 * dout [batch, d + n(n-1)/2], X and dX [batch, n, d]. */
int ctr_dot_interaction_bwd(const float* dout, const float* X, int32_t batch, int32_t n, int32_t d, float* dX,
                            void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Interaction variants.  CTR_INTERACT_CROSS is ctr_dot_interaction above.
 * CTR_INTERACT_WITH_SELF keeps the diagonal too ("DHEN" notes, section 3.1:
 * the AdvancedDLRM module takes all inner products <x_i, x_j> for i <= j):
 *   out[b] = [ X[b,0,:] | Z ],  Z[i(i+1)/2 + j] = <X[b,i,:], X[b,j,:]>, 0 <= j <= i < n
 * CTR_INTERACT_FULL_GRAM emits the whole Gram matrix ("DHEN" notes, section
 * 3.3, Eq. (7): the cross network's input X X^T), no dense vector:
 *   out[b] = Z,  Z[i n + j] = <X[b,i,:], X[b,j,:]>,  0 <= i, j < n
 * The order of the products and the leading dense vector are layout choices.
 * ctr_interaction_width(n, d, mode) is the output row length (-1 for bad
 * arguments).  The kernels, dtypes and alignment rules are those of
 * ctr_dot_interaction.  The derivative (fp32) is, with G the upstream gradient
 * of the emitted products (0 for products the mode omits) and S = G + G^T:
 *   dX[b,i,:] = sum_j S[i][j] X[b,j,:]  (+ dout[b, 0:d] for i = 0, first two modes). */
typedef enum { CTR_INTERACT_CROSS = 0, CTR_INTERACT_WITH_SELF = 1, CTR_INTERACT_FULL_GRAM = 2 } ctr_interaction_mode;
int64_t ctr_interaction_width(int32_t n, int32_t d, int mode);
int ctr_dot_interaction_mode(const void* X, ctr_dtype dtype, int32_t batch, int32_t n, int32_t d, int mode, void* out,
                             void* ws, size_t ws_bytes, ctr_stream_t stream);
int ctr_dot_interaction_bwd_mode(const float* dout, const float* X, int32_t batch, int32_t n, int32_t d, int mode,
                                 float* dX, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* a5. Sparse backward: per-unique-row gradient reduce + SGD row update       */
/* ------------------------------------------------------------------------ */
/* Source: "How TensorNet ...", Synchronous Architecture (only the sparse
 * features present in the batch are synchronised) and Core Optimizations (the
 * batch-sized matrix of unique rows).  The SGD rule is not on the pages.
 *
 * For each unique u < *n_unique, over its run of sorted occurrences s (from
 * ctr_dedup):
 *   g_u = sum_s scale(bag_s) * grad_pooled(bag_s),  scale = 1 (SUM) or
 *         1 / len(bag) (MEAN),   bag_s = sorted_bag[s] = f*B + b,
 *         grad_pooled(bag) = the fp32 d-vector at grad_pooled + b*g_stride_b + f*g_stride_f
 *   table[unique_rows[u]] <- table[unique_rows[u]] - lr * g_u
 * Each row is written exactly once; no float atomics.  The sum runs in a fixed
 * order (pieces of at most 128 occurrences summed in sorted order, then a fixed
 * tree over the pieces of a long run), so results are deterministic.
 * fp32 tables: one fused multiply-add, rounded once.  bf16 tables: the update
 * is computed in fp32 and rounded to bf16 (nearest even).
 * grad_unique_out (optional, [n_ids, d] fp32): receives g_u in row u.
 * n_ids (host) is the capacity used to size grids; *n_unique <= n_ids.
 * Workspace: ctr_bwd_update_workspace_size(n_ids, d) bytes. */
size_t ctr_bwd_update_workspace_size(int64_t n_ids, int32_t d);
int ctr_embedding_bag_bwd_update(const float* grad_pooled, int64_t g_stride_b, int64_t g_stride_f,
                                 const int64_t* offsets, int32_t num_fields, int32_t batch, ctr_pool pool,
                                 const int64_t* unique_rows, const int64_t* n_unique, const int32_t* run_offsets,
                                 const int32_t* sorted_bag, int64_t n_ids, float lr, void* table, ctr_dtype dtype,
                                 int32_t d, int64_t total_rows, float* grad_unique_out, void* ws, size_t ws_bytes,
                                 ctr_stream_t stream);

/* The same update in phases, for callers that overlap them on two streams.
 *   CTR_BWD_SHORT_RUNS  runs of at most 128 occurrences: summed and their rows
 *                       updated
 *   CTR_BWD_LONG_RUNS   every longer run: listed, cut into pieces of 128 and
 *                       each piece summed into the workspace
 *   CTR_BWD_FINISH      the long runs' pieces combined and their rows updated
 * ctr_embedding_bag_bwd_update runs all three in this order (short runs first:
 * the long runs then find many pooled-gradient rows still in L2).  LONG_RUNS and
 * SHORT_RUNS touch disjoint rows and disjoint workspace words, so they may run
 * concurrently on two streams with the same arguments and workspace; FINISH
 * must be ordered after LONG_RUNS (and both after the dedup that produced the
 * runs).  `phases` is a non-empty mask of the three; the phases it names run
 * in the order above on `stream`. */
typedef enum { CTR_BWD_SHORT_RUNS = 2, CTR_BWD_LONG_RUNS = 1, CTR_BWD_FINISH = 4 } ctr_bwd_phase;
int ctr_embedding_bag_bwd_update_phases(const float* grad_pooled, int64_t g_stride_b, int64_t g_stride_f,
                                        const int64_t* offsets, int32_t num_fields, int32_t batch, ctr_pool pool,
                                        const int64_t* unique_rows, const int64_t* n_unique,
                                        const int32_t* run_offsets, const int32_t* sorted_bag, int64_t n_ids, float lr,
                                        void* table, ctr_dtype dtype, int32_t d, int64_t total_rows,
                                        float* grad_unique_out, int phases, void* ws, size_t ws_bytes,
                                        ctr_stream_t stream);

/* The same update under an optimizer with per-row state, kept only for the
 * rows the batch touches (the pages name no update rule; these are readings):
 *   CTR_OPT_SGD               w -= lr g                                   (no state)
 *   CTR_OPT_ADAGRAD           s += g^2;  w -= lr g / (sqrt(s) + eps)      state0 [total_rows, d]
 *   CTR_OPT_ROWWISE_ADAGRAD   s += mean over the row of g^2;
 *                             w -= lr g / (sqrt(s) + eps)                state0 [total_rows]
 *   CTR_OPT_ADAM              m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
 *                             w -= lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
 *                             (Kingma and Ba 2015)          state0 = m, state1 = v [total_rows, d]
 * g is the row's reduced gradient (as in ctr_embedding_bag_bwd_update); state
 * arrays are fp32 device memory owned by the caller, indexed by global row,
 * 16-byte aligned, and only the batch's rows are read and written.  t = step
 * (>= 1) is this update's step number for Adam's bias correction; eps > 0.
 * phases as in ctr_embedding_bag_bwd_update_phases.  The optimizer
 * arithmetic is fp32.
 *
 * Stochastic rounding ("DHEN" notes, section 6.4: low-precision embeddings
 * with stochastic rounding; applied here to bf16 tables, with any kind): the
 * new value x (fp32) of element (row, c) becomes the bf16 neighbour above it
 * in magnitude with probability f = (|x| - lo) / (hi - lo), lo and hi its bf16
 * neighbours, else lo: with u the element's 16 random bits, x rounds up when
 * f + u / 2^16 >= 1, i.e. u is added to the 16 bits bf16 drops and the carry
 * kept.  The 4 values of column chunk q = c / 4 take bits 16 (c mod 4) ..
 * 16 (c mod 4) + 15 of splitmix64(sr_seed ^ (row d / 4 + q)).  Values at or
 * beyond the largest finite bf16 round to nearest.  fp32 tables ignore it. */
typedef enum { CTR_OPT_SGD = 0, CTR_OPT_ADAGRAD = 1, CTR_OPT_ROWWISE_ADAGRAD = 2, CTR_OPT_ADAM = 3 } ctr_opt_kind;
typedef struct {
  int kind;       /* ctr_opt_kind */
  float eps;
  float beta1;    /* Adam */
  float beta2;    /* Adam */
  int64_t step;   /* Adam: t >= 1 */
  float* state0;  /* Adagrad sum of squares, or Adam m */
  float* state1;  /* Adam v */
  int32_t stochastic_rounding;  /* bf16 tables: round the new rows stochastically (below) */
  uint64_t sr_seed;             /* its random bits; use a new seed every step */
} ctr_optimizer;
int ctr_embedding_bag_bwd_update_opt(const float* grad_pooled, int64_t g_stride_b, int64_t g_stride_f,
                                     const int64_t* offsets, int32_t num_fields, int32_t batch, ctr_pool pool,
                                     const int64_t* unique_rows, const int64_t* n_unique, const int32_t* run_offsets,
                                     const int32_t* sorted_bag, int64_t n_ids, float lr, void* table, ctr_dtype dtype,
                                     int32_t d, int64_t total_rows, float* grad_unique_out, int phases,
                                     const ctr_optimizer* opt, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* b. Expert layer on the interaction output                                  */
/* ------------------------------------------------------------------------ */
/* Source: "DHEN" notes, the mixture-of-experts section (a gate sends each
 * sample to a few experts and adds their results up).  The pages give no
 * shapes or kernels; the formulas below are this library's.
 *
 * A sample is called a token here; a token's k chosen experts are its choices.
 * Row order: the (token, choice) pairs sorted by expert, then by token.  Row r
 * of that order belongs to token[r], expert e owns rows offsets[e] ..
 * offsets[e+1]-1, and choice j of token t is row slot[t*k + j] (-1: no row).
 * offsets[experts] = routed rows <= tokens*k; token[r] = -1 beyond them.
 * All maps are int32; tokens*k < 2^31; 1 <= experts <= CTR_MAX_EXPERTS,
 * 1 <= k <= min(experts, CTR_MAX_CHOICES).  Matrices are row-major with a row
 * stride ld >= the row's elements (in elements); any alignment of the element
 * type is accepted (16-byte aligned rows take wider loads).
 * A NULL pointer is refused unless the text says optional; a call with zero
 * tokens or rows writes what has no token (offsets, norms) and succeeds. */
#define CTR_MAX_EXPERTS 512
#define CTR_MAX_CHOICES 16

/* Routing.  With l = scores[t, :] (fp32 or bf16; fp32 arithmetic) and A = the
 * experts with l_e > -inf:
 *   choice j = the j-th largest l_e over A, ties to the lower index
 *   weight_j = exp(l_e - m) / sum over B of exp(l_i - m),   m = max l,
 *              B = A, or the choices alone if renormalize != 0
 * A token with fewer than k experts in A gets expert -1, weight 0, slot -1 for
 * the rest (all of them where A is empty).  A token with a NaN or +inf score is
 * treated as if A were empty, and flagged CTR_ERR_BAD_VALUE.
 * Outputs: expert int32, weight fp32, slot int32 [tokens, k] (dense), token
 * int32 [tokens*k], offsets int32 [experts + 1].
 * Workspace: ctr_expert_route_workspace_size(tokens, experts, k) bytes.
 * Batches of 257 to 4096 tokens (and smaller ones of many experts) run as one
 * thread-block cluster where the device can place one of 16 blocks, else as
 * three launches like larger ones; ctr_set_route_cluster(0) takes the three
 * always (diagnostics; process-wide, returns the previous setting). */
int ctr_set_route_cluster(int on);
size_t ctr_expert_route_workspace_size(int64_t tokens, int32_t experts, int32_t k);
int ctr_expert_route(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts, int64_t ld_scores,
                     int32_t k, int renormalize, int32_t* expert, float* weight, int32_t* slot, int32_t* token,
                     int32_t* offsets, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Its gradient, the choices held fixed: with p = the softmax over B (0 outside),
 * g_e = dweight_j for the expert of choice j (0 for the others),
 *   dscores[t, e] = p_e (g_e - sum_i p_i g_i)
 * in the scores' type.  Masked scores and tokens with nothing routed get 0.
 * expert is the output of ctr_expert_route on the same scores; ws: as there or
 * ctr_expert_workspace_size() bytes. */
int ctr_expert_route_bwd(const float* dweight, const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts,
                         int64_t ld_scores, int32_t k, int renormalize, const int32_t* expert, void* dscores,
                         int64_t ld_dscores, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Tokens into row order: out[slot[t*k+j], :] = x[t, :], and zeros in the rows
 * r with token[r] = -1.  out is [tokens*k, d].  ws (these calls and
 * ctr_expert_combine*): ctr_expert_workspace_size() bytes, the error word.
 * Device errors: CTR_ERR_INDEX_OUT_OF_RANGE (a slot >= tokens*k: skipped). */
size_t ctr_expert_workspace_size(void);
int ctr_expert_dispatch(const void* x, ctr_dtype dtype, int64_t tokens, int32_t d, int64_t ldx, int32_t k,
                        const int32_t* slot, const int32_t* token, void* out, int64_t ldo, void* ws, size_t ws_bytes,
                        ctr_stream_t stream);

/* Rows back to tokens: y[t, :] = sum over j with slot >= 0 of weight[t*k+j] *
 * rows[slot[t*k+j], :], summed in fp32 in the order of j and rounded once; a
 * token without rows gets zeros.  weight NULL: all 1 (then this is also the
 * gradient of ctr_expert_dispatch: dx from the rows' gradient). */
int ctr_expert_combine(const void* rows, ctr_dtype dtype, int64_t tokens, int32_t d, int64_t ld_rows, int32_t k,
                       const int32_t* slot, const float* weight, void* y, int64_t ldy, void* ws, size_t ws_bytes,
                       ctr_stream_t stream);

/* Gradient of ctr_expert_combine:
 *   drows[slot[t*k+j], :] = weight[t*k+j] dy[t, :]   (zeros in rows with token[r] = -1)
 *   dweight[t*k+j] = <dy[t, :], rows[slot[t*k+j], :]>  (fp32; 0 where slot = -1) */
int ctr_expert_combine_bwd(const void* dy, ctr_dtype dtype, int64_t tokens, int32_t d, int64_t ld_dy, int32_t k,
                           const void* rows, int64_t ld_rows, const int32_t* slot, const float* weight,
                           const int32_t* token, void* drows, int64_t ld_drows, float* dweight, void* ws,
                           size_t ws_bytes, ctr_stream_t stream);

/* ---- 8-bit products with a scale per block of 128 ----------------------- */
/* Codes are e4m3 (4 exponent bits, 3 mantissa bits, largest value 448), one
 * byte each.  A block's scale and codes are, in fp32 with m = the block's
 * largest |x| but at least 2^-100,
 *   scale = m / 448,   code = e4m3(x * (448 / m))   (nearest even)
 * so the value that a code stands for is code * scale.  A block with a NaN or
 * an infinity gives NaN results for the rows it enters.
 * Layouts (P(n) = n rounded up to a multiple of 128, B(n) = P(n) / 128):
 *   row codes      [rows, P(cols)], zeros past cols; row scales fp32 [B(cols),
 *                  ld_scale], one per row and 128 columns: scale[c/128][r]
 *   block codes    [groups, n, P(k)] with scales [groups, B(n), B(k)], one per
 *                  128 x 128 block; their transpose [groups, k, P(n)] with
 *                  scales [groups, B(k), B(n)]
 *   column codes   [cols, P_rows], the transpose of grouped rows: each group's
 *                  rows start at a multiple of 128 along the row axis and are
 *                  filled up with zeros; P_rows = ctr_fp8_padded_rows(rows,
 *                  groups).  Scales by column, [P_rows / 128, cols], or by
 *                  128 x 128 block, [B(cols), P_rows / 128].
 * Codes must be 16-byte aligned. */
int64_t ctr_fp8_padded_rows(int64_t rows, int32_t groups);

/* Row codes of x [x_rows, cols], or of its rows row_index[r] for r < rows
 * (optional, int32; -1 gives a zero row).  Device errors:
 * CTR_ERR_INDEX_OUT_OF_RANGE (an index >= x_rows: a zero row).  ws: the error
 * word (256 bytes), in every ctr_fp8_quantize_* call. */
int ctr_fp8_quantize_rows(const void* x, ctr_dtype dtype, int64_t x_rows, int64_t rows, int64_t cols, int64_t ldx,
                          const int32_t* row_index, uint8_t* q, float* scale, int64_t ld_scale, void* ws,
                          size_t ws_bytes, ctr_stream_t stream);

/* Row codes and column codes of the same rows in one read, for a training
 * step.  offsets: int32 [groups + 1], offsets[0] = 0, rows of group g are
 * offsets[g] .. offsets[g+1]-1, offsets[groups] <= rows (rows beyond have no
 * group: their row codes are not written).  cols_by_block: 0 = a scale per
 * column and 128 rows (the left operand of ctr_fp8_matmul_wgrad), 1 = a scale
 * per 128 x 128 block (the right one).  Device errors: as above, and
 * CTR_ERR_BAD_OFFSETS (nothing is written). */
int ctr_fp8_quantize_rows_cols(const void* x, ctr_dtype dtype, int64_t x_rows, int64_t rows, int64_t cols, int64_t ldx,
                               const int32_t* row_index, const int32_t* offsets, int32_t groups, int cols_by_block,
                               uint8_t* q, float* scale, int64_t ld_scale, uint8_t* qc, float* scale_c, void* ws,
                               size_t ws_bytes, ctr_stream_t stream);

/* Block codes of w [groups, n, k] (dense), and of its transpose where qt and
 * scale_t (both or neither) are given. */
int ctr_fp8_quantize_blocks(const void* w, ctr_dtype dtype, int32_t groups, int64_t n, int64_t k, uint8_t* q,
                            float* scale, uint8_t* qt, float* scale_t, void* ws, size_t ws_bytes,
                            ctr_stream_t stream);

/* out[r, :] = W_g a_r for the rows r of group g: with a, b the values that the
 * row codes (a, [rows, P(k)]) and block codes (b, [groups, n, P(k)]) stand for,
 *   out[r, i] = sum over c < k of a[r, c] b[g, i, c],
 * blocks of 128 summed by the tensor cores in fp32, the blocks' sums scaled and
 * added in fp32, one rounding to out_dtype (a row's and a block's scale are
 * multiplied first: a product of theirs that is no normal fp32 number, as of
 * blocks whose largest magnitudes multiply to less than 2.4e-33, loses bits, and
 * one that overflows gives infinities or NaN).  offsets as above; NULL means that
 * all rows are group 0 (groups = 1).  Rows past offsets[groups] get zeros.
 * out [rows, n], row stride ldo.  Device errors: CTR_ERR_BAD_OFFSETS (zeros are
 * written), CTR_ERR_TIMEOUT.  The input gradient of out = W x is the same call
 * with dout's row codes and the transposed block codes.
 * Workspace (both products): ctr_fp8_matmul_workspace_size(rows, groups, n, k),
 * asked on the device of the call: the error word and, for a weight gradient
 * whose tiles are few and sums long, the partial sums (up to 20 MB).  Of it
 * ctr_fp8_matmul takes the error word alone. */
size_t ctr_fp8_matmul_workspace_size(int64_t rows, int32_t groups, int64_t n, int64_t k);
int ctr_fp8_matmul(const uint8_t* a, const float* a_scale, int64_t ld_scale, const uint8_t* b, const float* b_scale,
                   const int32_t* offsets, int64_t rows, int32_t groups, int64_t n, int64_t k, void* out,
                   ctr_dtype out_dtype, int64_t ldo, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Weight gradient: out[g, i, j] = sum over the rows r of group g of d[r, i]
 * x[r, j], from column codes of d (by column, [n, P_rows]) and of x (by block,
 * [k, P_rows]) made with the same offsets.  out [groups, n, k], dense; zeros
 * for a group without rows, and everywhere after CTR_ERR_BAD_OFFSETS. */
int ctr_fp8_matmul_wgrad(const uint8_t* d, const float* d_scale, const uint8_t* x, const float* x_scale,
                         const int32_t* offsets, int64_t rows, int32_t groups, int64_t n, int64_t k, void* out,
                         ctr_dtype out_dtype, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* ---- Global gradient norm and clipping ---------------------------------- */
/* norm = sqrt(sum over every element of every tensor of g^2), and
 *   outs[i] = grads[i] * c,   c = norm > max_norm ? max_norm / norm : 1
 * (the product in fp32, rounded once to the tensor's type).  grads, outs,
 * dtypes and counts are host arrays of n_tensors entries (outs optional: norm
 * only; outs[i] may be grads[i] but must not overlap anything else).  Blocks of
 * elements are squared and added in fp32, what is joined is joined in fp64, and
 * magnitudes whose squares leave fp32's range are squared in fp64, so norm is
 * right wherever it is an fp32 number.  A norm that is not finite leaves the
 * gradients as they are (c = 1) for the caller to see: norm (fp32 [1], device)
 * reports it.  max_norm >= 0 and not NaN.  Tensors need element alignment only.
 * Workspace: ctr_clip_grads_workspace_size() bytes. */
size_t ctr_clip_grads_workspace_size(void);
int ctr_clip_grads(const void* const* grads, void* const* outs, const int32_t* dtypes, const int64_t* counts,
                   int32_t n_tensors, float max_norm, float* norm, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* c. Layers around the experts                                               */
/* ------------------------------------------------------------------------ */
/* Source: "DHEN" notes, section 2.2 (a layer's output is Norm(Ensemble(...) +
 * ShortCut)) and the mixture-of-experts section; "Meta DLRM", section 02 (the
 * dense stacks below and above the interaction).  The pages give no shapes and
 * no norm; the formulas below are this library's.  Matrices, types, alignment
 * and NULL pointers as in section b. */

/* ---- Balanced routing ----------------------------------------------------- */
/* ctr_expert_route with a score function, a bias for balance and groups of
 * experts.  With l = scores[t, :] and A = the experts with l_e > -inf:
 *   p_e   = softmax over A of l (CTR_SCORE_SOFTMAX), or 1 / (1 + exp(-l_e))
 *   key_e = p_e + bias_e, for e in A with bias_e > -inf (bias fp32 [experts],
 *           optional; the program moves it towards even loads, it has no gradient)
 * Experts are `groups` groups of experts / groups neighbours.  The group_k groups
 * with the largest sums of their two largest keys (of the one that they have)
 * stay; choice j is the j-th largest key in them.  Keys and sums are those of
 * 64-bit arithmetic (choices without a bias go by the scores themselves, whose
 * order is the keys'); ties go to the lower index.
 *   weight_j = factor p_j, divided by the sum of the choices' p if renormalize != 0
 * Maps, missing choices, NaN or +inf scores, limits and workspace as in
 * ctr_expert_route; a NaN or +inf in bias is taken for -inf and flagged
 * CTR_ERR_BAD_VALUE.  experts is a multiple of groups, 1 <= group_k <= groups <=
 * CTR_MAX_GROUPS, k <= group_k experts / groups; factor is finite. */
#define CTR_MAX_GROUPS 32
typedef enum { CTR_SCORE_SOFTMAX = 0, CTR_SCORE_SIGMOID = 1 } ctr_score;
int ctr_expert_route_balanced(const void* scores, ctr_dtype dtype, int64_t tokens, int32_t experts, int64_t ld_scores,
                              int32_t k, int score, const float* bias, int32_t groups, int32_t group_k,
                              int renormalize, float factor, int32_t* expert, float* weight, int32_t* slot,
                              int32_t* token, int32_t* offsets, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Its gradient, the choices held fixed: dscores = the gradient of sum over j of
 * dweight_j weight_j, in the scores' type; 0 for masked scores, for tokens with
 * nothing routed and, with sigmoids or renormalized weights, for experts that
 * were not chosen.  ws: as ctr_expert_route_bwd. */
int ctr_expert_route_balanced_bwd(const float* dweight, const void* scores, ctr_dtype dtype, int64_t tokens,
                                  int32_t experts, int64_t ld_scores, int32_t k, int score, int renormalize,
                                  float factor, const int32_t* expert, void* dscores, int64_t ld_dscores, void* ws,
                                  size_t ws_bytes, ctr_stream_t stream);

/* ---- Dense layers ---------------------------------------------------------- */
typedef enum {
  CTR_ACT_NONE = 0,
  CTR_ACT_RELU = 1,    /* max(z, 0) */
  CTR_ACT_SILU = 2,    /* z / (1 + exp(-z)) */
  CTR_ACT_GELU = 3,    /* z (1 + erf(z / sqrt 2)) / 2 */
  CTR_ACT_SIGMOID = 4  /* 1 / (1 + exp(-z)) */
} ctr_activation;

/* z = x W^T + bias and y = act(z) + residual:
 *   z[t, i] = sum over c < k of x[t, c] w[i, c]  + bias[i],    y[t, i] = act(z[t, i]) + residual[t, i]
 * x [rows, k], w [n, k], bias [n] (optional), residual (optional), y and pre
 * [rows, n], all of `dtype`.  pre (optional) gets z, which the backward call
 * needs where there is an activation.  Sums are fp32, bias, activation and
 * residual are applied to them in fp32, y and pre are rounded once.
 * bf16: products of the tensor cores, whose additions drop what fp32 cannot hold:
 * sums of up to 65536 terms are up to 1.8e-4 of their terms' magnitudes too near
 * to zero; longer ones, and all of fp32's, are read back as they go and added up
 * with rounding.  fp32: also there, x and w each as three bf16 numbers that add up
 * to it, six of their nine products: what is dropped is below 2^-24 of |x| |w|, so
 * results are as near as those of fp32 sums, but for numbers below 2^-109, which
 * the three hold to within 2^-134 (half of bf16's smallest step).  A NaN or an
 * infinity in x or w, or a sum past fp32's range, makes what it enters NaN, or the
 * infinity that the formula gives.  Activations and their derivatives: within 16
 * and 20 times 2^-24 of themselves (of their terms, where those cancel) for fp32;
 * for bf16 below the result's rounding, but gelu's tail, which is within 1.5e-7; 0
 * where an exponential is below 2^-126.  y may be residual itself (the same rows
 * and stride); nothing else may overlap.
 * Device errors: CTR_ERR_TIMEOUT.
 * Workspace: ctr_dense_workspace_size(rows, n, k, dtype, train, packed) bytes,
 * asked on the device of the call: train != 0 for ctr_dense_bwd (with room for
 * ctr_dense too), packed != 0 where rows of a bf16 matrix do not start at
 * multiples of 16 bytes.  Enough for any call of at most `rows` rows; a call that
 * needs more than it is given is refused (CTR_ERR_WORKSPACE). */
size_t ctr_dense_workspace_size(int64_t rows, int64_t n, int64_t k, ctr_dtype dtype, int train, int packed);
int ctr_dense(const void* x, ctr_dtype dtype, int64_t rows, int64_t k, int64_t ldx, const void* w, int64_t n,
              int64_t ldw, const void* bias, int act, const void* residual, int64_t ld_residual, void* y, int64_t ld_y,
              void* pre, int64_t ld_pre, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Its gradients.  With dz = dy act'(pre) (relu: 1 where pre > 0, else 0; pre as
 * ctr_dense wrote it, not read without an activation):
 *   dx[t, c] = sum over i of dz[t, i] w[i, c]      (dtype)
 *   dw[i, c] = sum over t of dz[t, i] x[t, c]      (grad_dtype)
 *   dbias[i] = sum over t of dz[t, i]              (grad_dtype)
 * each optional; the residual's gradient is dy.  grad_dtype is dtype or CTR_F32.
 * For bf16, dz is rounded to bf16 for the two products (not for dbias); sums are
 * fp32 in an order that is the same in every run.  No rows: dw and dbias are
 * zeros.  Outputs may not overlap anything. */
int ctr_dense_bwd(const void* dy, ctr_dtype dtype, int64_t rows, int64_t n, int64_t ld_dy, const void* x, int64_t k,
                  int64_t ldx, const void* w, int64_t ldw, const void* pre, int64_t ld_pre, int act, void* dx,
                  int64_t ld_dx, ctr_dtype grad_dtype, void* dw, int64_t ld_dw, void* dbias, void* ws, size_t ws_bytes,
                  ctr_stream_t stream);

/* ---- Root-mean-square norm on a residual stream ------------------------- */
/* For each row:
 *   s = x + residual, rounded to the rows' type (s = x where residual is NULL)
 *   v = s / sqrt(mean(s^2) + eps) * gamma        (fp32; gamma NULL: all 1)
 *   y = v in the rows' type (optional), and/or its row codes q [rows, P(d)]
 *       (dense) with scale [B(d), ld_scale]: the left operand of ctr_fp8_matmul,
 *       as ctr_fp8_quantize_rows would write it for v
 * s is written where it is wanted (the stream's new value).  x, residual, s and
 * y are [rows, d] of `dtype`; gamma is fp32 [d].  s and y may be x or residual
 * themselves (the same rows and stride); nothing else may overlap.  One of y and
 * q is needed; q and scale go together.  eps > 0.  Squares that leave fp32's
 * range do not: such a row is summed again with scaled values.  A row with a NaN
 * or an infinity gets what the formula gives (NaN among it), other rows do not
 * see it.  d up to CTR_MAX_NORM_WIDTH.
 * Workspace: of ctr_rms_norm_workspace_size(rows, d) bytes ctr_rms_norm takes the
 * first 256 alone, ctr_rms_norm_bwd all of them for dgamma. */
#define CTR_MAX_NORM_WIDTH 16384
size_t ctr_rms_norm_workspace_size(int64_t rows, int32_t d);
int ctr_rms_norm(const void* x, ctr_dtype dtype, int64_t rows, int32_t d, int64_t ldx, const void* residual,
                 int64_t ld_residual, const float* gamma, float eps, void* s, int64_t ld_s, void* y, int64_t ld_y,
                 uint8_t* q, float* scale, int64_t ld_scale, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* Its gradient.  With u = s / sqrt(mean(s^2) + eps), g = dy gamma and ds the
 * gradient that arrives on the stream (optional):
 *   dx = ds + (g - u mean(g u)) / sqrt(mean(s^2) + eps)
 * the gradient of s, and so of x and of the residual; in the rows' type.
 *   dgamma = sum over rows of dy u     (fp32 [d]; optional; zeros of no rows)
 * in a fixed order.  s is what the forward wrote (x without a residual), gamma
 * and eps as there.  dx may be dy, ds or s themselves. */
int ctr_rms_norm_bwd(const void* dy, ctr_dtype dtype, int64_t rows, int32_t d, int64_t ld_dy, const void* ds,
                     int64_t ld_ds, const void* s, int64_t ld_s, const float* gamma, float eps, void* dx,
                     int64_t ld_dx, float* dgamma, void* ws, size_t ws_bytes, ctr_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Allocation-free dedup (no counterpart in the paper)                       */
/* ------------------------------------------------------------------------ */
/* ctr_dedup for callers that may not allocate device memory on this path: a
 * plugin inside a runtime that owns every device allocation, a server whose
 * memory budget is fixed at start-up, or a latency-critical loop where an
 * allocation could stall the device.  Same inputs and outputs as ctr_dedup,
 * but the scratch space is a fixed array inside the library (48 MB per GPU
 * that loads the library, held until exit) instead of a caller workspace.
 *   n_ids            at most 1048576 (2^20), for any total row count (the
 *                    array covers the largest scratch ctr_dedup_workspace_size
 *                    gives at 2^20 IDs, 46 MB at total rows = 64 x 2^20);
 *                    larger calls return CTR_ERR_UNSUPPORTED and launch
 *                    nothing.
 *   device_status    optional device int32: receives this call's device-side
 *                    error code (0, CTR_ERR_INDEX_OUT_OF_RANGE or
 *                    CTR_ERR_BAD_OFFSETS) once the call's work has run.
 * All calls share the array and it keeps the previous call's contents; its
 * error word is cleared at the start of every call.  Calls that overlap on
 * the GPU race on the array: order them (one stream, or explicit events).
 * The first call on a device looks up the array's address with that device
 * current and caches it; make that first call before any stream capture, and
 * do not call this entry point on a device again after cudaDeviceReset in the
 * same process (the cached address belongs to the old context).
 * Nothing here calls cudaMalloc, cudaFree or any other allocator. */
int ctr_dedup_static(const int64_t* ids, const int64_t* offsets, int32_t num_fields, int32_t batch,
                     const int32_t* bag_to_table, const int64_t* row_base, int32_t num_tables, int64_t n_ids,
                     int64_t* unique_rows, int64_t* n_unique, int32_t* inverse, int32_t* sorted_pos,
                     int32_t* sorted_bag, int32_t* run_offsets, int64_t* unique_offsets, int32_t* device_status,
                     ctr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CTR_H */
