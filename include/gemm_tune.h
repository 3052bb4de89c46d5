/*
 * gemm_tune.h -- C ABI of the shape-keyed autotuned matmul for MI355X (gfx950).
 *
 * The library computes C = op(A) * op(B) on one GPU with hand-written HIP
 * kernels and picks, per tuning key, the fastest of its candidate kernels by
 * measuring them on the device.  The design follows the matmul autotuner of
 * the Burn book's "autotune" page (tuning key with power-of-two buckets and
 * alignment factors; candidates ordered by group and priority; roofline time
 * bound; adaptive benchmark; winners cached in memory and on disk with a
 * checksum of the candidate list) and the result-file format and control
 * surface of the PyTorch TunableOp guide (validator lines, enable vs tuning
 * switches, max tuning duration and iterations, rotating buffers, read/write
 * file).  The kernels are this library's own.
 *
 * Conventions for every entry point
 *   - All matrices are row-major.  A layout names the storage of lhs then rhs:
 *     N = stored as used (A is M x K, B is K x N), T = stored transposed
 *     (A stored K x M, B stored N x K).  The output C is M x N.  "NT" is
 *     the case of the "cubecl-backend" page's worked example, a product with
 *     the transposed view of a matrix, read in place with no copy.
 *   - Leading dimensions are in elements; a value <= 0 selects the dense
 *     default (lhs: K for N, M for T; rhs: N for N, K for T; out: N).
 *   - Operand, output and workspace pointers are device pointers owned by the
 *     caller, who keeps them alive until the work on the stream is done.  The
 *     library never frees them.  It owns its tuning tables, the measured
 *     device peaks, a split-K workspace per device (grown on demand, kept
 *     until the process ends or gt_reset) and, during a tune only, rotating
 *     copies of the inputs and a scratch output.
 *   - Nothing throws across this boundary.  Every entry point returns a
 *     gt_status; gt_last_error() gives a message for the calling thread.
 *   - Thread safety: every entry point may be called from any thread.  A tune
 *     of one key blocks only the other callers of that key.
 *   - Degenerate shapes: M == 0 or N == 0 is a no-op; K == 0 writes zeros
 *     (the empty sum) to C.  Neither builds a key.
 */
#ifndef GEMM_TUNE_H
#define GEMM_TUNE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gt_status {
  GT_OK = 0,
  GT_ERR_INVALID_ARG = 1, /* null pointer, negative dim, ld too small, bad enum    */
  GT_ERR_UNSUPPORTED = 2, /* input/output type combination the library lacks        */
  GT_ERR_HIP = 3,         /* a HIP runtime call failed (message in gt_last_error)   */
  GT_ERR_NOT_FOUND = 4,   /* tune_lookup: no entry for this key                      */
  GT_ERR_IO = 5,          /* results file cannot be read or written                 */
  GT_ERR_VALIDATION = 6,  /* results file rejected by its validator lines           */
  GT_ERR_OOM = 7,         /* device memory exhausted                                */
  GT_ERR_NO_DEVICE = 8    /* no usable GPU                                          */
} gt_status;

/* Element types.  Inputs: all four.  Outputs: f32, f16, bf16. */
typedef enum gt_dtype { GT_F32 = 0, GT_F16 = 1, GT_BF16 = 2, GT_FP8_E4M3 = 3 } gt_dtype;

/* Storage of (lhs, rhs); see the conventions above. */
typedef enum gt_layout { GT_NN = 0, GT_NT = 1, GT_TN = 2, GT_TT = 3 } gt_layout;

/* Full problem description for gemm_tuned_ex and the query entry points.
 * out_dtype < 0 selects the default: the input type for f32/f16/bf16, f32
 * for fp8.  scale_a / scale_b are the per-tensor scales of fp8 inputs
 * (C = (acc * scale_a) * scale_b); they are ignored for other inputs.
 * stream is a hipStream_t; NULL means the stream set by gt_set_stream (the
 * default stream if none was set).  ldc is the output's leading dimension. */
typedef struct gt_gemm_desc {
  const void* lhs;
  const void* rhs;
  void* out;
  int64_t M, N, K;
  int64_t lda, ldb, ldc;
  int32_t layout;    /* gt_layout */
  int32_t in_dtype;  /* gt_dtype  */
  int32_t out_dtype; /* gt_dtype, or -1 for the default */
  float scale_a, scale_b;
  void* stream;
} gt_gemm_desc;

/* Packed tuning key: u32 m, n, k (bucketed, little endian), then one byte
 * each for lhs_pow2, lhs_stride, rhs_pow2, rhs_stride, elem_lhs, elem_rhs,
 * elem_out, layout_lhs, layout_rhs, scale, kind; the rest is zero. */
typedef struct gt_key {
  uint8_t bytes[32];
} gt_key;

/* Counters since the last gt_reset (launches are counted per kind, the way
 * the "autotune" page counts its cold run's launches). */
typedef struct gt_stats {
  uint64_t calls;             /* gemm_tuned / gemm_tuned_ex calls                    */
  uint64_t hits;              /* key found in the in-memory table                    */
  uint64_t misses;            /* key not found                                       */
  uint64_t tunes;             /* keys tuned                                          */
  uint64_t launches_probe;    /* peak / bandwidth / launch-overhead probe launches   */
  uint64_t launches_bench;    /* candidate launches while tuning (warm-up included)  */
  uint64_t launches_winner;   /* launches of a table entry on the caller's output    */
  uint64_t launches_fallback; /* launches of the naive kernel as a fallback          */
  uint64_t cands_measured;    /* candidates that produced at least one sample        */
  uint64_t cands_failed;      /* candidates that failed to launch or time            */
  uint64_t cands_eliminated;  /* candidates dropped for being > 1.5x the best        */
  uint64_t cands_not_run;     /* candidates of the set that no round reached         */
  uint64_t rows_loaded;       /* results-file rows accepted                          */
  uint64_t rows_skipped;      /* results-file rows ignored (stale checksum, garbage) */
  double last_tune_s;         /* wall time of the last tune (probes included)        */
  double total_tune_s;        /* wall time of all tunes                              */
  double last_limit_s;        /* time bound of the last tune                         */
  int32_t last_winner;        /* candidate index chosen by the last tune             */
  int32_t last_set_size;      /* candidates in the set of the last tune              */
  uint64_t cands_mismatch;    /* candidates dropped by the numerical check           */
  uint64_t wildcard_hits;     /* untuned calls served by a wildcard entry            */
  uint64_t launches_flush;    /* instruction-cache flush launches while tuning       */
} gt_stats;

/* Candidate description (for tests and reports). */
typedef struct gt_candidate_info {
  const char* name;
  int32_t group;  /* 0 naive, 1 gemv, 2 tile                                  */
  int32_t layout; /* gt_layout the kernel is built for; -1 any; -2 rhs stored
                     as is, lhs either (GEMV); -3 rhs stored transposed, lhs
                     either (GEMV)                                           */
  int32_t BM, BN, BK, waves, stages;
  int32_t splitk;    /* k-slices (1 = none; 0 = chosen at launch)            */
  int32_t va_bytes;  /* alignment its lhs loads need (bytes), 0 = none      */
  int32_t vb_bytes;  /* alignment its rhs loads need (bytes), 0 = none      */
  int32_t rows;      /* gemv: most rows it handles                           */
  int32_t lds_bytes; /* shared memory it uses                                */
} gt_candidate_info;

/* ---- the hot path ------------------------------------------------------- */

/* C = op(A) * op(B) with dense leading dimensions, output type = input type
 * (f32 for fp8 inputs, scales 1), on the stream set by gt_set_stream and the
 * current device.  On a key seen before this is a table lookup plus one
 * launch of the winner; on a new key (tuning enabled) it tunes first, which
 * synchronises the stream.  With tuning disabled a new key runs the naive
 * kernel.  Once the arguments are valid the call returns GT_OK unless HIP
 * itself fails: candidate failures fall back, the last fallback being the
 * naive kernel, which takes any shape, layout and alignment. */
gt_status gemm_tuned(const void* lhs, const void* rhs, void* out, int64_t M, int64_t N, int64_t K,
                     gt_layout layout, gt_dtype dtype);

/* Same with every option of gt_gemm_desc. */
gt_status gemm_tuned_ex(const gt_gemm_desc* d);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * call as gemm_tuned_ex, except that it allocates nothing.  It never tunes:
 * a key with a table entry (tuned, or loaded from a results file) runs its
 * winner; a miss runs what a miss with tuning off runs (the zero-search
 * default of option "untuned").  Every workspace it needs (GEMV slice
 * counters, split-K partial sums, transposed operand copies) comes from one
 * fixed device array per GPU of 64 MiB, held from the first call on that GPU
 * until the process ends.  That first call looks up the array's address and
 * clears its counter region with a kernel on the call's stream; make it
 * outside stream capture.  Errors: as gemm_tuned_ex, plus GT_ERR_INVALID_ARG
 * (nothing launched) when the chosen candidate needs more than 64 MiB of
 * workspace for this problem.  Calls on one GPU share the array: calls that
 * overlap in time on that GPU (other streams, other threads) race on it and
 * must be ordered by the caller. */
gt_status gemm_tuned_noalloc(const gt_gemm_desc* d);

/* The tuning key of a problem: the packed key and its compact text (the form
 * used in the results file).  Either output may be NULL.  Host only. */
gt_status gt_make_key(const gt_gemm_desc* d, gt_key* key, char* text, size_t text_len);

/* The key in the "autotune" page's print style (layout printed as
 * "MildlyPermuted { transposed: true, batch_swap: false }").  Host only. */
gt_status gt_key_display(const gt_gemm_desc* d, char* text, size_t text_len);

/* Look up the current device's table without tuning.  GT_ERR_NOT_FOUND on a
 * miss.  Any output pointer may be NULL.  *median_us is the winner's
 * measured median per launch (NaN if the row carried none). */
gt_status tune_lookup(const gt_gemm_desc* d, int* cand_index, char* cand_name, size_t name_len,
                      double* median_us);

/* Write every entry of the current device's table (and its measured peaks)
 * to a results file: validator lines, then one row per key.  The file is
 * written to a temporary name and renamed into place.  path NULL: the file
 * named by the option "cache_file" (env GT_CACHE_FILE). */
gt_status tune_save(const char* path);

/* The results-file text of the current device's table, as tune_save would
 * write it with no file there before: validator lines ("Validator,<name>,
 * <value>"), measured peaks ("Throughput,..."), then one "GemmTuned,<key>,
 * <candidate>,<median us>,<checksum>" row per key (the TunableOp guide's
 * get_results and get_validators, section 7.2, read from memory).  Writes at
 * most text_len bytes, NUL-terminated and cut short if it does not fit;
 * *needed = the whole text's length + 1.  text may be NULL when text_len is
 * 0 (a size query).  The caller owns both buffers. */
gt_status tune_results(char* text, size_t text_len, size_t* needed);

/* Read a results file into the current device's table.  A missing or
 * different validator rejects the whole file (GT_ERR_VALIDATION, nothing
 * loaded).  Rows whose candidate-list checksum differs from the current one,
 * that name an unknown candidate, or do not parse, are skipped and counted.
 * Entries already in memory are kept.  path NULL: option "cache_file". */
gt_status tune_load(const char* path);

/* Offline tuning of recorded problems (the record-then-tune timeline of the
 * TunableOp guide, section 6, and the offline, shipped results file of the
 * "autotune end to end" page).  With option record_untuned=1 and tuning off,
 * the first problem of every key that misses is appended to option
 * untuned_file as
 *   GemmUntuned,<compact key>,<in type>,<out type>,<layout>,M,N,K,lda,ldb,ldc,<A addr % 256>,<B addr % 256>
 * gt_tune_file reads such a file and, on the current device, tunes every
 * recorded problem whose key (at the current key level) has no entry yet:
 * device operands of the recorded shape, leading dimensions and alignment
 * are allocated, filled with seeded synthetic values (uniform in [-1, 1);
 * fp8 of magnitude at most 3.75), tuned exactly as a miss with tuning on
 * would be (whatever the "tuning" switch says), and freed.  Then the whole
 * table is written as a results file to results_path (NULL: option
 * cache_file; no file when that is empty too), for a serving process to
 * load (option cache_file, read on its first miss even with tuning off, or
 * tune_load).  Counts go to *report (may be NULL).  Errors: GT_ERR_INVALID_ARG
 * for a NULL untuned_path, GT_ERR_IO when it cannot be read or the results
 * file cannot be written, GT_ERR_HIP when a launch or copy fails (the pass
 * stops there; the results file is not written).  A row that does not parse,
 * or whose operands do not fit in device memory, is skipped and counted. */
typedef struct gt_tune_file_report {
  int64_t rows;    /* GemmUntuned rows read                                  */
  int64_t tuned;   /* keys tuned by this call                               */
  int64_t present; /* rows whose key already had an entry (or came earlier) */
  int64_t skipped; /* rows that did not parse or fit                        */
} gt_tune_file_report;
gt_status gt_tune_file(const char* untuned_path, const char* results_path, gt_tune_file_report* report);

/* ---- operators around the product --------------------------------------- */

/* What a language model runs directly before and around a product of this
 * library: the RMS norm with the residual's addition, whose output is a
 * product's left operand (e4m3 with its scales included), that norm's
 * backward pass, the product of a few rows with 4-bit weights, and the
 * expansion of such weights into a right operand of gemm_tuned.
 *
 * They follow the conventions above (row-major, leading dimensions in
 * elements with <= 0 for dense, caller-owned device pointers, the stream of
 * the descriptor or of gt_set_stream, every failure a gt_status).  No table
 * and no tuning is involved; nothing is launched when a check fails.
 * Pointers must be aligned to their element.  Inputs and outputs must not
 * overlap, except where a descriptor says so.  Results do not depend on the
 * order in which workgroups run: equal inputs give equal bits. */

/* How gt_rmsnorm's output is stored in 8 bits (e4m3, round to nearest even):
 * not at all; over one given scale, saturating at +-448; or over a scale per
 * row, max(max |y|, 2^-100) / 448, which the call writes. */
typedef enum gt_quant { GT_QUANT_NONE = 0, GT_QUANT_TENSOR = 1, GT_QUANT_ROW = 2 } gt_quant;

/* h = x + residual, rstd[m] = 1 / sqrt(mean_n h[m,n]^2 + eps),
 * y = h * rstd * (weight + weight_offset), all in fp32 and rounded once.
 * sum_out receives h rounded to in_dtype (the norm itself uses the unrounded
 * h).  Elements whose squares sum past fp32's range (about 1e19 each) give
 * rstd 0.  A product of the stored e4m3 rows takes the scale back as scale_a
 * (GT_QUANT_TENSOR, gemm_tuned_ex) or row_scale (GT_QUANT_ROW,
 * gt_w4_matmul); gemm_tuned_ex takes no scale per row. */
typedef struct gt_rmsnorm_desc {
  const void* x;        /* M x N, ldx                                        */
  const void* residual; /* M x N, ldr, or NULL                               */
  const void* weight;   /* N, or NULL for y = h * rstd                       */
  void* sum_out;        /* M x N, lds, or NULL; may be x or residual itself
                           (same leading dimension)                          */
  void* y;              /* M x N, ldy; may be x itself (same type and ld)    */
  float* rstd;          /* M, or NULL                                        */
  float* row_scale;     /* M; required by and only used with GT_QUANT_ROW    */
  int64_t M, N;         /* N <= 65536                                        */
  int64_t ldx, ldr, lds, ldy;
  int32_t in_dtype;     /* f32, f16, bf16: x, residual, sum_out              */
  int32_t weight_dtype; /* f32, f16, bf16; -1: in_dtype                      */
  int32_t out_dtype;    /* f32, f16, bf16, or e4m3 with a gt_quant; -1: e4m3
                           with a gt_quant, in_dtype without                 */
  int32_t quant;        /* gt_quant                                          */
  float eps;            /* finite, >= 0                                      */
  float weight_offset;  /* 0, or 1 where weights are stored less one         */
  float scale;          /* GT_QUANT_TENSOR: finite, > 0                      */
  void* stream;
} gt_rmsnorm_desc;

/* GT_ERR_INVALID_ARG: NULL x or y, a bad enum, dimension, leading dimension,
 * eps or scale, a misaligned pointer, e4m3 output without a gt_quant (or the
 * reverse), GT_QUANT_ROW without row_scale.  GT_ERR_UNSUPPORTED: e4m3 inputs
 * or weights, N > 65536.  M == 0 or N == 0 is a no-op. */
gt_status gt_rmsnorm(const gt_rmsnorm_desc* d);

/* The gradients of y = h * rstd * (weight + weight_offset), given dy, the h
 * and the rstd of the forward pass: with g = dy * (weight + weight_offset)
 * and n = h * rstd,
 *   dx = rstd * (g - n * mean_n(g * n)) + dsum,  dweight = sum_m dy * n.
 * dx is the gradient of x and of the residual alike; dsum is the gradient
 * that reaches h past the norm (sum_out's other uses).  dweight is summed
 * in fp32 in a fixed order; its partial sums may take a workspace of the
 * stream, which the first (largest) call allocates: make that call outside
 * stream capture. */
typedef struct gt_rmsnorm_bwd_desc {
  const void* dy;       /* M x N, lddy                                       */
  const void* h;        /* M x N, ldh: sum_out, or x without a residual      */
  const void* weight;   /* N, or NULL                                        */
  const float* rstd;    /* M                                                 */
  const void* dsum;     /* M x N, ldds, or NULL                              */
  void* dx;             /* M x N, lddx, or NULL; may be dy, h or dsum itself
                           (same type and leading dimension)                 */
  void* dweight;        /* N, or NULL                                        */
  int64_t M, N;         /* N <= 65536                                        */
  int64_t lddy, ldh, ldds, lddx;
  int32_t in_dtype;      /* f32, f16, bf16: h, dsum, dx                      */
  int32_t dy_dtype;      /* in_dtype or f32; -1: in_dtype                    */
  int32_t weight_dtype;  /* f32, f16, bf16; -1: in_dtype                     */
  int32_t dweight_dtype; /* f32, f16, bf16; -1: f32                          */
  float weight_offset;
  void* stream;
} gt_rmsnorm_bwd_desc;

/* GT_ERR_INVALID_ARG: NULL dy, h or rstd, neither dx nor dweight, and as
 * gt_rmsnorm; also when the workspace would have to grow while the stream is
 * being captured.  GT_ERR_OOM: no memory for the workspace.  M == 0 writes
 * zeros to dweight; N == 0 is a no-op. */
gt_status gt_rmsnorm_backward(const gt_rmsnorm_bwd_desc* d);

/* 4-bit weights: row n holds weight (n, k) in byte k / 2, the even k in the
 * low nibble; (K + 1) / 2 bytes a row, rows ldq bytes apart.  A nibble is a
 * two's complement integer (-8..7), or an e2m1 float (sign, then 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6).  Every `group` of consecutive k in a row shares a scale:
 * weight = scale * value, so integers are symmetric (there are no zero
 * points), and groups are of 32, 64 or 128 (neither 16 nor a whole row, nor k
 * in another order). */
typedef enum gt_w4_format { GT_W4_INT4 = 0, GT_W4_E2M1 = 1 } gt_w4_format;

/* y[m,n] = x_scale * row_scale[m] * sum_k x[m,k] * weight[n,k]: a product
 * with a transposed right operand (GT_NT) for a few rows, as one token or a
 * decode batch has.  The nibbles are expanded exactly, the products are
 * summed per group in fp32 and the scales applied to the fp32 sums (so a sum
 * of x * value past 2^128 is infinite, whatever its scale).  Any M
 * is taken, up to 256 rows at a time; from 64 to 96 rows on gemm_tuned is
 * faster with expanded weights that the program keeps (8192 x 8192: 25 and 32
 * us for 64 rows, 41 and 35 for 96), from 256 to 512 rows on also with a
 * gt_w4_expand in each call.  A long K may take a workspace of the stream, as
 * above, for at most 64 MiB of partial sums: a call that has more runs over
 * fewer rows or columns at a time. */
typedef struct gt_w4_desc {
  const void* x;          /* M x K, ldx                                      */
  const float* row_scale; /* M, or NULL                                      */
  const void* qweight;    /* N x K in 4 bits, ldq bytes (<= 0: (K + 1) / 2)  */
  const void* scales;     /* N x ceil(K / group): (n, g) at
                             n * scale_ldn + g * scale_ldg                   */
  void* y;                /* M x N, ldy                                      */
  int64_t M, N, K;
  int64_t ldx, ldq, ldy;
  int64_t scale_ldn, scale_ldg; /* elements; <= 0: ceil(K / group) and 1     */
  int32_t x_dtype;     /* f16, bf16, e4m3                                    */
  int32_t out_dtype;   /* f32, f16, bf16; -1: x_dtype, f32 for e4m3          */
  int32_t format;      /* gt_w4_format                                       */
  int32_t scale_dtype; /* f32, f16, bf16                                     */
  int32_t group;       /* 32, 64 or 128                                      */
  float x_scale;       /* 1, or the scale of e4m3 rows                       */
  void* stream;
} gt_w4_desc;

/* GT_ERR_INVALID_ARG: a NULL operand, a bad enum, dimension, leading
 * dimension or group, a misaligned pointer; also when a workspace would have
 * to grow while the stream is being captured.  GT_ERR_UNSUPPORTED: f32 rows,
 * e4m3 output or scales.  GT_ERR_OOM: no memory for the workspace.  M == 0 or
 * N == 0 is a no-op; K == 0 writes zeros. */
gt_status gt_w4_matmul(const gt_w4_desc* d);

/* out[n,k] = weight (n, k) as an fp32 product (exact unless the scales are
 * fp32), rounded to out_dtype: N x K row-major, the right operand of a GT_NT
 * product.  There is no e4m3 output. */
typedef struct gt_w4_expand_desc {
  const void* qweight;
  const void* scales;
  void* out;           /* N x K, ldo                                         */
  int64_t N, K;
  int64_t ldq, ldo, scale_ldn, scale_ldg;
  int32_t out_dtype;   /* f32, f16, bf16                                     */
  int32_t format;
  int32_t scale_dtype;
  int32_t group;
  void* stream;
} gt_w4_expand_desc;

/* Errors as gt_w4_matmul.  N == 0 or K == 0 is a no-op. */
gt_status gt_w4_expand(const gt_w4_expand_desc* d);

/* ---- experts and adapters beside the product ---------------------------- */

/* What a batch of requests meets beside the shared products: the choice of
 * experts from a router's logits (a product of gemm_tuned), a whole layer of
 * gated experts for a few tokens, and the low-rank adapters that requests
 * bring to a shared projection.  All are in the manner of the operators
 * above.  Indices are int32 in device memory, where the host cannot check
 * them: one outside its range means "none" and is never followed. */
typedef enum gt_score { GT_SCORE_SOFTMAX = 0, GT_SCORE_SIGMOID = 1 } gt_score;

/* For every row the topk experts of the largest logits, in descending order,
 * equal logits by ascending index, and their weights:
 *   softmax: exp(l_i) / sum exp(l), over all experts, or over the chosen ones
 *            with normalise;
 *   sigmoid: 1 / (1 + exp(-l_i)), over their sum with normalise;
 * times scale, in fp32.  A logit of -infinity masks its expert: it is never
 * chosen, and slots for which none is left get index -1 and weight 0.  A NaN
 * ranks above every number and its weight, with a softmax or normalise all
 * weights of its row, are NaN (as +infinity's are with a softmax). */
typedef struct gt_route_desc {
  const void* logits; /* M x E, ldl                                          */
  int32_t* index;     /* M x topk, ldi                                       */
  float* weight;      /* M x topk, ldw                                       */
  int64_t M, E, topk; /* topk <= E <= 1024, topk <= 64                       */
  int64_t ldl, ldi, ldw;
  int32_t dtype;     /* f32, f16, bf16                                       */
  int32_t score;     /* gt_score                                             */
  int32_t normalise; /* 0 or 1                                               */
  float scale;       /* finite                                               */
  void* stream;
} gt_route_desc;

/* GT_ERR_INVALID_ARG: NULL operands, a bad enum, dimension, leading dimension
 * or scale, topk outside 1..E, a misaligned pointer.  GT_ERR_UNSUPPORTED:
 * e4m3 logits, E > 1024, topk > 64.  M == 0 is a no-op. */
gt_status gt_route(const gt_route_desc* d);

/* How weights of experts are stored: 16 bits as the rows, or 4 bits with
 * group scales as gt_w4_matmul's (gt_w4_format's two). */
#define GT_WEIGHTS_16BIT (-1)
typedef enum gt_activation { GT_ACT_SILU = 0, GT_ACT_GELU = 1 /* its tanh form */ } gt_activation;

/* A layer of gated experts: with e = index[t,j],
 *   y[t] = base[t] + sum_j weight[t,j] * down_e (act(gate_e x[t]) * (up_e x[t]))
 * Each expert's gate_up holds the H rows of gate, then the H rows of up, K
 * long; its down holds K rows of H.  Sums, activations and what passes
 * between the products are fp32.  Where tokens share experts the down product
 * takes them in 16-bit parts that hold all of a value (bf16 experts) or at least
 * 22 bits of it beside the row's largest; 16 bits only below a 16-bit y, where
 * bf16 experts have 16 rows or more on average.  y is rounded once.  A token may
 * name an expert twice; a slot whose index is outside 0..E-1 adds nothing.  x may
 * be y itself (same type and leading dimension); else they must not overlap.
 *
 * The weights of the experts that are named are read once for up to 16 of
 * their rows (64 where 16-bit experts have 16 rows or more on average; for each
 * row where up to 8 tokens hardly share experts, and where a row of weights has
 * less than 16 bytes or rows are 2^27 bytes apart), so this is for the few
 * tokens of a decode batch: any M is taken, in ranges of tokens whose
 * intermediate values take about 64 MiB (one token's activations, topk * H
 * floats, may be more), but a prompt's rows belong in one product per expert.
 *
 * The intermediate values take gt_moe_workspace bytes of device memory (fewer
 * tokens may take more than many, whose sums are cut into fewer slices: ask
 * for each M): the caller's workspace (16-byte aligned), or, where that is
 * NULL, the stream's, which a call that needs more than those before
 * allocates: make one of the same sizes outside stream capture first.  Calls
 * and graph replays that overlap in time must not share a workspace: graphs
 * captured on one stream and replayed on several need the caller's, one each. */
typedef struct gt_moe_desc {
  const void* x;              /* M x K, ldx                                  */
  const int32_t* index;       /* M x topk, ldi                               */
  const float* weight;        /* M x topk, ldw                               */
  const void* gate_up;        /* E matrices of 2 H x K, rows gate_up_ld      */
  const void* gate_up_scales; /* 4 bits: (e, n, g) at e * _lde + n * _ldn + g * _ldg */
  const void* down;           /* E matrices of K x H, rows down_ld           */
  const void* down_scales;    /* magnitudes up to 2^100, or infinite         */
  const void* base;           /* M x K, ldb, of y's type, or NULL; may be y
                                 itself (same leading dimension)             */
  void* y;                    /* M x K, ldy                                  */
  void* workspace;            /* or NULL                                     */
  int64_t workspace_bytes;
  int64_t M, K, H, E, topk;   /* E <= 4096, topk <= 64, K and H <= 2^24      */
  int64_t ldx, ldi, ldw, ldb, ldy;
  int64_t gate_up_ld, gate_up_stride; /* of rows and of experts, in elements */
  int64_t down_ld, down_stride;       /* (4 bits: bytes); <= 0: dense        */
  int64_t gate_up_scale_lde, gate_up_scale_ldn, gate_up_scale_ldg; /* elements; <= 0: _ldn the groups of a row, _ldg 1,
                                 _lde rows * _ldn or, if that is more, groups * _ldg */
  int64_t down_scale_lde, down_scale_ldn, down_scale_ldg;
  int32_t x_dtype;     /* f16, bf16: x, and 16-bit weights                   */
  int32_t out_dtype;   /* f32, f16, bf16; -1: x_dtype                        */
  int32_t format;      /* GT_WEIGHTS_16BIT or a gt_w4_format                 */
  int32_t scale_dtype; /* f32, f16, bf16 (4 bits)                            */
  int32_t group;       /* 32, 64 or 128 (4 bits)                             */
  int32_t activation;  /* gt_activation                                      */
  void* stream;
} gt_moe_desc;

/* GT_ERR_INVALID_ARG: a NULL operand, a bad enum, dimension, leading
 * dimension, stride or group, a misaligned pointer, a workspace that is too
 * small; also when the stream's would have to grow while the stream is being
 * captured.  GT_ERR_UNSUPPORTED: f32 or e4m3 rows, e4m3 output or scales, E >
 * 4096, topk > 64, K or H > 2^24.  GT_ERR_OOM: no memory for the workspace.  M == 0 or K ==
 * 0 is a no-op; H, E or topk == 0 leaves y = base (zeros without one). */
gt_status gt_moe(const gt_moe_desc* d);
/* The workspace's bytes (0 for none); pointers are not looked at, the weights'
 * strides are. */
gt_status gt_moe_workspace(const gt_moe_desc* d, int64_t* bytes);

/* Adapters of many requests beside a shared projection: with a = index[m],
 *   y[m] = base[m] + scale[a] * b_a (a_a x[m])
 * where a_a is rank x K and b_a is N x rank (smaller ranks are padded with
 * zeros).  base is the projection's own result, y itself to add in place (x
 * must not overlap y: all of a row is read for each of its results); a
 * row without an adapter (an index outside 0..adapters-1) is left as base, not
 * written at all in place.  Sums and what passes between the products are
 * fp32 (in the second 16-bit parts that hold all of it, or at least 22 bits of
 * it with f16 rows, as gt_moe); y is rounded once.
 * An adapter's b is read once for up to 16 of its rows, its a once a row or, in
 * larger calls, for up to 16 or 64 rows; a few rows of small matrices read b once
 * a row and a once for 1024 columns of each.  Workspace as gt_moe, asked for also
 * where the kernel that the sizes get leaves it alone. */
typedef struct gt_lora_desc {
  const void* x;        /* M x K, ldx                                        */
  const int32_t* index; /* M                                                 */
  const void* a;        /* adapters of rank x K, rows a_ld, matrices a_stride */
  const void* b;        /* adapters of N x rank, rows b_ld, matrices b_stride */
  const float* scale;   /* adapters, or NULL for 1                           */
  const void* base;     /* M x N, ldb, of y's type, or NULL; may be y itself */
  void* y;              /* M x N, ldy                                        */
  void* workspace;      /* or NULL                                           */
  int64_t workspace_bytes;
  int64_t M, K, N, adapters, rank; /* adapters <= 4096, rank <= 256, K and N <= 2^24 */
  int64_t ldx, ldb, ldy;
  int64_t a_ld, a_stride, b_ld, b_stride; /* elements; <= 0: dense           */
  int32_t x_dtype;   /* f16, bf16: x, a and b                                */
  int32_t out_dtype; /* f32, f16, bf16; -1: x_dtype                          */
  void* stream;
} gt_lora_desc;

/* Errors as gt_moe, and GT_ERR_INVALID_ARG where y is x (GT_ERR_UNSUPPORTED: adapters > 4096, rank > 256, K or N >
 * 2^24).  M == 0 or N == 0 is a no-op; K, adapters or rank == 0 leaves y = base. */
gt_status gt_lora(const gt_lora_desc* d);
gt_status gt_lora_workspace(const gt_lora_desc* d, int64_t* bytes);

/* ---- control ------------------------------------------------------------ */

/* Enable or disable tuning on a miss (the enable-vs-tuning split of the
 * TunableOp guide: lookups still hit when tuning is off, and the first miss
 * on a device reads the results file named by option cache_file either way).
 * A miss with tuning off runs the zero-search default of option "untuned"
 * (below). */
gt_status gt_set_tuning(int enabled);

/* The candidate a miss with tuning off runs under untuned=heuristic, for the
 * problem *desc on the current device, without launching anything: the one
 * with the smallest analytic time estimate (a roofline per candidate family
 * with the quantisation of blocks over the CUs, the k-split's reduction and
 * the transposes' extra pass) among those the problem's key and operand
 * alignment allow; 0 (the naive kernel) when none is left.  This is the
 * "heuristic default on a miss" of the TunableOp guide and the pages'
 * zero-search designs.  GT_ERR_INVALID_ARG for a NULL cand_index, a desc
 * that does not validate, or an empty problem (M, N or K zero). */
gt_status gt_default_candidate(const gt_gemm_desc* desc, int* cand_index);

/* Default stream (hipStream_t) for gemm_tuned and for descs with a NULL
 * stream.  NULL restores the default stream. */
gt_status gt_set_stream(void* stream);

/* Set an option by name; every option is also read once from the
 * environment variable GT_<NAME uppercased> when the library first runs.
 *   tuning           0|1 (1)          tune on a miss
 *   untuned          heuristic|naive  what a miss runs with tuning off: the
 *                                     analytic pick (gt_default_candidate,
 *                                     kept per key) or the naive kernel
 *                                     (heuristic)
 *   level            minimal|balanced|extensive|full  key bucketing level:
 *                                     m, n, k rounded up to the next power of
 *                                     2.5 / 2 / 1.5 (as an integer), or kept
 *                                     (balanced)
 *   wildcard_dims    "" or letters of "mnk" (""): each tuned winner is also
 *                    stored under its key with those dimensions as "*"; a
 *                    miss with tuning off then tries the stored wildcard
 *                    entries (one dimension, then two, then all three) whose
 *                    candidate can run the problem, before the default
 *   tune_mode        adaptive|exhaustive  exhaustive: no early stop, no
 *                                     elimination, every candidate timed
 *   max_tuning_ms    per-candidate measured-time budget (30)
 *   max_tuning_iters per-candidate launch budget (100)
 *   warmup_ms / warmup_iters          extra untimed launches (0 / 0)
 *   rotating_mb      MiB of input copies rotated while tuning (512; 0 =
 *                    none; < 0 = the device's reported L2 size, the TunableOp
 *                    guide's default, section 7.1; reads back as -1)
 *   sample_us        target length of one timed sample (500)
 *   cache_file       results file for tune_save/tune_load(NULL), read on a
 *                    device's first miss ("")
 *   cache_file_ordinal 0|1 (0)      1: each device's results file has the
 *                    device ordinal before the extension of cache_file's
 *                    name ("results.csv" -> "results0.csv", "res" -> "res0"),
 *                    so one process per GPU never shares a file (the
 *                    TunableOp guide, sections 3.1 and 7.2); explicit paths
 *                    of tune_save / tune_load are used as given
 *   save_at_exit     0|1 (0)          1: when the process exits, every
 *                                     device's table is written to its
 *                                     cache_file as tune_save(NULL) would
 *                                     (the TunableOp guide, section 3.1)
 *   cache            1: write cache_file after every tune; 0: memory only (0)
 *   log_decisions    ""|stdout|stderr|<path>  one JSON line per tune
 *   fault_inject     "<candidate name>:launch_err|no_timing|slow", ";"-joined
 *   screen2          0 or a ratio >= 1 (0 = off): second screen, a candidate
 *                    with screen2_iters timed launches is dropped when
 *                    slower than this times the best median (TunableOp's 1.15)
 *   screen2_iters    timed launches before the second screen applies (10)
 *   finalists        0 = off, else how many of the fastest candidates are
 *                    re-measured after a round, the winner re-chosen by the
 *                    mean of the new samples (the winner's-curse remedy; 5)
 *   finalist_samples samples per finalist (5)
 *   numeric_check    "" = off, else "atol_rtol" (e.g. "1e-2_1e-2"): before
 *                    timing, each candidate's output on the caller's inputs
 *                    must be within atol + rtol*|ref| of the naive kernel's,
 *                    element by element, or it is dropped
 *   icache_flush     0|1 (0)          1: before each timed launch, a kernel
 *                                     invalidates the instruction caches of
 *                                     the CUs, and each launch is timed by
 *                                     its own event pair (the flush is not
 *                                     timed); the TunableOp guide's
 *                                     instruction-cache flush (section 7.1)
 *   record_untuned   0|1 (0)          append the problems that miss with
 *                                     tuning off to untuned_file
 *   untuned_file     path ("gemm_untuned.csv")
 * Unknown names or bad values give GT_ERR_INVALID_ARG. */
gt_status gt_set_option(const char* name, const char* value);
gt_status gt_get_option(const char* name, char* value, size_t value_len);

/* Counters; gt_reset clears them and, on request, the current device's
 * in-memory table and its measured peaks. */
gt_status gt_get_stats(gt_stats* out);
gt_status gt_reset(int clear_table, int clear_probes);

/* ---- candidates (tests, reports, forced runs) --------------------------- */

/* Number of candidates for an input type (registration order = index;
 * index 0 is always the naive kernel). -1 for an unknown type. */
int gt_candidate_count(gt_dtype dtype);
/* Candidate name, or NULL when out of range.  The string lives as long as the
 * library. */
const char* gt_candidate_name(gt_dtype dtype, int index);
gt_status gt_candidate_info_get(gt_dtype dtype, int index, gt_candidate_info* info);

/* Run one named candidate on the problem (no table, no tuning).  Returns
 * GT_ERR_UNSUPPORTED (nothing launched) when the candidate cannot take this
 * problem: wrong layout, alignment, shared-memory fit or shape class. */
gt_status gemm_candidate(const gt_gemm_desc* d, int cand_index);

/* The plan for a problem: candidate indices in the order they would be
 * tried, with the round each belongs to.  *count gets the total; at most cap
 * entries are written.  Host only. */
gt_status gt_plan(const gt_gemm_desc* d, int* cands, int* rounds, int cap, int* count);

/* Roofline bound of a problem on the current device: ops = M*N*(2K-1),
 * bytes = inputs once + output once, limit = max(ops/peak_ops,
 * bytes/peak_bytes)/0.8 + launch overhead.  Runs the peak probes on a miss
 * of the measured-peak cache.  Any output may be NULL. */
gt_status gt_time_limit(const gt_gemm_desc* d, double* limit_s, double* ops, double* bytes);

/* Thread-local message of the last failure ("" if none). */
const char* gt_last_error(void);
/* Library version string (also the GT_LIB_VERSION validator). */
const char* gt_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GEMM_TUNE_H */
