/*
 * rvq.h -- C ABI of the MI355X (gfx950) residual vector quantization library.
 *
 * What the library computes.  Visual feature vectors become multi-level
 * discrete token IDs by residual vector quantization (RVQ): at each level
 * the nearest codeword of that level's codebook is chosen, its index is
 * recorded, and it is subtracted so the residual passes on to the next
 * level ("LongCat-2.5 发布：面向智能体任务的原生多模态大模型", section
 * "Visual Primitive Modeling", paragraph "Discrete Native Resolution Vision
 * Transformer"; "LongCat-2.5 Open Source Release: Meituan's 1.6T Multimodal
 * Agent Model with 1M Context", section "02 Visual Coding and 3D": detail is
 * added level by level).  Token IDs are turned
 * back into vectors by summing the chosen codewords (same blog, Figure 1:
 * the token sequences are reconstructed).  The tokenizer is fixed and its
 * IDs are precomputed offline (same blog, paragraph "Offline Visual
 * Preprocessing"), so encoding here is a deterministic, batch-invariant
 * function of (row, codebooks): a row's IDs do not depend on the other rows
 * in the call or on its position.
 *
 * Readings taken where the pages are silent: the distance is the squared
 * Euclidean distance; there is one [K][d] codebook per level; search is
 * greedy level by level; among codewords at the same distance the lower
 * index wins.
 *
 * Conventions for every entry point:
 *   - Pointers named as device pointers are device memory owned by the
 *     caller (any allocator).  The library allocates no device memory and
 *     keeps no global mutable state; scratch memory is a caller-provided
 *     workspace.  (The host-side ID cache uses short-lived host buffers, and
 *     the streaming encoder creates and destroys its own copy streams and
 *     events within the call.)
 *   - All arrays are dense and row-major.  Codebooks are [L][K][d] fp32;
 *     token IDs are [n][L] int32 (level-minor); rows are [n][d].
 *   - Work is enqueued on `stream` and the call returns without waiting.
 *     Concurrent calls on different streams must use different workspaces.
 *   - The device entry points issue only kernel launches on `stream` (no
 *     memset, copy, allocation or host synchronisation), so a caller may
 *     capture them in a HIP graph; the streaming encoder is the exception.
 *   - Arguments are validated on the host before any HIP call; a non-OK
 *     status means nothing was enqueued, except RVQ_ERR_HIP, which reports
 *     a failed launch (the stream may then hold part of the work).
 *   - n == 0 is a valid no-op (outputs of size zero; hist and msr are still
 *     written for level statistics).
 *   - Inputs must be finite; results for NaN or Inf inputs are unspecified
 *     but every memory access stays in bounds.
 */
#ifndef RVQ_H
#define RVQ_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rvq_status {
    RVQ_OK = 0,
    RVQ_ERR_INVALID_ARGUMENT = 1,   /* null pointer, bad size, misaligned pointer */
    RVQ_ERR_UNSUPPORTED = 2,        /* valid request outside what the library supports */
    RVQ_ERR_WORKSPACE_TOO_SMALL = 3,
    RVQ_ERR_HIP = 4                 /* a HIP launch failed */
} rvq_status;

typedef enum rvq_dtype {
    RVQ_F32 = 0,
    RVQ_BF16 = 1,
    RVQ_F8E4M3 = 2   /* 8 bits (4 exponent, 3 mantissa, largest 448): only where named */
} rvq_dtype;

/* Static text for a status code. */
const char *rvq_status_string(rvq_status s);

/* Detail of the last non-OK status returned on the calling host thread
 * (thread-local, overwritten by the next failing call). */
const char *rvq_last_error(void);

/* ------------------------------------------------------------------------
 * Codebook preparation (once per fixed codebook set).
 *
 * The tokenizer is fixed ("Offline Visual Preprocessing"), so per-codeword
 * data derived from the codebooks is computed once and reused by every
 * encode call: the squared norms ||c||^2 in fp32 and a bf16 copy of the
 * codewords in the layout the distance kernel reads.
 * ---------------------------------------------------------------------- */

/* Bytes of the prepared buffer for L levels of K codewords of dimension d. */
rvq_status rvq_prepared_size(int32_t L, int32_t K, int32_t d, size_t *bytes);

/*
 * codebooks : device, [L][K][d] fp32, 16-byte aligned.
 * prepared  : device, >= rvq_prepared_size bytes, 256-byte aligned.  For
 *             d <= 1280 fully overwritten; for wider rows only an fp32 copy
 *             of the codebooks with rows padded to a multiple of 16 is
 *             written (when d is not one), the only part the exact fp32
 *             encoder reads.  Owned by the caller; pass it to rvq_encode with
 *             the same codebooks, L, K and d (not checked: a buffer prepared
 *             from other codebooks gives wrong IDs, never a fault).
 */
rvq_status rvq_prepare_codebooks(const float *codebooks, int32_t L, int32_t K, int32_t d,
                                 void *prepared, size_t prepared_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Encode: greedy multi-level nearest-codeword search with residual update.
 *
 * Per level l and row r the nearest codeword under ||r - c||^2 is chosen,
 * its index recorded, and it is subtracted from the fp32 residual, which
 * feeds the next level.
 *
 * Rows of at most 1280 features: the codewords are ranked by the score
 * ||c||^2 - 2 r.c (||r||^2 is the same for every codeword), with the dot
 * products taken on the matrix cores from bf16 copies of r and c with fp32
 * accumulation.  Per row and level the encoder bounds how far this
 * screening can move a score (from the row's and the level's rounding
 * terms: the residual's and the codewords' bf16 rounding, the fp32
 * accumulation, the hi/lo split of ||c||^2 and the tag bits of the ranking
 * keys), and every codeword whose key lies within the resulting band of the
 * smallest key is rescored exactly in fp32 as sum_i (r_i - c_i)^2; the
 * smallest distance wins.  A level whose candidates cannot all be kept
 * (a crowded band) is rescanned exactly over all K codewords after the
 * distance launch.  So the nearest codeword is returned wherever it beats
 * every other by more than 1e-4 ||r||^2.  (The bound treats the rounding
 * errors of different features as independent, a reading of the typical
 * case; its Cauchy-Schwarz worst case is used where it is smaller, at
 * widths below about 25.)
 *
 * Rows of 1281 to 8192 features: every distance sum_i (r_i - c_i)^2 is
 * computed exactly in fp32 on the vector ALUs, with no screening (slower).
 *
 * On both paths, among codewords at the same fp32 distance the lower index
 * wins (duplicated codewords return the lowest index), and a row's IDs and
 * fp32 residual depend only on the row and the codebooks, not on the other
 * rows of the call or on its position.
 * ---------------------------------------------------------------------- */

/* Workspace bytes needed by rvq_encode for n rows. */
rvq_status rvq_encode_workspace_size(int64_t n, int32_t d, int32_t L, int32_t K, size_t *bytes);

/*
 * x            : device, [n][d] rows in x_dtype (fp32 or bf16), aligned to
 *                the element size; rows that do not start 16-byte aligned
 *                (e.g. a slice of a larger batch) are first copied to the
 *                workspace.
 * codebooks    : device, [L][K][d] fp32 (the exact values used for rescoring
 *                and for the residual update), 16-byte aligned.
 * prepared     : device, filled by rvq_prepare_codebooks for these codebooks.
 * ids          : device, [n][L] int32 output; ids[row*L + l] in [0, K).
 * residual_out : device, [n][d] fp32 output x - sum_l codebooks[l][ids[l]],
 *                or NULL when not wanted.  4-byte aligned (16-byte alignment
 *                can save a final copy).
 * d            : 1..8192 (RVQ_ERR_UNSUPPORTED above).  Up to 1280 a row's
 *                features stay resident in registers during the matrix-core
 *                sweep; wider rows take the exact fp32 path.  One level of
 *                codewords, K x (d rounded up to 16) fp32, must be below
 *                4 GiB (RVQ_ERR_UNSUPPORTED otherwise; the same checks apply
 *                to rvq_prepared_size, rvq_prepare_codebooks and
 *                rvq_encode_workspace_size).
 * workspace    : device, >= rvq_encode_workspace_size bytes, 256-byte
 *                aligned; contents on entry are ignored.
 */
rvq_status rvq_encode(const void *x, rvq_dtype x_dtype, int64_t n, int32_t d,
                      const float *codebooks, const void *prepared, int32_t L, int32_t K,
                      int32_t *ids, float *residual_out,
                      void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Same as rvq_encode, and additionally times the distance stage with
 * caller-created events (hipEventCreate).  The encoder runs either one
 * launch for all levels (enough rows to fill the GPU: the launch includes
 * each level's rescoring and residual update) or one distance launch per
 * level (few rows, or rows wider than 1280 features).  events[2*i] is recorded on `stream` immediately before
 * and events[2*i + 1] immediately after distance launch i; `events` must
 * hold 2*L events, or be NULL to record nothing.  *launches (may be NULL)
 * receives the number of launches recorded (1 or L; 0 when n == 0).
 */
rvq_status rvq_encode_profiled(const void *x, rvq_dtype x_dtype, int64_t n, int32_t d,
                               const float *codebooks, const void *prepared, int32_t L, int32_t K,
                               int32_t *ids, float *residual_out,
                               void *workspace, size_t workspace_bytes, hipStream_t stream,
                               hipEvent_t *events, int32_t *launches);

/* ------------------------------------------------------------------------
 * Decode: out[row] = sum_{l < levels} codebooks[l][ids[row*L + l]], summed in
 * fp32 in level order, then stored as fp32 or rounded to nearest-even bf16.
 * `levels` in [0, L] reconstructs from the first `levels` levels only
 * (coarse-to-fine; levels == L is the full reconstruction).
 *
 * ids       : device, [n][L] int32.  An ID outside [0, K) contributes
 *             nothing and is counted in *bad_ids.
 * codebooks : device, [L][K][d] fp32, 16-byte aligned.
 * out       : device, [n][d] in out_dtype, 16-byte aligned.
 * bad_ids   : device uint32 counter incremented by the number of out-of-range
 *             IDs seen, or NULL.  The caller zeroes it.
 * ---------------------------------------------------------------------- */
rvq_status rvq_decode(const int32_t *ids, int64_t n, const float *codebooks,
                      int32_t L, int32_t K, int32_t d, int32_t levels,
                      void *out, rvq_dtype out_dtype, uint32_t *bad_ids, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Level statistics.
 *   hist[l][k] = number of rows whose level-l ID is k (exact integer count;
 *                out-of-range IDs are not counted and go to *bad_ids).
 *   msr[l]     = mean over rows of ||x_row - sum_{j <= l} codebooks[j][ids[row][j]]||^2,
 *                the mean squared residual left after levels 0..l (an
 *                out-of-range ID subtracts nothing).  Per-row residuals are
 *                fp32, squared norms and the mean are fp64, reduced in an
 *                order that depends only on n (bitwise reproducible).
 * Each out-of-range ID is counted once in *bad_ids per call.
 * ---------------------------------------------------------------------- */

/* Workspace bytes needed by rvq_level_stats (with_msr != 0 when msr is requested). */
rvq_status rvq_level_stats_workspace_size(int64_t n, int32_t L, int32_t K, int32_t d,
                                          int32_t with_msr, size_t *bytes);

/*
 * ids       : device, [n][L] int32.
 * hist      : device, [L][K] int64 output, fully overwritten.  Required.
 * msr       : device, [L] fp64 output, or NULL to compute the counts only.
 *             With n == 0 it is all zeros.
 * x         : device, [n][d] rows (x_dtype), aligned to the element size;
 *             required when msr is non-NULL and n > 0, ignored otherwise.
 *             Rows that do not start 16-byte (fp32) or 8-byte (bf16)
 *             aligned, or d not a multiple of 4, take a per-element path:
 *             the counts are the same and msr may differ in the last bits
 *             of its fp64 sum.
 * codebooks : device, [L][K][d] fp32; required when msr is non-NULL.
 * bad_ids   : as for rvq_decode.
 * workspace : device, >= rvq_level_stats_workspace_size bytes, 256-byte aligned.
 */
rvq_status rvq_level_stats(const int32_t *ids, int64_t n, int32_t L, int32_t K, int64_t *hist,
                           const void *x, rvq_dtype x_dtype, int32_t d, const float *codebooks,
                           double *msr, uint32_t *bad_ids,
                           void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Decode and level statistics of the same IDs in one pass.
 *
 * Produces exactly (bit for bit) what rvq_decode with levels == L followed by
 * rvq_level_stats with msr would: out[row] = sum of the row's codewords in
 * level order (fp32, out-of-range IDs skipped, stored as out_dtype), hist and
 * msr as defined above.  The msr pass already gathers every level's codeword
 * of every row, so the decode costs only its output writes.  Each
 * out-of-range ID is counted once in *bad_ids.
 *
 * Arguments are those of rvq_decode and rvq_level_stats; x, msr and out are
 * required (n > 0), and the workspace is sized by
 * rvq_level_stats_workspace_size(n, L, K, d, 1).
 * ---------------------------------------------------------------------- */
rvq_status rvq_decode_level_stats(const int32_t *ids, int64_t n, const float *codebooks,
                                  int32_t L, int32_t K, int32_t d, void *out, rvq_dtype out_dtype,
                                  int64_t *hist, const void *x, rvq_dtype x_dtype, double *msr,
                                  uint32_t *bad_ids, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/* ------------------------------------------------------------------------
 * Unified token embedding of a mixed text / visual sequence.
 *
 * Visual signals are multi-level discrete tokens that the backbone takes in
 * the same token format as text, and the visual codebook embeddings are
 * learned jointly with the backbone ("LongCat-2.5 发布：面向智能体任务的原生多模态大模型",
 * section "Visual Primitive Modeling", paragraph "Native
 * Visual Representation").  Token t of a sequence of T tokens becomes one
 * row of D values:
 *   visual token: out[t] = sum over l of level_tables[l][ids[t][l]], added
 *                 in fp32 in level order (bit for bit rvq_decode's sum when
 *                 the tables are fp32); an out-of-range ID adds nothing;
 *   text token:   out[t] = text_table[ids[t][0]] (ids[t][1..L-1] are not
 *                 read); an out-of-range ID gives a row of zeros.
 * bf16 outputs are the fp32 values rounded to nearest even.  Each
 * out-of-range ID that is read is counted once in *bad_ids.
 *
 * ids          : device, [T][L] int32.
 * is_visual    : device, [T] uint8, nonzero for a visual token; NULL means
 *                every token is visual.
 * text_table   : device, [V][D] in table_dtype, 16-byte aligned; may be NULL
 *                when V == 0 (every text ID is then out of range).
 * level_tables : device, [L][K][D] in table_dtype, 16-byte aligned.
 * table_dtype  : RVQ_F32 or RVQ_BF16 (both tables).
 * out          : device, [T][D] in out_dtype (RVQ_F32 or RVQ_BF16), 16-byte
 *                aligned, fully overwritten.
 * bad_ids      : device uint32 counter (added to), or NULL.
 * Limits: 1 <= L <= 64 (RVQ_ERR_UNSUPPORTED above), K >= 1, D >= 1, V >= 0.
 * ---------------------------------------------------------------------- */
rvq_status rvq_embed_tokens(const int32_t *ids, const uint8_t *is_visual, int64_t T, int32_t L,
                            const void *text_table, int64_t V, const void *level_tables,
                            int32_t K, int32_t D, rvq_dtype table_dtype, void *out,
                            rvq_dtype out_dtype, uint32_t *bad_ids, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Learning the token embedding.
 *
 * "Visual codebook embeddings are learned jointly with the backbone"
 * ("LongCat-2.5 发布：面向智能体任务的原生多模态大模型", paragraph "Native Visual
 * Representation").  The calls below are the parts of one training step
 * around the embedded rows: the norm that a model's first layer applies to
 * them and its gradient, the gradient of the embedding tables, and the
 * optimizer's step.  Pointers need only the alignment of their elements;
 * 16-byte alignment is fastest.
 * ---------------------------------------------------------------------- */

/*
 * RMS norm of rows, with the residual's addition and an 8-bit output:
 *   h = x + residual (or x),  r = 1 / sqrt(mean(h^2) + eps),  y = h r weight,
 * in fp32; each output is rounded once (y uses the unrounded h).  h has to be
 * within fp32's range, its squares need not be.
 *
 * x, residual  : device, [n][d] rows in x_dtype (RVQ_F32 or RVQ_BF16);
 *                residual may be NULL.
 * weight       : device, [d] in weight_dtype (RVQ_F32 or RVQ_BF16), or NULL
 *                for ones.
 * eps          : > 0.
 * sum_out      : device, [n][d] in x_dtype: h, the residual stream that goes
 *                on; or NULL.  May be x or residual itself (in place), not
 *                another overlap (y least of all).
 * y            : device, [n][d] in y_dtype.  RVQ_F8E4M3: row i holds
 *                e4m3(y / y_scale[i]), nearest even, with
 *                y_scale[i] = max(max|y| / 448, 2^-100) (NaN where a value of
 *                the row's y is NaN or infinite, by x, residual or weight).
 *                May be x itself if the types agree.
 * y_scale      : device, [n] fp32, required for RVQ_F8E4M3, else ignored.
 * rstd         : device, [n] fp32: r of every row, for the gradient; or NULL.
 * Limits: n <= 2^25, d <= 2^20.
 */
rvq_status rvq_rms_norm(const void *x, const void *residual, rvq_dtype x_dtype, int64_t n,
                        int32_t d, const void *weight, rvq_dtype weight_dtype, float eps,
                        void *sum_out, void *y, rvq_dtype y_dtype, float *y_scale, float *rstd,
                        hipStream_t stream);

/* Workspace bytes of rvq_rms_norm_backward with dweight. */
rvq_status rvq_rms_norm_backward_workspace_size(int64_t n, int32_t d, size_t *bytes);

/*
 * Gradient of rvq_rms_norm.  With g = dy weight and u = h rstd:
 *   dx = rstd (g - u mean(g u)) + dsum,   dweight = sum over rows of dy u.
 * dx is the gradient of x and of residual alike.
 *
 * dy, h        : device, [n][d] in dtype; h is the norm's sum_out (x where
 *                there was no residual).
 * rstd         : device, [n] fp32, from rvq_rms_norm.
 * weight       : as for rvq_rms_norm.
 * dsum         : device, [n][d] in dtype: the gradient that arrives at
 *                sum_out; or NULL.
 * dx           : device, [n][d] in dtype.  May be dy or dsum itself.
 * dweight      : device, [d] fp32, overwritten; NULL when not wanted (the
 *                workspace is then not used).  Summed in an order that
 *                depends on n, d and dtype only (bitwise reproducible).
 */
rvq_status rvq_rms_norm_backward(const void *dy, const void *h, rvq_dtype dtype, int64_t n,
                                 int32_t d, const float *rstd, const void *weight,
                                 rvq_dtype weight_dtype, const void *dsum, void *dx,
                                 float *dweight, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Workspace bytes of rvq_embed_tokens_backward. */
rvq_status rvq_embed_tokens_backward_workspace_size(int64_t T, int32_t L, int32_t K, int64_t V,
                                                    int32_t D, size_t *bytes);

/*
 * Gradient of rvq_embed_tokens with respect to its tables:
 *   dlevel[l][k] = sum of dout[t] over visual tokens t with ids[t][l] == k,
 *   dtext[v]     = sum of dout[t] over text tokens t with ids[t][0] == v,
 * in fp32, without float atomics: the order of a row's sum depends on the
 * IDs only (bitwise reproducible).  Every row of the tables is written.
 *
 * dout         : device, [T][D] in dout_dtype.
 * ids, is_visual : as for rvq_embed_tokens.
 * dlevel       : device, [L][K][D] in grad_dtype, or NULL (frozen tables).
 * dtext        : device, [V][D] in grad_dtype, or NULL.  Not both NULL.
 * accumulate   : nonzero adds to what dlevel and dtext hold (rows without a
 *                token are left as they are); zero overwrites.
 * bad_ids      : device uint32 counter (added to): out-of-range IDs, each
 *                once, of the tables whose gradient is asked for; or NULL.
 *                Such an ID adds to no row.
 * Limits: L <= 64, D <= 2^20, T <= 2^25, T (L + 1) <= 2^30, L K + V <= 2^28.
 */
rvq_status rvq_embed_tokens_backward(const void *dout, rvq_dtype dout_dtype, const int32_t *ids,
                                     const uint8_t *is_visual, int64_t T, int32_t L, int32_t K,
                                     int64_t V, int32_t D, void *dlevel, void *dtext,
                                     rvq_dtype grad_dtype, int32_t accumulate, uint32_t *bad_ids,
                                     void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One AdamW step over many tensors:
 *   g' = f grad,  f = grad_scale min(1, max_norm / (norm + 1e-6))
 *   m = beta1 m + (1 - beta1) g',   v = beta2 v + (1 - beta2) g'^2
 *   param = param (1 - lr weight_decay)
 *           - lr m / (1 - beta1^step) / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32, the update using m and v before they are rounded.  norm is the
 * 2-norm of grad_scale times all gradients of the call; without max_norm the
 * factor f is grad_scale.
 *
 * States.  state_bits 32: m and v are fp32.  state_bits 8: m and sqrt(v) are
 * held as e4m3 values with an fp32 scale for every 256 consecutive elements
 * of the tensor: m = m[i] m_scale[i / 256], sqrt(v) = v[i] v_scale[i / 256],
 * where a scale is max(largest magnitude of the 256 / 448, 2^-100).  All
 * zeros is a valid start of both.  Where m is not stored as 0, a sqrt(v) above 0
 * is not either: it becomes at least the smallest e4m3 value, 2^-9 of its scale.
 * (lr m / eps is a step without bounds: a state that a caller builds has to
 * keep to that too; a zero that comes beside an m is stepped by the formula alone.)
 * Squares may leave fp32: sqrt(v) of 8-bit
 * states has fp32's whole range, and a v of 32-bit states is held at the
 * largest fp32 at most.  A moment that is not finite (of such a gradient) is
 * stored as NaN in 8 bits and leaves the scale to the other elements.
 *
 * Rounding.  8-bit states and bf16 parameters are rounded to nearest even, or
 * where `stochastic` is nonzero at random (up with the probability of the
 * remainder), from bits that depend on (seed, step, tensor's place in the
 * call, element) only; roots below the smallest e4m3 value take m's bits, so that
 * they are seldom raised.  With beta2 = 0.999, 8-bit states need it: one step
 * moves sqrt(v) by far less than half a step of its grid.
 */
typedef struct rvq_adamw_tensor {
    void *param;          /* device, [numel] in param_dtype, updated */
    const void *grad;     /* device, [numel] in grad_dtype */
    void *m, *v;          /* device, [numel], updated: fp32 or e4m3 */
    float *m_scale, *v_scale; /* device, [ceil(numel / 256)], updated; 8-bit states only */
    void *copy;           /* device, [numel] bf16: the new parameters, nearest even; or NULL */
    int64_t numel;        /* 0 .. 2^34 */
    float weight_decay;
    int32_t reserved;     /* 0 */
} rvq_adamw_tensor;

typedef struct rvq_adamw_options {
    double lr, beta1, beta2, eps;  /* lr / (1 - beta1^step) within fp32, eps >= 1e-12 */
    int64_t step;                  /* 1 for the first */
    double grad_scale;             /* 1 for none; within fp32 */
    double max_norm;               /* <= 0: no clipping */
    int32_t stochastic;
    uint32_t seed;
} rvq_adamw_options;

/* Workspace bytes of rvq_adamw_step with max_norm or grad_norm (16 KB for every
 * 160 tensors). */
rvq_status rvq_adamw_workspace_size(int32_t count, size_t *bytes);

/*
 * tensors   : host, [count]; read before the call returns.  Tensors must not
 *             overlap.
 * options   : host.
 * grad_norm : device, fp32: the norm before clipping; or NULL.  Where
 *             max_norm > 0 or grad_norm is given and the norm is not finite,
 *             no parameter and no state is written (the step is skipped).
 * workspace : device, >= rvq_adamw_workspace_size bytes, 256-byte aligned;
 *             used (and required) with max_norm > 0 or grad_norm only.
 *
 * In a captured graph: tensors and options travel as kernel arguments, so every
 * replay repeats one step: its lr, step number, bias corrections and random bits
 * (the same elements round up every time, which is no longer right on average).
 * A training loop makes this call anew for each step, beside a graph of the rest.
 */
rvq_status rvq_adamw_step(const rvq_adamw_tensor *tensors, int32_t count, rvq_dtype param_dtype,
                          rvq_dtype grad_dtype, int32_t state_bits,
                          const rvq_adamw_options *options, float *grad_norm, void *workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * The head of a model that takes and predicts token IDs.
 *
 * Rows of features or hidden states are layer-normed, 8-bit rows are multiplied
 * with a table (8-bit values with a scale for each block of 128), and the logits
 * that come out score the IDs: their log probabilities, entropy and best
 * alternatives, or the distance from a teacher's best.  Each comes with its
 * gradient, for one training step around a model; conventions are those of the
 * calls above.  Pointers need only the alignment of their elements; 16-byte
 * alignment is fastest.
 * ---------------------------------------------------------------------- */

/*
 * Layer norm of rows, with the residual's addition and an 8-bit output:
 *   h = x + residual (or x),  m = mean(h),  r = 1 / sqrt(mean((h - m)^2) + eps),
 *   y = (h - m) r weight + bias,
 * in fp32, the variance taken of the centred values; each output is rounded once
 * (y uses the unrounded h).  h has to be within fp32's range, its squares need not.
 *
 * x, residual, sum_out, y, y_dtype, y_scale, eps : as for rvq_rms_norm.
 * weight, bias : device, [d] in weight_dtype (RVQ_F32 or RVQ_BF16), or NULL for
 *                ones and zeros.
 * mean, rstd   : device, [n] fp32: m and r of every row, for the gradient; or NULL.
 * Limits: n <= 2^25, d <= 2^20.
 */
rvq_status rvq_layer_norm(const void *x, const void *residual, rvq_dtype x_dtype, int64_t n,
                          int32_t d, const void *weight, const void *bias, rvq_dtype weight_dtype,
                          float eps, void *sum_out, void *y, rvq_dtype y_dtype, float *y_scale,
                          float *mean, float *rstd, hipStream_t stream);

/* Workspace bytes of rvq_layer_norm_backward with dweight or dbias. */
rvq_status rvq_layer_norm_backward_workspace_size(int64_t n, int32_t d, size_t *bytes);

/*
 * Gradient of rvq_layer_norm.  With g = dy weight and u = (h - mean) rstd:
 *   dx = rstd (g - mean(g) - u mean(g u)) + dsum,
 *   dweight = sum over rows of dy u,   dbias = sum over rows of dy.
 * dx is the gradient of x and of residual alike.
 *
 * dy, h, dsum, dx : as for rvq_rms_norm_backward.
 * mean, rstd      : device, [n] fp32, from rvq_layer_norm.
 * dweight, dbias  : device, [d] fp32, overwritten; either may be NULL (with both
 *                   NULL the workspace is not used).  Summed in an order that
 *                   depends on n, d and dtype only (bitwise reproducible).
 */
rvq_status rvq_layer_norm_backward(const void *dy, const void *h, rvq_dtype dtype, int64_t n,
                                   int32_t d, const float *mean, const float *rstd,
                                   const void *weight, rvq_dtype weight_dtype, const void *dsum,
                                   void *dx, float *dweight, float *dbias, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* Scales of an 8-bit operand [rows][k] of rvq_matmul_f8. */
typedef enum rvq_scale_layout {
    RVQ_SCALE_ROW = 0,      /* [rows]: one a row (as the norms' 8-bit outputs have) */
    RVQ_SCALE_ROW_128 = 1,  /* [rows][ceil(k / 128)]: one for 128 elements of a row */
    RVQ_SCALE_128_128 = 2   /* [ceil(rows / 128)][ceil(k / 128)]: one for 128 x 128 */
} rvq_scale_layout;

/*
 * 8-bit values (e4m3) with one scale for each block of 128:
 *   scale = max(max|x| / 448, 2^-100) of the block (NaN where a value of it is NaN
 *   or infinite),  q = e4m3(x / scale), nearest even.
 *
 * x         : device, [rows][cols] in x_dtype (RVQ_F32 or RVQ_BF16).
 * layout    : RVQ_SCALE_ROW_128 or RVQ_SCALE_128_128, of q's rows.
 * transpose : nonzero: q is x's transpose, [cols][rows], with blocks along its rows
 *             (what the gradient of a weight contracts are the rows of x).
 * q         : device, [rows][cols] (or [cols][rows]), rows q_stride bytes apart;
 *             bytes between a row's end and the next row are left as they are.
 * scale     : device, fp32, as layout says for q's rows and columns.
 * Limits: rows, cols <= 2^30, rows cols <= 2^40.
 */
rvq_status rvq_quantize_f8(const void *x, rvq_dtype x_dtype, int64_t rows, int64_t cols,
                           rvq_scale_layout layout, int32_t transpose, void *q, int64_t q_stride,
                           float *scale, hipStream_t stream);

/*
 * Product of 8-bit operands:
 *   out[i][j] = sum over blocks c of sa(i, c) sb(j, c) sum_{k in block c} a[i][k] b[j][k],
 * both sums in fp32, one rounding to out_dtype.  The forward pass of a linear
 * layer (a: rows, b: weight [n][k]) and, with transposed operands, both its gradients.
 * Every product is exact, and a bf16 result is the fp32 result rounded once.
 *
 * a, b         : device, [m][k] and [n][k] e4m3, rows a_stride, b_stride bytes
 *                apart (>= k).  Fastest with 16-byte aligned rows (address and stride
 *                multiples of 16): then each row, the last too, has to be readable up
 *                to a multiple of 16 bytes; what stands behind its end is not used.
 * a_scale, b_scale : device, fp32, laid out as a_layout and b_layout say; a product
 *                of two scales has to be within fp32.
 * out          : device, [m][n] in out_dtype (RVQ_F32 or RVQ_BF16).  k == 0 gives zeros.
 * Limits: m, n <= 2^27, m n <= 2^36, k <= 2^30.
 */
rvq_status rvq_matmul_f8(const void *a, int64_t a_stride, const float *a_scale,
                         rvq_scale_layout a_layout, const void *b, int64_t b_stride,
                         const float *b_scale, rvq_scale_layout b_layout, int64_t m, int64_t n,
                         int64_t k, void *out, rvq_dtype out_dtype, hipStream_t stream);

/* Workspace bytes of rvq_token_logprobs (0 for many rows). */
rvq_status rvq_token_logprobs_workspace_size(int64_t n, int32_t V, int32_t top, size_t *bytes);

/*
 * Log probabilities of given tokens under softmax(logits / temperature), with the
 * entropy and the best alternatives of each row.
 *
 * logits      : device, [n][V] in dtype (RVQ_F32 or RVQ_BF16).  -inf masks a token.
 * ids         : device, [n] int32: the token of each row; or NULL.  -1: no token
 *               (logprob 0); any other ID outside [0, V) also gives 0 and is counted
 *               in *bad_ids.
 * temperature : 1e-4 .. 1e4.
 * logprob     : device, [n] fp32 (-inf of a masked token); required with ids.
 * entropy     : device, [n] fp32, in nats; or NULL.
 * stats       : device, [n][2] fp32: the row's largest logit M and log S, S = sum of
 *               exp((logit - M) / temperature); the log of the row's sum of
 *               exponentials is M / temperature + log S.
 * top         : 0 .. 64 alternatives.
 * top_logprob, top_ids : device, [n][top] fp32 and int32: the largest logits, larger
 *               first and the lower ID first among equals; -inf and -1 behind the last
 *               token that is not masked.  Not read with top == 0.
 * bad_ids     : device uint32 counter (added to), or NULL.
 * A row that holds NaN or +inf gives NaN (and IDs of -1); a row of nothing but -inf
 * gives log probabilities of -inf and entropy 0.  Rows do not touch one another.
 * Limits: n <= 2^25, 1 <= V <= 2^24.
 */
rvq_status rvq_token_logprobs(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                              const int32_t *ids, float temperature, float *logprob,
                              float *entropy, float *stats, int32_t top, float *top_logprob,
                              int32_t *top_ids, uint32_t *bad_ids, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * Gradient of rvq_token_logprobs with respect to the logits:
 *   dlogits[j] = (dlogprob ([j == id] - p_j) - dentropy p_j (log p_j + entropy)) / temperature
 *
 * logits, ids, temperature, stats, entropy : as given to and by the forward call;
 *             entropy is read with dentropy only.
 * dlogprob, dentropy : device, [n] fp32; either may be NULL, not both.  dlogprob
 *             needs ids; rows without a valid ID take none.  Rows with both 0, and
 *             rows of nothing but -inf, get zeros whatever their logits are.
 * dlogits   : device, [n][V] in dtype.  May be logits itself, not another overlap.
 */
rvq_status rvq_token_logprobs_backward(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                                       const int32_t *ids, float temperature, const float *stats,
                                       const float *dlogprob, const float *entropy,
                                       const float *dentropy, void *dlogits, hipStream_t stream);

/*
 * Distillation loss of a teacher's top tokens, with p = softmax(logits / temperature):
 *   tail == 0: q = softmax(teacher / temperature) over the row's entries
 *              (teacher: logits, or log probabilities at temperature 1),
 *              loss = sum over entries of q (log q - log p);
 *   tail != 0: q = exp(teacher) (teacher: log probabilities at this temperature, as
 *              rvq_token_logprobs gives them), and all other tokens are one more
 *              outcome: rest = max(0, 1 - sum q), against the sum of their p.
 *              Where the other tokens have no weight (a sum below 2^-149: the entries
 *              name all that are not masked, by -inf or a large negative value), a
 *              rest of up to 2^-16 is taken as the logarithms' rounding.
 *
 * logits      : as for rvq_token_logprobs.
 * teacher_ids : device, [n][k] int32.  -1: no entry; any other ID outside [0, V) is
 *               left out and counted in *bad_ids; a repeated ID counts where it
 *               comes first.
 * teacher     : device, [n][k] fp32.
 * k           : 1 .. 256.
 * loss        : device, [n] fp32; 0 of a row without an entry (or, with tail == 0,
 *               whose entries are all -inf), +inf where the teacher's weight meets a
 *               masked token.
 * stats       : device, [n][4] fp32, for the gradient.
 * Limits: n <= 2^25, 1 <= V <= 2^24.
 */
rvq_status rvq_distill_loss(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                            const int32_t *teacher_ids, const float *teacher, int32_t k,
                            int32_t tail, float temperature, float *loss, float *stats,
                            uint32_t *bad_ids, hipStream_t stream);

/*
 * Gradient of rvq_distill_loss with respect to the logits, times dloss of the row:
 *   dlogits[j] = dloss (p_j - q_j) / temperature  (q_j: of a token outside the entries 0
 *   or, with tail, rest p_j / (sum of p over those tokens)).
 *
 * dloss    : device, [n] fp32.  A row of 0, one without an entry and one of nothing
 *            but -inf get zeros whatever their logits are.
 * dlogits  : device, [n][V] in dtype.  May be logits itself, not another overlap.
 * All else as given to and by the forward call.
 */
rvq_status rvq_distill_loss_backward(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                                     const int32_t *teacher_ids, const float *teacher, int32_t k,
                                     int32_t tail, float temperature, const float *stats,
                                     const float *dloss, void *dlogits, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Resumable ID cache (host files).
 *
 * The visual tokenizer is fixed, so token IDs are computed ahead of time
 * and cached offline ("LongCat-2.5 发布：面向智能体任务的原生多模态大模型",
 * paragraph "Offline Visual Preprocessing").  An ID cache file holds the
 * IDs [n][L] of n rows in chunks of chunk_rows rows (the last chunk may be
 * shorter), appended in chunk order, each with a CRC-32, so that an
 * interrupted writer resumes after its last complete chunk.  Host code
 * only: these calls make no HIP call and touch no device memory; each
 * opens and closes the file.  Errors (bad arguments, I/O failure, a header
 * that does not match) return RVQ_ERR_INVALID_ARGUMENT.
 * ---------------------------------------------------------------------- */

/* Creates the file (header only) when it does not exist.  Otherwise checks
 * that its header matches (n, L, K, chunk_rows), cuts off a torn or corrupt
 * tail, and reports in *chunks_done how many leading chunks it holds. */
rvq_status rvq_idcache_resume(const char *path, int64_t n, int32_t L, int32_t K,
                              int64_t chunk_rows, int64_t *chunks_done);

/* Appends chunk `chunk`: its rows x L IDs from host memory.  The file must
 * hold exactly chunks 0 .. chunk-1. */
rvq_status rvq_idcache_append(const char *path, int64_t n, int32_t L, int32_t K,
                              int64_t chunk_rows, int64_t chunk, const int32_t *ids);

/* Reads the valid leading chunks into ids (host, [n][L]; the rows of
 * missing chunks are left as they are) and reports their count. */
rvq_status rvq_idcache_read(const char *path, int64_t n, int32_t L, int32_t K,
                            int64_t chunk_rows, int32_t *ids, int64_t *chunks_done);

/* ------------------------------------------------------------------------
 * Streaming encode of host-resident rows (the offline tokenisation pass).
 *
 * Token IDs are computed ahead of training and cached ("LongCat-2.5 发布：面向智能体任务的原生多模态大模型",
 * paragraph "Offline Visual Preprocessing").  rvq_stream_encode encodes rows [0, n) of a host array
 * in chunks of chunk_rows rows: while chunk c is encoded on `stream`, chunk
 * c+1 is copied in and the IDs of chunk c-1 are copied out, each on a copy
 * stream of its own that the call creates (default priority) and destroys,
 * ordered by events.  The IDs are bit for bit those of one rvq_encode call
 * over all n rows (the encoder is batch-invariant).  The call is
 * synchronous: it returns when its chunks are done and every stream it used
 * is idle.
 * ---------------------------------------------------------------------- */

/* Called on the calling thread once chunk `chunk` (rows row0 .. row0+rows-1)
 * has its IDs in host memory at `ids` ([rows][L]).  A nonzero return stops
 * the call after this chunk (which counts as done). */
typedef int (*rvq_chunk_callback)(void *user, int64_t chunk, int64_t row0, int64_t rows,
                                  const int32_t *ids);

/* Device workspace bytes for rvq_stream_encode with chunks of chunk_rows rows:
 * two row buffers, two ID buffers and rvq_encode's workspace. */
rvq_status rvq_stream_workspace_size(int64_t chunk_rows, int32_t d, int32_t L, int32_t K,
                                     size_t *bytes);

/*
 * x_host      : host, [n][d] rows (x_dtype).  Pinned memory (hipHostMalloc)
 *               lets the copies overlap the encoder; pageable memory works,
 *               with copies that may not overlap.
 * codebooks, prepared, L, K : as for rvq_encode (device).
 * ids_host    : host, [n][L] int32 output; chunks not run are left as they are.
 * chunk_rows  : rows per chunk (>= 1); chunk c holds rows c*chunk_rows ...
 * first_chunk : the first chunk to run (earlier ones are skipped: resume).
 * max_chunks  : run at most this many chunks (<= 0: all that remain).
 * on_chunk    : callback per finished chunk, or NULL; user is passed to it.
 * workspace   : device, >= rvq_stream_workspace_size bytes, 256-byte aligned.
 * stream      : the stream the encoder runs on; work the caller queued on it
 *               before the call is done before the first copy.
 * chunks_done : out: chunks 0 .. *chunks_done - 1 are done (those before
 *               first_chunk included), also when an error is returned.
 */
rvq_status rvq_stream_encode(const void *x_host, rvq_dtype x_dtype, int64_t n, int32_t d,
                             const float *codebooks, const void *prepared, int32_t L, int32_t K,
                             int32_t *ids_host, int64_t chunk_rows, int64_t first_chunk,
                             int64_t max_chunks, rvq_chunk_callback on_chunk, void *user,
                             void *workspace, size_t workspace_bytes, hipStream_t stream,
                             int64_t *chunks_done);

/* rvq_stream_encode into a resumable ID cache file: rvq_idcache_resume on
 * `path`, then the chunks the file does not hold yet (at most max_chunks of
 * them), each appended to the file as it finishes.  Rerun after an
 * interruption to continue.  *chunks_done: the chunks the file holds. */
rvq_status rvq_stream_encode_to_cache(const char *path, const void *x_host, rvq_dtype x_dtype,
                                      int64_t n, int32_t d, const float *codebooks,
                                      const void *prepared, int32_t L, int32_t K,
                                      int32_t *ids_host, int64_t chunk_rows, int64_t max_chunks,
                                      void *workspace, size_t workspace_bytes, hipStream_t stream,
                                      int64_t *chunks_done);

/* ------------------------------------------------------------------------
 * rvq_encode with no workspace argument, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation.  The workspace is the library's own
 * file-scope device array of 256 MiB (268,435,456 bytes; one on every
 * device the library runs on, held until the process ends): enough for one
 * image of up to 84 x 84 patches (7,056 rows) at d = 1152, L = 8,
 * K = 8192.  Arguments, layouts, results and errors are rvq_encode's; a call
 * whose workspace (rvq_encode_workspace_size) exceeds the array returns
 * RVQ_ERR_UNSUPPORTED before any HIP call.  No hipMalloc or hipFree.  The
 * device address of the array is looked up on a device's first call (with
 * that device current).  Every call on one device shares the array: calls
 * that overlap on one GPU (several streams or threads) race, and must not
 * be made.
 * ---------------------------------------------------------------------- */
rvq_status rvq_encode_noalloc(const void *x, rvq_dtype x_dtype, int64_t n, int32_t d,
                              const float *codebooks, const void *prepared, int32_t L, int32_t K,
                              int32_t *ids, float *residual_out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Token-count-aware packing across data-parallel ranks (host code).
 *
 * With the visual tokenizer out of the training graph, every sample's
 * image-token count is known when batches are packed, so the share of
 * visual tokens on each data-parallel rank can be kept close to the
 * batch's ("LongCat-2.5 Released", section 4 "Infrastructure: Under 80 GB
 * Per Card", "Supernode-aware parallelism", last paragraph; "LongCat-2.5
 * 发布：面向智能体任务的原生多模态大模型", "Supernode-Aware Parallelism",
 * last paragraph).  The pages state the goal only; the objective is this
 * library's reading of it.  Sample i has t_i text and v_i image tokens,
 * n_i = t_i + v_i; the batch has N = sum n_i tokens, V = sum v_i of them
 * visual, p = V / N.  Rank r receives N_r tokens, V_r of them visual, and
 * at most `capacity` tokens.  The planner minimises
 *     max_r |V_r - p N_r|      (the rank's tokens beyond the batch's
 *                               modality proportion),
 * then max_r N_r, computing the excesses exactly in integers
 * (N (V_r - p N_r) = sum over the rank of v_i N - V n_i).
 *
 * text_tokens, image_tokens: host arrays [samples], each >= 0, at most
 * 2^30 tokens in all.  ranks >= 1.  Inputs of at most exact_max samples
 * are solved exactly (exhaustive search with a bound; keep exact_max small,
 * about 12: the search is exponential); larger ones by a greedy
 * assignment (samples by decreasing modality excess, each to the rank
 * that keeps its excess smallest) followed by moves and swaps that lower
 * the largest excess.  rank_of (host, [samples]) receives each sample's
 * rank.  summary (host, [3], or NULL): max_r |sum of v_i N - V n_i| (the
 * objective times N), N, and max_r N_r.  Returns RVQ_ERR_INVALID_ARGUMENT
 * for bad arguments and RVQ_ERR_UNSUPPORTED when a sample exceeds the
 * capacity, the samples do not fit, or the counts are too large.  No HIP
 * call; thread-safe.
 * ---------------------------------------------------------------------- */
rvq_status rvq_pack_ranks(const int64_t *text_tokens, const int64_t *image_tokens,
                          int64_t samples, int32_t ranks, int64_t capacity, int32_t exact_max,
                          int32_t *rank_of, int64_t *summary);

/* ------------------------------------------------------------------------
 * Measurement aid: the matrix cores' achievable bf16 rate.
 *
 * Not a step of the path.  The published dense bf16 peak assumes the
 * nominal clock; under a full matrix load the chip holds a clock that
 * depends on how much the operands switch.  rvq_mfma_rate runs a
 * register-only loop of v_mfma_f32_32x32x16_bf16 (the instruction of the
 * encoder's distance stage) on `blocks` workgroups of four waves (use one
 * per compute unit: one wave per SIMD), four independent accumulator chains
 * per wave, `iters` iterations of eight instructions, no memory traffic in
 * the loop.  zero_operands != 0 uses all-zero operands, otherwise random
 * bf16 values (random sign, magnitude in [0.25, 4), random mantissa).
 * A short untimed run precedes the timed one.
 *
 * workspace: device memory of at least rvq_mfma_rate_workspace_size(blocks)
 * bytes, 8-byte aligned (per-workgroup clock readings and a result sink).
 * tflops (host) receives the timed launch's rate from HIP events; clock_ghz
 * (host) the shader clock over the loop (s_memtime ticks over
 * s_memrealtime's 100 MHz, averaged over workgroups).  Unlike the other
 * device entry points this call waits for its work and copies the clock
 * readings to the host.  Returns RVQ_ERR_INVALID_ARGUMENT for blocks
 * outside 1 .. 65536, iters outside 10 .. 10^7 or a null or misaligned
 * pointer, RVQ_ERR_WORKSPACE_TOO_SMALL, or RVQ_ERR_HIP.
 * ---------------------------------------------------------------------- */
size_t rvq_mfma_rate_workspace_size(int32_t blocks);
rvq_status rvq_mfma_rate(int32_t blocks, int32_t iters, int32_t zero_operands, void *workspace,
                         size_t workspace_bytes, hipStream_t stream, double *tflops,
                         double *clock_ghz);

#ifdef __cplusplus
}
#endif

#endif /* RVQ_H */
