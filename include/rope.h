/*
 * rope.h -- C ABI of librope: rotary position embedding (RoPE) on the GPU.
 *
 * What the library computes.  For a token at table row r and pair index i,
 * the pair (x1, x2) of a query or key head row becomes
 *     (x1 cos t - x2 sin t,  x1 sin t + x2 cos t),   t = angle(r, i)
 * ("Rotary Embedding (RoPE) Kernel Optimization", Overview).  Queries and
 * keys are rotated in one launch ("How Unsloth Optimizes RoPE Embedding
 * Computations in Triton Kernels", Triton Kernel Architecture for RoPE:
 * the fused Q+K kernel), and the backward pass is the same rotation by -t
 * (same page, Frequently Asked Questions: gradients use the same kernel
 * with the backward flag).
 *
 * Conventions shared by every entry point:
 *   - Pointers marked "device" must point to memory of the current CUDA
 *     device.  The caller owns every buffer; the library allocates nothing
 *     and never synchronises the stream, except in rope_check_errors.
 *   - `stream` is a cudaStream_t passed as void*; NULL is the default stream.
 *     Work is enqueued asynchronously on that stream.
 *   - Tensors are dense and contiguous.  seq_before_head = 0: [B, H, S, D]
 *     (Unsloth page, Usage Examples; "rotary-embedding-torch", Input Tensor
 *     Shapes); seq_before_head = 1: [B, S, H, D] ("rotary-embedding-torch",
 *     RotaryEmbedding / Key Parameters: seq_before_head_dim).
 *   - Element types: ROPE_F32, ROPE_BF16, ROPE_F16.  Arithmetic is fp32;
 *     each output element is rounded once to the element type.
 *   - Pair layouts ("Rotary Embedding (RoPE) Kernel Optimization", Core
 *     Technique / Paired Element Layout): ROPE_SPLIT_HALF pairs
 *     (x[i], x[i + rotary_dim/2]); ROPE_INTERLEAVED pairs (x[2i], x[2i+1]).
 *   - Partial rotation ("rotary-embedding-torch", RotaryEmbedding / Key
 *     Parameters: dim is the size of the rotated part): only the first
 *     rotary_dim features of each head row are rotated; features
 *     [rotary_dim, D) are neither read nor written.
 *   - Errors detected on the host are returned before anything is enqueued;
 *     nothing is modified then.
 */
#ifndef ROPE_H
#define ROPE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ROPE_OK = 0,
    ROPE_ERR_INVALID_ARG = 1,      /* bad size, null pointer, overlap, ...       */
    ROPE_ERR_UNSUPPORTED = 2,      /* dtype or layout value outside the enums    */
    ROPE_ERR_CUDA = 3,             /* a CUDA call failed (launch, sync, ...)     */
    ROPE_ERR_POS_OUT_OF_RANGE = 4, /* a position index was outside the table     */
    ROPE_ERR_KERNEL_TIMEOUT = 5,   /* a bounded wait inside a kernel expired      */
    ROPE_ERR_BAD_INDEX = 6         /* a sequence offset, a length or a page number
                                      of a serving call was out of range          */
} rope_status;

typedef enum { ROPE_SPLIT_HALF = 0, ROPE_INTERLEAVED = 1 } rope_layout;
typedef enum { ROPE_F32 = 0, ROPE_BF16 = 1, ROPE_F16 = 2 } rope_dtype;
/* attention masks ("rotary-embedding-torch", flash_attn_with_rotary / Input
 * Tensor Shapes: attn_mask (batch, seq_len_k) or (batch, seq_len_q, seq_len_k)) */
typedef enum {
    ROPE_MASK_NONE = 0,
    ROPE_MASK_KEYS = 1,        /* uint8 [B, Sk]: one entry per key (key padding) */
    ROPE_MASK_QUERY_KEYS = 2   /* uint8 [B, Sq, Sk]: one entry per query and key */
} rope_mask_kind;
/* frequency modes ("rotary-embedding-torch", RotaryEmbedding: freqs_for) */
typedef enum { ROPE_FREQ_LANG = 0, ROPE_FREQ_PIXEL = 1, ROPE_FREQ_CONSTANT = 2 } rope_freq_mode;
/* rules for contexts longer than those trained on (rope_tables_build_scaled) */
typedef enum {
    ROPE_SCALE_LINEAR = 0,     /* every frequency over the factor                 */
    ROPE_SCALE_NTK = 1,        /* a larger base                                   */
    ROPE_SCALE_SMOOTH = 2,     /* low frequencies over the factor, high ones kept */
    ROPE_SCALE_YARN = 3        /* the same along the pairs, values scaled         */
} rope_scale_kind;

/*
 * rope_tables_build -- fill the cos/sin table.
 *
 * Source: "rotary-embedding-torch", RotaryEmbedding / Key Parameters (theta
 * is the frequency base, default 10000; interpolate_factor scales sequence
 * positions, default 1.0); "Rotary Embedding (RoPE) Kernel Optimization",
 * Common Pitfalls (cos/sin are [seq_len, D/2] and broadcast over batch and
 * heads).  The pages do not print the frequency formula; the library uses
 * the standard one: for row m and pair i (0 <= i < rotary_dim/2)
 *     angle = (m / interpolate_factor) * theta^(-2i / rotary_dim),
 * evaluated in fp64, and stores cos(angle), sin(angle) rounded to fp32.
 *
 * cos_out, sin_out: device, caller-owned, float[max_pos * rotary_dim/2]
 *   each, row-major [max_pos, rotary_dim/2].
 * Errors: ROPE_ERR_INVALID_ARG if theta <= 0, interpolate_factor <= 0 (or
 *   either is not finite), rotary_dim < 2 or odd, max_pos < 0, a null
 *   output with max_pos > 0, or overlapping outputs.  max_pos = 0 is a
 *   no-op.  ROPE_ERR_CUDA if the launch fails.
 */
rope_status rope_tables_build(double theta, int32_t rotary_dim, int64_t max_pos,
                              double interpolate_factor, float *cos_out, float *sin_out,
                              void *stream);

/*
 * rope_tables_build_ex -- the cos/sin table of a frequency mode, at given
 * row positions, optionally with the XPOS scale folded in.
 *
 * Source: "rotary-embedding-torch", RotaryEmbedding / Key Parameters names
 * freqs_for = 'lang' (default) | 'pixel' | 'constant' and use_xpos (length
 * extrapolation) without formulas; the published definitions are used.  For
 * row m and pair i (0 <= i < h = rotary_dim/2):
 *     p     = pos_offset + m / pos_divisor
 *     w_i   = theta^(-2i / rotary_dim)                     ROPE_FREQ_LANG
 *           = pi * (1 + i * (max_freq/2 - 1) / (h - 1))    ROPE_FREQ_PIXEL
 *             (pi when h = 1; Perceiver's Fourier features, positions
 *             usually in [-1, 1]: pos_offset = -1, pos_divisor = (rows-1)/2)
 *           = 1                                            ROPE_FREQ_CONSTANT
 *     s     = 1 when xpos_sign = 0, else (XPOS, Sun et al. 2022)
 *             zeta_i^(xpos_sign * (p - xpos_center) / xpos_scale_base),
 *             zeta_i = (2i/rotary_dim + xpos_gamma) / (1 + xpos_gamma)
 *     cos_out[m][i] = s * cos(p * w_i), sin_out[m][i] = s * sin(p * w_i),
 * all in fp64, each stored rounded once to fp32.  XPOS scales the query by
 * zeta^(+n/B) and the key by zeta^(-n/B): build one table with xpos_sign =
 * +1 for Q and one with -1 for K and rotate each with rope_apply_q (the
 * backward flag, which negates the sine, then gives the XPOS gradient too).
 * ROPE_FREQ_LANG with pos_offset = 0 and pos_divisor = interpolate_factor
 * reproduces rope_tables_build bit for bit.
 *
 * cos_out, sin_out: device, caller-owned, float[rows * rotary_dim/2] each.
 * Errors: ROPE_ERR_UNSUPPORTED for an unknown mode; ROPE_ERR_INVALID_ARG if
 *   rotary_dim < 2 or odd, rows < 0, theta <= 0 (lang), max_freq <= 0
 *   (pixel), pos_divisor <= 0, a non-finite pos_offset / pos_divisor,
 *   xpos_sign outside {-1, 0, 1}, and with xpos_sign != 0 a scale base or
 *   gamma <= 0 or a non-finite centre; null or overlapping outputs with
 *   rows > 0.  rows = 0 is a no-op.  ROPE_ERR_CUDA if the launch fails.
 */
rope_status rope_tables_build_ex(int32_t freq_mode, double theta, double max_freq,
                                 int32_t rotary_dim, int64_t rows, double pos_offset,
                                 double pos_divisor, int32_t xpos_sign, double xpos_scale_base,
                                 double xpos_gamma, double xpos_center, float *cos_out,
                                 float *sin_out, void *stream);

/*
 * rope_apply_qk -- rotate Q and K in place, in one launch.
 *
 * Source: Unsloth page, Triton Kernel Architecture for RoPE (Q and K in one
 * kernel) and Usage Examples (fast_rope_embedding(Q, K, cos, sin,
 * position_ids)); "rotary-embedding-torch", flash_attn_with_rotary / Key
 * Features (heads_q != heads_kv for GQA/MQA).
 *
 * q: device, [B, Hq, S, D] or [B, S, Hq, D] of `dtype`, updated in place.
 * k: device, [B, Hk, S, D] or [B, S, Hk, D] of `dtype`, updated in place;
 *    may be NULL when Hk = 0.  q and k must not overlap each other or the
 *    tables.
 * cos, sin: device, float[table_rows, rotary_dim/2] (as written by
 *    rope_tables_build with max_pos = table_rows).
 * pos_idx: device int32[S] or NULL.  Token s (in every batch) uses table
 *    row pos_idx[s] (Unsloth page, Support for Custom Position IDs;
 *    "rotary-embedding-torch", Input Tensor Shapes: rotary_pos_emb_indices
 *    (seq_len,)).  The value -1 leaves the token unrotated (the pos_mask of
 *    "rotary-embedding-torch", flash_attn_with_rotary): its rows are not
 *    written.  With NULL, token s uses row s and S <= table_rows is required.
 *    Any other value outside [0, table_rows) leaves that token unrotated and
 *    raises a device-side flag reported by rope_check_errors as
 *    ROPE_ERR_POS_OUT_OF_RANGE.
 * B, S >= 0; Hq, Hk >= 0; D >= 1; rotary_dim even, 2 <= rotary_dim <= D.
 *    An empty problem (B, S or Hq + Hk zero) returns ROPE_OK and enqueues
 *    nothing.
 * layout: rope_layout.  seq_before_head, backward: 0 or 1.  backward = 1
 *    rotates by the negated angle (the gradient of the forward rotation).
 * dtype: rope_dtype of q and k.
 * table_rows: rows of cos and sin (>= 1 for a non-empty problem).
 * Errors: ROPE_ERR_UNSUPPORTED for dtype/layout outside the enums;
 *    ROPE_ERR_INVALID_ARG for the size, flag, pointer and overlap rules
 *    above; ROPE_ERR_CUDA if the launch fails.  Pointers or rows that are
 *    not 16-byte aligned take a slower element-wise kernel, same results.
 */
rope_status rope_apply_qk(void *q, void *k, const float *cos, const float *sin,
                          const int32_t *pos_idx, int64_t B, int32_t Hq, int32_t Hk, int64_t S,
                          int32_t D, int32_t rotary_dim, int32_t layout, int32_t seq_before_head,
                          int32_t backward, int32_t dtype, int64_t table_rows, void *stream);

/*
 * rope_apply_qk_out -- rotate Q and K out of place (or in place), with
 * optional per-sequence position indices.
 *
 * Same computation as rope_apply_qk, reading q and k and writing q_out and
 * k_out.  An output may be exactly its input (that tensor is rotated in
 * place); otherwise it must not overlap any input, the tables, pos_idx or
 * the other output.  Out of place, the output receives every element: the
 * rotated span, the tail [rotary_dim, D) copied unchanged, and the rows of
 * unrotated tokens (position -1 or out of range) copied unchanged.
 *
 * Position indices (Unsloth page, Support for Custom Position IDs:
 * prefix-tuning and context shifting; "rotary-embedding-torch", Input Tensor
 * Shapes: indices into a padded frequency buffer):
 *   pos_batch_stride = 0: pos_idx is int32[S], shared by every batch (as in
 *     rope_apply_qk);
 *   pos_batch_stride >= S: pos_idx is int32[B][pos_batch_stride] and token
 *     (b, s) uses pos_idx[b * pos_batch_stride + s] -- one position vector per
 *     sequence, e.g. sequences decoded at different offsets.
 * Other strides return ROPE_ERR_INVALID_ARG.  Everything else (sizes, flags,
 * errors, range flag) as for rope_apply_qk.
 */
rope_status rope_apply_qk_out(const void *q, const void *k, void *q_out, void *k_out,
                              const float *cos, const float *sin, const int32_t *pos_idx,
                              int64_t pos_batch_stride, int64_t B, int32_t Hq, int32_t Hk,
                              int64_t S, int32_t D, int32_t rotary_dim, int32_t layout,
                              int32_t seq_before_head, int32_t backward, int32_t dtype,
                              int64_t table_rows, void *stream);

/*
 * rope_apply_q -- rotate one tensor in place (the query-only kernel of the
 * Unsloth page, Triton Kernel Architecture for RoPE).  Same rules as
 * rope_apply_qk with x in place of q, H in place of Hq, and no k.
 */
rope_status rope_apply_q(void *x, const float *cos, const float *sin, const int32_t *pos_idx,
                         int64_t B, int32_t H, int64_t S, int32_t D, int32_t rotary_dim,
                         int32_t layout, int32_t seq_before_head, int32_t backward, int32_t dtype,
                         int64_t table_rows, void *stream);

/*
 * rope_tables_build_scaled -- the cos/sin table for a context longer than the
 * one a model was trained on, by one of the published rules.
 *
 * With w_i = theta^(-2i / rotary_dim), f = factor and n_i = original_positions *
 * w_i / 2 pi (turns that pair i makes over the trained context), pair i turns by
 *     LINEAR   w_i / f
 *     NTK      (theta * f^(rotary_dim / (rotary_dim - 2)))^(-2i / rotary_dim)
 *     SMOOTH   (1 - m) w_i / f + m w_i,  m = clamp((n_i - low_turns) /
 *              (high_turns - low_turns), 0, 1)
 *     YARN     r w_i / f + (1 - r) w_i,  r = clamp((i - a) / (b - a), 0, 1), a
 *              = max(floor(j(high_turns)), 0), b = min(ceil(j(low_turns)),
 *              rotary_dim - 1), j(n) = rotary_dim ln(original_positions / 2 pi
 *              n) / (2 ln theta) the pair that makes n turns (b - a = 0.001
 *              where b <= a)
 * a position; row m stands for the position pos_offset + m.  Values are multiplied
 * by value_scale, or, when that is 0, by 1 (YARN: 0.1 ln f + 1).
 *
 * cos_out, sin_out: device, caller-owned, float[rows * rotary_dim/2] each.
 * Accuracy: frequencies in more than 100 bits on the host, phases as 64-bit fractions
 *   of a turn (p 2^-65 + 2^-57 turns off at position p), values within 6 * 2^-24 of
 *   themselves besides.
 * Errors: ROPE_ERR_UNSUPPORTED for an unknown kind or rotary_dim > 512;
 *   ROPE_ERR_INVALID_ARG if rotary_dim < 2 or odd (NTK: or 2), rows or
 *   pos_offset < 0 or their sum past 2^31 - 1, theta <= 1, factor < 1,
 *   value_scale < 0 (or any of them not finite), and for SMOOTH and YARN
 *   original_positions < 1, low_turns <= 0 or high_turns <= low_turns; null or
 *   overlapping outputs.  rows = 0 is a no-op.  ROPE_ERR_CUDA if the launch fails.
 */
rope_status rope_tables_build_scaled(int32_t kind, double theta, int32_t rotary_dim, int64_t rows,
                                     int64_t pos_offset, double factor, int64_t original_positions,
                                     double low_turns, double high_turns, double value_scale,
                                     float *cos_out, float *sin_out, void *stream);

/*
 * rope_norm_qk_fwd -- the RMS norm of every query and key head with the
 * rotation in the same pass, out of place (or in place).
 *
 *   n = x / sqrt(mean(x^2) + eps),  y = R(t) (w * n)
 *
 * q, k: device, B sequences of S tokens of Hq (Hk) heads of D features; the
 *    strides of batch, token and head, in elements, stand in q_strides and
 *    k_strides (host arrays of 3, or NULL: dense, [B, H, S, D] or with
 *    seq_before_head [B, S, H, D]); features are dense.  Strides of sizes of
 *    one are not looked at.  Either may be missing (NULL, with 0 heads).
 * q_out, k_out: device, dense, in the order that seq_before_head says.  They
 *    may be q and k themselves where those are dense.
 * wq, wk: device [D], of weight_dtype (ROPE_F32 or dtype), or NULL (ones).
 * pos_idx: device int32 [S] (pos_batch_stride 0) or one row per sequence,
 *    pos_batch_stride entries apart, or NULL (row = index in the sequence).  -1: the norm
 *    alone; other rows outside the table: the norm alone, and the flag is raised.
 * D, rotary_dim: multiples of 16, 16 <= rotary_dim <= D <= 256; features past
 *    rotary_dim are normalised and weighted too.  dtype: ROPE_F32, ROPE_BF16 or
 *    ROPE_F16.  eps: >= 0, finite.
 * Arithmetic: fp32 throughout, one rounding to dtype at the end.  So the sum of a
 *    row's squares has to lie in fp32's range: rows with elements past 10^18 come out
 *    as zeros, and with eps = 0 rows of elements below 10^-19 lose precision (all
 *    below 10^-23 they come out as infinities, all zeros as NaN).
 * Errors: ROPE_ERR_UNSUPPORTED for other types, layouts, D, rotary_dim, strides
 *    that are not whole 16-byte vectors or pointers not 16-byte aligned;
 *    ROPE_ERR_INVALID_ARG for bad sizes (B * S above 2^31 - 1, negative or zero
 *    strides, a pos_batch_stride below S), null pointers, an output overlapping
 *    another argument; ROPE_ERR_CUDA if the launch fails.
 */
rope_status rope_norm_qk_fwd(const void *q, const void *k, void *q_out, void *k_out, const void *wq,
                             const void *wk, const float *cos, const float *sin,
                             const int32_t *pos_idx, int64_t pos_batch_stride, int64_t B, int32_t Hq,
                             int32_t Hk, int64_t S, int32_t D, const int64_t *q_strides,
                             const int64_t *k_strides, int32_t rotary_dim, int32_t layout,
                             int32_t seq_before_head, float eps, int32_t dtype, int32_t weight_dtype,
                             int64_t table_rows, void *stream);

/*
 * rope_norm_qk_bwd -- gradients of rope_norm_qk_fwd.  With r = 1 / sqrt(mean(x^2)
 * + eps), n = r x and g = R(-t) dy,
 *   dx = r (w * g - n mean(w * g * n)),   dw = sum over rows of g * n.
 * gq, gk: gradients of the outputs; dq, dk: gradients of q and k, written: all
 *    device, dense, in the outputs' order.  q, k: the forward call's inputs.
 * dwq, dwk: device [D], of weight_dtype, written, or NULL (not wanted).
 * workspace: device, 16-byte aligned, rope_norm_qk_workspace(D) bytes (NULL where
 *    neither dwq nor dwk is given); overwritten.
 * Without tokens, or without heads of its kind, a weight's gradient is zeros.  Sums
 *    are fp32 in an order that the sizes alone give: the same call gives the same bits.
 * Everything else, and errors: as rope_norm_qk_fwd; an output may overlap no
 *    other argument.
 */
rope_status rope_norm_qk_bwd(const void *q, const void *k, const void *gq, const void *gk, void *dq,
                             void *dk, const void *wq, const void *wk, void *dwq, void *dwk,
                             const float *cos, const float *sin, const int32_t *pos_idx,
                             int64_t pos_batch_stride, int64_t B, int32_t Hq, int32_t Hk, int64_t S,
                             int32_t D, const int64_t *q_strides, const int64_t *k_strides,
                             int32_t rotary_dim, int32_t layout, int32_t seq_before_head, float eps,
                             int32_t dtype, int32_t weight_dtype, int64_t table_rows, void *workspace,
                             int64_t workspace_bytes, void *stream);

/* rope_norm_qk_workspace -- bytes of workspace of rope_norm_qk_bwd (-1 for a D
 * that it does not take). */
int64_t rope_norm_qk_workspace(int32_t D);

/*
 * rope_attention_fwd -- attention forward with the rotation fused into the
 * loads of Q and K ("rotary-embedding-torch", flash_attn_with_rotary: the
 * rotary transformation is applied to the loaded Q and K blocks inside the
 * attention kernel, so rotated Q and K are never written to global memory).
 *
 *   o = softmax(scale * rot(q) rot(k)^T + mask) v
 *
 * q: device [B, Hq, Sq, D]; k, v: device [B, Hk, Sk, D]; o: device
 *    [B, Hq, Sq, D], written; all of `dtype` (ROPE_BF16 or ROPE_F16), dense.
 *    Hq must be a multiple of Hk (GQA/MQA: query head h uses key/value head
 *    h / (Hq/Hk)).
 * cos, sin: the rotation table (rope_tables_build or rope_tables_build_ex, any
 *    frequency mode), [table_rows, rotary_dim/2].
 * pos_q, pos_k: device int32 [Sq], [Sk] or NULL (row = index); -1 leaves a
 *    token unrotated (pos_mask); other out-of-range values are not rotated and
 *    raise the flag that rope_check_errors reports.
 * rotary_dim: multiple of 16, 16 <= rotary_dim <= D; D is 64 or 128.
 * layout: pair layout of the rotation.  causal: 0 or 1; the mask is aligned
 *    to the bottom right (query i sees key j when j <= i + Sk - Sq); a query
 *    row that sees no key gets zeros.
 * softmax_scale: > 0, or <= 0 for 1/sqrt(D).
 * k_workspace: NULL, or a device buffer of workspace_bytes >= B * Hk * Sk *
 *    D * 2 bytes, 16-byte aligned, overlapping no other argument; owned by
 *    the caller and overwritten.  NULL: every CTA rotates the key tiles it
 *    reads in shared memory, and rot(K) is never written.  Given: rot(K) is
 *    written there once per call by the rotation kernel (rope_apply_qk's
 *    arithmetic, so the same bits), then the attention kernel reads the
 *    rotated keys (for D = 128 on pairs of SMs, with no CTA rotating key
 *    tiles).  Under GQA every key tile is read by many CTAs, so for long
 *    sequences the workspace path is the faster one; both give the same
 *    result bit for bit.  Q is rotated inside the attention kernel either way.
 * Arithmetic: the rotated q and k rows are rounded to `dtype`, S = q k^T is
 *    accumulated in fp32 in tensor memory, P is rounded to `dtype` for the
 *    P v product (fp32 accumulation), o is rounded once.
 * Errors: ROPE_ERR_UNSUPPORTED for other dtypes, D, rotary_dim, layouts or
 *    pointers not 16-byte aligned; ROPE_ERR_INVALID_ARG for bad sizes, null
 *    pointers, o overlapping an input, a workspace too small or overlapping;
 *    ROPE_ERR_CUDA if the launch fails, which includes more than 65535
 *    query tiles per head -- Sq > 65535 * 128 when Hq / Hk is even, else
 *    Sq > 65535 * 256.  B, Hq or Sq zero: nothing to do, ROPE_OK.  Asynchronous on `stream`; rope_check_errors later reports
 *    out-of-range positions and, should a wait inside the kernel expire (about
 *    2 s; o is then not written), ROPE_ERR_KERNEL_TIMEOUT.
 */
rope_status rope_attention_fwd(const void *q, const void *k, const void *v, void *o,
                               const float *cos, const float *sin, const int32_t *pos_q,
                               const int32_t *pos_k, int64_t B, int32_t Hq, int32_t Hk, int64_t Sq,
                               int64_t Sk, int32_t D, int32_t rotary_dim, int32_t layout,
                               int32_t causal, float softmax_scale, int32_t dtype,
                               int64_t table_rows, void *k_workspace, int64_t workspace_bytes,
                               void *stream);

/*
 * rope_attention_fwd_masked -- rope_attention_fwd with a boolean attention
 * mask ("rotary-embedding-torch", flash_attn_with_rotary / Input Tensor
 * Shapes: attn_mask, batch x seq_len_k or batch x seq_len_q x seq_len_k,
 * whose False entries are excluded like masked scores):
 *
 *   o = softmax(scale * rot(q) rot(k)^T + causal mask + attn_mask) v
 *
 * attn_mask: device bytes, 0 = the key is hidden from the query (its score
 *    becomes -inf), any other value = visible (torch.bool tensors qualify):
 *      mask_kind ROPE_MASK_KEYS:       [B, Sk], the same for every query
 *                                      (padded batches: key padding);
 *      mask_kind ROPE_MASK_QUERY_KEYS: [B, Sq, Sk], one row per query (read
 *                                      as 16-byte vectors when the pointer
 *                                      is 16-byte aligned and Sk % 16 == 0,
 *                                      else byte by byte);
 *      mask_kind ROPE_MASK_NONE:       ignored (may be NULL): rope_attention_fwd.
 *    Dense, contiguous, shared by all heads; it must not overlap o or the
 *    workspace.  The mask applies together with `causal`; a query row that
 *    sees no key gets zeros.
 * Key tiles a [B, Sk] mask hides entirely: with a k_workspace of at least
 *    W + 4 B bytes, W = B * Hk * Sk * D * 2 rounded up to a multiple of 16,
 *    the call also writes there (from byte W) the number of 128-key tiles up
 *    to each batch entry's last visible key, and the attention kernels skip
 *    the tiles past it (the result is the same bit for bit: hidden keys only
 *    add exact zeros).  With a smaller workspace, or none, every tile is
 *    computed.
 * Padding: with at least W + 8 B bytes, the call also writes (from byte
 *    W + 4 B) each entry's prefix length, L when its mask shows exactly the
 *    keys [0, L), else -1; the attention kernels of the workspace path
 *    then compute such an entry as an unmasked one with L keys, without
 *    reading its mask (the same bits).
 * Everything else as rope_attention_fwd.
 * Errors: as rope_attention_fwd; also ROPE_ERR_UNSUPPORTED for a mask_kind
 *    outside the enum and ROPE_ERR_INVALID_ARG for a NULL mask (with Sk > 0)
 *    or one that overlaps o or the workspace.
 */
rope_status rope_attention_fwd_masked(const void *q, const void *k, const void *v, void *o,
                                      const float *cos, const float *sin, const int32_t *pos_q,
                                      const int32_t *pos_k, int64_t B, int32_t Hq, int32_t Hk,
                                      int64_t Sq, int64_t Sk, int32_t D, int32_t rotary_dim,
                                      int32_t layout, int32_t causal, float softmax_scale,
                                      int32_t dtype, int64_t table_rows, const uint8_t *attn_mask,
                                      int32_t mask_kind, void *k_workspace,
                                      int64_t workspace_bytes, void *stream);

/*
 * rope_attention_fwd_noalloc -- rope_attention_fwd with the key workspace
 * taken from a fixed device array inside this library (32 MiB), for callers
 * that cannot allocate device memory at call time: an engine that has
 * reserved the device's memory for its own pool, plugin code limited to the
 * buffers its host framework hands it, or a latency-critical path that
 * cannot afford cudaMalloc.  The pages have no counterpart of this entry
 * point; it is an addition of this library.
 *
 * Arguments, result and errors: as rope_attention_fwd with k_workspace set,
 * except that rot(K) goes to the library's array.  The arguments are checked
 * first, exactly as rope_attention_fwd checks them (its error, if any, is
 * returned); then ROPE_ERR_UNSUPPORTED when B * Hk * Sk * D * 2 bytes exceed
 * 32 MiB (33554432 bytes).  Both happen before anything touches the device.
 * Nothing is allocated or freed, and no allocating library routine is called.
 * Set-up: the first call on a device (with that device current) looks up the
 *    array's device address once (cudaGetSymbolAddress) and caches it; make
 *    that first call before any stream capture.  The cached address belongs
 *    to the device's context as it was then: after cudaDeviceReset (or any
 *    reset of the primary context) the process must be restarted before this
 *    entry point is called again.
 * Sharing: every device that loads the library holds the 32 MiB array until
 *    the process exits.  All calls on a device share it; each call rewrites
 *    the part it uses before reading it (nothing needs to start at zero), and
 *    calls whose work overlaps on the GPU (on streams not ordered with each
 *    other) race on it.
 */
rope_status rope_attention_fwd_noalloc(const void *q, const void *k, const void *v, void *o,
                                       const float *cos, const float *sin, const int32_t *pos_q,
                                       const int32_t *pos_k, int64_t B, int32_t Hq, int32_t Hk,
                                       int64_t Sq, int64_t Sk, int32_t D, int32_t rotary_dim,
                                       int32_t layout, int32_t causal, float softmax_scale,
                                       int32_t dtype, int64_t table_rows, void *stream);

/*
 * Serving: packed sequences and a paged cache.
 *
 * Packed sequences.  The tokens of n_seqs sequences lie one after the other
 *   in [total, H, D] tensors; sequence b holds the tokens cu[b] .. cu[b+1] - 1
 *   (cu: device int32[n_seqs + 1], 0 <= cu[b] <= cu[b+1] <= total; lengths of
 *   zero are allowed, and so are rows before cu[0] and from cu[n_seqs] on,
 *   which belong to no sequence: the rows of an output there keep what they
 *   hold).  A token stride, in elements and a multiple of 8, lets an input be
 *   a view of a fused projection's output; heads and features are dense.
 * Paged cache.  k_pages, v_pages: device [n_pages, Hk, page_size, D] of the
 *   element type; page_size is 16, 32, 64 or 128.  A block list (device
 *   int32) names the pages of a sequence in order: its key i lies in row
 *   i mod page_size of page list[i / page_size].  Entries past a sequence's
 *   last key, and rows of a page past it, may hold anything.  Cached keys are
 *   rotated keys.
 * Element types ROPE_BF16 and ROPE_F16; D is 64 or 128; rotary_dim is a
 *   multiple of 16, 16 <= rotary_dim <= D; pointers to 16-bit and fp32 data
 *   are 16-byte aligned.  What only the device can see -- offsets, lengths,
 *   page numbers, positions -- is checked there: nothing out of range is read
 *   or written, and rope_check_errors reports ROPE_ERR_BAD_INDEX (positions:
 *   ROPE_ERR_POS_OUT_OF_RANGE).
 */

/*
 * rope_cache_append -- rotate new keys and write them, and their values, into
 * the pages of a cache.
 *
 * Token t of sequence b becomes key s = cache_lens[b] + t - cu[b] of its
 * sequence:
 *   k_pages[p, h, s mod page_size, :] = rot(k[t, h, :]),
 *   v_pages[p, h, s mod page_size, :] = v[t, h, :],
 *   p = block_table[b * max_blocks + s / page_size].
 * k, v: device [total, Hk, D], token strides k_stride, v_stride.
 * block_table: device int32[n_seqs, max_blocks].
 * cache_lens: device int32[n_seqs], the keys each sequence holds already
 *   (read only: the caller advances it).
 * pos: device int32[total] or NULL.  The key of token t is rotated with table
 *   row pos[t] (-1: not rotated), or pos_offset + s when pos is NULL
 *   (pos_offset >= 0: the length of a prefix kept elsewhere).  A row outside
 *   the table leaves the key unrotated (it is written) and raises the flag.
 * Tokens with a page number or a block outside the ranges are not written
 *   and raise the flag.  When two tokens go to the same row of the same page,
 *   either may be the one that remains.
 * Arithmetic: as rope_apply_qk (one rounding; the same bits); values are copied.
 * total = 0 or n_seqs = 0 or Hk = 0: nothing to do, ROPE_OK.
 * Errors: ROPE_ERR_UNSUPPORTED for other dtypes, layouts, D, rotary_dim,
 *   page_size, strides not a multiple of 8 or pointers not 16-byte aligned;
 *   ROPE_ERR_INVALID_ARG for bad sizes, a token stride below Hk * D, null
 *   pointers, a pool overlapping another argument; ROPE_ERR_CUDA if the
 *   launch fails.
 */
rope_status rope_cache_append(const void *k, const void *v, void *k_pages, void *v_pages,
                              const int32_t *block_table, const int32_t *cu_seqlens,
                              const int32_t *cache_lens, const float *cos, const float *sin,
                              const int32_t *pos, int64_t pos_offset, int64_t n_seqs,
                              int64_t total, int64_t k_stride, int64_t v_stride, int32_t Hk,
                              int32_t D, int32_t rotary_dim, int32_t layout, int32_t page_size,
                              int64_t n_pages, int64_t max_blocks, int32_t dtype,
                              int64_t table_rows, void *stream);

/*
 * rope_norm_cache_append -- rope_cache_append for a model that normalises
 * queries and keys: the new tokens' queries, normalised and rotated, into a dense
 * tensor, their keys, normalised and rotated, and values into the pages.
 *
 * q: device [total, Hq, D], token stride q_stride; q_out: device [total, Hq, D],
 *    dense, written for tokens of the sequences; it may be q itself where that is
 *    dense.  A token's query is rotated with the table row of its key.
 * wq, wk, eps, weight_dtype: as rope_norm_qk_fwd.  Hq or Hk may be 0.
 * Everything else, and errors: as rope_cache_append.  A token whose page is bad has
 *    its query written and its key and value not.
 */
rope_status rope_norm_cache_append(const void *q, const void *k, const void *v, void *q_out,
                                   void *k_pages, void *v_pages, const void *wq, const void *wk,
                                   const int32_t *block_table, const int32_t *cu_seqlens,
                                   const int32_t *cache_lens, const float *cos, const float *sin,
                                   const int32_t *pos, int64_t pos_offset, int64_t n_seqs,
                                   int64_t total, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, int32_t Hq, int32_t Hk, int32_t D,
                                   int32_t rotary_dim, int32_t layout, float eps, int32_t page_size,
                                   int64_t n_pages, int64_t max_blocks, int32_t dtype,
                                   int32_t weight_dtype, int64_t table_rows, void *stream);

/*
 * rope_attention_packed_fwd -- attention with rotary Q/K over packed
 * sequences of different lengths (whole prompts, or their last tokens).
 *
 *   o_i = softmax(scale * rot(q_i) rot(K_b)^T + mask) V_b
 *
 * for the tokens i of sequence b, whose queries are tokens cu_seqlens_q[b] ..
 * and whose keys are tokens cu_seqlens_k[b] .. of their tensors.  With causal,
 * query i of Lq sees key j of Lk when j <= i + Lk - Lq; a query that sees no
 * key gets zeros.
 * q: device [total_q, Hq, D], token stride q_stride; k, v: device [total_k,
 *    Hk, D], token strides k_stride, v_stride; o: device [total_q, Hq, D],
 *    dense, written (rows of no sequence are not).  Hq is a multiple of Hk.
 * cu_seqlens_q, cu_seqlens_k: device int32[n_seqs + 1]; they may be the same.
 * pos_q, pos_k: device int32[total_q], int32[total_k] or NULL.  NULL: a
 *    token's table row is its index among its sequence's queries (keys).
 *    -1: not rotated; other rows outside the table are not rotated and raise
 *    the flag.  Entries of tokens of no sequence are not looked at.
 * causal, softmax_scale: as rope_attention_fwd.
 * workspace: device, 128-byte aligned, at least
 *    rope_attention_packed_workspace(...) bytes; overwritten (the rotated
 *    keys, the list of work and the copy engine's maps).
 * A sequence offset out of range or out of order (ROPE_ERR_BAD_INDEX), or a
 *    sequence longer than the table when its positions are NULL
 *    (ROPE_ERR_POS_OUT_OF_RANGE), is found on the device: the flag is raised
 *    and nothing of o is written.
 * Arithmetic: as rope_attention_fwd.  Nothing of another sequence reaches a
 *    query, whatever it holds; a NaN or infinity in v may reach queries of its
 *    own sequence that do not see its key (their probability 0 times it).
 * Errors: ROPE_ERR_UNSUPPORTED for other dtypes, D, rotary_dim, layouts,
 *    strides not a multiple of 8 or unaligned pointers; ROPE_ERR_INVALID_ARG
 *    for bad sizes, token strides below a token's row, null pointers, a
 *    workspace too small, o or the workspace overlapping another argument;
 *    ROPE_ERR_CUDA if a launch fails.  Asynchronous on `stream`; a wait inside
 *    the kernel is bounded as in rope_attention_fwd.
 */
rope_status rope_attention_packed_fwd(const void *q, const void *k, const void *v, void *o,
                                      const float *cos, const float *sin, const int32_t *pos_q,
                                      const int32_t *pos_k, const int32_t *cu_seqlens_q,
                                      const int32_t *cu_seqlens_k, int64_t n_seqs, int64_t total_q,
                                      int64_t total_k, int64_t q_stride, int64_t k_stride,
                                      int64_t v_stride, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t rotary_dim, int32_t layout, int32_t causal,
                                      float softmax_scale, int32_t dtype, int64_t table_rows,
                                      void *workspace, int64_t workspace_bytes, void *stream);

/* rope_attention_packed_workspace -- bytes of workspace for a call of these
 * sizes (0 when there is nothing to do, -1 for sizes it does not take). */
int64_t rope_attention_packed_workspace(int64_t n_seqs, int64_t total_q, int64_t total_k, int32_t Hq,
                                        int32_t Hk, int32_t D);

/*
 * rope_attention_decode_fwd -- attention of one new token per sequence, over
 * a prefix that all sequences of the batch share and a suffix of each one's
 * own, both in the pages of a cache of rotated keys (rope_cache_append).
 *
 *   o_b = softmax(scale * rot(q_b) [K_prefix; K_b]^T) [V_prefix; V_b]
 *
 * The prefix's keys and values are read once for every 256 rows (sequence, head)
 * of a key head, not once for every sequence: rows of up to 16 heads of a group
 * (the largest power of two that divides its size) and of as many sequences as fit.
 * q: device [B, Hq, D], row stride q_stride (elements, a multiple of 8);
 *    o: device [B, Hq, D], dense, written.  Hq is a multiple of Hk.
 * k_pages, v_pages: the cache, [n_pages, Hk, page_size, D].
 * prefix_table, prefix_len: device int32, ceil(prefix_len / page_size) pages;
 *    prefix_len = 0: no prefix (the table may be NULL).
 * block_table: device int32[B, max_blocks]; seq_lens: device int32[B], the
 *    keys of each suffix, the new token's own among them (0 <= seq_lens[b] <=
 *    max_blocks * page_size; 0: the prefix alone).  A sequence without any key
 *    gets zeros.  Sequences may share pages.
 * pos_q: device int32[B] or NULL.  Query b is rotated with table row pos_q[b]
 *    (-1: not rotated), or prefix_len + seq_lens[b] - 1 when NULL.
 * softmax_scale: > 0, or <= 0 for 1/sqrt(D).
 * workspace: device, 128-byte aligned, at least
 *    rope_attention_decode_workspace(...) bytes; overwritten.
 * A length out of range is cut to the range, a page number out of range reads
 *    as zeros: the flag is raised (ROPE_ERR_BAD_INDEX), and the outputs of the
 *    sequences that use it mean nothing.  A query position outside the table
 *    is not rotated and raises ROPE_ERR_POS_OUT_OF_RANGE.
 * Arithmetic: rot(q) and the softmax probabilities are rounded to `dtype`
 *    for the products; sums, maxima and partial outputs are fp32; o is rounded
 *    once.  The split of the work depends on the sizes and the lengths alone:
 *    the same call gives the same bits.
 * Errors: ROPE_ERR_UNSUPPORTED for other dtypes, D, rotary_dim, layouts, page
 *    sizes, B > 4096, a stride not a multiple of 8 or unaligned pointers;
 *    ROPE_ERR_INVALID_ARG for bad sizes, null pointers, a workspace too small,
 *    o or the workspace overlapping another argument; ROPE_ERR_CUDA if a
 *    launch fails.  Asynchronous on `stream`; waits inside the kernels are
 *    bounded as in rope_attention_fwd.
 */
rope_status rope_attention_decode_fwd(const void *q, const void *k_pages, const void *v_pages, void *o,
                                      const int32_t *block_table, const int32_t *seq_lens,
                                      const int32_t *prefix_table, int64_t prefix_len,
                                      const float *cos, const float *sin, const int32_t *pos_q,
                                      int64_t B, int64_t q_stride, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t rotary_dim, int32_t layout, float softmax_scale,
                                      int32_t page_size, int64_t n_pages, int64_t max_blocks,
                                      int32_t dtype, int64_t table_rows, void *workspace,
                                      int64_t workspace_bytes, void *stream);

/* rope_attention_decode_workspace -- bytes of workspace for a call of these
 * sizes (0 when there is nothing to do, -1 for sizes it does not take). */
int64_t rope_attention_decode_workspace(int64_t B, int32_t Hq, int32_t Hk, int32_t D, int32_t page_size,
                                        int64_t max_blocks, int64_t prefix_len);

/*
 * rope_attention_paged_fwd -- attention of every sequence's new tokens, one or a
 * chunk of a prompt, over its keys in a paged cache (rope_cache_append or
 * rope_norm_cache_append them first).
 *
 *   o_i = softmax(scale * rot(q_i) K_b^T + mask) V_b
 *
 * for the tokens i of sequence b, whose queries are tokens cu_seqlens_q[b] .. of q
 * and whose seq_lens[b] keys, the new tokens' own among them, lie in its pages.
 * With causal, query i of Lq sees key j of Lk when j <= i + Lk - Lq; a query that
 * sees no key gets zeros.
 * q: device [total_q, Hq, D], token stride q_stride; o: device [total_q, Hq, D],
 *    dense, written (rows of no sequence are not).  Hq is a multiple of Hk.
 * k_pages, v_pages: the cache, [n_pages, Hk, page_size, D] of rotated keys.
 *    Sequences may share pages.
 * block_table: device int32[n_seqs, max_blocks]; cu_seqlens_q: device
 *    int32[n_seqs + 1]; seq_lens: device int32[n_seqs], 0 <= seq_lens[b] <=
 *    max_blocks * page_size.  A sequence may have no new tokens.
 * cos, sin: the rotation table, or both NULL: the queries are rotated already
 *    (rotary_dim and table_rows are not looked at then).
 * pos_q: device int32[total_q] table rows (-1: not rotated), or NULL for a query's index
 *    among its sequence's keys, Lk - Lq + i.
 * causal, softmax_scale: as rope_attention_fwd.
 * workspace: device, 128-byte aligned, at least
 *    rope_attention_paged_workspace(...) bytes; overwritten.
 * An offset or a length out of range (ROPE_ERR_BAD_INDEX) is found on the device:
 *    the flag is raised and nothing of o is written.  A page number out of range
 *    reads as zeros and raises the flag: outputs of sequences that use it mean
 *    nothing.  A table row out of range (but for rows before a sequence's first key
 *    when causal): the query is not rotated and ROPE_ERR_POS_OUT_OF_RANGE raised.
 * Arithmetic: rot(q) and the softmax probabilities are rounded to `dtype` for the
 *    products (for sequences of at most 8 rows, tokens * Hq / Hk, or one token of a
 *    group of up to 8 heads, they go in as two parts each and are not); sums, maxima
 *    and partial outputs are fp32; o is rounded once.  What lies behind a sequence's
 *    last key, and in other pages, reaches no query; a NaN or infinity in a value may
 *    reach queries of its sequence that do not see its key.  The split of the
 *    work depends on the sizes and the lengths alone: the same call gives the same
 *    bits.
 * Errors: ROPE_ERR_UNSUPPORTED for other dtypes, D, rotary_dim, layouts, page
 *    sizes, n_seqs > 4096, a stride not a multiple of 8 or unaligned pointers;
 *    ROPE_ERR_INVALID_ARG for bad sizes, null pointers, a workspace too small,
 *    o or the workspace overlapping another argument; ROPE_ERR_CUDA if a
 *    launch fails.  Asynchronous on `stream`; waits inside the kernels are
 *    bounded as in rope_attention_fwd.
 */
rope_status rope_attention_paged_fwd(const void *q, const void *k_pages, const void *v_pages, void *o,
                                     const int32_t *block_table, const int32_t *cu_seqlens_q,
                                     const int32_t *seq_lens, const float *cos, const float *sin,
                                     const int32_t *pos_q, int64_t n_seqs, int64_t total_q,
                                     int64_t q_stride, int32_t Hq, int32_t Hk, int32_t D,
                                     int32_t rotary_dim, int32_t layout, int32_t causal,
                                     float softmax_scale, int32_t page_size, int64_t n_pages,
                                     int64_t max_blocks, int32_t dtype, int64_t table_rows,
                                     void *workspace, int64_t workspace_bytes, void *stream);

/* rope_attention_paged_workspace -- bytes of workspace for a call of these
 * sizes (0 when there is nothing to do, -1 for sizes it does not take). */
int64_t rope_attention_paged_workspace(int64_t n_seqs, int64_t total_q, int32_t Hq, int32_t Hk, int32_t D,
                                       int32_t page_size, int64_t max_blocks);

/*
 * rope_check_errors -- synchronise `stream`, then report and clear the
 * current device's error flag.
 * Returns ROPE_ERR_CUDA if the stream reports an error, else
 * ROPE_ERR_KERNEL_TIMEOUT if a wait inside an attention kernel expired
 * (about 2 s; that launch stopped early and its output is incomplete), else
 * ROPE_ERR_BAD_INDEX if a serving call since the last check met a sequence
 * offset, a length or a page number out of range, else
 * ROPE_ERR_POS_OUT_OF_RANGE if any launch since the last check met an
 * out-of-range position index, else ROPE_OK.  The flag is shared by all
 * streams of the device.
 */
rope_status rope_check_errors(void *stream);

/*
 * rope_probe_wait_expiry -- diagnostic: exercise the path an expired wait
 * takes, without stalling any real kernel.  Two threads of one CTA wait, one
 * with each of the bounded mbarrier waits that the attention kernels use, on a
 * barrier that nothing arrives at; after `cycles` SM clock cycles (1 .. 4e9; 2e6
 * is about a millisecond), or about as long, the waits give up, and the timeout
 * bit of the device error flag is set, as by an expired wait inside those
 * kernels.  The next rope_check_errors then returns
 * ROPE_ERR_KERNEL_TIMEOUT and clears the flag.  The pages have no
 * counterpart; this is an addition of this library, for tests and for
 * callers that want to check their error handling.
 * Errors: ROPE_ERR_INVALID_ARG for cycles outside 1 .. 4e9 (nothing is
 *    launched); ROPE_ERR_CUDA if the launch fails.  Asynchronous on `stream`.
 */
rope_status rope_probe_wait_expiry(int64_t cycles, void *stream);

/* rope_status_string -- static, NUL-terminated name of a status value. */
const char *rope_status_string(rope_status status);

/*
 * rope_qk_kernel_variant -- which kernel rope_apply_qk would launch for
 * these arguments, without launching anything or touching the device.
 * Returns 0 when nothing would be launched (error or empty problem),
 * 2 for the element-wise kernel (any shape or alignment),
 * 3 for the register-staged 16-byte vector kernel (the automatic choice
 * for 16-byte aligned shapes whose rotary span is whole pairs of vectors).
 * Useful for tests and for callers checking that their tensors are aligned.
 */
int32_t rope_qk_kernel_variant(const void *q, const void *k, const float *cos, const float *sin,
                               const int32_t *pos_idx, int64_t B, int32_t Hq, int32_t Hk,
                               int64_t S, int32_t D, int32_t rotary_dim, int32_t layout,
                               int32_t seq_before_head, int32_t backward, int32_t dtype,
                               int64_t table_rows);

/*
 * rope_force_kernel_variant -- process-wide choice of the rotation kernel,
 * for tests and tuning: 0 = automatic (default), 2 or 3 as returned by
 * rope_qk_kernel_variant.  While 3 is forced, calls whose shapes or pointers
 * do not qualify for it return ROPE_ERR_UNSUPPORTED.  Both kernels compute
 * bit-identical results.  ROPE_ERR_INVALID_ARG for other values.
 */
rope_status rope_force_kernel_variant(int32_t variant);

/*
 * rope_tune_rotation_launch -- process-wide grid sizing of the vector
 * rotation kernel, for tuning and measurement; the results do not depend on
 * it.  The kernel splits its work, units of (TT consecutive tokens, one
 * head), into balanced contiguous runs, one per lane group of TT rows.
 *   ctas_per_sm: cap the grid at this many CTAs per SM (0 = as many as can
 *     be resident at once, the default; 1 .. 64 otherwise);
 *   min_units: the fewest units a run holds before the grid grows (0 = the
 *     default, 1);
 *   prefetch_next: 1 or 0 = while rotating a tile, prefetch the first heads
 *     of the run's next tile into L2 (the default); -1 = do not.
 * ROPE_ERR_INVALID_ARG for values outside these ranges (nothing changes).
 * The pages have no counterpart; this is an addition of this library.
 */
rope_status rope_tune_rotation_launch(int32_t ctas_per_sm, int32_t min_units,
                                      int32_t prefetch_next);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_H */
