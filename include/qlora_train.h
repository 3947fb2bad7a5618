/*
 * qlora_train.h — C ABI of what a training step needs next to the QLoRA
 * linears: the loss head with its gradient, and 8-bit checkpoints of the
 * linears' inputs with the backward pass that reads them.
 *
 * Sources (web pages, cited by title and section):
 *  - "QLoRA" encyclopedia entry (tonho.wtf), section "a ideia": the base is
 *    frozen and the gradient crosses it into the adapters; the head is part of
 *    the base, so its operator has a gradient towards the hidden states and
 *    none towards the weight.
 *  - same entry, section "como funciona": memory, not arithmetic, is what the
 *    method saves (FP8 constants, checkpointed activations, paged optimizer
 *    states).
 * The pages fix neither operator's arithmetic; the readings are stated here.
 *
 * Conventions as in qlora_nf4.h: the caller owns every buffer; calls only
 * enqueue work on `stream`; errors are reported before any work is enqueued;
 * pointers are 16-byte aligned; device-side conditions are OR-ed into the
 * optional device word d_status.  Results do not depend on the timing of the
 * GPU: sums run in a fixed order or are of integers, and repeated calls are
 * bitwise identical.
 */
#ifndef QLORA_TRAIN_H
#define QLORA_TRAIN_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bit: a label outside 0 .. vocab - 1 that is not ignore_index
 * (its token is then treated as ignored). */
#define QLORA_DEV_LABEL 4

/* ------------------------------------------------ 8-bit activation checkpoints
 *
 * A linear's input X is kept between forward and backward only for
 * dA = dU^T X.  Its 8-bit checkpoint holds, per row, blocks of 64 elements:
 *
 *   e    = the smallest integer with max|x| <= 448 * 2^e, at least -118 and at
 *          most 120 (an all-zero block: -118)
 *   exps [M, K/64] uint8   e + 127
 *   codes[M, K]    uint8   E4M3 round-to-nearest-even, saturating, of x * 2^-e
 *
 * 1 + 1/64 bytes per element instead of 2.  The value a code stands for,
 * x' = e4m3(code) * 2^e, is exact in bf16: a power of two only moves E4M3's
 * exponent.  (Above 1.9375 * 2^127 the nearest such value is 2^128, an infinity.)
 * A NaN keeps its place, an infinity comes back as one; both set
 * QLORA_DEV_NONFINITE.
 *
 * act8_quantize    X [M, K] bf16, row stride ldx elements (>= K, % 8 == 0)
 * act8_dequantize  x' as bf16 [M, K], row stride ldx; the gap between rows is
 *                  left as it was
 * K % 64 == 0, K >= 64, M >= 0 (0 = no-op), M < 2^31, M * K < 2^40, else
 * QLORA_ERR_SHAPE.  Bit-exact with the CPU oracle.
 */
QLORA_API qlora_status act8_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                                     uint8_t* exps, int32_t* d_status, void* stream);
QLORA_API qlora_status act8_dequantize(const uint8_t* codes, const uint8_t* exps, int64_t M, int64_t K,
                                       uint16_t* X, int64_t ldx, void* stream);

/*
 * The backward passes of qlora_nf4.h with the adapter's input given as its
 * 8-bit checkpoint (of X; for the dropout form, of X_drop, whose zeros stay
 * zeros): dA = dU^T X', everything else by the same formulas.  The rank-r
 * products (dU, dB, dA) take dU and s U as three bf16 parts (24 bits) and join
 * their accumulator's sums every 512 terms in fp32 with rounding to nearest: dA
 * and dB within 4e-6 of the sums of their terms' absolute values, whatever the
 * number of tokens (dA_jk: s sum_mn |dY_mn B_nj X'_mk|, dB_nj: s sum_m |dY_mn
 * U_mj|), and of random data within 4e-6 relative Frobenius error.
 * Arguments, constraints and errors as for qlora_linear_bwd, qlora_group_bwd
 * and qlora_linear_bwd_dropout; the workspace is
 * qlora_bwd_act8_workspace_size(M, N, K, members, r, dropout) bytes (members 1
 * for a single linear; dropout nonzero for the dropout form): the plain pass's
 * and 8 M members r more.
 */
QLORA_API size_t qlora_bwd_act8_workspace_size(int64_t M, int64_t N, int64_t K, int32_t members, int32_t r,
                                               int32_t dropout);
QLORA_API qlora_status qlora_linear_bwd_act8(const uint16_t* dY, const uint8_t* codes, const uint8_t* exps,
                                             const float* U, int64_t M, nf4_weight W, const uint16_t* A,
                                             const uint16_t* B, int32_t r, float s, void* dX, int32_t dx_dtype,
                                             float* dA, float* dB, void* ws, size_t ws_bytes, int32_t* d_status,
                                             void* stream);
QLORA_API qlora_status qlora_group_bwd_act8(const uint16_t* dY, const uint8_t* codes, const uint8_t* exps,
                                            const float* U, int64_t M, nf4_weight W, int32_t members,
                                            const int64_t* n_member, const uint16_t* A, const uint16_t* B, int32_t r,
                                            float s, void* dX, int32_t dx_dtype, float* dA, float* dB, void* ws,
                                            size_t ws_bytes, int32_t* d_status, void* stream);
QLORA_API qlora_status qlora_linear_bwd_dropout_act8(const uint16_t* dY, const uint8_t* codes, const uint8_t* exps,
                                                     const float* U, int64_t M, nf4_weight W, const uint16_t* A,
                                                     const uint16_t* B, int32_t r, float s, float p, uint64_t seed,
                                                     void* dX, int32_t dx_dtype, float* dA, float* dB, void* ws,
                                                     size_t ws_bytes, int32_t* d_status, void* stream);

/* ------------------------------------------------------------------ loss head
 *
 * Softmax cross entropy of the head's logits, in pieces of the vocabulary;
 * the [T, vocab] logits never exist:
 *
 *   l_tv   = sum_d H_td W_vd              (fp32 accumulation)
 *   lse_t  = log sum_v exp(l_tv)
 *   loss_t = lse_t - l_{t, label_t}       (0 for an ignored token)
 *   mean   = sum_t loss_t / count         (0 when count = 0)
 *   dH_t   = g_t sum_v (exp(l_tv - lse_t) - [v = label_t]) W_v
 *
 * A token counts unless its label is ignore_index (or out of range, see
 * QLORA_DEV_LABEL).  An ignored token's row of H may hold anything, NaN
 * included: its loss and its row of dH are exactly 0 (its lse is that of the
 * row as it stands).  Larger calls leave ignored rows out of the products that
 * make dH: a batch whose prompts are ignored costs that much less.  A
 * non-finite lse of a token that counts, made by the forward or the step or
 * given to the backward, sets QLORA_DEV_NONFINITE.
 *
 * The head: W [vocab, dim], either bf16 rows (`w`, row stride ld elements,
 * ld % 8 == 0, dim % 8 == 0) or, with w == NULL, NF4 (codes, c8, s2 and an
 * optional mean as in nf4_weight; dim % 64 == 0), dequantised inside the
 * products (up to 128 tokens) or piece by piece before them.
 */
typedef struct {
  const uint16_t* w;    /* bf16 rows, or NULL for an NF4 head */
  int64_t ld;           /* row stride of w in elements (ignored for NF4) */
  const uint8_t* codes; /* NF4 storage of [vocab, dim], used when w is NULL */
  const uint8_t* c8;
  const float* s2;
  const float* mean;
  int64_t vocab;
  int64_t dim;
} qlora_head;

/*
 * qlora_head_loss_fwd — per-token losses and their mean.
 *   H      [T, dim] bf16, row stride ldh elements (>= dim, % 8 == 0)
 *   labels [T] int64
 *   loss   [T] fp32 out;  lse [T] fp32 out (keep it for the backward)
 *   stats  [2] fp32 out: the mean over the tokens that count, and their number
 *
 * qlora_head_loss_bwd — dH from the saved lse and any gradient of the losses.
 *   dloss  [T] fp32, the gradient of every token's loss (stats NULL), or [1],
 *          the gradient of the mean (stats from the forward: g_t = dloss / count)
 *   dH     [T, dim] bf16 out, row stride lddh (>= dim, % 8 == 0)
 *
 * qlora_head_loss_step — both in one call, with two products of T x vocab x dim
 *   instead of the pair's three, for a gradient that is known beforehand:
 *   g_t = scale * weight_t (weight [T] fp32), or, with weight NULL,
 *   g_t = scale / count (the gradient of scale * mean).  loss, lse and stats
 *   are those of the forward, unscaled and unweighted.
 *
 * T >= 0 (0 = no-op; stats is then {0, 0}), vocab >= 1, both below 2^31 - 256,
 * dim in 8 .. 2^20, vocab * dim < 2^40, ld / ldh / lddh < 2^31, else
 * QLORA_ERR_SHAPE; so does ceil(T / 256) x ceil(max(vocab, dim) / 256) from
 * 2^23.  dH may be H itself (the same rows).  The per-token vectors and stats need
 * their type's alignment only (a shifted view of the labels is fine).
 * Workspaces: qlora_head_loss_workspace_size(T, vocab, dim, nf4, op) bytes with
 * nf4 nonzero for an NF4 head and op one of QLORA_HEAD_FWD / _BWD / _STEP.
 * Beside per-token words it holds per half tile of logits (128, or fewer
 * columns where that fills the GPU) 8 bytes (forward) or 12 (step), a piece of the
 * probabilities (backward, step: about 128 MB in bf16, at least 2048 columns),
 * the rows of H that count (backward of larger calls: bf16 [T, dim]), fp32 sums
 * [T, dim] (with several pieces) and of tiles of dH whose contraction is
 * divided (at most 39 MB), and, for more than 128 tokens, a dequantised piece of an
 * NF4 head (at most 128 MB, at least 2048 rows).
 * Accuracy: exact bf16 inputs, fp32 accumulation and softmax; a small loss keeps
 * its digits (the label's logit stays out of the sum).  The probabilities of the
 * others enter the second product as bf16, the label's coefficient in fp32 with
 * their roundings in it, so that what W's rows share cancels in dH.  Beside what
 * the logits' fp32 errors make of p, an element of dH is off by at most
 *   |g_t| (2^-8 sum_v p_tv |W_vd - W_label,d| + e sum_v p_tv |W_vd|) + 2^-8 |dH_td|
 * (2 2^-8 in a row of the step that has logits beyond +-40), with e = 2^-23 for
 * every 16 columns of a piece (measured: about 2^-26): the fp32 sum.  On random
 * data that is 1.7e-3 relative (Frobenius).  The backward's label coefficient,
 * expm1(l_label - lse), has the rounding of the lse that it is given, 2^-24
 * |lse| absolute, the step's has not: it keeps its digits for any token.
 */
#define QLORA_HEAD_FWD 0
#define QLORA_HEAD_BWD 1
#define QLORA_HEAD_STEP 2
QLORA_API size_t qlora_head_loss_workspace_size(int64_t T, int64_t vocab, int64_t dim, int32_t nf4, int32_t op);
QLORA_API qlora_status qlora_head_loss_fwd(const uint16_t* H, int64_t ldh, int64_t T, qlora_head head,
                                           const int64_t* labels, int64_t ignore_index, float* loss, float* lse,
                                           float* stats, void* ws, size_t ws_bytes, int32_t* d_status, void* stream);
QLORA_API qlora_status qlora_head_loss_bwd(const uint16_t* H, int64_t ldh, int64_t T, qlora_head head,
                                           const int64_t* labels, int64_t ignore_index, const float* lse,
                                           const float* dloss, const float* stats, uint16_t* dH, int64_t lddh,
                                           void* ws, size_t ws_bytes, int32_t* d_status, void* stream);
QLORA_API qlora_status qlora_head_loss_step(const uint16_t* H, int64_t ldh, int64_t T, qlora_head head,
                                            const int64_t* labels, int64_t ignore_index, const float* weight,
                                            float scale, float* loss, float* lse, float* stats, uint16_t* dH,
                                            int64_t lddh, void* ws, size_t ws_bytes, int32_t* d_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_TRAIN_H */
