// train.h — host-side launch functions of the training-step kernels (internal
// to the library): 8-bit activation checkpoints (act8.cu) and the loss head
// (head_loss.cu).
#pragma once

#include "../../include/qlora_train.h"
#include "kernels.h"

namespace qnf4 {

// ------------------------------------------------------------------ act8.cu

cudaError_t launch_act8_quantize(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, uint8_t* exps,
                                 int32_t* status, cudaStream_t stream);
cudaError_t launch_act8_dequantize(const uint8_t* codes, const uint8_t* exps, int64_t M, int64_t K, uint16_t* x,
                                   int64_t ldx, cudaStream_t stream);

// dA[j, k] = sum_m dU[m, j] X'[m, k] from the checkpoint (SkinnyArgs as for
// mode DA of skinny.cu): tm_du the bf16 hi/lo of dU [M, 2 ra] box {64, 64}
// SW128, tm_du3 its third parts the same, tm_x the codes [M, K] u8 box {128,
// 64}; exps [M, K / 64].
cudaError_t launch_act8_da(const CUtensorMap& tm_du, const CUtensorMap& tm_du3, const CUtensorMap& tm_x,
                           const uint8_t* exps, const SkinnyArgs& a, int grid_rows, int splits, cudaStream_t stream);

// ------------------------------------------------------------- head_loss.cu

constexpr int kHeadTile = 256;  // tokens, and columns, of a CTA pair's tile

enum HeadMode {
  kHeadLoss = 0,  // logits of a piece -> per-tile softmax statistics
  kHeadProb = 1,  // logits of a piece -> probabilities, bf16 (0 at the label)
  kHeadExp = 2,   // logits of a piece -> exponentials, bf16, and the statistics
  kHeadGrad = 3   // those times the piece's weight -> dH (or its fp32 sum so far)
};

// CTA pairs, or CTAs, of a persistent launch: one per TPC, one per SM.
constexpr int head_workers(bool pair) { return pair ? 74 : 148; }

// How dH's tiles go over the workers: whole tiles in turn, `full` each, then
// the `rest` that do not fill a wave, in parts of their contraction where the
// parts' sums (about 24 stages' time to write and join) cost less than the idle
// workers.  Up to half a wave: as many slices of `per` stages as there are
// workers for.  More: a worker a tile does the first `per` stages, and every
// worker left over the remaining ones of `help` tiles.  Either way the workers
// on one operand's rows walk the same stages together (ranges that start
// anywhere balance better, and read the operands from memory once per tile:
// 2048 x 50000 x 1024 412 us against 375).  8192 x 50257 x 1024, three quarters
// of the tokens counting: 96 tiles, 92 us a piece in parts, 105 whole.
struct HeadTail {
  int full, rest, parts, per, help;
};
constexpr int kHeadPartCost = 24;

inline __host__ __device__ HeadTail head_tail(int tiles, int kst, int workers) {
  HeadTail t{tiles / workers, tiles % workers, 1, kst, 0};
  if (t.rest == 0) return t;
  int parts = workers / t.rest, per = 0, help = 0;
  if (parts > 1) {
    per = (kst + parts - 1) / parts;
    per = per < 8 ? 8 : per;
    parts = (kst + per - 1) / per;
  } else {
    help = (t.rest + workers - t.rest - 1) / (workers - t.rest);
    per = (kst * help + help) / (help + 1);
    parts = 2;
  }
  if (per + kHeadPartCost < kst) {
    t.parts = parts;
    t.per = per;
    t.help = help;
  }
  return t;
}

struct HeadArgs {
  int pair, nf4;          // which kernel: tiles of 256 tokens on CTA pairs; (single CTAs) W from its codes
  int T;                  // tokens
  // The rows that count (see head_loss.cu), or null where the operand's rows
  // are the tokens: their number, the token of a row (Prob, Grad), and the row
  // of a token or -1 (Exp).
  const int32_t* nrows;
  const int32_t* rows;
  const int32_t* place;
  int arows;              // token rows of a copy: 128, or for fewer tokens those, to a multiple of 8
  int ncols;              // columns of this product: the piece's vocabulary rows, or dim (Grad)
  int kst;                // 64-deep contraction stages
  int kchunk;             // stages summed in one accumulator
  int kfull, workers;     // Grad: stages of a full piece, and CTA pairs or CTAs, for head_tail
  int b_row0;             // the piece's first row in W's tensor map
  int64_t v0;             // the piece's first vocabulary index
  int wrows;              // the piece's vocabulary rows
  int64_t vocab;
  int mtiles, ntiles;
  int tw;                 // columns of a tile: a multiple of 32 up to 256, NF4 128 (Grad: 256)
  const int64_t* labels;
  int64_t ignore;
  float2* part;           // Loss, Exp: (reference, sum of the others' exponentials) [half tile][T] of the piece
  float* rsum;            // Exp: their sum as rounded to bf16, [half tile][T]
  // Prob, Grad (backward): what rounding the probabilities added to their sum, [T] integers, cleared before
  unsigned long long* rounding;
  const float* lse;       // Prob: [T]
  float* coef_out;        // Prob: [T] probability of the label less 1, or null
  const uint16_t* h;      //   from the operand's rows, stride ldh
  int64_t ldh;
  uint16_t* g;            // Prob, Exp: [rows, ldg]
  int64_t ldg;
  uint32_t* zero;         // Loss, Exp: words cleared by the first CTA (combine's counters)
  int zero_count;
  // Grad
  int first, last;        // of the pieces
  float* acc;             // fp32 sums of the pieces so far, and of parts (blocked by tile)
  const float* alpha;     // [T] factor of the sum so far (null: 1)
  uint16_t* dh;           // [T, ldd]
  int64_t ldd;
  const float* dloss;     // per-token gradients, or one number with `stats` (backward)
  const float* stats;
  const float* row_root;  // [T] 1 / root of the softmax denominators (step), null in the backward
  const float* coef;      // [T] coefficient of W[label] beside the sum: backward, probability of the label less 1
  const float* weight;    // [T] or null (step)
  float scale;
  const int32_t* count;   // tokens that count (step, weight null)
  qlora_head head;        // the label's row of W; NF4: its codes
  Nf4Tables tab;
  int32_t* status;
};

//   tm_a: H [T, dim] (Grad: the piece's [T, ntiles tw]) box {64, arows} SW128;
//   tm_b: W rows, box {64, tw / 2 (pair) or tw} SW128 (Grad: {64, 64}); with
//   nf4 W's codes [vocab, dim / 2], box {32, tw} SW32 (Grad: {128, 64} SW128).
cudaError_t launch_head_gemm(int mode, const CUtensorMap& tm_a, const CUtensorMap& tm_b, const HeadArgs& a,
                             cudaStream_t stream);

// The tokens that count: rows [T], place [T], nrows [1]; with `out` their rows
// of h to out [T, dim], and zeros to the other rows of dh (which may be h).
struct HeadRowsArgs {
  const int64_t* labels;
  int64_t ignore, vocab, T, chunk;
  int32_t *rows, *place, *nrows, *status;
  unsigned long long* rounding;  // [T] to be cleared, or null
  const uint16_t* h;
  int64_t ldh, dim;
  uint16_t *out, *dh;
  int64_t ldd;
};
cudaError_t launch_head_rows(HeadRowsArgs a, cudaStream_t stream);
cudaError_t launch_head_clear(unsigned long long* rounding, int64_t T, cudaStream_t stream);

// Joins the parts of Grad's tiles after the last piece; `tiles`: an upper bound
// of those in parts.
cudaError_t launch_head_finish(const HeadArgs& a, int tiles, cudaStream_t stream);

// Joins the per-tile statistics of every row; see head_loss.cu.
struct HeadCombineArgs {
  int T, nparts;
  int part_cols;           // columns a part covers
  const float2* part;      // [nparts][T]
  const uint16_t* h;       // H [T, ldh], and the head: the label's logit
  int64_t ldh;
  qlora_head head;
  Nf4Tables tab;
  const int64_t* labels;
  int64_t ignore;
  int64_t vocab;
  int first, last;         // of the pieces (the forward combines once: both)
  const float* rsum;       // step: [nparts][T] sum of the exponentials as rounded
  float2* run;             // step: running (reference, sum) [T], and of the rounded
  float* run_rsum;
  float* alpha;            // step: [T]
  uint16_t* e;             // step: the piece's exponentials [rows, lde], or null
  int64_t lde;
  const int32_t* place;    // step: row of a token in e or -1, or null; then, with the last piece,
  uint16_t* dh;            //   the other rows of dH become zero
  int64_t ldd, dim;
  float* row_root;         // step: [T] 1 / root of the softmax denominator
  float* coef;             // step: [T] coefficient of the label's row of W
  int32_t* counters;       // [2]: tokens that count, blocks done; cleared before
  double* block_sum;       // [blocks]
  float* loss;
  float* lse;
  float* stats;
  int32_t* status;
};
int head_combine_blocks(int64_t T);
cudaError_t launch_head_combine(const HeadCombineArgs& a, cudaStream_t stream);

}  // namespace qnf4
