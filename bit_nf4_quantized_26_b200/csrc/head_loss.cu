// head_loss.cu — softmax cross entropy of the head's logits and its gradient
// towards the hidden states, in pieces of the vocabulary ("QLoRA" encyclopedia
// entry, tonho.wtf, section "a ideia": the base is frozen and the gradient
// crosses it into the adapters).
//
//   l = H W^T    lse = log sum exp l    loss = lse - l[label]
//   dH = g (exp(l - lse) - onehot) W
//
// The logits exist only as fp32 tiles in tensor memory.  One GEMM kernel makes
// every product; what its epilogue does with a tile is the mode:
//
//   Loss  per row and half tile the maximum m and sum exp(l - m): 8 bytes (the
//         label's column apart: head_combine_kernel makes its logit)
//   Prob  exp(l - lse), 0 at the label, rounded to bf16
//   Exp   exp(l - ref), 0 at the label, rounded to bf16, and (ref, sum), the
//         label apart: the gradient's operand before lse is known.  ref is 0 while the maximum
//         of the row's half tile lies within +-40 (exp then stays far inside
//         bf16's and fp32's range, and the reference costs no precision: both
//         types float), else that maximum
//   Grad  (second product) the piece's bf16 [T, piece] operand times W's rows
//         of the piece, added to the fp32 sum of the pieces before
//
// The step joins each piece's (ref, sum) per row (head_combine_kernel); rows
// whose tiles took different references have those tiles' exponentials
// rescaled to a common one, and `alpha` rescales the sum of earlier pieces:
// both leave ordinary rows alone.
//
// The label's column stays apart: loss = log1p(sum over the others of exp(l -
// l_label)), which keeps its digits where the label dominates (lse - l_label
// would leave 1e-6 of a logit of 14, whatever the loss), and its term of dH,
// (p_label - 1) W[label], is added after the last piece in fp32: rounding p to
// bf16 first would lose the gradient of a well-predicted token.
//
// A row's coefficients sum to zero, and so have the rounded ones to: what all of
// W's rows share (a head's rows have a mean) cancels in dH, and would come
// through with what the roundings leave, up to 2^-8 of the large ones (512 x 8000
// x 512, a label and a rival of like size, relative error of dH with a mean of 0,
// 3, 10 and 30 times the rows' own part: 0.20, 0.40, 1.2 and 3.4%; as it is 0.23%
// throughout).  The label's coefficient therefore takes the others' roundings up: in the step it is minus the sum of the
// others as rounded, in the backward (whose lse is the caller's, so that the
// others need not sum to 1 - p_label) expm1(l_label - lse) less the sum of the
// roundings.
#include <algorithm>

#include "train.h"

namespace qnf4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// The backward's sums of roundings are integers in units of 2^-40, added by
// atomics: in any order the same.  (A half tile's is below 2^-8; of something
// that is no probability, 1 and more, nothing is added.)
constexpr float kRoundingUnit = 1.0f / static_cast<float>(int64_t(1) << 40);
constexpr float kRefRange = 40.0f;  // tile maxima within +-kRefRange share the reference 0

// PAIR: tiles of 256 tokens on CTA pairs; otherwise of 128 on single CTAs.
// NF4 (single CTAs only): W's tile is dequantised into the ring from its codes.
template <int MODE, bool PAIR, bool NF4>
struct HeadPlan {
  static_assert(!(PAIR && NF4), "no such kernel");
  static constexpr bool kGrad = MODE == kHeadGrad;
  // columns of a tile at most: an NF4 kernel's extra warps leave the epilogue
  // registers for 64 sums a thread
  static constexpr int kMaxTw = NF4 && !kGrad ? 128 : 256;
  static constexpr int kCols = kMaxTw / 2;                       // an epilogue thread's
  static constexpr int kBRows = PAIR ? kMaxTw / 2 : kMaxTw;      // columns of the tile in this CTA's ring
  static constexpr uint32_t kA = 16384;                          // 128 tokens x 64
  static constexpr uint32_t kB = kBRows * 128;
  static constexpr uint32_t kC = NF4 ? kBRows * 32 : 0;          // packed codes of the same
  static constexpr uint32_t kStage = kA + kB + kC;
  // Warp 0: copies; warp 1: MMAs; then eight epilogue warps (two per quarter of
  // the rows, each with half of the columns); NF4: eight that dequantise.
  // Prob: two more, for the labels' logits.
  static constexpr int kLabelWarp = 2 + 8 + (NF4 ? 8 : 0);
  static constexpr int kLabelWarps = MODE == kHeadProb ? 2 : 0;
  static constexpr int kThreads = 32 * (kLabelWarp + kLabelWarps);
  // The dequantisers as groups that take the stages in turn, a 64-weight block
  // a thread; the ring is a multiple of the groups, so a slot's earlier stages
  // are the same group's and its parity waits cannot run a phase ahead.
  static constexpr int kGroups = NF4 ? 256 / kBRows : 1;
  static constexpr int kArrive = 8 / kGroups;                    // their arrivals on a stage
  static constexpr uint32_t kStages = (232448 - 2048) / kStage / (NF4 ? kGroups : 2) * (NF4 ? kGroups : 2);
  static constexpr uint32_t kBarOff = kStages * kStage;
  static constexpr uint32_t kSmem = 1024 + kBarOff + 512;
  static_assert(kSmem <= 232448u && kStages >= 4, "the ring does not fit");
};

constexpr int kEpiWarps = 8;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tile order: groups of token tiles, tokens first within a group, so the pairs
// at work share a few panels of each operand in L2.  Groups of 16 for logits
// (8192 x 32000 x 4096, forward: 1584-1621 us, of 8 1635-1650, of 32 1800), of
// 8 for dH, whose token panels are a piece wide.
template <bool GRAD>
__device__ __forceinline__ void head_tile(int tile, int mtiles, int ntiles, int& m, int& n) {
  constexpr int kGroup = GRAD ? 8 : 16;
  const int per = kGroup * ntiles;
  const int grp = tile / per, rem = tile - grp * per;
  const int gsz = min(kGroup, mtiles - grp * kGroup);
  n = rem / gsz;
  m = grp * kGroup + rem - n * gsz;
}

__device__ __forceinline__ bool counts(int64_t label, int64_t ignore, int64_t vocab) {
  return label != ignore && label >= 0 && label < vocab;
}

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Adds this thread's columns (a multiple of 16) of a finished accumulator to
// its registers (16 at a time: 128 sums leave few registers beside them).
template <int N>
__device__ __forceinline__ void add_chunk(uint32_t taddr, bool first, int cols, float (&l)[N]) {
#pragma unroll
  for (int cb = 0; cb < N / 16; ++cb) {
    if (cb * 16 >= cols) break;
    uint32_t v[16];
    tmem_ld_32x32b_x16(taddr + cb * 16, v);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = __uint_as_float(v[j]);
      l[cb * 16 + j] = first ? x : __fadd_rn(l[cb * 16 + j], x);
    }
  }
}

template <int N>
__device__ __forceinline__ float max_all(const float (&l)[N]) {
  float m[4] = {l[0], l[1], l[2], l[3]};
#pragma unroll
  for (int j = 4; j < N; ++j) m[j & 3] = fmaxf(m[j & 3], l[j]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 32 bf16 (64 bytes, 16-byte aligned) from fp32; `n` valid (a multiple of 8).
__device__ __forceinline__ void store_bf16x32(uint16_t* dst, const float (&v)[32], int n) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (8 * j < n)
      reinterpret_cast<uint4*>(dst)[j] =
          make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                     pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
}

// Two fp32 sums in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 c;
  asm("{.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(c.x), "=f"(c.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return c;
}

// `cols` bf16 (a multiple of 16; 32-byte aligned) from fp32, whole sectors a
// store; returns the sum of the rounded values (RESIDUE: less the values').
template <bool RESIDUE, int N>
__device__ __forceinline__ float store_bf16(uint16_t* dst, int cols, const float (&v)[N]) {
  float2 d[2] = {};
#pragma unroll
  for (int j = 0; j < N; j += 16) {
    if (j >= cols) break;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = pack_bf16x2(v[j + 2 * i], v[j + 2 * i + 1]);
      float2 r = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      if (RESIDUE) r = add2(r, make_float2(-v[j + 2 * i], -v[j + 2 * i + 1]));
      d[i & 1] = add2(d[i & 1], r);
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + j), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
  return (d[0].x + d[0].y) + (d[1].x + d[1].y);
}

// fp32 sums between pieces and of parts of a contraction: per tile or part and
// CTA, the epilogue threads' registers as 32 rows of 256 float4, so that every
// access of a warp is 512 contiguous bytes.
constexpr int kSumCols = kHeadTile / 2;                 // a thread's columns
constexpr int kSumStride = 32 * kEpiWarps;              // float4 per row
constexpr int kSumBlock = kSumCols / 4 * kSumStride;    // float4 per CTA of a tile

// Rows of a product's token-side operand.
__device__ __forceinline__ int operand_rows(const HeadArgs& a) { return a.nrows ? __ldcg(a.nrows) : a.T; }

// A worker's tiles, or parts of tiles, of a product in turn: for logits every
// workers-th tile, for dH as head_tail says (train.h).
template <bool GRAD>
struct HeadItems {
  int kst, workers, i, end;           // whole tiles in turn
  int j = 0, j_end = 0, part = 0;     // then tiles in parts, counted from `end`
  int t0 = 0, t1 = 0;                 //   and the part's stages
  int base = 0, parts = 1;
  int tile, k0, kn;  // the item: its tile, first stage, and stages (none: a short piece ends before)
  int slot;          // Grad: of its sums
  bool whole;        // the tile is not in parts

  __device__ __forceinline__ HeadItems(const HeadArgs& a, int mn, int worker, int workers_)
      : kst(a.kst), workers(workers_), i(worker), end(mn) {
    if (!GRAD) return;
    const HeadTail t = head_tail(mn, a.kfull, workers);
    end = t.full * workers;
    base = a.first && a.last ? 0 : end;  // (whole tiles of an only piece need no sums)
    parts = t.parts;
    if (t.help && worker >= t.rest) {
      part = 1;
      j = (worker - t.rest) * t.help;
      j_end = min(j + t.help, t.rest);
      t0 = t.per;
      t1 = a.kfull;
    } else if (worker < t.rest * parts) {
      part = worker / t.rest;
      j = worker - part * t.rest;
      j_end = j + 1;
      t0 = part * t.per;
      t1 = min(t0 + t.per, a.kfull);
    }
  }
  __device__ __forceinline__ bool next() {
    if (i < end) {
      tile = slot = i;
      i += workers;
      k0 = 0;
      kn = kst;
      whole = true;
      return true;
    }
    if (!GRAD || j >= j_end) return false;
    tile = end + j;
    k0 = t0;
    kn = min(kst, t1) - t0;
    whole = parts == 1;
    slot = base + j * parts + part;
    ++j;
    return true;
  }
};

// dH_t = cs * cn * (the row's sum over the vocabulary but the label + cl *
// W[label]).  Step: cn is the root of the sum's normalisation (head_combine_kernel).
__device__ __forceinline__ void grad_row_factors(const HeadArgs& a, int t, float& cn, float& cs, float& cl) {
  cl = __ldcg(a.coef + t);
  if (a.row_root) {
    const float g = a.weight ? a.scale * __ldcg(a.weight + t) : a.scale / static_cast<float>(__ldcg(a.count));
    cn = __ldcg(a.row_root + t);
    cs = g * cn;
  } else {
    cs = a.stats ? __ldcg(a.dloss) / __ldcg(a.stats + 1) : __ldcg(a.dloss + t);
    cn = 1.0f;
    cl -= static_cast<float>(static_cast<long long>(__ldcg(a.rounding + t))) * kRoundingUnit;
  }
}

// Columns d .. d + 31 of row `row` of the head as fp32 (`n` valid, a multiple of 8).
__device__ __forceinline__ void load_head_row(const qlora_head& h, const Nf4Tables& tab, int64_t row, int d, int n,
                                              float (&w)[32]) {
  uint4 v[4];
  if (h.w) {
    const uint4* src = reinterpret_cast<const uint4*>(h.w + row * h.ld + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 8 * j < n ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
  } else {  // half of a 64-element block
    const int64_t e = row * h.dim + d, b = e >> 6;
    const float chat = nf4_block_scale(__ldg(h.c8 + b), __ldg(h.s2 + (b >> 8)), nf4_load_mean(h.mean));
    const Nf4Lut lut = nf4_make_lut(tab, chat);
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(h.codes + (e >> 1)));
    v[0] = nf4_lookup8(c.x, lut);
    v[1] = nf4_lookup8(c.y, lut);
    v[2] = nf4_lookup8(c.z, lut);
    v[3] = nf4_lookup8(c.w, lut);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[8 * j + 2 * i] = __uint_as_float(u[i] << 16);
      w[8 * j + 2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

// A lane's share of the logit of label `label` for the row h: columns 8 first ..
// and every 8 lanes-th run of 8 on.  fp32 sums rounded to nearest, four a lane
// (shorter chains, smaller errors).
__device__ __forceinline__ float label_dot(const qlora_head& head, const Nf4Tables& tab, const uint16_t* h,
                                           int64_t label, int first, int lanes) {
  float z[4] = {};
  const int dim = static_cast<int>(head.dim);
  auto add = [&z](const uint4& x, const uint4& y) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), z[i]);
      z[i] = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), z[i]);
    }
  };
  const int d0 = first * 8, step = lanes * 8;
  if (head.w) {
    const uint16_t* w = head.w + label * head.ld;
#pragma unroll 8
    for (int d = d0; d < dim; d += step)
      add(__ldcg(reinterpret_cast<const uint4*>(h + d)), __ldg(reinterpret_cast<const uint4*>(w + d)));
  } else {
    const Nf4Mean mean = nf4_load_mean(head.mean);
#pragma unroll 2
    for (int d = d0; d < dim; d += step) {
      const int64_t e = label * head.dim + d, b = e >> 6;
      const Nf4Lut lut = nf4_make_lut(tab, nf4_block_scale(__ldg(head.c8 + b), __ldg(head.s2 + (b >> 8)), mean));
      add(__ldcg(reinterpret_cast<const uint4*>(h + d)),
          nf4_lookup8(__ldg(reinterpret_cast<const uint32_t*>(head.codes + (e >> 1))), lut));
    }
  }
  return (z[0] + z[1]) + (z[2] + z[3]);
}

// Columns d .. d + 31 (`n` of them valid) of dH's row t from its sums l and the
// label's row of W.
__device__ __forceinline__ void store_grad32(const HeadArgs& a, int t, bool counted, float cn, float cs, float cl,
                                             int d, int n, const float (&w)[32], float (&l)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) l[j] = counted ? cs * (cn * fmaf(cl, w[j], l[j])) : 0.0f;
  store_bf16x32(a.dh + static_cast<int64_t>(t) * a.ldd + d, l, n);
}

// Place in a ring of N slots: the slot, and the parity of its round.  (Counted
// on: a division per stage would take the MMA warp a fifth of a stage's time.)
template <uint32_t N>
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void advance(uint32_t by = 1) {
    slot += by;
    if (slot >= N) {
      slot -= N;
      parity ^= 1;
    }
  }
};

}  // namespace

// A tile is 256 tokens (a CTA pair's; 128 of a single CTA) x tw columns: 256,
// or for products of few tiles the width that fills the last wave.  Per 64-deep
// stage each CTA holds its 128 token rows (A; rows without a token hold
// whatever the ring held: rows do not mix) and its columns (B: half of the
// tile's in a pair), one thread issues the MMAs (in a pair the leader's, M =
// 256), and each CTA's tensor memory gets its 128 rows.  Persistent: one pair
// per TPC, or one CTA per SM.
//
// The tensor core truncates when it adds to its fp32 accumulator: the sum
// drifts towards zero by about 2^-26 of itself per K = 16 step (measured:
// -8e-7 relative at dim 1024, -8e-6 at 8192, on random data).  A tile's
// contraction of a loss is therefore cut into chunks that alternate between two
// accumulators, and the epilogue threads add each finished one to their
// registers, rounding to nearest, while the next runs.  Pairs: 768 deep (48
// steps, a drift of 6e-7; 512 deep costs the products 2-3%, 1024 nothing).
// Single CTAs: 256 deep, which is free where the products wait for W (64 x 32000
// x 4096, forward: 56.5 us, with 768 56.4) and costs 3% above (300 x 32000 x 4096:
// 95.1 against 92.2; step 192 against 187), for losses 3e-7 instead of 8e-7
// off.  Results rounded to bf16 take longer ones: the backward's probabilities
// 1024, dH all of its tile's or part's contraction.
//
// Barriers (leader: the pair's first CTA, or the single one): full[s] (leader:
// the stage's copies landed, and its dequantised tiles are written), empty[s]
// (all: the stage's MMAs are done), cfull[s] (each: an NF4 stage's codes
// landed), accf[b] (all: the chunk's accumulator is final), acce[b] (leader: all
// epilogue warps have read it), done (leader: the last commit).  What an earlier
// kernel of the same call wrote is read past L1 (__ldcg): launches overlap, and
// nothing is kept there from one to the next.
template <int MODE, bool PAIR, bool NF4>
__global__ void __launch_bounds__(HeadPlan<MODE, PAIR, NF4>::kThreads, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ HeadArgs a) {
  using P = HeadPlan<MODE, PAIR, NF4>;
  constexpr bool kGrad = P::kGrad;
  constexpr uint32_t kCtas = PAIR ? 2 : 1;
  constexpr int kTokens = 128 * kCtas;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kBarOff);
  uint64_t* empty = full + P::kStages;
  uint64_t* accf = empty + P::kStages;
  uint64_t* acce = accf + 2;
  uint64_t* done = acce + 2;
  uint64_t* cfull = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cfull + P::kStages);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const int worker = blockIdx.x / kCtas, workers = kGrad ? a.workers : gridDim.x / kCtas;
  const int tw = kGrad ? kHeadTile : a.tw;  // columns of a tile

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < P::kStages; ++s) {
      mbar_init(&full[s], 1 + (NF4 ? P::kArrive : 0));
      mbar_init(&empty[s], 1);
      mbar_init(&cfull[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], kCtas * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncwarp();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  const WaitCtx wc{abort_flag, a.status};
  grid_dependency_wait();
  grid_dependents_launch();
  const int T = operand_rows(a);
  const int mtiles = (T + kTokens - 1) / kTokens;
  HeadItems<kGrad> it(a, mtiles * a.ntiles, worker, workers);
  if ((MODE == kHeadLoss || MODE == kHeadExp) && blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.zero_count; i += blockDim.x) a.zero[i] = 0u;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      Ring<P::kStages> at;
      uint32_t issued = 0;  // stages, up to a full ring
      bool ok = true;
      while (ok && it.next()) {
        int m, n;
        head_tile<kGrad>(it.tile, mtiles, a.ntiles, m, n);
        const int arow = m * kTokens + static_cast<int>(rank) * 128;
        const int bcol = n * tw + static_cast<int>(rank) * (tw / 2);
        const int k1 = it.k0 + it.kn;
        const bool mine = arow < T;  // else the CTA's rows hold no token: nothing to copy
        const uint32_t bytes = (PAIR && arow + 128 < T ? 2 : 1) * a.arows * 128u + (NF4 ? 0 : tw * 128u);
        for (int kt = it.k0; kt < k1; ++kt, at.advance()) {
          const uint32_t s = at.slot;
          if (issued == P::kStages && !mbar_wait(&empty[s], at.parity ^ 1, wc)) {
            ok = false;
            break;
          }
          issued = min(issued + 1, P::kStages);
          uint8_t* st = smem + s * P::kStage;
          const uint32_t full0 = PAIR ? dsmem_addr(&full[s], 0) : 0;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
            if constexpr (PAIR) tma_load_2d_pair(dst, map, full0, x, y);
            else tma_load_2d(dst, map, &full[s], x, y);
          };
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          if (mine) load(st, &tm_a, kt * 64, arow);
          if constexpr (NF4) {
            mbar_arrive_expect_tx(&cfull[s], kGrad ? P::kC : tw * 32u);
            uint8_t* codes = st + P::kA + P::kB;
            if constexpr (kGrad) tma_load_2d(codes, &tm_b, &cfull[s], bcol / 2, a.b_row0 + kt * 64);
            else tma_load_2d(codes, &tm_b, &cfull[s], kt * 32, a.b_row0 + bcol);
          } else {
            if constexpr (kGrad) {  // W's rows are the contraction: 64-column atoms
#pragma unroll
              for (int i = 0; i < P::kBRows / 64; ++i)
                load(st + P::kA + i * 8192, &tm_b, bcol + i * 64, a.b_row0 + kt * 64);
            } else {
              load(st + P::kA, &tm_b, kt * 64, a.b_row0 + bcol);
            }
          }
        }
      }
      // The full barriers of an NF4 ring also count the dequantisers'
      // arrivals, which may never come after an abort: a short limit then (the
      // copies land in microseconds).
      const uint64_t lim = *abort_flag ? 1000000ull : kWaitTimeoutNs;
      for (uint32_t s = 0; s < issued; ++s) {  // each slot's last copy
        const uint32_t parity = s < at.slot ? at.parity : at.parity ^ 1;
        if (NF4) mbar_drain(&cfull[s], parity, a.status, lim);
        if (rank == 0) mbar_drain(&full[s], parity, a.status, lim);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA (leader)
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(kTokens, tw, 0, kGrad ? 1 : 0);
      constexpr uint32_t b_step = kGrad ? (2048u >> 4) : (32u >> 4);
      auto commit = [&](uint64_t* bar) {
        if constexpr (PAIR) umma_commit_pair(bar, 0x3);
        else umma_commit(bar);
      };
      Ring<P::kStages> at;
      int acc = 0;  // chunks begun
      bool ok = true;
      while (ok && it.next()) {
        const int kn = it.kn;
        for (int k0 = 0; ok && k0 < kn; k0 += a.kchunk, ++acc) {
          const int buf = acc & 1;
          if (acc >= 2 && !mbar_wait_all(&acce[buf], ((acc >> 1) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_d + buf * 256;
          const int kc = min(a.kchunk, kn - k0);
          for (int kt = 0; kt < kc; ++kt, at.advance()) {
            const uint32_t s = at.slot;
            if (!mbar_wait_all(&full[s], at.parity, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + s * P::kStage);
            const uint64_t ad = sdesc_sw128(sa, 16, 1024);
            const uint64_t bd = kGrad ? sdesc_sw128(sa + P::kA, 8192, 1024) : sdesc_sw128(sa + P::kA, 16, 1024);
            if (elect_one()) {
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk) {
                const uint32_t more = (kt | static_cast<int>(kk)) != 0 ? 1u : 0u;
                if constexpr (PAIR) umma_bf16_pair(d, ad + kk * 2, bd + kk * b_step, idesc, more);
                else umma_bf16(d, ad + kk * 2, bd + kk * b_step, idesc, more);
              }
              commit(&empty[s]);
              if (kt == kc - 1) commit(&accf[buf]);
            }
            __syncwarp();
          }
        }
      }
      if (elect_one()) {  // nothing is in flight when the tensor memory is freed
        if constexpr (PAIR) umma_commit_pair(done, 0x1);
        else umma_commit(done);
        mbar_drain(done, 0, a.status);
      }
      __syncwarp();
    }
  } else if (MODE == kHeadProb && warp >= P::kLabelWarp) {
    // ------------------------------------------------------------- label's term
    // p_label - 1 = expm1(l_label - lse) of the tokens that count, with the
    // label's logit in fp32 rounded to nearest, as the losses and so lse have it
    // (head_combine_kernel); eight lanes a token.  Beside the products they
    // cost nothing; a launch of their own took 4-20 us.
    if (a.coef_out) {
      const int stride = 4 * P::kLabelWarps * gridDim.x;
      for (int r0 = 4 * (blockIdx.x * P::kLabelWarps + warp - P::kLabelWarp); r0 < T; r0 += stride) {
        const int row = r0 + (lane >> 3);
        float z = 0.0f;
        int t = 0;
        bool counted = false;
        if (row < T) {
          t = a.rows ? __ldcg(a.rows + row) : row;
          const int64_t label = __ldg(a.labels + t);
          counted = counts(label, a.ignore, a.vocab);
          if (counted) z = label_dot(a.head, a.tab, a.h + row * a.ldh, label, lane & 7, 8);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
        if (counted && (lane & 7) == 0) a.coef_out[t] = expm1f(z - __ldcg(a.lse + t));
      }
    }
  } else if (NF4 && warp >= 2 + kEpiWarps) {
    // ----------------------------------------------------------- dequantisers
    // A thread turns one 64-weight block a stage into a 128-byte row of the
    // tile.  Logits: the block of column bcol + i at depth 64 kt (a K-major
    // row).  Grad: columns 64 (i / 64) .. of W's row 64 kt + i % 64 (a row of an
    // MN-major atom).  The codes come with the stage (swizzled, so that the
    // lanes' 16-byte reads spread over the banks), the block constants from
    // global memory, kAhead of the thread's stages ahead.
    const int di = threadIdx.x - 64 - 32 * kEpiWarps;
    constexpr int kSize = 256 / P::kGroups;  // threads of a group
    const int grp = di / kSize, i = di % kSize;
    const int blocks = kGrad ? P::kBRows : tw;  // of a stage
    const int64_t kbpr = a.head.dim / 64;
    const Nf4Mean wmean = nf4_load_mean(a.head.mean);
    // this thread's codes in the stage: byte offset of its row, 16-byte chunk
    const uint32_t c_at = P::kB + (kGrad ? (i & 63) * 128 : i * 32);
    const uint32_t c_0 = (kGrad ? ((i >> 6) * 2) ^ (i & 7) : (i >> 2) & 1) << 4;
    const uint32_t d_0 = i * 128 + ((i & 7) << 4);  // its row of the tile (Grad: atom i / 64, row i % 64), swizzled
    const int64_t b_step = kGrad ? P::kGroups * 64 * kbpr : P::kGroups;
    constexpr int kAhead = 4;
    Ring<P::kStages> at;
    at.advance(grp);
    int begun = 0;  // stages of the tiles before, modulo the groups
    bool ok = true;
    while (ok && it.next()) {
      int m, n;
      head_tile<kGrad>(it.tile, mtiles, a.ntiles, m, n);
      const int kt0 = it.k0, kn = it.kn;
      if (kn <= 0) continue;
      const int g0 = (grp + P::kGroups - begun) % P::kGroups;         // the group's first stage of the tile
      const int count = (kn - g0 + P::kGroups - 1) / P::kGroups;      // and its number of them
      begun = (begun + kn) % P::kGroups;
      // the thread's block of its first stage, and how many stages have one
      const int row = kGrad ? (kt0 + g0) * 64 + (i & 63) : n * tw + i;  // of the piece
      const int64_t kb = kGrad ? n * tw / 64 + (i >> 6) : kt0 + g0;
      int64_t b = (a.v0 + row) * kbpr + kb;
      int left = i < blocks && row < a.wrows && kb < kbpr ? count : 0;
      if (kGrad) left = min(left, (a.wrows - row + 64 * P::kGroups - 1) / (64 * P::kGroups));
      uint32_t pk[kAhead];
      float ps[kAhead];
      auto fetch = [&](uint32_t& k8, float& s2) {
        k8 = 0x100;  // outside: zeros, whatever the codes
        s2 = 0.0f;
        if (left-- > 0) {
          k8 = __ldg(a.head.c8 + b);
          s2 = __ldg(a.head.s2 + (b >> 8));
          b += b_step;
        }
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(pk[j], ps[j]);
      // (Unrolled over the slots, so that each is refilled in place: moving a
      // register that a load is still filling waits for the load.)
      for (int k = 0; ok && k < count; k += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (k + j >= count) break;
          const uint32_t s = at.slot;
          const Nf4Lut lut =
              nf4_make_lut(a.tab, pk[j] == 0x100u ? 0.0f : nf4_block_scale(pk[j], ps[j], wmean));
          fetch(pk[j], ps[j]);
          if (!mbar_wait_all(&cfull[s], at.parity, wc)) {
            ok = false;
            break;
          }
          if (i < blocks) {
            uint8_t* st = smem + s * P::kStage + P::kA;
            const uint4 c0 = *reinterpret_cast<const uint4*>(st + c_at + c_0);
            const uint4 c1 = *reinterpret_cast<const uint4*>(st + c_at + (c_0 ^ 16));
            const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (uint32_t c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(st + (d_0 ^ (c << 4))) = nf4_lookup8(cw[c], lut);
          }
          fence_proxy_async_smem();  // this lane's row -> async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          at.advance(P::kGroups);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;             // TMEM lanes 32 q ..
    const int half = (warp - 2) >> 2;   // columns hw half ..
    const int hw = tw / 2;
    const int et = threadIdx.x - 64;
    const uint32_t tq = tmem_d + (static_cast<uint32_t>(q * 32) << 16) + half * hw;
    int acc = 0;
    auto release = [&](int buf) {  // this warp's reads of the accumulator are done
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_remote(dsmem_addr(&acce[buf], 0));
        else mbar_arrive(&acce[buf]);
      }
    };
    while (it.next()) {
      int m, n;
      head_tile<kGrad>(it.tile, mtiles, a.ntiles, m, n);
      const int kn = it.kn;
      const int row = m * kTokens + static_cast<int>(rank) * 128 + q * 32 + lane;  // of the operand
      const bool rok = row < T;
      const int n0 = n * tw + half * hw;
      const int nv = min(hw, a.ncols - n0);  // this thread's columns (may be none)
      int t = row;  // the token
      int64_t label = -1;
      bool counted = false;
      if (rok) {
        if (a.rows) t = __ldcg(a.rows + row);
        label = __ldg(a.labels + t);
        counted = counts(label, a.ignore, a.vocab);
      }
      // the label's place among this thread's columns, or none
      int64_t lc = counted ? label - a.v0 - n0 : -1;
      const int lj = lc >= 0 && lc < nv ? static_cast<int>(lc) : -1;

      if (MODE == kHeadGrad) {
        // one chunk per item (bf16 results), 32 columns at a time
        const int buf = acc & 1;
        if (kn > 0) {  // an empty part (of a short last piece) adds nothing
          if (!mbar_wait_warp(&accf[buf], (acc >> 1) & 1, wc)) break;
          tc_fence_after();
        }
        float4* sum =
            reinterpret_cast<float4*>(a.acc) + (static_cast<int64_t>(it.slot) * kCtas + rank) * kSumBlock + et;
        const float al = (!a.first && a.alpha && rok) ? __ldcg(a.alpha + t) : 1.0f;
        const bool out = a.last && it.whole;
        float cn = 0.0f, cs = 0.0f, cl = 0.0f;
        if (out && counted) grad_row_factors(a, t, cn, cs, cl);
        for (int cb = 0; cb < kSumCols / 32; ++cb) {
          float l[32] = {};
          if (kn > 0) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tq + buf * 256 + cb * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) l[j] = __uint_as_float(v[j]);
          }
          float4* at = sum + cb * 8 * kSumStride;
          if (!a.first) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 o = __ldcg(at + j * kSumStride);
              l[4 * j] = fmaf(al, o.x, l[4 * j]);
              l[4 * j + 1] = fmaf(al, o.y, l[4 * j + 1]);
              l[4 * j + 2] = fmaf(al, o.z, l[4 * j + 2]);
              l[4 * j + 3] = fmaf(al, o.w, l[4 * j + 3]);
            }
          }
          if (!out) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              __stcg(at + j * kSumStride, make_float4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]));
          } else if (rok && cb * 32 < nv) {
            const int d = n0 + cb * 32, nd = min(32, nv - cb * 32);
            float w[32] = {};
            if (counted) load_head_row(a.head, a.tab, label, d, nd, w);
            store_grad32(a, t, counted, cn, cs, cl, d, nd, w, l);
          }
        }
        if (kn > 0) {
          release(buf);
          ++acc;
        }
        continue;
      }

      constexpr int kCols = P::kCols;
      float l[kCols];
      bool ok = true;
      for (int k0 = 0; k0 < kn; k0 += a.kchunk, ++acc) {
        const int buf = acc & 1;
        if (!mbar_wait_warp(&accf[buf], (acc >> 1) & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        add_chunk(tq + buf * 256, k0 == 0, hw, l);
        release(buf);
      }
      if (!ok) break;

      if (nv < kCols) {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          if (j >= nv) l[j] = -INFINITY;
      }
      if (lj >= 0) {  // the label's column leaves the tile
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          if (j == lj) l[j] = -INFINITY;
      }
      if (MODE == kHeadLoss) {
        const float mx = max_all(l);
        const float base = mx == -INFINITY ? 0.0f : mx * kLog2e;
        float p[4] = {};
#pragma unroll
        for (int j = 0; j < kCols; ++j) p[j & 3] += exp2_fast(fmaf(l[j], kLog2e, -base));
        if (rok) a.part[static_cast<int64_t>(2 * n + half) * a.T + t] = make_float2(mx, (p[0] + p[1]) + (p[2] + p[3]));
      } else if (MODE == kHeadExp) {
        const float mx = max_all(l);
        const float ref = (fabsf(mx) <= kRefRange || mx == -INFINITY) ? 0.0f : mx;
        const float base = ref * kLog2e;
        float p[4] = {};
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          l[j] = exp2_fast(fmaf(l[j], kLog2e, -base));
          p[j & 3] += l[j];
        }
        if (rok) {
          a.part[static_cast<int64_t>(2 * n + half) * a.T + t] = make_float2(ref, (p[0] + p[1]) + (p[2] + p[3]));
          const int at = a.place ? __ldcg(a.place + t) : t;
          if (at >= 0)
            a.rsum[static_cast<int64_t>(2 * n + half) * a.T + t] =
                store_bf16<false>(a.g + static_cast<int64_t>(at) * a.ldg + n0, hw, l);
        }
      } else if (MODE == kHeadProb) {
        const float lse = rok ? __ldcg(a.lse + t) : 0.0f;
        const float base = lse * kLog2e;
#pragma unroll
        for (int j = 0; j < kCols; ++j) l[j] = counted ? exp2_fast(fmaf(l[j], kLog2e, -base)) : 0.0f;
        if (rok) {
          const float d = store_bf16<true>(a.g + static_cast<int64_t>(row) * a.ldg + n0, hw, l);
          if (counted && fabsf(d) < 1.0f)  // (no NaN either)
            atomicAdd(a.rounding + t, static_cast<unsigned long long>(__float2ll_rn(d / kRoundingUnit)));
          if (n0 == 0 && a.v0 == 0 && a.status) {
            if (!counted && label != a.ignore) atomicOr(a.status, QLORA_DEV_LABEL);
            if (counted && !isfinite(lse)) atomicOr(a.status, QLORA_DEV_NONFINITE);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_d, 512);
    else tmem_dealloc(tmem_d, 512);
  }
}

// ------------------------------------------------------------- rows that count
//
// An ignored token has no gradient: its row is left out of the products that
// make dH (a fine-tuning batch ignores its prompts).  One launch lists the
// tokens that count in order (rows[i] the i-th, place[t] its i or -1, their
// number kept on the device) and, for the backward, copies their rows of H
// together.  A block takes `chunk` tokens and counts the ones before them
// itself (8192 labels are 64 KB from L2).  8192 tokens of width 1024: 18 us, 31
// with the scan in a launch of its own, one block; 1000 tokens: 13 either way,
// most of it start and end.

constexpr int kRowsThreads = 512;

__global__ void __launch_bounds__(kRowsThreads) head_rows_kernel(const __grid_constant__ HeadRowsArgs a) {
  __shared__ int warp_sum[kRowsThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t T = a.T, begin = static_cast<int64_t>(blockIdx.x) * a.chunk, end = min(begin + a.chunk, T);
  int n = 0;
  for (int64_t t0 = threadIdx.x; t0 < begin; t0 += 8 * kRowsThreads) {
    int64_t label[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = t0 + i * kRowsThreads;
      label[i] = t < begin ? __ldg(a.labels + t) : a.ignore;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) n += counts(label[i], a.ignore, a.vocab) ? 1 : 0;
  }
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if (lane == 0) warp_sum[warp] = n;
  __syncthreads();
  int at = 0;  // tokens that count before the chunk
  for (int w = 0; w < kRowsThreads / 32; ++w) at += warp_sum[w];

  // (every warp walks the chunk alike; `each` warps copy a row)
  const int each = a.chunk >= kRowsThreads / 32 ? 1 : kRowsThreads / 32 / static_cast<int>(a.chunk);
  const int sub = warp % each * 32 + lane, step = each * 32;
  for (int64_t t0 = begin; t0 < end; t0 += 32) {
    const int64_t label = t0 + lane < end ? __ldg(a.labels + t0 + lane) : a.ignore;
    const bool in = counts(label, a.ignore, a.vocab);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
    if (warp == 0 && t0 + lane < end) {
      const int mine = at + __popc(mask & ((1u << lane) - 1));
      a.place[t0 + lane] = in ? mine : -1;
      if (a.rounding) a.rounding[t0 + lane] = 0;
      if (in) a.rows[mine] = static_cast<int32_t>(t0 + lane);
      if (!in && label != a.ignore && a.status) atomicOr(a.status, QLORA_DEV_LABEL);
    }
    if (a.out) {
      for (int i = warp / each; i < 32 && t0 + i < end; i += kRowsThreads / 32 / each) {
        const bool one = mask >> i & 1;
        const int64_t t = t0 + i;
        const uint4* src = reinterpret_cast<const uint4*>(a.h + t * a.ldh);
        uint4* dst = reinterpret_cast<uint4*>(
            one ? a.out + (at + __popc(mask & ((1u << i) - 1))) * a.dim : a.dh + t * a.ldd);
        for (int64_t j0 = sub; j0 < a.dim / 8; j0 += 4 * step) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = one && j0 + k * step < a.dim / 8 ? src[j0 + k * step] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (j0 + k * step < a.dim / 8) dst[j0 + k * step] = v[k];
        }
      }
    }
    at += __popc(mask);
  }
  if (end == T && threadIdx.x == 0) *a.nrows = at;
}

// The backward's sums of roundings, cleared where the rows are not listed.
__global__ void __launch_bounds__(kRowsThreads) head_clear_kernel(unsigned long long* rounding, int64_t T) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsThreads + threadIdx.x;
  if (t < T) rounding[t] = 0;
}

// ------------------------------------------------------------------- finish
//
// The parts of a tile joined in order, and dH's rows from them.  blockIdx.x:
// (tile of those that fill no wave, CTA of it); blockIdx.y: 32 of a thread's 128
// columns.
__global__ void __launch_bounds__(kSumStride) head_finish_kernel(const __grid_constant__ HeadArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int ctas = a.pair ? 2 : 1;
  const int T = operand_rows(a);
  const int mtiles = (T + 128 * ctas - 1) / (128 * ctas);
  const HeadTail tail = head_tail(mtiles * a.ntiles, a.kfull, a.workers);
  const int j = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  if (j >= tail.rest || tail.parts == 1) return;
  const int tile = tail.full * a.workers + j;
  const int slot = (a.first && a.last ? 0 : tail.full * a.workers) + j * tail.parts;
  int m, n;
  head_tile<true>(tile, mtiles, a.ntiles, m, n);
  const int et = threadIdx.x, w = et >> 5, lane = et & 31;
  const int row = (m * ctas + rank) * 128 + ((w + 2) & 3) * 32 + lane;  // as in the product's epilogue
  const int d = n * kHeadTile + (w >> 2) * kSumCols + blockIdx.y * 32;
  if (row >= T || d >= a.ncols) return;
  const int t = a.rows ? __ldcg(a.rows + row) : row;
  const int at_row = static_cast<int>(blockIdx.y) * 8 * kSumStride + et;
  // the first part's sums on their way beside the chain of token, label and its row of W
  const float4* part0 = reinterpret_cast<const float4*>(a.acc) +
                        (static_cast<int64_t>(slot) * ctas + rank) * kSumBlock + at_row;
  float4 o0[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o0[j] = __ldcg(part0 + j * kSumStride);
  const int64_t label = __ldg(a.labels + t);
  const bool counted = counts(label, a.ignore, a.vocab);
  const int nd = min(32, a.ncols - d);
  float cn = 0.0f, cs = 0.0f, cl = 0.0f;
  float l[32] = {}, wr[32] = {};
  if (counted) {
    load_head_row(a.head, a.tab, label, d, nd, wr);
    grad_row_factors(a, t, cn, cs, cl);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    l[4 * j] = o0[j].x;
    l[4 * j + 1] = o0[j].y;
    l[4 * j + 2] = o0[j].z;
    l[4 * j + 3] = o0[j].w;
  }
  for (int part = 1; part < tail.parts; ++part) {
    const float4* at = reinterpret_cast<const float4*>(a.acc) +
                       (static_cast<int64_t>(slot + part) * ctas + rank) * kSumBlock + at_row;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 o = __ldcg(at + j * kSumStride);
      l[4 * j] += o.x;
      l[4 * j + 1] += o.y;
      l[4 * j + 2] += o.z;
      l[4 * j + 3] += o.w;
    }
  }
  store_grad32(a, t, counted, cn, cs, cl, d, nd, wr, l);
}

// ------------------------------------------------------------------ combine
//
// Joins the (reference, sum) pairs of a row's parts (half tiles): R = max ref,
// S = sum of s exp(ref - R), of all columns but the label's.  Step: R, S and the
// sum of the exponentials as rounded run over the pieces, exponentials of parts whose
// reference is not R are rescaled in place (rows with logits beyond +-40 only),
// and alpha = exp(R_old - R).  With the last piece: lse, loss, and
// the mean in fp64 (per-block sums, added in block order by the block that
// finishes last).  The label's logit is made here, in fp32 rounded to nearest:
// the tensor core's drift grows with a logit, and the label's is the one that
// stands out (with the tiles' own, losses of some tenths were 2-5e-6 off at dim
// 640 to 4096; so, below 1e-6).  Made in the tiles it took the products 5-10%
// (a wait for two rows in the epilogue, while the next chunk is due).  It reads
// nothing of the kernel before, and runs while that ends.
// A block takes TB tokens; its threads split their parts.  TB
// is 32 (whole sectors of a part's row) or, for few tokens, where the chain of
// loads is what takes the time, fewer, so that a thread has a few parts only.

namespace {

constexpr int kCombineWarps = 16;

// Reference, sum of exponentials, and their sum as rounded to bf16.
struct Part {
  float ref, sum, rsum;
};

template <bool STEP>
__device__ __forceinline__ void join(Part& a, const Part& b) {
  if (b.sum == 0.0f) return;          // (a NaN is not equal and joins)
  if (!STEP || a.ref != b.ref) {      // (the step's ordinary rows: all 0)
    const float top = fmaxf(a.ref, b.ref);
    // a.ref = -inf (nothing yet): the factor is 0
    const float fa = a.ref == top ? 1.0f : expf(a.ref - top), fb = b.ref == top ? 1.0f : expf(b.ref - top);
    a.sum = a.sum * fa + b.sum * fb;
    if (STEP) a.rsum = a.rsum * fa + b.rsum * fb;
    a.ref = top;
  } else {
    a.sum += b.sum;
    a.rsum += b.rsum;
  }
}

__device__ __forceinline__ void store_mean(const HeadCombineArgs& a, double sum, int count) {
  a.stats[0] = count > 0 ? static_cast<float>(sum / count) : 0.0f;
  a.stats[1] = static_cast<float>(count);
}

}  // namespace

template <int TB, bool STEP>
__global__ void __launch_bounds__(kCombineWarps * 32) head_combine_kernel(const HeadCombineArgs a) {
  __shared__ float2 sm[kCombineWarps][TB];
  __shared__ float sm_rsum[STEP ? kCombineWarps : 1][TB];
  __shared__ float again[STEP ? kCombineWarps : 1][TB];  // what a second rounding added
  __shared__ float ref_s[TB];
  __shared__ bool last_block;
  __shared__ double sums[kCombineWarps];
  constexpr int kSlices = kCombineWarps * 32 / TB;
  constexpr int kDotParts = TB < kCombineWarps ? kCombineWarps / TB : 1;  // warps on a token's label
  __shared__ float dot[TB][kDotParts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.last) {
    for (int i = warp / kDotParts; i < TB && blockIdx.x * TB + i < a.T; i += kCombineWarps / kDotParts) {
      const int64_t row = blockIdx.x * TB + i, label = a.labels[row];
      float z = 0.0f;
      if (counts(label, a.ignore, a.vocab))
        z = label_dot(a.head, a.tab, a.h + row * a.ldh, label, warp % kDotParts * 32 + lane, kDotParts * 32);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
      if (lane == 0) dot[i][warp % kDotParts] = z;
    }
  }
  grid_dependency_wait();
  grid_dependents_launch();
  const int tok = threadIdx.x % TB, slice = threadIdx.x / TB;
  const int t0 = blockIdx.x * TB, t = t0 + tok;
  const bool rok = t < a.T;

  Part all{-INFINITY, 0.0f, 0.0f};
  float lo = INFINITY;  // smallest reference of a part with a sum
  if (rok) {
    for (int j0 = slice; j0 < a.nparts; j0 += 8 * kSlices) {
      float2 p[8];
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i * kSlices;
        const int64_t at = static_cast<int64_t>(j) * a.T + t;
        p[i] = j < a.nparts ? __ldcg(a.part + at) : make_float2(0.0f, 0.0f);
        d[i] = STEP && j < a.nparts ? __ldcg(a.rsum + at) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        join<STEP>(all, {p[i].x, p[i].y, d[i]});
        if (p[i].y != 0.0f) lo = fminf(lo, p[i].x);
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= TB; o >>= 1) {  // lanes of the same token
    const Part other{__shfl_xor_sync(0xFFFFFFFFu, all.ref, o), __shfl_xor_sync(0xFFFFFFFFu, all.sum, o),
                     STEP ? __shfl_xor_sync(0xFFFFFFFFu, all.rsum, o) : 0.0f};
    // the lower lane's value first, so that both get the same bits
    Part both = (lane & o) ? other : all;
    join<STEP>(both, (lane & o) ? all : other);
    all = both;
  }
  if (lane < TB) {
    sm[warp][lane] = make_float2(all.ref, all.sum);
    if (STEP) {
      sm_rsum[warp][lane] = all.rsum;
      again[warp][lane] = 0.0f;
    }
  }
  __syncthreads();
  if (warp == 0) {
    bool counted = false;
    double sum = 0.0;
    if (lane < TB) {
      for (int w = 1; w < kCombineWarps; ++w) {
        const float2 v = sm[w][lane];
        join<STEP>(all, {v.x, v.y, STEP ? sm_rsum[w][lane] : 0.0f});
      }
      if (STEP && rok && !a.first) {
        const float2 old = __ldcg(a.run + t);
        join<STEP>(all, {old.x, old.y, __ldcg(a.run_rsum + t)});
        a.alpha[t] = (old.y == 0.0f || old.x == all.ref) ? 1.0f : expf(old.x - all.ref);
      }
      ref_s[lane] = all.ref;
      if (a.last && rok) {
        const int64_t label = a.labels[t];
        counted = counts(label, a.ignore, a.vocab);
        const float R = all.ref, S = all.sum;
        float lse = R + logf(S), loss = 0.0f;
        if (counted) {
          float z = dot[lane][0];
          for (int i = 1; i < kDotParts; ++i) z += dot[lane][i];
          const float top = fmaxf(R, z);
          // exp(l - l_label) over the others; where that is near overflow, its log is log S + R - l_label.
          // The reference may lie far below the others' maximum (0 for 40), so S exp(R - z) can be large
          // where exp(R - z) is not a number of fp32: the exponential in two halves.
          // (A label logit that overflowed: no number, as lse.)
          const float e = z == INFINITY ? NAN : expf(0.5f * (R - z));
          const float x = (S * e) * e;
          loss = x >= 1e30f ? (R - z) + logf(S) : log1pf(x);
          lse = top + logf(S * expf(R - top) + expf(z - top));  // (no others: R = -inf, S = 0)
          // and the root of 1 / (S + exp(z - R)), which overflows no earlier than it should
          if (STEP) a.row_root[t] = z > R ? e * rsqrtf(1.0f + x) : rsqrtf(S + expf(z - R));
        }
        a.lse[t] = lse;
        a.loss[t] = loss;
        sum = loss;
        if (a.status) {
          if (counted && !isfinite(lse)) atomicOr(a.status, QLORA_DEV_NONFINITE);
          if (!counted && label != a.ignore) atomicOr(a.status, QLORA_DEV_LABEL);
        }
      }
    }
    if (a.last) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      const uint32_t votes = __ballot_sync(0xFFFFFFFFu, counted);
      if (lane == 0) {
        const int count = __popc(votes);
        last_block = false;
        if (gridDim.x == 1) {
          a.counters[0] = count;
          store_mean(a, sum, count);
        } else {
          a.block_sum[blockIdx.x] = sum;
          atomicAdd(&a.counters[0], count);
          __threadfence();
          last_block = atomicAdd(&a.counters[1], 1) == static_cast<int>(gridDim.x) - 1;
        }
      }
    }
  }
  __syncthreads();
  if constexpr (STEP) {
    const float ref = ref_s[tok];
    // (no part of this thread: lo = inf)
    const bool rescale = __syncthreads_or(rok && lo < ref);
    if (rescale) {
      for (int j = slice; j - slice < a.nparts; j += kSlices) {
        const float2 p = rok && j < a.nparts ? __ldcg(a.part + static_cast<int64_t>(j) * a.T + t)
                                             : make_float2(0.0f, 0.0f);
        uint32_t todo = __ballot_sync(0xFFFFFFFFu, p.y != 0.0f && p.x != ref);
        const float f = expf(p.x - ref);
        while (todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          const float fr = __shfl_sync(0xFFFFFFFFu, f, src);
          const int js = __shfl_sync(0xFFFFFFFFu, j, src), ts = __shfl_sync(0xFFFFFFFFu, t, src);
          const int row = a.place ? __ldcg(a.place + ts) : ts;
          if (row < 0) continue;
          float d = 0.0f;
          if (4 * lane < a.part_cols) {
            uint2* at = reinterpret_cast<uint2*>(a.e + static_cast<int64_t>(row) * a.lde +
                                                 static_cast<int64_t>(js) * a.part_cols) + lane;
            const uint2 v = __ldcg(at);
            const float x[4] = {__uint_as_float(v.x << 16) * fr, __uint_as_float(v.x & 0xFFFF0000u) * fr,
                                __uint_as_float(v.y << 16) * fr, __uint_as_float(v.y & 0xFFFF0000u) * fr};
            const uint2 y = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            *at = y;
            d = ((__uint_as_float(y.x << 16) - x[0]) + (__uint_as_float(y.x & 0xFFFF0000u) - x[1])) +
                ((__uint_as_float(y.y << 16) - x[2]) + (__uint_as_float(y.y & 0xFFFF0000u) - x[3]));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
          if (lane == 0) again[warp][ts - t0] += d;
        }
      }
      __syncthreads();
    }
    if (warp == 0 && lane < TB && rok) {
#pragma unroll 1
      for (int w = 0; rescale && w < kCombineWarps; ++w) all.rsum += again[w][lane];
      a.run[t] = make_float2(all.ref, all.sum);
      a.run_rsum[t] = all.rsum;
      if (a.last) a.coef[t] = -all.rsum;
    }
  }
  if (a.last && a.place) {  // rows of dH that no product writes
    for (int i = 0; i < TB && t0 + i < a.T; ++i) {
      if (__ldcg(a.place + t0 + i) >= 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(a.dh + static_cast<int64_t>(t0 + i) * a.ldd);
      for (int64_t j = threadIdx.x; j < a.dim / 8; j += kCombineWarps * 32) dst[j] = make_uint4(0, 0, 0, 0);
    }
  }
  if (a.last && last_block) {
    __threadfence();
    double sum = 0.0;
    for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += kCombineWarps * 32) sum += __ldcg(a.block_sum + b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kCombineWarps; ++w) sum += sums[w];
      store_mean(a, sum, __ldcg(a.counters));
    }
  }
}

template <int MODE, bool PAIR, bool NF4>
static cudaError_t launch_head_gemm_impl(const CUtensorMap& tm_a, const CUtensorMap& tm_b, const HeadArgs& a,
                                         cudaStream_t stream) {
  using P = HeadPlan<MODE, PAIR, NF4>;
  static uint64_t done = 0;
  if (cudaError_t e = allow_smem(head_gemm_kernel<MODE, PAIR, NF4>, P::kSmem, done)) return e;
  const int tiles = a.mtiles * a.ntiles;
  int workers = std::min(tiles, head_workers(PAIR));
  if (MODE == kHeadGrad) {
    const HeadTail t = head_tail(tiles, a.kfull, a.workers);
    workers = t.full > 0 || t.help || a.nrows ? a.workers : t.rest * t.parts;
  }
  return launch_kernel(head_gemm_kernel<MODE, PAIR, NF4>, dim3((PAIR ? 2 : 1) * workers), dim3(P::kThreads), P::kSmem,
                       stream, dim3(PAIR ? 2 : 1, 1, 1), tm_a, tm_b, a);
}

template <int MODE>
static cudaError_t launch_head_gemm_mode(const CUtensorMap& tm_a, const CUtensorMap& tm_b, const HeadArgs& a,
                                         cudaStream_t stream) {
  if (a.pair) return a.nf4 ? cudaErrorInvalidValue : launch_head_gemm_impl<MODE, true, false>(tm_a, tm_b, a, stream);
  return a.nf4 ? launch_head_gemm_impl<MODE, false, true>(tm_a, tm_b, a, stream)
               : launch_head_gemm_impl<MODE, false, false>(tm_a, tm_b, a, stream);
}

cudaError_t launch_head_gemm(int mode, const CUtensorMap& tm_a, const CUtensorMap& tm_b, const HeadArgs& a,
                             cudaStream_t stream) {
  switch (mode) {
    case kHeadLoss: return launch_head_gemm_mode<kHeadLoss>(tm_a, tm_b, a, stream);
    case kHeadProb: return launch_head_gemm_mode<kHeadProb>(tm_a, tm_b, a, stream);
    case kHeadExp: return launch_head_gemm_mode<kHeadExp>(tm_a, tm_b, a, stream);
    case kHeadGrad: return launch_head_gemm_mode<kHeadGrad>(tm_a, tm_b, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_head_finish(const HeadArgs& a, int tiles, cudaStream_t stream) {
  return launch_kernel(head_finish_kernel, dim3((a.pair ? 2 : 1) * tiles, kSumCols / 32), dim3(kSumStride), 0, stream,
                       dim3(1, 1, 1), a);
}

cudaError_t launch_head_clear(unsigned long long* rounding, int64_t T, cudaStream_t stream) {
  return launch_kernel(head_clear_kernel, dim3(static_cast<unsigned>((T + kRowsThreads - 1) / kRowsThreads)),
                       dim3(kRowsThreads), 0, stream, dim3(1, 1, 1), rounding, T);
}

cudaError_t launch_head_rows(HeadRowsArgs a, cudaStream_t stream) {
  a.chunk = (a.T + 591) / 592;  // four blocks an SM
  return launch_kernel(head_rows_kernel, dim3(static_cast<unsigned>((a.T + a.chunk - 1) / a.chunk)),
                       dim3(kRowsThreads), 0, stream, dim3(1, 1, 1), a);
}

// Tokens of a combine block: 32, or for few tokens 4 (then at most 512 blocks).
static int combine_tokens(int64_t T) { return T > 2048 ? 32 : 4; }

int head_combine_blocks(int64_t T) {
  const int tb = combine_tokens(T);
  return static_cast<int>((T + tb - 1) / tb);
}

cudaError_t launch_head_combine(const HeadCombineArgs& a, cudaStream_t stream) {
  const bool wide = combine_tokens(a.T) == 32;
  return launch_kernel(a.run ? (wide ? head_combine_kernel<32, true> : head_combine_kernel<4, true>)
                             : (wide ? head_combine_kernel<32, false> : head_combine_kernel<4, false>),
                       dim3(head_combine_blocks(a.T)), dim3(kCombineWarps * 32), 0, stream, dim3(1, 1, 1), a);
}

}  // namespace qnf4
