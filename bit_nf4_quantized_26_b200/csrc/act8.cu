// act8.cu — 8-bit checkpoints of a linear's input and the adapter gradient
// that reads them ("QLoRA" encyclopedia entry, tonho.wtf, section "como
// funciona": memory is what the method saves; the adapters' gradients are the
// only use of the saved input).
//
// Per row, blocks of 64 elements share one power of two: with a = max|x| and
// e the smallest integer such that a <= 448 2^e, code = E4M3(x 2^-e).  A power
// of two leaves E4M3's three mantissa bits where they are, so x' = e4m3(code)
// 2^e has four significant bits and is exact in bf16: the tensor core reads
// exactly the value the checkpoint stands for, and the scale costs one byte.
// From the bits of a bf16 a = 1.m 2^E: 448 = 1.75 2^8, so e = E - 8, plus 1
// when 1.m > 1.75 (m > 0x60 of seven bits).
#include <algorithm>

#include "train.h"

namespace qnf4 {

namespace {

constexpr int kActThreads = 256;
constexpr int kExpBias = 127;
constexpr int kExpMin = -118, kExpMax = 120;

// Two E4M3 codes (low 16 bits) -> two fp32 values, exact.
__device__ __forceinline__ void e4m3x2_to_float(uint32_t pair, float& lo, float& hi) {
  uint32_t h2;
  const uint16_t in = static_cast<uint16_t>(pair);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  lo = f.x;
  hi = f.y;
}

// Four codes (one word) times 2^e (`scale`) -> four bf16, exact.
__device__ __forceinline__ uint2 codes4_to_bf16(uint32_t w, float scale) {
  float a, b, c, d;
  e4m3x2_to_float(w & 0xFFFFu, a, b);
  e4m3x2_to_float(w >> 16, c, d);
  return make_uint2(pack_bf16x2(a * scale, b * scale), pack_bf16x2(c * scale, d * scale));
}

// Two fp32 -> two E4M3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}

__device__ __forceinline__ float exp_scale(uint32_t byte) { return __uint_as_float(byte << 23); }  // 2^(byte - 127)

// Element offset of 16-element unit u (four per block) in rows of stride ld.
__device__ __forceinline__ int64_t unit_offset(int64_t u, int64_t units_per_row, int64_t K, int64_t ld) {
  if (ld == K) return u * 16;
  const int64_t row = u / units_per_row;
  return row * ld + (u - row * units_per_row) * 16;
}

// 16 elements (32 bytes).  WIDE (rows 32-byte aligned): one access of a whole
// sector a thread; as two 16-byte ones a warp's access touches every sector
// half, and L2 sees each twice (dequantiser: 811 MB for 405 MB).
template <bool WIDE>
__device__ __forceinline__ void load16(const uint16_t* src, uint32_t (&w)[8]) {
  if (WIDE) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(src));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store16(uint16_t* dst, const uint32_t (&w)[8]) {
  if (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Four threads share a block (16 elements each, one 16-byte store of codes).
// 3 + 1/64 bytes per element: HBM-bound.
template <bool WIDE>
__global__ void __launch_bounds__(kActThreads) act8_quantize_kernel(const uint16_t* __restrict__ x, int64_t units,
                                                                    int64_t units_per_row, int64_t K, int64_t ldx,
                                                                    uint8_t* __restrict__ codes,
                                                                    uint8_t* __restrict__ exps,
                                                                    int32_t* __restrict__ status) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kActThreads + threadIdx.x;
  const bool in = u < units;  // units is a multiple of 4: a block's lanes agree
  uint32_t w[8] = {};
  if (in) load16<WIDE>(x + unit_offset(u, units_per_row, K, ldx), w);
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
  uint32_t a = max(m2 & 0xFFFFu, m2 >> 16);  // magnitudes order like their bits
  a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
  a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
  if (!in) return;
  int e = static_cast<int>(a >> 7) - 127 - 8 + ((a & 0x7Fu) > 0x60u ? 1 : 0);
  e = min(max(e, kExpMin), kExpMax);
  const float inv = __uint_as_float(static_cast<uint32_t>(kExpBias - e) << 23);  // 2^-e
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = w[2 * i], q = w[2 * i + 1];
    c[i] = float2_to_e4m3x2(__uint_as_float(p << 16) * inv, __uint_as_float(p & 0xFFFF0000u) * inv) |
           (float2_to_e4m3x2(__uint_as_float(q << 16) * inv, __uint_as_float(q & 0xFFFF0000u) * inv) << 16);
  }
  reinterpret_cast<uint4*>(codes)[u] = make_uint4(c[0], c[1], c[2], c[3]);
  if ((threadIdx.x & 3) == 0) {
    exps[u >> 2] = static_cast<uint8_t>(e + kExpBias);
    if (a >= 0x7F80u && status) atomicOr(status, QLORA_DEV_NONFINITE);
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(kActThreads) act8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ exps, int64_t units,
                                                                      int64_t units_per_row, int64_t K,
                                                                      uint16_t* __restrict__ x, int64_t ldx) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kActThreads + threadIdx.x;
  if (u >= units) return;
  const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes) + u);
  const float s = exp_scale(__ldg(exps + (u >> 2)));
  const uint2 a = codes4_to_bf16(c.x, s), b = codes4_to_bf16(c.y, s), d = codes4_to_bf16(c.z, s),
              f = codes4_to_bf16(c.w, s);
  const uint32_t w[8] = {a.x, a.y, b.x, b.y, d.x, d.y, f.x, f.y};
  store16<WIDE>(x + unit_offset(u, units_per_row, K, ldx), w);
}

// ------------------------------------------------------------ dA from codes
//
// dA[j, k] = sum_m dU[m, j] X'[m, k]: the GEMM of skinny.cu's mode DA (128 rows
// of dU's bf16 hi/lo columns, tiles of 128 input features, the tokens split
// over a cluster and summed in rank order through distributed shared memory),
// with the token-side operand turned from codes into bf16 on the way: copies
// bring 64 tokens x 128 codes (8 KB) beside dU's three parts (32 KB), and two
// groups of four warps taking alternate stages write them as the MN-major
// 128-byte-swizzled tile the tensor core reads.  A stage is a chain (copy,
// convert, multiply) and runs beside the dX GEMM on few SMs, so what counts is
// how many are in flight: four copies and four converted tiles, one CTA per SM.
// (Three and two with one group, two CTAs per SM, took 193 us for 16384 tokens
// of 4096 features on 64 CTAs.)  The rings are even, so a slot's earlier stages are
// the same group's and its parity waits cannot run a phase ahead.
// Summed as DU and DB are (skinny.cu): two accumulators of eight stages each
// in turn, joined in registers.
struct ActDaPlan {
  static constexpr uint32_t kA = 16384;    // dU hi/lo: 64 tokens x 128 columns; its third parts the same
  static constexpr uint32_t kRaw = 8192;   // codes: 64 tokens x 128 features
  static constexpr uint32_t kCopy = 2 * kA + kRaw;
  static constexpr uint32_t kCopies = 4;
  static constexpr uint32_t kB = 16384;    // converted: 64 tokens x 128 features
  static constexpr uint32_t kTiles = 4;
  static constexpr uint32_t kTileOff = kCopies * kCopy;
  static constexpr uint32_t kBarOff = kTileOff + kTiles * kB;
  static constexpr uint32_t kSmem = 1024 + kBarOff + 256;
  static constexpr int kSumStages = 8;
  static constexpr int kLd = 132;  // floats per row of the parked partial tile
  static_assert(kSmem <= 232448u, "too much shared memory");
  static_assert(kCopies % 2 == 0 && kTiles % 2 == 0, "two alternating groups need even rings");
  static_assert(64 * kLd * 4 <= kTileOff, "the partial tile lies in the copy ring");
};
constexpr int kActDaThreads = 320;  // copy warp, MMA warp, 2 x 4 converting warps

__global__ void __launch_bounds__(kActDaThreads, 1)
    act8_da_kernel(const __grid_constant__ CUtensorMap tm_du, const __grid_constant__ CUtensorMap tm_du3,
                   const __grid_constant__ CUtensorMap tm_x,
                   const uint8_t* __restrict__ exps, const SkinnyArgs a) {
  using P = ActDaPlan;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kBarOff);  // copies landed
  uint64_t* empty = full + P::kCopies;                              // copies read (by the MMAs)
  uint64_t* bfull = empty + P::kCopies;                             // tile converted
  uint64_t* bempty = bfull + P::kTiles;                             // tile read
  uint64_t* accf = bempty + P::kTiles;                              // accumulator final
  uint64_t* acce = accf + 2;                                        // accumulator read
  uint64_t* done = acce + 2;                                        // the last commit of an aborted CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.groups;
  const int row0 = static_cast<int>(blockIdx.x) / G * 128;  // first input feature
  const int g = static_cast<int>(blockIdx.x) % G;           // member, or rank chunk
  const int ucol = g * 2 * a.r;
  const int rw = a.chunks ? min(a.r, a.r_total - g * a.r) : a.r;
  const int st0 = static_cast<int>(blockIdx.y) * a.stages_per_split;
  const int T = min(a.stages_total, st0 + a.stages_per_split) - st0;  // <= 0: no MMA, the partial is zero
  const bool wide = 2 * rw > 64;                                      // columns of dU in one or two boxes

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < P::kCopies; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (uint32_t s = 0; s < P::kTiles; ++s) {
      mbar_init(&bfull[s], 4);
      mbar_init(&bempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 8);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_du);
    tma_prefetch_desc(&tm_du3);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  const WaitCtx wc{abort_flag, a.status};
  // The kernel launched just before this one (dB) writes nothing that is read
  // here, and it let this one launch after everything older (dU, the
  // checkpoint) had completed: dA runs beside dB, and passes the wait at its
  // end, before it lets the next kernel launch.

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int t = 0; t < T; ++t) {
        const uint32_t s = t % P::kCopies, u = t / P::kCopies;
        if (t >= static_cast<int>(P::kCopies) && !mbar_wait(&empty[s], (u - 1) & 1, wc)) break;
        uint8_t* st = smem + s * P::kCopy;
        const int m0 = (st0 + t) * 64;
        mbar_arrive_expect_tx(&full[s], (wide ? 32768u : 16384u) + P::kRaw);
        tma_load_2d(st + 2 * P::kA, &tm_x, &full[s], row0, m0);
        tma_load_2d(st, &tm_du, &full[s], ucol, m0);
        if (wide) tma_load_2d(st + 8192, &tm_du, &full[s], ucol + 64, m0);
        tma_load_2d(st + P::kA, &tm_du3, &full[s], ucol, m0);
        if (wide) tma_load_2d(st + P::kA + 8192, &tm_du3, &full[s], ucol + 64, m0);
        issued = t + 1;
      }
      for (int t = max(0, issued - static_cast<int>(P::kCopies)); t < issued; ++t)
        mbar_drain(&full[t % P::kCopies], (t / P::kCopies) & 1, a.status);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 1, 1);
    bool aborted = false;
    for (int t = 0; t < T; ++t) {
      const uint32_t s = t % P::kCopies, b = t % P::kTiles;
      const int ch = t / P::kSumStages, buf = ch & 1;
      if ((t % P::kSumStages == 0 && ch >= 2 && !mbar_wait_all(&acce[buf], ((ch >> 1) - 1) & 1, wc)) ||
          !mbar_wait_all(&full[s], (t / P::kCopies) & 1, wc) || !mbar_wait_all(&bfull[b], (t / P::kTiles) & 1, wc)) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const uint64_t ad = sdesc_sw128(smem_u32(smem + s * P::kCopy), 8192, 1024);
      const uint64_t bd = sdesc_sw128(smem_u32(smem + P::kTileOff + b * P::kB), 8192, 1024);
      const uint64_t ad3 = sdesc_sw128(smem_u32(smem + s * P::kCopy + P::kA), 8192, 1024);
      if (elect_one()) {
#pragma unroll
        for (uint32_t kk = 0; kk < 4; ++kk) {  // 16 tokens = 16 rows of 128 bytes
          const uint32_t more = (t % P::kSumStages | kk) != 0 ? 1u : 0u;
          umma_bf16(tmem_d + buf * 128, ad + kk * (2048u >> 4), bd + kk * (2048u >> 4), idesc, more);
          // third parts onto the second ones' rows (zero in the first ones')
          umma_bf16(tmem_d + buf * 128, ad3 + kk * (2048u >> 4), bd + kk * (2048u >> 4), idesc, 1u);
        }
        umma_commit(&empty[s]);
        umma_commit(&bempty[b]);
        if (t % P::kSumStages == P::kSumStages - 1 || t == T - 1) umma_commit(&accf[buf]);
      }
      __syncwarp();
    }
    if (aborted && elect_one()) {
      umma_commit(done);
      mbar_drain(done, 0, a.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ converting warps
    // Unit i of a stage: 16 codes of row i / 8, columns 16 (i % 8); a thread
    // takes rows dt/8, dt/8 + 16, .. of one column unit, all in one block.
    const int grp = (warp - 2) >> 2;  // stages t with t % 2 == grp
    const int dt = (threadIdx.x - 64) & 127;
    const int cu = dt & 7, r0 = dt >> 3;
    const int kb = (row0 >> 6) + (cu >> 2);  // block along K
    const int64_t kbpr = a.K / 64;
    const bool kok = kb < kbpr;
    const uint32_t c0 = (cu & 3) * 2, flip = cu >> 2;  // first of two 16-byte chunks; the order alternates
    uint32_t pe[4];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = static_cast<int64_t>(st0 + t) * 64 + r0 + 16 * i;
        pe[i] = (t < T && kok && m < a.M) ? __ldg(exps + m * kbpr + kb) : 0u;  // outside: codes are zero-filled
      }
    };
    // TMEM row c = 32 q + lane holds part (lane / 16) of j = 16 q + lane % 16
    // (the second with the third).  The groups join 64 columns each; lanes 0-15 keep the first 32 of them,
    // lanes 16-31 the rest.
    const int q = warp & 3;
    float sum[32] = {};
    auto add_chunk = [&](int ch) {
      const int buf = ch & 1;
      if (!mbar_wait_warp(&accf[buf], (ch >> 1) & 1, wc)) return false;
      tc_fence_after();
      const uint32_t tq = tmem_d + buf * 128 + (static_cast<uint32_t>(q * 32) << 16) + grp * 64;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tq + cb * 32, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = __uint_as_float(v[i]);
          const float both = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
          if ((lane >= 16) == (cb == 1)) sum[i] = __fadd_rn(sum[i], both);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[buf]);
      return true;
    };
    bool ok = true;
    fetch(grp);
    for (int t = grp; t < T; t += 2) {
      // one chunk in flight, one final or nearly: join it while the MMAs go on
      if (t % P::kSumStages == 2 + grp && t > P::kSumStages && !(ok = add_chunk(t / P::kSumStages - 1))) break;
      const uint32_t s = t % P::kCopies, b = t % P::kTiles;
      float sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = exp_scale(pe[i]);
      fetch(t + 2);
      if (!mbar_wait_all(&full[s], (t / P::kCopies) & 1, wc) ||
          (t >= static_cast<int>(P::kTiles) && !mbar_wait_all(&bempty[b], ((t / P::kTiles) - 1) & 1, wc))) {
        ok = false;
        break;
      }
      const uint8_t* raw = smem + s * P::kCopy + 2 * P::kA;
      uint8_t* tile = smem + P::kTileOff + b * P::kB + (cu >> 2) * 8192;  // 64-feature atom
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r0 + 16 * i;
        const uint4 c = *reinterpret_cast<const uint4*>(raw + row * 128 + cu * 16);
        const uint2 p = codes4_to_bf16(c.x, sc[i]), q2 = codes4_to_bf16(c.y, sc[i]), v = codes4_to_bf16(c.z, sc[i]),
                    w = codes4_to_bf16(c.w, sc[i]);
        const uint4 lo = make_uint4(p.x, p.y, q2.x, q2.y), hi = make_uint4(v.x, v.y, w.x, w.y);
        uint8_t* dst = tile + row * 128;
        const uint32_t sw = row & 7;
        *reinterpret_cast<uint4*>(dst + (((c0 + flip) ^ sw) << 4)) = flip ? hi : lo;
        *reinterpret_cast<uint4*>(dst + (((c0 + 1 - flip) ^ sw) << 4)) = flip ? lo : hi;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bfull[b]);
    }
    // -------------------------------------------------- sums -> partial tile
    if (ok && T > 0) {  // the chunks the loop did not reach: the last, and the one before a short last
      const int last = (T - 1) / P::kSumStages;
      const int first = last - ((last > 0 && (T - 1) % P::kSumStages < 2 + grp) ? 1 : 0);
      for (int ch = first; ok && ch <= last; ++ch) ok = add_chunk(ch);
    }
    if (ok) {  // the copy ring is idle: its last stage's MMAs are done
      float* part = reinterpret_cast<float*>(smem);
      const int j = 16 * q + (lane & 15);
      if (j < rw) {
        float* dst = part + j * P::kLd + grp * 64 + (lane >> 4) * 32;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(dst + i) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
      }
    }
  }

  // ---------------------------------------------- fixed-order sum (cluster)
  __syncwarp();
  cluster_sync_all();
  {
    const float* part = reinterpret_cast<const float*>(smem);
    const uint32_t S = gridDim.y, self = cluster_ctarank();
    const int rows_per = (rw + static_cast<int>(S) - 1) / static_cast<int>(S);
    const int j0 = static_cast<int>(blockIdx.y) * rows_per, j1 = min(rw, j0 + rows_per);
    for (int i = threadIdx.x; i < (j1 - j0) * 32; i += blockDim.x) {
      const int row = j0 + i / 32, col = (i % 32) * 4;
      const float* loc = part + row * P::kLd + col;
      // with S = 1 the cluster (of two tiles, or none) does not span the splits
      float4 acc = dsmem_ld_f4(dsmem_addr(loc, S == 1 ? self : 0));
      for (uint32_t z = 1; z < S; ++z) {
        const float4 v = dsmem_ld_f4(dsmem_addr(loc, z));
        acc.x = __fadd_rn(acc.x, v.x);
        acc.y = __fadd_rn(acc.y, v.y);
        acc.z = __fadd_rn(acc.z, v.z);
        acc.w = __fadd_rn(acc.w, v.w);
      }
      const int k = row0 + col;
      if (k < a.K) *reinterpret_cast<float4*>(a.out_f32 + static_cast<int64_t>(g * a.r + row) * a.K + k) = acc;
    }
  }
  __syncwarp();
  cluster_sync_all();  // peers may still be reading this CTA's partial tile

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_d, 256);
  }
  grid_dependency_wait();
  grid_dependents_launch();
}

}  // namespace

// Rows 32-byte aligned (a vector access must be; 16 is what callers promise).
static bool wide_rows(const void* x, int64_t ldx) { return reinterpret_cast<uintptr_t>(x) % 32 == 0 && ldx % 16 == 0; }

cudaError_t launch_act8_quantize(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, uint8_t* exps,
                                 int32_t* status, cudaStream_t stream) {
  const int64_t units = M * (K / 16);
  const int64_t ctas = (units + kActThreads - 1) / kActThreads;
  return launch_kernel(wide_rows(x, ldx) ? act8_quantize_kernel<true> : act8_quantize_kernel<false>,
                       dim3(static_cast<unsigned>(ctas)), dim3(kActThreads), 0, stream, dim3(1, 1, 1), x, units, K / 16, K, ldx, codes, exps, status);
}

cudaError_t launch_act8_dequantize(const uint8_t* codes, const uint8_t* exps, int64_t M, int64_t K, uint16_t* x,
                                   int64_t ldx, cudaStream_t stream) {
  const int64_t units = M * (K / 16);
  const int64_t ctas = (units + kActThreads - 1) / kActThreads;
  return launch_kernel(wide_rows(x, ldx) ? act8_dequantize_kernel<true> : act8_dequantize_kernel<false>,
                       dim3(static_cast<unsigned>(ctas)), dim3(kActThreads), 0, stream, dim3(1, 1, 1), codes, exps, units, K / 16, K, x, ldx);
}

cudaError_t launch_act8_da(const CUtensorMap& tm_du, const CUtensorMap& tm_du3, const CUtensorMap& tm_x,
                           const uint8_t* exps, const SkinnyArgs& a, int grid_rows, int splits, cudaStream_t stream) {
  static uint64_t done = 0;
  if (cudaError_t e = allow_smem(act8_da_kernel, ActDaPlan::kSmem, done)) return e;
  if (splits < 1 || splits > 8) return cudaErrorInvalidValue;
  // unsplit products as clusters of two tiles, as in skinny.cu: they run
  // beside a CTA-pair GEMM and then sit on both SMs of a TPC
  const dim3 cluster = (splits == 1 && grid_rows % 2 == 0) ? dim3(2, 1, 1) : dim3(1, static_cast<unsigned>(splits), 1);
  return launch_kernel(act8_da_kernel, dim3(grid_rows, splits, 1), dim3(kActDaThreads), ActDaPlan::kSmem, stream,
                       cluster, tm_du, tm_du3, tm_x, exps, a);
}

}  // namespace qnf4
