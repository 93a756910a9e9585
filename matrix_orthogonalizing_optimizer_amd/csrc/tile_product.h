// The product of two matrices whose rows both run along the contraction, a
// tile of outputs per workgroup (gfx950): 8-bit codes with a scale byte per
// 128 on the scaled matrix instruction, or bf16.  What becomes of a tile's sums
// is the caller's: stored, or turned into a softmax's statistics or gradient.
#pragma once

#include "product.h"

namespace mo {

typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef int i32x8v __attribute__((ext_vector_type(8)));

// Both operands have rows of whole stages of 64 bytes (32 bf16 or 64 codes).
struct ProductArgs {
  const uint8_t *a, *b;          // 16-byte aligned
  uint32_t pitch_a, pitch_b;     // bytes from a row to the next
  const uint8_t *sa, *sb;        // 8-bit: scale bytes of each row
  uint32_t sp;                   // bytes of a row of them
  int m, n;
  int stages;                    // of 64 bytes of a row, even
  int stages_b;                  // of b's rows, which then repeat (even): b = [b b ..] for a = [hi lo ..]
  int tiles_m, tiles_n;
  int splits;                    // workgroups that share a tile's contraction
};

// A wave's 32 x 32 outputs from 64 bytes of each row: lane l gives row l & 31 and
// two chunks of 16 bytes, at 32 (l / 32) bytes of the stage.  (Any order of the
// contraction is right as long as both operands agree.)
// Two instructions a stage: first one for every output block, then the other,
// as two in a row on the same sums would wait for each other.
__device__ __forceinline__ f32x16v mma_bf16(u32x4v a, u32x4v b, f32x16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
struct OpBf16 {
  static constexpr bool kScaled = false, kDecoded = false;
  static constexpr int kSteps = 2;
  template <int kStep>
  static __device__ __forceinline__ f32x16v mma(const u32x4v (&a)[2], const u32x4v (&b)[2], f32x16v c, uint32_t, uint32_t) {
    return mma_bf16(a[kStep], b[kStep], c);
  }
};
// 8-bit codes as they are: the instruction adds the products of 8 columns at a time
// and cuts them at 2^(E - 13), E the largest sum of their codes' exponents (-6 for
// subnormal ones): 2^-13 of the largest product, 2^-10 where it has a subnormal
// code.  The sums are off by 1.4e-5 of their size (2-norm) for normal values, 8e-5
// where a few values are a thousand times the others: enough for bf16 outputs.
struct OpFp8 {
  static constexpr bool kScaled = true, kDecoded = false;
  static constexpr int kSteps = 1;
  static __device__ __forceinline__ i32x8v codes(const u32x4v (&x)[2]) {
    return i32x8v{static_cast<int>(x[0][0]), static_cast<int>(x[0][1]), static_cast<int>(x[0][2]), static_cast<int>(x[0][3]),
                  static_cast<int>(x[1][0]), static_cast<int>(x[1][1]), static_cast<int>(x[1][2]), static_cast<int>(x[1][3])};
  }
  template <int>
  static __device__ __forceinline__ f32x16v mma(const u32x4v (&a)[2], const u32x4v (&b)[2], f32x16v c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes(a), codes(b), c, 0, 0, 0, static_cast<int>(sa), 0, static_cast<int>(sb));
  }
};
// 8-bit codes turned into the bf16 numbers that they stand for, exactly, on
// their way from LDS to the matrix cores: exact products in fp32 sums, at half
// the rate.
struct OpFp8Exact {
  static constexpr bool kScaled = true, kDecoded = true;
};

// 16 codes under a scale as two operands of 8 bf16.
__device__ __forceinline__ void decode16(u32x4v x, float s, u32x4v& lo, u32x4v& hi) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    lo[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[w], s, false));
    lo[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[w], s, true));
    hi[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 + w], s, false));
    hi[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 + w], s, true));
  }
}
// TM x TN outputs, WM x WN waves, in LDS rings of NA stages of A (odd) and one
// less of B.  Sliced: each wave
// takes a part of the contraction for all outputs, with a ring of its own, and
// the waves' sums meet at the end; a wave then has its WM x WN part of them.
template <class OpT, int TMv, int TNv, int WMv, int WNv, int NAv, bool kSlicedv = false>
struct TileCfgT {
  typedef OpT Op;
  static constexpr int TM = TMv, TN = TNv, WM = WMv, WN = WNv, NA = NAv, NB = NA - 1, NW = WM * WN;
  static constexpr bool kSliced = kSlicedv;
  static constexpr int FM = TM / (32 * WM), FN = TN / (32 * WN);
  static constexpr int kThreads = 64 * NW;
  static constexpr int kMinWaves = FM * FN >= 16 ? 1 : 2;        // per SIMD: 256 sums a lane leave room for one
  static constexpr int kStageA = TM * 64, kStageB = TN * 64, kScaleGroup = Op::kScaled ? (TM + TN) * 16 : 0;
  // what the epilogues need to turn 32 rows per wave
  static constexpr int kTurnPitch = TN / WN * 4 + 16;
  static constexpr int kRings = NA * kStageA + NB * kStageB + 2 * kScaleGroup, kRing = (kSliced ? NW : 1) * kRings, kTurn = NW * 32 * kTurnPitch;
  static constexpr int kLds = kRing > kTurn ? kRing : kTurn;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
};

// What a tile costs, from measurements of this file's kernels with few and with
// many tiles and short and long contractions: `fixed` us for a round of as many
// tiles as the chip's 256 CUs hold (`resident` each), and per stage `alone` us,
// or `shared` for every tile that a CU has where that is more.
struct TileCost {
  int size, resident;
  double fixed, alone, shared;
};
inline double tile_us(const TileCost& c, int64_t m, int64_t n, int64_t stages, int splits) {
  const int64_t tiles = ((m + c.size - 1) / c.size) * ((n + c.size - 1) / c.size) * splits;
  const int64_t rounds = (tiles + 256 * c.resident - 1) / (256 * c.resident), per_cu = (tiles + 255) / 256;
  const double stage = c.shared * static_cast<double>(per_cu);
  return c.fixed * static_cast<double>(rounds) + static_cast<double>(stages) * (stage > c.alone ? stage : c.alone);
}

// Where a workgroup's tile is: its first row and column, the last ones inside
// it that exist, the wave's and the lane's place.
struct TilePlace {
  int split, tm, tn, wm, wn, lane, r32, half, mlast, nlast;
  int64_t m0, n0;
};

template <class C>
__device__ __forceinline__ TilePlace tile_place(const ProductArgs& p) {
  TilePlace q;
  q.lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  q.wm = wave / C::WN;
  q.wn = wave % C::WN;
  q.r32 = q.lane & 31;
  q.half = q.lane >> 5;
  {
    // one split after the other; of its tiles each XCD (workgroup index mod 8)
    // takes a contiguous range, walked in bands of 4 tile rows so that its L2
    // shares panels of both operands (a contiguous range of splits and tiles per
    // XCD: 1021 x 2045 x 32512 in 8 splits 262 instead of 222 us; blocks of 16 x
    // 16 tiles for the whole chip: nothing for 8192 x 8192 x 8192, 2% longer for
    // 8192 x 32000 x 2048)
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * static_cast<uint32_t>(p.tiles_n);
    q.split = __builtin_amdgcn_readfirstlane(static_cast<int>(blockIdx.x / tiles));
    const uint32_t id = blockIdx.x % tiles, x = id % 8, y = id / 8;
    const uint32_t t = x * (tiles / 8) + min(x, tiles % 8) + y;
    constexpr uint32_t kBand = 4;
    const uint32_t band = t / (kBand * p.tiles_n);
    const uint32_t rows = min(kBand, p.tiles_m - band * kBand);
    const uint32_t in = t - band * kBand * p.tiles_n;
    q.tm = __builtin_amdgcn_readfirstlane(static_cast<int>(band * kBand + in % rows));
    q.tn = __builtin_amdgcn_readfirstlane(static_cast<int>(in / rows));
  }
  q.m0 = static_cast<int64_t>(q.tm) * C::TM;
  q.n0 = static_cast<int64_t>(q.tn) * C::TN;
  q.mlast = static_cast<int>(min(static_cast<int64_t>(C::TM), p.m - q.m0)) - 1;
  q.nlast = static_cast<int>(min(static_cast<int64_t>(C::TN), p.n - q.n0)) - 1;
  return q;
}

// The stages of split `s`: an odd number of 256 bytes of each row, so that the
// splits, which advance together, use different channels of the memory.
__device__ __forceinline__ void split_range(const ProductArgs& p, int s, int& k0, int& k1) {
  if (p.splits == 1) {
    k0 = 0;
    k1 = p.stages;
    return;
  }
  const int per = 4 * ((((p.stages + 3) / 4 + p.splits - 1) / p.splits) | 1);
  k0 = min(s * per, p.stages);
  k1 = min(s * per + per, p.stages);
}

// acc[i][j]: lane (r32, half), element 4 e + k of the tile's row
// wm TM / WM + 32 i + r32, column wn TN / WN + 32 j + 8 e + 4 half + k.
//
// LDS holds rings of NA (odd) stages of 64 bytes of every row of A and of NB = NA
// - 1 of B, filled by loads that bypass the registers:
//   * a row of a stage is 4 chunks of 16 bytes, stored at chunk ^ ((row / 4) &
//     3): the 16 rows that a 16-byte read serves at a time then touch each of
//     the 64 banks once;
//   * scale bytes come for 16 blocks (32 stages) of a row at a time, and are read
//     a block ahead, behind its first product (as the last reads of a block, which
//     every wave then waits for: 8192 x 28672 x 8192 1456 instead of 1425 us);
//   * a line of 128 bytes holds two stages of a row.  Stages are requested in
//     pairs, both halves of a line one after the other, so that a line is fetched
//     once: a stage of 512 rows at a time fills the first-level cache twice over
//     before its other half is asked for (8192 x 8192 x 8192 in bf16 takes 856 us
//     with stages one by one and 806 in pairs, 8192 x 28672 x 8192 in codes 1525
//     and 1425, 8192 x 8192 x 8192 in tiles of 128 1219 and 966);
//   * at stage t, whose fragments are in registers, the wave waits for its
//     requests of stage t + 1 and the workgroup meets.  The places of stages t - 1
//     and t are then free: at an even stage of A, for stages t + NB and t + NA, at
//     an odd one of B, for t + NB - 1 and t + NB, the same pair.  Meanwhile the
//     fragments of t + 1 are read; products, reads and requests are interleaved
//     one by one.  (Both operands at the even stages: 2048 x 8192 x 32000 843
//     instead of 783 us.)
// Past the end no lane requests, and the number of loads in flight is still the
// same at every wait.  Rows past the end repeat the last row; what comes of them
// is not stored.
//
// C: the waves that share the ring at `smem`; `wave` of them, at wm, wn, which
// add up stages k0 to k1.
template <class C>
__device__ __forceinline__ void ring_sums(const ProductArgs& p, const TilePlace& q, int wave, int wm, int wn, int k0, int k1, uint8_t* smem,
                                          f32x16v (&acc)[C::FM][C::FN]) {
  typedef typename C::Op Op;
  constexpr int TM = C::TM, TN = C::TN, NW = C::NW, FM = C::FM, FN = C::FN, NA = C::NA, NB = C::NB;
  constexpr int kStageA = C::kStageA, kStageB = C::kStageB;
  constexpr int D = TM / (16 * NW), DP = 2 * D;                               // requests of a wave for a stage and a pair of one operand
  constexpr int DS = Op::kScaled ? ((TM + TN) / 64 + NW - 1) / NW : 0;        // and of a group of scales
  constexpr int kRingB = NA * kStageA, kScales = kRingB + NB * kStageB;
  static_assert(TM == TN && NA % 2 == 1 && NA >= 5, "pairs of stages, of both operands alike");
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16v{};
  const int stages = __builtin_amdgcn_readfirstlane(k1 - k0);
  if (stages <= 0) return;                                // the same for all waves of the ring
  const int lane = q.lane;
  const uint8_t* a0 = uniform_ptr(p.a + q.m0 * p.pitch_a + static_cast<int64_t>(k0) * 64);
  const uint8_t* b00 = uniform_ptr(p.b + q.n0 * p.pitch_b);

  // Requests.  Lane l copies chunk l & 3 of row l / 4 of 16 rows, so it fetches
  // the chunk that is stored there.
  const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
  uint32_t arow[D], brow[D];
#pragma unroll
  for (int i = 0; i < D; ++i) {
    arow[i] = min(16 * (wave * D + i) + lane / 4, q.mlast) * p.pitch_a + chunk * 16;
    brow[i] = min(16 * (wave * D + i) + lane / 4, q.nlast) * p.pitch_b + chunk * 16;
  }
  const uint32_t lds0 = lds_addr(smem);
  const uint32_t dst = lds0 + wave * D * 1024, dstb = dst + kRingB;
  int tp = 0, kb = __builtin_amdgcn_readfirstlane(k0 % p.stages_b);           // the pair being requested: its first stage, and b's
  const uint8_t *pa = a0, *pb = uniform_ptr(b00 + static_cast<int64_t>(kb) * 64);
  uint64_t lanes = ~uint64_t{0};                            // which of them request
  auto advance = [&]() __attribute__((always_inline)) {
    tp += 2;
    kb += 2;
    pa = uniform_ptr(pa + 128);
    const bool wrap = kb == p.stages_b;
    kb = wrap ? 0 : kb;
    pb = uniform_ptr(wrap ? b00 : pb + 128);
    const uint32_t half_wave = __builtin_amdgcn_readfirstlane(tp < stages ? -1 : 0);
    lanes = static_cast<uint64_t>(half_wave) << 32 | half_wave;
  };
  // request I of a pair's DP: the two stages of the same rows in turn
  auto request_a = [&](auto I, uint32_t to0, uint32_t to1) __attribute__((always_inline)) {
    constexpr int i = I / 2;
    if constexpr (I % 2 == 0) lds_dma16_masked<i * 1024>(pa, arow[i], dst + to0, lanes);
    else lds_dma16_masked<i * 1024>(uniform_ptr(pa + 64), arow[i], dst + to1, lanes);
  };
  auto request_b = [&](auto I, uint32_t to0, uint32_t to1) __attribute__((always_inline)) {
    constexpr int i = I / 2;
    if constexpr (I % 2 == 0) lds_dma16_masked<i * 1024>(pb, brow[i], dstb + to0, lanes);
    else lds_dma16_masked<i * 1024>(uniform_ptr(pb + 64), brow[i], dstb + to1, lanes);
  };
  // Scale bytes: 64 rows a request, 16 bytes of each (groups of 16 blocks); two
  // groups in turn.
  const int block0 = k0 / 2, blocks = k1 / 2, groups = (blocks + 15) / 16;
  auto request_scales = [&](int g) __attribute__((always_inline)) {
    if constexpr (Op::kScaled) {
#pragma unroll
      for (int i = 0; i < DS; ++i) {
        const int r = (wave * DS + i) % ((TM + TN) / 64);                     // small tiles: some twice, the same bytes
        const bool is_a = r < TM / 64;
        const int row = is_a ? min(r * 64 + lane, q.mlast) : min((r - TM / 64) * 64 + lane, q.nlast);
        const uint8_t* base = uniform_ptr(is_a ? p.sa + q.m0 * p.sp : p.sb + q.n0 * p.sp);
        lds_dma16_at<0>(base, static_cast<uint32_t>(row) * p.sp + g * 16, lds0 + kScales + (g & 1) * C::kScaleGroup + r * 1024);
      }
    }
  };

  // Fragments: 32 rows, lane l holds row l & 31.
  const uint8_t* abase = smem + (wm * (TM / C::WM) + q.r32) * 64;
  const uint8_t* bbase = smem + kRingB + (wn * (TN / C::WN) + q.r32) * 64;
  const uint8_t* asbase = smem + kScales + (wm * (TM / C::WM) + q.r32) * 16;
  const uint8_t* bsbase = smem + kScales + (TM + wn * (TN / C::WN) + q.r32) * 16;
  uint32_t xs[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) xs[s] = static_cast<uint32_t>(((q.half * 2 + s) ^ ((q.r32 >> 2) & 3)) * 16);
  u32x4v af[2][FM][2], bf[2][FN][2];
  uint32_t sa[FM] = {}, sb[FN] = {}, san[FM] = {}, sbn[FN] = {};
  // reading r of a stage's 2 (FM + FN), in the order of need: A's first rows, B, the rest of A
  constexpr int NR = 2 * (FM + FN);
  auto read = [&](auto R, auto set, uint32_t at, uint32_t at_b) __attribute__((always_inline)) {
    constexpr int f = R / 2, s = R % 2, S = set;
    constexpr int fa = f == 0 ? 0 : f > FN ? f - FN : -1, fb = f >= 1 && f <= FN ? f - 1 : -1;
    if constexpr (fa >= 0) af[S][fa][s] = *reinterpret_cast<const u32x4v*>(abase + (at + xs[s]) + fa * 32 * 64);
    if constexpr (fb >= 0) bf[S][fb][s] = *reinterpret_cast<const u32x4v*>(bbase + (at_b + xs[s]) + fb * 32 * 64);
  };
  auto read_scales = [&](int block) __attribute__((always_inline)) {
    if constexpr (Op::kScaled) {
      const int b = min(block, blocks - 1);                                   // past the end: the last again, unused
      const uint32_t off = ((b >> 4) & 1) * C::kScaleGroup + (b & 15);
#pragma unroll
      for (int i = 0; i < FM; ++i) san[i] = asbase[off + i * 512];
#pragma unroll
      for (int j = 0; j < FN; ++j) sbn[j] = bsbase[off + j * 512];
    }
  };
  auto take_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = san[i];
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = sbn[j];
  };
  auto meet = [&]() __attribute__((always_inline)) {       // no memory fence: it would drain the loads
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (NW > 1) __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  request_scales(block0 >> 4);
  if ((block0 & 15) && (block0 >> 4) + 1 < groups) request_scales((block0 >> 4) + 1);
  unroll<NB / 2>([&](auto Q) __attribute__((always_inline)) {
    if constexpr (Q > 0) advance();
    unroll<DP>([&](auto I) __attribute__((always_inline)) { request_a(I, 2 * Q * kStageA, (2 * Q + 1) * kStageA); });
    unroll<DP>([&](auto I) __attribute__((always_inline)) { request_b(I, 2 * Q * kStageB, (2 * Q + 1) * kStageB); });
  });
  wait_loads<(NB - 2) * DP>();
  meet();
  unroll<NR>([&](auto R) __attribute__((always_inline)) { read(R, std::integral_constant<int, 0>{}, 0u, 0u); });
  read_scales(block0);
  take_scales();

  constexpr int NP = FM * FN;
  // columns forth and back, so that a product keeps one operand of the last
  constexpr auto snake = [](int p) constexpr { return p / FN % 2 ? FN - 1 - p % FN : p % FN; };
  uint32_t at = 0, at_b = 0;                               // places of the stage in registers
  for (int t = 0; t < stages; t += 2) {
    unroll<2>([&](auto S) __attribute__((always_inline)) {
      constexpr int cur = S, nxt = cur ^ 1;
      // this wave's reads of the stage are done, its part of the next has come
      wait_loads<(NB - 2 - cur) * DP>();
      meet();
      uint32_t next = 0, next_b = 0, last = 0;
      // what goes with product P of N; the stage's bookkeeping too comes behind
      // its first product, as nothing else would keep the matrix cores busy
      auto besides = [&](auto P, auto N) __attribute__((always_inline)) {
        constexpr int n = N, r0 = P * NR / n, r1 = (P + 1) * NR / n, l0 = P * DP / n, l1 = (P + 1) * DP / n;
        if constexpr (P == 0) {
          next = at + kStageA == NA * kStageA ? 0u : at + kStageA;
          next_b = cur == 1 && at_b + kStageB == NB * kStageB ? 0u : at_b + kStageB;
          last = at == 0 ? (NA - 1) * kStageA : at - kStageA;
          if constexpr (Op::kScaled && cur == 0)
            if (const int b = block0 + t / 2; (b & 15) == 0 && (b >> 4) + 1 < groups) request_scales((b >> 4) + 1);
          if constexpr (cur == 0) advance();
        }
        unroll<r1 - r0>([&](auto R) __attribute__((always_inline)) {
          read(std::integral_constant<int, r0 + decltype(R)::value>{}, std::integral_constant<int, nxt>{}, next, next_b);
        });
        unroll<l1 - l0>([&](auto L) __attribute__((always_inline)) {
          constexpr auto l = std::integral_constant<int, l0 + decltype(L)::value>{};
          if constexpr (cur == 0) request_a(l, last, at);
          else request_b(l, at_b - kStageB, at_b);
        });
        if constexpr (cur == 0 && P == 0) read_scales(block0 + t / 2 + 1);
      };
      if constexpr (Op::kDecoded) {
        float fa[FM], fb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = scale_of(sa[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = scale_of(sb[j]);
        unroll<2>([&](auto H) __attribute__((always_inline)) {
          constexpr int s = H;
          u32x4v a[FM][2], b[FN][2];
#pragma unroll
          for (int j = 0; j < FN; ++j) decode16(bf[cur][j][s], fb[j], b[j][0], b[j][1]);
#pragma unroll
          for (int i = 0; i < FM; ++i) decode16(af[cur][i][s], fa[i], a[i][0], a[i][1]);
          unroll<2 * NP>([&](auto P) __attribute__((always_inline)) {
            constexpr int i = P % NP / FN, j = snake(P), h = P / NP;
            acc[i][j] = mma_bf16(b[j][h], a[i][h], acc[i][j]);
            besides(std::integral_constant<int, 2 * s * NP + decltype(P)::value>{}, std::integral_constant<int, 4 * NP>{});
          });
        });
      } else {
        // a product at a time, and behind each a little of everything else
        unroll<Op::kSteps * NP>([&](auto P) __attribute__((always_inline)) {
          constexpr int i = P % NP / FN, j = snake(P);
          acc[i][j] = Op::template mma<P / NP>(bf[cur][j], af[cur][i], acc[i][j], sb[j], sa[i]);
          besides(P, std::integral_constant<int, Op::kSteps * NP>{});
          __builtin_amdgcn_sched_barrier(0);
        });
      }
      if constexpr (cur == 1) take_scales();
      at = next;
      at_b = next_b;
    });
  }
  wait_loads<0>();                                         // no request outlives the workgroup
}

template <class C>
__device__ __forceinline__ void tile_sums(const ProductArgs& p, const TilePlace& q, uint8_t* smem, f32x16v (&acc)[C::FM][C::FN]) {
  const int wave = q.wm * C::WN + q.wn;
  int k0, k1;
  split_range(p, q.split, k0, k1);
  if constexpr (!C::kSliced) {
    ring_sums<C>(p, q, wave, q.wm, q.wn, k0, k1, smem, acc);
  } else {
    static_assert(C::FM == 1 && C::FN == 1, "a wave keeps one block of 32 x 32");
    typedef TileCfgT<typename C::Op, C::TM, C::TN, 1, 1, C::NA> One;
    const int pairs = (k1 - k0) / 2, per = (pairs + C::NW - 1) / C::NW;
    const int s0 = k0 + 2 * min(wave * per, pairs), s1 = k0 + 2 * min(wave * per + per, pairs);
    f32x16v sums[One::FM][One::FN];
    uint8_t* ring = smem + wave * C::kRings;
    ring_sums<One>(p, q, 0, 0, 0, s0, s1, ring, sums);
    // each block to the wave that keeps it; sums in the waves' order
    static_assert(C::NW * 4096 <= C::kRings, "the blocks fit the wave's ring");
    unroll<C::NW>([&](auto B) __attribute__((always_inline)) {
      constexpr int b = B;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x16v& s = sums[b / C::WN][b % C::WN];
        *reinterpret_cast<f32x4v*>(ring + b * 4096 + g * 1024 + q.lane * 16) = f32x4v{s[4 * g], s[4 * g + 1], s[4 * g + 2], s[4 * g + 3]};
      }
    });
    __syncthreads();
    acc[0][0] = f32x16v{};
#pragma unroll
    for (int w = 0; w < C::NW; ++w)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4v v = *reinterpret_cast<const f32x4v*>(smem + w * C::kRings + wave * 4096 + g * 1024 + q.lane * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[0][0][4 * g + k] += v[k];
      }
  }
  __syncthreads();
}


// Stores the sums, times a factor in device memory where one is given.  Each
// wave turns 32 rows at a time through LDS of its own, so that rows leave as
// whole lines; the 16 bytes of padding per row spread 16 rows over all banks.
template <typename T>
struct StoreArgs {
  T* out;
  int64_t ldo, split_stride;     // elements from a split's outputs to the next split's
  int accumulate;
  const float* scale;            // or null
  int stream;                    // past the caches
};
// Outputs larger than the L2s whose rows are whole lines: 8192 x 32000 x 2048 in
// bf16 (524 MB) 918 to 878 us, 8192 x 8192 x 8192 816 to 812.  Rows that share
// lines gain nothing (129283 x 2045 x 1022 in three terms to fp32 1470 us both ways) and meet in
// the caches.
template <typename T>
int worth_streaming(const T* out, int64_t ldo, int64_t m, int64_t n) {
  constexpr int kSize = sizeof(T);
  return m * n * kSize > (int64_t{32} << 20) && reinterpret_cast<uintptr_t>(out) % 128 == 0 && ldo * kSize % 128 == 0;
}
template <class C, typename T>
__device__ __forceinline__ void tile_store(const StoreArgs<T>& e, const TilePlace& q, uint8_t* smem, const f32x16v (&acc)[C::FM][C::FN]) {
  constexpr int W = C::TN / C::WN, kPitch = C::kTurnPitch, kLanes = W / 4;       // columns, and lanes to a row
  uint8_t* turn = smem + (q.wm * C::WN + q.wn) * 32 * kPitch;
  T* out = e.out + q.split * e.split_stride + q.m0 * e.ldo + q.n0;
  const float f = e.scale ? *e.scale : 1.0f;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4v*>(turn + q.r32 * kPitch + (32 * j + 8 * g + 4 * q.half) * 4) =
            f32x4v{acc[i][j][4 * g] * f, acc[i][j][4 * g + 1] * f, acc[i][j][4 * g + 2] * f, acc[i][j][4 * g + 3] * f};
    // four rows of stores at a time, before which what is added to comes at once
    constexpr int K = 32 * kLanes / 64, kStep = 64 / kLanes, kAtOnce = K < 4 ? K : 4;
    const int row = q.lane / kLanes, col = q.lane % kLanes * 4, c = q.wn * W + col, left = q.nlast + 1 - c;
    const int r = q.wm * (C::TM / C::WM) + 32 * i + row, rows = left > 0 ? q.mlast + 1 - r : 0;
    T* to = out + r * e.ldo + c;
#pragma unroll
    for (int k0 = 0; k0 < K; k0 += kAtOnce) {
      f32x4v v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) v[k] = *reinterpret_cast<const f32x4v*>(turn + ((k0 + k) * kStep + row) * kPitch + col * 4);
      if (e.accumulate) {
        f32x4v add[kAtOnce] = {};
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if ((k0 + k) * kStep < rows) add[k] = load4_out(to + (k0 + k) * kStep * e.ldo, left);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) v[k] += add[k];
      }
      if (e.stream && left >= 4) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if ((k0 + k) * kStep < rows) stream4_out(to + (k0 + k) * kStep * e.ldo, v[k]);
      } else {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if ((k0 + k) * kStep < rows) store4_out(to + (k0 + k) * kStep * e.ldo, v[k], left, 0);
      }
    }
  }
}

// The product of nothing: rows of zeros.
template <typename T>
__global__ void __launch_bounds__(256) product_zero_kernel(T* out, int64_t ldo, int64_t rows, int64_t cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += 256) out[r * ldo + c] = static_cast<T>(0.0f);
}
template <typename T>
hipError_t run_product_zero(T* out, int64_t ldo, int64_t rows, int64_t cols, hipStream_t s) {
  product_zero_kernel<T><<<static_cast<uint32_t>(rows < 4096 ? rows : 4096), 256, 0, s>>>(out, ldo, rows, cols);
  return hipGetLastError();
}

template <class C, typename T>
__global__ void __launch_bounds__(C::kThreads, C::kMinWaves) product_store_kernel(const ProductArgs p, const StoreArgs<T> e) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds];
  const TilePlace q = tile_place<C>(p);
  f32x16v acc[C::FM][C::FN];
  tile_sums<C>(p, q, smem, acc);
  tile_store<C, T>(e, q, smem, acc);
}

template <class C, typename T>
hipError_t run_product_store(ProductArgs p, const StoreArgs<T>& e, hipStream_t s) {
  p.tiles_m = (p.m + C::TM - 1) / C::TM;
  p.tiles_n = (p.n + C::TN - 1) / C::TN;
  const dim3 g(static_cast<uint32_t>(static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.splits));
  product_store_kernel<C, T><<<g, C::kThreads, 0, s>>>(p, e);
  return hipGetLastError();
}

}  // namespace mo
