// MX4: quantisation to microscaled 4-bit images, reading back, and the
// product of two images on the matrix cores (gfx950).  Layout and rounding
// are those of include/muon.h.
#include "mo_internal.h"
#include "mx4_internal.h"
#include "ns_common.h"

namespace mo {

namespace {

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef int i32x8v __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__bf16>(__bf16 v) { return static_cast<float>(v); }

// Scale byte of a block from the bits of its largest magnitude: the biased
// exponent less 2 (the list's largest binade starts at 4 = 2^2), 255 for a
// NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const uint32_t e = amax_bits >> 23;
  return e > 2u ? e - 2u : 0u;
}

// One block of 32 values, `n` of them present, `step` elements apart.
template <typename T>
__device__ void quant_block(const T* p, int64_t step, int n, uint8_t* codes, uint8_t* scale) {
  float v[32];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = j < n ? to_f(p[j * step]) : 0.0f;
    amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  const uint32_t sb = scale_byte(amax);
  u32x4v q = {0u, 0u, 0u, 0u};
  if (sb != 255u) {
    const float s = __uint_as_float(sb << 23);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t r = 0;
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 0], v[8 * w + 1], s, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 2], v[8 * w + 3], s, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 4], v[8 * w + 5], s, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 6], v[8 * w + 7], s, 3);
      q[w] = r;
    }
  }
  *reinterpret_cast<u32x4v*>(codes) = q;
  *scale = static_cast<uint8_t>(sb);
}

}  // namespace

// One thread per block: the row image's blocks first, then the transpose's.
// The thread of a row's last block also clears the row's scale padding.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quant_kernel(const Mx4QuantArgs a) {
  int i = 0;
  while (i + 1 < a.count && static_cast<int64_t>(blockIdx.x) >= a.item[i + 1].tile0) ++i;
  const Mx4QuantItem& it = a.item[i];
  const T* src = static_cast<const T*>(it.src);
  int64_t t = (static_cast<int64_t>(blockIdx.x) - it.tile0) * 256 + threadIdx.x;
  const int64_t nb = mx4_blocks(it.cols), nbt = mx4_blocks(it.rows);
  if (it.codes) {
    if (t < it.rows * nb) {
      const int64_t r = t / nb, b = t % nb;
      const int64_t sp = mx4_scale_pitch(it.cols);
      quant_block(src + r * it.ld + b * 32, 1, static_cast<int>(min(int64_t{32}, it.cols - b * 32)),
                  it.codes + (r * nb + b) * 16, it.scales + r * sp + b);
      if (b == nb - 1)
        for (int64_t p = nb; p < sp; ++p) it.scales[r * sp + p] = 0;
      return;
    }
    t -= it.rows * nb;
  }
  if (it.codes_t && t < it.cols * nbt) {
    const int64_t c = t % it.cols, b = t / it.cols;
    const int64_t sp = mx4_scale_pitch(it.rows);
    quant_block(src + b * 32 * it.ld + c, it.ld, static_cast<int>(min(int64_t{32}, it.rows - b * 32)),
                it.codes_t + (c * nbt + b) * 16, it.scales_t + c * sp + b);
    if (b == nbt - 1)
      for (int64_t p = nbt; p < sp; ++p) it.scales_t[c * sp + p] = 0;
  }
}

int64_t mx4_quant_tiles(int64_t rows, int64_t cols, bool row_image, bool col_image) {
  const int64_t t = (row_image ? rows * mx4_blocks(cols) : 0) + (col_image ? cols * mx4_blocks(rows) : 0);
  return (t + 255) / 256;
}

hipError_t launch_mx4_quant(int dt, const Mx4QuantArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (dt == F32) mx4_quant_kernel<float><<<g, 256, 0, s>>>(a);
  else mx4_quant_kernel<__bf16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

// Value of a code: sign, two exponent bits, one mantissa bit.
__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * static_cast<float>(m);
  return (c & 8u) ? -v : v;
}

// 2^(byte - 127); NaN for 255.  Byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t sb) {
  return sb == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(sb ? sb << 23 : 0x00400000u);
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const Mx4DequantArgs a) {
  int i = 0;
  while (i + 1 < a.count && static_cast<int64_t>(blockIdx.x) >= a.item[i + 1].tile0) ++i;
  const Mx4DequantItem& it = a.item[i];
  const int64_t nb = mx4_blocks(it.cols), sp = mx4_scale_pitch(it.cols);
  const int64_t t = (static_cast<int64_t>(blockIdx.x) - it.tile0) * 256 + threadIdx.x;
  if (t >= it.rows * nb) return;
  const int64_t r = t / nb, b = t % nb;
  const float s = scale_value(it.scales[r * sp + b]);
  T* dst = static_cast<T*>(it.dst) + r * it.cols + b * 32;
  const int n = static_cast<int>(min(int64_t{32}, it.cols - b * 32));
  for (int j = 0; j < n; ++j) {
    const uint32_t c = it.codes[(r * nb + b) * 16 + j / 2] >> (4 * (j & 1));
    dst[j] = static_cast<T>(code_value(c & 15u) * s);
  }
}

int64_t mx4_dequant_tiles(int64_t rows, int64_t cols) { return (rows * mx4_blocks(cols) + 255) / 256; }

hipError_t launch_mx4_dequant(int dt, const Mx4DequantArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (dt == F32) mx4_dequant_kernel<float><<<g, 256, 0, s>>>(a);
  else mx4_dequant_kernel<__bf16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ product
// C = A B^T on the scaled matrix instruction, whose operands are 32 codes and
// one scale byte per lane.  Two kernels:
//  * tile: TM x TN outputs per workgroup, both operands staged through LDS;
//  * skinny (few rows of A): B streamed once from memory into registers.
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ i32x8v codes8(u32x4v x) {
  return i32x8v{static_cast<int>(x[0]), static_cast<int>(x[1]), static_cast<int>(x[2]), static_cast<int>(x[3]), 0, 0, 0, 0};
}

// Byte `kSel` of each scale operand belongs to the lane's block.
template <int kSel>
__device__ __forceinline__ f32x16v mfma32(u32x4v a, u32x4v b, f32x16v c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes8(a), codes8(b), c, 4, 4, kSel, static_cast<int>(sa), kSel,
                                                         static_cast<int>(sb));
}

template <typename T>
__device__ __forceinline__ void store_out(T* o, float v, int accumulate) {
  if (accumulate) v += to_f(*o);
  *o = static_cast<T>(v);
}

// Tile kernel.  The contraction is cut into super-stages of 32 blocks (1024
// columns) of up to four stages of 8 blocks.  Any order of the blocks is
// right as long as A and B agree, so lanes 0..31 of a wave take the first
// half of a super-stage and lanes 32..63 the second: a lane's scale bytes of
// a super-stage are then 16 consecutive bytes (one load), a dword per stage,
// a byte per instruction.  In the last, partial super-stage the halves are h
// = 4, 8, 12 or 16 blocks.  Blocks past the end load the last block's codes
// under zero scale bytes in both operands: 2^-254 of a value of at most 36
// is zero in fp32.
// LDS holds two stages; a row of a stage is 8 chunks of 16 bytes, stored at
// chunk ^ (row & 7) so that the 8 rows of a fragment read touch all banks.
// Stage t + 2 is requested once every wave has read stage t, during the last
// of its four steps, while the first fragments of t + 1 are read: one
// barrier per stage, no wait on memory unless it is late by a whole stage.
constexpr int kTileChunk = 128;        // bytes of a row in one stage

// A wave-uniform address, said to be one.
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32));
}

template <int TM, int TN, int WM, int WN, typename T>
__global__ void __launch_bounds__(64 * WM * WN, 1) mx4_tile_kernel(const Mx4MatmulArgs p) {
  constexpr int NW = WM * WN, FM = TM / (32 * WM), FN = TN / (32 * WN);
  constexpr int DA = TM / (8 * NW), DB = TN / (8 * NW);
  constexpr int kStage = (TM + TN) * kTileChunk;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r32 = lane & 31, half = lane >> 5;

  int tm, tn;
  {
    // each XCD (workgroup index mod 8) takes a contiguous range of tiles,
    // walked in bands of 4 tile rows so that its L2 shares panels of both
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * static_cast<uint32_t>(p.tiles_n);
    const uint32_t x = blockIdx.x % 8, y = blockIdx.x / 8;
    const uint32_t t = x * (tiles / 8) + min(x, tiles % 8) + y;
    constexpr uint32_t kBand = 4;
    const uint32_t band = t / (kBand * p.tiles_n);
    const uint32_t rows = min(kBand, p.tiles_m - band * kBand);
    const uint32_t in = t - band * kBand * p.tiles_n;
    tm = __builtin_amdgcn_readfirstlane(static_cast<int>(band * kBand + in % rows));
    tn = __builtin_amdgcn_readfirstlane(static_cast<int>(in / rows));
  }
  const int64_t m0 = static_cast<int64_t>(tm) * TM, n0 = static_cast<int64_t>(tn) * TN;
  const uint32_t pitch = static_cast<uint32_t>(p.nb) * 16u;
  const uint8_t* a0 = p.a + m0 * pitch;
  const uint8_t* b0 = p.b + n0 * pitch;
  const uint8_t* sa0 = p.sa + m0 * p.sp;
  const uint8_t* sb0 = p.sb + n0 * p.sp;
  const int mlast = static_cast<int>(min(static_cast<int64_t>(TM), p.m - m0)) - 1;
  const int nlast = static_cast<int>(min(static_cast<int64_t>(TN), p.n - n0)) - 1;

  // rows past the end repeat the last row; their products are not stored
  uint32_t arow[DA], brow[DB];
#pragma unroll
  for (int i = 0; i < DA; ++i) arow[i] = min(8 * (wave * DA + i) + lane / 8, mlast) * pitch;
#pragma unroll
  for (int i = 0; i < DB; ++i) brow[i] = min(8 * (wave * DB + i) + lane / 8, nlast) * pitch;
  uint32_t asrow[FM], bsrow[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) asrow[f] = min(wm * (TM / WM) + 32 * f + r32, mlast) * static_cast<uint32_t>(p.sp);
#pragma unroll
  for (int f = 0; f < FN; ++f) bsrow[f] = min(wn * (TN / WN) + 32 * f + r32, nlast) * static_cast<uint32_t>(p.sp);

  const int full = p.nb / 32, rest = p.nb % 32;
  const int htail = (rest + 7) / 8 * 4;                // blocks in a half of the last super-stage
  const int stages = 4 * full + htail / 4;

  const int slot = (lane & 7) ^ (lane >> 3);           // the chunk this lane fetches
  auto request = [&](int t) __attribute__((always_inline)) {
    t = __builtin_amdgcn_readfirstlane(t);
    const uint8_t *pa = uniform_ptr(a0), *pb = uniform_ptr(b0);
    const int h = t < 4 * full ? 16 : htail;
    const int blk = (t >> 2) * 32 + (t & 3) * 4 + (slot < 4 ? slot : h + slot - 4);
    const uint32_t off = static_cast<uint32_t>(min(blk, p.nb - 1)) * 16u;
    const uint32_t base = lds_addr(smem) + (t & 1) * kStage;
#pragma unroll
    for (int i = 0; i < DA; ++i) lds_dma16(pa, arow[i] + off, base + (wave * DA + i) * 1024);
#pragma unroll
    for (int i = 0; i < DB; ++i) lds_dma16(pb, brow[i] + off, base + TM * kTileChunk + (wave * DB + i) * 1024);
  };
  auto scales = [&](const uint8_t* base, uint32_t row, int s) __attribute__((always_inline)) -> u32x4v {
    if (s < full) return *reinterpret_cast<const u32x4a4*>(base + row + s * 32 + half * 16);
    u32x4v v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int blk = s * 32 + half * htail + 4 * q;
      if (4 * q < htail && blk < p.nb) {
        uint32_t w = *reinterpret_cast<const uint32_t*>(base + row + blk);
        if (p.nb - blk < 4) w &= (1u << (8 * (p.nb - blk))) - 1u;
        v[q] = w;
      }
    }
    return v;
  };
  // fragment f of step s: the rows of a fragment are 32 apart, so its chunk
  // order is the same and only a constant is added
  const uint8_t* abase = smem + (wm * (TM / WM) + r32) * kTileChunk;
  const uint8_t* bbase = smem + TM * kTileChunk + (wn * (TN / WN) + r32) * kTileChunk;
  uint32_t xs[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) xs[s] = static_cast<uint32_t>(((half * 4 + s) ^ (r32 & 7)) * 16);
  uint32_t buf = 0;                                    // byte offset of the stage being read
  auto frag = [&](const uint8_t* base, int f, int s) __attribute__((always_inline)) -> u32x4v {
    return *reinterpret_cast<const u32x4v*>(base + (buf + xs[s]) + f * 32 * kTileChunk);
  };

  f32x16v acc[FM][FN] = {};
  u32x4v af[2][FM], bf[2][FN], as[FM], bs[FN], asn[FM] = {}, bsn[FN] = {};

  request(0);
#pragma unroll
  for (int f = 0; f < FM; ++f) as[f] = scales(sa0, asrow[f], 0);
#pragma unroll
  for (int f = 0; f < FN; ++f) bs[f] = scales(sb0, bsrow[f], 0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if (stages > 1) request(1);
#pragma unroll
  for (int f = 0; f < FM; ++f) af[0][f] = frag(abase, f, 0);
#pragma unroll
  for (int f = 0; f < FN; ++f) bf[0][f] = frag(bbase, f, 0);

  for (int t = 0; t < stages; ++t) {
    // the next super-stage's scales, three stages ahead
    if ((t & 3) == 0 && t + 4 < stages) {
#pragma unroll
      for (int f = 0; f < FM; ++f) asn[f] = scales(sa0, asrow[f], t / 4 + 1);
#pragma unroll
      for (int f = 0; f < FN; ++f) bsn[f] = scales(sb0, bsrow[f], t / 4 + 1);
    }
    unroll<4>([&](auto S) __attribute__((always_inline)) {
      constexpr int s = S, cur = s & 1, nxt = cur ^ 1;
      if constexpr (s == 3) {
        // this wave's reads of stage t are done, stage t + 1 has arrived
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (t + 2 < stages) request(t + 2);
        buf ^= kStage;
      }
      // (the last stage reads its first step again, for nothing)
#pragma unroll
      for (int f = 0; f < FM; ++f) af[nxt][f] = frag(abase, f, (s + 1) & 3);
#pragma unroll
      for (int f = 0; f < FN; ++f) bf[nxt][f] = frag(bbase, f, (s + 1) & 3);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma32<s>(af[cur][i], bf[cur][j], acc[i][j], as[i][0], bs[j][0]);
    });
    // the next stage's scale dwords move to the front
    const bool turn = (t & 3) == 3;
#pragma unroll
    for (int f = 0; f < FM; ++f) as[f] = turn ? asn[f] : u32x4v{as[f][1], as[f][2], as[f][3], 0u};
#pragma unroll
    for (int f = 0; f < FN; ++f) bs[f] = turn ? bsn[f] : u32x4v{bs[f][1], bs[f][2], bs[f][3], 0u};
  }

  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = wm * (TM / WM) + 32 * i + 8 * (e / 4) + 4 * half + e % 4;
        const int c = wn * (TN / WN) + 32 * j + r32;
        if (r <= mlast && c <= nlast) store_out(out + (m0 + r) * p.ldo + n0 + c, acc[i][j][e], p.accumulate);
      }
}

// Skinny kernel: MT x 16 rows of A (all of them), 16 rows of B per
// workgroup, whose waves share the contraction and add up through LDS.  B's
// codes go from memory to registers once; the instruction's lane groups take
// adjacent blocks, so a row's 64 bytes of a step are one segment, and 16
// blocks of a row (one scale load) are in flight at a time.
template <int MT, typename T>
__global__ void __launch_bounds__(1024) mx4_skinny_kernel(const Mx4MatmulArgs p) {
  extern __shared__ __attribute__((aligned(16))) float part[];     // [waves - 1][MT][64][4]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int r16 = lane & 15, kb = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t br = min(n0 + r16, static_cast<int64_t>(p.n) - 1);
  const uint8_t* b = p.b + br * p.nb * 16;
  const uint8_t* sb = p.sb + br * p.sp;
  const uint8_t *a[MT], *sa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t ar = min(16 * i + r16, p.m - 1);
    a[i] = p.a + ar * p.nb * 16;
    sa[i] = p.sa + ar * p.sp;
  }
  f32x4v acc[MT] = {};
  const int groups = (p.nb + 15) / 16;
  for (int g = wave; g < groups; g += waves) {
    const int k0 = g * 16;
    u32x4v bv[4], bsv = {}, av[MT][4], asv[MT];
    const bool whole = k0 + 16 <= p.nb;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t blk = min(k0 + 4 * s + kb, p.nb - 1);
      bv[s] = *reinterpret_cast<const u32x4v*>(b + blk * 16);
#pragma unroll
      for (int i = 0; i < MT; ++i) av[i][s] = *reinterpret_cast<const u32x4v*>(a[i] + blk * 16);
    }
    if (whole) {
      bsv = *reinterpret_cast<const u32x4a4*>(sb + k0);
#pragma unroll
      for (int i = 0; i < MT; ++i) asv[i] = *reinterpret_cast<const u32x4a4*>(sa[i] + k0);
    } else {
      // blocks past the end: the last block's codes under zero scale bytes
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int blk = k0 + 4 * s, left = p.nb - blk;
        const uint32_t keep = left >= 4 ? ~0u : left > 0 ? (1u << (8 * left)) - 1u : 0u;
        bsv[s] = left > 0 ? *reinterpret_cast<const uint32_t*>(sb + blk) & keep : 0u;
#pragma unroll
        for (int i = 0; i < MT; ++i) asv[i][s] = left > 0 ? *reinterpret_cast<const uint32_t*>(sa[i] + blk) & keep : 0u;
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(av[i][s]), codes8(bv[s]), acc[i], 4, 4, 0,
                                                                  static_cast<int>(asv[i][s] >> (8 * kb)), 0,
                                                                  static_cast<int>(bsv[s] >> (8 * kb)));
  }
  if (waves > 1) {
    f32x4v* q = reinterpret_cast<f32x4v*>(part);
    if (wave) {
#pragma unroll
      for (int i = 0; i < MT; ++i) q[((wave - 1) * MT + i) * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (wave) return;
    for (int w = 0; w < waves - 1; ++w)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] += q[(w * MT + i) * 64 + lane];
  }
  T* out = static_cast<T*>(p.out);
  if (n0 + r16 < p.n) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * i + 4 * kb + e;
        if (r < p.m) store_out(out + r * p.ldo + n0 + r16, acc[i][e], p.accumulate);
      }
  }
}

// A grid holds fewer than 2^32 threads, whichever kernel is taken.
bool mx4_matmul_fits(int64_t m, int64_t n) {
  return ((m + 63) / 64) * ((n + 63) / 64) <= int64_t{0xffffffff} / 256 && (n + 15) / 16 <= int64_t{0xffffffff} / 1024;
}

template <int TM, int TN, int WM, int WN>
static hipError_t run_tile(int out_dt, Mx4MatmulArgs a, hipStream_t s) {
  a.tiles_m = (a.m + TM - 1) / TM;
  a.tiles_n = (a.n + TN - 1) / TN;
  const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
  const dim3 g(static_cast<uint32_t>(tiles));
  if (out_dt == F32) mx4_tile_kernel<TM, TN, WM, WN, float><<<g, 64 * WM * WN, 0, s>>>(a);
  else mx4_tile_kernel<TM, TN, WM, WN, __bf16><<<g, 64 * WM * WN, 0, s>>>(a);
  return hipGetLastError();
}

template <int MT>
static hipError_t run_skinny(int out_dt, const Mx4MatmulArgs& a, int waves, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>((a.n + 15) / 16));
  const size_t lds = static_cast<size_t>(waves - 1) * MT * 64 * 16;
  if (out_dt == F32) mx4_skinny_kernel<MT, float><<<g, 64 * waves, lds, s>>>(a);
  else mx4_skinny_kernel<MT, __bf16><<<g, 64 * waves, lds, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx4_matmul(int out_dt, const Mx4MatmulArgs& a, hipStream_t s) {
  if (a.m <= 64) {
    // waves per workgroup: enough for about 16 on every CU, none without a
    // group of 16 blocks of its own
    const int64_t wgs = (a.n + 15) / 16, groups = (a.nb + 15) / 16;
    int waves = 1;
    while (waves < 16 && waves * 2 <= groups && wgs * waves < 4096) waves *= 2;
    if (a.m <= 16) return run_skinny<1>(out_dt, a, waves, s);
    if (a.m <= 32) return run_skinny<2>(out_dt, a, min(waves, 8), s);
    return run_skinny<4>(out_dt, a, min(waves, 8), s);
  }
  const int64_t t256 = ((a.m + 255) / 256) * static_cast<int64_t>((a.n + 255) / 256);
  const int64_t t128 = ((a.m + 127) / 128) * static_cast<int64_t>((a.n + 127) / 128);
  if (t256 >= 192) return run_tile<256, 256, 2, 2>(out_dt, a, s);
  if (t128 >= 192) return run_tile<128, 128, 2, 2>(out_dt, a, s);
  return run_tile<64, 64, 2, 2>(out_dt, a, s);
}

}  // namespace mo
