// Device code shared by the grouped products: element conversions, the
// activations, the lookup of a block's group and rows, and the LDS-tiled
// matrix-core kernel.
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "products.h"

namespace moe {

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_any;
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <Num T> struct Acc { using t4 = f32x4; };
template <> struct Acc<Num::kInt8> { using t4 = i32x4; };

// Round to nearest even, NaN kept (hardware conversions).
__device__ __forceinline__ uint32_t pack_f16_rne(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, (f16x2){(_Float16)lo, (_Float16)hi});
}
__device__ __forceinline__ uint32_t pack_half(bool fp16, float lo, float hi) {
  return fp16 ? pack_f16_rne(lo, hi) : pack_bf16_rne(lo, hi);
}
__device__ __forceinline__ float half_to_f32(bool fp16, uint16_t b) { return fp16 ? fp16_to_f32(b) : bf16_to_f32(b); }

// act(g) = g s(z) with s the sigmoid: z = g (silu), z = 2c (g + b g^3) (gelu:
// the tanh form with 1 + tanh(y) = 2 s(2y), no cancellation for negative g).
// With t = exp(-|z|) and r = 1 / (1 + t), s is r or t r by the sign of z and
// 1 - s the other, so neither overflows nor cancels.  The hardware exp2 and
// reciprocal flush subnormal results: t is carried as t 2^64, so that act(g)
// goes as far down as fp32 does.  Adding 64 rounds exp2's argument to 2^-19 for
// |z| < 22: t is off by up to 2^-19 ln 2 = 1.3e-6 of itself, act(g) by 1 - s
// times that, 370 times less than the half step of an fp16 result.
constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;
constexpr float kDrop = 0x1p-64f;
struct Gate {
  float z, dz, r, low;  // low = t r 2^64
};
__device__ __forceinline__ Gate gate_of(int act, float g) {
  Gate s;
  s.z = g;
  s.dz = 1.0f;
  if (act != MOE_ACT_SILU) {
    const float g2 = fminf(g * g, 1e30f);  // keeps dz finite
    s.z = kGeluC2 * fmaf(kGeluB * g2, g, g);
    s.dz = kGeluC2 * fmaf(3.0f * kGeluB, g2, 1.0f);
  }
  const float t = __builtin_amdgcn_exp2f(fmaf(-fabsf(s.z), 1.4426950408889634f, 64.0f));
  s.r = __builtin_amdgcn_rcpf(fmaf(t, kDrop, 1.0f));
  s.low = t * s.r;
  return s;
}
__device__ __forceinline__ float activate(int act, float g) {
  const Gate s = gate_of(act, g);
  return s.z < 0.0f ? g * s.low * kDrop : g * s.r;
}
// act(g) and act'(g) = s + g z' s (1 - s)
__device__ __forceinline__ void activate_slope(int act, float g, float& value, float& slope) {
  const Gate s = gate_of(act, g);
  const bool neg = s.z < 0.0f;
  const float sig = neg ? s.low : s.r;  // 2^64 times s where negative
  const float rest = neg ? s.r : s.low * kDrop;
  const float unit = neg ? kDrop : 1.0f;
  value = g * sig * unit;
  slope = fmaf(g * sig * rest, s.dz, sig) * unit;
}

// The power of two that a group's fp16 slopes were divided by, from the bits of
// the largest (0: none passes 65504): that one is in [2^14, 2^15) afterwards.
constexpr float kHalfMax = 65504.0f;
__device__ __forceinline__ float group_lift(uint32_t top) {
  return top ? __builtin_amdgcn_ldexpf(1.0f, __builtin_amdgcn_frexp_expf(__uint_as_float(top)) - 15) : 1.0f;
}

// 16 x 16 of A (lane l: row l % 16, 16 bytes of the contraction at
// 16 (l / 16)) times B (the same for its columns): D holds column l % 16, rows
// 4 (l / 16) + i.
template <Num T>
__device__ __forceinline__ typename Acc<T>::t4 mfma16x16(u32x4 a, u32x4 b, typename Acc<T>::t4 c) {
  if constexpr (T == Num::kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else if constexpr (T == Num::kFp16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Buffer descriptor of raw byte offsets below 2^31 from `base`; a lane with
// nothing to load passes kNoLoad, which is out of range and reads zeros.
constexpr uint32_t kNoLoad = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const char* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7FFFFFFF, 0x00020000);
}
// 16 bytes per lane, global -> LDS: lane l writes dst + 16 l.
__device__ __forceinline__ void buffer_to_lds16(__amdgpu_buffer_rsrc_t r, lds_char* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_any*)dst, 16, voff, soff, 0, 0);
}

// Transposing LDS read.  `__restrict` (true here: nothing else is accessed in
// the function) keeps the compiler from making the read wait for every copy
// into LDS in flight; the stage's own copies are waited for explicitly.
__device__ __forceinline__ u32x2 read_transposed(lds_char* __restrict p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// Waits for this wave's vector-memory operations, all but the newest N.
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// Barrier that waits for this wave's LDS operations but leaves copies in flight.
__device__ __forceinline__ void lds_only_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Group e's rows, clamped to the row matrices: offsets out of range or order
// give an empty or shortened group.
__device__ __forceinline__ void group_rows(const int32_t* offsets, int rows, int e, int& begin, int& end) {
  if (!offsets) {
    begin = 0;
    end = rows;
    return;
  }
  begin = min(max(offsets[e], 0), rows);
  end = max(begin, min(offsets[e + 1], rows));
}

// Block b of a grid whose blocks the hardware deals to the 8 XCDs in turn ->
// a unit such that each XCD takes one contiguous run of the `units` (their
// operands then share its L2); -1 past the end.
__device__ __forceinline__ int xcd_unit(int b, int units) {
  const int x = b & 7, i = b >> 3, q = units >> 3, r = units & 7;
  return i < q + (x < r) ? x * q + min(x, r) + i : -1;
}

// One unit of a tiled product: a tile, or one part of a tile's contraction.
struct RowTile {
  int group, row0, end, tile_n;  // group; first row; end of the group's rows; column tile
  int part, parts;               // this unit's share of the contraction
  int slot, slot_step;           // parts > 1: where its raw sums go, and from one part to the next
};

// How the tiles of a forward product or an input gradient go to the compute
// units, which hold `slots` blocks at a time: the tiles beyond the last full
// round would occupy rem = tiles mod slots of them for a whole tile's time, so
// their contraction is split in up to slots / rem parts.  Worth it where the
// saved stages outweigh the raw sums' way through memory and the joining
// kernel; a part keeps at least 4 stages.
struct Rounds {
  int full, rem, parts;
};
template <int BM, int BN>
__host__ __device__ __forceinline__ Rounds rounds_of(int tiles, int stages, int max_parts) {
  constexpr int slots = BM == 256 ? 256 : 512;
  Rounds r;
  r.full = tiles / slots * slots;
  r.rem = tiles - r.full;
  r.parts = 1;
  if (r.rem) {
    int s = slots / r.rem;
    s = s < max_parts ? s : max_parts;
    s = s < stages / 4 ? s : stages / 4;
    const int cost = BM == 256 ? 6 + r.rem * s / 8 : 12 + r.rem * s / 32;  // in stages
    if (s > 1 && stages * (s - 1) / s > cost) r.parts = s;
  }
  return r;
}

// This block's row tile (BM rows of one group) and column tile: tiles are
// counted over the groups (at most 256, one thread each), dealt by xcd_unit,
// and walked in bands of kBand row tiles so that blocks running side by side
// share weight columns and rows.  JOIN: block b has the b-th split tile.
// `scratch`: 28 bytes of LDS, free again after the caller's next barrier.
// Every thread calls it.
constexpr int kBand = 8;
template <int BM, int BN, int THREADS, bool JOIN>
__device__ __forceinline__ bool find_row_tile(const ProductArgs& a, int tiles_n, int stages, lds_char* scratch, RowTile& t) {
  typedef __attribute__((address_space(3))) int lds_int;
  lds_int* wsum = (lds_int*)scratch;  // [4] tiles of 64 groups each
  lds_int* found = wsum + 4;          // [3]
  const int tid = threadIdx.x;
  int tiles_m;
  int begin = 0, end = a.rows, mine = 0, upto = 0;
  if (a.groups == 1) {
    group_rows(a.offsets, a.rows, 0, begin, end);
    tiles_m = (end - begin + BM - 1) / BM;
  } else {
    static_assert(THREADS >= 256, "one thread per group");
    if (tid < 256) {
      if (tid < a.groups) group_rows(a.offsets, a.rows, tid, begin, end);
      mine = tid < a.groups ? (end - begin + BM - 1) / BM : 0;
      upto = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d, 64);
        if ((tid & 63) >= d) upto += v;
      }
      if ((tid & 63) == 63) wsum[tid >> 6] = upto;
    }
    __syncthreads();
    tiles_m = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < (tid >> 6)) upto += wsum[w];
      tiles_m += wsum[w];
    }
  }
  // the grid and the raw sums' space are sized for offsets in order, which
  // have at most this many tiles: with others some rows stay unspecified
  tiles_m = __builtin_amdgcn_readfirstlane(min(tiles_m, row_tile_bound(a.rows, a.groups, BM)));
  const Rounds r = rounds_of<BM, BN>(tiles_m * tiles_n, stages, a.splits);
  const int whole = r.full + (r.parts == 1 ? r.rem : 0);
  int unit;
  t.part = 0;
  t.parts = 1;
  t.slot = t.slot_step = 0;
  const int b = blockIdx.x, padded = (whole + 7) / 8 * 8;
  if (JOIN) {
    if (r.parts == 1 || b >= r.rem) return false;
    unit = whole + b;
  } else if (b < padded) {
    unit = xcd_unit(b, whole);
  } else {
    if (r.parts == 1) return false;
    const int u = xcd_unit(b - padded, r.rem * r.parts);
    if (u < 0) return false;
    // neighbours take the same part of neighbouring tiles: they share operands
    t.part = u / r.rem;
    unit = whole + u % r.rem;
  }
  if (unit < 0) return false;
  if (unit >= whole) {
    t.parts = r.parts;
    t.slot = t.part * r.rem + (unit - whole);
    t.slot_step = r.rem;
  }
  const int band = unit / (kBand * tiles_n), in = unit % (kBand * tiles_n);
  const int high = min(kBand, tiles_m - band * kBand);
  const int m = band * kBand + in % high;
  t.tile_n = in / high;
  if (a.groups == 1) {
    // uniform, but the compiler cannot see it: the copies' descriptors must
    // stay in scalar registers
    t.group = 0;
    t.row0 = __builtin_amdgcn_readfirstlane(begin + m * BM);
    t.end = __builtin_amdgcn_readfirstlane(end);
    return true;
  }
  if (tid < 256 && m < upto && m >= upto - mine) {
    found[0] = tid;
    found[1] = begin + (m - (upto - mine)) * BM;
    found[2] = end;
  }
  __syncthreads();
  t.group = __builtin_amdgcn_readfirstlane(found[0]);
  t.row0 = __builtin_amdgcn_readfirstlane(found[1]);
  t.end = __builtin_amdgcn_readfirstlane(found[2]);
  return true;
}

// ---- LDS-tiled product ------------------------------------------------------
// A block computes BM x BN of a group's product on WM x WN waves, each wave a
// grid of 16 x 16 matrix-core tiles.  The contraction is walked in stages of
// 128 bytes a row (64 16-bit values, 128 codes).  One operand's stage is a slot
// of a ring of kRing LDS buffers that direct global -> LDS copies fill: the
// current stage, the next one, and the one after for P.  An operand comes in
// one of two layouts:
//  - contraction contiguous in memory (x, codes, w in the forward product):
//    LDS rows of 128 bytes, 16-byte chunks swizzled by the row so that the 16
//    rows of one read cycle fall on different banks;
//  - contraction across the rows (w in the input gradient; dy and x in the
//    weight gradient): LDS holds 64 rows of BM (or BN) values and the
//    transposing LDS read hands each lane 4 consecutive contraction values of
//    its column; chunks are swizzled by row, so that the 8 rows that one read
//    cycle covers fall on different banks.  No operand is ever transposed in
//    memory.
// Missing rows, columns, the contraction's tail and stages past the end are
// zeros (out of range buffer loads), so they add nothing to the sums.
//
// The matrix cores take Q's values as A and P's as B: a lane then holds four
// consecutive columns of one result row.  16-bit results go through LDS and
// leave as whole rows of 16-byte stores; fp32 ones leave from registers.
//
// Gated: the block's columns are BN/2 gate and the same BN/2 up columns,
// interleaved by 16 so that a wave holds g and u of the same elements.
//
// What bounds it: power.  At 8192^3 in bf16 (random values) the chip holds
// 1.85 GHz with the matrix cores busy 78% of the cycles: 1500 TFLOP/s forward,
// 1480 input gradient, 1460 weight gradient (a large library product on the
// same card: 1570, 86% at 1.77 GHz), codes 2800 TOP/s (library: 2390).  What it
// took, each step timed at that size (forward / weight gradient / codes, us):
//  - 32 x 32 tiles, two buffers of both operands, all copies issued after the
//    barrier: 854 / 941 / 462.  A compute unit accepts a 1 KB copy every 16
//    cycles, so eight waves that issue eight each wait for each other with the
//    matrix cores idle; a deeper ring of half stages did not help (884);
//  - copies and fragment reads spread between the products: 824 / 790 / 438;
//  - 16 x 16 tiles: 777 / 749 / 401.  In a loop of products alone they run
//    at 2010 TFLOP/s, 32 x 32 ones at 1800: less power per product;
//  - products at raised wave priority, and the hand-over to the next stage
//    three eighths into its second step: 750 / 763 / 397.
// Four waves of 128 x 128 (fewer LDS reads, one wave per SIMD) spilled and lost
// a third.  128 x 128 blocks, two per compute unit, reach 1180 TFLOP/s (half
// the products per byte copied) and serve where few 256-wide ones would run.
// A tile costs about 8 us beside its stages (start 1.5, first copies 1.3, the
// results' way through LDS 1.8 and out 3), as much as 5 of them.  One block
// per compute unit that takes tiles from a queue and copies the next tile's
// first stages under the results' writing was no faster (its bookkeeping took
// registers from the loop).
//
// JOIN: the block adds the raw sums of a split tile's parts, in order, instead
// of computing them, and writes the result.
constexpr int kRing = 5;  // LDS buffers of one operand's stage
template <Num T, Pass PASS, Result RES, bool JOIN, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_tile_kernel(ProductArgs a) {
  constexpr int NW = WM * WN, THREADS = 64 * NW;
  constexpr int MI = BM / 16 / WM, NJ = BN / 16 / WN;
  constexpr bool P_STR = PASS == Pass::kWeightGrad, Q_STR = PASS != Pass::kForward;
  constexpr bool GATED = RES == Result::kGated;
  constexpr int ES = T == Num::kInt8 ? 1 : 2;
  constexpr int BK = 128 / ES;  // contraction values per stage
  constexpr int kPBytes = BM * 128, kQBytes = BN * 128;
  constexpr int kSlot = kPBytes;  // ring slot: one operand's stage
  constexpr int PI = kPBytes / 1024 / NW, QI = kQBytes / 1024 / NW;  // 1 KB copies per wave and stage
  constexpr int NO = GATED ? BN / 2 : BN;                            // result columns per block
  static_assert(NJ <= MI && MI % PI == 0 && MI >= 4, "a read of Q and a copy of P per row block");
  static_assert(PI * NW * 1024 == kPBytes && QI * NW * 1024 == kQBytes, "even copy split");
  static_assert(!GATED || NJ % 2 == 0, "gate and up blocks in pairs");
  static_assert(T != Num::kInt8 || PASS == Pass::kForward, "codes have no backward pass");
  using acc_t = typename Acc<T>::t4;
  __shared__ __attribute__((aligned(1024))) char smem_raw[kRing * kSlot];
  static_assert(PI == QI && BM * BN * 2 <= kRing * kSlot, "equal slots; the 16-bit result fits the ring");
  lds_char* smem = (lds_char*)smem_raw;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, quad = lane >> 4;
  const int F = a.cols / 2;  // gated: gate rows of W
  const int ncols = GATED ? F : a.cols;
  const int tiles_n = (ncols + NO - 1) / NO;

  // this block's rows [row0, row0 + live) and columns [n0, ...), its group,
  // the contraction's length and this block's stages of it
  int group, row0, live, n0, klen, part, parts, slot, slot_step;
  int gbegin = 0;
  if constexpr (PASS == Pass::kWeightGrad) {
    // every group's tiles are spread over all XCDs: the groups' contractions
    // differ in length
    const int tiles_m = (a.wrows + BM - 1) / BM, tiles = tiles_m * tiles_n;
    const int in = JOIN ? blockIdx.x : xcd_unit(blockIdx.x, tiles);
    if (in < 0) return;
    group = blockIdx.y;
    parts = a.splits;
    part = JOIN ? 0 : blockIdx.z;
    slot = (part * a.groups + group) * tiles + in;
    slot_step = a.groups * tiles;
    const int band = in / (kBand * tiles_n), high = min(kBand, tiles_m - band * kBand);
    row0 = (band * kBand + in % (kBand * tiles_n) % high) * BM;
    n0 = in % (kBand * tiles_n) / high * NO;
    live = min(BM, a.wrows - row0);
    int gend;
    group_rows(a.offsets, a.rows, group, gbegin, gend);
    klen = __builtin_amdgcn_readfirstlane(gend - gbegin);
    gbegin = __builtin_amdgcn_readfirstlane(gbegin);
  } else {
    klen = a.contract;
    RowTile t;
    if (!find_row_tile<BM, BN, THREADS, JOIN>(a, tiles_n, (klen + BK - 1) / BK, smem, t)) return;
    group = t.group;
    row0 = t.row0;
    live = min(BM, t.end - t.row0);
    n0 = t.tile_n * NO;
    part = t.part;
    parts = t.parts;
    slot = t.slot;
    slot_step = t.slot_step;
    if (a.groups > 1) __syncthreads();  // the lookup's LDS is free
  }
  const int stages = (klen + BK - 1) / BK;
  // (at most 2^16 stages and 8 parts; short contractions feel a division)
  const int st0 = parts == 1 ? 0 : stages * part / parts, st1 = parts == 1 ? stages : stages * (part + 1) / parts;
  // raw sums of a part: every lane's, 16 bytes each
  auto raw = [&](int at, int i, int j) {
    return reinterpret_cast<acc_t*>(a.partial + (int64_t)at * (BM * BN * 4)) + ((wave * MI + i) * NJ + j) * 64 + lane;
  };

  acc_t acc[MI][NJ];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = acc_t{};
  };
  if constexpr (JOIN) {
    clear();
    for (int s = 0; s < parts; ++s)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] += *raw(slot + s * slot_step, i, j);
  } else {
  // ---- copies ----
  const char* pbase = P_STR ? a.p + (int64_t)gbegin * a.ldp + (int64_t)row0 * ES : a.p + (int64_t)row0 * a.ldp;
  const char* qbase;
  if constexpr (PASS == Pass::kForward)
    qbase = a.q + (int64_t)group * a.q_group + (int64_t)n0 * a.ldq;
  else if constexpr (PASS == Pass::kInputGrad)
    qbase = a.q + (int64_t)group * a.q_group + (int64_t)n0 * ES;
  else
    qbase = a.q + (int64_t)gbegin * a.ldq + (int64_t)n0 * ES;
  uint32_t pv[PI], qv[QI];  // byte offsets of this lane's copies in stage 0, or kNoLoad
  int pk[PI], qk[QI];       // their contraction position: first value (contiguous) or row (strided)
  auto place = [&](bool strided, int j, int per_wave, int width, int64_t ld, int limit, bool gated, uint32_t& v, int& k) {
    const int inst = wave * per_wave + j;
    if (strided) {
      const int cpr = width / 8;  // 16-byte chunks per LDS row
      const int kr = inst * (64 / cpr) + lane / cpr;
      const int c = (lane % cpr) ^ (((kr & 3) | ((kr >> 1) & 4)) << 1);
      v = 8 * c < limit ? (uint32_t)(kr * ld + 16 * c) : kNoLoad;
      k = kr;
    } else {
      const int r = inst * 8 + lane / 8;
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      int src = r;
      if (gated) {  // LDS row r: block r / 16 belongs to wave column (r / 16) / NJ
        const int jb = r / 16;
        src = (jb / NJ * (NJ / 2) + jb % NJ / 2) * 16 + r % 16;
      }
      v = src < limit ? (uint32_t)(src * ld + 16 * c) : kNoLoad;
      k = c * (16 / ES);
    }
  };
#pragma unroll
  for (int j = 0; j < PI; ++j) place(P_STR, j, PI, BM, a.ldp, live, false, pv[j], pk[j]);
#pragma unroll
  for (int j = 0; j < QI; ++j) place(Q_STR, j, QI, BN, a.ldq, ncols - n0, GATED, qv[j], qk[j]);
  // The copies of an operand's stage: begin_p / begin_q set the descriptor
  // (and, in the contraction's last stage and past it, drop the lanes with
  // nothing to load: in place, so that the copies' offsets live in registers
  // of their own -- an offset in a temporary register makes the compiler wait
  // for the copy before the register's next use), then copy_p(slot, c) is this
  // wave's c-th copy into ring slot `slot`.
  __amdgpu_buffer_rsrc_t pr, qr, ur;
  auto values_from = [&](int st) { return st < st1 ? klen - st * BK : 0; };
  auto begin_p = [&](int st) {
    const int left = values_from(st);
    if (left < BK) {
#pragma unroll
      for (int j = 0; j < PI; ++j) pv[j] = pk[j] < left ? pv[j] : kNoLoad;
    }
    pr = buffer_at(P_STR ? pbase + (int64_t)st * BK * a.ldp : pbase + (int64_t)st * 128);
  };
  auto begin_q = [&](int st) {
    const int left = values_from(st);
    if (left < BK) {
#pragma unroll
      for (int j = 0; j < QI; ++j) qv[j] = qk[j] < left ? qv[j] : kNoLoad;
    }
    const char* q = Q_STR ? qbase + (int64_t)st * BK * a.ldq : qbase + (int64_t)st * 128;
    qr = buffer_at(q);
    if (GATED) ur = buffer_at(q + (int64_t)F * a.ldq);
  };
  auto copy_p = [&](int slot, int c) { buffer_to_lds16(pr, smem + slot * kSlot + (wave * PI + c) * 1024, pv[c], 0); };
  auto copy_q = [&](int slot, int c) {  // gated: the copy's 8 rows are gate or up
    buffer_to_lds16(GATED && (wave * QI + c) / 2 % 2 ? ur : qr, smem + slot * kSlot + (wave * QI + c) * 1024, qv[c], 0);
  };

  // ---- fragments ----
  // contiguous: lane l reads chunk 4s + l / 16 of row (block row) + l % 16
  const int row_at = l16 * 128, chunk_sw = (l16 >> 1) & 7;
  // strided: lane l reads, for columns 4 (l % 4) .. of its block, row
  // 32s + 8 (l / 16) + 4t + l % 16 / 4 (t = 0, 1)
  const int sj = l16 >> 2, fold = sj | (quad & 1) << 2;
  auto strided_at = [&](int width, int block) {
    return (8 * quad + sj) * width * 2 + 32 * (block ^ fold) + 8 * (l16 & 3);
  };
  int pat[MI], qat[NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i) pat[i] = P_STR ? strided_at(BM, wm * MI + i) : (wm * MI + i) * 2048 + row_at;
#pragma unroll
  for (int j = 0; j < NJ; ++j) qat[j] = Q_STR ? strided_at(BN, wn * NJ + j) : (wn * NJ + j) * 2048 + row_at;
  auto fragment = [&](bool strided, int width, lds_char* at, int s) -> u32x4 {
    if (strided) {
      lds_char* q = at + s * 32 * width * 2;
      const u32x2 lo = read_transposed(q), hi = read_transposed(q + 8 * width);
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    }
    return *(__attribute__((address_space(3))) u32x4*)(at + 16 * ((4 * s + quad) ^ chunk_sw));
  };
  // One row block's products.  The fences keep the order written here: each
  // read and copy issues while products run.
  u32x4 pf[MI], qf[2][NJ];
  auto row = [&](int i, int step) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = mfma16x16<T>(qf[step][j], pf[i], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };

  const int nst = st1 - st0;
  const bool busy = wm * MI * 16 < live;  // this wave has rows
  if (nst > 0) {
    begin_p(st0);
#pragma unroll
    for (int c = 0; c < PI; ++c) copy_p(0, c);
    begin_q(st0);
#pragma unroll
    for (int c = 0; c < QI; ++c) copy_q(1, c);
    begin_p(st0 + 1);
#pragma unroll
    for (int c = 0; c < PI; ++c) copy_p(2, c);
    begin_q(st0 + 1);
#pragma unroll
    for (int c = 0; c < QI; ++c) copy_q(3, c);
    __builtin_amdgcn_sched_barrier(0);
    clear();  // while the first copies are under way
    wait_copies<PI + QI>();
    lds_only_barrier();
    // Iteration i: ps and qs hold stage i, pn and qn stage i + 1, `spare` is
    // free and takes P's stage i + 2 during the first of the stage's two
    // steps.  Three eighths into the second step (all of stage i's fragments are
    // in registers by then) every wave has to be done with stage i and stage
    // i + 1 to have landed (that newest P may be in flight): ps takes Q's stage
    // i + 2, and qs is the next spare one.  A row block's next P fragment
    // replaces the current one as soon as its products are issued; Q's, which
    // every row block uses, alternate between two sets.
    int ps = 0, qs = 1, pn = 2, qn = 3, spare = 4;
    auto turn = [&](int i) {
      wait_copies<PI>();
      lds_only_barrier();
      begin_q(st0 + i + 2);
    };
    auto rotate = [&]() {
      const int p = ps, q = qs;
      ps = pn;
      qs = qn;
      pn = spare;
      qn = p;
      spare = q;
    };
    if (busy) {
      constexpr int kHead = MI * 3 / 8;  // row blocks of the second step before the turn
      auto read_p = [&](int slot, int i, int s) { pf[i] = fragment(P_STR, BM, smem + slot * kSlot + pat[i], s); };
      auto read_q = [&](int slot, int j, int s) { qf[s][j] = fragment(Q_STR, BN, smem + slot * kSlot + qat[j], s); };
#pragma unroll
      for (int j = 0; j < NJ; ++j) read_q(qs, j, 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) read_p(ps, i, 0);
      for (int i = 0; i < nst; ++i) {
        begin_p(st0 + i + 2);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
          row(m, 0);
          read_p(ps, m, 1);
          if (m < NJ) read_q(qs, m, 1);
          if (m % (MI / PI) == 0) copy_p(spare, m / (MI / PI));
        }
#pragma unroll
        for (int m = 0; m < kHead; ++m) row(m, 1);
        turn(i);
#pragma unroll
        for (int m = 0; m < kHead; ++m) read_p(pn, m, 0);
#pragma unroll
        for (int m = kHead; m < MI; ++m) {
          constexpr int kRest = MI - kHead;
          row(m, 1);
          read_p(pn, m, 0);
#pragma unroll
          for (int j = NJ * (m - kHead) / kRest; j < NJ * (m - kHead + 1) / kRest; ++j) read_q(qn, j, 0);
#pragma unroll
          for (int c = QI * (m - kHead) / kRest; c < QI * (m - kHead + 1) / kRest; ++c) copy_q(ps, c);
        }
        rotate();
      }
    } else {
      // a wave without rows only copies
      for (int i = 0; i < nst; ++i) {
        begin_p(st0 + i + 2);
#pragma unroll
        for (int c = 0; c < PI; ++c) copy_p(spare, c);
        turn(i);
#pragma unroll
        for (int c = 0; c < QI; ++c) copy_q(ps, c);
        rotate();
      }
    }
    wait_copies<0>();  // the zeros of stages past the end
  } else {
    clear();
  }
  if (parts > 1) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) *raw(slot, i, j) = acc[i][j];
    return;
  }
  }  // !JOIN

  // ---- results ----
  // element e of acc[i][j]: row rowl(i), column coll(j) + e
  auto rowl = [&](int i) { return (wm * MI + i) * 16 + l16; };
  auto coll = [&](int j) {
    return (GATED ? (wn * (NJ / 2) + j / 2) * 16 : (wn * NJ + j) * 16) + 4 * quad;
  };
  {
    const bool fp16 = T == Num::kFp16 || (T == Num::kInt8 && a.out_type == MOE_TYPE_FP16);
    // codes: the sum times the row's and the column's scale
    float prow[MI];
    if constexpr (T == Num::kInt8) {
#pragma unroll
      for (int i = 0; i < MI; ++i) prow[i] = rowl(i) < live ? a.pscale[row0 + rowl(i)] : 0.0f;
    }
    // the gated block's fp16 slopes may stand divided by a power of two
    constexpr bool LIFT = T == Num::kFp16 && PASS != Pass::kForward;
    const float lift = LIFT && a.tops ? group_lift(a.tops[group]) : 1.0f;
    const float* qs = T == Num::kInt8 ? a.qscale + (int64_t)group * a.cols : nullptr;
    auto value = [&](int i, int j) -> f32x4 {
      f32x4 v;
      if constexpr (T == Num::kInt8) {
        const int c = n0 + coll(j);
        const f32x4 s = c < ncols ? *reinterpret_cast<const f32x4*>(qs + c + (GATED && j % 2 ? F : 0)) : f32x4{};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * prow[i] * s[e];
      } else {
        v = acc[i][j];
        if constexpr (LIFT) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= lift;
        }
      }
      return v;
    };
    if constexpr (RES == Result::kWide) {
      char* outp = (char*)a.out;
      if constexpr (PASS == Pass::kWeightGrad) outp += (int64_t)group * a.wrows * a.cols * 4;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (rowl(i) >= live) continue;
        char* rowp = outp + ((int64_t)row0 + rowl(i)) * a.ldout * 4;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int c = n0 + coll(j);
          if (c < ncols) *reinterpret_cast<f32x4*>(rowp + (int64_t)c * 4) = value(i, j);
        }
      }
    } else {
      uint16_t* outp = (uint16_t*)a.out;
      if constexpr (PASS == Pass::kWeightGrad) outp += (int64_t)group * a.wrows * a.cols;
      __syncthreads();  // the stage buffers are free
      // LDS rows of W values, 16-byte chunks swizzled by the row
      auto put = [&](int width, int row, int col, f32x4 v) {
        const u32x2 h = {pack_half(fp16, v[0], v[1]), pack_half(fp16, v[2], v[3])};
        *(__attribute__((address_space(3))) u32x2*)(smem + row * width * 2 +
                                                    16 * ((col >> 3) ^ (row & (width / 8 - 1))) + 2 * (col & 7)) = h;
      };
      auto get = [&](int width, int row, int chunk) -> u32x4 {
        return *(__attribute__((address_space(3))) u32x4*)(smem + row * width * 2 + 16 * (chunk ^ (row & (width / 8 - 1))));
      };
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; j += GATED ? 2 : 1) {
          f32x4 v = value(i, j);
          if constexpr (GATED) {
            const f32x4 u = value(i, j + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]) * u[e];
          }
          put(NO, rowl(i), coll(j), v);
        }
      __syncthreads();
      for (int x = tid; x < BM * (NO / 8); x += THREADS) {
        const int r = x / (NO / 8), c = x % (NO / 8);
        if (r < live && n0 + 8 * c < ncols)
          *reinterpret_cast<u32x4*>(outp + ((int64_t)row0 + r) * a.ldout + n0 + 8 * c) = get(NO, r, c);
      }
      if constexpr (GATED && T != Num::kInt8) {
        if (a.keep) {
          __syncthreads();
          // gate columns in the left half of the LDS rows, up in the right
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) put(BN, rowl(i), coll(j) + (j % 2 ? NO : 0), value(i, j));
          __syncthreads();
          for (int x = tid; x < BM * (BN / 8); x += THREADS) {
            const int r = x / (BN / 8), c = x % (BN / 8);
            const int up = c >= NO / 8, col = n0 + 8 * (c - up * (NO / 8));
            if (r < live && col < F)
              *reinterpret_cast<u32x4*>(a.keep + ((int64_t)row0 + r) * a.ldkeep + up * F + col) = get(BN, r, c);
          }
        }
      }
    }
  }
}

template <Num T, Pass PASS, Result RES, int BM, int BN, int WM, int WN>
void launch_tile(const ProductArgs& a, hipStream_t s) {
  const int no = RES == Result::kGated ? BN / 2 : BN;
  const int tiles_n = ((RES == Result::kGated ? a.cols / 2 : a.cols) + no - 1) / no;
  const int threads = 64 * WM * WN;
  dim3 blocks, joins;
  if (PASS == Pass::kWeightGrad) {
    const int tiles = (a.wrows + BM - 1) / BM * tiles_n;
    blocks = dim3((tiles + 7) / 8 * 8, a.groups, a.splits);  // xcd_unit deals units in rounds of 8
    joins = dim3(tiles, a.groups);
  } else {
    const int tiles = row_tile_bound(a.rows, a.groups, BM) * tiles_n;
    blocks = dim3((tiles + 7) / 8 * 8 + (a.splits > 1 ? split_units(BM, tiles, a.splits) + 8 : 0));
    joins = dim3(std::min(tiles, (BM == 256 ? 256 : 512) / 2));  // a split tile has at least two parts
  }
  product_tile_kernel<T, PASS, RES, false, BM, BN, WM, WN><<<blocks, threads, 0, s>>>(a);
  if (a.splits > 1) product_tile_kernel<T, PASS, RES, true, BM, BN, WM, WN><<<joins, threads, 0, s>>>(a);
}

// The 128 x 128 (4 waves, two blocks per compute unit) or 256 x 256 (8 waves)
// block.
template <Num T, Pass PASS, Result RES>
void launch_tiles(const ProductArgs& a, const ProductPlan& p, hipStream_t s) {
  if (p.family == Family::kTile256)
    launch_tile<T, PASS, RES, 256, 256, 2, 4>(a, s);
  else
    launch_tile<T, PASS, RES, 128, 128, 2, 2>(a, s);
}

}  // namespace moe
