// Device code shared by the grouped products: element conversions, the
// activations, the lookup of a block's group and rows, and the LDS-tiled
// matrix-core kernel.
#pragma once

#include <algorithm>

#include "device_common.h"
#include "products.h"

namespace moe {

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_any;
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <Num T> struct Acc { using t16 = f32x16; using t4 = f32x4; using t1 = float; };
template <> struct Acc<Num::kInt8> { using t16 = i32x16; using t4 = i32x4; using t1 = int; };

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
// keeps its precision as far down as fp32 goes.
constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;
constexpr float kLift = 0x1p64f, kDrop = 0x1p-64f;
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

// 32 x 32 of A (lane l: row l % 32, 16 bytes of the contraction at 16 (l / 32))
// times B (the same for its columns): D holds column l % 32, rows
// 8 (i / 4) + 4 (l / 32) + i % 4 in element i.
template <Num T>
__device__ __forceinline__ typename Acc<T>::t16 mfma32x32(u32x4 a, u32x4 b, typename Acc<T>::t16 c) {
  if constexpr (T == Num::kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else if constexpr (T == Num::kFp16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
// The same at 16 x 16 (lane l: row l % 16, 16 bytes at 16 (l / 16)): D holds
// column l % 16, rows 4 (l / 16) + i.
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
    const int cost = BM == 256 ? 6 + r.rem * s / 8 : 6 + r.rem * s / 32;  // in stages
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
// grid of 32 x 32 matrix-core tiles.  The contraction is walked in stages of
// 128 bytes a row (64 16-bit values, 128 codes) through two LDS buffers filled
// by direct global -> LDS copies.  An operand comes in one of two layouts:
//  - contraction contiguous in memory (x, codes, w in the forward product):
//    LDS rows of 128 bytes, 16-byte chunks swizzled by the row so that the 16
//    rows of one read cycle fall on different banks;
//  - contraction across the rows (w in the input gradient; dy and x in the
//    weight gradient): LDS holds 64 rows of BM (or BN) values and the
//    transposing LDS read hands each lane 4 consecutive contraction values of
//    its column; chunks are swizzled by row % 4, the 4 rows that one read
//    cycle covers.  No operand is ever transposed in memory.
// In the last of a stage's four steps the block waits for the next stage's
// copies, refills the buffer just read and reads the next stage's first
// fragments before the step's products, which hide the LDS latency behind the
// barrier.  Missing rows, columns and the contraction's tail are zeros (out of
// range buffer loads), so they add nothing to the sums.
//
// The matrix cores take Q's values as A and P's as B: a lane then holds four
// consecutive columns of one result row.  16-bit results go through LDS and
// leave as whole rows of 16-byte stores; fp32 ones leave from registers.
//
// Gated: the block's columns are BN/2 gate and the same BN/2 up columns,
// interleaved by 32 so that a wave holds g and u of the same elements.
//
// JOIN: the block adds the raw sums of a split tile's parts, in order, instead
// of computing them, and writes the result.
template <Num T, Pass PASS, Result RES, bool JOIN, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_tile_kernel(ProductArgs a) {
  constexpr int NW = WM * WN, THREADS = 64 * NW;
  constexpr int MI = BM / 32 / WM, NJ = BN / 32 / WN;
  constexpr bool P_STR = PASS == Pass::kWeightGrad, Q_STR = PASS != Pass::kForward;
  constexpr bool GATED = RES == Result::kGated;
  constexpr int ES = T == Num::kInt8 ? 1 : 2;
  constexpr int BK = 128 / ES;  // contraction values per stage
  constexpr int kPBytes = BM * 128, kQBytes = BN * 128, kStage = kPBytes + kQBytes;
  constexpr int PI = kPBytes / 1024 / NW, QI = kQBytes / 1024 / NW;  // 1 KB copies per wave and stage
  constexpr int NO = GATED ? BN / 2 : BN;                            // result columns per block
  static_assert(PI * NW * 1024 == kPBytes && QI * NW * 1024 == kQBytes, "even copy split");
  static_assert(!GATED || (QI == 4 && NJ % 2 == 0), "a wave's copies of W lie in one block of 32 rows");
  static_assert(T != Num::kInt8 || PASS == Pass::kForward, "codes have no backward pass");
  using acc_t = typename Acc<T>::t16;
  __shared__ __attribute__((aligned(1024))) char smem_raw[2 * kStage];
  lds_char* smem = (lds_char*)smem_raw;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l32 = lane & 31, hh = lane >> 5;
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
    const int tiles_m = (a.wrows + BM - 1) / BM, tiles = tiles_m * tiles_n, padded = (tiles + 7) / 8 * 8;
    const int b = blockIdx.x;
    const int in = JOIN ? b % tiles : xcd_unit(b % padded, tiles);
    if (in < 0) return;
    group = (JOIN ? b / tiles : b / padded) % a.groups;
    parts = a.splits;
    part = JOIN ? 0 : b / (padded * a.groups);
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
  const int st0 = (int)((int64_t)stages * part / parts), st1 = (int)((int64_t)stages * (part + 1) / parts);
  // raw sums of a part: every lane's, 16 bytes each
  auto raw = [&](int at, int i, int j, int q) {
    using t4 = typename Acc<T>::t4;
    return reinterpret_cast<t4*>(a.partial + (int64_t)at * (BM * BN * 4)) +
           (((wave * MI + i) * NJ + j) * 4 + q) * 64 + lane;
  };

  acc_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = acc_t{};
  if constexpr (JOIN) {
    for (int s = 0; s < parts; ++s)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const typename Acc<T>::t4 v = *raw(slot + s * slot_step, i, j, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
          }
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
  // gated: this wave copies 32 W rows, all gate or all up
  const int qhalf = GATED ? (wave % NJ) % 2 : 0;
  if (GATED && qhalf) qbase += (int64_t)F * a.ldq;
  uint32_t pv[PI], qv[QI];  // byte offsets of this lane's copies in stage 0, or kNoLoad
  int pk[PI], qk[QI];       // their contraction position: first value (contiguous) or row (strided)
  auto place = [&](bool strided, int j, int per_wave, int width, int64_t ld, int limit, bool gated, uint32_t& v, int& k) {
    const int inst = wave * per_wave + j;
    if (strided) {
      const int cpr = width / 8;  // 16-byte chunks per LDS row
      const int kr = inst * (64 / cpr) + lane / cpr;
      const int c = (lane % cpr) ^ ((kr & 3) << 2);
      v = 8 * c < limit ? (uint32_t)(kr * ld + 16 * c) : kNoLoad;
      k = kr;
    } else {
      const int r = inst * 8 + lane / 8;
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      int src = r;
      if (gated) {  // LDS row r: block r / 32 belongs to wave column (r / 32) / NJ
        const int jb = r / 32;
        src = (jb / NJ * (NJ / 2) + jb % NJ / 2) * 32 + r % 32;
      }
      v = src < limit ? (uint32_t)(src * ld + 16 * c) : kNoLoad;
      k = c * (16 / ES);
    }
  };
#pragma unroll
  for (int j = 0; j < PI; ++j) place(P_STR, j, PI, BM, a.ldp, live, false, pv[j], pk[j]);
#pragma unroll
  for (int j = 0; j < QI; ++j) place(Q_STR, j, QI, BN, a.ldq, ncols - n0, GATED, qv[j], qk[j]);
  auto issue = [&](int st, int buf) {
    lds_char* dst = smem + buf * kStage;
    const int left = klen - st * BK;  // contraction values from this stage on
    const __amdgpu_buffer_rsrc_t pr = buffer_at(P_STR ? pbase + (int64_t)st * BK * a.ldp : pbase + (int64_t)st * 128);
    const __amdgpu_buffer_rsrc_t qr = buffer_at(Q_STR ? qbase + (int64_t)st * BK * a.ldq : qbase + (int64_t)st * 128);
    if (left >= BK) {
#pragma unroll
      for (int j = 0; j < PI; ++j) buffer_to_lds16(pr, dst + (wave * PI + j) * 1024, pv[j], 0);
#pragma unroll
      for (int j = 0; j < QI; ++j) buffer_to_lds16(qr, dst + kPBytes + (wave * QI + j) * 1024, qv[j], 0);
    } else {
#pragma unroll
      for (int j = 0; j < PI; ++j)
        buffer_to_lds16(pr, dst + (wave * PI + j) * 1024, pk[j] < left ? pv[j] : kNoLoad, 0);
#pragma unroll
      for (int j = 0; j < QI; ++j)
        buffer_to_lds16(qr, dst + kPBytes + (wave * QI + j) * 1024, qk[j] < left ? qv[j] : kNoLoad, 0);
    }
  };

  // ---- fragments ----
  // contiguous: lane l reads chunk 2s + hh of row (block row) + l % 32
  const int row_at = l32 * 128, chunk_sw = (l32 >> 1) & 7;
  // strided: lane 16g + j reads, for columns 16 (g % 2) + 4 (j % 4) .., row
  // 16s + 8 (g / 2) + 4t + j / 4 (t = 0, 1)
  const int sj = lane & 15, sg = lane >> 4;
  auto strided_at = [&](int width, int block) {
    return (8 * (sg >> 1) + (sj >> 2)) * width * 2 + 64 * (block ^ (sj >> 2)) + 32 * (sg & 1) + 8 * (sj & 3);
  };
  int pat[MI], qat[NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i) pat[i] = P_STR ? strided_at(BM, wm * MI + i) : (wm * MI + i) * 4096 + row_at;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    qat[j] = kPBytes + (Q_STR ? strided_at(BN, wn * NJ + j) : (wn * NJ + j) * 4096 + row_at);
  auto fragment = [&](bool strided, int width, lds_char* at, int s) -> u32x4 {
    if (strided) {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      lds_char* q = at + s * 16 * width * 2;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)q));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(q + 8 * width)));
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    }
    return *(__attribute__((address_space(3))) u32x4*)(at + 16 * ((2 * s + hh) ^ chunk_sw));
  };
  auto read_step = [&](int buf, int s, u32x4(&pf)[MI], u32x4(&qf)[NJ]) {
    lds_char* b = smem + buf * kStage;
#pragma unroll
    for (int j = 0; j < NJ; ++j) qf[j] = fragment(Q_STR, BN, b + qat[j], s);
#pragma unroll
    for (int i = 0; i < MI; ++i) pf[i] = fragment(P_STR, BM, b + pat[i], s);
  };

  auto products = [&](u32x4(&pf)[MI], u32x4(&qf)[NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mfma32x32<T>(qf[j], pf[i], acc[i][j]);
  };

  const int nst = st1 - st0;
  const bool busy = wm * MI * 32 < live;  // this wave has rows
  if (nst > 0) {
    issue(st0, 0);
    wait_copies<0>();
    lds_only_barrier();
    if (nst > 1) issue(st0 + 1, 1);
    u32x4 pf[2][MI], qf[2][NJ];
    if (busy) {
      read_step(0, 0, pf[0], qf[0]);
      for (int i = 0; i < nst; ++i) {
        const int buf = i & 1;
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          read_step(buf, s + 1, pf[(s + 1) & 1], qf[(s + 1) & 1]);
          products(pf[s & 1], qf[s & 1]);
        }
        if (i + 1 < nst) {
          wait_copies<0>();
          lds_only_barrier();
          if (i + 2 < nst) issue(st0 + i + 2, buf);
          read_step(buf ^ 1, 0, pf[0], qf[0]);
        }
        products(pf[1], qf[1]);
      }
    } else {
      // a wave without rows only copies
      for (int i = 0; i + 1 < nst; ++i) {
        wait_copies<0>();
        lds_only_barrier();
        if (i + 2 < nst) issue(st0 + i + 2, i & 1);
      }
    }
  }

  if (parts > 1) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *raw(slot, i, j, q) = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    return;
  }
  }  // !JOIN

  // ---- results ----
  // element e of acc[i][j]: row rowl(i), column coll(j) + 8 (e / 4) + e % 4
  auto rowl = [&](int i) { return (wm * MI + i) * 32 + l32; };
  auto coll = [&](int j) {
    return (GATED ? (wn * (NJ / 2) + j / 2) * 32 : (wn * NJ + j) * 32) + 4 * hh;
  };
  {
    const bool fp16 = T == Num::kFp16 || (T == Num::kInt8 && a.out_type == MOE_TYPE_FP16);
    // codes: the sum times the row's and the column's scale
    float prow[MI];
    if constexpr (T == Num::kInt8) {
#pragma unroll
      for (int i = 0; i < MI; ++i) prow[i] = rowl(i) < live ? a.pscale[row0 + rowl(i)] : 0.0f;
    }
    const float* qs = T == Num::kInt8 ? a.qscale + (int64_t)group * a.cols : nullptr;
    auto value = [&](int i, int j, int q) -> f32x4 {
      f32x4 v;
      if constexpr (T == Num::kInt8) {
        const int c = n0 + coll(j) + 8 * q;
        const f32x4 s = c < ncols ? *reinterpret_cast<const f32x4*>(qs + c + (GATED && j % 2 ? F : 0)) : f32x4{};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][4 * q + e] * prow[i] * s[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
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
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = n0 + coll(j) + 8 * q;
            if (c < ncols) *reinterpret_cast<f32x4*>(rowp + (int64_t)c * 4) = value(i, j, q);
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
        for (int j = 0; j < NJ; j += GATED ? 2 : 1)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4 v = value(i, j, q);
            if constexpr (GATED) {
              const f32x4 u = value(i, j + 1, q);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]) * u[e];
            }
            put(NO, rowl(i), coll(j) + 8 * q, v);
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
            for (int j = 0; j < NJ; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) put(BN, rowl(i), coll(j) + 8 * q + (j % 2 ? NO : 0), value(i, j, q));
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
  int blocks, joins;
  if (PASS == Pass::kWeightGrad) {
    const int tiles = (a.wrows + BM - 1) / BM * tiles_n;
    blocks = a.splits * a.groups * ((tiles + 7) / 8 * 8);  // xcd_unit deals units in rounds of 8
    joins = a.groups * tiles;
  } else {
    const int tiles = row_tile_bound(a.rows, a.groups, BM) * tiles_n;
    blocks = (tiles + 7) / 8 * 8 + (a.splits > 1 ? split_units(BM, tiles, a.splits) + 8 : 0);
    joins = std::min(tiles, (BM == 256 ? 256 : 512) / 2);  // a split tile has at least two parts
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
