// Grouped products of few rows per group: bound by reading each used group's
// weights once.
//
// A block owns 16 NC columns of one group (gated: 16 gate and the same 16 up
// columns) and up to 16 MT of the group's rows.  Its 4 waves each take a
// quarter of the contraction, in 64-byte steps (32 16-bit values, 64 codes),
// and read w straight into registers: the weights pass the compute unit once
// and nothing is reused through LDS.  kRun steps are loaded while the previous
// kRun are multiplied; a wave's steps are consecutive, so that it reads
// kilobytes of each row in turn.  The rows come from the caches in the same
// way.  The waves' sums meet in LDS and are added in wave order, so the result
// does not depend on timing.
//
// A load is 16 bytes a lane of 16 rows.  The matrix cores want row l % 16 in
// lane l, but the address unit takes four neighbouring lanes at a time, and if
// these ask for four rows it looks up four lines for 64 bytes: 16 bytes a clock
// and compute unit, which bounded blocks of more rows (64 rows x 1024 columns
// of 4096 in bf16: 21.5 us).  So four neighbours load 64 bytes of one row, and
// each fragment is exchanged between the lanes afterwards (ds_bpermute: LDS's
// crossbar, none of its memory): 14.7 us, with 16-row blocks 8.6.  Whole
// 128-byte lines (eight lanes a row, two more moves a fragment) gained 6% where
// memory is the bound (16 x 12800 of 4096: 25.1 against 26.6) and lost 10-25%
// elsewhere; 8 waves a block: 28.3 -> 29.5 at 16 x 4096 of 14336, 16 x 8192 of
// 4096: 17.0 -> 19.0.  The exchange itself costs where rows are short and groups
// many: 96 rows over 64 groups of 4096 columns of 2048 codes 50.6 -> 54.5 us,
// the one shape of those timed that lost by it.
//
// 32 rows over 8 groups of 14336 gated columns of 4096 codes: 160 us, 5.9 TB/s
// (a read-only stream reaches 6.7); 16 rows x one group of 6400 gated columns
// of 4096 in bf16: 25.8 us from memory (4.1 TB/s: 400 blocks, whose start and
// end show), 19.4 from the last-level cache.
// The non-temporal hint, which drops a line's second half before it is asked
// for, cost 15%.
#include <type_traits>

#include "product_core.h"

namespace moe {

namespace {

constexpr int kStreamWaves = 4;

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

template <Num T, Result RES, int MT, int NC>
__global__ __launch_bounds__(64 * kStreamWaves, MT == 4 ? 2 : 4) void product_stream_kernel(ProductArgs a) {
  constexpr bool GATED = RES == Result::kGated;
  static_assert(!GATED || NC == 2, "a gated block holds one gate and one up tile");
  constexpr int ES = T == Num::kInt8 ? 1 : 2;
  constexpr int NO = GATED ? 16 : 16 * NC;
  using acc_t = typename Acc<T>::t4;
  __shared__ __attribute__((aligned(16))) acc_t part[kStreamWaves][MT * NC][64];
  const int group = blockIdx.y;
  int begin, end;
  group_rows(a.offsets, a.rows, group, begin, end);
  begin = __builtin_amdgcn_readfirstlane(begin) + blockIdx.z * 16 * MT;
  end = __builtin_amdgcn_readfirstlane(end);
  if (begin >= end) return;
  const int F = a.cols / 2, ncols = GATED ? F : a.cols;
  const int n0 = blockIdx.x * NO;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, quad = lane >> 4;

  // lane l loads 16 bytes of row l / 4 of a tile, so that four neighbours ask
  // for 64 bytes in a row, and multiplies those of row l % 16
  const int lrow = lane >> 2, lbyte = 16 * (lane & 3);
  const int from = 4 * (4 * l16 + quad);  // the lane that loaded them, in bytes
  const char* wbase = a.q + (int64_t)group * a.q_group + (int64_t)n0 * a.ldq;
  __amdgpu_buffer_rsrc_t wr[NC];
  uint32_t wv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    wr[c] = buffer_at(GATED ? wbase + (c ? (int64_t)F * a.ldq : 0) : wbase);
    const int r = (GATED ? 0 : 16 * c) + lrow;
    wv[c] = n0 + r < ncols ? (uint32_t)(r * a.ldq + lbyte) : kNoLoad;
  }
  // the group's row tiles: this block's and every gridDim.z-th after it (the
  // grid has one for every tile with MT < 4, whose registers are full)
  for (bool first = true; first || (MT == 4 && begin < end); begin += gridDim.z * 16 * MT, first = false) {
    const int live = min(16 * MT, end - begin);
    if (!first) __syncthreads();  // the last tile's sums have been read
    const __amdgpu_buffer_rsrc_t xr = buffer_at(a.p + (int64_t)begin * a.ldp);
    uint32_t xv[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = 16 * m + lrow < live ? (uint32_t)((16 * m + lrow) * a.ldp + lbyte) : kNoLoad;

    acc_t acc[MT][NC];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[m][c] = acc_t{};

    const int bytes = a.contract * ES;  // of a row
    const int steps = (bytes + 63) / 64;
    // the row tiles in use are a compile-time count, so that the loop holds no branches
    auto body = [&](auto tag) {
      constexpr int ML = decltype(tag)::value;
      constexpr int kRun = ML == 1 && NC == 1 ? 4 : 2;  // steps loaded together, as the registers allow
      // this wave's steps [s, s1): contiguous, so that a wave reads long runs of
      // each row
      const int s1 = (int)((int64_t)steps * (wave + 1) / kStreamWaves);
      int s = (int)((int64_t)steps * wave / kStreamWaves);
      u32x4 w[2][kRun][NC], x[2][kRun][ML];
      auto load = [&](int b, int at) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
          const bool in = (at + u) * 64 + lbyte < bytes && at + u < s1;  // bytes: a multiple of 16
#pragma unroll
          for (int c = 0; c < NC; ++c) w[b][u][c] = load16(wr[c], in ? wv[c] : kNoLoad, (uint32_t)(at + u) * 64);
#pragma unroll
          for (int m = 0; m < ML; ++m) x[b][u][m] = load16(xr, in ? xv[m] : kNoLoad, (uint32_t)(at + u) * 64);
        }
      };
      auto fragment = [&](u32x4 v) {
        u32x4 f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __builtin_amdgcn_ds_bpermute(from, v[e]);
        return f;
      };
      auto multiply = [&](int b) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
          u32x4 wf[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) wf[c] = fragment(w[b][u][c]);
#pragma unroll
          for (int m = 0; m < ML; ++m) {
            const u32x4 xf = fragment(x[b][u][m]);
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[m][c] = mfma16x16<T>(wf[c], xf, acc[m][c]);
          }
        }
      };
      if (s < s1) load(0, s);
      while (s < s1) {
        if (s + kRun < s1) load(1, s + kRun);
        multiply(0);
        s += kRun;
        if (s >= s1) break;
        if (s + kRun < s1) load(0, s + kRun);
        multiply(1);
        s += kRun;
      }
    };
    const int tiles = (live + 15) / 16;
    if (MT == 1 || tiles == 1)
      body(std::integral_constant<int, 1>{});
    else if (MT == 2 || tiles == 2)
      body(std::integral_constant<int, MT < 2 ? 1 : 2>{});
    else
      body(std::integral_constant<int, MT>{});

#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) part[wave][m * NC + c][lane] = acc[m][c];
    __syncthreads();

    // lane l of tile (m, c): row 16m + l % 16, columns 16c + 4 (l / 16) ..
    const bool fp16 = T == Num::kFp16 || (T == Num::kInt8 && a.out_type == MOE_TYPE_FP16);
    constexpr int kTiles = GATED ? MT : MT * NC;  // result tiles
    for (int tile = wave; tile < kTiles; tile += kStreamWaves) {
      const int m = GATED ? tile : tile / NC, c = GATED ? 0 : tile % NC;
      const int row = 16 * m + l16, col = n0 + 16 * c + 4 * quad;
      if (row >= live || col >= ncols) continue;
      auto total = [&](int t, int up) -> f32x4 {
        acc_t v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < kStreamWaves; ++w) v += part[w][t][lane];
        f32x4 f;
        if constexpr (T == Num::kInt8) {
          const float ps = a.pscale[begin + row];
          const f32x4 s = *reinterpret_cast<const f32x4*>(a.qscale + (int64_t)group * a.cols + (up ? F : 0) + col);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = (float)v[e] * ps * s[e];
        } else {
          f = v;
        }
        return f;
      };
      f32x4 v = total(GATED ? m * NC : tile, 0);
      if constexpr (RES == Result::kWide) {
        *reinterpret_cast<f32x4*>((float*)a.out + (int64_t)(begin + row) * a.ldout + col) = v;
      } else {
        if constexpr (GATED) {
          const f32x4 u = total(m * NC + 1, 1);
          if (T != Num::kInt8 && a.keep) {
            uint16_t* k = a.keep + (int64_t)(begin + row) * a.ldkeep + col;
            *reinterpret_cast<u32x2*>(k) = u32x2{pack_half(fp16, v[0], v[1]), pack_half(fp16, v[2], v[3])};
            *reinterpret_cast<u32x2*>(k + F) = u32x2{pack_half(fp16, u[0], u[1]), pack_half(fp16, u[2], u[3])};
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]) * u[e];
        }
        *reinterpret_cast<u32x2*>((uint16_t*)a.out + (int64_t)(begin + row) * a.ldout + col) =
            u32x2{pack_half(fp16, v[0], v[1]), pack_half(fp16, v[2], v[3])};
      }
    }
  }
}

// Blocks of `no` columns and 16 mt rows that have rows, at least: the offsets
// are on the device.
int64_t live_blocks(const ProductArgs& a, int ncols, int no, int mt) {
  return (int64_t)((ncols + no - 1) / no) * std::max(a.groups, (a.rows + 16 * mt - 1) / (16 * mt));
}

// 64 rows x 256 columns of 4096 in bf16: blocks of 16 rows 8.1 us, of 64 14.5;
// 64 x 2048 (256 blocks of 32 rows): 11.2 against 11.5 with 512 of 16; 64 x
// 6400 (200 blocks of 64 rows and 32 columns): 24.4 against 25.9 with 32 rows.
constexpr int kFullChip = 256;
template <Num T, Result RES, int NC>
void launch_mt(const ProductArgs& a, hipStream_t s) {
  const int ncols = RES == Result::kGated ? a.cols / 2 : a.cols;
  const int no = RES == Result::kGated ? 16 : 16 * NC;
  // row tiles of 16 of the largest possible group, up to 4 a block; fewer while
  // that leaves compute units idle
  int mt = a.rows <= 16 ? 1 : a.rows <= 32 ? 2 : 4;
  while (mt > 1 && live_blocks(a, ncols, no, mt / 2) <= kFullChip) mt /= 2;
  // a block for every row tile that a group might have; of the high blocks,
  // which walk on over a group's tiles, four for each of an average group:
  // blocks beyond a group's rows cost 0.7 ns each (1024 rows over 64 groups of
  // 2048 gated columns of 4096, codes: 225 us with all of them, 203 without)
  int tiles = (a.rows + 16 * mt - 1) / (16 * mt);
  if (mt == 4 && a.groups > 1) tiles = std::min(tiles, 2 + 4 * tiles / a.groups);
  const dim3 grid((ncols + no - 1) / no, a.groups, tiles);
  const int threads = 64 * kStreamWaves;
  if (mt == 1)
    product_stream_kernel<T, RES, 1, NC><<<grid, threads, 0, s>>>(a);
  else if (mt == 2)
    product_stream_kernel<T, RES, 2, NC><<<grid, threads, 0, s>>>(a);
  else
    product_stream_kernel<T, RES, 4, NC><<<grid, threads, 0, s>>>(a);
}

// A block of 32 columns reads the rows half as often, one of 16 makes twice as
// many blocks.  With more than 4 rows a group and blocks for most compute units
// the wide ones win: 64 rows x 4096 columns of 4096 in bf16: 13.9 against 15.8
// us; 128 x 4096 codes of 4096: 12.0 against 15.6; 16 x 12800: 26.6 against
// 28.8; 256 over 16 groups of 4096 columns of 2048: 54.8 against 58.7.  16 x
// 4096 of 14336 (128 blocks): 40.5 against 29.1; 64 x 1024 of 4096 (128): 10.7
// against 8.6.
constexpr int kWideBlocks = 192, kWideRows = 4;
template <Num T, Result RES>
void launch_stream(const ProductArgs& a, hipStream_t s) {
  if constexpr (RES == Result::kGated)
    launch_mt<T, RES, 2>(a, s);
  else if (live_blocks(a, a.cols, 32, 1) >= kWideBlocks && a.rows > kWideRows * a.groups)
    launch_mt<T, RES, 2>(a, s);
  else
    launch_mt<T, RES, 1>(a, s);
}

}  // namespace

void launch_product_stream(const ProductArgs& a, Num num, Result res, hipStream_t s) {
  if (num == Num::kInt8) {
    if (res == Result::kGated)
      launch_stream<Num::kInt8, Result::kGated>(a, s);
    else if (res == Result::kWide)
      launch_stream<Num::kInt8, Result::kWide>(a, s);
    else
      launch_stream<Num::kInt8, Result::kHalf>(a, s);
  } else if (num == Num::kFp16) {
    if (res == Result::kGated)
      launch_stream<Num::kFp16, Result::kGated>(a, s);
    else
      launch_stream<Num::kFp16, Result::kHalf>(a, s);
  } else {
    if (res == Result::kGated)
      launch_stream<Num::kBf16, Result::kGated>(a, s);
    else
      launch_stream<Num::kBf16, Result::kHalf>(a, s);
  }
}

}  // namespace moe
