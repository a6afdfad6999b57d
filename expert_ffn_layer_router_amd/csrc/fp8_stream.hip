// Products of e4m3 codes with few rows per group: bound by reading each used
// group's weights once.
//
// As the streaming products of integer codes: a block owns 16 NC columns of one
// group (gated: 16 gate and the same 16 up columns) and up to 16 MT of its
// rows, its 4 waves a quarter of the contraction each, here in whole blocks of
// 128, whose products are scaled as they come from the matrix cores.  Weights
// and rows go straight to registers, four neighbouring lanes loading 64 bytes
// of one row, and are exchanged between the lanes afterwards.  The waves' sums
// meet in LDS and are added in wave order.
//
// Measured: 32 rows over 8 groups, gated, 14336 of 4096 (0.94 GB of weights) 165
// us, 5.7 TB/s (a read-only stream of that size: 5.15; an 8-bit integer product
// 162 us); one row, 4096 of 2048, 4.2 us, the launch itself about 2.5.  No gain:
// two blocks of 128 at a time before the exchange; lanes loading whole lines of
// 128 bytes; 8 waves a block (64 groups of one row 100 -> 163 us, too few blocks
// on a unit).
#include <type_traits>

#include "fp8_device.h"

namespace moe {

namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

template <Result RES, int MT, int NC>
__global__ __launch_bounds__(64 * kWaves, MT == 4 ? 2 : MT * NC == 4 ? 3 : 4) void fp8_stream_kernel(Fp8Args a) {
  constexpr bool GATED = RES == Result::kGated;
  static_assert(!GATED || NC == 2, "a gated block holds one gate and one up tile");
  constexpr int NO = GATED ? 16 : 16 * NC;
  __shared__ __attribute__((aligned(16))) f32x4 part[kWaves][MT * NC][64];
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

  // lane l loads 16 bytes of row l / 4 of a tile and multiplies those of row l % 16
  const int lrow = lane >> 2, lbyte = 16 * (lane & 3);
  const int from = 4 * (4 * l16 + quad);  // the lane that loaded them, in bytes
  const char* wbase = a.q + (int64_t)group * a.q_group + (int64_t)n0 * a.ldq;
  const float* sbase = a.qscale + (int64_t)group * a.qs_group;
  __amdgpu_buffer_rsrc_t wr[NC];
  uint32_t wv[NC];
  const float* wsp[NC];  // the tile's scales (NO divides the block of 128, so a tile has one row of them)
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    wr[c] = buffer_at(GATED ? wbase + (c ? (int64_t)F * a.ldq : 0) : wbase);
    const int r = (GATED ? 0 : 16 * c) + lrow;
    wv[c] = n0 + r < ncols ? (uint32_t)(r * a.ldq + lbyte) : kNoLoad;
    // a tile past the last column takes the first one's: its products are zero and not stored
    const int col = GATED || n0 + 16 * c >= ncols ? n0 : n0 + 16 * c;
    wsp[c] = sbase + (GATED ? c * a.qs_half : 0) + (int64_t)(col / kScaleBlock) * a.qs_cols;
  }
  for (bool first = true; first || (MT == 4 && begin < end); begin += gridDim.z * 16 * MT, first = false) {
    const int live = min(16 * MT, end - begin);
    if (!first) __syncthreads();  // the last tile's sums have been read
    const __amdgpu_buffer_rsrc_t xr = buffer_at(a.p + (int64_t)begin * a.ldp);
    uint32_t xv[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = 16 * m + lrow < live ? (uint32_t)((16 * m + lrow) * a.ldp + lbyte) : kNoLoad;

    f32x4 acc[MT][NC];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[m][c] = f32x4{};

    const int bytes = a.contract;  // of a row
    const int blocks = (bytes + kScaleBlock - 1) / kScaleBlock;
    // the row tiles in use are a compile-time count, so that the loop holds no branches
    auto body = [&](auto tag) {
      constexpr int ML = decltype(tag)::value;
      constexpr int kRun = ML == 1 && NC == 1 ? 2 : 1;  // blocks loaded together, as the registers allow
      // this wave's blocks [s, s1)
      const int s1 = blocks * (wave + 1) / kWaves;
      int s = blocks * wave / kWaves;
      u32x4 w[2][kRun][NC][2], x[2][kRun][ML][2];
      float ws[2][kRun][NC], xs[2][kRun][ML];
      auto load = [&](int b, int at) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
          const int blk = at + u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t byte = (uint32_t)blk * kScaleBlock + 64 * h;
            const bool in = (int)byte + lbyte < bytes && blk < s1;  // bytes: a multiple of 16
#pragma unroll
            for (int c = 0; c < NC; ++c) w[b][u][c][h] = load16(wr[c], in ? wv[c] : kNoLoad, byte);
#pragma unroll
            for (int m = 0; m < ML; ++m) x[b][u][m][h] = load16(xr, in ? xv[m] : kNoLoad, byte);
          }
          const int sb = min(blk, s1 - 1);
          const __amdgpu_buffer_rsrc_t r = scales_at(a.pscale + (int64_t)sb * a.ldscale + begin, live);
#pragma unroll
          for (int m = 0; m < ML; ++m) xs[b][u][m] = load_scale(r, (16 * m + l16) * 4);
#pragma unroll
          for (int c = 0; c < NC; ++c) ws[b][u][c] = wsp[c][sb];
        }
      };
      auto fragment = [&](const u32x4* v) {
        u32x4 f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) f[h][e] = __builtin_amdgcn_ds_bpermute(from, v[h][e]);
        return join_halves(f[0], f[1]);
      };
      auto multiply = [&](int b, int at) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
          if (kRun > 1 && at + u >= s1) break;
          i32x8 wf[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) wf[c] = fragment(w[b][u][c]);
#pragma unroll
          for (int m = 0; m < ML; ++m) {
            const i32x8 xf = fragment(x[b][u][m]);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const f32x4 d = block_product(wf[c], xf);
              const float f = xs[b][u][m] * ws[b][u][c];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[m][c][e] = fmaf(d[e], f, acc[m][c][e]);
            }
          }
        }
      };
      if (s < s1) load(0, s);
      while (s < s1) {
        if (s + kRun < s1) load(1, s + kRun);
        multiply(0, s);
        s += kRun;
        if (s >= s1) break;
        if (s + kRun < s1) load(0, s + kRun);
        multiply(1, s);
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
    const bool fp16 = a.out_type == MOE_TYPE_FP16;
    constexpr int kTiles = GATED ? MT : MT * NC;  // result tiles
    for (int tile = wave; tile < kTiles; tile += kWaves) {
      const int m = GATED ? tile : tile / NC, c = GATED ? 0 : tile % NC;
      const int row = 16 * m + l16, col = n0 + 16 * c + 4 * quad;
      if (row >= live || col >= ncols) continue;
      auto total = [&](int t) {
        f32x4 v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += part[w][t][lane];
        return v;
      };
      f32x4 v = total(GATED ? m * NC : tile);
      {
        if constexpr (GATED) {
          const f32x4 u = total(m * NC + 1);
          if (a.keep) {
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
int64_t live_blocks(const Fp8Args& a, int ncols, int no, int mt) {
  return (int64_t)((ncols + no - 1) / no) * std::max(a.groups, (a.rows + 16 * mt - 1) / (16 * mt));
}

// (the rules of the integer codes' streaming kernel, product_stream.hip, where both
// sides' times stand)
constexpr int kFullChip = 256;
template <Result RES, int NC>
void launch_mt8(const Fp8Args& a, hipStream_t s) {
  const int ncols = RES == Result::kGated ? a.cols / 2 : a.cols;
  const int no = RES == Result::kGated ? 16 : 16 * NC;
  int mt = a.rows <= 16 ? 1 : a.rows <= 32 ? 2 : 4;
  while (mt > 1 && live_blocks(a, ncols, no, mt / 2) <= kFullChip) mt /= 2;
  int tiles = (a.rows + 16 * mt - 1) / (16 * mt);
  if (mt == 4 && a.groups > 1) tiles = std::min(tiles, 2 + 4 * tiles / a.groups);
  const dim3 grid((ncols + no - 1) / no, a.groups, tiles);
  const int threads = 64 * kWaves;
  if (mt == 1)
    fp8_stream_kernel<RES, 1, NC><<<grid, threads, 0, s>>>(a);
  else if (mt == 2)
    fp8_stream_kernel<RES, 2, NC><<<grid, threads, 0, s>>>(a);
  else
    fp8_stream_kernel<RES, 4, NC><<<grid, threads, 0, s>>>(a);
}

constexpr int kWideBlocks = 192, kWideRows = 4;
template <Result RES>
void launch_nc8(const Fp8Args& a, hipStream_t s) {
  if constexpr (RES == Result::kGated)
    launch_mt8<RES, 2>(a, s);
  else if (live_blocks(a, a.cols, 32, 1) >= kWideBlocks && a.rows > kWideRows * a.groups)
    launch_mt8<RES, 2>(a, s);
  else
    launch_mt8<RES, 1>(a, s);
}

}  // namespace

void launch_fp8_stream(const Fp8Args& a, Result res, hipStream_t s) {
  if (res == Result::kGated)
    launch_nc8<Result::kGated>(a, s);
  else
    launch_nc8<Result::kHalf>(a, s);
}

}  // namespace moe
