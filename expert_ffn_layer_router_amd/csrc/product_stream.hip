// Grouped products of few rows (up to 64 in the call): bound by reading each
// used group's weights once.
//
// A block owns 16 NC columns of one group (gated: 16 gate and the same 16 up
// columns) and all of the group's rows, in up to MT tiles of 16.  Its 8 waves
// take the contraction's 64-byte steps (32 16-bit values, 64 codes) in runs of
// kRun, dealt round-robin, and read w straight into registers: the weights
// pass the compute unit once and nothing is reused through LDS.  kRun steps
// of loads are in flight per wave while the previous ones are multiplied.
// The rows come from the caches in the same fragment layout.  The waves' sums
// meet in LDS and are added in wave order, so the result does not depend on
// timing.
#include <type_traits>

#include "product_core.h"

namespace moe {

namespace {

constexpr int kStreamWaves = 8;
constexpr int kRun = 4;  // 64-byte steps in flight per wave

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

template <Num T, Result RES, int MT, int NC>
__global__ __launch_bounds__(64 * kStreamWaves, MT >= 4 ? 2 : 4) void product_stream_kernel(ProductArgs a) {
  constexpr bool GATED = RES == Result::kGated;
  static_assert(!GATED || NC == 2, "a gated block holds one gate and one up tile");
  constexpr int ES = T == Num::kInt8 ? 1 : 2;
  constexpr int NO = GATED ? 16 : 16 * NC;
  using acc_t = typename Acc<T>::t4;
  __shared__ __attribute__((aligned(16))) acc_t part[kStreamWaves][MT * NC][64];
  const int group = blockIdx.y;
  int begin, end;
  group_rows(a.offsets, a.rows, group, begin, end);
  const int live = __builtin_amdgcn_readfirstlane(end - begin);
  if (live <= 0) return;
  begin = __builtin_amdgcn_readfirstlane(begin);
  const int F = a.cols / 2, ncols = GATED ? F : a.cols;
  const int n0 = blockIdx.x * NO;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, quad = lane >> 4;

  const char* wbase = a.q + (int64_t)group * a.q_group + (int64_t)n0 * a.ldq;
  __amdgpu_buffer_rsrc_t wr[NC];
  uint32_t wv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    wr[c] = buffer_at(GATED ? wbase + (c ? (int64_t)F * a.ldq : 0) : wbase);
    const int r = (GATED ? 0 : 16 * c) + l16;
    wv[c] = n0 + r < ncols ? (uint32_t)(r * a.ldq + 16 * quad) : kNoLoad;
  }
  const __amdgpu_buffer_rsrc_t xr = buffer_at(a.p + (int64_t)begin * a.ldp);
  uint32_t xv[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xv[m] = 16 * m + l16 < live ? (uint32_t)((16 * m + l16) * a.ldp + 16 * quad) : kNoLoad;

  acc_t acc[MT][NC];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[m][c] = acc_t{};

  const int bytes = a.contract * ES;  // of a row; a multiple of 16
  const int steps = (bytes + 63) / 64;
  // the row tiles in use are a compile-time count, so that the loop holds no branches
  auto body = [&](auto tag) {
    constexpr int ML = decltype(tag)::value;
    u32x4 w0[kRun][NC], x0[kRun][ML];
    for (int s0 = wave * kRun; s0 < steps; s0 += kStreamWaves * kRun) {
      const uint32_t at = (uint32_t)s0 * 64;
      const bool whole = s0 * 64 + kRun * 64 <= bytes;
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        const bool in = whole || s0 * 64 + u * 64 + 16 * quad < bytes;
#pragma unroll
        for (int c = 0; c < NC; ++c) w0[u][c] = load16(wr[c], in ? wv[c] : kNoLoad, at + u * 64);
#pragma unroll
        for (int m = 0; m < ML; ++m) x0[u][m] = load16(xr, in ? xv[m] : kNoLoad, at + u * 64);
      }
#pragma unroll
      for (int u = 0; u < kRun; ++u)
#pragma unroll
        for (int m = 0; m < ML; ++m)
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[m][c] = mfma16x16<T>(w0[u][c], x0[u][m], acc[m][c]);
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
  if (wave >= kTiles) return;
  static_assert(kTiles <= kStreamWaves, "one wave per result tile");
  const int m = GATED ? wave : wave / NC, c = GATED ? 0 : wave % NC;
  const int row = 16 * m + l16, col = n0 + 16 * c + 4 * quad;
  if (row >= live || col >= ncols) return;
  auto total = [&](int tile, int up) -> f32x4 {
    acc_t v = part[0][tile][lane];
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w) v += part[w][tile][lane];
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
  if constexpr (RES == Result::kWide) {
    *reinterpret_cast<f32x4*>((float*)a.out + (int64_t)(begin + row) * a.ldout + col) = total(wave, 0);
  } else {
    f32x4 v = total(GATED ? m * NC : wave, 0);
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

template <Num T, Result RES, int NC>
void launch_mt(const ProductArgs& a, hipStream_t s) {
  const int ncols = RES == Result::kGated ? a.cols / 2 : a.cols;
  const int no = RES == Result::kGated ? 16 : 16 * NC;
  const dim3 grid((ncols + no - 1) / no, a.groups);
  const int threads = 64 * kStreamWaves;
  if (a.rows <= 16)
    product_stream_kernel<T, RES, 1, NC><<<grid, threads, 0, s>>>(a);
  else if (a.rows <= 32)
    product_stream_kernel<T, RES, 2, NC><<<grid, threads, 0, s>>>(a);
  else
    product_stream_kernel<T, RES, 4, NC><<<grid, threads, 0, s>>>(a);
}

template <Num T, Result RES>
void launch_stream(const ProductArgs& a, hipStream_t s) {
  if constexpr (RES == Result::kGated)
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
