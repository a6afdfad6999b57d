// Values into e4m3 codes with a scale for each block of 128: rows, weights, and
// the gated block's slopes.
//
// A block's scale is s = a / 448 with a its largest magnitude, its codes the
// exact quotients 448 x / a rounded to e4m3.  With both scaled by a power of two
// so that a is in [1/2, 1), p = 448 x is exact in fp32 (a 16-bit float has at
// most 11 significant bits and 448 three), r = RN(1/a), q0 = RN(p r), and
// q0 + (p - q0 a) r, whose remainder is exact by FMA, is the correctly rounded
// quotient (Markstein's division).  Rounding that to e4m3 equals rounding the
// exact quotient: unless the quotient is a tie, which fp32 holds exactly, it is
// relatively further than 2^-16 from one (a tie has 5 significant bits and the
// quotient's denominator 11), the fp32 one's error 2^-24.
//
// Sixteen lanes hold a block, 8 values each, so its largest magnitude takes four
// steps within a row of lanes.
//
// All three kernels are bound by memory: rows 8192 x 14336 take 66 to 80 us (4.5
// to 5.4 TB/s, by how much of them the last-level cache still holds), 16 matrices
// of 14336 x 4096 528 us (5.3 TB/s; a copy 4.9), the slopes of 4096 x 14336 with
// their 16-bit copy 111 us (6.4 TB/s).
#include <type_traits>

#include "fp8_device.h"

namespace moe {

namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

// The largest of 16 lanes, in each of them (bits of magnitudes: NaN is larger
// than infinity, infinity than the rest).
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // rotations by 8, 4, 2, 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
  return v;
}

// Largest magnitude of 8 16-bit values, as fp32 bits.
__device__ __forceinline__ uint32_t top_of(bool fp16, u32x4 w) {
  uint32_t hi = 0, lo = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi = max(hi, w[i] & 0x7FFF0000u);
    lo = max(lo, w[i] & 0x00007FFFu);
  }
  return __float_as_uint(half_to_f32(fp16, (uint16_t)max(hi >> 16, lo)));
}

// Codes of a block whose largest magnitude has the bits `top`.
struct Coder {
  float an, r;
  int e;
  bool some;  // otherwise the codes are 0
  __device__ __forceinline__ explicit Coder(uint32_t top) {
    some = top < kInfBits && top > 0;
    const float a = __uint_as_float(top);
    e = some ? __builtin_amdgcn_frexp_expf(a) : 0;
    an = some ? __builtin_amdgcn_ldexpf(a, -e) : 1.0f;
    r = 1.0f / an;
  }
  __device__ __forceinline__ float quotient(float x) const {
    const float p = 448.0f * __builtin_amdgcn_ldexpf(x, -e);
    const float q0 = p * r;
    return fmaf(fmaf(-q0, an, p), r, q0);
  }
  __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) const {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(a), quotient(b), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(c), quotient(d), w, true);
    return some ? (uint32_t)w : 0u;
  }
  __device__ __forceinline__ u32x2 eight(bool fp16, u32x4 w) const {
    auto v = [&](int i) { return half_to_f32(fp16, (uint16_t)(w[i / 2] >> (16 * (i & 1)))); };
    return u32x2{four(v(0), v(1), v(2), v(3)), four(v(4), v(5), v(6), v(7))};
  }
};
__device__ __forceinline__ float scale_of(uint32_t top) {
  return top < kInfBits ? __uint_as_float(top) / 448.0f : __uint_as_float(0x7FC00000u);
}

// ---- rows ---------------------------------------------------------------------
// A block of threads takes 4 PER rows of 4 scale blocks: a wave reads 1 KB of a
// row at a time, and the scales leave as runs of 4 PER rows.  One row a wave and
// more blocks where there are few, two otherwise (us in a captured graph, 1 / 2 /
// 4 rows): 16 x 4096 2.0 / 2.4 / 3.1, 512 x 4096 3.0 / 3.1 / 3.4, 1024 x 4096 4.2 /
// 4.1 / 4.4, 16384 x 4096 35.2 / 32.5 / 35.5, 8192 x 14336 71.5 / 65.1 / 65.5.
constexpr int kBlocks = 4;  // scale blocks of a row that a wave covers
// The blocks of threads go across the columns first; a grid has fewer than 2^32
// threads in x, which the largest matrices pass, so row blocks go on in y.
constexpr int kRowBlocks = 1 << 16;
__device__ __forceinline__ int row_block(int across) { return blockIdx.y * kRowBlocks + blockIdx.x / across; }
dim3 row_grid(int rows, int per_block, int across) {
  const int blocks = (rows + per_block - 1) / per_block;
  return dim3(across * (blocks < kRowBlocks ? blocks : kRowBlocks), (blocks + kRowBlocks - 1) / kRowBlocks);
}
template <int PER>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(int rows, int k, bool fp16, const uint16_t* __restrict__ x,
                                                              int64_t ldx, uint8_t* __restrict__ codes, int64_t ldcodes,
                                                              float* __restrict__ scale, int64_t ldscale) {
  constexpr int kRows = 4 * PER;
  __shared__ float scales[kBlocks][kRows];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int across = (scale_blocks(k) + kBlocks - 1) / kBlocks;
  const int row0 = row_block(across) * kRows, kb0 = blockIdx.x % across * kBlocks;
  const int col = kb0 * kScaleBlock + lane * 8;
  u32x4 v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = row0 + wave * PER + i;
    v[i] = row < rows && col < k ? *reinterpret_cast<const u32x4*>(x + (int64_t)row * ldx + col) : u32x4{};
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = row0 + wave * PER + i;
    const uint32_t top = max16(top_of(fp16, v[i]));
    const Coder code(top);
    const u32x2 w = code.eight(fp16, v[i]);
    if (row < rows && col < k) *reinterpret_cast<u32x2*>(codes + (int64_t)row * ldcodes + col) = w;
    if ((lane & 15) == 0) scales[lane >> 4][wave * PER + i] = scale_of(top);
  }
  __syncthreads();
  if (tid < kRows * kBlocks) {
    const int b = kb0 + tid / kRows, row = row0 + tid % kRows;
    if (b * kScaleBlock < k && row < rows) scale[(int64_t)b * ldscale + row] = scales[tid / kRows][tid % kRows];
  }
}

// ---- weights ------------------------------------------------------------------
// A block of threads takes a tile of 128 x 128, 64 values a thread.
__global__ __launch_bounds__(256) void quantize_tiles_kernel(int n, int k, bool fp16, const uint16_t* __restrict__ x,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scale) {
  __shared__ uint32_t tops[4];
  const int tid = threadIdx.x;
  const int col = blockIdx.x * kScaleBlock + (tid & 15) * 8;
  const int64_t first = (int64_t)blockIdx.z * n * k;
  u32x4 v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = blockIdx.y * kScaleBlock + i * 16 + (tid >> 4);
    v[i] = row < n && col < k ? *reinterpret_cast<const u32x4*>(x + first + (int64_t)row * k + col) : u32x4{};
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, top_of(fp16, v[i]));
  top = max16(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const Coder code(top);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = blockIdx.y * kScaleBlock + i * 16 + (tid >> 4);
    if (row < n && col < k) *reinterpret_cast<u32x2*>(codes + first + (int64_t)row * k + col) = code.eight(fp16, v[i]);
  }
  if (tid == 0) scale[((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = scale_of(top);
}

// ---- slopes of the gated block ------------------------------------------------
// dg = dh u act'(g), du = dh act(g) in fp32, from there into codes and, where
// they are asked for (the weights' gradient takes them), into 16 bits.  Rows
// before the first group and behind the last are skipped.  A wave takes one row's
// 4 scale blocks: with two and four rows 4096 x 14336 took 3 and 9 us more, 24576 x
// 2048 3 and 13, 300 x 1008 1.2 and 4.2 (three loads a row hold enough registers).
__global__ __launch_bounds__(256) void fp8_slopes_kernel(int rows, int n, bool fp16, int act,
                                                         const uint16_t* __restrict__ dh, int64_t lddh,
                                                         const uint16_t* __restrict__ gu, int64_t ldgu,
                                                         const int32_t* __restrict__ offsets, int groups,
                                                         uint16_t* __restrict__ slopes, int64_t ldslopes,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scale,
                                                         int64_t ldscale) {
  constexpr int kRows = 4;
  __shared__ float scales[2][kBlocks][kRows];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int first = offsets ? max(offsets[0], 0) : 0;
  const int last = offsets ? min(offsets[groups], rows) : rows;
  const int nb = scale_blocks(n), across = (nb + kBlocks - 1) / kBlocks;
  const int row0 = row_block(across) * kRows, kb0 = blockIdx.x % across * kBlocks;
  if (row0 >= last || row0 + kRows <= first) return;
  const int col = kb0 * kScaleBlock + lane * 8;
  const int64_t half = (int64_t)nb * kScaleBlock, ldcodes = 2 * half;
  const int row = row0 + wave;
  const bool in = row >= first && row < last, inside = in && col < n;
  const u32x4 d = inside ? *reinterpret_cast<const u32x4*>(dh + (int64_t)row * lddh + col) : u32x4{};
  const u32x4 g = inside ? *reinterpret_cast<const u32x4*>(gu + (int64_t)row * ldgu + col) : u32x4{};
  const u32x4 u = inside ? *reinterpret_cast<const u32x4*>(gu + (int64_t)row * ldgu + n + col) : u32x4{};
  float dg[8], du[8];
  uint32_t gtop = 0, utop = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    auto at = [&](u32x4 v) { return half_to_f32(fp16, (uint16_t)(v[e / 2] >> (16 * (e & 1)))); };
    float value, slope;
    activate_slope(act, at(g), value, slope);
    dg[e] = at(d) * at(u) * slope;
    du[e] = at(d) * value;
    gtop = max(gtop, __float_as_uint(dg[e]) & 0x7FFFFFFFu);
    utop = max(utop, __float_as_uint(du[e]) & 0x7FFFFFFFu);
  }
  if (slopes && inside) {
    u32x4 og, ou;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      og[e] = pack_half(fp16, dg[2 * e], dg[2 * e + 1]);
      ou[e] = pack_half(fp16, du[2 * e], du[2 * e + 1]);
    }
    *reinterpret_cast<u32x4*>(slopes + (int64_t)row * ldslopes + col) = og;
    *reinterpret_cast<u32x4*>(slopes + (int64_t)row * ldslopes + n + col) = ou;
  }
  if (!codes) return;
  gtop = max16(gtop);
  utop = max16(utop);
  const Coder cg(gtop), cu(utop);
  if (in && col < half) {  // zeros behind the columns, up to whole blocks
    uint8_t* to = codes + (int64_t)row * ldcodes + col;
    *reinterpret_cast<u32x2*>(to) = u32x2{cg.four(dg[0], dg[1], dg[2], dg[3]), cg.four(dg[4], dg[5], dg[6], dg[7])};
    *reinterpret_cast<u32x2*>(to + half) = u32x2{cu.four(du[0], du[1], du[2], du[3]), cu.four(du[4], du[5], du[6], du[7])};
  }
  if ((lane & 15) == 0) {
    scales[0][lane >> 4][wave] = scale_of(gtop);
    scales[1][lane >> 4][wave] = scale_of(utop);
  }
  __syncthreads();
  if (tid < 2 * kRows * kBlocks) {
    const int h = tid / (kRows * kBlocks), in = tid % (kRows * kBlocks);
    const int b = kb0 + in / kRows, row = row0 + in % kRows;
    if (b < nb && row < rows) scale[(int64_t)(h * nb + b) * ldscale + row] = scales[h][in / kRows][in % kRows];
  }
}

}  // namespace

void launch_quantize_blocks(int rows, int k, int type, const uint16_t* x, int64_t ldx, uint8_t* codes, int64_t ldcodes,
                            float* scale, int64_t ldscale, hipStream_t s) {
  const int across = (scale_blocks(k) + kBlocks - 1) / kBlocks;
  auto go = [&](auto per) {
    constexpr int P = decltype(per)::value;
    quantize_blocks_kernel<P><<<row_grid(rows, 4 * P, across), 256, 0, s>>>(
        rows, k, type == MOE_TYPE_FP16, x, ldx, codes, ldcodes, scale, ldscale);
  };
  if ((int64_t)across * ((rows + 7) / 8) < 1024)
    go(std::integral_constant<int, 1>{});
  else
    go(std::integral_constant<int, 2>{});
}

void launch_quantize_tiles(int matrices, int n, int k, int type, const uint16_t* x, uint8_t* codes, float* scale,
                           hipStream_t s) {
  const dim3 grid(scale_blocks(k), scale_blocks(n), matrices);
  quantize_tiles_kernel<<<grid, 256, 0, s>>>(n, k, type == MOE_TYPE_FP16, x, codes, scale);
}

void launch_fp8_slopes(int rows, int n, int type, int act, const uint16_t* dh, int64_t lddh, const uint16_t* gate_up,
                       int64_t ldgu, const int32_t* offsets, int groups, uint16_t* slopes, int64_t ldslopes,
                       uint8_t* codes, float* scale, int64_t ldscale, hipStream_t s) {
  const int across = (scale_blocks(n) + kBlocks - 1) / kBlocks;
  fp8_slopes_kernel<<<row_grid(rows, 4, across), 256, 0, s>>>(rows, n, type == MOE_TYPE_FP16, act, dh, lddh, gate_up, ldgu,
                                                             offsets, groups, slopes, ldslopes, codes, scale, ldscale);
}

}  // namespace moe
