// The element-wise parts of the grouped products: quantising rows, joining
// the parts of a split contraction, and the gated block's slopes.
#include <type_traits>

#include "product_core.h"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d, 64));
  return v;
}

// ---- quantise rows ------------------------------------------------------------
// WPR waves share a row; each thread keeps CH chunks of 8 values in registers,
// so the row is read once (longer rows read what does not fit a second time,
// from the caches).  Bound by memory: 3 bytes per value.
//
// The code is the exact quotient 127 x / a rounded to nearest even.  With the
// row scaled by a power of two so that a is in [1/2, 1) (no overflow or
// underflow), p = 127 x is exact in fp32 (a 16-bit float has at most 11
// significant bits), r = RN(1/a), q0 = RN(p r), and q0 + (p - q0 a) r, whose
// remainder is exact by FMA, is the correctly rounded quotient (Markstein's
// division).  Rounding that to an integer equals rounding the exact quotient v:
// write v = 127 m / D with integers m < 2^11 and D (x = m, a = D up to the
// same power of two, or both times one).  Unless v is a tie, which fp32 holds
// exactly, it is at least 1 / (2D) away from one.  The quotient's error is at
// most v 2^-24: with D < 2^11 that is below 2^-17 < 2^-12, and a larger D is
// m_a 2^t with m below 2^11, so v < 2^18 / D and the error < 2^-6 / D.
template <int WPR, int CH>
__global__ __launch_bounds__(256) void quantize_kernel(int rows, int k, bool fp16, const uint16_t* __restrict__ x,
                                                       int64_t ldx, int8_t* __restrict__ codes, int64_t ldcodes,
                                                       float* __restrict__ scale) {
  constexpr int kThreads = 64 * WPR, kRows = 4 / WPR;
  __shared__ uint32_t wmax[4];
  const int tid = threadIdx.x, t = tid % kThreads;
  const int64_t row = (int64_t)blockIdx.x * kRows + tid / kThreads;
  const bool live = row < rows;
  const u32x4* src = reinterpret_cast<const u32x4*>(x + (live ? row : 0) * ldx);
  const int chunks = live ? k / 8 : 0;
  u32x4 v[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) v[c] = t + c * kThreads < chunks ? src[t + c * kThreads] : u32x4{};
  // the largest magnitude, as the larger 15-bit pattern (infinities and NaN
  // are the largest patterns of all)
  uint32_t hi = 0, lo = 0;
  auto fold = [&](u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi = max(hi, w[i] & 0x7FFF0000u);
      lo = max(lo, w[i] & 0x00007FFFu);
    }
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) fold(v[c]);
  for (int i = t + CH * kThreads; i < chunks; i += kThreads) fold(src[i]);
  uint32_t top = max_lanes(max(hi >> 16, lo));
  if constexpr (WPR > 1) {
    if ((tid & 63) == 0) wmax[tid >> 6] = top;
    __syncthreads();
    top = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  }
  if (!live) return;
  const float a = half_to_f32(fp16, (uint16_t)top);
  const bool finite = top < (fp16 ? 0x7C00u : 0x7F80u);
  if (t == 0) scale[row] = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);
  const bool some = finite && a > 0.0f;
  const int e = some ? __builtin_amdgcn_frexp_expf(a) : 0;
  const float an = some ? __builtin_amdgcn_ldexpf(a, -e) : 1.0f;
  const float r = 1.0f / an;
  // a row without a scale has codes 0: its values are not looked at
  const uint32_t keep = some ? 0xFFFFFFFFu : 0u;
  auto code = [&](uint16_t b) -> uint32_t {
    const float p = 127.0f * __builtin_amdgcn_ldexpf(half_to_f32(fp16, b), -e);
    const float q0 = p * r;
    const float q = fmaf(fmaf(-q0, an, p), r, q0);
    return (uint32_t)(int)rintf(q) & 0xFFu;
  };
  auto store = [&](int i, u32x4 w) {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w0 = w[2 * h] & keep, w1 = w[2 * h + 1] & keep;
      o[h] = code((uint16_t)w0) | (code((uint16_t)(w0 >> 16)) << 8) | (code((uint16_t)w1) << 16) |
             (code((uint16_t)(w1 >> 16)) << 24);
    }
    *reinterpret_cast<u32x2*>(codes + row * ldcodes + 8 * (int64_t)i) = o;
  };
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (t + c * kThreads < chunks) store(t + c * kThreads, v[c]);
  for (int i = t + CH * kThreads; i < chunks; i += kThreads) store(i, src[i]);
}

// ---- join of a split contraction ------------------------------------------------
// out = result of the sum of `splits` raw parts, four columns per thread, the
// parts added in order.
template <Num T, Result RES, bool WEIGHT_GRAD>
__global__ __launch_bounds__(256) void join_kernel(ProductArgs a) {
  constexpr bool GATED = RES == Result::kGated;
  using t4 = typename Acc<T>::t4;
  const int F = a.cols / 2, quads = (GATED ? F : a.cols) / 4;
  const int64_t all = WEIGHT_GRAD ? (int64_t)a.groups * a.wrows : a.rows;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row = at / quads;
  const int col = (int)(at % quads) * 4;
  if (row >= all) return;
  if constexpr (!WEIGHT_GRAD) {
    // rows outside every group have no parts
    int begin, end;
    group_rows(a.offsets, a.rows, 0, begin, end);
    if (a.offsets) end = max(0, min(a.offsets[a.groups], a.rows));
    if (row < begin || row >= end) return;
  }
  int group = 0;
  if (T == Num::kInt8 && a.offsets) {
    // the last group that begins at or before the row: its own (ascending offsets)
    int lo = 0, hi = a.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.offsets[mid] <= row) lo = mid; else hi = mid;
    }
    group = lo;
  }
  auto total = [&](int c) -> f32x4 {
    const char* src = a.partial + (row * a.cols + c) * 4;
    t4 v = *reinterpret_cast<const t4*>(src);
    for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const t4*>(src + (int64_t)s * all * a.cols * 4);
    f32x4 f;
    if constexpr (T == Num::kInt8) {
      const float ps = a.pscale[row];
      const f32x4 qs = *reinterpret_cast<const f32x4*>(a.qscale + (int64_t)group * a.cols + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = (float)v[e] * ps * qs[e];
    } else {
      f = v;
    }
    return f;
  };
  f32x4 v = total(col);
  const bool fp16 = T == Num::kFp16 || (T == Num::kInt8 && a.out_type == MOE_TYPE_FP16);
  if constexpr (GATED) {
    const f32x4 u = total(F + col);
    if (T != Num::kInt8 && a.keep) {
      uint16_t* k = a.keep + row * a.ldkeep + col;
      *reinterpret_cast<u32x2*>(k) = u32x2{pack_half(fp16, v[0], v[1]), pack_half(fp16, v[2], v[3])};
      *reinterpret_cast<u32x2*>(k + F) = u32x2{pack_half(fp16, u[0], u[1]), pack_half(fp16, u[2], u[3])};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]) * u[e];
  }
  if constexpr (RES == Result::kWide)
    *reinterpret_cast<f32x4*>((float*)a.out + row * a.ldout + col) = v;
  else
    *reinterpret_cast<u32x2*>((uint16_t*)a.out + row * a.ldout + col) =
        u32x2{pack_half(fp16, v[0], v[1]), pack_half(fp16, v[2], v[3])};
}

// ---- slopes of the gated block ------------------------------------------------
// dg = dh u act'(g), du = dh act(g); 8 columns per thread.  Bound by memory:
// 10 bytes per element of dh.
__global__ __launch_bounds__(256) void gated_slopes_kernel(int rows, int n, bool fp16, int act,
                                                           const uint16_t* __restrict__ dh, int64_t lddh,
                                                           const uint16_t* __restrict__ gu, int64_t ldgu,
                                                           uint16_t* __restrict__ dgu) {
  const int per_row = n / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = at / per_row;
  const int col = (int)(at % per_row) * 8;
  if (row >= rows) return;
  const u32x4 d = *reinterpret_cast<const u32x4*>(dh + row * lddh + col);
  const u32x4 g = *reinterpret_cast<const u32x4*>(gu + row * ldgu + col);
  const u32x4 u = *reinterpret_cast<const u32x4*>(gu + row * ldgu + n + col);
  u32x4 og, ou;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a[2], b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float dv = half_to_f32(fp16, (uint16_t)(d[i] >> (16 * h)));
      const float gv = half_to_f32(fp16, (uint16_t)(g[i] >> (16 * h)));
      const float uv = half_to_f32(fp16, (uint16_t)(u[i] >> (16 * h)));
      float value, slope;
      activate_slope(act, gv, value, slope);
      a[h] = dv * uv * slope;
      b[h] = dv * value;
    }
    og[i] = pack_half(fp16, a[0], a[1]);
    ou[i] = pack_half(fp16, b[0], b[1]);
  }
  *reinterpret_cast<u32x4*>(dgu + row * 2 * n + col) = og;
  *reinterpret_cast<u32x4*>(dgu + row * 2 * n + n + col) = ou;
}

template <Num T, Result RES, bool WG>
void launch_join(const ProductArgs& a, hipStream_t s) {
  const int64_t rows = WG ? (int64_t)a.groups * a.wrows : a.rows;
  const int64_t quads = rows * ((RES == Result::kGated ? a.cols / 2 : a.cols) / 4);
  join_kernel<T, RES, WG><<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(a);
}

}  // namespace

void launch_product_join(const ProductArgs& a, Num num, Pass pass, Result res, hipStream_t s) {
  if (num == Num::kInt8) {
    if (res == Result::kGated)
      launch_join<Num::kInt8, Result::kGated, false>(a, s);
    else if (res == Result::kWide)
      launch_join<Num::kInt8, Result::kWide, false>(a, s);
    else
      launch_join<Num::kInt8, Result::kHalf, false>(a, s);
    return;
  }
  const bool wg = pass == Pass::kWeightGrad;
  if (res == Result::kWide) {
    launch_join<Num::kBf16, Result::kWide, true>(a, s);  // fp32 sums to fp32: the operands' type is gone
  } else if (num == Num::kFp16) {
    if (res == Result::kGated)
      launch_join<Num::kFp16, Result::kGated, false>(a, s);
    else if (wg)
      launch_join<Num::kFp16, Result::kHalf, true>(a, s);
    else
      launch_join<Num::kFp16, Result::kHalf, false>(a, s);
  } else {
    if (res == Result::kGated)
      launch_join<Num::kBf16, Result::kGated, false>(a, s);
    else if (wg)
      launch_join<Num::kBf16, Result::kHalf, true>(a, s);
    else
      launch_join<Num::kBf16, Result::kHalf, false>(a, s);
  }
}

void launch_quantize(int rows, int k, int type, const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldcodes,
                     float* scale, hipStream_t s) {
  const bool fp16 = type == MOE_TYPE_FP16;
  auto go = [&](auto wpr, auto ch) {
    constexpr int W = decltype(wpr)::value, C = decltype(ch)::value;
    const int per = 4 / W;
    quantize_kernel<W, C><<<(rows + per - 1) / per, 256, 0, s>>>(rows, k, fp16, x, ldx, codes, ldcodes, scale);
  };
  using std::integral_constant;
  if (k <= 1024)  // one wave a row
    go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  else if (k <= 4096)
    go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  else
    go(integral_constant<int, 4>{}, integral_constant<int, 8>{});
}

void launch_gated_slopes(int rows, int n, int type, int act, const uint16_t* dh, int64_t lddh, const uint16_t* gate_up,
                         int64_t ldgu, uint16_t* dgu, hipStream_t s) {
  const int64_t threads = (int64_t)rows * (n / 8);
  gated_slopes_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(rows, n, type == MOE_TYPE_FP16, act, dh, lddh,
                                                                        gate_up, ldgu, dgu);
}

}  // namespace moe
