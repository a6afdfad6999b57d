// The element-wise parts of the grouped products: quantising rows and the
// gated block's slopes.
#include <algorithm>
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
// from the caches).  Bound by memory, 3 bytes per value: 8192 rows of 14336 in
// 66 us, 5.3 TB/s (a large copy reaches 4.8); 16 rows of 4096 in 3.1 us, which
// is a launch and two trips to memory.
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

// ---- slopes of the gated block ------------------------------------------------
// dg = dh u act'(g), du = dh act(g); 8 columns per thread.  Bound by memory:
// 10 bytes per element of dh (4096 rows of 14336: 93-117 us, 5.0-6.3 TB/s).
// Rows before the first group and behind the last are skipped: nothing reads
// their slopes, and a captured call may have many spare rows.
//
// They are operands of 16-bit matrix products and rounded to that type.  In
// fp16 a product of finite values may pass 65504, where dx and dw do not: the
// largest such slope of each group is kept (tops, 0 without one; the maximum
// does not depend on the order), gated_slopes_far_kernel writes that group's
// again, divided by the power of two group_lift, and the products' epilogues
// multiply it back.  That costs the group's smaller slopes 2^-25 of the lift
// (half of the smallest subnormal) and nothing where no slope is that large.
__device__ __forceinline__ void slopes8(bool fp16, int act, int n, const uint16_t* dh, const uint16_t* gu, uint16_t* dgu,
                                        float unit, float& far) {
  const u32x4 d = *reinterpret_cast<const u32x4*>(dh);
  const u32x4 g = *reinterpret_cast<const u32x4*>(gu);
  const u32x4 u = *reinterpret_cast<const u32x4*>(gu + n);
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
      if (fp16) {
        // infinities and NaN of the inputs are no large slopes
        const float ma = fabsf(a[h]), mb = fabsf(b[h]);
        if (ma > kHalfMax && ma < __builtin_inff()) far = fmaxf(far, ma);
        if (mb > kHalfMax && mb < __builtin_inff()) far = fmaxf(far, mb);
        a[h] *= unit;
        b[h] *= unit;
      }
    }
    og[i] = pack_half(fp16, a[0], a[1]);
    ou[i] = pack_half(fp16, b[0], b[1]);
  }
  *reinterpret_cast<u32x4*>(dgu) = og;
  *reinterpret_cast<u32x4*>(dgu + n) = ou;
}

__global__ __launch_bounds__(256) void clear_tops_kernel(uint32_t* tops, int groups) {
  if ((int)threadIdx.x < groups) tops[threadIdx.x] = 0;
}

__global__ __launch_bounds__(256) void gated_slopes_kernel(int rows, int n, bool fp16, int act,
                                                           const uint16_t* __restrict__ dh, int64_t lddh,
                                                           const uint16_t* __restrict__ gu, int64_t ldgu,
                                                           const int32_t* __restrict__ offsets, int groups,
                                                           uint16_t* __restrict__ dgu, uint32_t* tops) {
  const int per_row = n / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = at / per_row;
  const int col = (int)(at % per_row) * 8;
  const int first = offsets ? max(offsets[0], 0) : 0;
  const int last = offsets ? min(offsets[groups], rows) : rows;
  if (row < first || row >= last) return;
  float far = 0.0f;
  slopes8(fp16, act, n, dh + row * lddh + col, gu + row * ldgu + col, dgu + row * 2 * n + col, 1.0f, far);
  if (far > 0.0f) {
    int e = 0;  // the row's group: the last that begins at or before it
    if (offsets)
      for (int past = groups; past - e > 1;) {
        const int mid = (e + past) / 2;
        if (offsets[mid] <= row) e = mid;
        else past = mid;
      }
    // positive floats order as their bits; most threads find a larger one there
    const uint32_t bits = __float_as_uint(far);
    if (__hip_atomic_load(tops + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < bits) atomicMax(tops + e, bits);
  }
}

__global__ __launch_bounds__(256) void gated_slopes_far_kernel(int rows, int n, int act, const uint16_t* __restrict__ dh,
                                                               int64_t lddh, const uint16_t* __restrict__ gu,
                                                               int64_t ldgu, const int32_t* __restrict__ offsets,
                                                               uint16_t* __restrict__ dgu,
                                                               const uint32_t* __restrict__ tops) {
  const int group = blockIdx.y;
  const uint32_t top = tops[group];
  if (top == 0) return;
  const float unit = 1.0f / group_lift(top);  // exact
  int begin, end;
  group_rows(offsets, rows, group, begin, end);
  const int per_row = n / 8;
  const int64_t chunks = (int64_t)(end - begin) * per_row;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < chunks; at += (int64_t)gridDim.x * 256) {
    const int64_t row = begin + at / per_row;
    const int col = (int)(at % per_row) * 8;
    float far = 0.0f;
    slopes8(true, act, n, dh + row * lddh + col, gu + row * ldgu + col, dgu + row * 2 * n + col, unit, far);
  }
}

}  // namespace

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
                         int64_t ldgu, const int32_t* offsets, int groups, uint16_t* dgu, uint32_t* tops, hipStream_t s) {
  const int64_t threads = (int64_t)rows * (n / 8);
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  if (tops) clear_tops_kernel<<<1, 256, 0, s>>>(tops, groups);
  gated_slopes_kernel<<<blocks, 256, 0, s>>>(rows, n, type == MOE_TYPE_FP16, act, dh, lddh, gate_up, ldgu, offsets, groups,
                                             dgu, tops);
  // seldom more than a look at tops: few blocks, which walk over the group
  if (tops)
    gated_slopes_far_kernel<<<dim3(std::min(blocks, std::max(16u, 1024u / groups)), groups), 256, 0, s>>>(
        rows, n, act, dh, lddh, gate_up, ldgu, offsets, dgu, tops);
}

}  // namespace moe
