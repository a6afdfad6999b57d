// AdamW over many tensors (moe_optim.h): C entry point and kernel.
//
// Bound by memory: each value's weight, gradient and states pass once.  A block
// of threads takes kChunk consecutive values of one tensor, 8 a thread; the
// tensors of a launch and where their chunks begin stand in the kernel's
// arguments, so that one launch serves up to kTensors tensors of the same types
// and nothing is copied to the device before it.
//
// 8-bit states have a scale for each 128 values, which 16 neighbouring lanes
// hold.  A state x with scale s is coded as sign(x) n 2^e, where 2^e is the
// spacing of the codes around |x| / s and n = floor(|x| / (s 2^e) + u), u the
// random fraction of 2^16: n is the next whole number up with the probability
// that |x| / (s 2^e) lies above the one below.
//
// Measured on one tensor of 2^28 values: fp32 weights and states 1390 us, 5.4 TB/s
// of what has to pass (a copy reaches 4.9); bf16 weights with fp32 ones beside
// them 1402 us, 5.35 TB/s, with 8-bit states 793 us, 5.45 TB/s.  bf16 weights with
// 8-bit states alone, 10 bytes a value, 472 to 500 us by box, 5.4 to 5.7 TB/s; there
// the arithmetic counts: by the compiler's exact divisions and roots, and with
// ordinary instructions rounding the codes, 719 us; with two passes of 8 values a
// thread and the step's numbers worked out by every block, not by the host, 550.
// 4096 values a block in two passes: 524 us, 1% to 3% more for the others; blocks of
// 128 and of 512 threads, and stores past the caches, change nothing.
//
// A step with numbers on the device has every thread work all of them out, in 64
// bits: bf16 weights with 8-bit states 577 us where the host's numbers take 472 (623
// at a step past 10^6, whose powers are longer), with fp32 ones beside them 801
// (793; 844), with fp32 states 1406 (1402), all in fp32 1383 (1393).
#include <algorithm>
#include <cmath>
#include <vector>

#include "api_checks.h"
#include "moe_optim.h"
#include "product_core.h"

namespace moe {

namespace {

constexpr int kStateBlock = 128;  // values that share a scale
constexpr int kThreads = 256, kChunk = kThreads * 8;
constexpr int kTensors = 36;

struct AdamTensor {
  void* param;
  const void* grad;
  float* master;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t count;
  int32_t number;  // in the call
  uint32_t first;  // the first of its chunks
};
// What all values of a step share.
struct Numbers {
  float b1, c1, b2, c2;  // beta, 1 - beta
  float keep;            // 1 - lr weight_decay
  float rate;            // lr / (1 - beta1^t)
  float root;            // 1 / sqrt(1 - beta2^t)
  float eps, grad_scale;
  uint32_t key;  // of seed and step
};
struct AdamArgs {
  double lr, beta1, beta2, weight_decay;
  float eps, grad_scale;
  uint64_t seed;
  int32_t step, tensors;
  const float *device_lr, *device_grad_scale;
  const int32_t* device_step;
  Numbers numbers;  // without numbers on the device
  AdamTensor t[kTensors];
};
static_assert(sizeof(AdamArgs) <= 4096 - 256, "kernel arguments");

// The halves of x c, XORed; twice of it, with a key, makes a value's draw.
__host__ __device__ __forceinline__ uint32_t fold(uint32_t x, uint32_t c) {
  const uint64_t p = (uint64_t)x * c;
  return (uint32_t)(p >> 32) ^ (uint32_t)p;
}
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x, uint32_t key) {
  return fold(fold(x ^ key, 0x9E3779B9u) + key, 0xBB67AE85u);
}

// beta^t by squaring, which takes few steps and the same ones everywhere.
__host__ __device__ inline double power(double b, uint32_t t) {
  double r = 1.0;
  for (; t; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}
// The same operations on the host and on the device: a step with its numbers in
// device memory gives the bits of one that was given them.
__host__ __device__ inline Numbers numbers_of(const AdamArgs& a, double lr, float grad_scale, int step) {
#pragma clang fp contract(off)
  Numbers n;
  n.b1 = (float)a.beta1;
  n.c1 = (float)(1.0 - a.beta1);
  n.b2 = (float)a.beta2;
  n.c2 = (float)(1.0 - a.beta2);
  n.keep = (float)(1.0 - lr * a.weight_decay);
  n.rate = (float)(lr / (1.0 - power(a.beta1, step)));
  n.root = (float)(1.0 / sqrt(1.0 - power(a.beta2, step)));
  n.eps = a.eps;
  n.grad_scale = grad_scale;
  n.key = mix((uint32_t)step, mix((uint32_t)(a.seed >> 32), (uint32_t)a.seed));
  return n;
}
__host__ __device__ inline bool on_device(const AdamArgs& a) { return a.device_lr || a.device_grad_scale || a.device_step; }

// The largest of 16 lanes, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // rotations by 8, 4, 2, 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
  return v;
}

// e4m3 (m) and e5m2 (v): largest and smallest positive value.  The conversions
// that take random bits add them to the bits that a code has no room for, the
// highest first, and cut off what is left: floor(|x| / unit + u) units, subnormal
// codes included (2^24 random values of either type: no other result).
struct E4M3 {
  static constexpr float kMost = 448.0f;
  static constexpr float kLeast = 0x1p-9f;
  static __device__ __forceinline__ void wide(uint32_t w, float* f) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
  }
  static __device__ __forceinline__ uint32_t narrow(const float* f, const uint32_t* u) {
    int w = __builtin_amdgcn_cvt_sr_fp8_f32(f[0], u[0], 0, 0);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(f[1], u[1], w, 1);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(f[2], u[2], w, 2);
    return __builtin_amdgcn_cvt_sr_fp8_f32(f[3], u[3], w, 3);
  }
};
struct E5M2 {
  static constexpr float kMost = 57344.0f;
  static constexpr float kLeast = 0x1p-16f;
  static __device__ __forceinline__ void wide(uint32_t w, float* f) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_bf8(w, true);
    f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
  }
  static __device__ __forceinline__ uint32_t narrow(const float* f, const uint32_t* u) {
    int w = __builtin_amdgcn_cvt_sr_bf8_f32(f[0], u[0], 0, 0);
    w = __builtin_amdgcn_cvt_sr_bf8_f32(f[1], u[1], w, 1);
    w = __builtin_amdgcn_cvt_sr_bf8_f32(f[2], u[2], w, 2);
    return __builtin_amdgcn_cvt_sr_bf8_f32(f[3], u[3], w, 3);
  }
};

// Codes of 8 states of a block whose scale comes out as `scale`; u: random bits,
// the highest 16 of each.  The quotient x / s is the correctly rounded one
// (Markstein's division, on values scaled by a power of two), as are m and v
// before it: the codes do not depend on how the compiler would contract or divide.
template <typename F, bool SQUARES>
__device__ __forceinline__ u32x2 code8(const float* x, const uint32_t* u, float& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  top = max16(top);
  const bool finite = top < 0x7F800000u;
  scale = finite ? __uint_as_float(top) * (1.0f / F::kMost) : __uint_as_float(0x7FC00000u);
  const bool some = finite && scale > 0.0f;
  const int se = some ? __builtin_amdgcn_frexp_expf(scale) : 0;
  const float sn = some ? __builtin_amdgcn_ldexpf(scale, -se) : 1.0f;
  const float r = 1.0f / sn;
  float c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = __builtin_amdgcn_ldexpf(x[e], -se);
    const float q0 = p * r;
    const float y = fmaf(fmaf(-q0, sn, p), r, q0);
    // a quotient may pass the largest code by its rounding
    if (SQUARES)
      c[e] = fminf(fmaxf(y, x[e] > 0.0f ? F::kLeast : 0.0f), F::kMost);
    else
      c[e] = __builtin_amdgcn_fmed3f(y, -F::kMost, F::kMost);
  }
  return some ? u32x2{F::narrow(c, u), F::narrow(c + 4, u + 4)} : u32x2{};
}

template <typename T> struct Wide {  // 8 values of a 16-bit type
  static __device__ __forceinline__ void load(const T* p, float* f) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = half_to_f32(std::is_same<T, _Float16>::value, (uint16_t)(w[e / 2] >> (16 * (e & 1))));
  }
  static __device__ __forceinline__ void store(T* p, const float* f) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_half(std::is_same<T, _Float16>::value, f[2 * e], f[2 * e + 1]);
    *reinterpret_cast<u32x4*>(p) = w;
  }
};
template <> struct Wide<float> {
  static __device__ __forceinline__ void load(const float* p, float* f) {
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = lo[e], f[4 + e] = hi[e];
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
  }
};
// The last values of a tensor, fewer than 8: one by one.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, float* f) {
  if (left >= 8) return Wide<T>::load(p, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = e < left ? (float)p[e] : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int left, const float* f) {
  if (left >= 8) return Wide<T>::store(p, f);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = (T)f[e];
}
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int left) {
  if (left >= 8) return *reinterpret_cast<const u32x2*>(p);
  u32x2 w = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) w[e / 4] |= (uint32_t)p[e] << (8 * (e & 3));
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int left, u32x2 w) {
  if (left >= 8) {
    *reinterpret_cast<u32x2*>(p) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
}

// Whether the hardware's root and reciprocal, each within one unit in the last
// place of normal numbers, will do: the root of a subnormal v is below 2^-63,
// less than 2^-25 of eps / root, and root and eps up to 1 keep the denominator
// of a finite v normal and its reciprocal too.
__device__ __forceinline__ bool plain_roots(const Numbers& n) { return n.eps >= n.root * 0x1p-38f && n.eps <= 1.0f; }

template <typename P, typename G, bool MASTER, bool CODES>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamArgs a) {
#pragma clang fp contract(off)
  const uint32_t chunk = blockIdx.y * gridDim.x + blockIdx.x;
  int i = 0;  // its tensor: the last that begins at or before it
  for (int past = a.tensors; past - i > 1;) {
    const int mid = (i + past) / 2;
    if (a.t[mid].first <= chunk)
      i = mid;
    else
      past = mid;
  }
  const AdamTensor& t = a.t[i];
  const int64_t begin = (int64_t)(chunk - t.first) * kChunk;
  const Numbers n = !on_device(a) ? a.numbers
                                  : numbers_of(a, a.device_lr ? (double)*a.device_lr : a.lr,
                                               a.device_grad_scale ? *a.device_grad_scale : a.grad_scale,
                                               a.device_step ? max(*a.device_step, 1) : a.step);
  // (a chunk does not cross a multiple of 2^32)
  const uint32_t key = mix((uint32_t)(begin >> 32), mix((uint32_t)t.number, n.key));
  P* param = (P*)t.param;
  const G* grad = (const G*)t.grad;
  const int64_t at = begin + threadIdx.x * 8;
  const int left = (int)min((int64_t)8, t.count - at);
  // 16 lanes share a scale: they leave together
  if (t.count <= at / kStateBlock * kStateBlock) return;
  float p[8] = {}, g[8] = {}, m[8] = {}, v[8] = {};
  if (left > 0) {
    load8(grad + at, left, g);
    if (MASTER)
      load8(t.master + at, left, p);
    else
      load8(param + at, left, p);
    if (CODES) {
      const u32x2 cm = load_codes((const uint8_t*)t.m + at, left), cv = load_codes((const uint8_t*)t.v + at, left);
      const float sm = t.m_scale[at / kStateBlock], sv = t.v_scale[at / kStateBlock];
      E4M3::wide(cm[0], m);
      E4M3::wide(cm[1], m + 4);
      E5M2::wide(cv[0], v);
      E5M2::wide(cv[1], v + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] *= sm, v[e] *= sv;
      if (left < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= left) m[e] = v[e] = 0.0f;
      }
    } else {
      load8((const float*)t.m + at, left, m);
      load8((const float*)t.v + at, left, v);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float gs = g[e] * n.grad_scale;
    m[e] = m[e] * n.b1 + gs * n.c1;
    v[e] = v[e] * n.b2 + (gs * gs) * n.c2;
  }
  if (plain_roots(n)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p[e] = fmaf(-n.rate * m[e], __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_sqrtf(v[e]), n.root, n.eps)), p[e] * n.keep);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = p[e] * n.keep - n.rate * m[e] / (sqrtf(v[e]) * n.root + n.eps);
  }
  if (left > 0) {
    if (MASTER) store8(t.master + at, left, p);
    store8(param + at, left, p);
  }
  if (CODES) {
    uint32_t um[8], uv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t d = mix((uint32_t)at + e, key);
      um[e] = d << 16;
      uv[e] = d & 0xFFFF0000u;
    }
    float sm, sv;
    const u32x2 cm = code8<E4M3, false>(m, um, sm), cv = code8<E5M2, true>(v, uv, sv);
    if (left > 0) {
      store_codes((uint8_t*)t.m + at, left, cm);
      store_codes((uint8_t*)t.v + at, left, cv);
    }
    if ((threadIdx.x & 15) == 0) {
      t.m_scale[at / kStateBlock] = sm;
      t.v_scale[at / kStateBlock] = sv;
    }
  } else if (left > 0) {
    store8((float*)t.m + at, left, m);
    store8((float*)t.v + at, left, v);
  }
}

constexpr int64_t kMaxChunks = (int64_t)1 << 24;  // of a launch
constexpr int64_t kMaxCount = (int64_t)1 << 35;
static_assert(kMaxCount / kChunk <= kMaxChunks, "a tensor fits a launch");
// A grid has fewer than 2^32 threads in x.  The blocks that y adds behind the
// last chunk find nothing.
dim3 grid_of(int64_t chunks) {
  const int64_t x = std::min<int64_t>(chunks, 1 << 20);
  return dim3((unsigned)x, (unsigned)((chunks + x - 1) / x));
}

template <typename P, typename G, bool MASTER>
void launch(const AdamArgs& a, int64_t chunks, bool codes, hipStream_t s) {
  if (codes)
    adamw_kernel<P, G, MASTER, true><<<grid_of(chunks), kThreads, 0, s>>>(a);
  else
    adamw_kernel<P, G, MASTER, false><<<grid_of(chunks), kThreads, 0, s>>>(a);
}
template <typename P>
void launch_half(const AdamArgs& a, int64_t chunks, bool wide_grad, bool master, bool codes, hipStream_t s) {
  if (wide_grad)
    master ? launch<P, float, true>(a, chunks, codes, s) : launch<P, float, false>(a, chunks, codes, s);
  else
    master ? launch<P, P, true>(a, chunks, codes, s) : launch<P, P, false>(a, chunks, codes, s);
}

size_t size_of(int type) { return type == MOE_TYPE_FP32 ? 4 : 2; }

moe_status check_numbers(const moe_adamw* n) {
  if (!n) return api_fail(MOE_ERR_INVALID_ARG, "null pointer argument");
  auto finite = [](double x) { return std::isfinite(x); };
  if (!n->device_lr && !finite(n->lr)) return api_fail(MOE_ERR_INVALID_ARG, "lr=%g is not finite", n->lr);
  if (!(n->beta1 >= 0.0 && n->beta1 < 1.0) || !(n->beta2 >= 0.0 && n->beta2 < 1.0))
    return api_fail(MOE_ERR_INVALID_ARG, "beta1=%g, beta2=%g must be in [0, 1)", n->beta1, n->beta2);
  if (!finite(n->eps) || n->eps < 0.0) return api_fail(MOE_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", n->eps);
  if (!finite(n->weight_decay)) return api_fail(MOE_ERR_INVALID_ARG, "weight_decay=%g is not finite", n->weight_decay);
  if (!n->device_step && n->step < 1) return api_fail(MOE_ERR_INVALID_ARG, "step=%d must be at least 1", n->step);
  if (n->state_bits != 8 && n->state_bits != 32)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "state_bits=%d must be 8 or 32", n->state_bits);
  for (const void* p : {(const void*)n->device_lr, (const void*)n->device_grad_scale, (const void*)n->device_step})
    if (reinterpret_cast<uintptr_t>(p) % 4) return api_fail(MOE_ERR_INVALID_ARG, "a device number is not 4-byte aligned");
  return MOE_OK;
}

moe_status check_tensor(const moe_adamw_tensor& t, int i, bool codes) {
  if (t.count < 0 || t.count > kMaxCount)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "tensor %d: count=%lld outside [0, %lld]", i, (long long)t.count,
                    (long long)kMaxCount);
  if (t.param_type != MOE_TYPE_BF16 && t.param_type != MOE_TYPE_FP16 && t.param_type != MOE_TYPE_FP32)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "tensor %d: param_type=%d is no moe_type", i, t.param_type);
  if (t.grad_type != t.param_type && t.grad_type != MOE_TYPE_FP32)
    return api_fail(MOE_ERR_UNSUPPORTED_SHAPE, "tensor %d: grad_type=%d must be param_type or MOE_TYPE_FP32", i, t.grad_type);
  if (t.master && t.param_type == MOE_TYPE_FP32)
    return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: a param in fp32 has no master", i);
  if (t.count == 0) return MOE_OK;
  struct {
    const char* name;
    const void* p;
    bool needed;
    unsigned align;
  } const all[] = {{"param", t.param, true, 16},      {"grad", t.grad, true, 16}, {"master", t.master, false, 16},
                   {"m", t.m, true, 16},              {"v", t.v, true, 16},       {"m_scale", t.m_scale, codes, 4},
                   {"v_scale", t.v_scale, codes, 4}};
  for (const auto& x : all) {
    if (x.needed && !x.p) return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: %s is null", i, x.name);
    if (reinterpret_cast<uintptr_t>(x.p) % x.align)
      return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: %s is not %u-byte aligned", i, x.name, x.align);
  }
  if (!codes && (t.m_scale || t.v_scale))
    return api_fail(MOE_ERR_INVALID_ARG, "tensor %d: states in 32 bits have no scales", i);
  return MOE_OK;
}

// What a step writes overlaps nothing else that it reads or writes.
moe_status check_apart(int count, const moe_adamw_tensor* tensors, bool codes) {
  struct Range {
    uintptr_t begin, end;
    int tensor;
    bool written;
  };
  std::vector<Range> all;
  all.reserve((size_t)count * 7);
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.count == 0) continue;
    auto add = [&](const void* p, size_t bytes, bool written) {
      const uintptr_t b = reinterpret_cast<uintptr_t>(p);
      if (p) all.push_back({b, b + bytes, i, written});
    };
    const size_t scales = (size_t)((t.count + kStateBlock - 1) / kStateBlock) * 4;
    add(t.param, t.count * size_of(t.param_type), true);
    add(t.master, t.count * 4, true);
    add(t.m, t.count * (codes ? 1 : 4), true);
    add(t.v, t.count * (codes ? 1 : 4), true);
    add(t.m_scale, scales, true);
    add(t.v_scale, scales, true);
    add(t.grad, t.count * size_of(t.grad_type), false);
  }
  std::sort(all.begin(), all.end(), [](const Range& x, const Range& y) { return x.begin < y.begin; });
  // the range that reaches furthest so far, among all and among the written ones
  const Range *far = nullptr, *far_written = nullptr;
  for (const Range& r : all) {
    const Range* hit = r.written ? far : far_written;
    if (hit && r.begin < hit->end)
      return api_fail(MOE_ERR_INVALID_ARG, "tensors %d and %d share memory", hit->tensor, r.tensor);
    if (!far || r.end > far->end) far = &r;
    if (r.written && (!far_written || r.end > far_written->end)) far_written = &r;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_EXPORT moe_status moe_adamw_step(const moe_adamw* n, int32_t count, const moe_adamw_tensor* tensors,
                                     moe_stream stream) {
  MOE_TRY(check_numbers(n));
  if (count < 0 || (count > 0 && !tensors)) return api_fail(MOE_ERR_INVALID_ARG, "%d tensors at %p", count, (const void*)tensors);
  const bool codes = n->state_bits == 8;
  try {
    for (int i = 0; i < count; ++i) MOE_TRY(check_tensor(tensors[i], i, codes));
    MOE_TRY(check_apart(count, tensors, codes));
  } catch (const std::bad_alloc&) {
    return api_fail(MOE_ERR_INVALID_ARG, "no memory to check %d tensors", count);
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  AdamArgs a;
  a.lr = n->lr;
  a.beta1 = n->beta1;
  a.beta2 = n->beta2;
  a.weight_decay = n->weight_decay;
  a.eps = (float)n->eps;
  a.grad_scale = (float)n->grad_scale;
  a.seed = n->seed;
  a.step = n->step;
  a.device_lr = n->device_lr;
  a.device_grad_scale = n->device_grad_scale;
  a.device_step = n->device_step;
  if (!on_device(a)) a.numbers = numbers_of(a, a.lr, a.grad_scale, a.step);
  // tensors of the same types share launches, in their order
  for (int type = MOE_TYPE_BF16; type <= MOE_TYPE_FP32; ++type)
    for (int kind = 0; kind < (type == MOE_TYPE_FP32 ? 1 : 4); ++kind) {
      const bool wide_grad = type == MOE_TYPE_FP32 || (kind & 1), master = kind & 2;
      int64_t chunks = 0;
      a.tensors = 0;
      auto flush = [&]() {
        if (a.tensors == 0) return MOE_OK;
        if (type == MOE_TYPE_FP32)
          launch<float, float, false>(a, chunks, codes, s);
        else if (type == MOE_TYPE_FP16)
          launch_half<_Float16>(a, chunks, wide_grad, master, codes, s);
        else
          launch_half<__bf16>(a, chunks, wide_grad, master, codes, s);
        a.tensors = 0;
        chunks = 0;
        return check_launch();
      };
      for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.count == 0 || t.param_type != type || (t.grad_type == MOE_TYPE_FP32) != wide_grad ||
            (t.master != nullptr) != master)
          continue;
        const int64_t mine = (t.count + kChunk - 1) / kChunk;
        if (a.tensors == kTensors || chunks + mine > kMaxChunks) MOE_TRY(flush());
        a.t[a.tensors++] = {t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale, t.count, i, (uint32_t)chunks};
        chunks += mine;
      }
      MOE_TRY(flush());
    }
  return MOE_OK;
}
