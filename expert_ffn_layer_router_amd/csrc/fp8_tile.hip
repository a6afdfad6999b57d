// LDS-tiled products of e4m3 codes with a scale for each block of 128.
#include "fp8_device.h"

namespace moe {

namespace {

// Transposing LDS read of 8-bit values: 16 lanes read 8 rows of 16, lane l the
// 8 values from 8 (l % 2) on of row l / 2, and lane l receives column l.
__device__ __forceinline__ u32x2 read_transposed8(lds_char* __restrict p) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)p));
}
template <Pass PASS, Result RES, bool JOIN, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(Fp8Args a) {
  constexpr int NW = WM * WN, THREADS = 64 * NW;
  constexpr int MI = BM / 16 / WM, NJ = BN / 16 / WN;
  constexpr bool Q_STR = PASS == Pass::kInputGrad;
  constexpr bool GATED = RES == Result::kGated;
  constexpr int BK = kScaleBlock;  // contraction values, and bytes of a row, per stage
  constexpr int kPBytes = BM * BK, kQBytes = BN * BK;
  constexpr int kSlot = kPBytes + kQBytes;
  constexpr int PI = kPBytes / 1024 / NW, QI = kQBytes / 1024 / NW;  // 1 KB copies per wave and stage
  constexpr int NO = GATED ? BN / 2 : BN;                            // result columns per block
  constexpr int NS = GATED ? 2 : 1;                                  // column scales of a wave
  static_assert(PI * NW * 1024 == kPBytes && QI * NW * 1024 == kQBytes, "even copy split");
  static_assert(!GATED || NJ % 2 == 0, "gate and up tiles in pairs");
  static_assert(NO % (16 * NJ / NS) == 0 && kScaleBlock % (16 * NJ / NS) == 0 && (!GATED || kScaleBlock % NO == 0),
                "a wave's columns share a scale");
  static_assert(BM * BN * 2 <= 2 * kSlot, "the 16-bit result fits the stages' LDS");
  __shared__ __attribute__((aligned(1024))) char smem_raw[2 * kSlot];
  lds_char* smem = (lds_char*)smem_raw;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, quad = lane >> 4;
  const int F = a.cols / 2;  // gated: gate rows of w
  const int ncols = GATED ? F : a.cols;
  const int tiles_n = (ncols + NO - 1) / NO;
  const int half_stages = (a.contract + BK - 1) / BK;
  const int stages = a.halves * half_stages;
  RowTile t;
  if (!find_row_tile<BM, BN, THREADS, JOIN>(a, tiles_n, stages, smem, t)) return;
  const int row0 = t.row0, live = min(BM, t.end - t.row0), n0 = t.tile_n * NO;
  const int parts = t.parts;
  if (a.groups > 1) __syncthreads();  // the lookup's LDS is free
  const int st0 = parts == 1 ? 0 : stages * t.part / parts, st1 = parts == 1 ? stages : stages * (t.part + 1) / parts;
  auto raw = [&](int at, int i, int j) {
    return reinterpret_cast<f32x4*>(a.partial + (int64_t)at * (BM * BN * 4)) + ((wave * MI + i) * NJ + j) * 64 + lane;
  };

  f32x4 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
  if constexpr (JOIN) {
    for (int s = 0; s < parts; ++s)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] += *raw(t.slot + s * t.slot_step, i, j);
  } else {
    // ---- copies ----
    const char* pbase = a.p + (int64_t)row0 * a.ldp;
    const char* qbase = a.q + (int64_t)t.group * a.q_group + (Q_STR ? (int64_t)n0 : (int64_t)n0 * a.ldq);
    uint32_t pv[PI], qv[QI];  // byte offsets of this lane's copies, or kNoLoad
    int pk[PI], qk[QI];       // their contraction position in the stage
#pragma unroll
    for (int c = 0; c < PI; ++c) {
      const int r = (wave * PI + c) * 8 + lane / 8, chunk = (lane & 7) ^ ((r >> 1) & 7);
      pv[c] = r < live ? (uint32_t)(r * a.ldp + 16 * chunk) : kNoLoad;
      pk[c] = 16 * chunk;
    }
#pragma unroll
    for (int c = 0; c < QI; ++c) {
      if constexpr (Q_STR) {
        constexpr int cpr = BN / 16;  // 16-byte chunks per LDS row
        const int kr = (wave * QI + c) * (64 / cpr) + lane / cpr;
        const int fold = cpr == 16 ? (kr & 7) | (kr >> 1 & 8) : (kr >> 1 & 3) | (kr >> 2 & 4);
        const int chunk = (lane % cpr) ^ fold;
        qv[c] = n0 + 16 * chunk < ncols ? (uint32_t)(kr * a.ldq + 16 * chunk) : kNoLoad;
        qk[c] = kr;
      } else {
        const int r = (wave * QI + c) * 8 + lane / 8, chunk = (lane & 7) ^ ((r >> 1) & 7);
        int src = r;
        if constexpr (GATED) {  // LDS row r: tile r / 16 belongs to wave column (r / 16) / NJ
          const int jb = r / 16;
          src = (jb / NJ * (NJ / 2) + jb % NJ / 2) * 16 + r % 16;
        }
        qv[c] = n0 + src < ncols ? (uint32_t)(src * a.ldq + 16 * chunk) : kNoLoad;
        qk[c] = 16 * chunk;
      }
    }
    auto copy_stage = [&](int slot, int st) {
      const int half = st >= half_stages ? 1 : 0, in = st - half * half_stages;
      const int left = a.contract - in * BK;
      lds_char* dst = smem + slot * kSlot;
      const __amdgpu_buffer_rsrc_t pr = buffer_at(pbase + (int64_t)st * BK);
#pragma unroll
      for (int c = 0; c < PI; ++c)
        buffer_to_lds16(pr, dst + (wave * PI + c) * 1024, a.halves == 2 || pk[c] < left ? pv[c] : kNoLoad, 0);
      const char* q = qbase + (Q_STR ? ((int64_t)half * a.contract + in * BK) * a.ldq : (int64_t)in * BK);
      const __amdgpu_buffer_rsrc_t qr = buffer_at(q), ur = buffer_at(GATED ? q + (int64_t)F * a.ldq : q);
#pragma unroll
      for (int c = 0; c < QI; ++c)
        buffer_to_lds16(GATED && (wave * QI + c) / 2 % 2 ? ur : qr, dst + kPBytes + (wave * QI + c) * 1024,
                        qk[c] < left ? qv[c] : kNoLoad, 0);
    };
    // ---- scales ----
    const float* psb = a.pscale + row0;
    const float* qsb = a.qscale + (int64_t)t.group * a.qs_group +
                       (int64_t)((n0 + (GATED ? 0 : wn * NJ * 16)) / kScaleBlock) * a.qs_cols;
    // a block's last columns may lie past the matrix: their scale is not read
    const bool cols_in = n0 + (GATED ? 0 : wn * NJ * 16) < ncols;
    float ps[2][MI], qs[2][NS];
    auto load_scales = [&](int b, int st) {
      const __amdgpu_buffer_rsrc_t r = scales_at(psb + (int64_t)st * a.ldscale, live);
#pragma unroll
      for (int i = 0; i < MI; ++i) ps[b][i] = load_scale(r, ((wm * MI + i) * 16 + l16) * 4);
#pragma unroll
      for (int h = 0; h < NS; ++h) qs[b][h] = cols_in ? qsb[h * a.qs_half + st * a.qs_stage] : 0.0f;
    };

    // ---- fragments ----
    auto pread = [&](int slot, int i) {
      lds_char* at = smem + slot * kSlot + ((wm * MI + i) * 16 + l16) * BK;
      const int sw = (l16 >> 1) & 7;
      return join_halves(*(__attribute__((address_space(3))) u32x4*)(at + 16 * (quad ^ sw)),
                         *(__attribute__((address_space(3))) u32x4*)(at + 16 * ((quad + 4) ^ sw)));
    };
    auto qread = [&](int slot, int j) {
      lds_char* base = smem + slot * kSlot + kPBytes;
      if constexpr (Q_STR) {
        // lane l reads half of 16 columns of row 16 (l / 16) + l % 16 / 2 (+ 8, + 64)
        u32x2 v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int kr = (s / 2) * 64 + quad * 16 + (s % 2) * 8 + (l16 >> 1);
          const int fold = BN == 256 ? (kr & 7) | (kr >> 1 & 8) : (kr >> 1 & 3) | (kr >> 2 & 4);
          v[s] = read_transposed8(base + kr * BN + 16 * ((wn * NJ + j) ^ fold) + 8 * (l16 & 1));
        }
        return join_halves(u32x4{v[0].x, v[0].y, v[1].x, v[1].y}, u32x4{v[2].x, v[2].y, v[3].x, v[3].y});
      } else {
        lds_char* at = base + ((wn * NJ + j) * 16 + l16) * BK;
        const int sw = (l16 >> 1) & 7;
        return join_halves(*(__attribute__((address_space(3))) u32x4*)(at + 16 * (quad ^ sw)),
                           *(__attribute__((address_space(3))) u32x4*)(at + 16 * ((quad + 4) ^ sw)));
      }
    };

    const bool busy = wm * MI * 16 < live;  // this wave has rows
    copy_stage(0, st0);
    load_scales(0, st0);
    auto stage = [&](int b, int st) {
      wait_copies<0>();
      __syncthreads();  // stage st has landed, and the other slot is free
      if (st + 1 < st1) {
        copy_stage(b ^ 1, st + 1);
        load_scales(b ^ 1, st + 1);
      }
      if (busy) {
        i32x8 q[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) q[j] = qread(b, j);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const i32x8 p = pread(b, i);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const f32x4 d = block_product(q[j], p);
            const float s = ps[b][i] * qs[b][GATED ? j % 2 : 0];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s, acc[i][j][e]);
          }
        }
      }
    };
    for (int st = st0; st < st1; st += 2) {
      stage(0, st);
      if (st + 1 < st1) stage(1, st + 1);
    }
    if (parts > 1) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) *raw(t.slot, i, j) = acc[i][j];
      return;
    }
  }

  // ---- results ----
  // element e of acc[i][j]: row rowl(i), column coll(j) + e
  auto rowl = [&](int i) { return (wm * MI + i) * 16 + l16; };
  auto coll = [&](int j) { return (GATED ? (wn * (NJ / 2) + j / 2) * 16 : (wn * NJ + j) * 16) + 4 * quad; };
  {
    const bool fp16 = a.out_type == MOE_TYPE_FP16;
    uint16_t* outp = (uint16_t*)a.out;
    __syncthreads();  // the stages' LDS is free
    // LDS rows of `width` values, 16-byte chunks swizzled by the row
    auto put = [&](int width, int row, int col, f32x4 v) {
      const u32x2 h = {pack_half(fp16, v[0], v[1]), pack_half(fp16, v[2], v[3])};
      *(__attribute__((address_space(3))) u32x2*)(smem + row * width * 2 + 16 * ((col >> 3) ^ (row & (width / 8 - 1))) +
                                                  2 * (col & 7)) = h;
    };
    auto get = [&](int width, int row, int chunk) -> u32x4 {
      return *(__attribute__((address_space(3))) u32x4*)(smem + row * width * 2 + 16 * (chunk ^ (row & (width / 8 - 1))));
    };
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; j += GATED ? 2 : 1) {
        f32x4 v = acc[i][j];
        if constexpr (GATED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]) * acc[i][j + 1][e];
        }
        put(NO, rowl(i), coll(j), v);
      }
    __syncthreads();
    for (int x = tid; x < BM * (NO / 8); x += THREADS) {
      const int r = x / (NO / 8), c = x % (NO / 8);
      if (r < live && n0 + 8 * c < ncols)
        *reinterpret_cast<u32x4*>(outp + ((int64_t)row0 + r) * a.ldout + n0 + 8 * c) = get(NO, r, c);
    }
    if constexpr (GATED) {
      if (a.keep) {
        __syncthreads();
        // gate columns in the left half of the LDS rows, up in the right
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j) put(BN, rowl(i), coll(j) + (j % 2 ? NO : 0), acc[i][j]);
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

template <Pass PASS, Result RES, int BM, int BN, int WM, int WN>
void launch_tile8(const Fp8Args& a, hipStream_t s) {
  const int no = RES == Result::kGated ? BN / 2 : BN;
  const int tiles_n = ((RES == Result::kGated ? a.cols / 2 : a.cols) + no - 1) / no;
  const int tiles = row_tile_bound(a.rows, a.groups, BM) * tiles_n;
  const int blocks = (tiles + 7) / 8 * 8 + (a.splits > 1 ? split_units(BM, tiles, a.splits) + 8 : 0);
  const int joins = std::min(tiles, (BM == 256 ? 256 : 512) / 2);  // a split tile has at least two parts
  fp8_tile_kernel<PASS, RES, false, BM, BN, WM, WN><<<blocks, 64 * WM * WN, 0, s>>>(a);
  if (a.splits > 1) fp8_tile_kernel<PASS, RES, true, BM, BN, WM, WN><<<joins, 64 * WM * WN, 0, s>>>(a);
}

template <Pass PASS, Result RES>
void launch_family(const Fp8Args& a, const ProductPlan& p, hipStream_t s) {
  if (p.family == Family::kTile256)
    launch_tile8<PASS, RES, 256, 256, 2, 4>(a, s);
  else
    launch_tile8<PASS, RES, 128, 128, 2, 2>(a, s);
}

}  // namespace

void launch_fp8_tiles(const Fp8Args& a, const ProductPlan& p, Pass pass, Result res, hipStream_t s) {
  if (pass == Pass::kInputGrad)
    launch_family<Pass::kInputGrad, Result::kHalf>(a, p, s);
  else if (res == Result::kGated)
    launch_family<Pass::kForward, Result::kGated>(a, p, s);
  else
    launch_family<Pass::kForward, Result::kHalf>(a, p, s);
}

}  // namespace moe
