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

// A block computes BM x BN of a group's product on WM x WN waves, each a grid of
// 16 x 16 tiles, as the products of integer codes do (product_core.h: the ring of
// operand stages that direct global -> LDS copies fill, the swizzles, the split
// of the last round's tiles).  What differs:
//  - A stage is 128 of the contraction, one scale block, and one matrix-core
//    instruction takes all of it: its 16 x 16 products start from zero and are
//    added to the sums by FMA, times the row's and the columns' scale.  All
//    columns of a wave share a scale (they lie in one block of 128, in the gated
//    block in one of gate's and one of up's).
//  - Which 32 of the 128 a lane holds is free, as long as both operands agree:
//    contiguous ones give it chunks l / 16 and 4 + l / 16 of a row, and w in the
//    input gradient (contraction across its rows) the same ones of a column, by
//    the transposing read of 8-bit values.
//  - A lane of the result holds four columns of one row, so a row block's scales
//    are one register; a lane loads one row's in 64 and the lanes exchange them.
//
// What bounds it: the matrix cores' feeding (they are busy 66% of the cycles) and
// the clock, which power lowers.  At 8192^3 with random codes 432 us, 2545
// TFLOP/s forward, 2510 input gradient and gated (a large library product of
// plain 8-bit floats, without scales: 2630; integer codes by this library, 2840);
// with all codes zero, where nothing switches and the clock stays up, the same
// launch takes 321 us.  Registers alone, the products reach 4350 TFLOP/s and with the FMAs 3650; the
// FMAs cost 13% in the whole kernel too, the copies 25%, LDS reads 2%.  Each
// step, timed at that size:
//  - two buffers, copies and fragment reads after the barrier: 630 us;
//  - the ring of stages, copies and reads spread between the products, and a
//    tile's FMAs three tiles later: 455;
//  - one scale load in 64 lanes instead of one for every row block: 450;
//  - the hand-over to the next stage half way, not before the last two row
//    blocks, and five row fragments in registers, not four: 432.
// Rows that a group's last tile has not cost two thirds of what its rows do: 256
// tiles of 14336 contracted and 4096 columns take 213 us for 8 groups of 512 rows,
// 187 of 384, 176 of 257; 64 groups' input gradient, 2048 columns of 4096, 158 for
// 256 rows each, 223 for 257.
// No gain: raised wave priority for the products; two tiles between the
// schedule's fences; the last two row blocks together, for earlier Q reads; a
// group's last tile with its rows spread over all waves and only as many row
// blocks as it has (the units stay as many: 4096 rows over 8 groups and 4096
// columns are one round of 256 and 64 tiles in 4 parts, from which a unit that ends
// early takes nothing away; a remainder of up to 128 rows counted as half a unit
// would, which is not built); units dealt to the XCDs round by round; staggered starts;
// four stages of 128 x 128 ahead where tiles are few (a stage takes 0.6 us either
// way); 64 x 64 blocks of one wave there (300 rows, 4096 and 4096, input gradient:
// 26.5 -> 35.5 us); splitting their contraction earlier than ops_api.hip's rule
// (300 rows over 5, 1008 and 1424: 20.2 -> 22.3 us with the join).
template <Pass PASS, Result RES, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(Fp8Args a) {
  constexpr int NW = WM * WN, THREADS = 64 * NW;
  constexpr int MI = BM / 16 / WM, NJ = BN / 16 / WN;
  constexpr bool Q_STR = PASS == Pass::kInputGrad;
  constexpr bool GATED = RES == Result::kGated;
  constexpr int BK = kScaleBlock;  // contraction values, and bytes of a row, per stage
  constexpr int kPBytes = BM * BK, kQBytes = BN * BK;
  constexpr int kSlot = kPBytes;  // ring slot: one operand's stage
  constexpr int PI = kPBytes / 1024 / NW, QI = kQBytes / 1024 / NW;  // 1 KB copies per wave and stage
  constexpr int NO = GATED ? BN / 2 : BN;                            // result columns per block
  constexpr int NS = GATED ? 2 : 1;                                  // column scales of a wave
  static_assert(PI * NW * 1024 == kPBytes && QI * NW * 1024 == kQBytes, "even copy split");
  static_assert(!GATED || NJ % 2 == 0, "gate and up tiles in pairs");
  static_assert(NO % (16 * NJ / NS) == 0 && kScaleBlock % (16 * NJ / NS) == 0 && (!GATED || kScaleBlock % NO == 0),
                "a wave's columns share a scale");
  static_assert(PI == QI && BM * BN * 2 <= kRing * kSlot, "equal slots; the 16-bit result fits the ring");
  constexpr int R = MI == 8 ? 5 : 4;      // P fragments in registers
  constexpr int kTurn = MI == 8 ? 4 : 1;  // row blocks before the turn
  constexpr int kPCopies = (PI + kTurn - 1) / kTurn;                // P copies of a row block before it
  constexpr int kQCopies = (QI + MI - kTurn - 1) / (MI - kTurn);    // Q copies of one after it
  static_assert(kTurn >= MI - R && kTurn >= 1, "at the turn all of the stage's fragments are read");
  static_assert(MI >= R && NJ == 4 && PI == 4, "the rows' schedule");
  __shared__ __attribute__((aligned(1024))) char smem_raw[kRing * kSlot];
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
  if (!find_row_tile<BM, BN, THREADS, false>(a, tiles_n, stages, smem, t)) return;
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
  // ---- copies ----
  const char* pbase = a.p + (int64_t)row0 * a.ldp;
  const char* qbase = a.q + (int64_t)t.group * a.q_group + (Q_STR ? (int64_t)n0 : (int64_t)n0 * a.ldq);
  uint32_t pv[PI], qv[QI];  // byte offsets of this lane's copies, or kNoLoad
  // where this lane's c-th copy lies in the stage's contraction: contiguous
  // operands (LDS row r holds chunk c of 16 bytes at c ^ (r / 2) % 8), strided
  const int chunk0 = 16 * ((lane & 7) ^ (lane >> 4));
  auto chunk_at = [&](int c) { return chunk0 ^ (c & 1) * 64; };
  constexpr int cpr = BN / 16;  // strided: 16-byte chunks per LDS row
  auto q_at = [&](int c) { return (wave * QI + c) * (64 / cpr) + lane / cpr; };
  static_assert(PI % 2 == 0, "a wave's copies begin at a multiple of 16 rows");
#pragma unroll
  for (int c = 0; c < PI; ++c) {
    const int r = (wave * PI + c) * 8 + lane / 8;
    pv[c] = r < live ? (uint32_t)(r * a.ldp + chunk_at(c)) : kNoLoad;
  }
#pragma unroll
  for (int c = 0; c < QI; ++c) {
    if constexpr (Q_STR) {
      const int kr = q_at(c);
      const int fold = cpr == 16 ? (kr & 7) | (kr >> 1 & 8) : (kr >> 1 & 3) | (kr >> 2 & 4);
      const int chunk = (lane % cpr) ^ fold;
      qv[c] = n0 + 16 * chunk < ncols ? (uint32_t)(kr * a.ldq + 16 * chunk) : kNoLoad;
    } else {
      const int r = (wave * QI + c) * 8 + lane / 8;
      int src = r;
      if constexpr (GATED) {  // LDS row r: tile r / 16 belongs to wave column (r / 16) / NJ
        const int jb = r / 16;
        src = (jb / NJ * (NJ / 2) + jb % NJ / 2) * 16 + r % 16;
      }
      qv[c] = n0 + src < ncols ? (uint32_t)(src * a.ldq + chunk_at(c)) : kNoLoad;
    }
  }
  // The copies of an operand's stage: begin_p / begin_q set the descriptor
  // (and, in the contraction's last stage and past it, drop the lanes with
  // nothing to load: in place, so that the copies' offsets live in registers
  // of their own, and without a branch, behind which the compiler would gather
  // the additions), then copy_p(slot, c) is this wave's c-th copy.  The first
  // of two halves ends in whole blocks too: P's codes behind it are zeros, and
  // what Q's stage holds there are the second half's first rows (a half shorter
  // than a stage: as many as it has, which drops no lane that the second needs).
  const int plen = a.halves == 2 ? stages * BK : a.contract;  // of P's rows
  __amdgpu_buffer_rsrc_t pr, qr, ur;
  auto begin_p = [&](int st) {
    const int left = min(plen, st1 * BK) - st * BK;
#pragma unroll
    for (int c = 0; c < PI; ++c) pv[c] = chunk_at(c) < left ? pv[c] : kNoLoad;
    pr = buffer_at(pbase + (int64_t)st * BK);
  };
  auto begin_q = [&](int st) {
    const int half = st >= half_stages ? 1 : 0, in = st - half * half_stages;
    const int left = min(a.contract * (a.halves - half) - in * BK, (st1 - st) * BK);
#pragma unroll
    for (int c = 0; c < QI; ++c)
      qv[c] = (Q_STR ? q_at(0) : chunk_at(c)) < left - (Q_STR ? c * (64 / cpr) : 0) ? qv[c] : kNoLoad;
    const char* q = qbase + (Q_STR ? ((int64_t)half * a.contract + in * BK) * a.ldq : (int64_t)in * BK);
    qr = buffer_at(q);
    if (GATED) ur = buffer_at(q + (int64_t)F * a.ldq);
  };
  auto copy_p = [&](int slot, int c) { buffer_to_lds16(pr, smem + slot * kSlot + (wave * PI + c) * 1024, pv[c], 0); };
  auto copy_q = [&](int slot, int c) {  // gated: the copy's 8 rows are gate or up
    buffer_to_lds16(GATED && (wave * QI + c) / 2 % 2 ? ur : qr, smem + slot * kSlot + (wave * QI + c) * 1024, qv[c], 0);
  };

  // ---- scales ----
  const float* psb = a.pscale + row0;
  // (columns past the matrix take the first ones' scale: nothing of them is stored)
  const int qcol = GATED || n0 + wn * NJ * 16 >= ncols ? n0 : n0 + wn * NJ * 16;
  const float* qsb = a.qscale + (int64_t)t.group * a.qs_group + (int64_t)(qcol / kScaleBlock) * a.qs_cols;
  // a lane loads the scale of one row in 64, the lanes exchange them afterwards
  constexpr int kLoads = MI / 4;
  const uint32_t prow = (wm * MI * 16 + lane) * 4;
  float pn[kLoads], qn[NS];  // the next stage's
  float ps[MI], qs[NS];      // this one's
  auto load_p = [&](int st) {
    const __amdgpu_buffer_rsrc_t r = scales_at(psb + (int64_t)min(st, st1 - 1) * a.ldscale, live);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) pn[i] = load_scale(r, prow + i * 256);
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // lanes 16 r .. of pn[i] hold row block 4 i + r: (r0 r0 r2 r2), (r1 r1 r3 r3), then each of them everywhere
      const uint32_t v = __float_as_uint(pn[i]);
      const auto even = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      const auto lo = __builtin_amdgcn_permlane32_swap(even[0], even[0], false, false);
      const auto hi = __builtin_amdgcn_permlane32_swap(even[1], even[1], false, false);
      ps[4 * i] = __uint_as_float(lo[0]);
      ps[4 * i + 1] = __uint_as_float(hi[0]);
      ps[4 * i + 2] = __uint_as_float(lo[1]);
      ps[4 * i + 3] = __uint_as_float(hi[1]);
    }
#pragma unroll
    for (int h = 0; h < NS; ++h) qs[h] = qn[h];
  };
  auto load_q = [&](int st) {
#pragma unroll
    for (int h = 0; h < NS; ++h)
      qn[h] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          buffer_at((const char*)(qsb + h * a.qs_half + (int64_t)min(st, st1 - 1) * a.qs_stage)), 0, 0, 0));
  };

  // ---- fragments ----
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
  // contiguous: lane l reads chunks l / 16 and 4 + l / 16 of row (row block) + l % 16
  const int flo = l16 * BK + 16 * (quad ^ (l16 >> 1 & 7)), fhi = flo ^ 64;
  // strided: lane l reads half of 16 columns of row 16 (l / 16) + l % 16 / 2 (+ 8, + 64, + 72)
  int fat = 0;  // of column tile 0; another's differs in two bits of the chunk
  if constexpr (Q_STR) {
    const int kr = quad * 16 + (l16 >> 1);
    const int fold = BN == 256 ? (kr & 7) | (kr >> 1 & 8) : (kr >> 1 & 3) | (kr >> 2 & 4);
    fat = kr * BN + 16 * ((wn * NJ) ^ fold) + 8 * (l16 & 1);
  }
  auto pread = [&](int slot, int i) {
    lds_char* at = smem + slot * kSlot + (wm * MI + i) * 16 * BK;
    return join_halves(*(lds_u32x4*)(at + flo), *(lds_u32x4*)(at + fhi));
  };
  auto qread = [&](int slot, int j) {
    lds_char* at = smem + slot * kSlot;
    if constexpr (Q_STR) {
      at = smem + ((slot * kSlot + fat) ^ (16 * j));
      const u32x2 v0 = read_transposed8(at), v1 = read_transposed8(at + 8 * BN);
      const u32x2 v2 = read_transposed8(at + 64 * BN), v3 = read_transposed8(at + 72 * BN);
      return join_halves(u32x4{v0.x, v0.y, v1.x, v1.y}, u32x4{v2.x, v2.y, v3.x, v3.y});
    } else {
      at += (wn * NJ + j) * 16 * BK;
      return join_halves(*(lds_u32x4*)(at + flo), *(lds_u32x4*)(at + fhi));
    }
  };

  const int nst = st1 - st0;
  const bool busy = wm * MI * 16 < live;  // this wave has rows
  begin_p(st0);
#pragma unroll
  for (int c = 0; c < PI; ++c) copy_p(0, c);
  begin_q(st0);
#pragma unroll
  for (int c = 0; c < QI; ++c) copy_q(1, c);
  load_p(st0);
  load_q(st0);
  begin_p(st0 + 1);
#pragma unroll
  for (int c = 0; c < PI; ++c) copy_p(2, c);
  begin_q(st0 + 1);
#pragma unroll
  for (int c = 0; c < QI; ++c) copy_q(3, c);
  __builtin_amdgcn_sched_barrier(0);
  wait_copies<PI + QI>();
  lds_only_barrier();
  // Iteration i: slots pc and qc hold stage i, pnx and qnx stage i + 1, `spare`
  // is free and takes P's stage i + 2 during the first row blocks.  At the
  // turn (all of stage i's fragments are in registers by then) every wave has to
  // be done with stage i, and stage i + 1 to have landed: newer than its copies
  // are the next scales and P's stage i + 2.  Then pc takes Q's stage i + 2, and
  // qc is the next spare one.  A tile's products are added to the sums, scaled,
  // while the next three tiles' are under way.
  int pc = 0, qc = 1, pnx = 2, qnx = 3, spare = 4;
  auto rotate = [&]() {
    const int p = pc, q = qc;
    pc = pnx;
    qc = qnx;
    pnx = spare;
    qnx = p;
    spare = q;
  };
  if (busy) {
    i32x8 pf[R], qf[NJ];
    f32x4 d[4] = {};
    float sc[2][NS] = {};  // the scales of this row block and of the one before
#pragma unroll
    for (int j = 0; j < NJ; ++j) qf[j] = qread(qc, j);
#pragma unroll
    for (int i = 0; i < R; ++i) pf[i] = pread(pc, i);
    for (int i = 0; i < nst; ++i) {
      begin_p(st0 + i + 2);
      take_scales();
      load_p(st0 + i + 1);
      load_q(st0 + i + 1);
#pragma unroll
      for (int m = 0; m < MI; ++m) {
        if (m == kTurn) {
          wait_copies<PI + kLoads + NS>();
          lds_only_barrier();
          begin_q(st0 + i + 2);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            bool used = false;  // by a row block to come
            for (int to = kTurn; to < MI; ++to) used = used || to % R == r;
            if (!used) pf[r] = pread(pnx, r);
          }
        }
#pragma unroll
        for (int h = 0; h < NS; ++h) sc[m & 1][h] = ps[m] * qs[h];
#pragma unroll
        for (int c = kPCopies * m; c < kPCopies * (m + 1) && c < PI; ++c) copy_p(spare, c);
        if (m >= kTurn) {
#pragma unroll
          for (int c = kQCopies * (m - kTurn); c < kQCopies * (m - kTurn + 1) && c < QI; ++c) copy_q(pc, c);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          __builtin_amdgcn_sched_barrier(0);
          d[j] = block_product(qf[j], pf[m % R]);
          // the tile three before: of this row block, or of the one before
          const int b = (j + 1) % NJ, row = j == 3 ? m : (m + MI - 1) % MI;
          const float s = sc[row & 1][GATED ? b % 2 : 0];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[row][b][e] = fmaf(d[b][e], s, acc[row][b][e]);
          if (m == MI - 1) qf[j] = qread(qnx, j);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (m + R < MI) pf[m % R] = pread(pc, m + R);
        if (m >= kTurn) pf[m % R] = pread(pnx, m % R);
      }
      rotate();
    }
#pragma unroll
    for (int b = 1; b < NJ; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[MI - 1][b][e] = fmaf(d[b][e], sc[(MI - 1) & 1][GATED ? b % 2 : 0], acc[MI - 1][b][e]);
  } else {
    // a wave without rows only copies
    for (int i = 0; i < nst; ++i) {
      begin_p(st0 + i + 2);
#pragma unroll
      for (int c = 0; c < PI; ++c) copy_p(spare, c);
      wait_copies<PI>();
      lds_only_barrier();
      begin_q(st0 + i + 2);
#pragma unroll
      for (int c = 0; c < QI; ++c) copy_q(pc, c);
      rotate();
    }
  }
  wait_copies<0>();  // the zeros of stages past the end
  if (parts > 1) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) *raw(t.slot, i, j) = acc[i][j];
    return;
  }

  // ---- results ----
  // element e of acc[i][j]: row rowl(i), column coll(j) + e
  auto rowl = [&](int i) { return (wm * MI + i) * 16 + l16; };
  auto coll = [&](int j) { return (GATED ? (wn * (NJ / 2) + j / 2) * 16 : (wn * NJ + j) * 16) + 4 * quad; };
  const bool fp16 = a.out_type == MOE_TYPE_FP16;
  uint16_t* outp = (uint16_t*)a.out;
  // barriers that leave the stores in flight: nothing waits for them but the
  // kernel's end
  lds_only_barrier();  // the stages' LDS is free
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
  lds_only_barrier();
  for (int x = tid; x < BM * (NO / 8); x += THREADS) {
    const int r = x / (NO / 8), c = x % (NO / 8);
    if (r < live && n0 + 8 * c < ncols)
      *reinterpret_cast<u32x4*>(outp + ((int64_t)row0 + r) * a.ldout + n0 + 8 * c) = get(NO, r, c);
  }
  if constexpr (GATED) {
    if (a.keep) {
      lds_only_barrier();
      // gate columns in the left half of the LDS rows, up in the right; not to be
      // read before the backward pass, so the caches need not keep them
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) put(BN, rowl(i), coll(j) + (j % 2 ? NO : 0), acc[i][j]);
      lds_only_barrier();
      for (int x = tid; x < BM * (BN / 8); x += THREADS) {
        const int r = x / (BN / 8), c = x % (BN / 8);
        const int up = c >= NO / 8, col = n0 + 8 * (c - up * (NO / 8));
        if (r < live && col < F)
          __builtin_nontemporal_store(get(BN, r, c), reinterpret_cast<u32x4*>(
                                                         a.keep + ((int64_t)row0 + r) * a.ldkeep + up * F + col));
      }
    }
  }
}

// Adds the raw sums of a split tile's parts, in order, and writes the result:
// block (b, i) has the i-th 16 rows of each wave of the b-th split tile, so that
// all compute units take part (64 tiles of 256 x 256 in 4 parts: 20 us as one
// block a tile).
template <Result RES, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void fp8_join_kernel(Fp8Args a) {
  constexpr int THREADS = 64 * WM * WN, MI = BM / 16 / WM, NJ = BN / 16 / WN;
  constexpr bool GATED = RES == Result::kGated;
  constexpr int NO = GATED ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) char scratch[32];
  const int F = a.cols / 2, ncols = GATED ? F : a.cols;
  const int stages = a.halves * scale_blocks(a.contract);
  RowTile t;
  if (!find_row_tile<BM, BN, THREADS, true>(a, (ncols + NO - 1) / NO, stages, (lds_char*)scratch, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.y;
  const int row = t.row0 + (wave / WN * MI + i) * 16 + (lane & 15);
  if (row >= t.end) return;
  const f32x4* from = reinterpret_cast<const f32x4*>(a.partial) + ((int64_t)(wave * MI + i) * NJ) * 64 + lane;
  f32x4 v[NJ] = {};
  for (int s = 0; s < t.parts; ++s) {
    const f32x4* p = from + (int64_t)(t.slot + s * t.slot_step) * (BM * BN / 4);
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] += p[j * 64];
  }
  const bool fp16 = a.out_type == MOE_TYPE_FP16;
  auto store = [&](uint16_t* p, f32x4 x) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_half(fp16, x[0], x[1]), pack_half(fp16, x[2], x[3])};
  };
  const int c0 = t.tile_n * NO + wave % WN * (NO / WN) + 4 * (lane >> 4);
#pragma unroll
  for (int j = 0; j < NJ; j += GATED ? 2 : 1) {
    const int c = c0 + (GATED ? j / 2 : j) * 16;
    if (c >= ncols) continue;
    f32x4 x = v[j];
    if constexpr (GATED) {
      if (a.keep) {
        store(a.keep + (int64_t)row * a.ldkeep + c, x);
        store(a.keep + (int64_t)row * a.ldkeep + F + c, v[j + 1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = activate(a.act, x[e]) * v[j + 1][e];
    }
    store((uint16_t*)a.out + (int64_t)row * a.ldout + c, x);
  }
}

template <Pass PASS, Result RES, int BM, int BN, int WM, int WN>
void launch_tile8(const Fp8Args& a, hipStream_t s) {
  const int no = RES == Result::kGated ? BN / 2 : BN;
  const int tiles_n = ((RES == Result::kGated ? a.cols / 2 : a.cols) + no - 1) / no;
  const int tiles = row_tile_bound(a.rows, a.groups, BM) * tiles_n;
  const int blocks = (tiles + 7) / 8 * 8 + (a.splits > 1 ? split_units(BM, tiles, a.splits) + 8 : 0);
  const int joins = std::min(tiles, (BM == 256 ? 256 : 512) / 2);  // a split tile has at least two parts
  fp8_tile_kernel<PASS, RES, BM, BN, WM, WN><<<blocks, 64 * WM * WN, 0, s>>>(a);
  if (a.splits > 1) fp8_join_kernel<RES, BM, BN, WM, WN><<<dim3(joins, BM / 16 / WM), 64 * WM * WN, 0, s>>>(a);
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
