// Grouped products of expert feed-forward blocks (moe_ops.h): the kernels'
// arguments and host-side plans, shared by the API and the kernel sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_ops.h"

namespace moe {

enum class Num { kBf16, kFp16, kInt8 };                          // operand type
enum class Pass { kForward, kInputGrad, kWeightGrad };
enum class Result { kHalf, kGated, kWide };                      // 16-bit, act(g) u in 16 bits, fp32

// One grouped product out = P Q: P's rows are the result's rows, Q's the
// result's columns.  Strides in bytes, except those of the results (elements).
struct ProductArgs {
  const char* p = nullptr;         // forward: x or codes; input gradient: dy; weight gradient: dy
  const char* q = nullptr;         // forward, input gradient: w; weight gradient: x
  int64_t ldp = 0, ldq = 0;
  int64_t q_group = 0;             // bytes from one group's w to the next
  const int32_t* offsets = nullptr;
  int groups = 1, rows = 0;        // rows of the row matrices
  int contract = 0;                // forward, input gradient: length of the sums
  int cols = 0;                    // columns of the product (gated: 2F)
  int wrows = 0;                   // weight gradient: rows of a group's result
  void* out = nullptr;
  int64_t ldout = 0;
  int out_type = 0;                // moe_type
  uint16_t* keep = nullptr;        // gated: (g, u), or null
  int64_t ldkeep = 0;
  const float* pscale = nullptr;   // codes: scale of each row, of each w row ([groups][cols])
  const float* qscale = nullptr;
  int act = 0;
  // fp16 gradients of the gated block, or null: bits of each group's largest
  // slope if it passes 65504 (P then holds the slopes over group_lift), else 0
  const uint32_t* tops = nullptr;
  // contraction split: weight gradient, into this many parts; otherwise the
  // most parts that the kernels may choose (rounds_of), 1 if none can pay.
  // The parts' raw sums go to `partial`; a second launch joins them.
  int splits = 1;
  char* partial = nullptr;
};

enum class Family { kStream, kTile128, kTile256 };

struct ProductPlan {
  Family family = Family::kTile128;
  int splits = 1;
  size_t partial_bytes = 0;
};

// Row tiles a grid must hold: sum_e ceil(rows_e / bm) is at most this.
__host__ __device__ inline int row_tile_bound(int rows, int groups, int bm) {
  return (rows + bm - 1) / bm + (rows < groups ? rows : groups) - (rows > 0 ? 1 : 0);
}
// Parts of split tiles that a product of at most `tiles` tiles can have.
inline int split_units(int bm, int tiles, int max_parts) {
  const int slots = bm == 256 ? 256 : 512;
  return (int64_t)tiles * max_parts < slots ? tiles * max_parts : slots;
}

// Pure host arithmetic.
ProductPlan plan_product(Num num, Pass pass, Result res, const ProductArgs& a);

// Enqueue only.
void launch_product_int8(const ProductArgs& a, const ProductPlan& p, Result res, hipStream_t s);
void launch_product_half(const ProductArgs& a, const ProductPlan& p, Num num, Result res, hipStream_t s);
void launch_product_grad(const ProductArgs& a, const ProductPlan& p, Num num, Pass pass, Result res, hipStream_t s);
void launch_product_stream(const ProductArgs& a, Num num, Result res, hipStream_t s);
void launch_quantize(int rows, int k, int type, const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldcodes,
                     float* scale, hipStream_t s);
// (dg, du) [rows][2n] of the groups' rows from dh [rows][n] and the saved (g, u);
// fp16: tops [groups] receives what ProductArgs::tops says, else it is null
void launch_gated_slopes(int rows, int n, int type, int act, const uint16_t* dh, int64_t lddh, const uint16_t* gate_up,
                         int64_t ldgu, const int32_t* offsets, int groups, uint16_t* dgu, uint32_t* tops, hipStream_t s);

}  // namespace moe
