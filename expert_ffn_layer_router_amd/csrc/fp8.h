// Grouped products in 8-bit floating point (moe_fp8.h): the kernels' arguments,
// shared by the API and the kernel sources.
#pragma once

#include "moe_fp8.h"
#include "products.h"

namespace moe {

constexpr int kScaleBlock = 128;  // values that share a scale, along the contraction and (weights) across it
inline __host__ __device__ int scale_blocks(int n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// ProductArgs with codes of e4m3 as P and Q and the blocks' scales: pscale
// [stages][ldscale], where a stage is 128 of the contraction; qscale as its
// strides say.  `contract` is the length of one half's sums and `halves` their
// number: the gated backward pass contracts over the gate's and the up
// projection's columns in turn, each in whole blocks (P's rows have both, padded
// to blocks; w's rows follow each other).
struct Fp8Args : ProductArgs {
  int64_t ldscale = 0;
  int64_t qs_group = 0;  // from one group's scales to the next, in values, and so on:
  int64_t qs_half = 0;   // forward, gated: gate's to up's
  int64_t qs_cols = 0;   // 128 result columns
  int64_t qs_stage = 0;  // 128 of the contraction
  int halves = 1;
};

// Enqueue only.
void launch_fp8_tiles(const Fp8Args& a, const ProductPlan& p, Pass pass, Result res, hipStream_t s);
void launch_fp8_stream(const Fp8Args& a, Result res, hipStream_t s);
void launch_quantize_blocks(int rows, int k, int type, const uint16_t* x, int64_t ldx, uint8_t* codes, int64_t ldcodes,
                            float* scale, int64_t ldscale, hipStream_t s);
void launch_quantize_tiles(int matrices, int n, int k, int type, const uint16_t* x, uint8_t* codes, float* scale,
                           hipStream_t s);
// (dg, du) of the groups' rows from dh [rows][n] and the saved (g, u): into
// slopes [rows][2n] and as codes [rows][2 nb 128] (zeros behind either half's
// n columns) with scale [2 nb][ldscale]; either may be null
void launch_fp8_slopes(int rows, int n, int type, int act, const uint16_t* dh, int64_t lddh, const uint16_t* gate_up,
                       int64_t ldgu, const int32_t* offsets, int groups, uint16_t* slopes, int64_t ldslopes,
                       uint8_t* codes, float* scale, int64_t ldscale, hipStream_t s);

}  // namespace moe
