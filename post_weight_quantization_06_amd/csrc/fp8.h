// 8-bit floating point in blocks of 128 and the routing of rows to experts: the host-side launchers
// that the C ABI calls after validating its arguments.
//
// FP8: e4m3 codes (1 sign, 4 exponent, 3 fraction bits, the largest value 448, 0x7f and 0xff NaN) with
// one fp32 scale for each block: 128 columns of a row, or a tile of 128 rows by 128 columns of a weight
// matrix; the last blocks of a row and of a matrix may be short.
#pragma once

#include "mxfp4.h"

namespace aaac {

constexpr int kFp8Block = 128;

__host__ __device__ __forceinline__ int64_t fp8_blocks(int64_t n) {
  return (n + kFp8Block - 1) / kFp8Block;
}

// Codes of X [E, M, C] (rows of ldx elements, matrices `stride_x` apart): whole 16-byte pieces up to
// column Cw (a multiple of 16 in [C, ldq]) are written, zeros past C. scales: element (row or tile row
// m, block b) at m * s_row + b * s_blk. tile: 128 x 128 blocks, else E is 1.
hipError_t launch_fp8_quantize(const void* X, int x_type, int64_t E, int64_t M, int64_t C,
                               int64_t ldx, int64_t stride_x, bool tile, uint8_t* codes, int64_t ldq,
                               int64_t Cw, float* scales, int64_t s_row, int64_t s_blk,
                               hipStream_t stream);
hipError_t launch_fp8_dequant(const uint8_t* codes, int64_t ldq, const float* scales, int64_t E,
                              int64_t M, int64_t C, bool tile, void* Y, int y_type, int64_t ldy,
                              hipStream_t stream);

struct RouteArgs {
  const void* logits;          // [T, E], rows of ldl elements
  int type;
  int64_t T, ldl;
  int E, k;
  const float* bias;           // [E] or NULL
  bool sigmoid, renormalize;
  int groups, top_groups, group_top;
  float scale;
  int32_t* experts;            // [T, k]
  float* weights;              // [T, k]
  int32_t* offsets;            // [E + 1]
  int32_t* rows;               // [T k]
  int32_t* places;             // [T, k]
  int32_t* counts;             // [blocks, E up to whole fours]: a block's rows of each expert; unused with one block
  int per_block;               // tokens of a block, set by the launcher
  bool vec;                    // set by the launcher: a lane's logits lie on their whole size
};

constexpr int kMaxExperts = 512, kMaxGroups = 64, kMaxChoices = 64;

size_t route_workspace_bytes(int64_t T, int E);
hipError_t launch_route(RouteArgs a, hipStream_t stream);

// out[places[t, j]] = x[t], rows of `bytes` bytes; strides in bytes.
hipError_t launch_rows_to_experts(const void* x, int64_t T, int64_t bytes, int64_t ldx,
                                  const int32_t* places, int k, void* out, int64_t N, int64_t ldo,
                                  int element, hipStream_t stream);
// out[t] = sum_j weights[t, j] y[places[t, j]].
hipError_t launch_rows_from_experts(const void* y, int type, int64_t N, int64_t C, int64_t ldy,
                                    const int32_t* places, const float* weights, int64_t T, int k,
                                    void* out, int out_type, int64_t ldo, hipStream_t stream);

}  // namespace aaac
