// Microscaled 4-bit floating point (OCP MX, format MXFP4) and the matrix products on 4-bit weights:
// the host-side launchers that the C ABI calls after validating its arguments.
//
// MXFP4: a row is cut into blocks of 32 columns, the last one padded with zeros, Cp = 32 ceil(C/32).
// A block holds one scale byte b (the value 2^(b - 127); 255 reads as NaN) and 32 e2m1 codes:
// bit 3 the sign, magnitudes {0, 1/2, 1, 3/2, 2, 3, 4, 6}. Codes lie two to a byte, the even column
// in the low nibble; codes [rows, Cp / 2] and scale bytes [rows, Cp / 32] are contiguous.
#pragma once

#include "common.h"

namespace aaac {

constexpr int kMxBlock = 32;

__host__ __device__ __forceinline__ int64_t mx_blocks(int64_t C) {
  return (C + kMxBlock - 1) / kMxBlock;
}

// A grid of `blocks` workgroups numbered by block_id(). A dimension of a grid holds fewer than 2^32
// threads (a launch of more is cut without an error), so long grids go over two; the last workgroups
// may then lie past `blocks`.
inline dim3 grid_of(int64_t blocks) {
  constexpr int64_t kRow = (int64_t)1 << 22;     // workgroups of at most 512 threads
  if (blocks <= kRow) return dim3((unsigned)blocks);
  return dim3((unsigned)kRow, (unsigned)((blocks + kRow - 1) / kRow));
}
__device__ __forceinline__ int64_t block_id() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

hipError_t launch_mxfp4_quantize(const void* X, int x_type, int64_t M, int64_t C, int64_t ldx,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t launch_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t C,
                                void* Y, int y_type, int64_t ldy, hipStream_t stream);

// One product call: y[t, r] = sum_c x[t, c] W[e(t)][r, c] for the rows t of expert e,
// offsets[e] <= t < offsets[e + 1] (offsets NULL: every row, one matrix). The offsets are clamped
// to [0, T] and to ascending order where they are read, so no value of theirs leads outside x or y.
struct MatmulArgs {
  const uint8_t* codes;        // [E, R, Cp / 2]
  const void* scales;          // MXFP4: bytes [E, R, Cp / 32]; packed: bf16 words [E, R, C / g]
  const uint8_t* bitmap;       // packed, S < g: [E, bitmap_stride]
  const uint16_t* tables;      // packed: [E, 2, n]
  int64_t bitmap_stride;
  int64_t R, C, Cp;
  int E;
  int log2g, log2S, n;
  const int32_t* offsets;      // [E + 1] on the device, or NULL
  const void* x;               // bf16 rows of ldx elements, or codes [T, Cp / 2]
  const uint8_t* x_scales;     // with codes: [T, Cp / 32]
  int64_t T, ldx;
  void* y;                     // [T, R] of y_type, rows of ldy elements
  int y_type;
  int64_t ldy;
  int y_vec;                   // four neighbours of a row go out in one store
  int y_row;                   // 16-bit y whose rows start on 16 bytes; 2: past the caches
  int split;                   // workgroups that share a tile's columns; their sums lie in parts
  float* parts;                // [split, T, part_row(R)], with split > 1
  int64_t row_blocks;          // set by the launcher: row blocks of one expert
  int64_t blocks;              // set by the launcher of tiles: workgroups that have one
  int x_rows;                  // set by the launcher: rows of x that the workgroup's LDS holds
};

__host__ __device__ __forceinline__ int64_t part_row(int64_t R) { return (R + 3) & ~(int64_t)3; }

// Token tiles of BN rows that a call can need at most: every expert's last tile may be partial.
inline int64_t token_tiles(const MatmulArgs& a, int BN) {
  if (!a.offsets) return (a.T + BN - 1) / BN;
  const int64_t e = a.E < a.T ? a.E : a.T;
  return a.T / BN + e;
}

// How a call is run. bn == 0: the few-row kernels with rt x 16 weight rows by nt x 16 rows of x a
// workgroup, `chunks` (4 or 1) chunks of columns a wave at a time. Else tiles of bm weight rows by bn
// rows of x, their columns split over `split` workgroups.
struct MatmulPlan {
  int bm, bn, split;
  int rt, nt, chunks;
};

enum MatmulKind { kMxBf16, kMxMxfp4, kPacked };

// can_split: a workspace for parts may be used.
MatmulPlan plan_matmul(const MatmulArgs& a, MatmulKind kind, bool can_split);
size_t parts_bytes(const MatmulArgs& a, const MatmulPlan& p);
hipError_t launch_matmul(MatmulArgs a, MatmulKind kind, const MatmulPlan& p, hipStream_t stream);

hipError_t launch_few_mxfp4(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream);
hipError_t launch_few_mx_bf16(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream);
hipError_t launch_few_packed(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream);
hipError_t launch_tile_mxfp4(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream);
hipError_t launch_tile_mx_bf16(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream);
hipError_t launch_tile_packed(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream);

}  // namespace aaac
