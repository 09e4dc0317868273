// Quantisation to 8-bit floating point (e4m3) in blocks of 128, and its inverse.
//
// quantise: scale = max(top / 448, 2^-126) in fp32 with top = max |x| over the block, code = the e4m3
// value nearest to the fp32 quotient x / scale, ties to even. The smallest normal number as the least
// scale keeps the quotient's divisor and its reciprocal normal and a block of zeros free of 0 / 0. The
// quotient never passes 448 by as much as half a step, so nothing saturates. A block with an infinity or
// a NaN has no finite scale: its scale and codes are NaN and all of it reads back as NaN.
//
// Both directions move each byte once and are bound by memory.
#include "aaac.h"
#include "fp8.h"
#include "fp8_encode.h"

namespace aaac {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kSteps = 2;                        // lane pieces in flight per thread
constexpr int kCols = 16;                        // columns a lane

__device__ __forceinline__ int64_t divide(int64_t i, int64_t n, int64_t total) {
  return total <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)n) : i / n;
}

// Blocks of 1 x 128. 16 columns a lane, so that a store of codes is 16 bytes (4096 x 4096 of bf16: 13 us, 9.6 of
// it the bytes' at a copy's rate, with 8 columns a lane 15; 1003 x 5003 of fp32 8.0, with 4 columns 9.6).
template <int TYPE, bool VEC>
__global__ __launch_bounds__(kBlock) void fp8_quantize_rows_kernel(
    const typename Elem<TYPE>::T* __restrict__ X, int64_t C, int64_t ldx, int64_t per_row,
    int64_t total, uint8_t* __restrict__ codes, int64_t ldq, int64_t Cw, float* __restrict__ scales,
    int64_t s_row, int64_t s_blk) {
  constexpr int V = kCols, kLanes = kFp8Block / V;
  const int64_t i0 = block_id() * (kBlock * kSteps) + threadIdx.x;
  float v[kSteps][V];
  int64_t row[kSteps], col[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t i = i0 + u * kBlock;
    if (i >= total) break;
    row[u] = divide(i, per_row, total);
    col[u] = (i - row[u] * per_row) * V;
    const int64_t left = C - col[u];
    load_lane<TYPE, VEC>(X + row[u] * ldx + col[u], left > V ? V : left < 0 ? 0 : (int)left, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    if (i0 + u * kBlock >= total) break;         // total is a multiple of kLanes: whole blocks leave
    const float s = scale_of(block_max_u32_t<kLanes>(top_bits(v[u]), kLanes));
    const int64_t left = C - col[u];
    if (col[u] < Cw) store_codes(v[u], s, left > V ? V : (int)left, codes + row[u] * ldq + col[u]);
    if (threadIdx.x % kLanes == 0) scales[row[u] * s_row + col[u] / kFp8Block * s_blk] = s;
  }
}

// Blocks of 128 x 128, one a workgroup, which holds it in registers between its maximum and its codes. 4096 x
// 14336 of bf16: 37 us, 4.8 TB/s (with 8 columns a lane 41); 4096 x 14335 44, tiles in turn over the dies 50.
template <int TYPE, bool VEC>
__global__ __launch_bounds__(kBlock) void fp8_quantize_tiles_kernel(
    const typename Elem<TYPE>::T* __restrict__ X, int64_t M, int64_t C, int64_t ldx, int64_t stride_x,
    int64_t tiles, uint8_t* __restrict__ codes, int64_t ldq, int64_t Cw, float* __restrict__ scales) {
  constexpr int V = kCols, kLanes = kFp8Block / V, kRows = kBlock / kLanes, kEach = kFp8Block / kRows;
  __shared__ uint32_t tops[kWavesPerBlock];
  if (block_id() >= tiles) return;
  const int64_t id = by_die(block_id(), tiles);  // neighbours share lines that rows start in
  const int64_t cb = fp8_blocks(C), rb = fp8_blocks(M);
  const int64_t e = id / (cb * rb), tr = id / cb % rb, tc = id % cb;
  const int64_t col = tc * kFp8Block + threadIdx.x % kLanes * V;
  const int64_t row0 = tr * kFp8Block + threadIdx.x / kLanes, left = C - col;
  const int valid = left > V ? V : left < 0 ? 0 : (int)left;
  float v[kEach][V];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int64_t r = row0 + u * kRows;
    load_lane<TYPE, VEC>(X + e * stride_x + r * ldx + col, r < M ? valid : 0, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) top = max(top, top_bits(v[u]));
  top = block_max_u32_t<kWave>(top, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) tops[wave_index()] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const float s = scale_of(top);
  if (threadIdx.x == 0) scales[id] = s;
  if (col >= Cw) return;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int64_t r = row0 + u * kRows;
    if (r >= M) break;
    store_codes(v[u], s, valid, codes + (e * M + r) * ldq + col);
  }
}

// per: rows that share a row of scales (128 with tiles, else 1). VEC: rows of Y start on 16 bytes; CV:
// rows of codes do. Values are the fp32 products of code and scale, rounded once more to a 16-bit type.
// fp32 values leave 16 bytes a lane, so that a wave's stores lie together (1003 x 5003: 7.9 us, with 64 bytes
// a lane 12.7); in 16 bits 32 bytes a lane are as good (4096 x 14336: 27 us, with 16 bytes a lane 30).
template <int TYPE> constexpr int kOutCols = TYPE == AAAC_F32 ? 4 : 16;
template <int TYPE> constexpr int kOutSteps = TYPE == AAAC_F32 ? 4 : 2;
template <int TYPE, bool VEC, bool CV>
__global__ __launch_bounds__(kBlock) void fp8_dequant_kernel(
    const uint8_t* __restrict__ codes, int64_t ldq, const float* __restrict__ scales, int64_t M,
    int64_t C, int per, int64_t per_row, int64_t total, typename Elem<TYPE>::T* __restrict__ Y,
    int64_t ldy) {
  typedef typename Elem<TYPE>::T T;
  constexpr int V = kOutCols<TYPE>, kWords = V / 4, kOut = V * sizeof(T) / 16, kSteps = kOutSteps<TYPE>;
  const int64_t i0 = block_id() * (kBlock * kSteps) + threadIdx.x;
  const int64_t cb = fp8_blocks(C), rb = (M + per - 1) / per;
  uint32_t w[kSteps][kWords];
  float s[kSteps];
  int64_t row[kSteps], col[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t i = i0 + u * kBlock;
    if (i >= total) break;
    row[u] = divide(i, per_row, total);
    col[u] = (i - row[u] * per_row) * V;
    const uint8_t* p = codes + row[u] * ldq + col[u];
    const int64_t left = C - col[u];
    if (left >= V) {
      if (CV) __builtin_memcpy(w[u], __builtin_assume_aligned(p, V), V);
      else __builtin_memcpy(w[u], p, V);
    } else {
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[u][k] = 0;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < left) w[u][k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
    }
    int64_t at = row[u];
    if (per > 1) {
      const int64_t e = divide(row[u], M, total);
      at = e * rb + (row[u] - e * M) / per;
    }
    s[u] = scales[at * cb + col[u] / kFp8Block];
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    if (i0 + u * kBlock >= total) break;
    float v[V];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][k], false);
      const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][k], true);
      v[4 * k] = a.x * s[u];
      v[4 * k + 1] = a.y * s[u];
      v[4 * k + 2] = b.x * s[u];
      v[4 * k + 3] = b.y * s[u];
    }
    Words4 o[kOut];
#pragma unroll
    for (int k = 0; k < 4 * kOut; ++k) {
      if (TYPE == AAAC_F32) {
        o[k >> 2][k & 3] = __float_as_uint(v[k]);
      } else {
        const f32x2 f = {v[(2 * k) % V], v[(2 * k + 1) % V]};
        o[k >> 2][k & 3] = TYPE == AAAC_BF16
                               ? __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2))
                               : __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
      }
    }
    T* p = Y + row[u] * ldy + col[u];
    const int64_t left = C - col[u];
    if (left >= V) {
#pragma unroll
      for (int k = 0; k < kOut; ++k) {
        if (VEC) reinterpret_cast<Words4*>(p)[k] = o[k];
        else __builtin_memcpy(reinterpret_cast<uint8_t*>(p) + 16 * k, &o[k], 16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < left)
          p[k] = sizeof(T) == 4 ? (T)o[0][k & 3] : (T)(o[(k >> 3) % kOut][(k >> 1) & 3] >> (16 * (k & 1)));
    }
  }
}

template <int TYPE>
hipError_t quantize_t(const void* X, int64_t E, int64_t M, int64_t C, int64_t ldx, int64_t stride_x,
                      bool tile, uint8_t* codes, int64_t ldq, int64_t Cw, float* scales, int64_t s_row,
                      int64_t s_blk, hipStream_t stream) {
  typedef typename Elem<TYPE>::T T;
  const T* x = static_cast<const T*>(X);
  const bool vec = (uintptr_t)X % 16 == 0 && (ldx * sizeof(T)) % 16 == 0 && (stride_x * sizeof(T)) % 16 == 0;
  if (tile) {
    const int64_t tiles = E * fp8_blocks(M) * fp8_blocks(C);
    if (vec)
      hipLaunchKernelGGL((fp8_quantize_tiles_kernel<TYPE, true>), grid_of(tiles), dim3(kBlock), 0,
                         stream, x, M, C, ldx, stride_x, tiles, codes, ldq, Cw, scales);
    else
      hipLaunchKernelGGL((fp8_quantize_tiles_kernel<TYPE, false>), grid_of(tiles), dim3(kBlock), 0,
                         stream, x, M, C, ldx, stride_x, tiles, codes, ldq, Cw, scales);
    return hipGetLastError();
  }
  const int64_t per_row = fp8_blocks(C) * (kFp8Block / kCols), total = M * per_row;
  const dim3 grid = grid_of((total + kBlock * kSteps - 1) / (kBlock * kSteps));
  if (vec)
    hipLaunchKernelGGL((fp8_quantize_rows_kernel<TYPE, true>), grid, dim3(kBlock), 0, stream, x, C, ldx,
                       per_row, total, codes, ldq, Cw, scales, s_row, s_blk);
  else
    hipLaunchKernelGGL((fp8_quantize_rows_kernel<TYPE, false>), grid, dim3(kBlock), 0, stream, x, C,
                       ldx, per_row, total, codes, ldq, Cw, scales, s_row, s_blk);
  return hipGetLastError();
}

template <int TYPE>
hipError_t dequant_t(const uint8_t* codes, int64_t ldq, const float* scales, int64_t E, int64_t M,
                     int64_t C, bool tile, void* Y, int64_t ldy, hipStream_t stream) {
  typedef typename Elem<TYPE>::T T;
  T* y = static_cast<T*>(Y);
  const bool vec = (uintptr_t)Y % 16 == 0 && (ldy * sizeof(T)) % 16 == 0;
  const bool cv = (uintptr_t)codes % 16 == 0 && ldq % 16 == 0;
  const int64_t per_row = (C + kOutCols<TYPE> - 1) / kOutCols<TYPE>, total = E * M * per_row;
  const int64_t each = kBlock * kOutSteps<TYPE>;
  const dim3 grid = grid_of((total + each - 1) / each);
  const int per = tile ? kFp8Block : 1;
  if (vec && cv)
    hipLaunchKernelGGL((fp8_dequant_kernel<TYPE, true, true>), grid, dim3(kBlock), 0, stream, codes,
                       ldq, scales, M, C, per, per_row, total, y, ldy);
  else if (cv)
    hipLaunchKernelGGL((fp8_dequant_kernel<TYPE, false, true>), grid, dim3(kBlock), 0, stream, codes,
                       ldq, scales, M, C, per, per_row, total, y, ldy);
  else
    hipLaunchKernelGGL((fp8_dequant_kernel<TYPE, false, false>), grid, dim3(kBlock), 0, stream, codes,
                       ldq, scales, M, C, per, per_row, total, y, ldy);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const void* X, int x_type, int64_t E, int64_t M, int64_t C, int64_t ldx,
                               int64_t stride_x, bool tile, uint8_t* codes, int64_t ldq, int64_t Cw,
                               float* scales, int64_t s_row, int64_t s_blk, hipStream_t stream) {
  if (E * M == 0) return hipSuccess;
  if (x_type == AAAC_BF16)
    return quantize_t<AAAC_BF16>(X, E, M, C, ldx, stride_x, tile, codes, ldq, Cw, scales, s_row, s_blk,
                                 stream);
  if (x_type == AAAC_F16)
    return quantize_t<AAAC_F16>(X, E, M, C, ldx, stride_x, tile, codes, ldq, Cw, scales, s_row, s_blk,
                                stream);
  return quantize_t<AAAC_F32>(X, E, M, C, ldx, stride_x, tile, codes, ldq, Cw, scales, s_row, s_blk,
                              stream);
}

hipError_t launch_fp8_dequant(const uint8_t* codes, int64_t ldq, const float* scales, int64_t E,
                              int64_t M, int64_t C, bool tile, void* Y, int y_type, int64_t ldy,
                              hipStream_t stream) {
  if (E * M == 0) return hipSuccess;
  if (y_type == AAAC_BF16)
    return dequant_t<AAAC_BF16>(codes, ldq, scales, E, M, C, tile, Y, ldy, stream);
  if (y_type == AAAC_F16)
    return dequant_t<AAAC_F16>(codes, ldq, scales, E, M, C, tile, Y, ldy, stream);
  return dequant_t<AAAC_F32>(codes, ldq, scales, E, M, C, tile, Y, ldy, stream);
}

}  // namespace aaac
