// MXFP4 quantisation and its inverse (OCP MX: blocks of 32 with a power-of-two scale).
//
// quantise: with top = max |x| over the block, e = clamp(floor(log2 top) - 2, -127, 127), so that
// the block's largest magnitude lies in [4, 8) after scaling; scale byte e + 127, code = the e2m1
// value nearest to x 2^-e (ties to the even code, magnitudes above 6 become 6). floor(log2 top) is
// the exponent field of top, x 2^-e is exact in fp32 (a subnormal result is far below 1/4 and
// rounds to zero either way), so the conversion's rounding is the only one. A block that holds an
// infinity or a NaN has no finite scale: it stores byte 255 and zero codes and reads back as NaN.
//
// Both directions move each byte once and are bound by memory: 13824 x 5120 bf16 takes 38 us one way
// (4.7 TB/s of the 5.2 that a copy reaches) and 26 us the other (6.7 TB/s, codes partly from the cache).
// Eight columns a lane make a block four neighbouring lanes, whose maximum two lane permutes find.
#include "aaac.h"
#include "mxfp4.h"

namespace aaac {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kMxLane = 8;                       // columns per lane: four lanes make a block
constexpr int kMxSteps = 4;                      // lane rows in flight per thread

template <int TYPE> struct Elem;
template <> struct Elem<AAAC_BF16> { typedef uint16_t T; };
template <> struct Elem<AAAC_F16> { typedef uint16_t T; };
template <> struct Elem<AAAC_F32> { typedef uint32_t T; };

template <int TYPE>
__device__ __forceinline__ float to_f32(typename Elem<TYPE>::T v) {
  if (TYPE == AAAC_F32) return __uint_as_float((uint32_t)v);
  if (TYPE == AAAC_BF16) return __uint_as_float((uint32_t)v << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
}

// Eight consecutive elements as fp32; those at or past `valid` read as zero. Eight inside the row are
// read in 16-byte words, aligned (VEC) or not (1003 x 5003 in fp32: 6.7 us, 14.5 element by element).
template <int TYPE, bool VEC>
__device__ __forceinline__ void load8(const typename Elem<TYPE>::T* p, int valid, float (&v)[8]) {
  typedef typename Elem<TYPE>::T T;
  if (VEC || valid == 8) {
    if (sizeof(T) == 2) {
      uint4 u;
      if (VEC) u = *reinterpret_cast<const uint4*>(p);
      else __builtin_memcpy(&u, p, 16);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = to_f32<TYPE>((T)(w[k] & 0xffffu));
        v[2 * k + 1] = to_f32<TYPE>((T)(w[k] >> 16));
      }
    } else {
      uint4 a, b;
      if (VEC) {
        a = reinterpret_cast<const uint4*>(p)[0];
        b = reinterpret_cast<const uint4*>(p)[1];
      } else {
        __builtin_memcpy(&a, p, 16);
        __builtin_memcpy(&b, p + 4, 16);
      }
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < valid ? to_f32<TYPE>(p[k]) : 0.0f;
  }
}

__device__ __forceinline__ void encode8(const float (&v)[8], uint32_t& word, uint32_t& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
  top = max(top, dpp_u32<kDppQuadXor1>(top));
  top = max(top, dpp_u32<kDppQuadXor2>(top));
  const uint32_t field = top >> 23;
  const bool bad = field == 255u;
  byte = bad ? 255u : (field > 2u ? field - 2u : 0u);
  const float mul = __uint_as_float((254u - (bad ? 127u : byte)) << 23);
  word = 0;
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[0] * mul, v[1] * mul, 1.0f, 0);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[2] * mul, v[3] * mul, 1.0f, 1);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[4] * mul, v[5] * mul, 1.0f, 2);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[6] * mul, v[7] * mul, 1.0f, 3);
  if (bad) word = 0;
}

// FLAT: rows are contiguous multiples of 32 columns, so the lanes walk one long row. Otherwise a
// lane finds its row by a division.
template <int TYPE, bool VEC, bool FLAT>
__global__ __launch_bounds__(kBlock) void mxfp4_quantize_kernel(
    const typename Elem<TYPE>::T* __restrict__ X, int64_t C, int64_t ldx, int64_t lanes_per_row,
    int64_t total, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t i0 = block_id() * (kBlock * kMxSteps) + threadIdx.x;
  float v[kMxSteps][8];
#pragma unroll
  for (int u = 0; u < kMxSteps; ++u) {
    const int64_t i = i0 + (int64_t)u * kBlock;
    if (i < total) {
      if (FLAT) {
        load8<TYPE, true>(X + i * kMxLane, 8, v[u]);
      } else {
        const int64_t r = total <= 0xffffffffll
                              ? (int64_t)((uint32_t)i / (uint32_t)lanes_per_row) : i / lanes_per_row;
        const int64_t c = (i - r * lanes_per_row) * kMxLane;
        const int64_t left = C - c;
        const int valid = left > 8 ? 8 : (left > 0 ? (int)left : 0);
        if (VEC && valid == 8) load8<TYPE, true>(X + r * ldx + c, 8, v[u]);
        else load8<TYPE, false>(X + r * ldx + c, valid, v[u]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kMxSteps; ++u) {
    const int64_t i = i0 + (int64_t)u * kBlock;
    if (i < total) {                             // total is a multiple of 4: whole quads leave
      uint32_t word, byte;
      encode8(v[u], word, byte);
      codes[i] = word;
      if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(typename Elem<TYPE>::T* p, bool vec, int valid,
                                       const float (&v)[8]) {
  typedef typename Elem<TYPE>::T T;
  if (TYPE == AAAC_F32) {
    if (vec) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (valid == 8) {
      __builtin_memcpy(p, v, 32);
    } else {
      for (int k = 0; k < 8; ++k)
        if (k < valid) p[k] = (T)__float_as_uint(v[k]);
    }
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const f32x2 f = {v[2 * k], v[2 * k + 1]};
    if (TYPE == AAAC_BF16) w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
    else w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
  }
  if (vec) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (valid == 8) {
    __builtin_memcpy(p, w, 16);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < valid) p[k] = (T)(w[k >> 1] >> (16 * (k & 1)));
  }
}

template <int TYPE, bool FLAT>
__global__ __launch_bounds__(kBlock) void mxfp4_dequant_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t C, int64_t ldy,
    int64_t lanes_per_row, int64_t total, bool vec, typename Elem<TYPE>::T* __restrict__ Y) {
  const int64_t i0 = block_id() * (kBlock * kMxSteps) + threadIdx.x;
  uint32_t word[kMxSteps], byte[kMxSteps];
#pragma unroll
  for (int u = 0; u < kMxSteps; ++u) {
    const int64_t i = i0 + (int64_t)u * kBlock;
    if (i < total) {
      word[u] = codes[i];
      byte[u] = scales[i >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kMxSteps; ++u) {
    const int64_t i = i0 + (int64_t)u * kBlock;
    if (i >= total) break;
    const uint32_t b = byte[u];
    // 2^(b - 127): byte 0 is the subnormal 2^-127, byte 255 a NaN
    const float s = __uint_as_float(b == 0 ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23));
    float v[8];
    const f32x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], 1.0f, 0);
    const f32x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], 1.0f, 1);
    const f32x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], 1.0f, 2);
    const f32x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], 1.0f, 3);
    v[0] = a0.x * s; v[1] = a0.y * s; v[2] = a1.x * s; v[3] = a1.y * s;
    v[4] = a2.x * s; v[5] = a2.y * s; v[6] = a3.x * s; v[7] = a3.y * s;
    if (FLAT) {
      store8<TYPE>(Y + i * kMxLane, true, 8, v);
    } else {
      const int64_t r = total <= 0xffffffffll
                            ? (int64_t)((uint32_t)i / (uint32_t)lanes_per_row) : i / lanes_per_row;
      const int64_t c = (i - r * lanes_per_row) * kMxLane;
      const int64_t left = C - c;
      const int valid = left > 8 ? 8 : (left > 0 ? (int)left : 0);
      store8<TYPE>(Y + r * ldy + c, vec && valid == 8, valid, v);
    }
  }
}

template <int TYPE>
hipError_t quantize_t(const void* X, int64_t M, int64_t C, int64_t ldx, uint8_t* codes,
                      uint8_t* scales, hipStream_t stream) {
  typedef typename Elem<TYPE>::T T;
  const T* x = static_cast<const T*>(X);
  const int64_t lpr = mx_blocks(C) * 4, total = M * lpr;
  const bool vec = ((uintptr_t)X % 16 == 0) && (ldx * sizeof(T)) % 16 == 0;
  const bool flat = vec && C % kMxBlock == 0 && (ldx == C || M == 1);
  const int64_t per = kBlock * kMxSteps;
  const dim3 grid = grid_of((total + per - 1) / per);
  uint32_t* cw = reinterpret_cast<uint32_t*>(codes);
  if (flat)
    hipLaunchKernelGGL((mxfp4_quantize_kernel<TYPE, true, true>), grid, dim3(kBlock), 0, stream, x,
                       C, ldx, lpr, total, cw, scales);
  else if (vec)
    hipLaunchKernelGGL((mxfp4_quantize_kernel<TYPE, true, false>), grid, dim3(kBlock), 0, stream,
                       x, C, ldx, lpr, total, cw, scales);
  else
    hipLaunchKernelGGL((mxfp4_quantize_kernel<TYPE, false, false>), grid, dim3(kBlock), 0, stream,
                       x, C, ldx, lpr, total, cw, scales);
  return hipGetLastError();
}

template <int TYPE>
hipError_t dequant_t(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t C, void* Y,
                     int64_t ldy, hipStream_t stream) {
  typedef typename Elem<TYPE>::T T;
  T* y = static_cast<T*>(Y);
  const int64_t lpr = mx_blocks(C) * 4, total = M * lpr;
  const bool vec = ((uintptr_t)Y % 16 == 0) && (ldy * sizeof(T)) % 16 == 0;
  const bool flat = vec && C % kMxBlock == 0 && (ldy == C || M == 1);
  const int64_t per = kBlock * kMxSteps;
  const dim3 grid = grid_of((total + per - 1) / per);
  const uint32_t* cw = reinterpret_cast<const uint32_t*>(codes);
  if (flat)
    hipLaunchKernelGGL((mxfp4_dequant_kernel<TYPE, true>), grid, dim3(kBlock), 0, stream, cw,
                       scales, C, ldy, lpr, total, vec, y);
  else
    hipLaunchKernelGGL((mxfp4_dequant_kernel<TYPE, false>), grid, dim3(kBlock), 0, stream, cw,
                       scales, C, ldy, lpr, total, vec, y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* X, int x_type, int64_t M, int64_t C, int64_t ldx,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  if (x_type == AAAC_BF16) return quantize_t<AAAC_BF16>(X, M, C, ldx, codes, scales, stream);
  if (x_type == AAAC_F16) return quantize_t<AAAC_F16>(X, M, C, ldx, codes, scales, stream);
  return quantize_t<AAAC_F32>(X, M, C, ldx, codes, scales, stream);
}

hipError_t launch_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t C,
                                void* Y, int y_type, int64_t ldy, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  if (y_type == AAAC_BF16) return dequant_t<AAAC_BF16>(codes, scales, M, C, Y, ldy, stream);
  if (y_type == AAAC_F16) return dequant_t<AAAC_F16>(codes, scales, M, C, Y, ldy, stream);
  return dequant_t<AAAC_F32>(codes, scales, M, C, Y, ldy, stream);
}

}  // namespace aaac
