// The FP8 encoder (fp8.hip describes the format's rounding), shared by the quantiser and by the products
// that quantise few rows of x themselves. A lane holds V neighbouring columns.
#pragma once

#include "aaac.h"
#include "fp8.h"

namespace aaac {

namespace {

typedef uint32_t Words4 __attribute__((ext_vector_type(4)));

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

// V consecutive elements, whole 16-byte words, as fp32; those at or past `valid` read as zero. VEC: p is
// aligned to 16 bytes.
template <int TYPE, bool VEC, int V>
__device__ __forceinline__ void load_lane(const typename Elem<TYPE>::T* p, int valid, float (&v)[V]) {
  typedef typename Elem<TYPE>::T T;
  if (valid < V) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < valid ? to_f32<TYPE>(p[i]) : 0.0f;
    return;
  }
  constexpr int kWords = V * sizeof(T) / 16;
  Words4 w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if (VEC) w[i] = reinterpret_cast<const Words4*>(p)[i];
    else __builtin_memcpy(&w[i], reinterpret_cast<const uint8_t*>(p) + 16 * i, 16);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (sizeof(T) == 4) v[i] = __uint_as_float(w[i >> 2][i & 3]);
    else v[i] = to_f32<TYPE>((T)(w[(i >> 3) % kWords][(i >> 1) & 3] >> (16 * (i & 1))));
  }
}

template <int V>
__device__ __forceinline__ uint32_t top_bits(const float (&v)[V]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}

__device__ __forceinline__ float scale_of(uint32_t top) {
  if (top >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(top) / 448.0f, 0x1p-126f);
}

// The codes of V elements, those at or past `valid` zeros, stored as V bytes. Their quotients are the
// correctly rounded ones: with r the rounded reciprocal of the scale, x r is within two units of the
// quotient, one correction by its remainder brings it within one and the second one rounds it correctly
// (Markstein). Scales so small that a remainder may underflow are divided by.
template <int V>
__device__ __forceinline__ void store_codes(const float (&v)[V], float scale, int valid, uint8_t* p) {
  float q[V];
  if (scale >= 0x1p-80f) {
    const float r = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float u = v[i] * r;
      u = __builtin_fmaf(__builtin_fmaf(-u, scale, v[i]), r, u);
      q[i] = __builtin_fmaf(__builtin_fmaf(-u, scale, v[i]), r, u);
      // a zero keeps its sign
      q[i] = v[i] == 0.0f ? v[i] : q[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = v[i] / scale;
  }
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], c, true);
    // no number: the scale of a block with an infinity or a NaN
    w[i] = scale == scale ? (uint32_t)c : 0x7f7f7f7fu;
    const int n = valid - 4 * i;
    if (n < 4) w[i] = n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1u);
  }
  __builtin_memcpy(__builtin_assume_aligned(p, V), w, V);
}

}  // namespace

}  // namespace aaac
