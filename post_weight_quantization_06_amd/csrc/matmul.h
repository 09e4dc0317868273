// Device helpers shared by the product kernels (matmul_few.hip, matmul_tile.hip).
#pragma once

#include "aaac.h"
#include "mxfp4.h"

namespace aaac {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kMfma = 16;                        // rows and columns of one matrix instruction

// Token tiles of BN rows that a call can need at most: every expert's last tile may be partial.
inline int64_t token_tiles(const MatmulArgs& a, int BN) {
  if (!a.offsets) return (a.T + BN - 1) / BN;
  const int64_t e = a.E < a.T ? a.E : a.T;
  return a.T / BN + e;
}

// The expert and the rows [t0, t1) of token tile `tile` (uniform over the wave), or false past the
// last one. Every wave counts the experts' tiles by itself, 64 experts at a time.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int64_t T, int BN,
                                          int64_t tile, int& e, int64_t& t0, int64_t& t1) {
  if (!offsets) {
    e = 0;
    t0 = tile * BN;
    t1 = T;
    return t0 < T;
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int top = (int)T;
  int64_t before = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int i = e0 + lane < E ? e0 + lane : E - 1;
    int lo = offsets[i], hi = offsets[i + 1];
    lo = lo < 0 ? 0 : (lo > top ? top : lo);
    hi = hi < lo ? lo : (hi > top ? top : hi);
    const int n = e0 + lane < E ? (int)(((int64_t)hi - lo + BN - 1) / BN) : 0;
    int sum = n;                                 // tiles of this and the lanes before it
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int v = __shfl_up(sum, d, kWave);
      if (lane >= d) sum += v;
    }
    const int64_t want = tile - before;
    const uint64_t past = __ballot((int64_t)sum > want);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(sum - n, l);
      const int l0 = __builtin_amdgcn_readlane(lo, l), h0 = __builtin_amdgcn_readlane(hi, l);
      e = e0 + l;
      t0 = l0 + (want - first) * BN;
      t1 = h0;
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, kWave - 1);
  }
  return false;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// y[t, r .. r + 3] = v, the columns at or past R left out; one rounding to the output's type.
__device__ __forceinline__ void store4(const MatmulArgs& a, int64_t t, int64_t r, f32x4 v) {
  const int64_t i = t * a.ldy + r;
  if (a.y_vec && r + 4 <= a.R) {
    if (a.y_type == AAAC_F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + i) = v;
    } else {
      const uint2 w = a.y_type == AAAC_BF16 ? make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w))
                                            : make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + i) = w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (r + k >= a.R) break;
    if (a.y_type == AAAC_F32) static_cast<float*>(a.y)[i + k] = v[k];
    else if (a.y_type == AAAC_BF16)
      static_cast<uint16_t*>(a.y)[i + k] = (uint16_t)pack_bf16(v[k], 0.0f);
    else static_cast<uint16_t*>(a.y)[i + k] = (uint16_t)pack_f16(v[k], 0.0f);
  }
}

inline int can_store4(const MatmulArgs& a) {
  const int b = a.y_type == AAAC_F32 ? 4 : 2;
  return (uintptr_t)a.y % (4 * b) == 0 && a.ldy % 4 == 0;
}

// B: which byte of the scale words counts.
template <int B>
__device__ __forceinline__ f32x4 mfma_fp4(u32x4 w, u32x4 x, f32x4 c, uint32_t sw, uint32_t sx) {
  const i32x8 aw = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
  const i32x8 ax = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aw, ax, c, 4, 4, B, (int)sw, B,
                                                          (int)sx);
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 w, u32x4 x, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                 __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
}

// ------------------------------------------------------------------------------------------------
// Weights of a lane's run of 32 consecutive columns (16 bytes of codes) as bf16, eight at a time.
// ------------------------------------------------------------------------------------------------

// MXFP4: the run is one block; code times power of two is exact in bf16.
struct MxRun {
  u32x4 codes;
  uint32_t byte;
};
struct MxDecoder {
  typedef MxRun Run;
  struct Row { const uint8_t* codes; const uint8_t* scales; };
  __device__ __forceinline__ void init(const MatmulArgs&, int) {}
  __device__ __forceinline__ Row row(const MatmulArgs& a, int e, int64_t r) const {
    const int64_t i = (int64_t)e * a.R + r;
    return {a.codes + i * (a.Cp >> 1), static_cast<const uint8_t*>(a.scales) + i * (a.Cp >> 5)};
  }
  __device__ __forceinline__ Run load(const MatmulArgs&, const Row& w, int64_t k) const {
    Run u;
    u.codes = *reinterpret_cast<const u32x4*>(w.codes + (k >> 1));
    u.byte = w.scales[k >> 5];
    return u;
  }
  static __device__ __forceinline__ float value(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23));
  }
  __device__ __forceinline__ void decode(const MatmulArgs&, const Run& u, u32x4 (&out)[4]) const {
    const float s = value(u.byte);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4];
      // code values are exact in fp32 and so is their product with the power of two
      const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.codes[j], 1.0f, 0);
      const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.codes[j], 1.0f, 1);
      const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.codes[j], 1.0f, 2);
      const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.codes[j], 1.0f, 3);
      o[0] = pack_bf16(v0.x * s, v0.y * s);
      o[1] = pack_bf16(v1.x * s, v1.y * s);
      o[2] = pack_bf16(v2.x * s, v2.y * s);
      o[3] = pack_bf16(v3.x * s, v3.y * s);
      out[j] = u32x4{o[0], o[1], o[2], o[3]};
    }
  }
};

// Packed dual-codebook weights: bf16(|s| T_sel[q]). The two tables of 16 bf16 entries lie in
// registers as planes of low and high bytes; a byte permute looks four codes up at once in eight
// entries, a second permute picks between the lower and the upper eight by bit 3 of the code, and a
// third puts the two bytes of an entry where fp32 keeps them. One product and one rounding follow,
// as in dequant.
// GPL, SPL: scale and selection groups in a run (1 for groups of 32 and more). SIGN: the selector
// is the scale's sign bit (S == g), else a bit of the bitmap.
template <int GPL, int SPL>
struct PackedRun {
  u32x4 codes;
  uint32_t scale[GPL];
  uint32_t bits, shift;                          // bitmap byte and the run's first bit in it
};
template <int GPL, int SPL, bool SIGN>
struct PackedDecoder {
  typedef PackedRun<GPL, SPL> Run;
  struct Row { const uint8_t* codes; const uint16_t* scales; const uint8_t* bitmap; int64_t first; };
  uint32_t lo[2][4], hi[2][4];

  __device__ __forceinline__ void init(const MatmulArgs& a, int e) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint16_t* t = a.tables + ((int64_t)e * 2 + c) * a.n;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t l = 0, h = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int q = 4 * v + k;
          const uint32_t b = t[q < a.n ? q : 0];
          l |= (b & 0xffu) << (8 * k);
          h |= (b >> 8) << (8 * k);
        }
        asm volatile("" : "+v"(l), "+v"(h));     // vector registers: a permute reads two of them
        lo[c][v] = l;
        hi[c][v] = h;
      }
    }
  }
  __device__ __forceinline__ Row row(const MatmulArgs& a, int e, int64_t r) const {
    const int64_t i = (int64_t)e * a.R + r;
    return {a.codes + i * (a.C >> 1),
            static_cast<const uint16_t*>(a.scales) + i * (a.C >> a.log2g),
            SIGN ? nullptr : a.bitmap + (int64_t)e * a.bitmap_stride, r * (a.C >> a.log2S)};
  }
  __device__ __forceinline__ Run load(const MatmulArgs& a, const Row& w, int64_t k) const {
    Run u;
    u.codes = *reinterpret_cast<const u32x4*>(w.codes + (k >> 1));
    const uint16_t* sp = w.scales + (k >> a.log2g);
#pragma unroll
    for (int i = 0; i < GPL; ++i) u.scale[i] = sp[i];
    if (!SIGN) {
      const int64_t h = w.first + (k >> a.log2S);
      u.bits = w.bitmap[h >> 3];
      u.shift = (uint32_t)h & 7u;
    }
    return u;                                    // as loaded: nothing here waits for the words
  }
  __device__ __forceinline__ void decode(const MatmulArgs&, const Run& u, u32x4 (&out)[4]) const {
    uint32_t L[4], H[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j % (4 / SPL) == 0) {
        const int i = j / (4 / SPL);             // SIGN: SPL == GPL
        const bool one = SIGN ? (u.scale[i < GPL ? i : 0] & 0x8000u) != 0
                              : ((u.bits >> (u.shift + i)) & 1u) != 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          L[v] = one ? lo[1][v] : lo[0][v];
          H[v] = one ? hi[1][v] : hi[0][v];
        }
      }
      const float s = __uint_as_float((u.scale[j / (4 / GPL)] & 0x7fffu) << 16);
      const uint32_t w = u.codes[j];
      uint32_t pl[2], ph[2];                     // entry bytes of the even and the odd columns
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        const uint32_t idx = (odd ? w >> 4 : w) & 0x07070707u;
        const uint32_t pick = ((odd ? w >> 5 : w >> 1) & 0x04040404u) | 0x03020100u;
        pl[odd] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(L[3], L[2], idx),
                                        __builtin_amdgcn_perm(L[1], L[0], idx), pick);
        ph[odd] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(H[3], H[2], idx),
                                        __builtin_amdgcn_perm(H[1], H[0], idx), pick);
      }
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // bytes: 0, 0, low, high (selector 12 is a zero byte; 0..3 index the low plane's word)
        const uint32_t sel = 0x00000c0cu | ((uint32_t)p << 16) | ((uint32_t)(4 + p) << 24);
        const float ve = __uint_as_float(__builtin_amdgcn_perm(ph[0], pl[0], sel));
        const float vo = __uint_as_float(__builtin_amdgcn_perm(ph[1], pl[1], sel));
        o[p] = pack_bf16(ve * s, vo * s);
      }
      out[j] = u32x4{o[0], o[1], o[2], o[3]};
    }
  }
};

}  // namespace aaac
