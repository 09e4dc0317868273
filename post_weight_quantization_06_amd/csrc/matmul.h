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

template <int N> struct Int { static constexpr int value = N; };

// Rows as a buffer: loads past its `bytes` give zeros, so rows past a tile's last and columns past a
// row's end need no branch. The ABI keeps a tile of 256 rows below 2^31 bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
// An offset past every such buffer, also with a tile's rows and columns added to it (below 2^29).
constexpr uint32_t kOutside = 0x80000000u;

typedef __attribute__((address_space(3))) void* LdsPtr;

// rows_rsrc as the four words that an assembly operand takes.
__device__ __forceinline__ u32x4 rows_buffer(const void* p, int64_t bytes) {
  const uint64_t b = (uint64_t)p;
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, (uint32_t)bytes, 0x00027000u};
}

// Any bytes as a buffer of whole words: the word that holds the first byte is word 0 and that byte
// lies `lead` bytes into it. The last word may reach past the last byte, never past its own address.
__device__ __forceinline__ u32x4 words_buffer(const void* p, int64_t bytes, uint32_t& lead) {
  lead = (uint32_t)(uintptr_t)p & 3u;
  return rows_buffer(static_cast<const uint8_t*>(p) - lead, (bytes + lead + 3) & ~(int64_t)3);
}

// Asynchronous loads from a buffer into LDS: lane l's bytes land at dst + l * size (dst uniform).
// `more` is a uniform offset below the buffer's bytes. The range check takes it from the buffer's bytes
// before it compares, so a larger one could wrap round to a range that kOutside lies in; a smaller one
// leaves kOutside outside whether it is counted or not.
// In assembly because the compiler would wait for them before any LDS read, of the other stage too;
// the caller waits (wait_loads, then step_barrier) before they are read. The move to m0 needs one
// wait state before the load.
__device__ __forceinline__ void load_lds16(u32x4 buf, uint32_t off, uint32_t more, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(dst), "v"(off), "s"(buf), "s"(more) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(u32x4 buf, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(dst), "v"(off), "s"(buf) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(LdsPtr)(void*)p;
}
// At most N of this wave's loads are still under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}
// After it, every wave's LDS writes, and the loads it waited for, can be read.
__device__ __forceinline__ void step_barrier() {
  __builtin_amdgcn_s_waitcnt(0xc07f);            // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Step `step` of 64 columns lies past the row's end: its loads are outside their buffers.
__device__ __forceinline__ bool past_row(const MatmulArgs& a, int step) {
  return step * 64 >= (int)a.Cp;
}

constexpr int kMfma = 16;                        // rows and columns of one matrix instruction

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

// A tile's result: y itself, or part `part` of a sum split over workgroups, kept in fp32 in rows of
// whole 16-byte words.
__device__ __forceinline__ void store_part(const MatmulArgs& a, int part, int64_t t, int64_t r,
                                           f32x4 v) {
  if (a.split == 1) store4(a, t, r, v);
  else *reinterpret_cast<f32x4*>(a.parts + ((int64_t)part * a.T + t) * part_row(a.R) + r) = v;
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
// Decoders: 4-bit weights to bf16, eight at a time. A kernel reads a weight row either by runs (32
// consecutive columns a thread: the tiles, which stage codes, scale and selector words of a run in
// LDS, `issue` and `fetch`, and pass the result on through LDS, `piece`) or by chunks (128
// consecutive columns a wave row of four lane groups: the few-row kernels, which feed it to the
// matrix instructions directly). In a chunk lane group q = lane >> 4 reads the 16 code bytes of run
// q; a transposition over the four groups then leaves it with the codes of columns 32 p + 8 q ..
// 32 p + 8 q + 7 in word p, the columns that instruction p of the chunk wants from it. Eight
// neighbouring columns never cross a scale or selection group.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ u32x4 over_groups(u32x4 v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const u32x2 b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const u32x2 c = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
  const u32x2 d = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
  return u32x4{c.x, c.y, d.x, d.y};
}

// Word p of the result: v of lane group p.
__device__ __forceinline__ u32x4 from_groups(uint32_t v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const u32x2 c = __builtin_amdgcn_permlane16_swap(a.x, a.x, false, false);
  const u32x2 d = __builtin_amdgcn_permlane16_swap(a.y, a.y, false, false);
  return u32x4{c.x, c.y, d.x, d.y};
}

// MXFP4: a run is one block; code times power of two is exact in bf16 (and in fp32 before it).
struct MxDecoder {
  static constexpr bool kFour = true;            // see load_four
  struct Row { const uint8_t* codes; const uint8_t* scales; };
  struct Run { u32x4 codes; uint32_t byte; };
  struct Chunk { u32x4 codes; uint32_t bytes; };
  __device__ __forceinline__ void init(const MatmulArgs&, int) {}
  __device__ __forceinline__ Row row(const MatmulArgs& a, int e, int64_t r) const {
    const int64_t i = (int64_t)e * a.R + r;
    return {a.codes + i * (a.Cp >> 1), static_cast<const uint8_t*>(a.scales) + i * (a.Cp >> 5)};
  }
  // 2^(b - 127): byte 0 is the subnormal 2^-127, byte 255 a NaN.
  static __device__ __forceinline__ float value(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23));
  }
  static __device__ __forceinline__ u32x4 eight(uint32_t w, uint32_t b) {
    const float s = value(b);
    const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    return u32x4{pack_bf16(v0.x * s, v0.y * s), pack_bf16(v1.x * s, v1.y * s),
                 pack_bf16(v2.x * s, v2.y * s), pack_bf16(v3.x * s, v3.y * s)};
  }

  static constexpr int kWords = 1;
  u32x4 codes_buf, scales_buf;
  uint32_t lead;                                 // bytes from the word that holds the first scale
  __device__ __forceinline__ void init_tile(const MatmulArgs& a, int e, int64_t r0, int64_t nr) {
    const int64_t i = (int64_t)e * a.R + r0, kb = a.Cp >> 5;
    codes_buf = rows_buffer(a.codes + i * (a.Cp >> 1), nr * (a.Cp >> 1));
    scales_buf = words_buffer(static_cast<const uint8_t*>(a.scales) + i * kb, nr * kb, lead);
  }
  // Loads of a run: columns 64 step + half .. + 31 of tile row `row`.
  __device__ __forceinline__ void issue(const MatmulArgs& a, int row, int step, int half, bool in,
                                        uint32_t dst, uint32_t words, int) const {
    const uint32_t kb = (uint32_t)(a.Cp >> 5);
    load_lds16(codes_buf, in ? row * (kb * 16) + half / 2 : kOutside, past_row(a, step) ? 0 : step * 32,
               dst);
    load_lds4(scales_buf, in ? (lead + row * kb + 2 * step + half / 32) & ~3u : kOutside, words);
  }
  __device__ __forceinline__ Run fetch(const MatmulArgs& a, int row, int step, int half, bool,
                                       const void* codes, const uint32_t* words, int) const {
    const uint32_t at = lead + row * (uint32_t)(a.Cp >> 5) + 2 * step + half / 32;
    return {*static_cast<const u32x4*>(codes), (*words >> (8 * (at & 3u))) & 0xffu};
  }
  struct Planes {};
  struct Eight { u32x4 out; };
  __device__ __forceinline__ void piece(const Run& u, int j, int n, Planes&, Eight& v) const {
    if (n == 0) v.out = eight(u.codes[j], u.byte);
  }
  __device__ __forceinline__ Chunk load_chunk(const MatmulArgs&, const Row& w, int c, int q) const {
    Chunk u;
    u.codes = *reinterpret_cast<const u32x4*>(w.codes + (int64_t)c * 64 + 16 * q);
    __builtin_memcpy(&u.bytes, w.scales + c * 4, 4);
    return u;
  }
  // Four chunks at once, the scales of chunk q read by lane group q: `Four` as loaded, `chunk` one of
  // them.
  struct Four { u32x4 codes[4]; uint32_t bytes; };
  __device__ __forceinline__ Four load_four(const MatmulArgs&, const Row& w, int c, int q) const {
    Four u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u.codes[i] = *reinterpret_cast<const u32x4*>(w.codes + (int64_t)(c + i) * 64 + 16 * q);
    __builtin_memcpy(&u.bytes, w.scales + (c + q) * 4, 4);
    return u;
  }
  static __device__ __forceinline__ Chunk chunk(const Four& u, const u32x4& bytes, int i) {
    return {u.codes[i], bytes[i]};
  }
  static __device__ __forceinline__ u32x4 spread(const Four& u) { return from_groups(u.bytes); }
  // The row's last chunk: runs at or past its end are zeros.
  __device__ __forceinline__ Chunk load_last(const MatmulArgs& a, const Row& w, int c, int q) const {
    Chunk u = {u32x4{0u, 0u, 0u, 0u}, 0u};
    const int left = (int)(a.Cp >> 5) - 4 * c;
    if (q < left) u.codes = *reinterpret_cast<const u32x4*>(w.codes + (int64_t)c * 64 + 16 * q);
    for (int i = 0; i < 4; ++i)
      if (i < left) u.bytes |= (uint32_t)w.scales[c * 4 + i] << (8 * i);
    return u;
  }
  __device__ __forceinline__ void decode_chunk(const Chunk& u, int, u32x4 (&out)[4]) const {
    const u32x4 w = over_groups(u.codes);
#pragma unroll
    for (int p = 0; p < 4; ++p) out[p] = eight(w[p], (u.bytes >> (8 * p)) & 0xffu);
  }
};

// Packed dual-codebook weights: bf16(|s| T_sel[q]). The two tables of 16 bf16 entries lie in scalar
// registers as planes of low and high bytes, the second as its difference to the first; a byte
// permute looks four codes up at once in eight entries, a second permute picks between the lower and
// the upper eight by bit 3 of the code, and a third puts the two bytes of an entry where fp32 keeps
// them. One product and one rounding follow, as in dequant.
// LG: log2 of the scale group, 7 for 128 and more. LS: the same of the selection group when its
// selectors are in the bitmap, 0 when they are the scales' sign bits (S == g). OFF: the scales start
// two bytes past a word, with LG < 5, where a run's scales are whole words otherwise (C / g is even
// there, so every row starts as the first one does); the tiles then read a word more a run.
template <int LG, int LS, bool OFF = false>
struct PackedDecoder {
  static constexpr bool kSign = LS == 0;
  static constexpr bool kFour = kSign && LG >= 6;                   // see load_four
  static constexpr int kGpl = LG >= 5 ? 1 : 32 >> LG;               // scale groups in a run
  static constexpr int kScaleBytes = LG >= 7 ? 2 : 256 >> LG;       // of a chunk
  static constexpr int kScaleWords = (kScaleBytes + 3) / 4;
  struct Row { const uint8_t* codes; const uint16_t* scales; int64_t first; };
  struct Run { u32x4 codes; uint32_t scale[kGpl]; uint32_t bits, pick; };
  struct Chunk { u32x4 codes; uint32_t scale[kScaleWords]; uint32_t bits, shift; };
  uint32_t lo[2][4], hi[2][4];                   // T0, and T0 ^ T1; uniform, in scalar registers
  const uint8_t* bitmap;
  int64_t bitmap_bytes;

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
        l = __builtin_amdgcn_readfirstlane(l);
        h = __builtin_amdgcn_readfirstlane(h);
        lo[c][v] = c == 0 ? l : l ^ lo[0][v];
        hi[c][v] = c == 0 ? h : h ^ hi[0][v];
      }
    }
    bitmap = kSign ? nullptr : a.bitmap + (int64_t)e * a.bitmap_stride;
    bitmap_bytes = a.bitmap_stride;
  }
  __device__ __forceinline__ Row row(const MatmulArgs& a, int e, int64_t r) const {
    const int64_t i = (int64_t)e * a.R + r;
    return {a.codes + i * (a.C >> 1), static_cast<const uint16_t*>(a.scales) + i * (a.C >> a.log2g),
            kSign ? 0 : r * (a.C >> a.log2S)};
  }
  struct Planes { uint32_t L[4], H[4]; };
  // The table of a selector in bit `bit` of word w, by a mask of that bit.
  __device__ __forceinline__ Planes planes(uint32_t w, int bit) const {
    const uint32_t one = (uint32_t)__builtin_amdgcn_sbfe((int)w, (uint32_t)bit, 1u);
    Planes p;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      p.L[v] = lo[0][v] ^ (lo[1][v] & one);
      p.H[v] = hi[0][v] ^ (hi[1][v] & one);
    }
    return p;
  }
  // Eight weights in four parts of equal work, which a kernel can place between matrix instructions:
  // the entry bytes of the even and of the odd columns, then two words of bf16 pairs twice.
  // from: kPick, or 0x0c0c0c0c (zero bytes) with codes of zero for columns past the row's end.
  static constexpr uint32_t kPick = 0x03020100u;
  struct Eight { uint32_t l[2], h[2]; u32x4 out; };
  static __device__ __forceinline__ void part(Eight& v, int n, uint32_t w, const Planes& t,
                                              uint32_t scale, uint32_t from) {
    if (n < 2) {
      const uint32_t idx = (n ? w >> 4 : w) & 0x07070707u;
      const uint32_t pick = ((n ? w >> 5 : w >> 1) & 0x04040404u) | from;
      v.l[n] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(t.L[3], t.L[2], idx),
                                     __builtin_amdgcn_perm(t.L[1], t.L[0], idx), pick);
      v.h[n] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(t.H[3], t.H[2], idx),
                                     __builtin_amdgcn_perm(t.H[1], t.H[0], idx), pick);
      return;
    }
    const float s = __uint_as_float((scale & 0x7fffu) << 16);
#pragma unroll
    for (int p = 2 * n - 4; p < 2 * n - 2; ++p) {
      // bytes: 0, 0, low, high (selector 12 is a zero byte; 0..3 index the low plane's word)
      const uint32_t sel = 0x00000c0cu | ((uint32_t)p << 16) | ((uint32_t)(4 + p) << 24);
      const float ve = __uint_as_float(__builtin_amdgcn_perm(v.h[0], v.l[0], sel));
      const float vo = __uint_as_float(__builtin_amdgcn_perm(v.h[1], v.l[1], sel));
      v.out[p] = pack_bf16(ve * s, vo * s);
    }
  }
  static __device__ __forceinline__ u32x4 eight(uint32_t w, const Planes& t, uint32_t scale,
                                                uint32_t from) {
    Eight v;
#pragma unroll
    for (int n = 0; n < 4; ++n) part(v, n, w, t, scale, from);
    return v.out;
  }

  static constexpr int kScaleLoads = (kGpl + 1) / 2 + (OFF ? 1 : 0);  // words with a run's scales
  static constexpr int kWords = kScaleLoads + (kSign ? 0 : 1);
  u32x4 codes_buf, scales_buf, bits_buf;
  uint32_t lead, bits_lead;                      // see words_buffer; bits_lead in bits
  __device__ __forceinline__ void init_tile(const MatmulArgs& a, int e, int64_t r0, int64_t nr) {
    const int64_t i = (int64_t)e * a.R + r0, per = a.C >> a.log2g;
    codes_buf = rows_buffer(a.codes + i * (a.C >> 1), nr * (a.C >> 1));
    scales_buf = words_buffer(static_cast<const uint16_t*>(a.scales) + i * per, nr * per * 2, lead);
    if (!kSign) {
      const int64_t h = r0 * (a.C >> a.log2S), bits = nr * (a.C >> a.log2S) + (h & 7);
      bits_buf = words_buffer(bitmap + (h >> 3), (bits + 7) >> 3, bits_lead);
      bits_lead = 8 * bits_lead + (uint32_t)(h & 7);
    }
  }
  __device__ __forceinline__ uint32_t scale_at(const MatmulArgs& a, int row, int step,
                                               int half) const {
    const uint32_t g = LG >= 6 ? (step * 64) >> a.log2g : (step * 64 + half) >> a.log2g;
    return lead + 2 * (row * (uint32_t)(a.C >> a.log2g) + g);
  }
  __device__ __forceinline__ uint32_t bit_at(const MatmulArgs& a, int row, int step, int half) const {
    const uint32_t h = LS >= 6 ? (step * 64) >> a.log2S : (step * 64 + half) >> a.log2S;
    return bits_lead + row * (uint32_t)(a.C >> a.log2S) + h;
  }
  __device__ __forceinline__ void issue(const MatmulArgs& a, int row, int step, int half, bool in,
                                        uint32_t dst, uint32_t words, int threads) const {
    load_lds16(codes_buf, in ? row * (uint32_t)(a.C >> 1) + half / 2 : kOutside,
               past_row(a, step) ? 0 : step * 32, dst);
    const uint32_t at = scale_at(a, row, step, half) & ~3u;
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i)
      load_lds4(scales_buf, in ? at + 4 * i : kOutside, words + i * threads * 4);
    if (!kSign)
      load_lds4(bits_buf, in ? (bit_at(a, row, step, half) >> 5) * 4 : kOutside,
                words + kScaleLoads * threads * 4);
  }
  __device__ __forceinline__ Run fetch(const MatmulArgs& a, int row, int step, int half, bool in,
                                       const void* codes, const uint32_t* words,
                                       int threads) const {
    Run u;
    u.codes = *static_cast<const u32x4*>(codes);
    u.pick = in ? kPick : 0x0c0c0c0cu;
    const uint32_t at = scale_at(a, row, step, half);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const uint32_t w = words[i * threads];
      if (kGpl == 1) {
        u.scale[0] = w >> (8 * (at & 2u));
      } else if (OFF) {
        if (i > 0) u.scale[2 * i - 1] = w;
        if (2 * i < kGpl) u.scale[2 * i] = w >> 16;
      } else {
        u.scale[2 * i] = w;
        u.scale[2 * i + 1] = w >> 16;
      }
    }
    if (!kSign) u.bits = words[kScaleLoads * threads] >> (bit_at(a, row, step, half) & 31u);
    return u;
  }
  // Part n of columns 8 j .. 8 j + 7 of a run, in ascending order; t carries the tables from one j
  // to the next of the same selection group.
  __device__ __forceinline__ void piece(const Run& u, int j, int n, Planes& t, Eight& v) const {
    const int gi = LG >= 5 ? 0 : (8 * j) >> LG, si = LS >= 5 ? 0 : (8 * j) >> LS;
    if (n == 0) {
      if (kSign) {
        if (j == 0 || (LG < 5 && (8 * j) % (1 << LG) == 0)) t = planes(u.scale[gi], 15);
      } else if (j == 0 || (LS < 5 && (8 * j) % (1 << LS) == 0)) {
        t = planes(u.bits, si);
      }
    }
    part(v, n, u.codes[j], t, u.scale[gi], u.pick);
  }

  __device__ __forceinline__ Chunk load_chunk(const MatmulArgs& a, const Row& w, int c, int q) const {
    Chunk u;
    u.codes = *reinterpret_cast<const u32x4*>(w.codes + (int64_t)c * 64 + 16 * q);
    const uint16_t* sp = w.scales + (((int64_t)c * 128) >> a.log2g);
    if (LG >= 7) u.scale[0] = sp[0];
    else __builtin_memcpy(u.scale, sp, kScaleBytes);
    if (!kSign) load_bits(a, w, c, u);
    return u;
  }
  // Four chunks at once (scale groups of 64 and more, selectors in the sign): lane group q reads the
  // scales of chunk q.
  struct Four { u32x4 codes[4]; uint32_t scale; };
  __device__ __forceinline__ Four load_four(const MatmulArgs& a, const Row& w, int c, int q) const {
    Four u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u.codes[i] = *reinterpret_cast<const u32x4*>(w.codes + (int64_t)(c + i) * 64 + 16 * q);
    const uint16_t* sp = w.scales + (((int64_t)(c + q) * 128) >> a.log2g);
    if (LG >= 7) u.scale = sp[0];
    else __builtin_memcpy(&u.scale, sp, 4);
    return u;
  }
  static __device__ __forceinline__ u32x4 spread(const Four& u) { return from_groups(u.scale); }
  static __device__ __forceinline__ Chunk chunk(const Four& u, const u32x4& scales, int i) {
    Chunk v;
    v.codes = u.codes[i];
    v.scale[0] = scales[i];
    return v;
  }
  // The selectors of a chunk as the low bits of bits >> shift: four bytes from the first one's, or
  // the four last bytes of this matrix's map where those would end past it.
  __device__ __forceinline__ void load_bits(const MatmulArgs& a, const Row& w, int c, Chunk& u) const {
    const int64_t h = w.first + (((int64_t)c * 128) >> a.log2S);
    if (bitmap_bytes >= 4) {
      const int64_t last = bitmap_bytes - 4, at = (h >> 3) < last ? (h >> 3) : last;
      __builtin_memcpy(&u.bits, bitmap + at, 4);
      u.shift = (uint32_t)(h - 8 * at);
    } else {
      u.bits = 0;
      for (int i = 0; i < (int)bitmap_bytes; ++i) u.bits |= (uint32_t)bitmap[i] << (8 * i);
      u.shift = (uint32_t)h;
    }
  }
  // The row's last chunk: runs at or past its end are zeros (and their codes entry 0: the caller
  // clears what it decodes to).
  __device__ __forceinline__ Chunk load_last(const MatmulArgs& a, const Row& w, int c, int q) const {
    Chunk u;
    u.codes = u32x4{0u, 0u, 0u, 0u};
    const int64_t k = (int64_t)c * 128 + 32 * q;
    if (k < a.C) u.codes = *reinterpret_cast<const u32x4*>(w.codes + (k >> 1));
    const int64_t g0 = ((int64_t)c * 128) >> a.log2g, gn = a.C >> a.log2g;
#pragma unroll
    for (int i = 0; i < kScaleWords; ++i) u.scale[i] = 0;
#pragma unroll
    for (int i = 0; i < kScaleBytes / 2; ++i)
      if (g0 + i < gn) u.scale[i >> 1] |= (uint32_t)w.scales[g0 + i] << (16 * (i & 1));
    if (!kSign) load_bits(a, w, c, u);
    return u;
  }
  __device__ __forceinline__ void decode_chunk(const Chunk& u, int q, u32x4 (&out)[4]) const {
    const u32x4 w = over_groups(u.codes);
    Planes t;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t s;
      if (LG >= 7) s = u.scale[0];
      else if (LG == 6) s = u.scale[0] >> (16 * (p >> 1));
      else if (LG == 5) s = u.scale[p >> 1] >> (16 * (p & 1));
      else if (LG == 4) s = u.scale[p] >> (16 * (q >> 1));
      else s = (q >> 1 ? u.scale[2 * p + 1] : u.scale[2 * p]) >> (16 * (q & 1));
      if (kSign) {
        if (p == 0 || LG < 6 || (LG == 6 && p == 2)) t = planes(s, 15);
      } else if (p == 0 || LS < 6 || (LS == 6 && p == 2)) {
        const int i = LS >= 7 ? 0 : LS >= 5 ? (32 * p) >> LS : ((32 * p) >> LS) + ((8 * q) >> LS);
        t = planes(u.bits, (int)u.shift + i);
      }
      out[p] = eight(w[p], t, s, kPick);
    }
  }
};

// Calls f with the decoder type of a packed call. TILES: f reads weights by runs.
template <bool TILES, class F>
hipError_t with_packed_decoder(const MatmulArgs& a, F f) {
  const int lg = a.log2g < 7 ? a.log2g : 7, ls = a.log2S < 7 ? a.log2S : 7;
  if constexpr (TILES) {
    if (lg < 5 && (uintptr_t)a.scales % 4 != 0)
      return a.bitmap ? f(PackedDecoder<4, 3, true>())
             : lg == 3 ? f(PackedDecoder<3, 0, true>()) : f(PackedDecoder<4, 0, true>());
  }
  if (!a.bitmap) {
    switch (lg) {
      case 3: return f(PackedDecoder<3, 0>());
      case 4: return f(PackedDecoder<4, 0>());
      case 5: return f(PackedDecoder<5, 0>());
      case 6: return f(PackedDecoder<6, 0>());
      default: return f(PackedDecoder<7, 0>());
    }
  }
  switch (8 * lg + ls) {
    case 8 * 4 + 3: return f(PackedDecoder<4, 3>());
    case 8 * 5 + 3: return f(PackedDecoder<5, 3>());
    case 8 * 5 + 4: return f(PackedDecoder<5, 4>());
    case 8 * 6 + 3: return f(PackedDecoder<6, 3>());
    case 8 * 6 + 4: return f(PackedDecoder<6, 4>());
    case 8 * 6 + 5: return f(PackedDecoder<6, 5>());
    case 8 * 7 + 3: return f(PackedDecoder<7, 3>());
    case 8 * 7 + 4: return f(PackedDecoder<7, 4>());
    case 8 * 7 + 5: return f(PackedDecoder<7, 5>());
    case 8 * 7 + 6: return f(PackedDecoder<7, 6>());
    default: return f(PackedDecoder<7, 7>());
  }
}

}  // namespace aaac
