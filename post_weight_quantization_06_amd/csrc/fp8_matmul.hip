// Products of rows of x and weights in 8-bit floating point with a scale for each block of 128: for
// every block b of 128 columns the matrix instruction sums the codes' products, and the block's sum goes
// into the result times sx[t, b] sw[r / 128, b], so fp32 sums are scaled, never codes.
//   y[t, r] = sum_b sx[t, b] sw[r / 128, b] sum_{c in b} qx[t, c] qw[r, c]
// Matrix instructions take weight rows as the A operand and rows of x as B. That of the few-row kernels takes
// 16 of each and 128 columns: one instruction is one block. Lane l holds, for weight row (and x row) l & 15,
// the same 32 of the 128 columns, and in the result four neighbouring weight rows of x row l & 15; a sum does
// not depend on which lane holds which columns.
#include "fp8.h"
#include "fp8_encode.h"
#include "matmul.h"

namespace aaac {

namespace {

// A fragment: a lane's 32 codes of a block, for the FP8 instruction as they are, for the bf16 one (WIDE)
// as bf16 numbers, eight of them for each of its four instructions.
//
// The FP8 instruction adds eight products at a time, aligned to the largest and cut below 2^-13 of it
// (measured: 2^16 + 2^2 gives 2^16, 2^16 + 2^3 does not), then in fp32: its sums are off by 2^-19.4 of the
// sum of magnitudes on average over normal values, 2^-15.8 at most. Over a product of normal values that is
// 1.4e-5 of the result's norm at any number of columns, a 118th of what the rounding to bf16 is off by (1.66e-3),
// so results of that type use it. It would be a fifteenth of the rounding to fp16 (2.1e-4), and 140 times what
// fp32 sums are off by (1e-7): those results take the bf16 instruction, whose sums of the same exact products are
// fp32 sums, at half the rate and with a conversion for every two codes (4096 x 14336 and one row of bf16: 14 us,
// with the FP8 instruction 13; 14336 x 4096 and 48 rows 25 and 18, 4096 rows 445 and 249 with fp16 results).
template <bool WIDE> struct Frag;
template <> struct Frag<false> { u32x4 v[2]; };
template <> struct Frag<true> { u32x4 v[4]; };

__device__ __forceinline__ uint32_t two_bf16(uint32_t w, bool hi) {
  return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
            : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
template <bool WIDE>
__device__ __forceinline__ Frag<WIDE> frag(u32x4 a, u32x4 b) {
  Frag<WIDE> f;
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = i < 2 ? a[2 * i] : b[2 * i - 4], hi = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
      f.v[i] = u32x4{two_bf16(lo, false), two_bf16(lo, true), two_bf16(hi, false), two_bf16(hi, true)};
    }
  } else {
    f.v[0] = a;
    f.v[1] = b;
  }
  return f;
}

__device__ __forceinline__ i32x8 operand(const Frag<false>& f) {
  return i32x8{(int)f.v[0].x, (int)f.v[0].y, (int)f.v[0].z, (int)f.v[0].w,
               (int)f.v[1].x, (int)f.v[1].y, (int)f.v[1].z, (int)f.v[1].w};
}

// The sum over a block by the bf16 instruction.
__device__ __forceinline__ f32x4 block_sum(const Frag<true>& w, const Frag<true>& x) {
  f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma_bf16(w.v[i], x.v[i], c);
  return c;
}

__device__ __forceinline__ f32x4 block_sum(const Frag<false>& w, const Frag<false>& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(x), f32x4{0.0f, 0.0f, 0.0f, 0.0f},
                                                          0, 0, 0, 0, 0, 0);
}

// A 16-byte piece without its bytes at or past `valid`.
__device__ __forceinline__ u32x4 first_bytes(u32x4 v, int valid) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = valid - 4 * i;
    if (n < 4) v[i] = n <= 0 ? 0u : v[i] & ((1u << (8 * n)) - 1u);
  }
  return v;
}

// The row of x that row t of y multiplies, -1 for none.
__device__ __forceinline__ int64_t x_row(const MatmulArgs& a, int64_t t) {
  if (!a.pick) return t;
  const int64_t p = a.pick[t];
  return p >= 0 && p < a.Tx ? p : -1;
}

// ------------------------------------------------------------------------------------------------
// Few rows of x per matrix: the weights are read once, straight into registers, and bound the time.
// A workgroup owns RT * 16 rows of one expert's matrix and up to 16 rows of x; its waves take the blocks of
// columns in turn, U at a time, the next U or 2 U on their way while these are multiplied, and add their sums
// in wave order through LDS.
// QUANTIZE: x is bf16, fp16 or fp32. Its rows are quantised into LDS, eight lanes a block, while the first
// weights are on their way; the same codes and scales that the quantiser writes.
// A load takes 64 neighbouring bytes of 16 rows. Measured, the kernel alone: 4096 x 14336 with one row of bf16 11.6
// to 12.0 us (4.9 TB/s, a copy's rate is 5.2), 64 experts of 2048 x 2048 with 92 rows 33 us. The choice of RT and
// W stands at the plan; U = 1 with RT = 4 makes the least registers, and two groups of two there take 39 us instead of 34.
// ------------------------------------------------------------------------------------------------
constexpr int few_x_bytes(int64_t C) { return (int)(fp8_blocks(C) * kFp8Block + 16); }   // of a row in LDS

// meanwhile: called once the thread's first elements are on their way (loads return in order, so what it
// loads does not hold them up).
template <int TYPE, class F>
__device__ __forceinline__ void quantize_rows(const MatmulArgs& a, int64_t t0, int nt, int cb, uint8_t* codes,
                                              int row_bytes, float* scales, int threads, F meanwhile) {
  typedef typename Elem<TYPE>::T T;
  constexpr int V = 16, kLanes = kFp8Block / V;
  const int per_row = cb * kLanes;
  float v[V];
  auto load = [&](int i) __attribute__((always_inline)) {
    if (i >= nt * per_row) return;
    const int row = i / per_row, col = (i - row * per_row) * V, left = (int)a.C - col;
    const int64_t x = x_row(a, t0 + row);
    load_lane<TYPE, false>(static_cast<const T*>(a.x) + (x < 0 ? 0 : x) * a.ldx + col,
                           x < 0 || left < 0 ? 0 : left > V ? V : left, v);
  };
  load(threadIdx.x);
  meanwhile();
  for (int i = threadIdx.x; i < nt * per_row; i += threads) {
    const int row = i / per_row, col = (i - row * per_row) * V, left = (int)a.C - col;
    if (i >= threads) load(i);
    const float s = scale_of(block_max_u32_t<kLanes>(top_bits(v), kLanes));
    store_codes(v, s, left > V ? V : left, codes + row * row_bytes + col);
    if (threadIdx.x % kLanes == 0) scales[row * cb + col / kFp8Block] = s;
  }
}

template <int RT, int U, int W, bool QUANTIZE, bool WIDE>
__global__ __launch_bounds__(W * kWave, 1) void few_fp8_kernel(MatmulArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t id = block_id(), tile = id / a.row_blocks, rb = id % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, kMfma, tile, e, t0, t1)) return;
  const int64_t r0 = rb * (RT * kMfma);
  const int l = lane & 15, q = lane >> 4;
  const int cb = (int)fp8_blocks(a.C), whole = (int)(a.C / kFp8Block);
  const uint8_t* wp[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = r0 + i * kMfma + l;
    wp[i] = a.codes + ((int64_t)e * a.R + (r < a.R ? r : a.R - 1)) * a.ldw + 16 * q;
  }
  const float* sw = static_cast<const float*>(a.scales) +
                    ((int64_t)e * fp8_blocks(a.R) + r0 / kFp8Block) * cb;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  // lane group q takes the 16-byte pieces q and q + 4 of a block: 64 neighbouring bytes of a row a load.
  // The row's last, short block keeps the columns that exist.
  typedef u32x4 Group[U][RT][2];
  auto load = [&](Group& w, int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int b = b0 + n * W;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4* p = reinterpret_cast<const u32x4*>(wp[i] + (int64_t)b * kFp8Block + 64 * h);
          w[n][i][h] = zero;
          if (b < whole) {
            w[n][i][h] = *p;
          } else if (b < cb) {
            const int left = (int)a.C - b * kFp8Block - 64 * h - 16 * q;
            if (left > 0) w[n][i][h] = first_bytes(*p, left < 16 ? left : 16);
          }
        }
    }
  };
  Group w[2];
  const int nt = (int)(t1 - t0 < kMfma ? t1 - t0 : kMfma);
  const int row_bytes = few_x_bytes(a.C);
  const uint8_t* xp;
  const float* sx;
  bool in;
  int64_t xs_blk = 1;
  if constexpr (QUANTIZE) {
    uint8_t* codes = smem;
    float* scales = reinterpret_cast<float*>(smem + a.x_rows * row_bytes);
    auto first = [&]() __attribute__((always_inline)) { load(w[0], wave); };
    constexpr int kThreads = W * kWave;
    if (a.x_type == AAAC_BF16)
      quantize_rows<AAAC_BF16>(a, t0, nt, cb, codes, row_bytes, scales, kThreads, first);
    else if (a.x_type == AAAC_F16)
      quantize_rows<AAAC_F16>(a, t0, nt, cb, codes, row_bytes, scales, kThreads, first);
    else
      quantize_rows<AAAC_F32>(a, t0, nt, cb, codes, row_bytes, scales, kThreads, first);
    load(w[1], wave + U * W);
    step_barrier();                              // does not wait for the weights
    in = l < nt;
    xp = codes + (in ? l : 0) * row_bytes + 16 * q;
    sx = scales + (in ? l : 0) * cb;
  } else {
    load(w[0], wave);
    load(w[1], wave + U * W);
    const int64_t x = t0 + l < t1 ? x_row(a, t0 + l) : -1;
    in = x >= 0;
    xp = static_cast<const uint8_t*>(a.x) + (in ? x : 0) * a.ldx + 16 * q;
    sx = a.x_blocks + (in ? x : 0) * a.xs_row;
    xs_blk = a.xs_blk;
  }
  f32x4 acc[RT][1];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Group& w, int b0) __attribute__((always_inline)) {
    u32x4 x[U][2];
    float f[U];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int b = b0 + n * W;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4* p = reinterpret_cast<const u32x4*>(xp + (int64_t)b * kFp8Block + 64 * h);
        x[n][h] = zero;
        if (QUANTIZE ? b < cb : b < whole) {
          if (in) x[n][h] = *p;
        } else if (b < cb) {
          const int left = (int)a.C - b * kFp8Block - 64 * h - 16 * q;
          if (left > 0 && in) x[n][h] = first_bytes(*p, left < 16 ? left : 16);
        }
      }
      // a row that is none has the scale 0, as in the tiles: by an infinite scale of weights it is NaN too
      f[n] = b < cb ? (in ? sx[b * xs_blk] : 0.0f) * sw[b] : 0.0f;
    }
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const Frag<WIDE> xf = frag<WIDE>(x[n][0], x[n][1]);
#pragma unroll
      for (int i = 0; i < RT; ++i)
        acc[i][0] += block_sum(frag<WIDE>(w[n][i][0], w[n][i][1]), xf) * f[n];
    }
  };
  for (int b = wave; b < cb; b += 2 * U * W) {
    multiply(w[0], b);
    if (b + U * W >= cb) break;
    load(w[0], b + 2 * U * W);
    multiply(w[1], b + U * W);
    load(w[1], b + 3 * U * W);
  }
  if (QUANTIZE) __syncthreads();                 // the rows of x give way to the waves' sums
  join_and_store<RT, 1, W>(a, acc, r0, t0, t1, reinterpret_cast<float*>(smem));
}

template <int RT, int U, int W>
hipError_t few_fp8(MatmulArgs a, hipStream_t stream) {
  static_assert(W * kWave <= kGridThreads, "a grid's threads");
  const bool quantize = a.x_type != AAAC_FP8, wide = a.y_type != AAAC_BF16;
  a.row_blocks = (a.R + RT * kMfma - 1) / (RT * kMfma);
  const int64_t grid = a.row_blocks * token_tiles(a, kMfma);
  a.x_rows = (int)(a.T < kMfma ? a.T : kMfma);
  const int x_lds = quantize ? a.x_rows * (few_x_bytes(a.C) + 4 * (int)fp8_blocks(a.C)) : 0;
  const int lds = x_lds > join_bytes<RT, 1, W>() ? x_lds : join_bytes<RT, 1, W>();
  const auto kernel =
      quantize ? (wide ? few_fp8_kernel<RT, U, W, true, true> : few_fp8_kernel<RT, U, W, true, false>)
               : (wide ? few_fp8_kernel<RT, U, W, false, true> : few_fp8_kernel<RT, U, W, false, false>);
  hipLaunchKernelGGL(kernel, grid_of(grid), dim3(W * kWave), lds, stream, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------
// More rows: tiles of BM weight rows by BN rows of x, both staged through LDS, a block of 128 columns a
// step, in a ring of NS stages. The 16-byte pieces of a row lie permuted by row bits 1 to 3 (piece_turn). A
// stage ends with the step's scales: those of the tile's rows of x, then of its blocks of weight rows.
//
// The instruction is that of 32 x 32 results and 64 columns, two of them a block. Its operands take 16 of
// its 64 cycles to read, in which no vector instruction starts; the one of 16 x 16 by 128 columns takes as
// long for its 32 cycles, and the four multiply-adds and the rest of a block's vector work do not fit into
// what is left (4 vector instructions to one take 35 cycles, 6 take 47, 8 take 54; in the other, 12 to 64
// cycles take 68).
//
// A wave holds its fragments of x for the whole step and takes the 2 FR half fragments of weights in
// turn, two of them in registers: the products of one run while the next is there and the one after it is
// read. A stage is given back in two parts, so that loads run NS - 1/2 steps ahead: point A, before the
// products of the first half of the weight rows' last two half fragments (everything of that half and of x
// has been read), frees these for the step NS later, and point B, before the last two, the rest. The
// products at these points come from registers, so the matrix units work through the barriers. At either
// point all but the (NS - 1) kLoads youngest loads of a wave have to have arrived, and the loads that follow
// it are spread between the products: 64 lanes of 16 bytes take the address unit 16 cycles, all of a step's
// at once half of a step. Loads past the last step lie outside their buffers, so every step has the same
// count. A wave with one fragment of weights (FR = 1) has no first half and only point B.
//
// Measured, the kernel alone: 4096 rows against 14336 x 4096 237 to 246 us (1.95 PFLOP/s; the matrix instructions
// alone take 165, with their LDS reads and factors 210, the loads alone 117; 896 tiles are 3.5 rounds of 256 CUs, and a round ends
// with 7 us of stores), 16380 rows over 32 experts of 4096 x 2048 187 to 193 us, 48 rows against 14336 x 4096 15.3 us
// (3.8 TB/s).
// ------------------------------------------------------------------------------------------------
constexpr int kBig = 32;                         // rows and columns of the tiles' matrix instruction
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Half of a block: 64 columns, 32 codes a lane.
template <bool WIDE>
__device__ __forceinline__ f32x16 half_sum(const Frag<WIDE>& w, const Frag<WIDE>& x, f32x16 c) {
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w.v[i]),
                                                  __builtin_bit_cast(bf16x8, x.v[i]), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(w), operand(x), c, 0, 0, 0, 0, 0, 0);
  }
}

// A wave's result, FR * 32 weight rows by FT * 32 rows of x. A lane has row lane & 31 of x and, in registers
// 4 g .. 4 g + 3 of a fragment, weight rows 8 g + 4 (lane >> 5) and the next three. In 16 bits the two lanes of
// a row of x exchange halves, so that each stores eight neighbours, 16 bytes. Where they do not start on four
// bytes (every second row of y where R is odd) a lane stores those from the second on, with the next lane's
// first: 4096 rows against 14335 x 4096 take 243 us, with the 16 bytes on odd addresses 272, element by element
// 366, and against 14336 x 4096 231.
template <int FR, int FT>
__device__ __forceinline__ void store_big(const MatmulArgs& a, int part, const f32x16 (&acc)[FR][FT],
                                          int64_t t0, int64_t t1, int64_t r0) {
  const int lane = threadIdx.x & (kWave - 1), l = lane & 31, q = lane >> 5;
  if (a.y_type == AAAC_F32 || a.split > 1) {
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
      for (int i = 0; i < FR; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16 c = acc[i][j];
          const f32x4 v = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
          const int64_t t = t0 + j * kBig + l, r = r0 + i * kBig + 8 * g + 4 * q;
          if (t < t1 && r + 4 <= a.R && a.split == 1 && !a.y_vec)
            __builtin_memcpy(static_cast<float*>(a.y) + t * a.ldy + r, &v, 16);
          else if (t < t1 && r < a.R)
            store_part(a, part, t, r, v);
        }
    return;
  }
  constexpr int kPieces = 2 * FR;                // a lane's pieces of a row of x
  const bool shift = !a.y_row && (((uintptr_t)a.y & 2) || (a.ldy & 1)) && r0 + FR * kBig <= a.R;
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t t = t0 + j * kBig + l;
    uint16_t* y = static_cast<uint16_t*>(a.y) + t * a.ldy + r0;
    auto piece = [&](int n) __attribute__((always_inline)) {
      const f32x16 c = acc[n / 2][j];
      const int k = n % 2 * 8;
      const uint2 u = pack_16(a, f32x4{c[k], c[k + 1], c[k + 2], c[k + 3]});
      const uint2 v = pack_16(a, f32x4{c[k + 4], c[k + 5], c[k + 6], c[k + 7]});
      const auto lo = __builtin_amdgcn_permlane32_swap(u.x, v.x, false, false);
      const auto hi = __builtin_amdgcn_permlane32_swap(u.y, v.y, false, false);
      return u32x4{lo[0], hi[0], lo[1], hi[1]};
    };
    u32x4 w = piece(0);
    if (shift) {
      const uint32_t odd = (uintptr_t)y >> 1 & 1, bits = 16 * odd;
      if (t < t1 && odd && q == 0) y[0] = (uint16_t)w.x;
      y += odd + 8 * q;
#pragma unroll
      for (int n = 0; n < kPieces; ++n) {
        const u32x4 after = n + 1 < kPieces ? piece(n + 1) : u32x4{0u, 0u, 0u, 0u};
        // the next eight neighbours' first: the other lane's, of its next piece for the upper one
        const auto firsts = __builtin_amdgcn_permlane32_swap(w.x, after.x, false, false);
        const uint32_t first = q ? firsts[0] : firsts[1];
        const u32x4 v = {__builtin_amdgcn_alignbit(w.y, w.x, bits), __builtin_amdgcn_alignbit(w.z, w.y, bits),
                         __builtin_amdgcn_alignbit(w.w, w.z, bits), __builtin_amdgcn_alignbit(first, w.w, bits)};
        if (t < t1) {
          if (n + 1 < kPieces || !(odd && q)) {
            __builtin_memcpy(y + 16 * n, &v, 16);
          } else {
            __builtin_memcpy(y + 16 * n, &v, 12);
            y[16 * n + 6] = (uint16_t)v.w;
          }
        }
        w = after;
      }
      continue;
    }
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      if (n > 0) w = piece(n);
      const int64_t r = r0 + 16 * n + 8 * q;
      uint16_t* p = y + 16 * n + 8 * q;
      if (t < t1 && r + 8 <= a.R) {
        if (a.y_row) *reinterpret_cast<u32x4*>(p) = w;
        else __builtin_memcpy(p, &w, 16);
      } else if (t < t1) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r + k < a.R) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
}

template <int WR, int WT, int FR, int FT, int NS, bool WIDE>
__global__ __launch_bounds__(WR * WT * kWave, 2) void tile_fp8_kernel(MatmulArgs a) {
  constexpr int NW = WR * WT, BM = WR * FR * kBig, BN = WT * FT * kBig;
  constexpr int kW = BM * 128, kX = BN * 128, kS = NW * 256, kStage = kW + kX + kS;
  // fragments of a wave's weight rows in the first half, loads a wave of either half and of x
  constexpr bool kTwo = FR > 1;
  constexpr int kFirst = kTwo ? FR / 2 : FR;
  constexpr int kW0 = kFirst * WR * kBig / 8 / NW, kW1 = (FR - kFirst) * WR * kBig / 8 / NW, kXl = BN / 8 / NW;
  constexpr int kA = kW0 + kXl + 1, kLoads = kA + kW1;
  constexpr int kXWaves = (BN + kWave - 1) / kWave;          // waves that load scales of x
  static_assert(kFirst * WR * kBig % (8 * NW) == 0 && (FR - kFirst) * WR * kBig % (8 * NW) == 0 &&
                BN % (8 * NW) == 0, "whole loads a wave");
  static_assert(kXWaves < NW && FR * kBig <= kFp8Block, "the scales' loads");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * kStage];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  if (block_id() >= a.blocks) return;
  // fewer than 2^32 workgroups have a tile (2^31 tiles of 16 x 16 at most)
  const uint32_t id = (uint32_t)by_die(block_id(), a.blocks), tiles = (uint32_t)a.blocks / (uint32_t)a.split;
  const uint32_t part = id / tiles, row_blocks = (uint32_t)a.row_blocks;
  // tiles go in bands of kBand token tiles by all row blocks, the band's token tiles innermost, so that
  // a die's run of tiles shares rows of x and weights alike
  constexpr uint32_t kBand = 4;
  const uint32_t n_tok = tiles / row_blocks, in_part = id - part * tiles;
  const uint32_t band = in_part / (kBand * row_blocks), in_band = in_part - band * kBand * row_blocks;
  const uint32_t wide = n_tok - band * kBand < kBand ? n_tok - band * kBand : kBand;
  const uint32_t rb = in_band / wide, tile = band * kBand + (in_band - rb * wide);
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, BN, tile, e, t0, t1)) return;
  const int64_t r0 = (int64_t)rb * BM;
  const int nr = (int)(a.R - r0 < BM ? a.R - r0 : BM), nt = (int)(t1 - t0 < BN ? t1 - t0 : BN);
  const int64_t cb = fp8_blocks(a.C), rbs = fp8_blocks(a.R);
  // buffers end with the 16-byte piece that holds their last column; x has a row (plan_matmul), so none is empty
  const u32x4 wr = rows_buffer(a.codes + ((int64_t)e * a.R + r0) * a.ldw,
                               ((nr - 1) * a.ldw + a.C + 15) & ~(int64_t)15);
  const int64_t x0 = a.pick ? 0 : t0, xn = a.pick ? a.Tx : nt;
  const u32x4 xr = rows_buffer(static_cast<const uint8_t*>(a.x) + x0 * a.ldx,
                               ((xn - 1) * a.ldx + a.C + 15) & ~(int64_t)15);
  const int first = (int)(cb * part / a.split), steps = (int)(cb * (part + 1) / a.split);
  // the tile row where load n of the weights starts: the first half of every wave row's fragments, then
  // the second
  auto w_row = [&](int n) {
    const int h = n < kW0 ? 0 : 1, rows = (h ? FR - kFirst : kFirst) * kBig;
    const int r = h ? (wave * kW1 + n - kW0) * 8 : (wave * kW0 + n) * 8;
    return r / rows * (FR * kBig) + h * kFirst * kBig + r % rows;
  };
  // the column of a lane's 16 bytes in rows from an even and from an odd multiple of eight on
  const int col[2] = {((lane & 7) ^ piece_turn(lane >> 3)) * 16, ((lane & 7) ^ piece_turn((lane >> 3) + 8)) * 16};
  uint32_t woff[kW0 + kW1], xoff[kXl];
#pragma unroll
  for (int i = 0; i < kW0 + kW1; ++i) {
    const int row = w_row(i);
    woff[i] = row + (lane >> 3) < nr ? (row + (lane >> 3)) * (uint32_t)a.ldw + col[row >> 3 & 1] : kOutside;
  }
#pragma unroll
  for (int i = 0; i < kXl; ++i) {
    const int row = (wave * kXl + i) * 8;
    const int64_t x = row + (lane >> 3) < nt ? x_row(a, t0 + row + (lane >> 3)) : -1;
    xoff[i] = x >= 0 ? (uint32_t)(x - x0) * (uint32_t)a.ldx + col[row >> 3 & 1] : kOutside;
  }
  // this wave's scales: 64 rows of x, or the tile's blocks of weight rows
  const float* sbase;
  int64_t sstep, sbytes;
  uint32_t soff = kOutside;
  if (wave < kXWaves) {
    const int row = wave * kWave + lane;
    const int64_t x = row < nt ? x_row(a, t0 + row) : -1;
    if (x >= 0) soff = (uint32_t)((x - x0) * a.xs_row) * 4u;
    sbase = a.x_blocks + x0 * a.xs_row;
    sstep = a.xs_blk;
    sbytes = ((xn - 1) * a.xs_row + 1) * 4;
  } else {
    const int64_t r = r0 / kFp8Block, left = rbs - r;
    const int n = left < (BM + kFp8Block - 1) / kFp8Block ? (int)left : (BM + kFp8Block - 1) / kFp8Block;
    if (wave == kXWaves && lane < n) soff = (uint32_t)(lane * cb) * 4u;
    sbase = static_cast<const float*>(a.scales) + ((int64_t)e * rbs + r) * cb;
    sstep = 1;
    sbytes = ((n - 1) * cb + 1) * 4;
  }
  const uint32_t lds0 = lds_address(&lds[0]);
  // Loads of a step, one at a time: 0 .. kA - 1 its part A, kA .. kLoads - 1 its part B.
  auto load = [&](int slot, int kt, int n) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + slot * kStage;
    const bool in = kt < steps;
    const uint32_t more = in ? (uint32_t)kt * kFp8Block : 0u;
    // columns from the step's first on; a row's last step may have fewer
    const int left = in ? (int)a.C - kt * kFp8Block : 0;
    auto at = [&](uint32_t off, int row) { return left >= kFp8Block || col[row >> 3 & 1] < left ? off : kOutside; };
    if (n == kW0 + kXl) {
      load_lds4(rows_buffer(sbase + (in ? kt : 0) * sstep, sbytes), in ? soff : kOutside,
                dst + kW + kX + wave * 256);
    } else if (n >= kW0 && n < kW0 + kXl) {
      const int i = n - kW0, row = (wave * kXl + i) * 8;
      load_lds16(xr, at(xoff[i], row), more, dst + kW + row * 128);
    } else {
      const int i = n < kW0 ? n : n - kXl - 1, row = w_row(i);
      load_lds16(wr, at(woff[i], row), more, dst + row * 128);
    }
  };
  // Loads n0 .. n1 - 1, part `at` of `of` of them.
  auto loads = [&](int slot, int kt, int n0, int n1, int at, int of) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < kLoads; ++n)
      if (n >= n0 + (n1 - n0) * at / of && n < n0 + (n1 - n0) * (at + 1) / of) load(slot, kt, n);
  };
  // Arrived are all but the youngest N loads. Where step kt is the row's last and ends inside a 16-byte
  // piece, that piece keeps the columns that exist: of half h of the weights, and of x with half 0.
  auto arrive = [&](auto n, int slot, int kt, int h) __attribute__((always_inline)) {
    wait_loads<decltype(n)::value>();
    step_barrier();
    if ((a.C & 15) && kt == (int)cb - 1) {
      int from = tid;
      asm volatile("" : "+v"(from));             // keeps what this needs out of the loop's registers
      for (int r = from; r < BM + BN; r += NW * kWave) {
        if (r < BM ? (r / kBig % FR >= kFirst) != h : h) continue;
        const int piece = ((int)a.C & 127) >> 4;
        u32x4* p = reinterpret_cast<u32x4*>(lds + slot * kStage + r * 128 +
                                            (piece ^ piece_turn(r < BM ? r : r - BM)) * 16);
        *p = first_bytes(*p, (int)a.C & 15);
      }
      step_barrier();
    }
  };
  typedef Int<kTwo ? (NS - 1) * kLoads : (NS - 2) * kLoads> Younger;
  f32x16 acc[FR][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x16{};
  // neighbouring waves, on different SIMDs, share their rows of x; those past a partial tile's last
  // row only help to load
  const int wm = (wave % WR) * FR * kBig, wn = (wave / WR) * FT * kBig;
  const bool busy = wn < nt;
  const int l = lane & 31, q = lane >> 5;
  // the first piece of a lane's half fragment s: pieces 4 s + 2 q and the next
  const int p0 = ((2 * q) ^ piece_turn(l)) * 16;
  auto read = [&](const uint8_t* row, int s) __attribute__((always_inline)) {
    return frag<WIDE>(*reinterpret_cast<const u32x4*>(row + (p0 ^ (64 * s))),
                      *reinterpret_cast<const u32x4*>(row + (p0 ^ (64 * s + 16))));
  };
  auto walk = [&](auto with_products) __attribute__((always_inline)) {
    constexpr bool kMul = decltype(with_products)::value != 0;
    constexpr int G = 2 * FR;                    // half fragments of weights: fragment g / 2, half g % 2
    Frag<WIDE> xf[FT][2], wf[2];
    f32x16 p[FT];                                // a fragment of weights' sums over the block
    float f[FT], sx[FT], fw = 0.0f;              // factors of the block; scales of the next step's
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(s, first + s, n);
    arrive(Int<(NS - 1) * kLoads>(), 0, first, 0);
    auto scales = [&](const uint8_t* stage) __attribute__((always_inline)) {
      const float* sb = reinterpret_cast<const float*>(stage + kW + kX);
      fw = sb[kXWaves * kWave + wm / kFp8Block];
#pragma unroll
      for (int j = 0; j < FT; ++j) sx[j] = sb[wn + j * kBig + l];
    };
    if (kMul) {
      scales(lds);
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        xf[j][0] = read(lds + kW + (wn + j * kBig + l) * 128, 0);
        xf[j][1] = read(lds + kW + (wn + j * kBig + l) * 128, 1);
        p[j] = f32x16{};
        f[j] = 0.0f;
      }
      wf[0] = read(lds + (wm + l) * 128, 0);
      wf[1] = read(lds + (wm + l) * 128, 1);
    }
    int slot = 0;
    for (int kt = first; kt < steps; ++kt) {
      const int next = slot + 1 == NS ? 0 : slot + 1;
      const uint8_t* wb = lds + slot * kStage + (wm + l) * 128;
      const uint8_t* nb = lds + next * kStage;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        constexpr int kPointA = kTwo ? 2 * kFirst - 2 : -1, kPointB = G - 2;
        if (g == kPointA) arrive(Younger(), slot, kt, 1);
        if (g == kPointB) arrive(Younger(), next, kt + 1, 0);
        if (kMul) {
          const int i = g / 2, s = g % 2;
#pragma unroll
          for (int j = 0; j < FT; ++j) {
            if (s == 0) {
              // the sums of the fragment before; its factors are the step before's for the last one
              f32x16& sum = acc[i > 0 ? i - 1 : FR - 1][j];
              sum += p[j] * f[j];
              asm volatile("" : "+v"(sum));      // here, not behind the barriers that follow
              if (i == 0) f[j] = sx[j] * fw;
              p[j] = half_sum<WIDE>(wf[0], xf[j][0], f32x16{});
            } else {
              p[j] = half_sum<WIDE>(wf[1], xf[j][1], p[j]);
            }
            if (g >= kPointB) xf[j][s] = read(nb + kW + (wn + j * kBig + l) * 128, s);
          }
          wf[s] = g + 2 < G ? read(wb + (i + 1) * kBig * 128, s) : read(nb + (wm + l) * 128, s);
          if (g == G - 1) scales(nb);
        }
        if (kTwo) {
          // after A: part A of the step NS later; after B: its part B
          if (g >= kPointA && g < kPointB) loads(slot, kt + NS, 0, kA, g - kPointA, kPointB - kPointA);
          if (g >= kPointB) loads(slot, kt + NS, kA, kLoads, g - kPointB, 2);
        } else {
          loads(slot, kt + NS, 0, kLoads, g, 2);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      slot = next;
    }
    if (kMul) {
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[FR - 1][j] += p[j] * f[j];
    }
  };
  if (busy) walk(Int<1>());
  else walk(Int<0>());
  wait_loads<0>();                               // none may reach LDS after the workgroup has ended
  store_big<FR, FT>(a, (int)part, acc, t0 + wn, t1, r0 + wm);
}

template <int WR, int WT, int FR, int FT, int NS, bool WIDE>
hipError_t tile_fp8(MatmulArgs a, hipStream_t stream) {
  constexpr int BM = WR * FR * kBig, BN = WT * FT * kBig;
  a.row_blocks = (a.R + BM - 1) / BM;
  a.blocks = a.row_blocks * token_tiles(a, BN) * a.split;
  hipLaunchKernelGGL((tile_fp8_kernel<WR, WT, FR, FT, NS, WIDE>), grid_of(a.blocks),
                     dim3(WR * WT * kWave), 0, stream, a);
  return hipGetLastError();
}

template <bool WIDE>
hipError_t tile_fp8_any(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  switch (p.bn) {
    case 64:
      return p.bm == 64 ? tile_fp8<2, 2, 1, 1, 4, WIDE>(a, stream) : tile_fp8<2, 2, 2, 1, 3, WIDE>(a, stream);
    case 128: return tile_fp8<2, 2, 2, 2, 2, WIDE>(a, stream);
    default:
      // fragments of bf16 numbers leave no registers for more
      if constexpr (WIDE) return tile_fp8<2, 2, 2, 2, 2, WIDE>(a, stream);
      else return tile_fp8<2, 4, 4, 2, 2, WIDE>(a, stream);
  }
}

}  // namespace

hipError_t launch_few_fp8(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  if (p.rt == 4) return few_fp8<4, 1, 8>(a, stream);
  return p.rt == 2 ? few_fp8<2, 2, 8>(a, stream) : few_fp8<1, 2, 16>(a, stream);
}

hipError_t launch_tile_fp8(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return a.y_type == AAAC_BF16 ? tile_fp8_any<false>(a, p, stream) : tile_fp8_any<true>(a, p, stream);
}

}  // namespace aaac
