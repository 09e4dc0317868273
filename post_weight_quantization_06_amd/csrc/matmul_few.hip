// Products with few rows of x per matrix: the weights are read once, straight into registers, and
// bound the time.
//
// A workgroup owns RT * 16 rows of one expert's matrix and up to NT * 16 rows of x; its waves split
// the columns in chunks and add their sums in wave order through LDS, so results are bitwise
// reproducible. Matrix instructions take 16 weight rows as the A operand and 16 rows of x as B: lane
// l holds, for weight row (and x row) l & 15, the columns of run l >> 4, and in the result four
// neighbouring weight rows of x row l & 15.
#include "matmul.h"

namespace aaac {

namespace {

// Adds the waves' sums acc[RT][NT] in wave order and stores them.
template <int RT, int NT, int W>
__device__ __forceinline__ void join_and_store(const MatmulArgs& a, const f32x4 (&acc)[RT][NT],
                                               int64_t r0, int64_t t0, int64_t t1) {
  constexpr int kRowsPad = RT * kMfma + 4;       // floats between x rows
  __shared__ float red[W][NT * kMfma][kRowsPad];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(&red[wave][j * kMfma + (lane & 15)][i * kMfma + 4 * (lane >> 4)]) =
          acc[i][j];
  __syncthreads();
  for (int u = tid; u < NT * kMfma * RT * 4; u += W * kWave) {
    const int t = u / (RT * 4), r = 4 * (u % (RT * 4));
    f32x4 v = *reinterpret_cast<const f32x4*>(&red[0][t][r]);
#pragma unroll
    for (int w = 1; w < W; ++w) v += *reinterpret_cast<const f32x4*>(&red[w][t][r]);
    if (t0 + t < t1 && r0 + r < a.R) store4(a, t0 + t, r0 + r, v);
  }
}

// ------------------------------------------------------------------------------------------------
// bf16 rows of x times decoded weights. A chunk is 128 columns: run q of a lane is the 32 columns
// 32 q .. 32 q + 31 of the chunk, and instruction j of a chunk takes columns 8 j .. 8 j + 7 of every
// run (weights and x in the same order, so the order does not matter to the sum).
// ------------------------------------------------------------------------------------------------
template <class D, int RT, int NT, int W>
__global__ __launch_bounds__(W * kWave) void few_bf16_kernel(MatmulArgs a) {
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t tile = blockIdx.x / a.row_blocks, rb = blockIdx.x % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, NT * kMfma, tile, e, t0, t1)) return;
  const int64_t r0 = rb * (RT * kMfma);
  D dec;
  dec.init(a, e);
  typename D::Row w[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = r0 + i * kMfma + (lane & 15);
    w[i] = dec.row(a, e, r < a.R ? r : a.R - 1);
  }
  const uint16_t* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = t0 + j * kMfma + (lane & 15);
    xp[j] = static_cast<const uint16_t*>(a.x) + (t < t1 ? t : t1 - 1) * a.ldx;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int run = 32 * (lane >> 4);
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int64_t c = (int64_t)wave * 128; c < a.Cp; c += W * 128) {
    const int64_t k = c + run;
    const bool whole = c + 128 <= a.C;           // uniform: every run of the chunk lies in the row
    const bool in = k < a.Cp;
    const int64_t kl = in ? k : 0;
    typename D::Run u[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) u[i] = dec.load(a, w[i], kl);
    u32x4 x[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (whole) {
          x[j][p] = *reinterpret_cast<const u32x4*>(xp[j] + k + 8 * p);
        } else {
          x[j][p] = zero;                        // columns past the row's end: zero times zero
          if (k + 8 * p < a.C) x[j][p] = *reinterpret_cast<const u32x4*>(xp[j] + k + 8 * p);
        }
      }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      u32x4 wv[4];
      dec.decode(a, u[i], wv);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (!whole && k + 8 * p >= a.C) wv[p] = zero;
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma_bf16(wv[p], x[j][p], acc[i][j]);
      }
    }
  }
  join_and_store<RT, NT, W>(a, acc, r0, t0, t1);
}

// ------------------------------------------------------------------------------------------------
// MXFP4 x times MXFP4 weights: the scaled matrix instruction takes codes and scale bytes as they
// are stored. Run q of a lane is one block of 32 columns; a chunk is 512 columns, so that a lane
// reads the 16 scale bytes of its row in one load and takes byte 4 j + q for instruction j.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ u32x4 load_scales(const uint8_t* p, int64_t left) {
  u32x4 v;
  if (left >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    v = u32x4{w[0], w[1], w[2], w[3]};
  }
  return v;
}

template <int RT, int NT, int W>
__global__ __launch_bounds__(W * kWave) void few_mxfp4_kernel(MatmulArgs a) {
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t tile = blockIdx.x / a.row_blocks, rb = blockIdx.x % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, NT * kMfma, tile, e, t0, t1)) return;
  const int64_t r0 = rb * (RT * kMfma);
  const int64_t kb = a.Cp >> 5;                  // blocks in a row
  const uint8_t *wp[RT], *wsp[RT], *xp[NT], *xsp[NT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = r0 + i * kMfma + (lane & 15);
    const int64_t row = (int64_t)e * a.R + (r < a.R ? r : a.R - 1);
    wp[i] = a.codes + row * (a.Cp >> 1);
    wsp[i] = static_cast<const uint8_t*>(a.scales) + row * kb;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    int64_t t = t0 + j * kMfma + (lane & 15);
    t = t < t1 ? t : t1 - 1;
    xp[j] = static_cast<const uint8_t*>(a.x) + t * (a.Cp >> 1);
    xsp[j] = a.x_scales + t * kb;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int q = lane >> 4;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int64_t b0 = (int64_t)wave * 16; b0 < kb; b0 += W * 16) {
    const int64_t left = kb - b0;
    u32x4 ws[RT], xs[NT], wc[RT][4], xc[NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      ws[i] = load_scales(wsp[i] + b0, left);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        wc[i][p] = zero;                         // past the row's end: zero codes, scale byte 0
        if (4 * p + q < left)
          wc[i][p] = *reinterpret_cast<const u32x4*>(wp[i] + (b0 + 4 * p + q) * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      xs[j] = load_scales(xsp[j] + b0, left);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        xc[j][p] = zero;
        if (4 * p + q < left)
          xc[j][p] = *reinterpret_cast<const u32x4*>(xp[j] + (b0 + 4 * p + q) * 16);
      }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t sx[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) sx[j] = xs[j][p] >> (8 * q);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const uint32_t sw = ws[i][p] >> (8 * q);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = mfma_fp4<0>(wc[i][p], xc[j][p], acc[i][j], sw, sx[j]);
      }
    }
  }
  join_and_store<RT, NT, W>(a, acc, r0, t0, t1);
}

template <int RT, int NT>
int64_t few_grid(MatmulArgs& a) {
  a.row_blocks = (a.R + RT * kMfma - 1) / (RT * kMfma);
  a.y_vec = can_store4(a);
  return a.row_blocks * token_tiles(a, NT * kMfma);
}

template <class D>
hipError_t few_bf16(MatmulArgs a, hipStream_t stream) {
  const int64_t grid = few_grid<1, 1>(a);
  hipLaunchKernelGGL((few_bf16_kernel<D, 1, 1, 4>), dim3((unsigned)grid), dim3(4 * kWave), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_mxfp4(MatmulArgs a, hipStream_t stream) {
  const int64_t grid = few_grid<1, 1>(a);
  hipLaunchKernelGGL((few_mxfp4_kernel<1, 1, 4>), dim3((unsigned)grid), dim3(4 * kWave), 0, stream,
                     a);
  return hipGetLastError();
}

hipError_t launch_few_mx_bf16(const MatmulArgs& a, hipStream_t stream) {
  return few_bf16<MxDecoder>(a, stream);
}

hipError_t launch_few_packed(const MatmulArgs& a, hipStream_t stream) {
  const int gpl = a.log2g >= 5 ? 1 : 32 >> a.log2g, spl = a.log2S >= 5 ? 1 : 32 >> a.log2S;
  if (!a.bitmap) {
    if (gpl == 1) return few_bf16<PackedDecoder<1, 1, true>>(a, stream);
    if (gpl == 2) return few_bf16<PackedDecoder<2, 2, true>>(a, stream);
    return few_bf16<PackedDecoder<4, 4, true>>(a, stream);
  }
  if (gpl == 1 && spl == 1) return few_bf16<PackedDecoder<1, 1, false>>(a, stream);
  if (gpl == 1 && spl == 2) return few_bf16<PackedDecoder<1, 2, false>>(a, stream);
  if (gpl == 1) return few_bf16<PackedDecoder<1, 4, false>>(a, stream);
  return few_bf16<PackedDecoder<2, 4, false>>(a, stream);
}

namespace {

// The 32-bit offsets of the tiles' loads reach every row of a tile.
bool tiles_fit(const MatmulArgs& a) { return a.ldx < ((int64_t)1 << 21); }

}  // namespace

hipError_t launch_mxfp4_matmul(const MatmulArgs& a, bool x_mxfp4, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const bool many = a.T > 64 * (int64_t)a.E;
  if (x_mxfp4) return many ? launch_tile_mxfp4(a, stream) : launch_few_mxfp4(a, stream);
  return many && tiles_fit(a) ? launch_tile_mx_bf16(a, stream) : launch_few_mx_bf16(a, stream);
}

hipError_t launch_packed_matmul(const MatmulArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const bool many = a.T > 64 * (int64_t)a.E && tiles_fit(a);
  return many ? launch_tile_packed(a, stream) : launch_few_packed(a, stream);
}

}  // namespace aaac
