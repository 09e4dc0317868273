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
// bf16 rows of x times decoded weights. Instruction p of a chunk of 128 columns takes columns
// 32 p + 8 q .. 32 p + 8 q + 7 from lane group q, so a load of x reads 64 neighbouring bytes of each
// row. The chunks go to the waves in turn, U at a time, so that U loads of each weight row are in
// flight. Rows past the tile's last lie outside the x buffer and load as zeros.
// ------------------------------------------------------------------------------------------------
template <class D, int RT, int NT, int W, int U>
__global__ __launch_bounds__(W * kWave, 1) void few_bf16_kernel(MatmulArgs a) {
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
  const int64_t nt = t1 - t0 < NT * kMfma ? t1 - t0 : NT * kMfma;
  const __amdgpu_buffer_rsrc_t xr = rows_rsrc(
      static_cast<const uint16_t*>(a.x) + t0 * a.ldx, (nt - 1) * a.ldx * 2 + a.C * 2);
  const int q = lane >> 4;
  uint32_t xoff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    xoff[j] = j * kMfma + (lane & 15) < nt
                  ? (uint32_t)(((j * kMfma + (lane & 15)) * a.ldx + 8 * q) * 2) : kOutside;
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4 zero = {0u, 0u, 0u, 0u};

  const int whole = (int)(a.C >> 7);             // chunks whose every run lies in the row
  auto chunks = [&](int c, auto n) {
    constexpr int N = decltype(n)::value;
    typename D::Chunk u[N][RT];
    u32x4 x[N][NT][4];
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i) u[s][i] = dec.load_chunk(a, w[i], c + s * W, q);
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p)
          x[s][j][p] = buffer_load16(xr, xoff[j] + (uint32_t)((c + s * W) * 256 + 64 * p));
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        u32x4 wv[4];
        dec.decode_chunk(u[s][i], q, wv);
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mfma_bf16(wv[p], x[s][j][p], acc[i][j]);
      }
  };
  int c = wave;
  for (; c + (U - 1) * W < whole; c += U * W) chunks(c, Int<U>());
  if (U > 1)
    for (; c < whole; c += W) chunks(c, Int<1>());
  if (c == whole && (int64_t)whole * 128 < a.Cp) {
    // the row's last columns: zero times zero past its end
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      u32x4 wv[4];
      dec.decode_chunk(dec.load_last(a, w[i], whole, q), q, wv);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const bool in = (int64_t)whole * 128 + 32 * p + 8 * q < a.C;
        if (!in) wv[p] = zero;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = mfma_bf16(
              wv[p], buffer_load16(xr, in ? xoff[j] + (uint32_t)(whole * 256 + 64 * p) : kOutside),
              acc[i][j]);
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
__device__ __forceinline__ u32x4 load_scales(const uint8_t* p, int left) {
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
__global__ __launch_bounds__(W * kWave, 1) void few_mxfp4_kernel(MatmulArgs a) {
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t tile = blockIdx.x / a.row_blocks, rb = blockIdx.x % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, NT * kMfma, tile, e, t0, t1)) return;
  const int64_t r0 = rb * (RT * kMfma);
  const int kb = (int)(a.Cp >> 5);               // blocks in a row
  const uint8_t *wp[RT], *wsp[RT], *xsp[NT];
  const int q = lane >> 4;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = r0 + i * kMfma + (lane & 15);
    const int64_t row = (int64_t)e * a.R + (r < a.R ? r : a.R - 1);
    wp[i] = a.codes + row * (a.Cp >> 1);
    wsp[i] = static_cast<const uint8_t*>(a.scales) + row * kb;
  }
  const int64_t nt = t1 - t0 < NT * kMfma ? t1 - t0 : NT * kMfma;
  const __amdgpu_buffer_rsrc_t xr =
      rows_rsrc(static_cast<const uint8_t*>(a.x) + t0 * (a.Cp >> 1), nt * (a.Cp >> 1));
  uint32_t xoff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = j * kMfma + (lane & 15);
    const bool in = t < nt;
    xoff[j] = in ? (uint32_t)(t * (a.Cp >> 1)) : kOutside;
    xsp[j] = a.x_scales + (t0 + (in ? t : 0)) * kb;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  auto chunk = [&](int b0, auto all) {
    constexpr bool ALL = decltype(all)::value;   // every block of the chunk lies in the row
    const int left = ALL ? 16 : kb - b0;
    u32x4 ws[RT], xs[NT], wc[RT][4], xc[NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      ws[i] = load_scales(wsp[i] + b0, left);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        wc[i][p] = zero;                         // past the row's end: zero codes, scale byte 0
        if (ALL || 4 * p + q < left)
          wc[i][p] = *reinterpret_cast<const u32x4*>(wp[i] + (b0 + 4 * p + q) * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      xs[j] = load_scales(xsp[j] + b0, left);
#pragma unroll
      for (int p = 0; p < 4; ++p)
        xc[j][p] = buffer_load16(xr, ALL || 4 * p + q < left
                                         ? xoff[j] + (uint32_t)((b0 + 4 * p + q) * 16) : kOutside);
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
  };
  int b0 = wave * 16;
  for (; b0 + 16 <= kb; b0 += W * 16) chunk(b0, Int<1>());
  if (b0 < kb) chunk(b0, Int<0>());
  join_and_store<RT, NT, W>(a, acc, r0, t0, t1);
}

template <int RT, int NT>
int64_t few_grid(MatmulArgs& a) {
  a.row_blocks = (a.R + RT * kMfma - 1) / (RT * kMfma);
  return a.row_blocks * token_tiles(a, NT * kMfma);
}

template <class D, int RT, int NT, int W, int U>
hipError_t few_bf16(MatmulArgs a, hipStream_t stream) {
  const int64_t grid = few_grid<RT, NT>(a);
  hipLaunchKernelGGL((few_bf16_kernel<D, RT, NT, W, U>), dim3((unsigned)grid), dim3(W * kWave), 0,
                     stream, a);
  return hipGetLastError();
}

template <class D>
hipError_t few_bf16_any(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  if (p.nt == 1) {
    if (p.rt == 2) return few_bf16<D, 2, 1, 8, 2>(a, stream);
    return p.waves == 16 ? few_bf16<D, 1, 1, 16, 1>(a, stream) : few_bf16<D, 1, 1, 8, 1>(a, stream);
  }
  if (p.rt == 2) return few_bf16<D, 2, 2, 8, 1>(a, stream);
  return p.waves == 16 ? few_bf16<D, 1, 2, 16, 1>(a, stream) : few_bf16<D, 1, 2, 8, 1>(a, stream);
}

template <int RT, int NT, int W>
hipError_t few_mxfp4(MatmulArgs a, hipStream_t stream) {
  const int64_t grid = few_grid<RT, NT>(a);
  hipLaunchKernelGGL((few_mxfp4_kernel<RT, NT, W>), dim3((unsigned)grid), dim3(W * kWave), 0, stream,
                     a);
  return hipGetLastError();
}

template <int NT>
hipError_t few_mxfp4_any(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  if (p.rt == 2) return few_mxfp4<2, NT, 8>(a, stream);
  return p.waves == 16 ? few_mxfp4<1, NT, 16>(a, stream) : few_mxfp4<1, NT, 8>(a, stream);
}

}  // namespace

hipError_t launch_few_mxfp4(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  switch (p.nt) {
    case 1: return few_mxfp4_any<1>(a, p, stream);
    case 2: return few_mxfp4_any<2>(a, p, stream);
    case 3: return few_mxfp4_any<3>(a, p, stream);
    default: return few_mxfp4_any<4>(a, p, stream);
  }
}

hipError_t launch_few_mx_bf16(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return few_bf16_any<MxDecoder>(a, p, stream);
}

hipError_t launch_few_packed(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return with_packed_decoder(a, [&](auto d) { return few_bf16_any<decltype(d)>(a, p, stream); });
}

}  // namespace aaac
