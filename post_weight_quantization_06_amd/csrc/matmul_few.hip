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

template <bool B, class X, class Y> struct Pick { typedef X type; };
template <class X, class Y> struct Pick<false, X, Y> { typedef Y type; };

constexpr int64_t kXLds = 64 << 10;              // LDS bytes for rows of x

// Adds the waves' sums acc[RT][NT] in wave order and stores them. red: join_bytes of LDS.
template <int RT, int NT, int W>
constexpr int join_bytes() { return W * NT * kMfma * (RT * kMfma + 4) * 4; }
template <int RT, int NT, int W>
__device__ __forceinline__ void join_and_store(const MatmulArgs& a, const f32x4 (&acc)[RT][NT],
                                               int64_t r0, int64_t t0, int64_t t1, float* red) {
  constexpr int kRow = RT * kMfma + 4;           // floats between x rows
  constexpr int kPart = NT * kMfma * kRow;       // and between waves
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(red + wave * kPart + (j * kMfma + (lane & 15)) * kRow + i * kMfma +
                                4 * (lane >> 4)) = acc[i][j];
  __syncthreads();
  for (int u = tid; u < NT * kMfma * RT * 4; u += W * kWave) {
    const int t = u / (RT * 4), r = 4 * (u % (RT * 4));
    const float* p = red + t * kRow + r;
    f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int w = 1; w < W; ++w) v += *reinterpret_cast<const f32x4*>(p + w * kPart);
    if (t0 + t < t1 && r0 + r < a.R) store4(a, t0 + t, r0 + r, v);
  }
}

// Bytes between the rows of x in LDS: whole 1 KB pieces, and 16 more to spread a column over banks.
__host__ __device__ __forceinline__ int64_t x_row_bytes(int64_t C) {
  return (2 * C + 1023) / 1024 * 1024 + 16;
}

// ------------------------------------------------------------------------------------------------
// bf16 rows of x times decoded weights. Instruction p of a chunk of 128 columns takes columns
// 32 p + 8 q .. 32 p + 8 q + 7 from lane group q. U chunks in a row go to one wave, the groups of U
// to the waves in turn, the loads of a wave's next group under way while it uses one. The count of
// load instructions bounds this kernel before their bytes do, hence one scale load for four chunks
// (U = 4), and x in LDS where the tile's rows fit into a.x_rows of them; otherwise x is read
// directly, 64 neighbouring bytes a row, and rows past the tile's last load as zeros.
// 14336 columns by 4096 rows in MXFP4, one row of x: 11.1 us, 2.8 TB/s (the reads of x and of the scales
// took 3 us each of 14 before they were gathered); 32 experts of 2048 x 4096, 61 rows: 28 us, 5.1 TB/s.
// In the packed format the decoding bounds it: some seven vector instructions a weight with scale
// groups of 16, five with 128.
// ------------------------------------------------------------------------------------------------
template <class D, int RT, int NT, int W, int U>
__global__ __launch_bounds__(W * kWave, 1) void few_bf16_kernel(MatmulArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t id = block_id(), tile = id / a.row_blocks, rb = id % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, NT * kMfma, tile, e, t0, t1)) return;
  const int64_t r0 = rb * (RT * kMfma);
  const int nt = (int)(t1 - t0 < NT * kMfma ? t1 - t0 : NT * kMfma);
  const int64_t x_bytes = (nt - 1) * a.ldx * 2 + a.C * 2;
  const void* x0 = static_cast<const uint16_t*>(a.x) + t0 * a.ldx;
  const int xstride = (int)x_row_bytes(a.C);
  const bool in_lds = nt <= a.x_rows;
  if (in_lds) {
    const u32x4 xb = rows_buffer(x0, x_bytes);
    const uint32_t base = lds_address(smem);
    const int pieces = xstride / 1024;
    for (int i = wave; i < nt * pieces; i += W) {
      const int row = i / pieces, col = (i % pieces) * 512 + lane * 8;
      load_lds16(xb, col < a.C ? (uint32_t)(row * a.ldx + col) * 2 : kOutside, 0,
                 base + row * xstride + (i % pieces) * 1024);
    }
  }
  const __amdgpu_buffer_rsrc_t xr = rows_rsrc(x0, x_bytes);
  D dec;
  dec.init(a, e);
  typename D::Row w[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = r0 + i * kMfma + (lane & 15);
    w[i] = dec.row(a, e, r < a.R ? r : a.R - 1);
  }
  const int q = lane >> 4;
  // where this lane's 16 bytes of x rows start: in LDS rows past the last repeat it
  uint32_t xoff[NT];
  const uint8_t* xlds[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = j * kMfma + (lane & 15);
    xoff[j] = t < nt ? (uint32_t)((t * a.ldx + 8 * q) * 2) : kOutside;
    xlds[j] = smem + (t < nt ? t : nt - 1) * xstride + 16 * q;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4 zero = {0u, 0u, 0u, 0u};

  // one chunk's products; `cut`: columns at or past the row's end are zero times zero
  auto multiply = [&](int c, const typename D::Chunk (&u)[RT], auto from_lds, bool cut)
      __attribute__((always_inline)) {
    u32x4 x[NT][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bool in = !cut || c * 128 + 32 * p + 8 * q < a.C;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (decltype(from_lds)::value)           // LDS rows are padded with zeros
          x[j][p] = in ? *reinterpret_cast<const u32x4*>(xlds[j] + c * 256 + 64 * p) : zero;
        else
          x[j][p] = buffer_load16(xr, in ? xoff[j] + (uint32_t)(c * 256 + 64 * p) : kOutside);
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      u32x4 wv[4];
      dec.decode_chunk(u[i], q, wv);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (cut && c * 128 + 32 * p + 8 * q >= a.C) wv[p] = zero;
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma_bf16(wv[p], x[j][p], acc[i][j]);
      }
    }
  };
  const int whole = (int)(a.C >> 7), groups = whole / U;
  typedef typename Pick<U == 4, typename D::Four, typename D::Chunk>::type Group;
  auto load = [&](int g, Group (&u)[RT]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if constexpr (U == 4) u[i] = dec.load_four(a, w[i], 4 * g, q);
      else u[i] = dec.load_chunk(a, w[i], g, q);
    }
  };
  auto use = [&](int g, const Group (&u)[RT], auto from_lds) __attribute__((always_inline)) {
    if constexpr (U == 4) {
      u32x4 s[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) s[i] = D::spread(u[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        typename D::Chunk v[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) v[i] = D::chunk(u[i], s[i], k);
        multiply(4 * g + k, v, from_lds, false);
      }
    } else {
      multiply(g, u, from_lds, false);
    }
  };
  Group even[RT], odd[RT];
  int g = wave;
  if (g < groups) load(g, even);
  auto run = [&](auto from_lds) __attribute__((always_inline)) {
    while (g < groups) {
      if (g + W < groups) load(g + W, odd);
      use(g, even, from_lds);
      g += W;
      if (g >= groups) break;
      if (g + W < groups) load(g + W, even);
      use(g, odd, from_lds);
      g += W;
    }
    // what is left of the row, a chunk a wave
    for (int c = groups * U + (wave + W - groups % W) % W; c * 128 < a.Cp; c += W) {
      typename D::Chunk v[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        v[i] = c < whole ? dec.load_chunk(a, w[i], c, q) : dec.load_last(a, w[i], c, q);
      multiply(c, v, from_lds, c >= whole);
    }
  };
  if (in_lds) {
    wait_loads<0>();
    step_barrier();
    run(Int<1>());
  } else {
    run(Int<0>());
  }
  __syncthreads();                               // the rows of x give way to the waves' sums
  join_and_store<RT, NT, W>(a, acc, r0, t0, t1, reinterpret_cast<float*>(smem));
}

// ------------------------------------------------------------------------------------------------
// MXFP4 x times MXFP4 weights: the scaled matrix instruction takes codes and scale bytes as they
// are stored. Run q of a lane is one block of 32 columns; a chunk is 512 columns, so that a lane
// reads the 16 scale bytes of its row in one load and takes byte 4 j + q for instruction j. One row
// against 14336 x 4096, quantised in the call: 12 us.
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
  const int64_t id = block_id(), tile = id / a.row_blocks, rb = id % a.row_blocks;
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
  __shared__ float red[join_bytes<RT, NT, W>() / 4];
  join_and_store<RT, NT, W>(a, acc, r0, t0, t1, red);
}

template <int RT, int NT>
int64_t few_grid(MatmulArgs& a) {
  a.row_blocks = (a.R + RT * kMfma - 1) / (RT * kMfma);
  return a.row_blocks * token_tiles(a, NT * kMfma);
}

template <class D, int RT, int NT, int W, int U>
hipError_t few_bf16(MatmulArgs a, hipStream_t stream) {
  const int64_t grid = few_grid<RT, NT>(a);
  // x rows in LDS, as many as leave two workgroups room on a CU
  const int64_t most = kXLds / x_row_bytes(a.C), want = a.T < NT * kMfma ? a.T : NT * kMfma;
  a.x_rows = (int)(most < want ? most : want);
  const int64_t x_lds = a.x_rows * x_row_bytes(a.C);
  const int lds = (int)(x_lds > join_bytes<RT, NT, W>() ? x_lds : join_bytes<RT, NT, W>());
  hipLaunchKernelGGL((few_bf16_kernel<D, RT, NT, W, U>), grid_of(grid), dim3(W * kWave), lds,
                     stream, a);
  return hipGetLastError();
}

// Only decoders that read their scales for four chunks at a time have the form with groups of four.
template <class D>
hipError_t few_bf16_any(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  if constexpr (D::kFour) {
    if (p.rt == 1 && p.chunks == 4) return few_bf16<D, 1, 1, 8, 4>(a, stream);
  }
  return p.rt == 2 ? few_bf16<D, 2, 1, 8, 1>(a, stream) : few_bf16<D, 1, 1, 8, 1>(a, stream);
}

template <int RT, int NT, int W>
hipError_t few_mxfp4(MatmulArgs a, hipStream_t stream) {
  const int64_t grid = few_grid<RT, NT>(a);
  hipLaunchKernelGGL((few_mxfp4_kernel<RT, NT, W>), grid_of(grid), dim3(W * kWave), 0, stream,
                     a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_mxfp4(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  if (p.nt == 1)
    return p.rt == 2 ? few_mxfp4<2, 1, 8>(a, stream) : few_mxfp4<1, 1, 8>(a, stream);
  return p.rt == 2 ? few_mxfp4<2, 2, 8>(a, stream) : few_mxfp4<1, 2, 8>(a, stream);
}

hipError_t launch_few_mx_bf16(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return few_bf16_any<MxDecoder>(a, p, stream);
}

hipError_t launch_few_packed(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return with_packed_decoder<false>(
      a, [&](auto d) { return few_bf16_any<decltype(d)>(a, p, stream); });
}

}  // namespace aaac
