// Products with many rows of x per matrix: tiles of weight rows by rows of x, both staged through
// LDS, bound by the matrix units.
#include "matmul.h"

namespace aaac {

namespace {

typedef __attribute__((address_space(3))) void* LdsPtr;

// rows_rsrc as the four words that an assembly operand takes.
__device__ __forceinline__ u32x4 rows_buffer(const void* p, int64_t bytes) {
  const uint64_t b = (uint64_t)p;
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, (uint32_t)bytes, 0x00027000u};
}

// Asynchronous loads from a buffer into LDS: lane l's bytes land at dst + l * size (dst uniform).
// In assembly because the compiler would wait for them before any LDS read, of the other stage too;
// the caller waits (stage_ready) before the barrier after which they are read. The move to m0 needs
// one wait state before the load.
__device__ __forceinline__ void load_lds16(u32x4 buf, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(dst), "v"(off), "s"(buf) : "memory");
}
__device__ __forceinline__ void load_lds4(u32x4 buf, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(dst), "v"(off), "s"(buf) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(LdsPtr)(void*)p;
}
// This wave's loads have landed; after the barrier every wave's have.
__device__ __forceinline__ void stage_ready() {
  __builtin_amdgcn_s_waitcnt(0x0f70);           // vmcnt(0)
  __syncthreads();
}

// Workgroups go to the eight dies in turn; numbering them so that a die gets consecutive tiles lets
// its L2 serve the rows that neighbouring tiles share.
constexpr int kDies = 8;
__device__ __forceinline__ int64_t by_die(int64_t b, int64_t n) {
  const int64_t per = n / kDies, rest = n % kDies, d = b % kDies, i = b / kDies;
  return d * per + (d < rest ? d : rest) + i;
}

// ------------------------------------------------------------------------------------------------
// MXFP4 x times MXFP4 weights. A tile is BM weight rows by BN rows of x; a step takes 256 columns
// (128 bytes of codes and 8 scale bytes a row). Lane l of a matrix instruction holds blocks 2 q and
// 2 q + 1 (q = l >> 4) of its row for the step's two halves, so its two scale bytes are neighbours.
// In LDS the eight 16-byte pieces of a row lie permuted by the row's low bits, which spreads a
// column of pieces over all banks.
// ------------------------------------------------------------------------------------------------
template <int WR, int WT, int FR, int FT, bool WHOLE>
__global__ __launch_bounds__(WR * WT * kWave, 1) void tile_mxfp4_kernel(MatmulArgs a) {
  constexpr int NW = WR * WT, BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  constexpr int kW = BM * 128, kX = BN * 128, kWs = BM * 8, kXs = BN * 8;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][kW + kX + kWs + kXs];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  const int64_t id = by_die(blockIdx.x, gridDim.x), tiles = gridDim.x / a.split;
  const int part = (int)(id / tiles);
  const int64_t tile = id % tiles / a.row_blocks, rb = id % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, BN, tile, e, t0, t1)) return;
  const int64_t r0 = rb * BM;
  const int64_t row_bytes = a.Cp >> 1, kb = a.Cp >> 5;
  const int64_t nr = a.R - r0 < BM ? a.R - r0 : BM, nt = t1 - t0 < BN ? t1 - t0 : BN;
  const int64_t wrow = (int64_t)e * a.R + r0;
  const u32x4 wr = rows_buffer(a.codes + wrow * row_bytes, nr * row_bytes);
  const u32x4 xr =
      rows_buffer(static_cast<const uint8_t*>(a.x) + t0 * row_bytes, nt * row_bytes);
  const uint8_t* ws = static_cast<const uint8_t*>(a.scales) + wrow * kb;
  const uint8_t* xs = a.x_scales + t0 * kb;
  const u32x4 wsr = rows_buffer(ws, nr * kb), xsr = rows_buffer(xs, nt * kb);

  const int piece = (lane & 7) ^ (lane >> 3);    // the 16-byte piece of the row that a lane loads
  const uint32_t lds0 = lds_address(&lds[0][0]);
  auto load = [&](int buf, int64_t kt) {
    const uint32_t dst = lds0 + buf * (kW + kX + kWs + kXs);
    const bool in = WHOLE || kt * 8 + piece < kb;
    const uint32_t col = (uint32_t)(kt * 128) + piece * 16;
    const uint32_t off0 = (uint32_t)(lane >> 3) * (uint32_t)row_bytes + col;
#pragma unroll
    for (int i = 0; i < BM / 8 / NW; ++i) {
      const int row = (wave * (BM / 8 / NW) + i) * 8;
      load_lds16(wr, in ? off0 + row * (uint32_t)row_bytes : kOutside, dst + row * 128);
    }
#pragma unroll
    for (int i = 0; i < BN / 8 / NW; ++i) {
      const int row = (wave * (BN / 8 / NW) + i) * 8;
      load_lds16(xr, in ? off0 + row * (uint32_t)row_bytes : kOutside, dst + kW + row * 128);
    }
    if (WHOLE) {
      const uint32_t soff = (uint32_t)(lane >> 1) * (uint32_t)kb + (uint32_t)(kt * 8) + 4 * (lane & 1);
#pragma unroll
      for (int i = 0; i < BM / 32; i += NW)
        if (BM / 32 % NW == 0 || i + wave < BM / 32)
          load_lds4(wsr, soff + (i + wave) * 32 * (uint32_t)kb, dst + kW + kX + (i + wave) * 256);
#pragma unroll
      for (int i = 0; i < BN / 32; i += NW)
        if (BN / 32 % NW == 0 || i + wave < BN / 32)
          load_lds4(xsr, soff + (i + wave) * 32 * (uint32_t)kb,
                    dst + kW + kX + kWs + (i + wave) * 256);
    } else {
      // scale rows of any length: byte by byte, zero past the row's end
      for (int i = tid; i < (BM + BN) * 8; i += NW * kWave) {
        const bool isw = i < BM * 8;
        const int row = (isw ? i : i - BM * 8) >> 3, b = i & 7;
        uint8_t v = 0;
        if (kt * 8 + b < kb && row < (isw ? nr : nt))
          v = (isw ? ws : xs)[(int64_t)row * kb + kt * 8 + b];
        lds[buf][kW + kX + i] = v;
      }
    }
  };

  f32x4 acc[FR][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int wm = (wave / WT) * FR * kMfma, wn = (wave % WT) * FT * kMfma;
  const int l = lane & 15, q = lane >> 4;
  const int64_t all = (kb + 7) / 8, first = all * part / a.split;
  const int64_t steps = all * (part + 1) / a.split;
  load(0, first);
  for (int64_t kt = first; kt < steps; ++kt) {
    const int buf = (int)((kt - first) & 1);
    stage_ready();
    if (kt + 1 < steps) load(buf ^ 1, kt + 1);
    const uint8_t* base = lds[buf];
    uint32_t sw[FR], sx[FT];
#pragma unroll
    for (int i = 0; i < FR; ++i)
      sw[i] = *reinterpret_cast<const uint16_t*>(base + kW + kX + (wm + i * kMfma + l) * 8 + 2 * q);
#pragma unroll
    for (int j = 0; j < FT; ++j)
      sx[j] = *reinterpret_cast<const uint16_t*>(base + kW + kX + kWs + (wn + j * kMfma + l) * 8 +
                                                 2 * q);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 wf[FR], xf[FT];
      const int p = ((2 * q + h) ^ (l & 7)) * 16;
#pragma unroll
      for (int i = 0; i < FR; ++i)
        wf[i] = *reinterpret_cast<const u32x4*>(base + (wm + i * kMfma + l) * 128 + p);
#pragma unroll
      for (int j = 0; j < FT; ++j)
        xf[j] = *reinterpret_cast<const u32x4*>(base + kW + (wn + j * kMfma + l) * 128 + p);
#pragma unroll
      for (int i = 0; i < FR; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j)
          acc[i][j] = h == 0 ? mfma_fp4<0>(wf[i], xf[j], acc[i][j], sw[i], sx[j])
                             : mfma_fp4<1>(wf[i], xf[j], acc[i][j], sw[i], sx[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t t = t0 + wn + j * kMfma + l;
    if (t >= t1) continue;
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      const int64_t r = r0 + wm + i * kMfma + 4 * q;
      if (r < a.R) store_part(a, part, t, r, acc[i][j]);
    }
  }
}

template <int WR, int WT, int FR, int FT>
hipError_t tile_mxfp4(MatmulArgs a, hipStream_t stream) {
  constexpr int BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  a.row_blocks = (a.R + BM - 1) / BM;
  const int64_t grid = a.row_blocks * token_tiles(a, BN) * a.split;
  const bool whole = a.Cp % 256 == 0 && (uintptr_t)a.scales % 4 == 0 && (uintptr_t)a.x_scales % 4 == 0;
  if (whole)
    hipLaunchKernelGGL((tile_mxfp4_kernel<WR, WT, FR, FT, true>), dim3((unsigned)grid),
                       dim3(WR * WT * kWave), 0, stream, a);
  else
    hipLaunchKernelGGL((tile_mxfp4_kernel<WR, WT, FR, FT, false>), dim3((unsigned)grid),
                       dim3(WR * WT * kWave), 0, stream, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------
// bf16 x times decoded weights. A step takes 64 columns (128 bytes of bf16 a row). Two threads share
// a weight row of the tile: each reads a run of 32 columns (16 bytes of codes) straight into
// registers, decodes it and writes it to LDS as bf16, one step ahead of its use, so a weight is
// decoded once per tile. Rows of x go to LDS unchanged. Both lie permuted as above. Instruction
// h of a step takes pieces 4 h + q (columns 32 h + 8 q ..) of a row.
// ------------------------------------------------------------------------------------------------
template <class D, int WR, int WT, int FR, int FT>
__global__ __launch_bounds__(WR * WT * kWave, 1) void tile_bf16_kernel(MatmulArgs a) {
  constexpr int NW = WR * WT, BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  static_assert(NW * kWave == 2 * BM, "two threads a weight row");
  static_assert(BN % (8 * NW) == 0, "whole loads of x a wave");
  constexpr int kW = BM * 128, kX = BN * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][kW + kX];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  const int64_t id = by_die(blockIdx.x, gridDim.x), tiles = gridDim.x / a.split;
  const int part = (int)(id / tiles);
  const int64_t tile = id % tiles / a.row_blocks, rb = id % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, BN, tile, e, t0, t1)) return;
  const int64_t r0 = rb * BM;
  const int64_t x_bytes = a.ldx * 2;
  const int64_t nt = t1 - t0 < BN ? t1 - t0 : BN;
  const u32x4 xr = rows_buffer(static_cast<const uint8_t*>(a.x) + t0 * x_bytes,
                               (nt - 1) * x_bytes + a.C * 2);
  const uint32_t lds0 = lds_address(&lds[0][0]);
  const int piece = (lane & 7) ^ (lane >> 3);
  auto load_x = [&](int buf, int64_t kt) {
    const uint32_t dst = lds0 + buf * (kW + kX) + kW;
    const uint32_t off0 =
        (uint32_t)(lane >> 3) * (uint32_t)x_bytes + (uint32_t)(kt * 128) + piece * 16;
    const bool in = kt * 64 + piece * 8 < a.C;
#pragma unroll
    for (int i = 0; i < BN / 8 / NW; ++i) {
      const int row = (wave * (BN / 8 / NW) + i) * 8;
      load_lds16(xr, in ? off0 + row * (uint32_t)x_bytes : kOutside, dst + row * 128);
    }
  };
  D dec;
  dec.init(a, e);
  const int wrow = tid >> 1, half = tid & 1;
  const typename D::Row wp = dec.row(a, e, r0 + wrow < a.R ? r0 + wrow : a.R - 1);
  auto load_w = [&](int64_t kt) {
    const int64_t k = kt * 64 + half * 32;
    return dec.load_run(a, wp, k < a.Cp ? k : 0);
  };
  auto put_w = [&](int buf, int64_t kt, const typename D::Run& u) {
    u32x4 v[4];
    dec.decode_run(u, v);
    const bool in = kt * 64 + half * 32 < a.Cp;  // columns past the row's end: zero times zero
    uint8_t* p = lds[buf] + wrow * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<u32x4*>(p + (((4 * half + j) ^ (wrow & 7)) * 16)) =
          in ? v[j] : u32x4{0u, 0u, 0u, 0u};
  };

  f32x4 acc[FR][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int wm = (wave / WT) * FR * kMfma, wn = (wave % WT) * FT * kMfma;
  const int l = lane & 15, q = lane >> 4;
  const int64_t all = (a.Cp + 63) / 64, first = all * part / a.split;
  const int64_t steps = all * (part + 1) / a.split;
  auto multiply = [&](int buf) {
    const uint8_t* base = lds[buf];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 wf[FR], xf[FT];
      const int p = ((4 * h + q) ^ (l & 7)) * 16;
#pragma unroll
      for (int i = 0; i < FR; ++i)
        wf[i] = *reinterpret_cast<const u32x4*>(base + (wm + i * kMfma + l) * 128 + p);
#pragma unroll
      for (int j = 0; j < FT; ++j)
        xf[j] = *reinterpret_cast<const u32x4*>(base + kW + (wn + j * kMfma + l) * 128 + p);
#pragma unroll
      for (int i = 0; i < FR; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = mfma_bf16(wf[i], xf[j], acc[i][j]);
    }
  };

  typename D::Run now = load_w(first);
  load_x(0, first);
  put_w(0, first, now);
  if (first + 1 < steps) now = load_w(first + 1);
  for (int64_t kt = first; kt < steps; ++kt) {
    const int buf = (int)((kt - first) & 1);
    stage_ready();
    const bool more = kt + 1 < steps;
    typename D::Run next = now;
    if (more) load_x(buf ^ 1, kt + 1);
    if (kt + 2 < steps) next = load_w(kt + 2);
    multiply(buf);
    if (more) put_w(buf ^ 1, kt + 1, now);
    now = next;
  }
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t t = t0 + wn + j * kMfma + l;
    if (t >= t1) continue;
#pragma unroll
    for (int i = 0; i < FR; ++i) {
      const int64_t r = r0 + wm + i * kMfma + 4 * q;
      if (r < a.R) store_part(a, part, t, r, acc[i][j]);
    }
  }
}

template <class D, int WR, int WT, int FR, int FT>
hipError_t tile_bf16(MatmulArgs a, hipStream_t stream) {
  constexpr int BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  a.row_blocks = (a.R + BM - 1) / BM;
  const int64_t grid = a.row_blocks * token_tiles(a, BN) * a.split;
  hipLaunchKernelGGL((tile_bf16_kernel<D, WR, WT, FR, FT>), dim3((unsigned)grid),
                     dim3(WR * WT * kWave), 0, stream, a);
  return hipGetLastError();
}

template <class D>
hipError_t tile_bf16_any(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  switch (p.bn) {
    case 32: return tile_bf16<D, 4, 1, 2, 2>(a, stream);
    case 64: return tile_bf16<D, 2, 2, 4, 2>(a, stream);
    case 128: return tile_bf16<D, 2, 2, 4, 4>(a, stream);
    default: return tile_bf16<D, 2, 4, 8, 4>(a, stream);
  }
}

}  // namespace

hipError_t launch_tile_mx_bf16(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return tile_bf16_any<MxDecoder>(a, p, stream);
}

hipError_t launch_tile_packed(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return with_packed_decoder(a, [&](auto d) { return tile_bf16_any<decltype(d)>(a, p, stream); });
}

hipError_t launch_tile_mxfp4(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  switch (p.bn) {
    case 64: return tile_mxfp4<2, 2, 4, 2>(a, stream);
    case 128: return tile_mxfp4<2, 2, 4, 4>(a, stream);
    default: return tile_mxfp4<2, 4, 8, 4>(a, stream);
  }
}

}  // namespace aaac
