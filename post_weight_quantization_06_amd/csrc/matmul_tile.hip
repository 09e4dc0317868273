// Products with many rows of x per matrix: tiles of weight rows by rows of x, both staged through
// LDS, bound by the matrix units.
#include "matmul.h"

namespace aaac {

namespace {

// ------------------------------------------------------------------------------------------------
// MXFP4 x times MXFP4 weights. A tile is BM weight rows by BN rows of x; a step takes 256 columns
// (128 bytes of codes and 8 scale bytes a row). Lane l of a matrix instruction holds blocks 2 q and
// 2 q + 1 (q = l >> 4) of its row for the step's two halves, so its two scale bytes are neighbours.
// In LDS the eight 16-byte pieces of a row lie permuted by row bits 1 to 3 (piece_turn). Permuted by
// bits 0 to 2, half of the LDS's cycles were bank conflicts (15.1 M of 30.3 M, now 4.1 M of 19.3 M; the
// case below took 149 us instead of 144).
// Fragments are half a step ahead of the matrix instructions: a barrier falls between the two halves
// of a step's instructions, and each register is read again as soon as it has been used.
//
// 4096 x 14336 x 4096: 144 us, 3.3 PFLOP/s, of the 8.8 that the instruction alone reaches here. What
// bounds it is the supply of the stages: without its matrix instructions it takes 87 % of the time,
// without its loads 79 %. Eight waves of 128 x 64 rather than four of 128 x 128: four need 512
// registers each and spill. Rows of x tiles advancing together (1 to 16 of them) and touching lines
// two to four steps ahead measured equal or slower.
//
// WHOLE: rows of whole steps whose scale bytes lie on words. Otherwise the scale bytes are loaded one by
// one through registers, and each waits for memory, the next stage's loads among it, in every step: half
// the rate (2048 x 2880 with 2816 columns 23 us, with 2880 or 2944 46 us; 32 experts, 4096 rows, 60 and 119).
// ------------------------------------------------------------------------------------------------
template <int WR, int WT, int FR, int FT, bool WHOLE>
__global__ __launch_bounds__(WR * WT * kWave, 2) void tile_mxfp4_kernel(MatmulArgs a) {
  constexpr int NW = WR * WT, BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  // LDS: two stages of codes, then the scale bytes of two times four steps, 32 a row; the halves of
  // these 32 are swapped in rows with bit 3 set, so that 16 rows' bytes of a step lie in 16 banks
  constexpr int kW = BM * 128, kX = BN * 128, kStage = kW + kX, kWs = BM * 32, kScales = kWs + BN * 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * (kStage + kScales)];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  if (block_id() >= a.blocks) return;
  const int64_t id = by_die(block_id(), a.blocks), tiles = a.blocks / a.split;
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

  const int64_t all = (kb + 7) / 8, first = all * part / a.split;
  const int64_t steps = all * (part + 1) / a.split;
  // the 16-byte piece of the row that a lane loads, in the even and the odd loads of eight rows
  const int piece[2] = {(lane & 7) ^ piece_turn(lane >> 3), (lane & 7) ^ piece_turn((lane >> 3) + 8)};
  static_assert(BM / 8 / NW % 2 == 0 && BN / 8 / NW % 2 == 0, "row bit 3 is the load's parity");
  const uint32_t lds0 = lds_address(&lds[0]);
  auto load = [&](int buf, int64_t kt) {
    const uint32_t dst = lds0 + buf * kStage;
    const int at4 = 2 * kStage + (int)(kt >> 2 & 1) * kScales;
    const uint32_t row0 = (uint32_t)(lane >> 3) * (uint32_t)row_bytes + (uint32_t)(kt * 128);
    const uint32_t off[2] = {
        WHOLE || kt * 8 + piece[0] < kb ? row0 + piece[0] * 16 : kOutside,
        WHOLE || kt * 8 + piece[1] < kb ? row0 + piece[1] * 16 : kOutside};
#pragma unroll
    for (int i = 0; i < BM / 8 / NW; ++i) {
      const int row = (wave * (BM / 8 / NW) + i) * 8;
      load_lds16(wr, off[i & 1] + row * (uint32_t)row_bytes, 0, dst + row * 128);
    }
#pragma unroll
    for (int i = 0; i < BN / 8 / NW; ++i) {
      const int row = (wave * (BN / 8 / NW) + i) * 8;
      load_lds16(xr, off[i & 1] + row * (uint32_t)row_bytes, 0, dst + kW + row * 128);
    }
    if (WHOLE) {
      // scale rows are read for four steps at a time: a load costs by its rows, not their bytes
      if (kt != first && (kt & 3) != 0) return;
      const uint32_t sdst = lds0 + at4;
      const uint32_t soff = (uint32_t)(lane >> 1) * (uint32_t)kb + (uint32_t)(kt >> 2) * 32 +
                            16 * ((lane ^ (lane >> 4)) & 1);
#pragma unroll
      for (int i = 0; i < BM / 32; i += NW)
        if (BM / 32 % NW == 0 || i + wave < BM / 32)
          load_lds16(wsr, soff + (i + wave) * 32 * (uint32_t)kb, 0, sdst + (i + wave) * 1024);
#pragma unroll
      for (int i = 0; i < BN / 32; i += NW)
        if (BN / 32 % NW == 0 || i + wave < BN / 32)
          load_lds16(xsr, soff + (i + wave) * 32 * (uint32_t)kb, 0, sdst + kWs + (i + wave) * 1024);
    } else {
      // scale rows of any length: byte by byte, zero past the row's end
      for (int i = tid; i < (BM + BN) * 8; i += NW * kWave) {
        const bool isw = i < BM * 8;
        const int row = (isw ? i : i - BM * 8) >> 3, b = i & 7;
        uint8_t v = 0;
        if (kt * 8 + b < kb && row < (isw ? nr : nt))
          v = (isw ? ws : xs)[(int64_t)row * kb + kt * 8 + b];
        lds[at4 + (isw ? 0 : kWs) + row * 32 + (((int)(kt & 3) * 8) ^ (row & 8) * 2) + b] = v;
      }
    }
  };

  f32x4 acc[FR][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // neighbouring waves, on different SIMDs, share their rows of x; those past a partial tile's last
  // row only help to load (and decode)
  const int wm = (wave % WR) * FR * kMfma, wn = (wave / WR) * FT * kMfma;
  const bool busy = wn < nt;
  const int l = lane & 15, q = lane >> 4;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  u32x4 wf[FR], xf[2][FT];
  uint32_t sw[FR], sx[2][FT];                    // scale words
#pragma unroll
  for (int i = 0; i < FR; ++i) {
    wf[i] = zero;
    sw[i] = 0;
  }
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    xf[1][j] = zero;
    sx[1][j] = 0;
  }
  load(0, first);
  auto walk = [&](auto with_products) __attribute__((always_inline)) {
    for (int64_t kt = first; kt < steps; ++kt) {
      const int buf = (int)((kt - first) & 1);
      wait_loads<0>();
      step_barrier();
      if (kt + 1 < steps) load(buf ^ 1, kt + 1);
      if (decltype(with_products)::value == 0) continue;
      const uint8_t* base = lds + buf * kStage;
      const uint8_t* wb = base + (wm + l) * 128;
      const uint8_t* sb = lds + 2 * kStage + (int)(kt >> 2 & 1) * kScales +
                          (((int)(kt & 3) * 8) ^ (l & 8) * 2) + 2 * q;
      const uint8_t *wsb = sb + (wm + l) * 32, *xsb = sb + kWs + (wn + l) * 32;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        sx[0][j] = sx[1][j];
        sx[1][j] = *reinterpret_cast<const uint16_t*>(xsb + j * kMfma * 32);
      }
      // half 0 of the pass: instructions of the step before, on its second half's fragments, while
      // this step's first half is read; half 1: this step's first half, while its second is read
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = ((2 * q + h) ^ piece_turn(l)) * 16;
#pragma unroll
        for (int j = 0; j < FT; ++j)
          xf[h][j] = *reinterpret_cast<const u32x4*>(base + kW + (wn + j * kMfma + l) * 128 + p);
#pragma unroll
        for (int i = 0; i < FR; ++i) {
          // the registers of the group before
          if (i > 0) {
            wf[i - 1] = *reinterpret_cast<const u32x4*>(wb + (i - 1) * kMfma * 128 + p);
            if (h == 0) sw[i - 1] = *reinterpret_cast<const uint16_t*>(wsb + (i - 1) * kMfma * 32);
          } else if (h == 1) {
            wf[FR - 1] = *reinterpret_cast<const u32x4*>(wb + (FR - 1) * kMfma * 128 + (p ^ 16));
            sw[FR - 1] = *reinterpret_cast<const uint16_t*>(wsb + (FR - 1) * kMfma * 32);
          }
#pragma unroll
          for (int j = 0; j < FT; ++j)
            acc[i][j] = h == 0 ? mfma_fp4<1>(wf[i], xf[1][j], acc[i][j], sw[i], sx[0][j])
                               : mfma_fp4<0>(wf[i], xf[0][j], acc[i][j], sw[i], sx[1][j]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      wf[FR - 1] = *reinterpret_cast<const u32x4*>(wb + (FR - 1) * kMfma * 128 +
                                                   ((2 * q + 1) ^ piece_turn(l)) * 16);
    }
  };
  if (busy) walk(Int<1>());
  else walk(Int<0>());
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j)
      acc[i][j] = mfma_fp4<1>(wf[i], xf[1][j], acc[i][j], sw[i], sx[1][j]);
  static_assert(sizeof(lds) >= NW * tile_bytes<FR, FT>(), "the waves' results fit");
  wait_loads<0>();
  step_barrier();                                // the stages give way to the results
  store_tile<FR, FT>(a, part, acc, &lds[0] + wave * tile_bytes<FR, FT>(), t0 + wn, t1, r0 + wm);
}

template <int WR, int WT, int FR, int FT>
hipError_t tile_mxfp4(MatmulArgs a, hipStream_t stream) {
  constexpr int BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  a.row_blocks = (a.R + BM - 1) / BM;
  a.blocks = a.row_blocks * token_tiles(a, BN) * a.split;
  const bool whole = a.Cp % 256 == 0 && (uintptr_t)a.scales % 4 == 0 && (uintptr_t)a.x_scales % 4 == 0;
  if (whole)
    hipLaunchKernelGGL((tile_mxfp4_kernel<WR, WT, FR, FT, true>), grid_of(a.blocks),
                       dim3(WR * WT * kWave), 0, stream, a);
  else
    hipLaunchKernelGGL((tile_mxfp4_kernel<WR, WT, FR, FT, false>), grid_of(a.blocks),
                       dim3(WR * WT * kWave), 0, stream, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------
// bf16 x times decoded weights. A step takes 64 columns (128 bytes of bf16 a row). Two threads share
// a weight row of the tile, a run of 32 columns each: a thread decodes its run and writes it to LDS
// as bf16 one step ahead of its use, so a weight is decoded once per tile. Rows of x go to LDS
// unchanged. The 16-byte pieces of both lie permuted by row bits 0 to 2. Instruction h of a step takes
// pieces 4 h + q (columns 32 h + 8 q ..) of a row.
// Memory is NS - 1 steps ahead: group j of asynchronous loads holds x of step j and the codes and
// scales of step j + 1, and at most NS - 2 younger groups are in flight when a step begins. Loads
// past the last step lie outside their buffers, so every group has the same count.
// Fragments are one half step ahead of the matrix instructions: a barrier falls between the two
// halves of a step's instructions, and each register is read again as soon as it has been used.
//
// 2048 x 14336 x 4096 packed: 245 us, 980 TFLOP/s; 448 tiles make 1.75 rounds of the 256 CUs, so a full
// round runs at 1.1 PFLOP/s, where a library bf16 product of 8192 x 8192 x 8192 reaches 1.18. Without
// decoding it takes 80 % of the time, without matrix instructions 70 %: the two share the issue slots
// of a SIMD (three byte permutes to one matrix instruction cost 30 % over the instructions alone).
// ------------------------------------------------------------------------------------------------
template <class D, int WR, int WT, int FR, int FT, int NS>
__global__ __launch_bounds__(WR * WT * kWave, 2) void tile_bf16_kernel(MatmulArgs a) {
  constexpr int NW = WR * WT, BM = WR * FR * kMfma, BN = WT * FT * kMfma, kThreads = NW * kWave;
  static_assert(kThreads == 2 * BM, "two threads a weight row");
  static_assert(BN % (8 * NW) == 0, "whole loads of x a wave");
  constexpr int kW = BM * 128, kX = BN * 128, kC = kThreads * 16, kS = D::kWords * kThreads * 4;
  constexpr int kSlot = kX + kC + kS;
  constexpr int kLoads = BN / 8 / NW + 1 + D::kWords;        // a wave's loads in a group
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kW + NS * kSlot];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  if (block_id() >= a.blocks) return;
  const int64_t id = by_die(block_id(), a.blocks), tiles = a.blocks / a.split;
  const int part = (int)(id / tiles);
  const int64_t tile = id % tiles / a.row_blocks, rb = id % a.row_blocks;
  int e;
  int64_t t0, t1;
  if (!find_tile(a.offsets, a.E, a.T, BN, tile, e, t0, t1)) return;
  const int64_t r0 = rb * BM;
  const int64_t x_bytes = a.ldx * 2;
  const int64_t nt = t1 - t0 < BN ? t1 - t0 : BN, nr = a.R - r0 < BM ? a.R - r0 : BM;
  const u32x4 xr = rows_buffer(static_cast<const uint8_t*>(a.x) + t0 * x_bytes,
                               (nt - 1) * x_bytes + a.C * 2);
  D dec;
  dec.init(a, e);
  dec.init_tile(a, e, r0, nr);
  const uint32_t slots = lds_address(&lds[2 * kW]);
  const int piece = (lane & 7) ^ (lane >> 3);
  // the weight row that this thread decodes; rows past the matrix repeat its last one
  const int wrow = tid >> 1, half = 32 * (tid & 1);
  const int mrow = wrow < nr ? wrow : (int)nr - 1;
  const int all = (int)((a.Cp + 63) / 64);
  const int first = (int)((int64_t)all * part / a.split);
  const int steps = (int)((int64_t)all * (part + 1) / a.split);
  const int cols = (int)a.C, wcols = (int)a.Cp;
  constexpr int kXl = BN / 8 / NW;
  uint32_t xoff[kXl];
#pragma unroll
  for (int i = 0; i < kXl; ++i) {
    const int row = (wave * kXl + i) * 8 + (lane >> 3);
    xoff[i] = (uint32_t)(row < nt ? row : (int)nt - 1) * (uint32_t)x_bytes + piece * 16;
  }
  auto load_w = [&](int slot, int kt) {
    const uint32_t dst = slots + slot * kSlot + kX;
    dec.issue(a, mrow, kt, half, kt < steps && kt * 64 + half < wcols, dst + wave * (kWave * 16),
              dst + kC + wave * (kWave * 4), kThreads);
  };
  auto load_group = [&](int slot, int kt) {
    const uint32_t dst = slots + slot * kSlot + wave * kXl * 1024;
    if (kt < steps && kt * 64 + 64 <= cols) {
#pragma unroll
      for (int i = 0; i < kXl; ++i) load_lds16(xr, xoff[i], kt * 128, dst + i * 1024);
    } else {
      const bool in = kt < steps && kt * 64 + piece * 8 < cols;
#pragma unroll
      for (int i = 0; i < kXl; ++i)
        load_lds16(xr, in ? xoff[i] : kOutside, kt * 64 < cols ? kt * 128 : 0, dst + i * 1024);
    }
    load_w(slot, kt + 1);
  };
  auto fetch = [&](int slot, int kt) {
    const uint8_t* p = lds + 2 * kW + slot * kSlot + kX;
    return dec.fetch(a, mrow, kt, half, kt < steps && kt * 64 + half < wcols, p + tid * 16,
                     reinterpret_cast<const uint32_t*>(p + kC) + tid, kThreads);
  };
  auto put = [&](int buf, int j, u32x4 v) {
    uint8_t* p = lds + buf * kW + wrow * 128;
    *reinterpret_cast<u32x4*>(p + (((half / 8 + j) ^ (wrow & 7)) * 16)) = v;
  };

  f32x4 acc[FR][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // neighbouring waves, on different SIMDs, share their rows of x; those past a partial tile's last
  // row only help to load (and decode)
  const int wm = (wave % WR) * FR * kMfma, wn = (wave / WR) * FT * kMfma;
  const bool busy = wn < nt;
  const int l = lane & 15, q = lane >> 4;

  load_w(NS - 1, first);
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) load_group(s, first + s);
  wait_loads<(NS - 1) * kLoads>();
  {
    typename D::Planes t;
    const typename D::Run u = fetch(NS - 1, first);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      typename D::Eight v;
#pragma unroll
      for (int n = 0; n < 4; ++n) dec.piece(u, j, n, t, v);
      put(0, j, v.out);
    }
  }
  const u32x4 zero = {0u, 0u, 0u, 0u};
  u32x4 wf[FR], xf[2][FT];
#pragma unroll
  for (int i = 0; i < FR; ++i) wf[i] = zero;
#pragma unroll
  for (int j = 0; j < FT; ++j) xf[1][j] = zero;
  auto walk = [&](auto with_products) __attribute__((always_inline)) {
    constexpr bool kMul = decltype(with_products)::value != 0;
    int slot = 0;
    for (int kt = first; kt < steps; ++kt) {
      const int buf = (kt - first) & 1;
      wait_loads<(NS - 2) * kLoads>();
      step_barrier();
      load_group(slot == 0 ? NS - 1 : slot - 1, kt + NS - 1);
      typename D::Planes t;
      typename D::Eight v;
      const typename D::Run u = fetch(slot, kt + 1);
      const uint8_t* wb = lds + buf * kW + (wm + l) * 128;
      const uint8_t* xb = lds + 2 * kW + slot * kSlot + (wn + l) * 128;
      __builtin_amdgcn_sched_barrier(0);
      // half 0 of the pass: instructions of the step before, on its second half's fragments, while
      // this step's first half is read; half 1: this step's first half, while its second is read
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = ((4 * h + q) ^ (l & 7)) * 16;
#pragma unroll
        for (int j = 0; j < FT; ++j)
          if (kMul) xf[h][j] = *reinterpret_cast<const u32x4*>(xb + j * kMfma * 128 + p);
#pragma unroll
        for (int i = 0; i < FR; ++i) {
          // the registers of the group before
          if (!kMul) {
          } else if (i > 0) {
            wf[i - 1] = *reinterpret_cast<const u32x4*>(wb + (i - 1) * kMfma * 128 + p);
          } else if (h == 1) {
            wf[FR - 1] = *reinterpret_cast<const u32x4*>(wb + (FR - 1) * kMfma * 128 + (p ^ 64));
          }
#pragma unroll
          for (int j = 0; j < FT; ++j)
            if (kMul) acc[i][j] = mfma_bf16(wf[i], xf[h ^ 1][j], acc[i][j]);
          // the decoding in sixteen parts beside the instructions; the barriers keep the compiler
          // from gathering the reads, or the vector work, of several parts
          constexpr int kParts = 8 / FR;
#pragma unroll
          for (int n = 0; n < kParts; ++n) {
            const int w = (h * FR + i) * kParts + n;
            dec.piece(u, w / 4, w % 4, t, v);
            if (w % 4 == 3) put(buf ^ 1, w / 4, v.out);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (kMul)
        wf[FR - 1] =
            *reinterpret_cast<const u32x4*>(wb + (FR - 1) * kMfma * 128 + (((4 + q) ^ (l & 7)) * 16));
      slot = slot + 1 == NS ? 0 : slot + 1;
    }
  };
  if (busy) walk(Int<1>());
  else walk(Int<0>());
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = mfma_bf16(wf[i], xf[1][j], acc[i][j]);
  static_assert(sizeof(lds) >= NW * tile_bytes<FR, FT>(), "the waves' results fit");
  wait_loads<0>();
  step_barrier();                                // the stages give way to the results
  store_tile<FR, FT>(a, part, acc, &lds[0] + wave * tile_bytes<FR, FT>(), t0 + wn, t1, r0 + wm);
}

template <class D, int WR, int WT, int FR, int FT, int NS>
hipError_t tile_bf16(MatmulArgs a, hipStream_t stream) {
  constexpr int BM = WR * FR * kMfma, BN = WT * FT * kMfma;
  a.row_blocks = (a.R + BM - 1) / BM;
  a.blocks = a.row_blocks * token_tiles(a, BN) * a.split;
  hipLaunchKernelGGL((tile_bf16_kernel<D, WR, WT, FR, FT, NS>), grid_of(a.blocks),
                     dim3(WR * WT * kWave), 0, stream, a);
  return hipGetLastError();
}

template <class D>
hipError_t tile_bf16_any(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  switch (p.bn) {
    case 32: return tile_bf16<D, 4, 1, 2, 2, 4>(a, stream);
    case 64: return tile_bf16<D, 2, 2, 4, 2, 3>(a, stream);
    case 128: return tile_bf16<D, 2, 2, 4, 4, 2>(a, stream);
    default: return tile_bf16<D, 2, 4, 8, 4, 2>(a, stream);
  }
}

}  // namespace

hipError_t launch_tile_mx_bf16(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return tile_bf16_any<MxDecoder>(a, p, stream);
}

hipError_t launch_tile_packed(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  return with_packed_decoder<true>(
      a, [&](auto d) { return tile_bf16_any<decltype(d)>(a, p, stream); });
}

hipError_t launch_tile_mxfp4(const MatmulArgs& a, const MatmulPlan& p, hipStream_t stream) {
  switch (p.bn) {
    case 64: return p.bm == 64 ? tile_mxfp4<1, 4, 4, 1>(a, stream) : tile_mxfp4<2, 2, 4, 2>(a, stream);
    case 128: return tile_mxfp4<2, 2, 4, 4>(a, stream);
    default: return tile_mxfp4<2, 4, 8, 4>(a, stream);
  }
}

}  // namespace aaac
