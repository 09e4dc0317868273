// How a product call is run: the choice of kernel and tile, and the kernel that adds the parts of a
// sum that was split over workgroups.
#include "fp8.h"
#include "matmul.h"

namespace aaac {

namespace {

constexpr int64_t kL2Bytes = (int64_t)32 << 20;   // the L2s of the eight dies together

// y = the sum of the parts in order, four columns a thread. Rows that no expert has were not written
// by the tiles and are left alone here.
__global__ __launch_bounds__(kBlock) void add_parts_kernel(MatmulArgs a) {
  const int64_t per = part_row(a.R) / 4;
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  const int64_t t = i / per, r = (i - t * per) * 4;
  if (t >= a.T) return;
  if (a.offsets && (t < a.offsets[0] || t >= a.offsets[a.E])) return;
  const f32x4* p = reinterpret_cast<const f32x4*>(a.parts) + i;
  const int64_t stride = a.T * per;
  f32x4 v = p[0];
  for (int s = 1; s < a.split; ++s) v += p[s * stride];
  store4(a, t, r, v);
}

// The choice. Up to 16 rows of x a matrix (32 for one matrix in MXFP4) go to the few-row kernels,
// which read each weight once for every 16 (32) rows: one row against 14336 x 4096 packed weights takes
// 18 us there and 26 in the best tiles, 16 rows 19 us there, 17 rows 26 us in tiles. The offsets lie on
// the device, so an average decides: 64 experts of 2048 x 2048 in MXFP4 with 1000 rows take 85 us spread
// unevenly, 109 with 938 of them at one expert (28 for 1000 rows at that one alone, in tiles). Two blocks
// of 16 weight rows a workgroup halve the reads of x, one block makes more workgroups: 32 experts of
// 2048 x 4096 (some 3500 blocks) take 33 us with two and 41 with one, 4096 x 14336 (256 blocks) 19
// and 12. Four chunks at a time pay on long rows: 12.6 us down to 11.9 at 14336 columns, 7.3 up to 7.8
// at 4096.
//
// FP8, whose tiles stream weights as fast: the few-row kernels where they save more than a second pass over an
// expert's weights costs. Those of an expert with more than 16 rows are read again, and the tile kernels read
// x from LDS, so up to kFewOne rows for one matrix and kFewMean rows an expert on average, and twice as many
// for fp32 and fp16 results, whose tiles are slower. 64 experts of 2048 x 2048, bf16 x: 33 us with 100 rows (tiles 36),
// 41 with 200 (43), 53 with 400 (46). One matrix, calls with FP8 and with bf16 x, three matrices in turn: 4096 x
// 14336 with 1 row 14.9 and 12.9 us (tiles 17.2 and 20.7), with 8 16.8 and 19.6 (17.4 and 21.0), with 16 20.8 and
// 21.6 (17.4 and 21.0); 14336 x 4096 with 8 12.9 and 16.6 (13.4 and 17.3); 28672 x 8192 with 8 48 and 52 (55 and
// 60); 8192 x 28672 with 8 52 and 55 (51 and 54). 8192 x 8192 would be faster in tiles with 2 rows already: 20.3 and
// 22.2 (17.6 and 21.1). fp32 results with 16 rows: 14336 x 4096 14.4 and 17.9 (20.6 and 24.3), 4096 x 14336 21.2
// and 22.5 (19.6 and 23.4). Up to kFewWeights codes a call is all latency, and no launch for the quantised x or
// the parts counts more: 4096 x 4096 with 16 rows 15.5 us (17).
// 16 weight rows a workgroup of 16 waves where that makes no more workgroups than the CUs, 32 up to twice as
// many, else 64, the longest run of loads for the time it takes to start and end, in calls of one matrix again and
// again (some of it stays in the last cache) with one row of bf16: 4096 x 14336 13.4 us (32: 18, 64: 30), 8000 x
// 8000 14.7 (16: 15.4, 64: 17.6), 14336 x 4096 13.1 (15.7, 14.1), 28672 x 8192 40 (63, 56).
//
// FP8 rows of x given in another type: a workgroup of the few-row kernels quantises its own where they have
// up to kFewQuantize elements, which saves a launch; more take longer than the launch does. An expert may have
// four times the average, and LDS holds 16 of its rows.
constexpr int64_t kFewOne = 8, kFewMean = 4, kFewWeights = (int64_t)1 << 25;
constexpr int64_t kFewQuantize = 32768, kFewLds = 65536;

// With small weights (kFewAgain; kFewWeights up to 16 rows an expert on average: 16 of 1000 x 1000 with 200
// rows 12.5 us, 16 in tiles) they also take more rows, 16 a workgroup, where that takes
// less than a launch (kQuantise, for rows of x in another type) more than the tiles do: 1000 x 1000 with 64 rows
// of bf16 10.8 us (tiles 15.4), with 250 10.7 (15.4), 2000 x 2000 with 128 rows 13.1 (15.4), with 250 17.1
// (15.2), 16 experts of 500 x 500 with 600 rows 10.9 (15.9); larger weights cost more to read again: 12866 x
// 2022 with 27 rows 22 (16). The times of a workgroup are measured ones, `two` those of more than one a CU. The
// choice does not look at the type of x, so that quantising inside the call and before it give the same bits.
constexpr int64_t kFewAgain = (int64_t)1 << 23;
struct FewCost { int rt; double start, block, two; };
constexpr FewCost kFewFp8[] = {{1, 2.2, 0.24, 1.00}, {2, 3.0, 0.27, 0.75}, {4, 3.0, 0.36, 0.72}};
constexpr double kQuantise = 5.0;

// Tiles: the least estimated time over tile widths and splits. A tile takes its steps times kStep
// (measured with every CU at work) and kTile to start and end; the busiest CU runs
// ceil(workgroups / CUs) of them, two at a time where LDS holds two, which takes kTwo of one after the
// other. A split adds a launch and the traffic of the parts. It picks, in microseconds and packed
// weights of 14336 x 4096: 64 rows: 64 wide, split 4 (32; unsplit 53); 512 rows: 256 wide, split 2
// (85; 128 wide unsplit 96); 2048 rows: 256 wide unsplit (250; 128 wide 334). Tiles of 64 weight rows
// double the workgroups of a short MXFP4 product: 48 rows against 14336 x 4096 in 16.2 us, 17.0 in 128.
// The MXFP4 step times are those of rows of whole steps; the other form's steps (tile_mxfp4_kernel) take
// about twice as long in every tile and have no table of their own.
//
// The FP8 tiles' times are their own, by results: bf16, or fp32 and fp16 (which take another instruction). They
// count that a chip at work in part runs faster (kIdle) and, on average over the experts, half a tile that is
// empty (kLastFp8). Measured: 14336 x 4096 with 300 rows 38 us in 128 wide tiles (128 by 64: 44, 256 wide: 52,
// split in two: 48), with 1024 rows 65 in 256 wide ones (128 wide: 79); 4096 x 14336 with 512 rows 50 in 128
// wide ones split in two (unsplit 71, 256 wide split 8: 54); 64 experts of 2048 x 2048 with 4000 rows 62 in 128
// wide ones (256 wide: 92), 32 of 4096 x 2048 with 16380 rows 192 in 256 wide ones (213).
struct TileCost { int bm, bn; double step, two, tile; };
constexpr double kOne = 0.0;                     // LDS holds one tile
constexpr double kTile = 2.3, kTwoBf16 = 0.80, kTwoMx = 0.95, kLaunch = 3.0;
constexpr TileCost kBf16Tiles[] = {{128, 32, 0.70, kTwoBf16, kTile}, {128, 64, 0.77, kTwoBf16, kTile},
                                   {128, 128, 0.96, kTwoBf16, kTile}, {256, 256, 1.85, kOne, kTile}};
constexpr TileCost kMxTiles[] = {{64, 64, 0.45, kTwoMx, kTile}, {128, 64, 0.60, kTwoMx, kTile},
                                 {128, 128, 0.75, kTwoMx, kTile}, {256, 256, 1.90, kOne, kTile}};
constexpr TileCost kFp8Tiles[] = {{64, 64, 0.30, 0.73, 3.5}, {128, 64, 0.46, 0.72, 4.5},
                                  {128, 128, 0.60, 0.79, 6.0}, {256, 256, 1.60, kOne, 12.0}};
constexpr TileCost kFp8WideTiles[] = {{64, 64, 0.49, 0.73, 3.5}, {128, 64, 0.66, 0.80, 6.0},
                                      {128, 128, 1.00, 0.88, 8.5}};
constexpr double kPartBytes = 6e6, kIdle = 0.4, kLast = 0.75, kLastFp8 = 0.5;

// The estimated time, and the plan.
template <int N>
double plan_tiles(const MatmulArgs& a, const TileCost (&tiles)[N], int cols, double idle, double last,
                bool can_split, MatmulPlan& p) {
  const int cus = device_cu_count();
  const int64_t steps = (a.Cp + cols - 1) / cols;
  // experts' last tiles: some are empty, and the split of the rows over the experts is not known here
  const double extra = a.E > 1 ? last * (double)(a.E < a.T ? a.E : a.T) : 0.0;
  double best = 1e30;
  for (const TileCost& t : tiles) {
    const double across = a.E > 1 ? (double)a.T / t.bn + extra : (double)((a.T + t.bn - 1) / t.bn);
    const double n = (double)((a.R + t.bm - 1) / t.bm) * across;
    for (int split = 1; split <= (can_split ? 16 : 1); ++split) {
      if (split > 1 && (steps < 4 * split || n * split > 4.0 * cus)) break;
      const double on_cu = n * split / cus;
      const double step = t.step * (on_cu < 1 ? 1.0 - idle * (1.0 - on_cu) : 1.0);
      const double each = (double)((steps + split - 1) / split) * step + t.tile;
      const double turns = on_cu <= 1 ? 1.0 : (double)(int64_t)(on_cu + 0.999);
      double time = turns * each * (on_cu > 1 && t.two > 0 ? t.two : 1.0);
      if (split > 1) time += kLaunch + 8.0 * split * (double)a.T * (double)a.R / kPartBytes;
      if (time < best) {
        best = time;
        p.bm = t.bm;
        p.bn = t.bn;
        p.split = split;
      }
    }
  }
  return best;
}

// The same of the few-row kernels for any number of rows.
double plan_few_fp8(const MatmulArgs& a, int& rt) {
  const int cus = device_cu_count();
  const double tiles = a.E > 1 ? (double)a.T / kMfma + kLastFp8 * (double)(a.E < a.T ? a.E : a.T)
                               : (double)((a.T + kMfma - 1) / kMfma);
  double best = 1e30;
  for (const FewCost& f : kFewFp8) {
    const double on_cu = (double)((a.R + f.rt * kMfma - 1) / (f.rt * kMfma)) * tiles / cus;
    const double each = f.start + f.block * (double)fp8_blocks(a.C);
    const double time = on_cu <= 1 ? each : each * f.two * (double)(int64_t)(on_cu + 0.999);
    if (time < best) {
      best = time;
      rt = f.rt;
    }
  }
  return best;
}

}  // namespace

MatmulPlan plan_matmul(const MatmulArgs& a, MatmulKind kind, bool can_split) {
  MatmulPlan p = {};
  p.split = 1;
  const int64_t rows = (a.T + a.E - 1) / a.E;    // rows of x an expert, on average
  if (kind == kFp8) {
    if (a.Tx == 0) {
      // no row of x: those that are picked are zeros. The few-row kernels read nothing of such an x; the
      // tiles' buffers of rows hold one row at least.
      p.rt = 4;
      p.nt = p.chunks = 1;
      return p;
    }
    const bool wide = a.y_type != AAAC_BF16;     // sums by the bf16 instruction
    const int64_t most = (a.E == 1 ? kFewOne : kFewMean) * (wide ? 2 : 1);
    const int64_t weights = a.E * a.R * a.C;
    if (rows <= (a.E == 1 && weights <= kFewWeights ? kMfma : most)) {
      const int64_t blocks = (a.R + kMfma - 1) / kMfma * (a.E < a.T ? a.E : a.T);
      const int cus = device_cu_count();
      const int64_t each = a.E == 1 ? rows : rows < kMfma / 4 ? 4 * rows : kMfma;
      p.nt = 1;
      p.rt = blocks <= cus ? 1 : blocks <= 2 * cus ? 2 : 4;
      p.chunks = 1;
      p.quantize = each * a.C <= kFewQuantize && (a.T < kMfma ? a.T : kMfma) * a.C <= kFewLds;
      return p;
    }
    const double time = wide ? plan_tiles(a, kFp8WideTiles, kFp8Block, kIdle, kLastFp8, can_split, p)
                             : plan_tiles(a, kFp8Tiles, kFp8Block, kIdle, kLastFp8, can_split, p);
    int rt;
    if (weights <= (rows <= kMfma ? kFewWeights : kFewAgain) && kMfma * a.C <= kFewQuantize &&
        plan_few_fp8(a, rt) < time + kQuantise) {
      p = {};
      p.split = 1;
      p.rt = rt;
      p.nt = p.chunks = 1;
      p.quantize = true;
    }
    return p;
  }
  if (rows <= kMfma || (kind == kMxMxfp4 && a.E == 1 && rows <= 2 * kMfma)) {
    const int64_t blocks = (a.R + kMfma - 1) / kMfma * (a.E < a.T ? a.E : a.T);
    p.nt = rows <= kMfma ? 1 : 2;
    p.rt = blocks > 2 * device_cu_count() ? 2 : 1;
    p.chunks = a.C >= 8192 ? 4 : 1;
    return p;
  }
  if (kind == kMxMxfp4) plan_tiles(a, kMxTiles, 256, 0.0, kLast, can_split, p);
  else plan_tiles(a, kBf16Tiles, 64, 0.0, kLast, can_split, p);
  return p;
}

size_t parts_bytes(const MatmulArgs& a, const MatmulPlan& p) {
  return p.split > 1 ? (size_t)p.split * a.T * part_row(a.R) * sizeof(float) : 0;
}

hipError_t launch_matmul(MatmulArgs a, MatmulKind kind, const MatmulPlan& p, hipStream_t stream) {
  a.y_vec = can_store4(a);
  a.y_row = a.y_type != AAAC_F32 && (uintptr_t)a.y % 16 == 0 && a.ldy % 8 == 0;
  if (a.y_row && a.T * a.R * 2 > kL2Bytes) a.y_row = 2;
  a.split = p.split;
  hipError_t e;
  if (p.bn == 0)
    e = kind == kPacked ? launch_few_packed(a, p, stream)
        : kind == kFp8 ? launch_few_fp8(a, p, stream)
        : kind == kMxMxfp4 ? launch_few_mxfp4(a, p, stream) : launch_few_mx_bf16(a, p, stream);
  else
    e = kind == kPacked ? launch_tile_packed(a, p, stream)
        : kind == kFp8 ? launch_tile_fp8(a, p, stream)
        : kind == kMxMxfp4 ? launch_tile_mxfp4(a, p, stream) : launch_tile_mx_bf16(a, p, stream);
  if (e != hipSuccess || p.split == 1) return e;
  const int64_t items = a.T * (part_row(a.R) / 4);
  hipLaunchKernelGGL(add_parts_kernel, dim3((unsigned)((items + kBlock - 1) / kBlock)), dim3(kBlock),
                     0, stream, a);
  return hipGetLastError();
}

}  // namespace aaac
