// How a product call is run: the choice of kernel and tile, and the kernel that adds the parts of a
// sum that was split over workgroups.
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
// Tiles: the least estimated time over tile widths and splits. A tile takes its steps times kStep
// (measured with every CU at work) and kTile to start and end; the busiest CU runs
// ceil(workgroups / CUs) of them, two at a time where LDS holds two, which takes kTwo of one after the
// other. A split adds a launch and the traffic of the parts. It picks, in microseconds and packed
// weights of 14336 x 4096: 64 rows: 64 wide, split 4 (32; unsplit 53); 512 rows: 256 wide, split 2
// (85; 128 wide unsplit 96); 2048 rows: 256 wide unsplit (250; 128 wide 334). Tiles of 64 weight rows
// double the workgroups of a short MXFP4 product: 48 rows against 14336 x 4096 in 16.2 us, 17.0 in 128.
// The MXFP4 step times are those of rows of whole steps; the other form's steps (tile_mxfp4_kernel) take
// about twice as long in every tile and have no table of their own.
struct TileCost { int bm, bn; double step; bool two; };
constexpr TileCost kBf16Tiles[] = {{128, 32, 0.70, true}, {128, 64, 0.77, true},
                                   {128, 128, 0.96, true}, {256, 256, 1.85, false}};
constexpr TileCost kMxTiles[] = {{64, 64, 0.45, true}, {128, 64, 0.60, true},
                                 {128, 128, 0.75, true}, {256, 256, 1.90, false}};
constexpr double kTile = 2.3, kTwoBf16 = 0.80, kTwoMx = 0.95, kLaunch = 3.0;
constexpr double kPartBytes = 6e6;

template <int N>
void plan_tiles(const MatmulArgs& a, const TileCost (&tiles)[N], double two, int cols, bool can_split,
                MatmulPlan& p) {
  const int cus = device_cu_count();
  const int64_t steps = (a.Cp + cols - 1) / cols;
  // experts' last tiles: some are empty, and the split of the rows over the experts is not known here
  const double extra = a.E > 1 ? 0.75 * (double)(a.E < a.T ? a.E : a.T) : 0.0;
  double best = 1e30;
  for (const TileCost& t : tiles) {
    const double across = a.E > 1 ? (double)a.T / t.bn + extra : (double)((a.T + t.bn - 1) / t.bn);
    const double n = (double)((a.R + t.bm - 1) / t.bm) * across;
    for (int split = 1; split <= (can_split ? 16 : 1); ++split) {
      if (split > 1 && (steps < 4 * split || n * split > 4.0 * cus)) break;
      const double each = (double)((steps + split - 1) / split) * t.step + kTile;
      const double on_cu = n * split / cus;
      double time = on_cu <= 1 ? each : (double)(int64_t)(on_cu + 0.999) * each * (t.two ? two : 1.0);
      if (split > 1) time += kLaunch + 8.0 * split * (double)a.T * (double)a.R / kPartBytes;
      if (time < best) {
        best = time;
        p.bm = t.bm;
        p.bn = t.bn;
        p.split = split;
      }
    }
  }
}

}  // namespace

MatmulPlan plan_matmul(const MatmulArgs& a, MatmulKind kind, bool can_split) {
  MatmulPlan p = {};
  p.split = 1;
  const int64_t rows = (a.T + a.E - 1) / a.E;    // rows of x an expert, on average
  if (rows <= kMfma || (kind == kMxMxfp4 && a.E == 1 && rows <= 2 * kMfma)) {
    const int64_t blocks = (a.R + kMfma - 1) / kMfma * (a.E < a.T ? a.E : a.T);
    p.nt = rows <= kMfma ? 1 : 2;
    p.rt = blocks > 2 * device_cu_count() ? 2 : 1;
    p.chunks = a.C >= 8192 ? 4 : 1;
    return p;
  }
  if (kind == kMxMxfp4) plan_tiles(a, kMxTiles, kTwoMx, 256, can_split, p);
  else plan_tiles(a, kBf16Tiles, kTwoBf16, 64, can_split, p);
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
        : kind == kMxMxfp4 ? launch_few_mxfp4(a, p, stream) : launch_few_mx_bf16(a, p, stream);
  else
    e = kind == kPacked ? launch_tile_packed(a, p, stream)
        : kind == kMxMxfp4 ? launch_tile_mxfp4(a, p, stream) : launch_tile_mx_bf16(a, p, stream);
  if (e != hipSuccess || p.split == 1) return e;
  const int64_t items = a.T * (part_row(a.R) / 4);
  hipLaunchKernelGGL(add_parts_kernel, dim3((unsigned)((items + kBlock - 1) / kBlock)), dim3(kBlock),
                     0, stream, a);
  return hipGetLastError();
}

}  // namespace aaac
