// How a product call is run: the choice of kernel and tile, and the kernel that adds the parts of a
// sum that was split over workgroups.
#include "matmul.h"
#ifdef TUNE
#include <stdlib.h>
#endif

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

}  // namespace

MatmulPlan plan_matmul(const MatmulArgs& a, MatmulKind kind, bool can_split) {
  MatmulPlan p = {};
  p.split = 1;
  const int64_t rows = (a.T + a.E - 1) / a.E;    // rows of x an expert, on average
#ifdef TUNE
  {
    auto v = [](const char* n, int d) { const char* s = getenv(n); return s ? atoi(s) : d; };
    p.bn = v("BN", 0); p.bm = p.bn == 256 ? 256 : 128; p.split = can_split ? v("SPLIT", 1) : 1;
    p.rt = v("RT", 1); p.nt = v("NT", 1); p.waves = v("WAVES", 8); p.chunks = v("U", 4);
    return p;
  }
#endif
  const bool fp4 = kind == kMxMxfp4;
  if (rows <= (fp4 ? 64 : kMfma)) {
    p.nt = (int)((rows + kMfma - 1) / kMfma);
    const int64_t blocks = (a.R + kMfma - 1) / kMfma * (a.E < a.T ? a.E : a.T);
    p.rt = blocks > 512 ? 2 : 1;
    p.waves = blocks > 256 ? 8 : 16;
    p.chunks = a.C >= 512 * p.waves ? 4 : 1;
    return p;
  }
  p.bn = rows <= 64 ? 64 : rows <= 512 ? 128 : 256;
  p.bm = p.bn == 256 ? 256 : 128;
  if (can_split) {
    const int64_t tiles = (a.R + p.bm - 1) / p.bm * ((a.T + p.bn - 1) / p.bn);
    const int64_t steps = (a.Cp + (fp4 ? 255 : 63)) / (fp4 ? 256 : 64);
    while (tiles * p.split < 256 && p.split * 8 <= steps) ++p.split;
  }
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
