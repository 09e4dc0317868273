// Routing of rows to experts: the choice of k experts for each token, the order of the chosen slots by
// expert, and the rows' way to their experts and back.
//
// The choice. With scores s = softmax(l) or sigmoid(l) over the E experts of a token, an expert's value
// is v = s + bias. An expert whose logit or bias is -inf is left out. With groups, a group's value is
// the largest v of its experts or the sum of the two largest; only the top_groups best groups take part.
// The k largest v are chosen in descending order, the lowest index first among equals. Weights are s
// (without the bias), over their sum where renormalised, times `scale`. Slots that no expert is left for
// hold expert -1 and weight 0.
//
// The choice is made on exact keys: scores are monotonous in the logits, so without a bias (and unless
// scores are added up for groups) the logits themselves are compared; otherwise the values are computed
// in 64 bits, where a single precision's rounding would reorder neighbours. A NaN ranks above every
// number and shows in the weights.
#include "aaac.h"
#include "fp8.h"

namespace aaac {

namespace {

constexpr int kMaxBlocks = 256;                  // blocks of tokens, each counted on its own
constexpr int kWaves = 8;                        // waves of a block

template <int N> struct Int { static constexpr int value = N; };

template <int TYPE>
__device__ __forceinline__ float load_f32(const void* p, int64_t i) {
  if (TYPE == AAAC_F32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return TYPE == AAAC_BF16 ? __uint_as_float((uint32_t)b << 16) : (float)__builtin_bit_cast(_Float16, b);
}

__device__ __forceinline__ float load_any(int type, const void* p, int64_t i) {
  return type == AAAC_F32 ? load_f32<AAAC_F32>(p, i)
         : type == AAAC_BF16 ? load_f32<AAAC_BF16>(p, i) : load_f32<AAAC_F16>(p, i);
}

// Order-preserving keys: larger value, larger key; zeros of both signs alike, every NaN the largest.
// Key 0 is no value's: it marks what is left out.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0), sign = 1ull << 63;
  if ((b & ~sign) > 0x7ff0000000000000ull) return ~0ull;
  return b & sign ? ~b : b | sign;
}
__device__ __forceinline__ double value_of(uint64_t key) {
  const uint64_t sign = 1ull << 63;
  return __longlong_as_double((long long)(key & sign ? key ^ sign : ~key));
}

// The largest of the wave's values, in a scalar register. Lanes shift within their rows of 16, then
// each row's last lane passes its maximum on; lanes without a source take the 0 that no key is below.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, kWave - 1);
}

// Keys of 32 bits (logits) or of 64 (values).
template <bool EXACT> struct Keys;
template <> struct Keys<false> { typedef uint32_t T; };
template <> struct Keys<true> { typedef uint64_t T; };

// The lanes that hold the wave's largest key, none where it is 0.
__device__ __forceinline__ uint64_t top_lanes(uint32_t key) {
  const uint32_t top = wave_max(key);
  return top ? __ballot(key == top) : 0;
}
__device__ __forceinline__ uint64_t top_lanes(uint64_t key) {
  const uint32_t hi = (uint32_t)(key >> 32), top = wave_max(hi);
  if (!top) return 0;
  uint64_t lanes = __ballot(hi == top);
  if (lanes & (lanes - 1)) {                     // equal in the upper half: the lower decides
    const uint32_t lo = hi == top ? (uint32_t)key : 0u, low = wave_max(lo);
    lanes = __ballot(hi == top && lo == low);
  }
  return lanes;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_top(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const float o = __shfl_xor(v, d);
    v = v != v ? v : o != o ? o : fmaxf(v, o);   // a NaN stays
  }
  return v;
}

// One token by one wave. Groups take 64 / 2^ceil(log2 G) neighbouring lanes each, NV neighbouring
// experts a lane, so that lane order is expert order and a group is a power of two of lanes.
// Returns the expert of slot `lane`, or -1, and its weight.
template <int NV, bool EXACT>
__device__ __forceinline__ int choose(const RouteArgs& a, int64_t t, int lanes_per_group, float& weight) {
  typedef typename Keys<EXACT>::T Key;
  const int lane = threadIdx.x & (kWave - 1);
  const int per_group = a.E / a.groups, group = lane / lanes_per_group;
  const int j0 = (lane % lanes_per_group) * NV, e0 = group * per_group + j0;
  const int n = group < a.groups ? per_group - j0 : 0;      // experts of this lane: NV, or fewer
  float l[NV];
  const int64_t at = t * a.ldl;
  auto load = [&](auto type) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      l[v] = v < n ? load_f32<decltype(type)::value>(a.logits, at + e0 + v) : -INFINITY;
  };
  if (a.type == AAAC_F32) load(Int<AAAC_F32>());
  else if (a.type == AAAC_BF16) load(Int<AAAC_BF16>());
  else load(Int<AAAC_F16>());
  float top = 0.0f;
  double total = 1.0;
  if (!a.sigmoid && (EXACT || !a.renormalize)) {
    top = l[0];
#pragma unroll
    for (int v = 1; v < NV; ++v) top = top != top ? top : l[v] != l[v] ? l[v] : fmaxf(top, l[v]);
    top = wave_top(top);
    total = 0.0;
    if (top != -INFINITY) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (v < n) total += EXACT ? exp((double)l[v] - top) : (double)expf(l[v] - top);
      }
    }
    total = wave_sum(total);
  }
  Key key[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    key[v] = 0;
    if (EXACT) {
      double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[v])) : exp((double)l[v] - top) / total;
      const float b = a.bias && v < n ? a.bias[e0 + v] : 0.0f;
      if (v < n && l[v] != -INFINITY && b != -INFINITY) key[v] = (Key)key_of(s + b);
    } else if (v < n && l[v] != -INFINITY) {
      key[v] = (Key)key_of(l[v]);
    }
  }
  if (a.top_groups < a.groups) {
    Key best = 0, next = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      next = max(next, min(best, key[v]));
      best = max(best, key[v]);
    }
    for (int d = 1; d < lanes_per_group; d <<= 1) {
      const Key ob = (Key)__shfl_xor((unsigned long long)best, d);
      const Key on = (Key)__shfl_xor((unsigned long long)next, d);
      next = max(min(best, ob), max(next, on));
      best = max(best, ob);
    }
    if (EXACT && a.group_top == 2 && next != 0)
      best = (Key)key_of(value_of(best) + value_of(next));
    // a group's place among the groups, the lower index first among equals
    int place = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)best, g * lanes_per_group);
      Key o = lo;
      if (EXACT)
        o |= (Key)__builtin_amdgcn_readlane((uint32_t)((uint64_t)best >> 32), g * lanes_per_group) << (EXACT ? 32 : 0);
      place += o > best || (o == best && g < group) ? 1 : 0;
    }
    if (place >= a.top_groups) {
#pragma unroll
      for (int v = 0; v < NV; ++v) key[v] = 0;
    }
  }
  int mine = -1;
  Key best = 0;
  int which = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (key[v] > best) best = key[v], which = v;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    const uint64_t lanes = top_lanes(best);
    if (!lanes) break;
    const int from = __builtin_ctzll(lanes);
    const int e = __builtin_amdgcn_readlane(e0 + which, from);
    if (lane == j) mine = e;
    if (lane == from) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v == which) key[v] = 0;
      best = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (key[v] > best) best = key[v], which = v;
    }
  }
  // weights in 64 bits, a lane each
  double s = 0.0;
  const float lm = mine >= 0 ? load_any(a.type, a.logits, at + mine) : -INFINITY;
  if (a.sigmoid) {
    s = mine >= 0 ? 1.0 / (1.0 + exp(-(double)lm)) : 0.0;
  } else {
    if (!EXACT && a.renormalize) top = wave_top(lm);
    s = mine >= 0 ? exp((double)lm - (double)top) / total : 0.0;
  }
  if (a.renormalize) {
    const double sum = wave_sum(s);
    s = sum == 0.0 ? 0.0 : s / sum;
  }
  weight = (float)(s * (double)a.scale);
  return mine;
}

// The order of a block's slots [s0, s1). counts: LDS int [waves][E], in which wave w's row holds, for
// each expert, the place of the first of its slots; lists of slots run in order over the waves. A wave
// takes 64 slots at a time: lanes with the same expert find each other by a ballot for every bit of the
// expert's number, count the ones before them, and the last one moves the expert's next place on.
__device__ __forceinline__ void place_slots(const RouteArgs& a, volatile int* next, int64_t s0, int64_t s1,
                                            int bits) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint64_t below = (1ull << lane) - 1;
  for (int64_t s = s0; s < s1; s += kWave) {
    const int64_t slot = s + lane;
    const int e = slot < s1 ? a.experts[slot] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    if (e >= 0) {
      const int before = __popcll(same & below), place = next[e] + before;
      if (before + 1 == __popcll(same)) next[e] = place + 1;
      a.places[slot] = place;
      a.rows[place] = (int32_t)(slot / a.k);
    } else if (slot < s1) {
      a.places[slot] = -1;
    }
  }
}

// Everything after the choice for one block of tokens: counts and their sums in LDS, then the places.
// lds: int [place_ints]. The rows of each expert in earlier blocks and in every block are read from
// a.counts; with one block (`alone`) they are its own.
__host__ __device__ constexpr int place_ints(int E) { return kWaves * E + kWaves; }
__device__ __forceinline__ void place_block(const RouteArgs& a, int* lds, int block, int blocks,
                                            bool alone) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  constexpr int kThreads = kWaves * kWave, kShare = kMaxExperts / kThreads;
  int* hist = lds;                               // [kWaves][E]: slots of each wave, then their places
  int* sums = lds + kWaves * a.E;                // [kWaves]
  const int64_t slots = a.T * a.k, per = (int64_t)a.per_block * a.k, b0 = block * per;
  const int64_t b1 = b0 + per < slots ? b0 + per : slots;
  const int64_t each = (b1 - b0 + kWaves - 1) / kWaves;
  const int64_t s0 = b0 + wave * each < b1 ? b0 + wave * each : b1;
  const int64_t s1 = s0 + each < b1 ? s0 + each : b1;
  for (int i = tid; i < kWaves * a.E; i += kThreads) hist[i] = 0;
  __syncthreads();
  for (int64_t s = s0 + lane; s < s1; s += kWave) {
    const int e = a.experts[s];
    if (e >= 0) atomicAdd(&hist[wave * a.E + e], 1);
  }
  __syncthreads();
  // a thread's experts: kShare neighbours
  int all[kShare], before[kShare], mine = 0;
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    const int e = tid * kShare + i;
    all[i] = before[i] = 0;
    if (e < a.E) {
      if (alone) {
        for (int w = 0; w < kWaves; ++w) all[i] += hist[w * a.E + e];
      } else {
        const int32_t* c = a.counts + e;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
          const int n = c[(int64_t)b * a.E];
          all[i] += n;
          before[i] += b < block ? n : 0;
        }
      }
      mine += all[i];
    }
  }
  int run = mine;                                // inclusive over the wave
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == kWave - 1) sums[wave] = run;
  __syncthreads();
  int first = run - mine, total = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) first += sums[w];
    total += sums[w];
  }
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    const int e = tid * kShare + i;
    if (e < a.E) {
      if (block == 0) a.offsets[e] = first;
      int at = first + before[i];
      for (int w = 0; w < kWaves; ++w) {
        const int n = hist[w * a.E + e];
        hist[w * a.E + e] = at;
        at += n;
      }
      first += all[i];
    }
  }
  if (block == 0 && tid == 0) a.offsets[a.E] = total;
  // places that no slot has
  for (int64_t i = total + (int64_t)block * kThreads + tid; i < slots; i += (int64_t)blocks * kThreads)
    a.rows[i] = -1;
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
  place_slots(a, hist + wave * a.E, s0, s1, bits);
}

// alone: the one block of a call with few tokens orders its slots too.
template <int NV, bool EXACT>
__global__ __launch_bounds__(kWaves * kWave) void route_kernel(RouteArgs a, int lanes_per_group,
                                                               bool alone) {
  extern __shared__ int lds[];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t t0 = (int64_t)blockIdx.x * a.per_block;
  const int64_t t1 = t0 + a.per_block < a.T ? t0 + a.per_block : a.T;
  if (!alone) {
    for (int i = threadIdx.x; i < a.E; i += kWaves * kWave) lds[i] = 0;
    __syncthreads();
  }
  for (int64_t t = t0 + wave; t < t1; t += kWaves) {
    float weight;
    const int e = choose<NV, EXACT>(a, t, lanes_per_group, weight);
    if (lane < a.k) {
      a.experts[t * a.k + lane] = e;
      a.weights[t * a.k + lane] = weight;
      if (!alone && e >= 0) atomicAdd(&lds[e], 1);
    }
  }
  __syncthreads();
  if (alone) {
    place_block(a, lds, 0, 1, true);
  } else {
    for (int i = threadIdx.x; i < a.E; i += kWaves * kWave)
      a.counts[(int64_t)blockIdx.x * a.E + i] = lds[i];
  }
}

__global__ __launch_bounds__(kWaves * kWave) void place_kernel(RouteArgs a, int blocks) {
  extern __shared__ int lds[];
  place_block(a, lds, blockIdx.x, blocks, false);
}

// A block's tokens: one a wave up to kMaxBlocks blocks, then equal shares. One block is one launch.
int tokens_per_block(int64_t T) {
  const int64_t n = (T + kMaxBlocks - 1) / kMaxBlocks;
  return (int)((n + kWaves - 1) / kWaves * kWaves);
}

template <int NV, bool EXACT>
hipError_t route_n(const RouteArgs& a, int lanes_per_group, hipStream_t stream) {
  const int blocks = (int)((a.T + a.per_block - 1) / a.per_block);
  const bool alone = blocks == 1;
  const size_t lds = sizeof(int) * place_ints(a.E);
  hipLaunchKernelGGL((route_kernel<NV, EXACT>), dim3(blocks), dim3(kWaves * kWave),
                     alone ? lds : sizeof(int) * a.E, stream, a, lanes_per_group, alone);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || alone) return e;
  hipLaunchKernelGGL(place_kernel, dim3(blocks), dim3(kWaves * kWave), lds, stream, a, blocks);
  return hipGetLastError();
}

template <bool EXACT>
hipError_t route_e(const RouteArgs& a, hipStream_t stream) {
  int groups = 1;
  while (groups < a.groups) groups <<= 1;
  const int lanes = kWave / groups, each = (a.E / a.groups + lanes - 1) / lanes;
  if (each <= 1) return route_n<1, EXACT>(a, lanes, stream);
  if (each <= 2) return route_n<2, EXACT>(a, lanes, stream);
  if (each <= 4) return route_n<4, EXACT>(a, lanes, stream);
  if (each <= 8) return route_n<8, EXACT>(a, lanes, stream);
  return route_n<16, EXACT>(a, lanes, stream);   // 512 experts in groups of any number
}

// no tokens: every expert's rows start and end at 0
__global__ void no_offsets_kernel(int32_t* offsets, int n) {
  for (int i = threadIdx.x; i < n; i += kBlock) offsets[i] = 0;
}

// ------------------------------------------------------------------------------------------------
// Rows to experts and back: bound by memory. A workgroup takes one token and 256 words of its row: the
// row is read once and written to each of its places, in words of 16, 4 or 2 bytes as the rows' addresses
// allow. Places outside [0, N) are skipped.
// ------------------------------------------------------------------------------------------------
template <class Word>
__global__ __launch_bounds__(kBlock) void rows_to_experts_kernel(
    const uint8_t* __restrict__ x, int64_t words, int64_t ldx, const int32_t* __restrict__ places, int k,
    uint8_t* __restrict__ out, int64_t N, int64_t ldo, int64_t chunks, int64_t blocks) {
  const int64_t id = block_id();
  if (id >= blocks) return;
  const int64_t t = id / chunks, w = (id - t * chunks) * kBlock + threadIdx.x;
  if (w >= words) return;
  const Word v = reinterpret_cast<const Word*>(x + t * ldx)[w];
  for (int j = 0; j < k; ++j) {
    const int64_t p = places[t * k + j];
    if (p >= 0 && p < N) reinterpret_cast<Word*>(out + p * ldo)[w] = v;
  }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// V neighbours of a row as fp32.
template <int TYPE, int V>
__device__ __forceinline__ void load_v(const void* p, int64_t i, float (&v)[V]) {
  if (V == 1) {
    v[0] = load_f32<TYPE>(p, i);
  } else if (TYPE == AAAC_F32) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = __uint_as_float(w[c & 3]);
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const uint16_t b = (uint16_t)(w[(c >> 1) & 3] >> (16 * (c & 1)));
      v[c] = TYPE == AAAC_BF16 ? __uint_as_float((uint32_t)b << 16)
                               : (float)__builtin_bit_cast(_Float16, b);
    }
  }
}
__device__ __forceinline__ uint16_t to_16(int type, float v) {
  return type == AAAC_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)v)
                           : __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <int TYPE, int V>
__global__ __launch_bounds__(kBlock) void rows_from_experts_kernel(
    const void* __restrict__ y, int64_t N, int64_t C, int64_t ldy, const int32_t* __restrict__ places,
    const float* __restrict__ weights, int k, void* __restrict__ out, int out_type, int64_t ldo,
    int64_t chunks, int64_t blocks) {
  const int64_t id = block_id();
  if (id >= blocks) return;
  const int64_t t = id / chunks, c = ((id - t * chunks) * kBlock + threadIdx.x) * V;
  if (c >= C) return;
  float sum[V] = {};
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int64_t p = places[t * k + j];
    if (p < 0 || p >= N) continue;
    const float w = weights[t * k + j];
    float v[V];
    load_v<TYPE, V>(y, p * ldy + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = __builtin_fmaf(w, v[i], sum[i]);
  }
  const int64_t at = t * ldo + c;
  if (out_type == AAAC_F32) {
    float* o = static_cast<float*>(out) + at;
    if (V == 1) {
      o[0] = sum[0];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4)
        *reinterpret_cast<u32x4*>(o + i) =
            u32x4{__float_as_uint(sum[i % V]), __float_as_uint(sum[(i + 1) % V]),
                  __float_as_uint(sum[(i + 2) % V]), __float_as_uint(sum[(i + 3) % V])};
    }
    return;
  }
  uint16_t* o = static_cast<uint16_t*>(out) + at;
  uint32_t w[(V + 1) / 2];
#pragma unroll
  for (int i = 0; i < V; i += 2)
    w[i / 2] = to_16(out_type, sum[i]) | (V > 1 ? (uint32_t)to_16(out_type, sum[(i + 1) % V]) << 16 : 0u);
  if (V == 8) *reinterpret_cast<u32x4*>(o) = u32x4{w[0], w[1 % ((V + 1) / 2)], w[2 % ((V + 1) / 2)], w[3 % ((V + 1) / 2)]};
  else if (V == 4) *reinterpret_cast<u32x2*>(o) = u32x2{w[0], w[1 % ((V + 1) / 2)]};
  else o[0] = (uint16_t)w[0];
}

template <int TYPE>
hipError_t from_experts(const void* y, int64_t N, int64_t C, int64_t ldy, const int32_t* places,
                        const float* weights, int64_t T, int k, void* out, int out_type, int64_t ldo,
                        hipStream_t stream) {
  constexpr int V = TYPE == AAAC_F32 ? 4 : 8;    // 16 bytes of y
  const int ob = out_type == AAAC_F32 ? 4 : 2, store = V * ob < 16 ? V * ob : 16;
  const bool vec = (uintptr_t)y % 16 == 0 && ldy % V == 0 && C % V == 0 && (uintptr_t)out % store == 0 &&
                   (ldo * ob) % store == 0;
  const int64_t chunks = (C + kBlock * (vec ? V : 1) - 1) / (kBlock * (vec ? V : 1)), blocks = T * chunks;
  if (vec)
    hipLaunchKernelGGL((rows_from_experts_kernel<TYPE, V>), grid_of(blocks), dim3(kBlock), 0, stream, y, N,
                       C, ldy, places, weights, k, out, out_type, ldo, chunks, blocks);
  else
    hipLaunchKernelGGL((rows_from_experts_kernel<TYPE, 1>), grid_of(blocks), dim3(kBlock), 0, stream, y, N,
                       C, ldy, places, weights, k, out, out_type, ldo, chunks, blocks);
  return hipGetLastError();
}

template <class Word>
hipError_t to_experts(const void* x, int64_t T, int64_t bytes, int64_t ldx, const int32_t* places, int k,
                      void* out, int64_t N, int64_t ldo, hipStream_t stream) {
  const int64_t words = bytes / sizeof(Word), chunks = (words + kBlock - 1) / kBlock, blocks = T * chunks;
  hipLaunchKernelGGL((rows_to_experts_kernel<Word>), grid_of(blocks), dim3(kBlock), 0, stream,
                     static_cast<const uint8_t*>(x), words, ldx, places, k, static_cast<uint8_t*>(out), N,
                     ldo, chunks, blocks);
  return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int E) {
  const int64_t per = tokens_per_block(T);
  return T <= per ? 0 : sizeof(int32_t) * (size_t)((T + per - 1) / per) * (size_t)E;
}

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  if (a.T == 0) {
    hipLaunchKernelGGL(no_offsets_kernel, dim3(1), dim3(kBlock), 0, stream, a.offsets, a.E + 1);
    return hipGetLastError();
  }
  a.per_block = tokens_per_block(a.T);
  const bool exact = a.bias || (a.top_groups < a.groups && a.group_top == 2);
  return exact ? route_e<true>(a, stream) : route_e<false>(a, stream);
}

hipError_t launch_rows_to_experts(const void* x, int64_t T, int64_t bytes, int64_t ldx,
                                  const int32_t* places, int k, void* out, int64_t N, int64_t ldo,
                                  int element, hipStream_t stream) {
  if (T == 0 || bytes == 0) return hipSuccess;
  const uint64_t low = (uintptr_t)x | (uintptr_t)out | (uint64_t)bytes | (uint64_t)ldx | (uint64_t)ldo;
  if (low % 16 == 0) return to_experts<u32x4>(x, T, bytes, ldx, places, k, out, N, ldo, stream);
  if (low % 4 == 0) return to_experts<uint32_t>(x, T, bytes, ldx, places, k, out, N, ldo, stream);
  if (element == 1) return to_experts<uint8_t>(x, T, bytes, ldx, places, k, out, N, ldo, stream);
  return to_experts<uint16_t>(x, T, bytes, ldx, places, k, out, N, ldo, stream);
}

hipError_t launch_rows_from_experts(const void* y, int type, int64_t N, int64_t C, int64_t ldy,
                                    const int32_t* places, const float* weights, int64_t T, int k,
                                    void* out, int out_type, int64_t ldo, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (type == AAAC_F32)
    return from_experts<AAAC_F32>(y, N, C, ldy, places, weights, T, k, out, out_type, ldo, stream);
  if (type == AAAC_BF16)
    return from_experts<AAAC_BF16>(y, N, C, ldy, places, weights, T, k, out, out_type, ldo, stream);
  return from_experts<AAAC_F16>(y, N, C, ldy, places, weights, T, k, out, out_type, ldo, stream);
}

}  // namespace aaac
