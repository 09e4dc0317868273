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
// number; a logit's shows in the weights, which no bias enters.
#include "aaac.h"
#include "fp8.h"

namespace aaac {

namespace {

constexpr int kMaxBlocks = 256;                  // blocks of tokens, each counted on its own
constexpr int kWaves = 16;                       // waves of a block: four a SIMD hide what one waits for

template <int N> struct Int { static constexpr int value = N; };
template <bool B, class X, class Y> struct Pick { typedef X type; };
template <class X, class Y> struct Pick<false, X, Y> { typedef Y type; };

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

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
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

// The partner's key in a block of 2 D lanes whose halves are alike within themselves.
template <int D>
__device__ __forceinline__ uint32_t other(uint32_t v) {
  if (D == 1) return dpp_u32<kDppQuadXor1>(v);
  if (D == 2) return dpp_u32<kDppQuadXor2>(v);
  if (D == 4) return dpp_u32<kDppRowHalfMirror>(v);
  if (D == 8) return dpp_u32<kDppRowMirror>(v);
  return (uint32_t)__shfl_xor((int)v, D);
}
template <int D>
__device__ __forceinline__ uint64_t other(uint64_t v) {
  return (uint64_t)other<D>((uint32_t)(v >> 32)) << 32 | other<D>((uint32_t)v);
}

// e^x for x <= 0 in 64 bits: x = n ln 2 + r with |r| <= ln 2 / 2, and the Taylor polynomial of e^r up to
// r^13 (what follows is below 2^-57). NaN gives some number: callers look for it in x.
__device__ __forceinline__ double exp64(double x) {
  x = fmax(x, -750.0);                           // 0 from there on
  const double n = rint(x * 1.4426950408889634);
  double r = __builtin_fma(-n, 0.6931471805599453, x);
  r = __builtin_fma(-n, 2.3190468138462996e-17, r);
  double p = 1.0 / 6227020800.0;
#pragma unroll
  for (int i = 0; i < 13; ++i) {
    const double c[] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                        1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
    double k = c[i];
    if (i < 10) asm("" : "+s"(k));               // a scalar operand: in vector registers each is copied first
    p = __builtin_fma(p, r, k);
  }
  return ldexp(p, (int)n);
}
// 1 / d, d normal: the instruction's estimate and two steps of Newton's method.
__device__ __forceinline__ double reciprocal(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
__device__ __forceinline__ double sigmoid64(float l) {
  const double e = exp64(-fabs((double)l)), r = reciprocal(1.0 + e);
  return l > 0.0f ? r : e * r;
}

// NV neighbouring logits; those at or past n are -inf. VEC: n is 0 or NV and they lie on their whole size.
template <int TYPE, int NV, bool VEC>
__device__ __forceinline__ void load_logits(const void* p, int64_t at, int n, float (&l)[NV]) {
  if (VEC) {
    typedef typename Pick<TYPE == AAAC_F32, uint32_t, uint16_t>::type T;
    T v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = -INFINITY;
    if (n > 0) {
      __builtin_memcpy(v, __builtin_assume_aligned(static_cast<const T*>(p) + at, sizeof(v) < 16 ? sizeof(v) : 16),
                       sizeof(v));
#pragma unroll
      for (int i = 0; i < NV; ++i)
        l[i] = TYPE == AAAC_F32 ? __uint_as_float((uint32_t)v[i])
               : TYPE == AAAC_BF16 ? __uint_as_float((uint32_t)v[i] << 16)
                                   : (float)__builtin_bit_cast(_Float16, (uint16_t)v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = i < n ? load_f32<TYPE>(p, at + i) : -INFINITY;
  }
}

// One token by one wave. Groups take 64 / 2^ceil(log2 G) neighbouring lanes each, NV neighbouring experts a
// lane, so that lane order is expert order and a group is a power of two of lanes. bias: of the lane's
// experts, -inf past the last. Returns the expert of slot `lane`, or -1, and its weight.
//
// Bound by vector instructions, some 780 a token with 256 experts in groups, a bias and k = 8 (16384 tokens:
// 32 us, 22 of them at full issue; the logits' bytes would take 3). A lane's few keys are sorted once, so that
// the k rounds of selection only look at each lane's first. Two tokens side by side in a wave took 30 us,
// and 11 instead of 8 us for one token.
template <int NV, bool EXACT>
__device__ __forceinline__ int choose(const RouteArgs& a, int64_t t, int lanes_per_group,
                                      const float (&bias)[NV], float& weight) {
  typedef typename Keys<EXACT>::T Key;
  constexpr bool kSorted = NV <= 4;
  const int lane = threadIdx.x & (kWave - 1);
  const int per_group = a.E / a.groups, group = lane / lanes_per_group;
  const int j0 = (lane % lanes_per_group) * NV, e0 = group * per_group + j0;
  const int n = group < a.groups ? per_group - j0 : 0;      // experts of this lane: NV, or fewer
  const int64_t at = t * a.ldl;
  float l[NV];
  auto load = [&](auto type) __attribute__((always_inline)) {
    if (a.vec) load_logits<decltype(type)::value, NV, true>(a.logits, at + e0, n, l);
    else load_logits<decltype(type)::value, NV, false>(a.logits, at + e0, n, l);
  };
  if (a.type == AAAC_F32) load(Int<AAAC_F32>());
  else if (a.type == AAAC_BF16) load(Int<AAAC_BF16>());
  else load(Int<AAAC_F16>());
  float top = 0.0f;
  double over = 1.0;
  if (!a.sigmoid && (EXACT || !a.renormalize)) {
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) best = max(best, key_of(l[v]));
    top = value_of(wave_max(best));
    double total = 0.0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const double x = (double)l[v] - top;
      total += x != x ? x : EXACT ? exp64(x) : (double)expf((float)x);
    }
    // a row of -inf has no scores; its x are NaN
    over = top == -INFINITY ? 0.0 : 1.0 / block_sum_f64(total, kWave);
  }
  Key key[NV];
  int which[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) which[v] = v;
  // l or bias -inf, a NaN beside it or not (the minimum is then the other): 0, also past the lane's last expert
  if constexpr (EXACT) {
    auto take = [&](int v, double s) __attribute__((always_inline)) {
      const Key k = key_of(s + (double)bias[v]);
      key[v] = fminf(l[v], bias[v]) == -INFINITY ? 0 : l[v] != l[v] ? ~(Key)0 : k;
    };
    if (a.sigmoid) {
#pragma unroll
      for (int v = 0; v < NV; ++v) take(v, sigmoid64(l[v]));
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const double x = (double)l[v] - top;
        take(v, x != x ? x : exp64(x) * over);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = l[v] == -INFINITY ? 0 : (Key)key_of(l[v]);
  }
  if (kSorted) {
    // neighbours in turn; equals keep their order
#pragma unroll
    for (int i = NV - 1; i > 0; --i)
#pragma unroll
      for (int v = 0; v < i; ++v) {
        const bool swap = key[v + 1] > key[v];
        const Key k = swap ? key[v] : key[v + 1];
        const int w = swap ? which[v] : which[v + 1];
        key[v] = swap ? key[v + 1] : key[v];
        which[v] = swap ? which[v + 1] : which[v];
        key[v + 1] = k;
        which[v + 1] = w;
      }
  }
  if (a.top_groups < a.groups) {
    Key best = key[0], next = 0;
#pragma unroll
    for (int v = 1; v < NV; ++v) {
      next = max(next, min(best, key[v]));
      best = max(best, key[v]);
      if (kSorted) break;
    }
    auto join = [&](auto d) __attribute__((always_inline)) {
      constexpr int D = decltype(d)::value;
      if (D >= lanes_per_group) return;
      const Key ob = other<D>(best);
      if (EXACT) next = max(min(best, ob), max(next, other<D>(next)));
      best = max(best, ob);
    };
    join(Int<1>());
    join(Int<2>());
    join(Int<4>());
    join(Int<8>());
    join(Int<16>());
    join(Int<32>());
    if constexpr (EXACT) {
      if (a.group_top == 2 && next != 0) best = key_of(value_of(best) + value_of(next));
    }
    // a group's place among the groups, the lower index first among equals
    int place = 0;
    for (int g = 0; g < a.groups; ++g) {
      Key o = (uint32_t)__builtin_amdgcn_readlane((uint32_t)best, g * lanes_per_group);
      if constexpr (EXACT) {
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(best >> 32), g * lanes_per_group);
        o |= (Key)hi << 32;
      }
      place += o > best || (o == best && g < group) ? 1 : 0;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = place >= a.top_groups ? 0 : key[v];
  }
  int mine = -1;
  Key best = key[0];
  int first = which[0];
  if (!kSorted) {
#pragma unroll
    for (int v = 1; v < NV; ++v)
      if (key[v] > best) best = key[v], first = v;
  }
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    const uint64_t lanes = top_lanes(best);
    if (!lanes) break;
    const int from = __builtin_ctzll(lanes);
    const int e = __builtin_amdgcn_readlane(e0 + first, from);
    if (lane == j) mine = e;
    if (lane == from) {
      if (kSorted) {
#pragma unroll
        for (int v = 0; v + 1 < NV; ++v) key[v] = key[v + 1], which[v] = which[v + 1];
        key[NV - 1] = 0;
        best = key[0];
        first = which[0];
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v == first) key[v] = 0;
        best = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (key[v] > best) best = key[v], first = v;
      }
    }
  }
  // weights in 64 bits, a lane each; `lanes`, a power of two, hold all of them
  int lanes = 1;
  while (lanes < a.k) lanes <<= 1;
  double s = 0.0;
  const float lm = mine >= 0 ? load_any(a.type, a.logits, at + mine) : -INFINITY;
  if (a.sigmoid) {
    s = lm != lm ? (double)lm : mine >= 0 ? sigmoid64(lm) : 0.0;
  } else {
    if (!EXACT && a.renormalize) top = value_of(block_max_u32(key_of(lm), lanes));
    const double x = (double)lm - (double)top;
    s = mine < 0 ? 0.0 : x != x ? x : exp64(x) * over;
  }
  if (a.renormalize) {
    const double sum = block_sum_f64(s, lanes);
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
__host__ __device__ constexpr int count_row(int E) { return (E + 3) & ~3; }
constexpr int kThreads = kWaves * kWave;
__host__ __device__ constexpr int place_ints(int E) { return kWaves * E + kWaves + 2 * 4 * kThreads; }
__device__ __forceinline__ void place_block(const RouteArgs& a, int* lds, int block, int blocks,
                                            bool alone) {
  static_assert(kMaxExperts <= kThreads, "an expert a thread");
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_index();
  int* sum = lds;                                // [kThreads][2][4]: a thread's part of the counts
  int* hist = lds + 2 * 4 * kThreads;            // [kWaves][E]: slots of each wave, then their places
  int* sums = hist + kWaves * a.E;               // [kWaves]
  const int64_t slots = a.T * a.k, per = (int64_t)a.per_block * a.k, b0 = block * per;
  const int64_t b1 = b0 + per < slots ? b0 + per : slots;
  const int64_t each = (b1 - b0 + kWaves - 1) / kWaves;
  const int64_t s0 = b0 + wave * each < b1 ? b0 + wave * each : b1;
  const int64_t s1 = s0 + each < b1 ? s0 + each : b1;
  for (int i = tid; i < kWaves * a.E; i += kThreads) hist[i] = 0;
  // four experts a thread, the blocks dealt out over what threads that leaves
  const int cols = count_row(a.E) / 4, room = kThreads / cols < 8 ? kThreads / cols : 8;
  const int ways = blocks < room ? blocks : room;
  if (!alone) {
    int4 all = {0, 0, 0, 0}, before = {0, 0, 0, 0};
    if (tid < cols * ways) {
      const int4* c = reinterpret_cast<const int4*>(a.counts) + tid % cols;
#pragma unroll 8
      for (int b = tid / cols; b < blocks; b += ways) {
        const int4 n = c[(int64_t)b * cols];
        const int m = b < block ? -1 : 0;
        all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
        before.x += n.x & m, before.y += n.y & m, before.z += n.z & m, before.w += n.w & m;
      }
    }
    reinterpret_cast<int4*>(sum)[2 * tid] = all;
    reinterpret_cast<int4*>(sum)[2 * tid + 1] = before;
  }
  __syncthreads();
  for (int64_t s = s0 + lane; s < s1; s += kWave) {
    const int e = a.experts[s];
    if (e >= 0) atomicAdd(&hist[wave * a.E + e], 1);
  }
  __syncthreads();
  int all = 0, before = 0;                       // of expert tid
  if (tid < a.E) {
    if (alone) {
      for (int w = 0; w < kWaves; ++w) all += hist[w * a.E + tid];
    } else {
      for (int i = tid / 4; i < cols * ways; i += cols) {
        all += sum[8 * i + (tid & 3)];
        before += sum[8 * i + 4 + (tid & 3)];
      }
    }
  }
  int run = all;                                 // inclusive over the wave
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == kWave - 1) sums[wave] = run;
  __syncthreads();
  int first = run - all, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) first += sums[w];
    total += sums[w];
  }
  if (tid < a.E) {
    if (block == 0) a.offsets[tid] = first;
    int at = first + before;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int n = hist[w * a.E + tid];
      hist[w * a.E + tid] = at;
      at += n;
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
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, int lanes_per_group, bool alone) {
  extern __shared__ int lds[];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_index();
  const int64_t t0 = (int64_t)blockIdx.x * a.per_block;
  const int64_t t1 = t0 + a.per_block < a.T ? t0 + a.per_block : a.T;
  if (!alone) {
    for (int i = threadIdx.x; i < a.E; i += kThreads) lds[i] = 0;
    __syncthreads();
  }
  float bias[NV];
  {
    const int group = lane / lanes_per_group, per_group = a.E / a.groups, j0 = lane % lanes_per_group * NV;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = group < a.groups && j0 + v < per_group;
      bias[v] = !in ? -INFINITY : EXACT && a.bias ? a.bias[group * per_group + j0 + v] : 0.0f;
    }
  }
  for (int64_t t = t0 + wave; t < t1; t += kWaves) {
    float weight;
    const int e = choose<NV, EXACT>(a, t, lanes_per_group, bias, weight);
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
    // a row of counts ends on 16 bytes; what follows the experts is never used
    for (int i = threadIdx.x; i < a.E; i += kThreads)
      a.counts[(int64_t)blockIdx.x * count_row(a.E) + i] = lds[i];
  }
}

__global__ __launch_bounds__(kThreads) void place_kernel(RouteArgs a, int blocks) {
  extern __shared__ int lds[];
  place_block(a, lds, blockIdx.x, blocks, false);
}

// A block's tokens: one a wave up to kMaxBlocks blocks, then equal shares. One block is one launch, so a
// block's waves take more tokens each where that is all of them: 48 tokens over 60 experts 13.6 us (in two
// launches 17.9), 24 over 256 in groups with a bias 15.3 (18.8), 32 of these 19.7 (18.8).
int tokens_per_block(int64_t T, int E) {
  const int alone = E <= 64 ? 4 * kWaves : E <= 128 ? 3 * kWaves : E <= 256 ? 3 * kWaves / 2 : kWaves;
  if (T <= alone) return alone;
  const int64_t n = (T + kMaxBlocks - 1) / kMaxBlocks;
  return (int)((n + kWaves - 1) / kWaves * kWaves);
}

template <int NV, bool EXACT>
hipError_t route_n(RouteArgs a, int lanes_per_group, hipStream_t stream) {
  const int b = a.type == AAAC_F32 ? 4 : 2, whole = NV * b < 16 ? NV * b : 16;
  a.vec = (uintptr_t)a.logits % whole == 0 && a.ldl % NV == 0 && a.E / a.groups % NV == 0;
  const int blocks = (int)((a.T + a.per_block - 1) / a.per_block);
  const bool alone = blocks == 1;
  const size_t lds = sizeof(int) * place_ints(a.E);
  hipLaunchKernelGGL((route_kernel<NV, EXACT>), dim3(blocks), dim3(kThreads),
                     alone ? lds : sizeof(int) * a.E, stream, a, lanes_per_group, alone);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || alone) return e;
  hipLaunchKernelGGL(place_kernel, dim3(blocks), dim3(kThreads), lds, stream, a, blocks);
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
// Rows to experts and back: bound by memory. A thread takes 16 bytes of a token's row, which are read once and
// written to each of the row's places; a workgroup one token or, where rows are short, several (16384 x 4 rows
// of 130 in bf16: 8 us there and 8 back, with one 23 and 21). Rows that do not start on 16 bytes but on four are
// moved by words, neighbouring ones by a wave's lanes (4096 x 4 rows of 4094: 27 and 28 us, in pieces of 16
// unaligned bytes 34 and 32, rows of 4096 26); two-byte elements on any address are put together to words there
// (rows of 4095: 28 us, 37 in unaligned pieces), and the rest goes in such pieces (back: 34).
// Places outside [0, N) are skipped. 8192 x 8 rows of 4096 in bf16: 87 us there and 161 back, together 4.9
// TB/s (some of what the first writes reaches memory while the second runs).
// ------------------------------------------------------------------------------------------------
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// What a thread takes: token t, and of its row the piece of `size` units that starts at `at`. A workgroup has
// one token's kBlock pieces, or several tokens where rows have fewer.
struct RowGrid {
  int64_t T, chunks, blocks;   // workgroups a token, all workgroups
  int per, tokens;             // threads a token, tokens a workgroup
};
RowGrid row_grid(int64_t T, int64_t pieces) {
  RowGrid g;
  g.T = T;
  g.chunks = (pieces + kBlock - 1) / kBlock;
  g.per = pieces < kBlock ? (int)pieces : kBlock;
  g.tokens = kBlock / g.per;
  g.blocks = (T + g.tokens - 1) / g.tokens * g.chunks;
  return g;
}
// The thread's token, and its number among the row's; false where it has none. ONE: one token a workgroup,
// whose places and weights are then scalar loads (8192 x 8 rows of 4096 back: 121 us, 133 otherwise).
template <bool ONE>
__device__ __forceinline__ bool row_place(const RowGrid& g, int64_t& t, int64_t& i) {
  const int64_t id = block_id();
  if (id >= g.blocks) return false;
  if (ONE) {
    t = id / g.chunks;
    i = (id - t * g.chunks) * kBlock + threadIdx.x;
    return true;
  }
  const int first = threadIdx.x / g.per;
  t = id / g.chunks * g.tokens + first;
  i = id % g.chunks * kBlock + threadIdx.x - first * g.per;
  return first < g.tokens && t < g.T;
}

// VEC: on 16 bytes. Of the row's last piece there may be only `bytes` < 16, a multiple of the element's.
template <bool VEC>
__device__ __forceinline__ u32x4 load_piece(const uint8_t* p, int bytes, int element) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (VEC) return *reinterpret_cast<const u32x4*>(p);
  if (bytes >= 16) {
    __builtin_memcpy(&v, p, 16);
    return v;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i >= bytes) break;
    if (element == 1) v[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    else if (i % 4 == 0 && element == 4) v[i >> 2] = *reinterpret_cast<const uint32_t*>(p + i);
    else if (i % 2 == 0 && element == 2)
      v[i >> 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + i) << (8 * (i & 3));
  }
  return v;
}
template <bool VEC>
__device__ __forceinline__ void store_piece(uint8_t* p, int bytes, int element, u32x4 v) {
  if (VEC) {
    *reinterpret_cast<u32x4*>(p) = v;
  } else if (bytes >= 16) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i >= bytes) break;
      if (element == 1) p[i] = (uint8_t)(v[i >> 2] >> (8 * (i & 3)));
      else if (i % 4 == 0 && element == 4) *reinterpret_cast<uint32_t*>(p + i) = v[i >> 2];
      else if (i % 2 == 0 && element == 2)
        *reinterpret_cast<uint16_t*>(p + i) = (uint16_t)(v[i >> 2] >> (8 * (i & 3)));
    }
  }
}

template <bool VEC, bool ONE>
__global__ __launch_bounds__(kBlock) void rows_to_experts_kernel(
    const uint8_t* __restrict__ x, int64_t bytes, int64_t ldx, const int32_t* __restrict__ places, int k,
    uint8_t* __restrict__ out, int64_t N, int64_t ldo, int element, RowGrid grid) {
  int64_t t, at;
  if (!row_place<ONE>(grid, t, at)) return;
  at *= 16;
  if (at >= bytes) return;
  const int left = bytes - at < 16 ? (int)(bytes - at) : 16;
  const u32x4 v = load_piece<VEC>(x + t * ldx + at, left, element);
  for (int j = 0; j < k; ++j) {
    const int64_t p = places[t * k + j];
    if (p >= 0 && p < N) store_piece<VEC>(out + p * ldo + at, left, element, v);
  }
}

// Rows on four bytes: a wave's 64 lanes take neighbouring words, four times.
template <bool ONE>
__global__ __launch_bounds__(kBlock) void rows_to_experts_words_kernel(
    const uint32_t* __restrict__ x, int64_t words, int64_t ldx, const int32_t* __restrict__ places, int k,
    uint32_t* __restrict__ out, int64_t N, int64_t ldo, RowGrid grid) {
  int64_t t, at;
  if (!row_place<ONE>(grid, t, at)) return;
  const int step = ONE ? kBlock : grid.per;
  at += at / kBlock * (3 * kBlock);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * step < words) v[i] = x[t * ldx + at + i * step];
  for (int j = 0; j < k; ++j) {
    const int64_t p = places[t * k + j];
    if (p < 0 || p >= N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * step < words) out[p * ldo + at + i * step] = v[i];
  }
}

// Rows of two-byte elements on any address: words at either end, put together from a thread's three elements.
template <bool ONE>
__global__ __launch_bounds__(kBlock) void rows_to_experts_halves_kernel(
    const uint16_t* __restrict__ x, int64_t C, int64_t ldx, const int32_t* __restrict__ places, int k,
    uint16_t* __restrict__ out, int64_t N, int64_t ldo, RowGrid grid) {
  int64_t t, at;
  if (!row_place<ONE>(grid, t, at)) return;
  const int step = ONE ? kBlock : grid.per;
  at += at / kBlock * (3 * kBlock);
  uint32_t even[4], odd[4];                      // elements 2 w and the next, 2 w + 1 and the next
  const uint16_t* row = x + t * ldx;
  const bool from_odd = (uintptr_t)row & 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c = 2 * (at + i * step);
    if (c >= C) break;
    const uint16_t* p = row + c;
    if (c + 2 >= C) {
      even[i] = p[0];
      odd[i] = c + 1 < C ? p[1] : 0;
      even[i] |= odd[i] << 16;
    } else if (from_odd) {
      odd[i] = *reinterpret_cast<const uint32_t*>(p + 1);
      even[i] = p[0] | odd[i] << 16;
    } else {
      even[i] = *reinterpret_cast<const uint32_t*>(p);
      odd[i] = even[i] >> 16 | (uint32_t)p[2] << 16;
    }
  }
  for (int j = 0; j < k; ++j) {
    const int64_t p = places[t * k + j];
    if (p < 0 || p >= N) continue;
    uint16_t* to = out + p * ldo;
    if ((uintptr_t)to & 2) {
      if (at == 0) to[0] = (uint16_t)even[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t c = 2 * (at + i * step) + 1;
        if (c + 1 < C) *reinterpret_cast<uint32_t*>(to + c) = odd[i];
        else if (c < C) to[c] = (uint16_t)odd[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t c = 2 * (at + i * step);
        if (c + 1 < C) *reinterpret_cast<uint32_t*>(to + c) = even[i];
        else if (c < C) to[c] = (uint16_t)even[i];
      }
    }
  }
}

template <int TYPE>
__device__ __forceinline__ float value_at(u32x4 w, int i) {
  if (TYPE == AAAC_F32) return __uint_as_float(w[i & 3]);
  const uint16_t b = (uint16_t)(w[(i >> 1) & 3] >> (16 * (i & 1)));
  return TYPE == AAAC_BF16 ? __uint_as_float((uint32_t)b << 16) : (float)__builtin_bit_cast(_Float16, b);
}
__device__ __forceinline__ uint32_t to_16(int type, float v) {
  return type == AAAC_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)v)
                           : __builtin_bit_cast(uint16_t, (_Float16)v);
}

// VEC: whole pieces of y and of out on their own size.
template <int TYPE, bool VEC, bool ONE>
__global__ __launch_bounds__(kBlock) void rows_from_experts_kernel(
    const uint8_t* __restrict__ y, int64_t N, int64_t C, int64_t ldy, const int32_t* __restrict__ places,
    const float* __restrict__ weights, int k, uint8_t* __restrict__ out, int out_type, int64_t ldo,
    RowGrid grid) {
  constexpr int B = TYPE == AAAC_F32 ? 4 : 2, V = 16 / B;
  int64_t t, c;
  if (!row_place<ONE>(grid, t, c)) return;
  c *= V;
  if (c >= C) return;
  const int left = C - c < V ? (int)(C - c) : V;
  float sum[V] = {};
  constexpr int U = 8;                           // rows on their way together
  for (int j0 = 0; j0 < k; j0 += U) {
    u32x4 v[U];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = u32x4{0u, 0u, 0u, 0u};
      w[u] = 0.0f;
      if (j0 + u < k) {
        const int64_t p = places[t * k + j0 + u];
        if (p >= 0 && p < N) {
          w[u] = weights[t * k + j0 + u];
          v[u] = load_piece<VEC>(y + (p * ldy + c) * B, left * B, B);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = __builtin_fmaf(w[u], value_at<TYPE>(v[u], i), sum[i]);
  }
  const int ob = out_type == AAAC_F32 ? 4 : 2;
  uint8_t* o = out + (t * ldo + c) * ob;
  if (ob == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const u32x4 w = {__float_as_uint(sum[i]), __float_as_uint(sum[i + 1]), __float_as_uint(sum[i + 2]),
                       __float_as_uint(sum[i + 3])};
      if (left > i) store_piece<VEC>(o + 4 * i, (left - i) * 4, 4, w);
    }
    return;
  }
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < V; i += 2) w[i / 2] = to_16(out_type, sum[i]) | to_16(out_type, sum[i + 1]) << 16;
  if (V == 8) {
    store_piece<VEC>(o, left * 2, 2, w);
  } else if (VEC) {
    *reinterpret_cast<u32x2*>(o) = u32x2{w.x, w.y};
  } else {
    store_piece<false>(o, left * 2, 2, w);       // eight bytes at most
  }
}

// The same for rows on four bytes, a word or its one or two columns at a time.
template <int TYPE, bool ONE>
__global__ __launch_bounds__(kBlock) void rows_from_experts_words_kernel(
    const uint32_t* __restrict__ y, int64_t N, int64_t words, int64_t ldy, const int32_t* __restrict__ places,
    const float* __restrict__ weights, int k, uint8_t* __restrict__ out, int out_type, int64_t ldo,
    RowGrid grid) {
  constexpr int V = TYPE == AAAC_F32 ? 1 : 2, W = 4, U = 8;
  int64_t t, at;
  if (!row_place<ONE>(grid, t, at)) return;
  const int step = ONE ? kBlock : grid.per;
  at += at / kBlock * ((W - 1) * kBlock);
  float sum[W][V] = {};
  for (int j0 = 0; j0 < k; j0 += U) {
    uint32_t v[U][W];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t p = j0 + u < k ? places[t * k + j0 + u] : -1;
      const bool in = p >= 0 && p < N;
      w[u] = in ? weights[t * k + j0 + u] : 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) v[u][i] = in && at + i * step < words ? y[p * ldy + at + i * step] : 0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int c = 0; c < V; ++c)
          sum[i][c] = __builtin_fmaf(w[u], value_at<TYPE>(u32x4{v[u][i], 0u, 0u, 0u}, c), sum[i][c]);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (at + i * step >= words) break;
    const int64_t c = (at + i * step) * V;
    if (out_type == AAAC_F32) {
      __builtin_memcpy(out + 4 * (t * ldo + c), sum[i], 4 * V);
    } else {
      uint32_t o = to_16(out_type, sum[i][0]);
      if (V == 2) o |= to_16(out_type, sum[i][V - 1]) << 16;
      __builtin_memcpy(out + 2 * (t * ldo + c), &o, 2 * V);
    }
  }
}

template <int TYPE, bool ONE>
hipError_t from_experts(const void* y, int64_t N, int64_t C, int64_t ldy, const int32_t* places,
                        const float* weights, int k, void* out, int out_type, int64_t ldo, const RowGrid& grid,
                        hipStream_t stream) {
  constexpr int B = TYPE == AAAC_F32 ? 4 : 2, V = 16 / B, P = 4 / B;   // bytes a column; columns of 16, of 4
  const int ob = out_type == AAAC_F32 ? 4 : 2, store = V * ob < 16 ? V * ob : 16;
  const bool vec = (uintptr_t)y % 16 == 0 && ldy % V == 0 && C % V == 0 && (uintptr_t)out % store == 0 &&
                   (ldo * ob) % store == 0;
  const bool word = (uintptr_t)y % 4 == 0 && ldy % P == 0 && C % P == 0;
  const uint8_t* in = static_cast<const uint8_t*>(y);
  uint8_t* to = static_cast<uint8_t*>(out);
  if (vec)
    hipLaunchKernelGGL((rows_from_experts_kernel<TYPE, true, ONE>), grid_of(grid.blocks), dim3(kBlock), 0,
                       stream, in, N, C, ldy, places, weights, k, to, out_type, ldo, grid);
  else if (word)
    hipLaunchKernelGGL((rows_from_experts_words_kernel<TYPE, ONE>), grid_of(grid.blocks), dim3(kBlock), 0,
                       stream, static_cast<const uint32_t*>(y), N, C / P, ldy / P, places, weights, k, to,
                       out_type, ldo, grid);
  else
    hipLaunchKernelGGL((rows_from_experts_kernel<TYPE, false, ONE>), grid_of(grid.blocks), dim3(kBlock), 0,
                       stream, in, N, C, ldy, places, weights, k, to, out_type, ldo, grid);
  return hipGetLastError();
}

template <bool ONE>
hipError_t to_experts(const void* x, int64_t bytes, int64_t ldx, const int32_t* places, int k, void* out,
                      int64_t N, int64_t ldo, int element, const RowGrid& grid, hipStream_t stream) {
  const uint64_t low = (uintptr_t)x | (uintptr_t)out | (uint64_t)bytes | (uint64_t)ldx | (uint64_t)ldo;
  const uint8_t* in = static_cast<const uint8_t*>(x);
  uint8_t* to = static_cast<uint8_t*>(out);
  if (low % 16 == 0)
    hipLaunchKernelGGL((rows_to_experts_kernel<true, ONE>), grid_of(grid.blocks), dim3(kBlock), 0, stream, in,
                       bytes, ldx, places, k, to, N, ldo, element, grid);
  else if (low % 4 == 0)
    hipLaunchKernelGGL((rows_to_experts_words_kernel<ONE>), grid_of(grid.blocks), dim3(kBlock), 0, stream,
                       static_cast<const uint32_t*>(x), bytes / 4, ldx / 4, places, k,
                       static_cast<uint32_t*>(out), N, ldo / 4, grid);
  else if (element == 2)
    hipLaunchKernelGGL((rows_to_experts_halves_kernel<ONE>), grid_of(grid.blocks), dim3(kBlock), 0, stream,
                       static_cast<const uint16_t*>(x), bytes / 2, ldx / 2, places, k,
                       static_cast<uint16_t*>(out), N, ldo / 2, grid);
  else
    hipLaunchKernelGGL((rows_to_experts_kernel<false, ONE>), grid_of(grid.blocks), dim3(kBlock), 0, stream, in,
                       bytes, ldx, places, k, to, N, ldo, element, grid);
  return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int E) {
  const int64_t per = tokens_per_block(T, E);
  return T <= per ? 0 : sizeof(int32_t) * (size_t)((T + per - 1) / per) * (size_t)count_row(E);
}

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  if (a.T == 0) {
    hipLaunchKernelGGL(no_offsets_kernel, dim3(1), dim3(kBlock), 0, stream, a.offsets, a.E + 1);
    return hipGetLastError();
  }
  a.per_block = tokens_per_block(a.T, a.E);
  const bool exact = a.bias || (a.top_groups < a.groups && a.group_top == 2);
  return exact ? route_e<true>(a, stream) : route_e<false>(a, stream);
}

hipError_t launch_rows_to_experts(const void* x, int64_t T, int64_t bytes, int64_t ldx,
                                  const int32_t* places, int k, void* out, int64_t N, int64_t ldo,
                                  int element, hipStream_t stream) {
  if (T == 0 || bytes == 0) return hipSuccess;
  const RowGrid grid = row_grid(T, (bytes + 15) / 16);
  return grid.tokens == 1 ? to_experts<true>(x, bytes, ldx, places, k, out, N, ldo, element, grid, stream)
                          : to_experts<false>(x, bytes, ldx, places, k, out, N, ldo, element, grid, stream);
}

template <int TYPE>
static hipError_t from_experts_of(const void* y, int64_t N, int64_t C, int64_t ldy, const int32_t* places,
                                  const float* weights, int64_t T, int k, void* out, int out_type,
                                  int64_t ldo, hipStream_t stream) {
  constexpr int V = TYPE == AAAC_F32 ? 4 : 8;
  const RowGrid grid = row_grid(T, (C + V - 1) / V);
  return grid.tokens == 1
             ? from_experts<TYPE, true>(y, N, C, ldy, places, weights, k, out, out_type, ldo, grid, stream)
             : from_experts<TYPE, false>(y, N, C, ldy, places, weights, k, out, out_type, ldo, grid, stream);
}

hipError_t launch_rows_from_experts(const void* y, int type, int64_t N, int64_t C, int64_t ldy,
                                    const int32_t* places, const float* weights, int64_t T, int k,
                                    void* out, int out_type, int64_t ldo, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (type == AAAC_F32)
    return from_experts_of<AAAC_F32>(y, N, C, ldy, places, weights, T, k, out, out_type, ldo, stream);
  if (type == AAAC_BF16)
    return from_experts_of<AAAC_BF16>(y, N, C, ldy, places, weights, T, k, out, out_type, ldo, stream);
  return from_experts_of<AAAC_F16>(y, N, C, ldy, places, weights, T, k, out, out_type, ldo, stream);
}

}  // namespace aaac
