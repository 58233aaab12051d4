// Routing of tokens to experts and back: the top experts of each token with their weights, the
// rows sorted by expert, the weighted sums of the experts' rows, and the gradients of both.
//
// Choosing: 16 lanes (up to 256 experts) or 64 share a token, each with 4, 8 or 16 adjacent experts'
// scores in registers; a round takes the largest score by DPP moves and, among the lanes that
// have it, the lowest, whose experts come first.  Sorting is a counting sort that keeps the
// tokens' order without an atomic whose order matters: a workgroup counts its block of tokens,
// and in a second launch each adds up the blocks before it and ranks its own entries by ballots
// over the bits of the expert's number.  One block of tokens needs one launch.
//
// All of it is short work in waves that wait: 32768 tokens to 4 of 64 (fp32) choose in 7.1 us and
// place in 6.4, where 13 MB need 2.5; to 8 of 256 (bf16) both take 28, of 512 60.  The gradient takes 5.1 us at 32768 x 64
// (bf16, 8 taken; 8 MB), 14.9 at 256 and 15.4 at 512: sums over the taken alone; where the weights are shares of all
// there is one exponential a score (5.7, 15.5 and 18.9).
#include "route.h"

#include <algorithm>

namespace i8mp {
namespace {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
// Lanes of a token: a row of 16, or the wave for more than 256 experts.  Tokens a workgroup takes at least (what its lanes
// take at a time), and workgroups at most, one for each CU.  (Whole calls, replayed: 512 tokens to 8 of 64 9.7 us with 64
// tokens a workgroup, 13.0 with 128; to 8 of 512 24 with 32 and 37 with 64.)
constexpr int route_lanes(int64_t E) { return E <= 256 ? 16 : 64; }
constexpr int64_t route_block(int64_t E) { return kRouteThreads / route_lanes(E); }
constexpr int64_t kRouteMaxBlocks = 256;
// Whether one workgroup takes all tokens, in one launch: a second costs the host 2 us.  (Replayed, one launch and two: 64
// tokens to 8 of 64 6.9 us and 9.5, 128 10.0 and 9.6, 256 17.2 and 9.7; 256 to 2 of 8 8.7 and 8.4; 64 to 8 of 128 8.8 and
// 10.7, to 8 of 256 11.3 and 13.5; 32 to 8 of 512 15.2 and 14.3.)
constexpr bool route_alone(int64_t T, int64_t E, int64_t k) {
  return E <= 64 ? T <= 256 && T * k <= 512 : T <= (E <= 256 ? 64 : 32);
}

template <int DT>
__device__ __forceinline__ float load_as_float(const void* p, int64_t i) {
  if constexpr (DT == I8MP_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  if constexpr (DT == I8MP_FP16) return (float)static_cast<const _Float16*>(p)[i];
  return static_cast<const float*>(p)[i];
}
template <int DT>
__device__ __forceinline__ void store_float(void* p, int64_t i, float v) {
  if constexpr (DT == I8MP_BF16) static_cast<__bf16*>(p)[i] = (__bf16)v;
  if constexpr (DT == I8MP_FP16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  if constexpr (DT == I8MP_FP32) static_cast<float*>(p)[i] = v;
}

// Over the 16 lanes of a DPP row (G = 16) or the wave (64); every lane gets the result.
template <int G, typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  const auto dpp = [&](int moved) { v = f(v, __int_as_float(moved)); };
  dpp(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
  dpp(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));
  dpp(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));
  dpp(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));
  if constexpr (G == 64) {  // the whole wave is here
    const auto row = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
    v = f(f(row(0), row(16)), f(row(32), row(48)));
  }
  return v;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
// For shares of a sum of sigmoids, of which the largest is that of m: sigmoid(x) / e^min(m, 0), so that the shares of
// scores far below zero, whose sigmoids fp32 does not hold, are there.  Below -700 a sigmoid is 0.
__device__ __forceinline__ float scaled_sigmoid(float x, float m) {
  return m < -700.0f ? 0.0f : m < 0.0f ? expf(x - m) / (1.0f + expf(x)) : sigmoid(x);
}

// A token's scores: lane l of its G has experts l J .. l J + J - 1.  VEC: J of them are there or none, and lie at a
// multiple of their size (of 16 bytes at most).
template <int DT, int J>
struct Lanes {
  static constexpr int kSize = DT == I8MP_FP32 ? 4 : 2, kPer = J * kSize > 16 ? 16 / kSize : J;  // elements of one load
};
template <int G, int J, int DT, bool VEC>
__device__ __forceinline__ void load_scores(const RouteArgs& a, int64_t t, int lane, float (&x)[J]) {
  typedef Lanes<DT, J> L;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = -INFINITY;
    if (lane * J < a.E) {
      typedef uint32_t words __attribute__((ext_vector_type(L::kPer * L::kSize / 4)));
      const char* p = static_cast<const char*>(a.logits) + (t * a.ld + lane * J) * L::kSize;
#pragma unroll
      for (int i = 0; i < J; i += L::kPer) {
        const words w = *reinterpret_cast<const words*>(p + i * L::kSize);
#pragma unroll
        for (int j = 0; j < L::kPer; ++j) {
          if constexpr (DT == I8MP_FP32) x[i + j] = __uint_as_float(w[j]);
          if constexpr (DT == I8MP_BF16) x[i + j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
          if constexpr (DT == I8MP_FP16) x[i + j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[j / 2] >> (16 * (j & 1))));
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane * J + j;
      x[j] = e < a.E ? load_as_float<DT>(a.logits, t * a.ld + e) : -INFINITY;
    }
  }
}

template <int J, int DT, bool VEC>
__device__ __forceinline__ void store_scores(const RouteArgs& a, void* d, int64_t at, int lane, const float (&v)[J]) {
  typedef Lanes<DT, J> L;
  if constexpr (VEC) {
    if (lane * J >= a.E) return;
    typedef uint32_t words __attribute__((ext_vector_type(L::kPer * L::kSize / 4)));
    char* p = static_cast<char*>(d) + (at + lane * J) * L::kSize;
#pragma unroll
    for (int i = 0; i < J; i += L::kPer) {
      __attribute__((aligned(16))) char buf[L::kPer * L::kSize];
#pragma unroll
      for (int j = 0; j < L::kPer; ++j) store_float<DT>(buf, j, v[i + j]);
      *reinterpret_cast<words*>(p + i * L::kSize) = *reinterpret_cast<const words*>(buf);
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane * J + j < a.E) store_float<DT>(d, at + lane * J + j, v[j]);
  }
}

// A lane's J scores, of which the best is asked for again and again: lists of four, each sorted, so that a best is among
// their firsts.  Exchanging neighbours only where the later is larger keeps equal ones in order.  (Searching 16 of them
// each round: 512 tokens to 8 of 128 21.5 us, 15.5 so and with 8 a lane; to 8 of 256 22.6 and 20.7.)
template <int J>
struct Best {
  static constexpr int kLists = J / 4;
  float v[kLists][4];
  int e[kLists][4];
  __device__ __forceinline__ void init(const float (&x)[J]) {
#pragma unroll
    for (int l = 0; l < kLists; ++l) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[l][i] = x[4 * l + i] == x[4 * l + i] ? x[4 * l + i] : -INFINITY, e[l][i] = 4 * l + i;  // NaN is never taken
      order(l, 0), order(l, 2), order(l, 1), order(l, 0), order(l, 2), order(l, 1);
    }
  }
  __device__ __forceinline__ void order(int l, int i) {
    const bool swap = v[l][i + 1] > v[l][i];
    const float a = v[l][i], b = v[l][i + 1];
    const int c = e[l][i], d = e[l][i + 1];
    v[l][i] = swap ? b : a, v[l][i + 1] = swap ? a : b;
    e[l][i] = swap ? d : c, e[l][i + 1] = swap ? c : d;
  }
  __device__ __forceinline__ float top() const {
    float t = v[0][0];
#pragma unroll
    for (int l = 1; l < kLists; ++l) t = fmaxf(t, v[l][0]);
    return t;
  }
  // The first of the scores `t`, taken away.
  __device__ __forceinline__ int pop(float t) {
    int first = 0;
    bool done = false;
#pragma unroll
    for (int l = 0; l < kLists; ++l) {
      const bool here = kLists == 1 || (!done && v[l][0] == t);
      done |= here;
      first = here ? e[l][0] : first;
#pragma unroll
      for (int i = 0; i < 3; ++i) v[l][i] = here ? v[l][i + 1] : v[l][i], e[l][i] = here ? e[l][i + 1] : e[l][i];
      v[l][3] = here ? -INFINITY : v[l][3];
    }
    return first;
  }
};

// The k choices of token t (G lanes, all of them here), written by the lanes that have them; counts in LDS.  Lane
// r % G keeps round r's score, so that exponentials and divisions are one for all rounds.
template <int G, int J>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t t, int lane, const float (&x)[J], int32_t* counts) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < J; ++j) bad |= !(x[j] < INFINITY);  // NaN, +inf
  Best<J> best;
  best.init(x);
  const int shift = (threadIdx.x & 63) & ~(G - 1);  // the group's first lane in the wave
  constexpr uint64_t kGroup = G == 64 ? ~uint64_t(0) : (uint64_t(1) << G) - 1;
  bad = (__ballot(bad) >> shift) & kGroup;
  constexpr int kKept = kRouteMaxK / G + (kRouteMaxK % G != 0);
  float m = 0.0f, kept[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) kept[i] = -INFINITY;
  for (int r = 0; r < a.k; ++r) {
    const float mine = best.top(), top = over_lanes<G>(mine, larger);
    const uint64_t who = (__ballot(mine == top) >> shift) & kGroup;
    const bool some = top > -INFINITY;
    if (r == 0) m = some ? top : 0.0f;
#pragma unroll
    for (int i = 0; i < kKept; ++i)
      if (lane + G * i == r) kept[i] = top;
    if (lane == __builtin_ctzll(who)) {
      const int e = lane * J + best.pop(top);
      a.experts[t * a.k + r] = some ? e : -1;
      if (some) atomicAdd(counts + e, 1);
    }
  }
  float s[kKept], taken = 0.0f;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    s[i] = !(kept[i] > -INFINITY) ? 0.0f
           : a.score != I8MP_SIGMOID ? expf(kept[i] - m)
           : a.normalize ? scaled_sigmoid(kept[i], m) : sigmoid(kept[i]);
    taken += s[i];
  }
  float total = 1.0f;
  if (a.normalize) {
    total = over_lanes<G>(taken, add);
  } else if (a.score == I8MP_SOFTMAX) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) sum += expf(x[j] - m);
    total = over_lanes<G>(sum, add);
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (lane + G * i < a.k) a.weights[t * a.k + lane + G * i] = bad ? NAN : s[i] > 0.0f ? s[i] / total : 0.0f;
}

// Ranks of the block's entries and where they go.  base[e]: first row of the block's entries
// for expert e; within[wave][e]: entries of a turn's waves, at most 64 each.
__device__ __forceinline__ void place_entries(const RouteArgs& a, int64_t first, int64_t n, int32_t* base, uint16_t* within) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, E = (int)a.E;  // E <= kRouteThreads
  const int bits = 32 - __builtin_clz(E);                                 // numbers 0 .. E
  for (int64_t i0 = 0; i0 < n; i0 += kRouteThreads) {
    for (int i = t; i < kRouteWaves * E; i += kRouteThreads) within[i] = 0;
    __syncthreads();
    const int64_t i = i0 + t;
    const int e = i < n ? a.experts[first + i] : -1;
    const int key = e < 0 ? E : e;
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (e >= 0 && rank == 0) within[wave * E + e] = (uint16_t)__popcll(same);
    __syncthreads();
    int32_t turn = 0;  // entries of expert t
    if (t < E) {
#pragma unroll
      for (int w = 0; w < kRouteWaves; ++w) {
        const int32_t c = within[w * E + t];
        within[w * E + t] = (uint16_t)turn;
        turn += c;
      }
    }
    __syncthreads();
    if (i < n) {
      int32_t at = -1;
      if (e >= 0) {
        at = base[e] + within[wave * E + e] + rank;
        a.rows[at] = (int32_t)((first + i) / a.k);
      }
      a.places[first + i] = at;
    }
    __syncthreads();
    if (t < E) base[t] += turn;
  }
}

// Exclusive sums of counts[0 .. E - 1] into first[0 .. E], by the first wave.
__device__ __forceinline__ void first_rows(const int32_t* counts, int32_t* first, int E) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int32_t before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int32_t c = e0 + lane < E ? counts[e0 + lane] : 0;
      int32_t s = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int32_t up = __shfl_up(s, o);
        if (lane >= o) s += up;
      }
      if (e0 + lane < E) first[e0 + lane] = before + s - c;
      before += __shfl(s, 63);
    }
    if (lane == 0) first[E] = before;
  }
}

// LDS: counts [E], first [E + 1], within [waves][E] (16 bits).
template <int G, int J, int DT, bool VEC, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void route_choose(RouteArgs a, int64_t per) {
  extern __shared__ int32_t lds[];
  const int E = (int)a.E, t = threadIdx.x;
  int32_t *counts = lds, *first = lds + E;
  uint16_t* within = reinterpret_cast<uint16_t*>(first + E + 1);
  for (int e = t; e < E; e += kRouteThreads) counts[e] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * per, n = min(per, a.T - t0);
  constexpr int kAtOnce = kRouteThreads / G;
  float x[J], next[J];
  if (t / G < n) load_scores<G, J, DT, VEC>(a, t0 + t / G, t & (G - 1), x);
  for (int64_t i = t / G; i < n; i += kAtOnce) {  // whole groups
    if (i + kAtOnce < n) load_scores<G, J, DT, VEC>(a, t0 + i + kAtOnce, t & (G - 1), next);
    choose<G, J>(a, t0 + i, t & (G - 1), x, counts);
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = next[j];
  }
  __syncthreads();
  if constexpr (!ONE) {
    for (int e = t; e < E; e += kRouteThreads) a.hist[blockIdx.x * a.E + e] = counts[e];
  } else {
    first_rows(counts, first, E);
    __threadfence_block();  // the choices, read again by other waves
    __syncthreads();
    for (int e = t; e <= E; e += kRouteThreads) a.offsets[e] = first[e];
    const int32_t used = first[E];
    __syncthreads();
    place_entries(a, 0, a.T * a.k, first, within);
    for (int64_t r = used + t; r < a.T * a.k; r += kRouteThreads) a.rows[r] = -1;
  }
}

__global__ __launch_bounds__(kRouteThreads) void route_place(RouteArgs a, int64_t per, int blocks) {
  extern __shared__ int32_t lds[];
  const int E = (int)a.E, t = threadIdx.x;
  int32_t *counts = lds, *first = lds + E, *before = first + E + 1;  // rows of the blocks before this one
  uint16_t* within = reinterpret_cast<uint16_t*>(before + E);
  for (int e = t; e < E; e += kRouteThreads) counts[e] = 0, before[e] = 0;
  __syncthreads();
  const int parts = kRouteThreads / E, e = t % E, part = t / E;  // E <= kRouteThreads
  if (part < parts) {
    int32_t all = 0, some = 0;
#pragma unroll 8
    for (int b = part; b < blocks; b += parts) {
      const int32_t c = a.hist[(int64_t)b * E + e];
      all += c;
      some += b < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(counts + e, all);
    atomicAdd(before + e, some);
  }
  __syncthreads();
  first_rows(counts, first, E);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int x = t; x <= E; x += kRouteThreads) a.offsets[x] = first[x];
  const int32_t used = first[E];
  __syncthreads();
  for (int x = t; x < E; x += kRouteThreads) first[x] += before[x];
  __syncthreads();
  const int64_t t0 = blockIdx.x * per, n = min(per, a.T - t0);
  place_entries(a, t0 * a.k, n * a.k, first, within);
  for (int64_t r = used + blockIdx.x * (int64_t)kRouteThreads + t; r < a.T * a.k; r += (int64_t)gridDim.x * kRouteThreads) a.rows[r] = -1;
}

// Gradient at a token's scores: with g the gradients of the taken weights w and S their sum,
// <g, w> = inner, softmax gives p (g - inner) (over all, or the taken alone with their w), the
// normalized sigmoid w (1 - s) (g - inner), the plain one g s (1 - s).  Lane r % G has the r-th taken expert and its
// score; what it gets goes among the lanes' adjacent scores through LDS.
template <int G, int J, int DT, bool VEC>
__global__ __launch_bounds__(256) void route_back(RouteArgs a, const int32_t* __restrict__ experts,
                                                  const float* __restrict__ dw, void* __restrict__ d, int64_t ldd, int64_t first) {
  __shared__ __attribute__((aligned(16))) float row_lds[256 / G][G * J];
  const int64_t t = first + (blockIdx.x * (int64_t)256 + threadIdx.x) / G;
  if (t >= a.T) return;  // whole groups
  const int lane = threadIdx.x & (G - 1);
  float x[J], v[J];
  constexpr int kKept = kRouteMaxK / G + (kRouteMaxK % G != 0);
  int e[kKept];
  float g[kKept], s[kKept], rest[kKept];
  bool bad = false;
  load_scores<G, J, DT, VEC>(a, t, lane, x);
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int r = lane + G * i;
    e[i] = r < a.k ? experts[t * a.k + r] : -1;
    g[i] = r < a.k ? dw[t * a.k + r] : 0.0f;
    if (e[i] >= a.E) e[i] = -1;
    s[i] = e[i] >= 0 ? load_as_float<DT>(a.logits, t * a.ld + e[i]) : -INFINITY;
  }
  const bool sig = a.score == I8MP_SIGMOID, all = !sig && !a.normalize;
  float m = -INFINITY;  // the largest score, of all or of the taken ones, which need not be the largest of all
#pragma unroll
  for (int j = 0; j < J; ++j) bad |= !(x[j] < INFINITY), m = larger(m, x[j]);
  if (!all) {
    m = s[0];
#pragma unroll
    for (int i = 1; i < kKept; ++i) m = larger(m, s[i]);
  }
  const int shift = (threadIdx.x & 63) & ~(G - 1);
  constexpr uint64_t kGroup = G == 64 ? ~uint64_t(0) : (uint64_t(1) << G) - 1;
  bad = (__ballot(bad) >> shift) & kGroup;
  m = over_lanes<G>(m, larger);
  m = m > -INFINITY ? m : 0.0f;
  if (sig) {
    // 1 - sigmoid(x) is formed from the score: 1 - s has no digits left where s is near 1 (6 % off at 16, 0 from 17 on).
    // Shares of a sum whose largest score lies below zero are formed as in scaled_sigmoid, where all scores have x < 0.
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const float z = s[i], t = expf(-fabsf(z)), q = 1.0f / (1.0f + t);
      rest[i] = z < 0.0f ? q : t * q;
      s[i] = z < 0.0f ? t * q : q;
      if (a.normalize && m < 0.0f) s[i] = m < -700.0f ? 0.0f : expf(z - m) * q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kKept; ++i) s[i] = expf(s[i] - m);
  }
  float sum = 0.0f, inner = 0.0f;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    s[i] = e[i] < 0 ? 0.0f : s[i];
    sum += s[i];
    inner += e[i] < 0 ? 0.0f : g[i] * s[i];
  }
  if (all) {
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = expf(x[j] - m), sum += v[j];
  }
  sum = over_lanes<G>(sum, add);
  inner = over_lanes<G>(inner, add);
  const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
  inner *= r;
  float* const row = row_lds[threadIdx.x / G];
#pragma unroll
  for (int j = 0; j < J; ++j) row[lane * J + j] = all ? v[j] * r * (0.0f - inner) : 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a token's lanes are one wave's, whose accesses of LDS stay in order
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    if (e[i] >= 0) row[e[i]] = sig ? (a.normalize ? (g[i] - inner) * r : g[i]) * (s[i] * rest[i]) : s[i] * r * (g[i] - inner);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int j = 0; j < J; ++j) v[j] = bad ? NAN : row[lane * J + j];
  store_scores<J, DT, VEC>(a, d, t * ldd, lane, v);
}

// ---- the weighted sums ------------------------------------------------------
//
// Bound by memory: 8192 tokens, 4 rows of 2048 each, bf16, 27 us (168 MB, 6.2 TB/s where some of them lie in the last
// level), the gradients at rows and weights 54 (302 MB, 5.6 TB/s); both from memory 95.  37 tokens 3.8 us, a launch.

// Rows are read W elements at a time: 16 bytes, or one element.
template <int DT, int W>
__device__ __forceinline__ void read_chunk(const void* p, int64_t i, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = load_as_float<DT>(p, i);
  } else if constexpr (DT == I8MP_FP32) {
    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == I8MP_BF16) {
        v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 h = __builtin_bit_cast(h2, w[j]);
        v[2 * j] = (float)h.x, v[2 * j + 1] = (float)h.y;
      }
    }
  }
}

template <int DT, int W>
__device__ __forceinline__ void write_chunk(void* p, int64_t i, const float (&v)[W]) {
  if constexpr (W == 1) {
    store_float<DT>(p, i, v[0]);
  } else if constexpr (DT == I8MP_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint16_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) store_float<DT>(h, j, v[j]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = __builtin_bit_cast(uint4, h);
  }
}

// A thread has one chunk of a token.
template <int DT, int W>
__global__ __launch_bounds__(256) void combine(CombineArgs a, int64_t chunks, int64_t first) {
  const int64_t i = first + blockIdx.x * (int64_t)256 + threadIdx.x;
  const int64_t t = i / chunks, c = (i - t * chunks) * W;
  if (t >= a.T) return;
  float s[W];
  if (a.residual) {
    read_chunk<DT, W>(a.residual, t * a.ldr + c, s);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j) s[j] = 0.0f;
  }
#pragma unroll 4
  for (int r = 0; r < a.k; ++r) {
    const int64_t at = a.places[t * a.k + r];
    if (at < 0 || at >= a.R) continue;
    const float w = a.weights ? a.weights[t * a.k + r] : 1.0f;
    float y[W];
    read_chunk<DT, W>(a.Y, at * a.ldy + c, y);
#pragma unroll
    for (int j = 0; j < W; ++j) s[j] = __builtin_fmaf(w, y[j], s[j]);
  }
  write_chunk<DT, W>(a.out, t * a.ldo + c, s);
}

// A wave has one (token, choice): its row of dY and its weight's gradient; then, with `rows`, the
// rows that nobody has, of no token or of one whose places do not name them (any more): eight a wave, of which
// eight lanes each look at a row's token (8192 tokens, 4 rows of 2048 each, with the sums: 94.5 us, 95.4 with a wave for each row).
constexpr int kFreeRows = 8;
template <int DT, int W>
__global__ __launch_bounds__(256) void combine_back(CombineArgs a, int64_t first) {
  const int64_t i = first + blockIdx.x * (int64_t)4 + (threadIdx.x >> 6), pairs = a.T * a.k;
  const int lane = threadIdx.x & 63;
  if (i < pairs) {
    const int64_t t = i / a.k, at = a.places[i];
    const bool some = at >= 0 && at < a.R;
    float dot = 0.0f;
    if (some) {
      const float w = a.weights ? a.weights[i] : 1.0f;
      for (int64_t c = lane * W; c < a.N; c += 64 * W) {
        float d[W], y[W];
        read_chunk<DT, W>(a.dout, t * a.ldd + c, d);
        if (a.dweights) {
          read_chunk<DT, W>(a.Y, at * a.ldy + c, y);
#pragma unroll
          for (int j = 0; j < W; ++j) dot = __builtin_fmaf(d[j], y[j], dot);
        }
        if (a.dY) {
#pragma unroll
          for (int j = 0; j < W; ++j) d[j] *= w;
          write_chunk<DT, W>(a.dY, at * a.ldg + c, d);
        }
      }
    }
    if (a.dweights) {
      dot = over_lanes<64>(dot, add);
      if (lane == 0) a.dweights[i] = dot;
    }
  } else if (a.rows && a.dY) {
    constexpr int kLook = 64 / kFreeRows;
    const int64_t r0 = (i - pairs) * kFreeRows, r = r0 + lane / kLook;
    const int64_t t = r < a.R ? a.rows[r] : -1;
    bool named = r >= a.R;
    if (t >= 0 && t < a.T)
      for (int j = lane % kLook; j < a.k; j += kLook) named |= a.places[t * a.k + j] == r;
    const uint64_t who = __ballot(named);
    float z[W];
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] = 0.0f;
    for (int n = 0; n < kFreeRows; ++n) {
      if (who >> (kLook * n) & ((1 << kLook) - 1)) continue;
      for (int64_t c = lane * W; c < a.N; c += 64 * W) write_chunk<DT, W>(a.dY, (r0 + n) * a.ldg + c, z);
    }
  }
}

template <int G, int J, int DT, bool VEC>
void choose_blocks(const RouteArgs& a, int64_t per, int blocks, hipStream_t stream) {
  const size_t small = (size_t)(2 * a.E + 1) * 4, ranks = (size_t)kRouteWaves * a.E * 2;
  if (blocks == 1) {
    route_choose<G, J, DT, VEC, true><<<1, kRouteThreads, small + ranks, stream>>>(a, per);
  } else {
    route_choose<G, J, DT, VEC, false><<<(unsigned)blocks, kRouteThreads, small, stream>>>(a, per);
    route_place<<<(unsigned)blocks, kRouteThreads, small + (size_t)a.E * 4 + ranks, stream>>>(a, per, blocks);
  }
}

// Whether a lane's J scores of a matrix can be moved at once.
template <int DT, int J>
bool whole_lanes(const RouteArgs& a, const void* p, int64_t ld) {
  typedef Lanes<DT, J> L;
  constexpr int64_t kBytes = L::kPer * L::kSize;
  return a.E % J == 0 && (reinterpret_cast<uintptr_t>(p) % kBytes) == 0 && ld * L::kSize % kBytes == 0;
}

template <int G, int J, int DT>
void choose_lanes(const RouteArgs& a, int64_t per, int blocks, hipStream_t stream) {
  if (whole_lanes<DT, J>(a, a.logits, a.ld))
    choose_blocks<G, J, DT, true>(a, per, blocks, stream);
  else
    choose_blocks<G, J, DT, false>(a, per, blocks, stream);
}

template <int DT>
void route_as(const RouteArgs& a, int64_t per, int blocks, hipStream_t stream) {
  if (a.E <= 64)
    choose_lanes<16, 4, DT>(a, per, blocks, stream);
  else if (a.E <= 128)
    choose_lanes<16, 8, DT>(a, per, blocks, stream);
  else if (a.E <= 256)
    choose_lanes<16, 16, DT>(a, per, blocks, stream);
  else if (a.E <= 512)
    choose_lanes<64, 8, DT>(a, per, blocks, stream);
  else
    choose_lanes<64, 16, DT>(a, per, blocks, stream);
}

constexpr int64_t kMaxGrid = int64_t(1) << 23;  // workgroups of 256: fewer than 2^32 work items

template <int G, int J, int DT>
void route_back_lanes(const RouteArgs& a, const int32_t* experts, const float* dw, void* d, int64_t ldd, hipStream_t stream) {
  constexpr int64_t kTokens = 256 / G;  // of a workgroup
  const int64_t n = (a.T + kTokens - 1) / kTokens;
  const bool vec = whole_lanes<DT, J>(a, a.logits, a.ld) && whole_lanes<DT, J>(a, d, ldd);
  for (int64_t b = 0; b < n; b += kMaxGrid) {
    const unsigned grid = (unsigned)std::min(kMaxGrid, n - b);
    if (vec)
      route_back<G, J, DT, true><<<grid, 256, 0, stream>>>(a, experts, dw, d, ldd, b * kTokens);
    else
      route_back<G, J, DT, false><<<grid, 256, 0, stream>>>(a, experts, dw, d, ldd, b * kTokens);
  }
}

template <int DT>
void route_back_as(const RouteArgs& a, const int32_t* experts, const float* dw, void* d, int64_t ldd, hipStream_t stream) {
  if (a.E <= 64)
    route_back_lanes<16, 4, DT>(a, experts, dw, d, ldd, stream);
  else if (a.E <= 128)
    route_back_lanes<16, 8, DT>(a, experts, dw, d, ldd, stream);
  else if (a.E <= 256)
    route_back_lanes<16, 16, DT>(a, experts, dw, d, ldd, stream);
  else if (a.E <= 512)
    route_back_lanes<64, 8, DT>(a, experts, dw, d, ldd, stream);
  else
    route_back_lanes<64, 16, DT>(a, experts, dw, d, ldd, stream);
}

template <int DT, int W>
void combine_as(const CombineArgs& a, hipStream_t stream) {
  const int64_t chunks = (a.N + W - 1) / W, n = (a.T * chunks + 255) / 256;
  for (int64_t b = 0; b < n; b += kMaxGrid)
    combine<DT, W><<<(unsigned)std::min(kMaxGrid, n - b), 256, 0, stream>>>(a, chunks, b * 256);
}

template <int DT, int W>
void combine_back_as(const CombineArgs& a, hipStream_t stream) {
  const int64_t n = (a.T * a.k + (a.rows && a.dY ? (a.R + kFreeRows - 1) / kFreeRows : 0) + 3) / 4;
  for (int64_t b = 0; b < n; b += kMaxGrid)
    combine_back<DT, W><<<(unsigned)std::min(kMaxGrid, n - b), 256, 0, stream>>>(a, b * 4);
}

}  // namespace

int64_t route_block_tokens(int64_t T, int64_t E, int64_t k) {
  if (route_alone(T, E, k)) return std::max<int64_t>(T, 1);
  return std::max(route_block(E), (T + kRouteMaxBlocks - 1) / kRouteMaxBlocks);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  const int64_t per = route_block_tokens(a.T, a.E, a.k);
  const int blocks = (int)std::max<int64_t>(1, (a.T + per - 1) / per);
  switch (a.dtype) {
    case I8MP_BF16: route_as<I8MP_BF16>(a, per, blocks, stream); break;
    case I8MP_FP16: route_as<I8MP_FP16>(a, per, blocks, stream); break;
    default: route_as<I8MP_FP32>(a, per, blocks, stream);
  }
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteArgs& a, const int32_t* experts, const float* dw, void* d, int64_t ldd, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  switch (a.dtype) {
    case I8MP_BF16: route_back_as<I8MP_BF16>(a, experts, dw, d, ldd, stream); break;
    case I8MP_FP16: route_back_as<I8MP_FP16>(a, experts, dw, d, ldd, stream); break;
    default: route_back_as<I8MP_FP32>(a, experts, dw, d, ldd, stream);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  switch (2 * a.dtype + a.vec) {
    case 2 * I8MP_BF16 + 1: combine_as<I8MP_BF16, 8>(a, stream); break;
    case 2 * I8MP_BF16: combine_as<I8MP_BF16, 1>(a, stream); break;
    case 2 * I8MP_FP16 + 1: combine_as<I8MP_FP16, 8>(a, stream); break;
    case 2 * I8MP_FP16: combine_as<I8MP_FP16, 1>(a, stream); break;
    case 2 * I8MP_FP32 + 1: combine_as<I8MP_FP32, 4>(a, stream); break;
    default: combine_as<I8MP_FP32, 1>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineArgs& a, hipStream_t stream) {
  switch (2 * a.dtype + a.vec) {
    case 2 * I8MP_BF16 + 1: combine_back_as<I8MP_BF16, 8>(a, stream); break;
    case 2 * I8MP_BF16: combine_back_as<I8MP_BF16, 1>(a, stream); break;
    case 2 * I8MP_FP16 + 1: combine_back_as<I8MP_FP16, 8>(a, stream); break;
    case 2 * I8MP_FP16: combine_back_as<I8MP_FP16, 1>(a, stream); break;
    case 2 * I8MP_FP32 + 1: combine_back_as<I8MP_FP32, 4>(a, stream); break;
    default: combine_back_as<I8MP_FP32, 1>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace i8mp
