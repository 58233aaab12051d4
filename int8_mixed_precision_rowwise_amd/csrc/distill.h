// Loss of a student's logits against a teacher's kept top logits, and its
// gradient: kernels, templated on the logits' type (distill_bf16.hip,
// distill_fp16.hip and distill_fp32.hip instantiate them).
//
// For one row x of V logits, temperature tau, kept entries j with logits t_j:
//   q = softmax(x / tau),  p_j = exp(t_j / tau - z)
// z = log sum_j exp(t_j / tau), or the whole teacher's log-sum-exp, when the
// mass p_rest = max(0, 1 - sum p_j) that is left is one more class, whose
// student is q_rest = sum of q over the entries not kept;
//   loss = tau^2 [sum_j p_j log(p_j / q_j) + p_rest log(p_rest / q_rest)]
//          + ce (log sum exp(x) - x_label)
//   dx_i = g tau [mass q_i - p_i]                     (i kept; mass = sum p_j + p_rest)
//        = g tau q_i [mass - p_rest / q_rest]         (i not kept)
//          + g ce (softmax(x)_i - [i = label]).
//
// A step has to read every logit and write every gradient once, and nothing
// else of size: it is bound by memory as long as a row is read once.  So one
// workgroup holds a whole row in registers between the sums and the gradient
// (a row of 131064 16-bit logits is half a CU's registers).  The sums are taken
// while the row arrives, each thread rescaling its own to the maximum it has seen
// so far; the kept entries are left out of them (a byte a chunk in LDS tells which
// elements they are) and are evaluated one per thread in 64 bits, which keeps
// q_rest and mass q_j - p_j free of cancellation.
//
// The other entries' sums are relative to the maximum of those entries, mo, and only
// joined in 64 bits with the kept ones, which are relative to the row's maximum m:
// where the kept logits stand 88 tau and more above the rest, fp32 sums relative to m
// would be 0 and p_rest / q_rest infinite.  With e' = exp((x - mo) / tau), S' their
// sum and S = S' exp((mo - m) / tau) + the kept entries' sum, the gradient outside is
//   g tau e'_i [mass exp((mo - m) / tau) / S - p_rest / S'],
// every factor of which is in range.  Rest entries that are all -inf have e' = 0.
//
// Measured: loss and gradient of 4096 x 128256 bf16 logits, temperature 2 with hard
// labels, 520 - 525 us in calls one after another for 2.1 GB, 4.0 TB/s where a copy of that
// size reaches 5.1 (the kernel alone under the profiler 537 - 590, 553 on average).  Two
// exponentials an element at a quarter of the vector rate and some 13 other operations
// are about 240 us of every CU's time; a row of this length fills a CU, so they
// overlap with memory only as far as the CUs are at different places of their rows.  Loss of
// 2000 x 32000 fp32 51 us (5.0 TB/s); loss, then gradient, of 1021 x 32003 fp16 26 and
// 27 us; three rows of 128256 in segments 4.5 and 8.7 us, bound by one load waiting
// for the other.
//
// Rows too long for that, and calls with too few rows to fill the chip, take
// two launches over (segment, row): partial sums, then the gradient with each
// workgroup joining its row's partial sums itself.  The gradient alone (the
// backward of an earlier forward) is the second of them with the sums given.
//
// Exponentials are 2^(c x - R), one fused operation, with c = log2(e) / tau and R =
// c mo (c m for the kept entries) rounded to fp32.  The same c and R stand in the
// 64-bit part: the rounding of c only scales the temperature by 2^-24, and that of
// each R cancels, as the two are joined by their exact difference.  Beyond |R| = 2^22 (a
// row masked with the type's lowest value) the rounding of R is no longer small
// against its terms: such a row is summed and swept once more from memory as
// 2^(c (x - mo)).  fp32 logits take x - mo first and carry the product's low part.
#pragma once

#include "internal.h"

#include <algorithm>
#include <utility>

namespace i8mp {
namespace distill {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;

// What a row's gradient needs besides its logits and kept entries.
struct RowStats {
  double ref;      // the maximum m of the logits (0 if all are -inf)
  double ref_out;  // the maximum mo of those not kept (0 if all are -inf)
  double kept;     // mass / S, S the sum of the exponentials (2^(c x - R), see Expo) relative to m
  double kept1;    // 1 / S at temperature 1
  double outside;  // mass exp((mo - m) / tau) / S - p_rest / (sum outside, relative to mo)
  double outside1; // exp(mo - m) / S at temperature 1
  double z;        // p_j = exp(t_j / tau - z)
  double spare;
};
static_assert(sizeof(RowStats) == 8 * I8MP_DISTILL_STATS, "one row of the caller's statistics");

struct Partial {  // sums of one segment without its kept entries, relative to its own maximum
  float max, sum, sum1;
  float pad;
};

// One LDS-only workgroup barrier: loads in flight from memory stay in flight.
__device__ __forceinline__ void lds_sync() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float uniform(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); }

// The row's element type: 16-byte chunks of E elements.
template <typename T>
struct Elem;
template <>
struct Elem<__bf16> {
  static constexpr int E = 8;
  static constexpr uint32_t kNegInf = 0xFF80u;
  static __device__ __forceinline__ uint32_t bits(const __bf16* p) { return *reinterpret_cast<const uint16_t*>(p); }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
  static __device__ __forceinline__ float get(const v4i& v, int e) {
    const uint32_t w = (uint32_t)v[e >> 1];
    return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};
template <>
struct Elem<_Float16> {
  static constexpr int E = 8;
  static constexpr uint32_t kNegInf = 0xFC00u;
  static __device__ __forceinline__ uint32_t bits(const _Float16* p) { return *reinterpret_cast<const uint16_t*>(p); }
  static __device__ __forceinline__ float value(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (unsigned short)b); }
  static __device__ __forceinline__ float get(const v4i& v, int e) {
    const uint32_t w = (uint32_t)v[e >> 1];
    return (float)__builtin_bit_cast(_Float16, (unsigned short)((e & 1) ? (w >> 16) : (w & 0xFFFFu)));
  }
};
template <>
struct Elem<float> {
  static constexpr int E = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ __forceinline__ uint32_t bits(const float* p) { return *reinterpret_cast<const uint32_t*>(p); }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b); }
  static __device__ __forceinline__ float get(const v4i& v, int e) { return __uint_as_float((uint32_t)v[e]); }
};

// Elements whose bit is set in mask become -inf.
template <typename T>
__device__ __forceinline__ void drop(v4i& v, uint32_t mask) {
  constexpr uint32_t inf = Elem<T>::kNegInf;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (Elem<T>::E == 4) {
      v[w] = mask >> w & 1 ? (int)inf : v[w];
    } else {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_sbfe((int)mask, 2 * w, 1), hi = (uint32_t)__builtin_amdgcn_sbfe((int)mask, 2 * w + 1, 1);
      const uint32_t m = (lo & 0xFFFFu) | (hi << 16);
      v[w] = (int)(((uint32_t)v[w] & ~m) | ((inf | inf << 16) & m));
    }
  }
}

// A row as 16-byte chunks of memory: chunk c holds elements c E - shift ...;
// elements before the row and behind it (in its first and last chunk) are
// read as -inf and never written.
template <typename T>
struct Row {
  const v4i* chunks;
  int shift;    // elements of the first chunk that lie before the row
  int nchunks;
  int V;
  __device__ __forceinline__ Row(const void* base, int64_t row, int64_t ld, int V_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(base) + (uintptr_t)(row * ld) * sizeof(T);
    chunks = reinterpret_cast<const v4i*>(a & ~(uintptr_t)15);
    shift = (int)(a & 15) / (int)sizeof(T);
    V = V_;
    nchunks = (V + shift + Elem<T>::E - 1) / Elem<T>::E;
  }
  // Elements of chunk c outside the row.
  __device__ __forceinline__ uint32_t outside(int c) const {
    constexpr int E = Elem<T>::E;
    uint32_t m = 0;
    if (c == 0) m = (1u << shift) - 1;
    const int left = V + shift - c * E;  // elements up to the row's end
    if (left < E) m |= ~0u << (left > 0 ? left : 0);
    return m;
  }
  __device__ __forceinline__ v4i load(int c) const {
    v4i v = chunks[c];
    if (c == 0 || c == nchunks - 1) drop<T>(v, outside(c));
    return v;
  }
};

// The chunks of a row held in registers, through a buffer descriptor of just
// that row: chunks past its end are read as zeros and their writes are dropped,
// with no branch around the access.  (A branch that may skip a load makes the
// compiler wait for every access in flight where it needs only an older one.)
struct RowBuffer {
  __amdgpu_buffer_rsrc_t rsrc;
  __device__ __forceinline__ RowBuffer(const void* p, int chunks)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, chunks * 16, 0x00020000)) {}
  // chunk `first` (the same in every lane) + t
  __device__ __forceinline__ v4i load(int first, int t) const {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc, t * 16, first * 16, 0));
  }
  __device__ __forceinline__ void store(int first, int t, v4i v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), rsrc, t * 16, first * 16, 2);  // non-temporal
  }
};

__device__ __forceinline__ v4i all_neg_inf(int elem_bytes, uint32_t inf) {
  const int w = elem_bytes == 4 ? (int)inf : (int)(inf | (inf << 16));
  return (v4i){w, w, w, w};
}

// Exponentials of a row: in its sweeps relative to the entries that are not kept,
// of kept entries in 64 bits relative to the whole row.  MODE 0: one temperature
// (no hard labels, or tau = 1); 1: tau = 2, exp(x) as the square; 2: two.
template <typename T, int MODE>
struct Expo {
  static constexpr bool kPrecise = sizeof(T) == 4;
  static constexpr float kFar = 0x1p22f;
  float c, c_lo, c1, c1_lo;  // log2(e) / tau and log2(e), with their low parts
  float m, r, r1;            // the sweep's maximum, R, and R at temperature 1
  float mk, rk, rk1;         // the same of the row
  bool rest;                 // the entries not kept are a class
  __device__ __forceinline__ Expo(const DistillArgs& a)
      : c(a.c), c_lo(a.c_lo), c1(a.c1), c1_lo(a.c1_lo), m(0), r(0), r1(0), mk(0), rk(0), rk1(0), rest(a.lse != nullptr) {}
  // A maximum so far.  The bound keeps R finite where everything is -inf or close to
  // the type's lowest value: exponentials there are 0.
  __device__ __forceinline__ void at(float max) {
    if constexpr (kPrecise) {
      m = max == -__builtin_inff() ? 0.0f : max;
    } else {
      r = fmaxf(c * max, -kFar);
      if constexpr (MODE == 2) r1 = fmaxf(c1 * max, -kFar);
    }
  }
  // The maxima of a row's entries that are not kept, and of all.
  __device__ __forceinline__ void at_row(float out, float all) {
    at(out);
    m = out == -__builtin_inff() ? 0.0f : out;
    mk = all == -__builtin_inff() ? 0.0f : all;
    rk = fmaxf(c * mk, -kFar);
    if constexpr (MODE == 2) rk1 = fmaxf(c1 * mk, -kFar);
  }
  // One value for all lanes: scalar registers.
  __device__ __forceinline__ void uniform_all() {
    m = uniform(m), r = uniform(r), r1 = uniform(r1), mk = uniform(mk), rk = uniform(rk), rk1 = uniform(rk1);
  }
  // Where the entries not kept are no class of their own, a maximum of theirs below the
  // bound does not matter: next to the row's they are then 0.
  __device__ __forceinline__ bool far() const {
    return !kPrecise && (__builtin_fabsf(c * mk) >= kFar || (MODE == 2 && __builtin_fabsf(c1 * mk) >= kFar) || (rest && c * m <= -kFar));
  }
  __device__ __forceinline__ static float precise(float y, float c, float c_lo) {
    const float h = y * c;
    const float l = __builtin_fmaf(y, c_lo, __builtin_fmaf(y, c, -h));
    const float e = exp2_fast(h);
    // y = -inf: h is -inf and l a NaN
    return h < -150.0f ? 0.0f : __builtin_fmaf(e, l * (float)kLn2, e);
  }
  // exp(x / tau) and, given that, exp(x), relative to the reference
  __device__ __forceinline__ float e(float x) const {
    if constexpr (kPrecise) return precise(x - m, c, c_lo);
    else return exp2_fast(__builtin_fmaf(x, c, -r));
  }
  __device__ __forceinline__ float e1(float x, float e) const {
    if constexpr (MODE == 1) return e * e;
    if constexpr (kPrecise) return precise(x - m, c1, c1_lo);
    else return exp2_fast(__builtin_fmaf(x, c1, -r1));
  }
  // the same for a row far out
  __device__ __forceinline__ float far_e(float x) const { return exp2_fast((x - m) * c); }
  __device__ __forceinline__ float far_e1(float x, float e) const { return MODE == 1 ? e * e : exp2_fast((x - m) * c1); }
  // log2 of the same exponentials relative to the whole row, in 64 bits
  __device__ __forceinline__ double log2e(double x, const DistillArgs& a) const {
    return kPrecise || far() ? (x - (double)mk) * a.cd : x * (double)c - (double)rk;
  }
  __device__ __forceinline__ double log2e1(double x, const DistillArgs& a) const {
    if constexpr (MODE == 0) return log2e(x, a);
    if constexpr (MODE == 1) return 2 * log2e(x, a);
    return kPrecise || far() ? (x - (double)mk) * kLog2e : x * (double)c1 - (double)rk1;
  }
  // log2 of what takes the sweep's exponentials there
  __device__ __forceinline__ double gap(const DistillArgs& a) const {
    return kPrecise || far() ? ((double)m - (double)mk) * a.cd : (double)r - (double)rk;
  }
  __device__ __forceinline__ double gap1(const DistillArgs& a) const {
    if constexpr (MODE == 0) return gap(a);
    if constexpr (MODE == 1) return 2 * gap(a);
    return kPrecise || far() ? ((double)m - (double)mk) * kLog2e : (double)r1 - (double)rk1;
  }
};

// 2^y in 64 bits: the Taylor polynomial of degree 10 of exp on |z| <= ln(2) / 2
// is off by less than 1e-12 relative, far inside what the sums' fp32 part has.
__device__ __forceinline__ double exp2_d(double y) {
  const double n = __builtin_rint(y), z = (y - n) * kLn2;
  double p = 1.0 / 3628800;
  p = __builtin_fma(p, z, 1.0 / 362880);
  p = __builtin_fma(p, z, 1.0 / 40320);
  p = __builtin_fma(p, z, 1.0 / 5040);
  p = __builtin_fma(p, z, 1.0 / 720);
  p = __builtin_fma(p, z, 1.0 / 120);
  p = __builtin_fma(p, z, 1.0 / 24);
  p = __builtin_fma(p, z, 1.0 / 6);
  p = __builtin_fma(p, z, 0.5);
  p = __builtin_fma(p, z, 1.0);
  p = __builtin_fma(p, z, 1.0);
  // -inf (where the polynomial is a NaN) and what underflows give 0; beyond the range: infinity
  return y < -1100 ? 0 : y > 1100 ? (double)__builtin_inff() : __builtin_amdgcn_ldexp(p, (int)n);
}
// 2^y within a few 2^-24 where fp32 holds it, 0 below: for y <= 0 whose power only adds to larger numbers.
__device__ __forceinline__ double exp2_f(double y) {
  const float h = (float)y, e = exp2_fast(h);
  return h < -150.0f ? 0.0 : (double)__builtin_fmaf(e, (float)(y - (double)h) * (float)kLn2, e);
}

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}

// Both at once: one after the other they would wait twice.
__device__ __forceinline__ void wave_max2(float& a, float& b) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const float x = __shfl_xor(a, off), y = __shfl_xor(b, off);
    a = fmaxf(a, x), b = fmaxf(b, y);
  }
}

__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t row, int j) {
  const int64_t at = row * a.t_ld + j;
  switch (a.t_dtype) {
    case I8MP_BF16: return __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.teacher)[at] << 16);
    case I8MP_FP16: return (float)static_cast<const _Float16*>(a.teacher)[at];
    default: return static_cast<const float*>(a.teacher)[at];
  }
}

// The class of kept entry j of a row, or -1 (also for classes the vocabulary does not have).
__device__ __forceinline__ int kept_at(const DistillArgs& a, int64_t row, int j) {
  const int64_t at = row * a.i_ld + j;
  const int64_t i = a.idx64 ? static_cast<const int64_t*>(a.idx)[at] : (int64_t) static_cast<const int32_t*>(a.idx)[at];
  return i >= 0 && i < a.V ? (int)i : -1;
}
__device__ __forceinline__ int label_at(const DistillArgs& a, int64_t row) {
  if (!a.labels) return -1;
  const int64_t i = a.lab64 ? static_cast<const int64_t*>(a.labels)[row] : (int64_t) static_cast<const int32_t*>(a.labels)[row];
  return i != a.ignore && i >= 0 && i < a.V ? (int)i : -1;
}

// The same for the row kernels, in two steps: the loads, of which none waits for
// another, and what they give.
struct RawIndex {
  uint32_t lo, hi;
  __device__ __forceinline__ void load(const void* p, int64_t at, bool wide) {
    const uint32_t* w = static_cast<const uint32_t*>(p);
    lo = w[wide ? 2 * at : at];
    hi = w[wide ? 2 * at + 1 : at];
  }
  // the class, or -1
  __device__ __forceinline__ int index(const DistillArgs& a, bool wide) const {
    return lo < (uint32_t)a.V && (!wide || hi == 0) ? (int)lo : -1;
  }
  __device__ __forceinline__ int64_t value(bool wide) const {
    return wide ? (int64_t)((uint64_t)hi << 32 | lo) : (int64_t)(int32_t)lo;
  }
};
__device__ __forceinline__ uint32_t teacher_bits(const DistillArgs& a, int64_t at) {
  return a.t_dtype == I8MP_FP32 ? static_cast<const uint32_t*>(a.teacher)[at] : (uint32_t) static_cast<const uint16_t*>(a.teacher)[at];
}
__device__ __forceinline__ float teacher_value(const DistillArgs& a, uint32_t bits) {
  switch (a.t_dtype) {
    case I8MP_BF16: return __uint_as_float(bits << 16);
    case I8MP_FP16: return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
    default: return __uint_as_float(bits);
  }
}

// What the joined sums of a row give: the loss and the statistics.
// sums over kept entries: W = sum w_j, A = sum w_j (ln w_j - ln e_j), e and e1;
// w_j = exp(t_j / tau - zref), kept: how many there are.
struct Joined {
  double out, out1;  // sums over the entries not kept, relative to their maximum
  double W, A, e, e1;
  double zref;
  int kept;
};
struct Totals {
  RowStats st;          // but for z
  double total, total1; // S, at both temperatures
  double p_rest;
};
template <typename T, int MODE>
__device__ __forceinline__ Totals join(const DistillArgs& a, const Joined& s, const Expo<T, MODE>& ex) {
  Totals r;
  // nothing outside: whatever the factors, they meet exponentials of 0
  const double g = s.out == 0 ? 0 : exp2_f(ex.gap(a)), g1 = MODE == 0 ? g : s.out == 0 ? 0 : exp2_f(ex.gap1(a));
  r.total = s.out * g + s.e;
  r.total1 = MODE == 0 ? r.total : s.out1 * g1 + s.e1;
  r.p_rest = !a.lse || s.W >= 1 || s.kept == 0 ? 0 : 1 - s.W;  // a NaN stays one
  const double i = 1 / r.total, i1 = MODE == 0 ? i : 1 / r.total1, rest = r.p_rest == 0 || s.out == 0 ? 0 : r.p_rest / s.out;
  RowStats& st = r.st;
  st.ref = (double)ex.mk, st.ref_out = (double)ex.m;
  st.kept1 = i1, st.outside1 = g1 * i1;
  st.kept = st.outside = st.z = st.spare = 0;
  if (s.kept != 0) {
    st.kept = a.lse ? (s.W + r.p_rest) * i : i;
    st.outside = st.kept * g - rest;
  }
  return r;
}
// A row's loss and statistics, by the 64 lanes of one wave: its five logarithms at
// once, a lane each (one after the other they took 2 us behind every row).
// gap: log2 of what takes s.out to the row's reference.
__device__ __forceinline__ void write_row(const DistillArgs& a, int64_t row, const Joined& s, Totals r, double gap,
                                          double label_log2e1, bool has_label) {
  const int lane = threadIdx.x & 63;
  const double p_rest = r.p_rest;
  const double of = lane == 0 ? r.total : lane == 1 ? s.W : lane == 2 ? p_rest : lane == 3 ? s.out : r.total1;
  const double ln = log(of);
  const double ln_total = __shfl(ln, 0), ln_w = __shfl(ln, 1), ln_rest = __shfl(ln, 2), ln_out = __shfl(ln, 3), ln_total1 = __shfl(ln, 4);
  if (lane != 0) return;
  double loss = 0;
  if (s.kept > 0) {
    if (a.lse) {
      loss = s.A + s.W * ln_total;
      if (!(p_rest == 0)) loss += p_rest * (ln_rest - (ln_out + gap * kLn2) + ln_total);
    } else {
      loss = s.A / s.W - ln_w + ln_total;
    }
    loss *= (double)a.tau * (double)a.tau;
  }
  if (has_label) loss += (double)a.ce * (ln_total1 - label_log2e1 * kLn2);
  if (a.loss) a.loss[row] = (float)loss;
  if (a.stats) {
    r.st.z = s.kept == 0 ? 0 : a.lse ? s.zref : s.zref + ln_w;  // p_j = exp(t_j / tau - z)
    static_cast<RowStats*>(a.stats)[row] = r.st;
  }
}

// The gradient's factors of a row, formed in 64 bits.
struct Factors {
  float out, out1;    // not kept: out * e + out1 * e1
  float kept, p, c1;  // kept: kept * e_j + c1 * e1_j - p * w_j
  float label;        // subtracted at the label
};
// w_scale: p_j = w_scale * w_j for the w_j in the slots.
__device__ __forceinline__ Factors factors(const DistillArgs& a, const RowStats& st, double w_scale, int64_t row, bool has_label,
                                           int mode) {
  const double g = (double)a.grad[row * a.grad_s], gt = g * (double)a.tau;
  const double label = has_label ? g * (double)a.ce : 0, out = gt * st.outside, out1 = has_label ? label * st.outside1 : 0;
  Factors f;
  f.label = (float)label;
  f.c1 = has_label ? (float)(label * st.kept1) : 0.0f;
  f.out1 = (float)out1;
  f.kept = (float)(gt * st.kept);
  f.p = (float)(gt * w_scale);
  f.out = (float)(mode == 0 ? out + out1 : out);
  return f;
}
__device__ __forceinline__ Factors uniform(const Factors& f) {
  return {uniform(f.out), uniform(f.out1), uniform(f.kept), uniform(f.p), uniform(f.c1), uniform(f.label)};
}

template <typename T, int MODE>
__device__ __forceinline__ float outside_grad(const Expo<T, MODE>& ex, const Factors& f, float x) {
  const float e = ex.e(x);
  if constexpr (MODE == 0) return e * f.out;
  if constexpr (MODE == 1) return e * __builtin_fmaf(e, f.out1, f.out);
  return __builtin_fmaf(ex.e1(x, e), f.out1, e * f.out);
}
template <typename T, int MODE>
__device__ __forceinline__ float far_outside_grad(const Expo<T, MODE>& ex, const Factors& f, float x) {
  const float e = ex.far_e(x);
  if constexpr (MODE == 0) return e * f.out;
  return __builtin_fmaf(ex.far_e1(x, e), f.out1, e * f.out);
}

// A byte for each chunk in LDS: the elements that are kept entries.
__device__ __forceinline__ void mark(uint32_t* table, int chunk, int elem) {
  atomicOr(table + (chunk >> 2), 1u << (8 * (chunk & 3) + elem));
}
__device__ __forceinline__ uint32_t marked(const uint32_t* table, int chunk) {
  return reinterpret_cast<const uint8_t*>(table)[chunk];
}

template <typename T, int MODE, bool FAR = false>
__device__ __forceinline__ v4i grad_chunk(const Expo<T, MODE>& ex, const Factors& f, v4i v) {
  constexpr int E = Elem<T>::E;
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef T t2 __attribute__((ext_vector_type(2)));
  struct __attribute__((aligned(16))) Out { t2 p[E / 2]; } o;
#pragma unroll
  for (int e = 0; e < E; e += 2) {  // pairs: one conversion instruction for both
    const float x0 = Elem<T>::get(v, e), x1 = Elem<T>::get(v, e + 1);
    f2 y;
    if constexpr (FAR) y = {far_outside_grad<T, MODE>(ex, f, x0), far_outside_grad<T, MODE>(ex, f, x1)};
    else y = {outside_grad<T, MODE>(ex, f, x0), outside_grad<T, MODE>(ex, f, x1)};
    o.p[e / 2] = __builtin_convertvector(y, t2);
  }
  return __builtin_bit_cast(v4i, o);
}
// The gradient at a label that is no kept entry.
template <typename T, int MODE>
__device__ __forceinline__ float label_grad(const Expo<T, MODE>& ex, const Factors& f, float x) {
  return (ex.far() ? far_outside_grad<T, MODE>(ex, f, x) : outside_grad<T, MODE>(ex, f, x)) - f.label;
}
// A kept entry's gradient; x, x1, w: its exp((x - m) / tau), exp(x - m) and w_j.
__device__ __forceinline__ float kept_grad(const Factors& f, float e, float e1, float w, bool is_label) {
  float value = __builtin_fmaf(f.kept, e, -(f.p * w));
  if (f.label != 0) value += __builtin_fmaf(f.c1, e1, is_label ? -f.label : 0.0f);
  return value;
}

// The elements of chunk c that lie in the row, one by one.
template <typename T>
__device__ __forceinline__ void store_elements(const Row<T>& row, v4i v, int c, T* __restrict__ d) {
  constexpr int E = Elem<T>::E, BITS = 8 * sizeof(T);
  T* at = d + (int64_t)c * E - row.shift;
  const uint32_t skip = row.outside(c);
#pragma unroll 1
  for (int e = 0; e < E; ++e) {  // rolled: it stands behind every chunk's store and hardly ever runs
    if (!(skip >> e & 1)) {
      if constexpr (E == 4) at[e] = __uint_as_float((uint32_t)v[0]);
      else at[e] = __builtin_bit_cast(T, (unsigned short)v[0]);
    }
    v[0] = (int)__builtin_amdgcn_alignbit((uint32_t)v[1], (uint32_t)v[0], BITS & 31);
    v[1] = (int)__builtin_amdgcn_alignbit((uint32_t)v[2], (uint32_t)v[1], BITS & 31);
    v[2] = (int)__builtin_amdgcn_alignbit((uint32_t)v[3], (uint32_t)v[2], BITS & 31);
    v[3] = (int)((uint32_t)v[3] >> (BITS & 31));
    if constexpr (E == 4) v = (v4i){v[1], v[2], v[3], 0};
  }
}
template <typename T>
__device__ __forceinline__ void store_chunk(const Row<T>& row, const DistillArgs& a, v4i v, int c, T* __restrict__ d) {
  if (a.d_aligned && c != 0 && c != row.nchunks - 1)
    __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(d + (int64_t)c * Elem<T>::E - row.shift));
  else
    store_elements<T>(row, v, c, d);
}
// Through the gradient row's buffer (which starts at the chunk that holds its
// first element) where both rows start at the same place in a chunk.
template <typename T>
__device__ __forceinline__ void store_chunk(const Row<T>& row, const RowBuffer& out, const DistillArgs& a, v4i v, int first,
                                            int t, T* __restrict__ d) {
  const int c = first + t;
  const bool edge = c == 0 || c == row.nchunks - 1;
  if (a.d_aligned) {
    out.store(first, edge ? row.nchunks : t, v);
    if (edge) store_elements<T>(row, v, c, d);
  } else if (c < row.nchunks) {
    store_elements<T>(row, v, c, d);
  }
}

// Running sums of one thread: four fp32 sums relative to the maximum so far,
// so none adds more than a few dozen terms before they are joined.
template <typename T, int MODE>
struct Running {
  static constexpr int E = Elem<T>::E, S = 4;
  float max = -__builtin_inff();
  float s[S], s1[MODE ? S : 1];
  __device__ __forceinline__ Running() {
#pragma unroll
    for (int e = 0; e < S; ++e) s[e] = 0;
#pragma unroll
    for (int e = 0; e < (MODE ? S : 1); ++e) s1[e] = 0;
  }
  template <int N>
  __device__ __forceinline__ void add(const v4i (&v)[N], Expo<T, MODE>& ex) {
    float m = max;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) m = fmaxf(m, Elem<T>::get(v[i], e));
    rescale(m, ex);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = Elem<T>::get(v[i], e);
        const float y = ex.e(x);
        s[e % S] += y;
        if constexpr (MODE == 1) s1[e % S] = __builtin_fmaf(y, y, s1[e % S]);
        if constexpr (MODE == 2) s1[e % S] += ex.e1(x, y);
      }
  }
  __device__ __forceinline__ void rescale(float m, Expo<T, MODE>& ex) {
    const Expo<T, MODE> was = ex;
    ex.at(m);
    float f, f1 = 1;
    if constexpr (Expo<T, MODE>::kPrecise) {
      f = ex.e(was.m);
      if constexpr (MODE != 0) f1 = ex.e1(was.m, f);
    } else {  // between the rounded references, which the terms so far were formed with
      f = exp2_fast(was.r - ex.r);
      if constexpr (MODE == 1) f1 = f * f;
      if constexpr (MODE == 2) f1 = exp2_fast(was.r1 - ex.r1);
    }
    if (max == -__builtin_inff()) f = f1 = 1;  // nothing summed yet
    max = m;
#pragma unroll
    for (int e = 0; e < S; ++e) s[e] *= f;
    if constexpr (MODE != 0) {
#pragma unroll
      for (int e = 0; e < S; ++e) s1[e] *= f1;
    }
  }
  __device__ __forceinline__ float sum() const { return (s[0] + s[1]) + (s[2] + s[3]); }
  __device__ __forceinline__ float sum1() const {
    if constexpr (MODE == 0) return 0;
    else return (s1[0] + s1[1]) + (s1[2] + s1[3]);
  }
};

// ---- one workgroup a row, the row in registers -----------------------------
//
// Kept entries are one (or a few) per thread, which holds their logits and writes
// their gradient over what the row's sweep has put there, behind a barrier.

template <int NT>
struct RowLds {
  double sums[NT / 64][6];
  Factors f;
  float wmax[NT / 64], kmax[NT / 64], tmax[NT / 64];
  int kept[NT / 64];
  int label_kept;  // whether the label is a kept entry
};

// f(0), f(1), ... with the index a constant: a row's chunks are registers, and a
// loop too long for the compiler to unroll would put them into memory.
template <typename F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, const F& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(const F& f) {
  each_of(std::make_integer_sequence<int, N>{}, f);
}

// Sums over chunks g .. g + G - 1 of a thread; the elements that the masks name
// (kept entries, and what lies outside the row) become -inf.
template <typename T, int MODE, int g, int G, int N>
__device__ __forceinline__ void stats_group(v4i (&v)[N], const uint32_t (&masks)[N / 4 + (N < 4)], Running<T, MODE>& run,
                                            Expo<T, MODE>& ex) {
  v4i u[G];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const uint32_t mask = masks[(g + i) / 4] >> (8 * ((g + i) % 4)) & 0xFFu;
    if (mask) drop<T>(v[g + i], mask);
    u[i] = v[g + i];
  }
  run.add(u, ex);
  // The sums are wanted now: left alone, the compiler takes them where they are
  // used, behind the barrier, and holds every term's inputs until then.
  asm volatile("" : "+v"(run.s[0]), "+v"(run.s[1]), "+v"(run.s[2]), "+v"(run.s[3]));
  if constexpr (MODE != 0) asm volatile("" : "+v"(run.s1[0]), "+v"(run.s1[1]), "+v"(run.s1[2]), "+v"(run.s1[3]));
}

// A row far out, from memory: this thread's part of its sums, over the chunks first,
// first + step, ... below end, without the elements that skip(chunk) names.
template <typename T, int MODE, typename F>
__device__ __forceinline__ void far_sums(const Row<T>& x, const Expo<T, MODE>& ex, int first, int end, int step, const F& skip,
                                         float& sum, float& sum1) {
#pragma unroll 1
  for (int c = first; c < end; c += step) {
    v4i v = x.load(c);
    drop<T>(v, skip(c));
#pragma unroll
    for (int e = 0; e < Elem<T>::E; ++e) {
      const float xe = Elem<T>::get(v, e), y = ex.far_e(xe);
      sum += y;
      if (MODE) sum1 += ex.far_e1(xe, y);
    }
  }
}

// Waves a SIMD: what the row, 4 registers a chunk, leaves room for (two of a
// workgroup of 512 stand on each).
constexpr int row_waves(int nv) { return nv <= 4 ? 5 : nv <= 16 ? 4 : 2; }

template <typename T, int NT, int NV, int KPT, int MODE>
__global__ __launch_bounds__(NT, row_waves(NV)) void distill_rows(DistillArgs a) {
  constexpr int W = NT / 64, E = Elem<T>::E;
  constexpr int WORDS = NV / 4 + (NV < 4), G = NV >= 24 ? 4 : 2;
  // a byte a chunk, each thread's chunks (t, t + NT, ...) together
  __shared__ __attribute__((aligned(16))) uint32_t table[NT * WORDS];
  __shared__ RowLds<NT> l;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int k = a.k;
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.logits) + row * a.ld;
  const Row<T> x(a.logits, row, a.ld, (int)a.V);
  // entries and label first: they are needed before the row has arrived
  RawIndex raw[KPT], raw_label{};
  uint32_t raw_t[KPT];
  if (k > 0) {
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int j = min(t + i * NT, k - 1);
      raw[i].load(a.idx, row * a.i_ld + j, a.idx64);
      raw_t[i] = teacher_bits(a, row * a.t_ld + j);
    }
  }
  if (a.labels) raw_label.load(a.labels, row, a.lab64);
  const float lse = a.lse ? a.lse[row] : 0.0f;
  const RowBuffer in(x.chunks, x.nchunks);
  v4i v[NV];
  each<NV>([&](auto i) __attribute__((always_inline)) {
    v[i] = in.load(i * NT, t);
    __builtin_amdgcn_sched_barrier(0);  // in the order in which they are waited for
  });
  const int label = a.labels && raw_label.value(a.lab64) != a.ignore ? raw_label.index(a, a.lab64) : -1;
  int id[KPT];
  float tv[KPT];
  uint32_t xraw[KPT];  // bits, a value only behind the row's sums: at once, it would wait for all of the row
  float tmax = -__builtin_inff();
  int kept = 0;
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    id[i] = t + i * NT < k ? raw[i].index(a, a.idx64) : -1;
    tv[i] = t + i * NT < k ? teacher_value(a, raw_t[i]) : 0.0f;
  }
  // what lies outside the row: chunks behind it, and parts of the first and last
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 4 * w; i < 4 * w + 4 && i < NV; ++i) {
      const int c = i * NT + t;
      if (c == 0 || c >= x.nchunks - 1) word |= (c < x.nchunks ? x.outside(c) & 0xFFu : 0xFFu) << (8 * (i % 4));
    }
    table[t * WORDS + w] = word;
  }
  if (t == 0) l.label_kept = 0;
#pragma unroll
  for (int i = 0; i < KPT; ++i)
    if (id[i] >= 0) tmax = fmaxf(tmax, tv[i]), ++kept;
  if (wave * 64 < k) tmax = wave_max(tmax), kept = wave_sum(kept);
  if (lane == 0) l.tmax[wave] = tmax, l.kept[wave] = kept;
  lds_sync();
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    xraw[i] = Elem<T>::kNegInf;
    if (id[i] < 0) continue;
    const int at = id[i] + x.shift;
    const int c = at / E, i_of = c / NT;
    atomicOr(table + (c % NT) * WORDS + i_of / 4, 1u << (8 * (i_of % 4) + at % E));
    xraw[i] = Elem<T>::bits(xr + id[i]);
    if (id[i] == label) l.label_kept = 1;
  }
  const uint32_t lab_raw = Elem<T>::bits(xr + (label >= 0 ? label : 0));
  tmax = l.tmax[0], kept = l.kept[0];
#pragma unroll
  for (int w = 1; w < W; ++w) tmax = fmaxf(tmax, l.tmax[w]), kept += l.kept[w];
  // scalar registers, and zref only where it is used: the row's sums leave no others
  tmax = uniform(a.lse ? lse : tmax), kept = __builtin_amdgcn_readfirstlane(kept);
  lds_sync();

  Expo<T, MODE> ex(a);
  Running<T, MODE> run;
  uint32_t masks[WORDS];
  if constexpr (NV >= 24) {  // all at once, where there are few waves to wait behind
#pragma unroll
    for (int w = 0; w < WORDS; ++w) masks[w] = table[t * WORDS + w];
  }
  each<NV / G>([&](auto g) __attribute__((always_inline)) {
    if constexpr (NV < 24 && G * g % 4 == 0) masks[G * g / 4] = table[t * WORDS + G * g / 4];
    stats_group<T, MODE, G * g, G>(v, masks, run, ex);
    __builtin_amdgcn_sched_barrier(0);  // mixed, several chunks' values would not fit the registers
  });
  __builtin_amdgcn_sched_barrier(0);  // nothing of what follows takes registers from the sums
  const float xlab = uniform(Elem<T>::value(lab_raw));
  float xj[KPT];
  float m = run.max, mk = -__builtin_inff();  // of the entries not kept, and of the kept
#pragma unroll
  for (int i = 0; i < KPT; ++i) mk = fmaxf(mk, xj[i] = Elem<T>::value(xraw[i]));
  wave_max2(m, mk);
  if (lane == 0) l.wmax[wave] = m, l.kmax[wave] = mk;
  lds_sync();
  m = l.wmax[0], mk = l.kmax[0];
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, l.wmax[w]), mk = fmaxf(mk, l.kmax[w]);
  m = uniform(m);
  run.rescale(m, ex);
  ex.at_row(m, uniform(fmaxf(m, mk)));
  ex.uniform_all();
  float ws = run.sum(), ws1 = run.sum1();
  const auto marked_here = [&](int c) {
    const int i = c / NT;
    return table[(c % NT) * WORDS + i / 4] >> (8 * (i % 4)) & 0xFFu;
  };
  if (ex.far()) ws = ws1 = 0, far_sums<T, MODE>(x, ex, t, x.nchunks, NT, marked_here, ws, ws1);
  ws = wave_sum(ws), ws1 = MODE ? wave_sum(ws1) : 0;
  const double zref = a.lse ? (double)tmax : (double)tmax * a.itau;
  float e0[KPT], e1[KPT], w0[KPT];
  double q[4] = {0, 0, 0, 0};
  if (wave * 64 < k) {  // kept entries in 64 bits
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (id[i] < 0) continue;
      const double lw = (double)tv[i] * a.itau - zref, w = exp2_d(lw * kLog2e);
      const double y = (double)xj[i], ye = ex.log2e(y, a), e = exp2_d(ye);
      const double f1 = MODE == 0 ? e : MODE == 1 ? e * e : exp2_d(ex.log2e1(y, a));
      q[0] += w;
      if (!(w == 0)) q[1] += w * (lw - ye * kLn2);
      q[2] += e;
      q[3] += f1;
      e0[i] = (float)e, e1[i] = (float)f1, w0[i] = (float)w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = wave_sum(q[i]);
  }
  if (lane == 0) {
    l.sums[wave][0] = (double)ws, l.sums[wave][1] = (double)ws1;
#pragma unroll
    for (int i = 0; i < 4; ++i) l.sums[wave][2 + i] = q[i];
  }
  lds_sync();
  const auto joined = [&]() -> Joined {
    return {l.sums[0][0], l.sums[0][1], l.sums[0][2], l.sums[0][3], l.sums[0][4], l.sums[0][5], zref, kept};
  };
  if (wave == 0) {
    if (lane < 6) {  // a sum a lane
      double b = l.sums[0][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) b += l.sums[w][lane];
      l.sums[0][lane] = b;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS operations stay in order
    if (lane == 0 && a.d) {
      const Joined s = joined();
      l.f = factors(a, join(a, s, ex).st, kept == 0 ? 0 : a.lse ? 1 : 1 / s.W, row, label >= 0, MODE);
    }
  }
  lds_sync();
  if (a.d) {
    const Factors f = uniform(l.f);
    T* d = static_cast<T*>(a.d) + row * a.d_ld;
    const RowBuffer out(a.d_aligned ? d - x.shift : d, x.nchunks);
    if (ex.far()) {
#pragma unroll 1
      for (int c = t; c < x.nchunks; c += NT) store_chunk<T>(x, a, grad_chunk<T, MODE, true>(ex, f, x.load(c)), c, d);
    } else {
      each<NV>([&](auto i) __attribute__((always_inline)) {
        // unpacked again: the values that the sums had unpacked are not to be kept for this
        asm volatile("" : "+v"(v[i]));
        if (i * NT < x.nchunks) store_chunk<T>(x, out, a, grad_chunk<T, MODE>(ex, f, v[i]), i * NT, t, d);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  }
  if (wave == W - 1) {  // while the sweep's stores arrive
    const Joined s = joined();
    write_row(a, row, s, join(a, s, ex), ex.gap(a), label >= 0 ? ex.log2e1((double)xlab, a) : 0, label >= 0);
  }
  if (a.d) {
    T* d = static_cast<T*>(a.d) + row * a.d_ld;
    const Factors f = uniform(l.f);
    __syncthreads();  // what follows is stored behind the sweep's stores
#pragma unroll
    for (int i = 0; i < KPT; ++i)
      if (id[i] >= 0) d[id[i]] = (T)kept_grad(f, e0[i], e1[i], w0[i], id[i] == label);
    if (t == 0 && label >= 0 && !l.label_kept) d[label] = (T)(label_grad<T, MODE>(ex, f, xlab));
  }
}

// ---- segments of rows ------------------------------------------------------

constexpr int kSegThreads = 512;
constexpr int kSegChunks = 4096;  // at most: a byte of the table each

struct SegLds {
  uint32_t table[kSegChunks / 4];
  double sums[kSegThreads / 64][6];
  float wmax[kSegThreads / 64], kmax[kSegThreads / 64];
  int kept[kSegThreads / 64];
  int label_kept;
  Joined joined;  // of thread 0, until it writes the loss
};

// Kept entries in chunks [c0, c1) go into the table.
template <typename T>
__device__ __forceinline__ void seg_table(SegLds& l, const DistillArgs& a, const Row<T>& x, int64_t row, int c0, int c1) {
  constexpr int E = Elem<T>::E;
  const int t = threadIdx.x;
  for (int c = t; 4 * c < c1 - c0; c += kSegThreads) l.table[c] = 0;
  __syncthreads();
  for (int j = t; j < a.k; j += kSegThreads) {
    const int id = kept_at(a, row, j);
    if (id < 0) continue;
    const int at = id + x.shift, c = at / E;
    if (c >= c0 && c < c1) mark(l.table, c - c0, at % E);
  }
  __syncthreads();
}

template <typename T, int MODE>
__global__ __launch_bounds__(kSegThreads) void distill_partial(DistillArgs a) {
  constexpr int W = kSegThreads / 64, GROUP = 4;
  __shared__ __attribute__((aligned(16))) SegLds l;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int seg = (int)(blockIdx.x % a.segs);
  const int64_t row = blockIdx.x / a.segs;
  const Row<T> x(a.logits, row, a.ld, (int)a.V);
  const int c0 = seg * a.seg_chunks, c1 = min(x.nchunks, c0 + a.seg_chunks);
  seg_table<T>(l, a, x, row, c0, c1);
  Expo<T, MODE> ex(a);
  Running<T, MODE> run;
  for (int g = c0 + t; g < c1; g += GROUP * kSegThreads) {
    v4i v[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const int c = g + i * kSegThreads;
      v[i] = c < c1 ? x.load(c) : all_neg_inf(sizeof(T), Elem<T>::kNegInf);
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const int c = g + i * kSegThreads;
      const uint32_t mask = c < c1 ? marked(l.table, c - c0) : 0;
      if (mask) drop<T>(v[i], mask);
    }
    run.add(v, ex);
  }
  const float wm = wave_max(run.max);
  if (lane == 0) l.wmax[wave] = wm;
  __syncthreads();
  float m = l.wmax[0];
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, l.wmax[w]);
  run.rescale(m, ex);  // a row far out: these sums are not used
  const float s = wave_sum(run.sum()), s1 = MODE ? wave_sum(run.sum1()) : 0;
  if (lane == 0) l.sums[wave][0] = s, l.sums[wave][1] = s1;
  __syncthreads();
  if (t == 0) {
    double b = 0, b1 = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) b += l.sums[w][0], b1 += l.sums[w][1];
    static_cast<Partial*>(a.partial)[blockIdx.x] = {m, (float)b, (float)b1, 0.0f};
  }
}

// A kept entry as memory holds it.
struct Kept {
  int id;  // or -1
  float t, x;
};
template <typename T>
__device__ __forceinline__ Kept fetch_kept(const DistillArgs& a, int64_t row, int j) {
  Kept e{-1, 0, 0};
  if (j < a.k) e.id = kept_at(a, row, j);
  if (e.id >= 0) e.t = teacher_at(a, row, j), e.x = (float)(static_cast<const T*>(a.logits) + row * a.ld)[e.id];
  return e;
}

// A row's partial sums and kept entries joined, by the whole workgroup; every
// thread returns the sums.  mine: entry threadIdx.x, held since the kernel's
// start: its loads wait for each other, and this is all latency.
template <typename T, int MODE>
__device__ __forceinline__ Joined seg_join(SegLds& l, const DistillArgs& a, int64_t row, const Kept& mine, Expo<T, MODE>& ex) {
  constexpr int W = kSegThreads / 64;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const Partial* part = static_cast<const Partial*>(a.partial) + row * a.segs;
  const Partial my_part = part[min(t, a.segs - 1)];
  const float lse = a.lse ? a.lse[row] : 0.0f;
  float tmax = -__builtin_inff(), m = -__builtin_inff(), mk = -__builtin_inff();
  int kept = 0;
  for (int j = t; j < a.k; j += kSegThreads)
    if (const Kept e = j == t ? mine : fetch_kept<T>(a, row, j); e.id >= 0) tmax = fmaxf(tmax, e.t), mk = fmaxf(mk, e.x), ++kept;
  for (int i = t; i < a.segs; i += kSegThreads) m = fmaxf(m, i == t ? my_part.max : part[i].max);
  wave_max2(m, mk);
  tmax = wave_max(tmax), kept = wave_sum(kept);
  if (lane == 0) l.wmax[wave] = tmax, l.kmax[wave] = mk, l.sums[wave][0] = m, l.kept[wave] = kept;
  __syncthreads();
  tmax = m = mk = -__builtin_inff(), kept = 0;
#pragma unroll
  for (int w = 0; w < W; ++w)
    tmax = fmaxf(tmax, l.wmax[w]), m = fmaxf(m, (float)l.sums[w][0]), mk = fmaxf(mk, l.kmax[w]), kept += l.kept[w];
  __syncthreads();
  tmax = uniform(tmax), m = uniform(m), kept = __builtin_amdgcn_readfirstlane(kept);
  ex.at_row(m, uniform(fmaxf(m, mk)));
  ex.uniform_all();
  double q[6] = {0, 0, 0, 0, 0, 0};
  if (ex.far()) {
    const Row<T> r(a.logits, row, a.ld, (int)a.V);
    float s = 0, s1 = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < r.nchunks; c0 += kSegChunks) {
      const int c1 = min(r.nchunks, c0 + kSegChunks);
      seg_table<T>(l, a, r, row, c0, c1);
      far_sums<T, MODE>(r, ex, c0 + t, c1, kSegThreads, [&](int c) { return marked(l.table, c - c0); }, s, s1);
      __syncthreads();
    }
    q[0] = s, q[1] = s1;
  } else {
    for (int i = t; i < a.segs; i += kSegThreads) {
      const Partial p = i == t ? my_part : part[i];
      Expo<T, MODE> own(a);
      own.at(p.max);
      // between the two references
      constexpr bool precise = Expo<T, MODE>::kPrecise;
      const double dm = (double)own.m - (double)ex.m;
      const double y = precise ? dm * a.cd : (double)own.r - (double)ex.r;
      const double y1 = MODE == 1 ? 2 * y : precise ? dm * kLog2e : (double)own.r1 - (double)ex.r1;
      q[0] += p.sum == 0 ? 0 : (double)p.sum * exp2_d(y);
      if (MODE) q[1] += p.sum1 == 0 ? 0 : (double)p.sum1 * exp2_d(y1);
    }
  }
  const double itau = a.itau, zref = a.lse ? (double)lse : (double)tmax * itau;
  for (int j = t; j < a.k; j += kSegThreads) {
    const Kept k = j == t ? mine : fetch_kept<T>(a, row, j);
    if (k.id < 0) continue;
    const double lw = (double)k.t * itau - zref, w = exp2_d(lw * kLog2e), xj = (double)k.x;
    const double y = ex.log2e(xj, a), e = exp2_d(y);
    q[2] += w;
    if (!(w == 0)) q[3] += w * (lw - y * kLn2);
    q[4] += e;
    q[5] += MODE == 0 ? e : exp2_d(ex.log2e1(xj, a));
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    q[i] = wave_sum(q[i]);
    if (lane == 0) l.sums[wave][i] = q[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    q[i] = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) q[i] += l.sums[w][i];
  }
  __syncthreads();
  return {q[0], q[1], q[2], q[3], q[4], q[5], zref, kept};
}

template <typename T, int MODE>
__global__ __launch_bounds__(kSegThreads) void distill_finish(DistillArgs a) {
  __shared__ __attribute__((aligned(16))) SegLds l;
  const int64_t row = blockIdx.x;
  const Kept mine = fetch_kept<T>(a, row, threadIdx.x);
  Expo<T, MODE> ex(a);
  const Joined s = seg_join<T, MODE>(l, a, row, mine, ex);
  if (threadIdx.x >= 64) return;
  const int label = label_at(a, row);
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  write_row(a, row, s, join(a, s, ex), ex.gap(a), label >= 0 ? ex.log2e1((double)(float)x[label], a) : 0, label >= 0);
}

// GIVEN: the row's statistics come from an earlier forward.
template <typename T, int MODE, bool GIVEN>
__global__ __launch_bounds__(kSegThreads, 4) void distill_grad(DistillArgs a) {
  constexpr int GROUP = 4;
  __shared__ __attribute__((aligned(16))) SegLds l;
  const int t = threadIdx.x;
  const int seg = (int)(blockIdx.x % a.segs);
  const int64_t row = blockIdx.x / a.segs;
  const Row<T> x(a.logits, row, a.ld, (int)a.V);
  const int c0 = seg * a.seg_chunks, c1 = min(x.nchunks, c0 + a.seg_chunks);
  const int label = label_at(a, row);
  const Kept mine = fetch_kept<T>(a, row, t);
  v4i v[GROUP];
  const auto fetch = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < GROUP; ++i)
      if (g + i * kSegThreads < c1) v[i] = x.load(g + i * kSegThreads);
  };
  fetch(c0 + t);  // on the way while the row's sums are joined
  Expo<T, MODE> ex(a);
  RowStats st;
  double w_ref, w_scale;  // p_j = w_scale exp(t_j / tau - w_ref)
  if constexpr (GIVEN) {
    st = static_cast<const RowStats*>(a.stats)[row];
    ex.at_row((float)st.ref_out, (float)st.ref);
    w_ref = st.z, w_scale = 1;
  } else {
    const Joined s = seg_join<T, MODE>(l, a, row, mine, ex);
    st = join(a, s, ex).st;
    if (t == 0) l.joined = s;
    w_ref = s.zref, w_scale = s.kept == 0 ? 0 : a.lse ? 1 : 1 / s.W;
  }
  const Factors f = uniform(factors(a, st, w_scale, row, label >= 0, MODE));
  T* d = static_cast<T*>(a.d) + row * a.d_ld;
  for (int g = c0 + t; g < c1;) {
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const int c = g + i * kSegThreads;
      if (c >= c1) continue;
      if (ex.far()) store_chunk<T>(x, a, grad_chunk<T, MODE, true>(ex, f, v[i]), c, d);
      else store_chunk<T>(x, a, grad_chunk<T, MODE>(ex, f, v[i]), c, d);
    }
    g += GROUP * kSegThreads;
    fetch(g);
  }
  // kept entries and the label over what the sweep has put there
  const T* xr = static_cast<const T*>(a.logits) + row * a.ld;
  const auto here = [&](int id) { const int c = (id + x.shift) / Elem<T>::E; return c >= c0 && c < c1; };
  if (t == 0) l.label_kept = 0;
  __syncthreads();
  if constexpr (!GIVEN) {
    if (t >= kSegThreads - 64 && seg == 0)
      write_row(a, row, l.joined, join(a, l.joined, ex), ex.gap(a), label >= 0 ? ex.log2e1((double)(float)xr[label], a) : 0, label >= 0);
  }
  for (int j = t; j < a.k; j += kSegThreads) {
    const Kept k = j == t ? mine : fetch_kept<T>(a, row, j);
    const int id = k.id;
    if (id < 0 || !here(id)) continue;
    const double y = (double)k.x;
    const float e = (float)exp2_d(ex.log2e(y, a)), e1 = MODE == 0 ? e : (float)exp2_d(ex.log2e1(y, a));
    const float w = (float)exp2_d(((double)k.t * a.itau - w_ref) * kLog2e);
    if (id == label) l.label_kept = 1;
    d[id] = (T)kept_grad(f, e, e1, w, id == label);
  }
  __syncthreads();
  if (t == 0 && label >= 0 && !l.label_kept && here(label)) d[label] = (T)(label_grad<T, MODE>(ex, f, (float)xr[label]));
}

// ---- launches ---------------------------------------------------------------

template <typename T, int MODE>
hipError_t launch_mode(const DistillArgs& a, hipStream_t stream) {
  switch (a.plan) {
    case kRows64x2: distill_rows<T, 64, 2, 2, MODE><<<(unsigned)a.T, 64, 0, stream>>>(a); break;
    case kRows64x4: distill_rows<T, 64, 4, 2, MODE><<<(unsigned)a.T, 64, 0, stream>>>(a); break;
    case kRows64x8: distill_rows<T, 64, 8, 2, MODE><<<(unsigned)a.T, 64, 0, stream>>>(a); break;
    case kRows256x4: distill_rows<T, 256, 4, 2, MODE><<<(unsigned)a.T, 256, 0, stream>>>(a); break;
    case kRows256x8: distill_rows<T, 256, 8, 2, MODE><<<(unsigned)a.T, 256, 0, stream>>>(a); break;
    case kRows512x8: distill_rows<T, 512, 8, 2, MODE><<<(unsigned)a.T, 512, 0, stream>>>(a); break;
    case kRows512x12: distill_rows<T, 512, 12, 2, MODE><<<(unsigned)a.T, 512, 0, stream>>>(a); break;
    case kRows512x16: distill_rows<T, 512, 16, 2, MODE><<<(unsigned)a.T, 512, 0, stream>>>(a); break;
    case kRows512x24: distill_rows<T, 512, 24, 2, MODE><<<(unsigned)a.T, 512, 0, stream>>>(a); break;
    case kRows512x32: distill_rows<T, 512, 32, 2, MODE><<<(unsigned)a.T, 512, 0, stream>>>(a); break;
    default: {
      const dim3 grid((unsigned)(a.T * a.segs));
      if (a.given) {
        distill_grad<T, MODE, true><<<grid, kSegThreads, 0, stream>>>(a);
        break;
      }
      distill_partial<T, MODE><<<grid, kSegThreads, 0, stream>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      if (a.d)
        distill_grad<T, MODE, false><<<grid, kSegThreads, 0, stream>>>(a);
      else
        distill_finish<T, MODE><<<(unsigned)a.T, kSegThreads, 0, stream>>>(a);
    }
  }
  return hipGetLastError();
}

// Rows [row, row + rows) of a call.
template <typename T>
DistillArgs rows_of(DistillArgs a, int64_t row, int64_t rows) {
  const auto at = [&](const void* p, int64_t per_row, int64_t elem) {
    return p ? static_cast<const char*>(p) + row * per_row * elem : nullptr;
  };
  const int64_t index = a.idx64 ? 8 : 4, label = a.lab64 ? 8 : 4;
  a.logits = at(a.logits, a.ld, sizeof(T));
  a.teacher = at(a.teacher, a.t_ld, a.t_dtype == I8MP_FP32 ? 4 : 2), a.idx = at(a.idx, a.i_ld, index);
  a.labels = at(a.labels, 1, label);
  if (a.lse) a.lse += row;
  if (a.grad) a.grad += row * a.grad_s;
  if (a.loss) a.loss += row;
  a.stats = const_cast<char*>(at(a.stats, 1, sizeof(RowStats)));
  a.d = const_cast<char*>(at(a.d, a.d_ld, sizeof(T)));
  a.partial = const_cast<char*>(at(a.partial, a.segs, sizeof(Partial)));
  a.T = rows;
  return a;
}

template <typename T>
hipError_t launch_typed(const DistillArgs& a, hipStream_t stream) {
  // A launch holds fewer than 2^32 work items; as many rows as that leaves at 512 a segment.
  const int64_t per = std::max<int64_t>(1, ((int64_t(1) << 32) - 1) / ((int64_t)kSegThreads * a.segs));
  for (int64_t row = 0; row < a.T; row += per) {
    const DistillArgs part = rows_of<T>(a, row, std::min(per, a.T - row));
    const hipError_t e = !part.labels || a.tau == 1.0f ? launch_mode<T, 0>(part, stream)
                         : a.tau == 2.0f               ? launch_mode<T, 1>(part, stream)
                                                       : launch_mode<T, 2>(part, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace distill
}  // namespace i8mp
