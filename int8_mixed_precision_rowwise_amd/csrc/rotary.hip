// Rotary positions of query and key heads, and their inverse (which is also
// the backward: the rotation is orthogonal, so its gradient is the rotation by
// the negative angle).
//
// Pair i of a head is (a, b); with t = position * freqs[i]
//   a' = a cos t - b sin t,   b' = a sin t + b cos t.
// "half" pairs are elements (i, i + rot / 2), "interleaved" ones (2i, 2i + 1);
// elements from rot on are copied.
//
// The angle of a position 10^6 out needs more than the 24 bits of a float: it
// is formed and reduced in 64 bits (t * 2/pi = n + f, n the nearest integer,
// |f| <= 1/2), and only the remainder f * pi/2 goes to fp32, where the Taylor
// polynomials of sine (to y^9) and cosine (to y^10) on [-pi/4, pi/4] are off
// by less than 2^-28.
//
// A pass reads and writes every head once and computes next to nothing, so it
// is bound by memory (by the launch, for one token per sequence).  The cosines
// and sines of a token serve all its heads: a workgroup takes a few whole
// tokens (or part of one token's heads), computes their table into LDS, then
// streams the heads with the widest access that the pairs' layout allows.  A
// token's place in each tensor stands in LDS too: with the division and the wide
// products in the streaming loop those were what bounded it (16 x 2048 tokens of 36
// bf16 heads of 64: 95 us, now 55 us for 302 MB, 5.5 TB/s; the backward of 2 x 4001
// tokens of 40 heads of 128, half of each rotated: 38 us, now 29 us for 164 MB, which
// partly stay in the last level).  One token of 64 sequences takes 3.7 us.
#include "internal.h"

#include <type_traits>

namespace i8mp {
namespace {

constexpr int kRotThreads = 256;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));

// Outputs of more bytes than this are written past the caches: with the inputs they
// would not stay in the last level of 256 MiB anyway.  82 MB out from inputs that are
// not in the caches: 34 us past them and 41 through them; 75 MB from inputs that
// are, then read again: 36 and 32; 151 MB: 68 and 73.
constexpr int64_t kPast = 64 << 20;

struct RotKernelArgs {
  RotaryTensor t[2];  // q, k
  int64_t tokens, S;
  int64_t first;     // token of the launch's first workgroup
  const void* pos;
  int64_t pos_b, pos_s;
  const double* freqs;
  int pos32, D, rot;
  float sign;
  int tpw;           // tokens per workgroup
  int rows_per_y;    // heads per workgroup along grid y (all of them unless tpw = 1)
  int slots;         // work items per head
  int rot_slots;     // of them, items that rotate
  int dslot, drow;   // kRotThreads = drow * slots + dslot
};

// fp32 cosine and sine of an angle given in 64 bits.
__device__ __forceinline__ float2 cos_sin(double angle) {
  const double turns = angle * 0.63661977236758134308;  // 2 / pi
  const double n = __builtin_rint(turns);
  const double f = __builtin_fma(angle, 0.63661977236758134308, -n);
  const float y = (float)(f * 1.57079632679489661923);
  // the quarter modulo 4 by a 64-bit remainder: exact for every n
  const int quarter = (int)(n - 4.0 * __builtin_floor(n * 0.25));
  const float y2 = y * y;
  float s = 1.0f / 362880.0f;
  s = __builtin_fmaf(s, y2, -1.0f / 5040.0f);
  s = __builtin_fmaf(s, y2, 1.0f / 120.0f);
  s = __builtin_fmaf(s, y2, -1.0f / 6.0f);
  s = __builtin_fmaf(s * y2, y, y);
  float c = -1.0f / 3628800.0f;
  c = __builtin_fmaf(c, y2, 1.0f / 40320.0f);
  c = __builtin_fmaf(c, y2, -1.0f / 720.0f);
  c = __builtin_fmaf(c, y2, 1.0f / 24.0f);
  c = __builtin_fmaf(c, y2, -0.5f);
  c = __builtin_fmaf(c, y2, 1.0f);
  const float cc = (quarter & 1) ? s : c, ss = (quarter & 1) ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -cc : cc, quarter >= 2 ? -ss : ss);
}

// V elements of type T, read and written in one access (WIDE) or one by one; PAST:
// written past the caches.
template <typename T, int V, bool WIDE, bool PAST>
struct Pack {
  template <int BYTES>
  using Word = std::conditional_t<BYTES == 16, v4i, std::conditional_t<BYTES == 8, v2i, int>>;
  struct __attribute__((aligned(WIDE ? sizeof(T) * V : sizeof(T)))) Mem { T v[V]; };
  static __device__ __forceinline__ void load(const T* p, T (&x)[V]) {
    const Mem m = *reinterpret_cast<const Mem*>(p);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = m.v[j];
  }
  static __device__ __forceinline__ void store(T* p, const T (&x)[V]) {
    Mem m;
#pragma unroll
    for (int j = 0; j < V; ++j) m.v[j] = x[j];
    if constexpr (PAST && WIDE && sizeof(Mem) >= 4)
      __builtin_nontemporal_store(__builtin_bit_cast(Word<sizeof(Mem)>, m), reinterpret_cast<Word<sizeof(Mem)>*>(p));
    else
      *reinterpret_cast<Mem*>(p) = m;
  }
};

// An fp32 value in T.  Left alone, the compiler gives some fp16 outputs a fused
// instruction that rounds once where the others round to fp32 first, and which ones
// differs between this kernel's forms: a call's bits would depend on its size.
template <typename T>
__device__ __forceinline__ T rounded(float x) {
  if constexpr (std::is_same_v<T, _Float16>) asm("" : "+v"(x));
  return (T)x;
}

// Every element is read before its pair's outputs are written, by the same
// thread, so the outputs may be the inputs themselves.
template <typename T, int V, bool WIDE, bool HALF, bool PAST>
__global__ __launch_bounds__(kRotThreads) void rotary_kernel(RotKernelArgs a) {
  // a token's first elements in q, k and their outputs; [tokens][rot / 2]: cosine, sine
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int64_t(*at0)[4] = reinterpret_cast<int64_t(*)[4]>(lds);
  float2* table = reinterpret_cast<float2*>(lds + a.tpw * sizeof(*at0));
  typedef Pack<T, V, WIDE, PAST> P;
  const int t = threadIdx.x;
  const int half = a.rot / 2;
  const int64_t token0 = a.first + (int64_t)blockIdx.x * a.tpw;
  const int tokens = (int)min((int64_t)a.tpw, a.tokens - token0);
  for (int i = t; i < tokens * half; i += kRotThreads) {
    const int tb = i / half, pair = i - tb * half;
    const int64_t token = token0 + tb;
    const int64_t b = a.tokens >> 31 ? token / a.S : (int64_t)((uint32_t)token / (uint32_t)a.S), s = token - b * a.S;
    const int64_t at = b * a.pos_b + s * a.pos_s;
    const int64_t p = a.pos32 ? (int64_t) static_cast<const int32_t*>(a.pos)[at] : static_cast<const int64_t*>(a.pos)[at];
    float2 cs = cos_sin((double)p * a.freqs[pair]);
    cs.y *= a.sign;
    table[i] = cs;
    if (pair == 0) {  // once a token: the streaming loop multiplies and divides nothing wide
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        at0[tb][w] = b * a.t[w].x_b + s * a.t[w].x_s;
        at0[tb][2 + w] = b * a.t[w].y_b + s * a.t[w].y_s;
      }
    }
  }
  __syncthreads();
  const int heads = a.t[0].heads + a.t[1].heads;
  const int row0 = (int)blockIdx.y * a.rows_per_y;
  const int rows = min(a.rows_per_y, heads - row0);
  int row = t / a.slots, slot = t - row * a.slots;
  int tb = row / rows;
  row -= tb * rows;
  while (tb < tokens) {
    const int which = row0 + row >= a.t[0].heads;
    const int h = row0 + row - (which ? a.t[0].heads : 0);
    const RotaryTensor& r = a.t[which];
    const T* x = static_cast<const T*>(r.x) + at0[tb][which] + h * r.x_h;
    T* y = static_cast<T*>(r.y) + at0[tb][2 + which] + h * r.y_h;
    const float2* cs = table + tb * half;
    if (slot >= a.rot_slots) {  // past the rotated part: copied
      const int e = a.rot + (slot - a.rot_slots) * V;
      T v[V];
      P::load(x + e, v);
      P::store(y + e, v);
    } else if constexpr (HALF) {
      const int e = slot * V;
      T u[V], v[V];
      P::load(x + e, u);
      P::load(x + e + half, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 k = cs[e + j];
        const float p = (float)u[j], q = (float)v[j];
        u[j] = rounded<T>(__builtin_fmaf(p, k.x, -(q * k.y)));
        v[j] = rounded<T>(__builtin_fmaf(p, k.y, q * k.x));
      }
      P::store(y + e, u);
      P::store(y + e + half, v);
    } else {
      const int e = slot * V;
      T v[V];
      P::load(x + e, v);
#pragma unroll
      for (int j = 0; j + 1 < V; j += 2) {
        const float2 k = cs[(e + j) / 2];
        const float p = (float)v[j], q = (float)v[j + 1];
        v[j] = rounded<T>(__builtin_fmaf(p, k.x, -(q * k.y)));
        v[j + 1] = rounded<T>(__builtin_fmaf(p, k.y, q * k.x));
      }
      P::store(y + e, v);
    }
    slot += a.dslot;
    row += a.drow;
    if (slot >= a.slots) slot -= a.slots, ++row;
    while (row >= rows) row -= rows, ++tb;
  }
}

template <typename T, int V, bool WIDE, bool PAST>
void launch_pairs(const RotKernelArgs& a, bool half, dim3 grid, size_t lds, hipStream_t stream) {
  if (half)
    rotary_kernel<T, V, WIDE, true, PAST><<<grid, kRotThreads, lds, stream>>>(a);
  else if constexpr (V >= 2)
    rotary_kernel<T, V, WIDE, false, PAST><<<grid, kRotThreads, lds, stream>>>(a);
}

template <typename T>
hipError_t launch_typed(RotKernelArgs a, bool half, hipStream_t stream) {
  // Elements per access: the widest power of two, up to 16 bytes, that divides
  // the rotated part (each half of it for half pairs), the head and every
  // stride, with aligned bases.
  constexpr int kWidest = 16 / (int)sizeof(T);
  int64_t any = a.D | (half ? a.rot / 2 : a.rot);
  for (const RotaryTensor& r : a.t)
    if (r.heads > 0) {
      any |= r.x_b | r.x_s | r.x_h | r.y_b | r.y_s | r.y_h;
      any |= (int64_t)((reinterpret_cast<uintptr_t>(r.x) | reinterpret_cast<uintptr_t>(r.y)) / sizeof(T));
    }
  int v = kWidest;
  while (v > 1 && any % v) v /= 2;
  const bool wide = half || v >= 2;
  if (!wide) v = 2;  // interleaved pairs at an odd address or stride: element by element
  a.rot_slots = (half ? a.rot / 2 : a.rot) / v;
  a.slots = a.rot_slots + (a.D - a.rot) / v;
  const int heads = a.t[0].heads + a.t[1].heads;
  // Workgroups of about 1024 items while that leaves 2048 of them (8 a CU);
  // with fewer tokens one token each, and with few of those the heads are
  // split so that one item falls to each thread.
  const int64_t items = (int64_t)heads * a.slots;
  a.tpw = (int)max((int64_t)1, min(min((int64_t)16, 1024 / items), a.tokens / 2048));
  a.tpw = (int)min((int64_t)a.tpw, max((int64_t)1, (int64_t)32768 / max(1, a.rot / 2 * 8)));
  a.rows_per_y = heads;
  if (a.tpw == 1 && a.tokens < 1024) a.rows_per_y = (int)max((int64_t)1, min((int64_t)heads, (int64_t)kRotThreads / a.slots));
  a.drow = kRotThreads / a.slots;
  a.dslot = kRotThreads - a.drow * a.slots;
  const size_t lds = (size_t)a.tpw * (a.rot / 2 * sizeof(float2) + 32);
  const bool past = kPast < (int64_t)sizeof(T) * a.tokens * heads * a.D;
  // a launch holds fewer than 2^32 work items
  const int64_t step = ((int64_t(1) << 32) / kRotThreads - 1) * a.tpw;
  for (a.first = 0; a.first < a.tokens; a.first += step) {
    const dim3 grid((unsigned)((min(step, a.tokens - a.first) + a.tpw - 1) / a.tpw),
                    (unsigned)((heads + a.rows_per_y - 1) / a.rows_per_y));
    if constexpr (kWidest >= 8) {
      if (v == 8 && past) launch_pairs<T, 8, true, true>(a, half, grid, lds, stream);
      if (v == 8 && !past) launch_pairs<T, 8, true, false>(a, half, grid, lds, stream);
    }
    if (v == 4 && past) launch_pairs<T, 4, true, true>(a, half, grid, lds, stream);
    if (v == 4 && !past) launch_pairs<T, 4, true, false>(a, half, grid, lds, stream);
    if (v == 2 && wide) launch_pairs<T, 2, true, false>(a, half, grid, lds, stream);
    if (v == 2 && !wide) launch_pairs<T, 2, false, false>(a, half, grid, lds, stream);
    if (v == 1) launch_pairs<T, 1, true, false>(a, half, grid, lds, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rotary(const RotaryTensor& q, const RotaryTensor& k, int64_t B, int64_t S, int D, int rot, int dtype,
                         bool half, bool inverse, const void* pos, int pos32, int64_t pos_b, int64_t pos_s,
                         const double* freqs, hipStream_t stream) {
  RotKernelArgs a{};
  a.t[0] = q, a.t[1] = k;
  a.tokens = B * S, a.S = S;
  a.pos = pos, a.pos32 = pos32, a.pos_b = pos_b, a.pos_s = pos_s;
  a.freqs = freqs;
  a.D = D, a.rot = rot;
  a.sign = inverse ? -1.0f : 1.0f;
  switch (dtype) {
    case I8MP_BF16: return launch_typed<__bf16>(a, half, stream);
    case I8MP_FP16: return launch_typed<_Float16>(a, half, stream);
    default: return launch_typed<float>(a, half, stream);
  }
}

}  // namespace i8mp
