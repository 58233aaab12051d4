// Device side of the quantization passes: scales, codes and maxima of bf16
// chunks (the method and its arithmetic are described in quantize.hip).
#pragma once

#include "internal.h"
#include "philox.h"

namespace i8mp {
namespace {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / 64;

__device__ __forceinline__ us2 as_us2(uint32_t w) { return __builtin_bit_cast(us2, w); }

// Largest |x| bit pattern among the 8 bf16 of a chunk, kept as two halves.
__device__ __forceinline__ us2 absmax_bits(us2 m, uint4 v) {
  m = __builtin_elementwise_max(m, as_us2(v.x & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, as_us2(v.y & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, as_us2(v.z & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, as_us2(v.w & 0x7FFF7FFFu));
  return m;
}

// Zero the bf16 elements at positions >= n (1 <= n < 8) of a chunk.
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lo = 2 * i, hi = 2 * i + 1;
    uint32_t mask = (lo < n ? 0x0000FFFFu : 0u) | (hi < n ? 0xFFFF0000u : 0u);
    w[i] &= mask;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Maximum over the 64 lanes of a wave (all lanes active), the same value in
// every lane.  DPP: within each row of 16 lanes DPP moves combine neighbours
// (quad permutes [1,0,3,2] and [2,3,0,1], then the half-row and row
// mirrors) and the four row maxima are read out with readlane, all in VALU /
// SALU latency; otherwise butterfly shuffles through LDS permutes.  Which is
// faster depends on the kernel (measured at 4096 x 4096: the one-row-per-wave
// pass, at 59 VGPRs and 8 waves per SIMD, runs 0.5 us faster with shuffles;
// the pass with column maxima, at 2-3 waves per SIMD, 0.3 us faster with DPP).
template <bool DPP>
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t m) {
  if constexpr (!DPP) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    return m;
  }
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)m, 0);
  const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)m, 16);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)m, 32);
  const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)m, 48);
  return max(max(a, b), max(c, d));
}

// Scale of one group and how its quotients are evaluated.
struct GroupScale {
  float s;    // RN32(amax / 127)
  float rcp;  // RN32(1 / s)
  int mode;   // 0: all-zero group, 1: FMA quotient, 2: direct division
};

__device__ __forceinline__ GroupScale scale_from_s(float s) {
  GroupScale g;
  g.s = s;
  if (s == 0.0f) {
    g.rcp = 0.0f;
    g.mode = 0;
  } else if (s >= 0x1p-100f) {
    g.rcp = 1.0f / s;  // IEEE division (correctly rounded)
    g.mode = 1;
  } else {
    g.rcp = 0.0f;
    g.mode = 2;
  }
  return g;
}

// Code formats: 0 = INT8 (codes in [-127, 127]), 1 = FP8 E4M3 (OCP "e4m3fn",
// values in [-448, 448]).  The scale divides amax by the largest code.
template <int FMT>
constexpr float code_max() { return FMT == 1 ? 448.0f : 127.0f; }

// amax is the bit pattern of a non-negative bf16; the scale is
// RN32(amax / code max) (an IEEE division, correctly rounded), 0 only for
// amax = 0.
template <int FMT = 0>
__device__ __forceinline__ GroupScale make_scale(uint32_t amax_bits) {
  return scale_from_s(__uint_as_float(amax_bits << 16) / code_max<FMT>());
}

// Quotient x / s under a known evaluation mode (1: FMA form, 2: division).
template <int MODE>
__device__ __forceinline__ float quotient(float x, float s, float rcp) {
  if constexpr (MODE == 1) {
    const float q0 = x * rcp;
    const float e = __builtin_fmaf(-q0, s, x);
    return __builtin_fmaf(e, rcp, q0);
  } else {
    return x / s;
  }
}

// int8 code of x under scale s with a known mode (1 or 2), in the low byte
// of the result (the upper bytes are not part of the code).
//
// Round half to even: rounding is monotone and +-127 are integers, so
// clamping the quotient first gives the same code.  Adding 1.5 * 2^23 to a
// value in [-127, 127] rounds it to an integer n (ties to even: the added
// constant is even), and the sum's bit pattern is that of 1.5 * 2^23 plus n,
// so its low byte is n in two's complement.
//
// Stochastic rounding: u is the uniform in units of 2^-24 (word_uniform_units);
// u * 2^-24 is exact, so the FMA rounds v + u * 2^-24 once, exactly as the
// addition of the uniform would.
template <bool SR, int MODE>
__device__ __forceinline__ uint32_t code_of(float x, float s, float rcp, float u) {
  const float v = quotient<MODE>(x, s, rcp);
  if constexpr (SR) {
    return (uint32_t)(int)__builtin_amdgcn_fmed3f(floorf(__builtin_fmaf(u, 0x1p-24f, v)), -127.0f, 127.0f);
  } else {
    return __float_as_uint(__builtin_amdgcn_fmed3f(v, -127.0f, 127.0f) + 0x1.8p23f);
  }
}

// Any mode, decided per element (0 gives code 0).
template <bool SR>
__device__ __forceinline__ uint32_t code_any(float x, const GroupScale& g, float u) {
  if (g.mode == 1) return code_of<SR, 1>(x, g.s, g.rcp, u);
  if (g.mode == 2) return code_of<SR, 2>(x, g.s, g.rcp, u);
  return 0;
}

// FP8 value of x under scale s with a known mode (1 or 2): the quotient
// clamped to [-448, 448]; a zero x gives +0 (the FMA form already does: the
// quotient of -0 comes out +0).  v_cvt_pk_fp8_f32 then rounds it to the
// nearest E4M3 value, ties to even.
template <int MODE>
__device__ __forceinline__ float f8_value(float x, float s, float rcp) {
  if constexpr (MODE == 2) {
    if (x == 0.0f) return 0.0f;
  }
  return __builtin_amdgcn_fmed3f(quotient<MODE>(x, s, rcp), -448.0f, 448.0f);
}

__device__ __forceinline__ float f8_any(float x, const GroupScale& g) {
  if (g.mode == 1) return f8_value<1>(x, g.s, g.rcp);
  if (g.mode == 2) return f8_value<2>(x, g.s, g.rcp);
  return 0.0f;
}

// Four E4M3 codes, first value in the lowest byte.
__device__ __forceinline__ uint32_t pack_f8x4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Low bytes of four words, a's in the lowest byte.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return (a & 0xFFu) | ((b & 0xFFu) << 8) | ((c & 0xFFu) << 16) | (d << 24);
}

__device__ __forceinline__ float elem(const uint4& v, int j) {
  const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
  return (j & 1) ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
}

// Uniforms (in units of 2^-24) of the 8 elements starting at logical index
// e0.  ALIGNED4: e0 is a multiple of 4, so the chunk needs exactly two Philox
// blocks.
template <bool ALIGNED4>
__device__ __forceinline__ void chunk_uniforms(uint64_t seed, uint64_t offset, uint64_t e0,
                                               float u[8]) {
  if constexpr (ALIGNED4) {
    const uint64_t b = offset + (e0 >> 2);
    const u32x4 w0 = philox_block(seed, b);
    const u32x4 w1 = philox_block(seed, b + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = word_uniform_units(w0.w[j]);
      u[4 + j] = word_uniform_units(w1.w[j]);
    }
  } else {
    // Elements e0 .. e0+7 take words s .. s+7 (s = e0 mod 4) of the three
    // consecutive blocks from block offset + e0 / 4 on.  s is the same in
    // every lane of a wave where the callers call this (e0 = row * cols + a
    // multiple of 8); each element selects among its four candidate words,
    // all at constant indices.
    const uint64_t b = offset + (e0 >> 2);
    const u32x4 w0 = philox_block(seed, b), w1 = philox_block(seed, b + 1), w2 = philox_block(seed, b + 2);
    const uint32_t w[12] = {w0.w[0], w0.w[1], w0.w[2], w0.w[3], w1.w[0], w1.w[1],
                            w1.w[2], w1.w[3], w2.w[0], w2.w[1], w2.w[2], w2.w[3]};
    const uint32_t s = (uint32_t)(e0 & 3);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t word = s == 0 ? w[j] : s == 1 ? w[j + 1] : s == 2 ? w[j + 2] : w[j + 3];
      u[j] = word_uniform_units(word);
    }
  }
}

// Codes of one chunk.  MODE 1 or 2: every element uses that quotient form
// with scale g[0] (g[j] when PER_ELEM_SCALE); MODE -1: each element's own
// GroupScale decides.  Returns 8 bytes.
template <bool SR, bool ALIGNED4, bool PER_ELEM_SCALE, int MODE, int FMT = 0>
__device__ __forceinline__ uint2 quantize_chunk(const uint4& v, const GroupScale* g,
                                                uint64_t seed, uint64_t offset, uint64_t e0) {
  if constexpr (FMT == 1) {  // FP8: round to nearest only
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const GroupScale& gj = g[PER_ELEM_SCALE ? j : 0];
      if constexpr (MODE < 0)
        f[j] = f8_any(elem(v, j), gj);
      else
        f[j] = f8_value<MODE>(elem(v, j), gj.s, gj.rcp);
    }
    return make_uint2(pack_f8x4(f[0], f[1], f[2], f[3]), pack_f8x4(f[4], f[5], f[6], f[7]));
  }
  float u[8];
  if constexpr (SR) {
    chunk_uniforms<ALIGNED4>(seed, offset, e0, u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = 0.0f;
  }
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const GroupScale& gj = g[PER_ELEM_SCALE ? j : 0];
    if constexpr (MODE < 0)
      c[j] = code_any<SR>(elem(v, j), gj, u[j]);
    else
      c[j] = code_of<SR, MODE>(elem(v, j), gj.s, gj.rcp, u[j]);
  }
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

__device__ __forceinline__ void store_partial(int8_t* dst, uint2 codes, int n) {
  const uint64_t all = ((uint64_t)codes.y << 32) | codes.x;
  for (int j = 0; j < n; ++j) dst[j] = (int8_t)(all >> (8 * j));
}

}  // namespace
}  // namespace i8mp
