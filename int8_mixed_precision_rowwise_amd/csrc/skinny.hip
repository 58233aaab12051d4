// A few tokens against a weight matrix of INT8 codes: Y = act(X W^T + bias) +
// residual for up to 64 rows of X.
//
// The weights are read once and everything else is small, so the kernel is
// bound by reading them.  A workgroup takes 16 CT columns of the output (rows of
// W) and all rows of X; its 8 waves share the contraction, wave w taking every
// eighth step of 64 codes, so that the workgroup reads 512 adjacent bytes of each
// weight row at a time and a short output still spreads over many waves.  Weights
// go from memory straight into the matrix instruction's registers: lane l holds
// 16 codes of row l % 16 at step offset 16 (l / 16), which is what
// v_mfma_i32_16x16x64_i8 wants of an operand.  The waves' int32 sums are joined in
// LDS (exact in any order).  One token against 14336 x 4096 codes: 15.7 us with the
// token's quantization (3.7 TB/s; the launch, the first weights' way and the join are 4
// of them), 64 tokens 35 us, where every workgroup reads all of X's codes again: twice the
// weights' bytes, from the cache.
#include "activation.h"
#include "internal.h"
#include "quant_device.h"

#include <algorithm>

namespace i8mp {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kSkWaves = 8, kSkThreads = 64 * kSkWaves;
// Chunks of X, 8 values each, that a thread quantizes at most.  Every workgroup
// does this work again, so it has to stay small against reading the weights.
// Both sides, all the call's kernels (a separate quantization is one more): one row against
// 14336 x 4096 codes (a chunk a thread) 16 us and 20, 8 rows (8 chunks) 19.5 and 20.7;
// 4 rows against 5003 x 2040 (2) 6.4 us and 8.8, 13 rows (8) 9.8 and 9.9.
constexpr int kSkChunks = 8;

// One tile of columns a workgroup while each CU gets at most one workgroup; beyond
// that two, which halve the reads of X's codes (every workgroup takes them from the
// cache) and the workgroups that quantize X.  Both sides, two tiles and one, all the
// call's kernels.  X quantized in the kernel: 1 row against 5003 x 2040 5.8 us and 7.7, 13
// rows 9.7 and 13.7, 8 rows against 6000 x 4096 12.3 and 13.5, 16 against 8191 x 2048
// 10.0 and 14.2, 8 against 14336 x 4096 19.8 and 24.8 (only 1 to 4 rows against
// 8191 x 4096 are better off with one: 10.4 and 9.2, 11.7 and 10.7).  Separately: 13 rows
// against 14336 x 4096 21.8 and 24.4, 64 rows 35.0 and 49.6, 64 against 5003 x 2040 13.8 and
// 17.3.  Up to 4096 columns, the other way: 13 against 4096 x 14336 34.5 and 26.7, 64
// rows 58.2 and 49.8, 1 row against 4096 x 4096 8.0 and 6.4.
constexpr int64_t kSkWideN = 16 * 256;

struct SkinnyArgs {
  const int8_t *A, *B;  // codes of X [M x K] and W [N x K]
  const float *sa, *sb;
  uint16_t* C;
  int64_t M, N, K, lda, ldb, ldc;
  Epilogue epi;
};

// The first n bytes of 16 (none for n <= 0).
__device__ __forceinline__ v4i first_bytes(v4i v, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    v[i] &= left >= 4 ? -1 : left <= 0 ? 0 : (int)((1u << (8 * left)) - 1u);
  }
  return v;
}

__device__ __forceinline__ float bf16_at(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }

__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return activation<kActRelu>(z);
    case kActGelu: return activation<kActGelu>(z);
    case kActGeluTanh: return activation<kActGeluTanh>(z);
    case kActSilu: return activation<kActSilu>(z);
    default: return z;
  }
}

// The waves' sums joined and finished; sa: scales of the rows of X.
template <int MT, int CT>
__device__ __forceinline__ void write_outputs(const SkinnyArgs& a, const v4i (*red)[MT * CT][64], const float* sa, int64_t n0) {
  // one group of 4 adjacent outputs per thread and turn
  for (int o = threadIdx.x; o < MT * CT * 64; o += kSkThreads) {
    const int tile = o >> 6, l = o & 63;
    v4i s = red[0][tile][l];
#pragma unroll
    for (int w = 1; w < kSkWaves; ++w) s += red[w][tile][l];
    const int64_t m = 16 * (tile / CT) + (l & 15), n = n0 + 16 * (tile % CT) + 4 * (l >> 4);
    if (m >= a.M) continue;
    const float sam = sa[m];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= a.N) break;
      const float z = __builtin_fmaf((float)s[e] * sam, a.sb[n + e], a.epi.bias ? bf16_at(a.epi.bias, n + e) : 0.0f);
      float y = activate(a.epi.act, z);
      if (a.epi.residual) y += bf16_at(a.epi.residual, m * a.epi.ld_residual + n + e);
      reinterpret_cast<__bf16*>(a.C)[m * a.ldc + n + e] = (__bf16)y;
      if (a.epi.z) reinterpret_cast<__bf16*>(a.epi.z)[m * a.epi.ld_z + n + e] = (__bf16)z;
    }
  }
}

template <int MT, int CT>
__global__ __launch_bounds__(kSkThreads) void skinny_gemm(SkinnyArgs a) {
  constexpr int U = MT * CT >= 8 ? 2 : 4;  // steps in flight per wave
  __shared__ __attribute__((aligned(16))) v4i red[kSkWaves][MT * CT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * CT;
  const int8_t *pa[MT], *pb[CT];  // rows past the last one repeat it: their outputs are not stored
#pragma unroll
  for (int i = 0; i < MT; ++i) pa[i] = a.A + min((int64_t)(16 * i + li), a.M - 1) * a.lda;
#pragma unroll
  for (int j = 0; j < CT; ++j) pb[j] = a.B + min(n0 + 16 * j + li, a.N - 1) * a.ldb;
  v4i acc[MT][CT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
  const int K = (int)a.K;
  for (int s0 = wave * 64; s0 < K; s0 += U * kSkWaves * 64) {
    v4i fa[U][MT], fb[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = s0 + u * kSkWaves * 64 + 16 * q;
      const bool in = k < K;
#pragma unroll
      for (int j = 0; j < CT; ++j) fb[u][j] = in ? *reinterpret_cast<const v4i*>(pb[j] + k) : (v4i){0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[u][i] = in ? *reinterpret_cast<const v4i*>(pa[i] + k) : (v4i){0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = s0 + u * kSkWaves * 64 + 16 * q;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        // codes behind the row's end are whatever its padding holds: one operand drops them
        if (k + 16 > K) fa[u][i] = first_bytes(fa[u][i], K - k);
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][j], fa[u][i], acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) red[wave][i * CT + j][lane] = acc[i][j];
  __syncthreads();
  write_outputs<MT, CT>(a, red, a.sa, n0);
}

// The same from X itself, for up to 16 short rows: every workgroup quantizes them
// (as quantize_rowwise does) into LDS while its first weights are on the way.
// Of the 8 waves, kSkWaves / G rows' worth of G waves each share a row.
template <int Q, int CT>
__global__ __launch_bounds__(kSkThreads) void skinny_raw(SkinnyArgs a, const uint16_t* __restrict__ x, int64_t ldx, int G, int C,
                                                         int stride) {
  constexpr int U = 8 / CT;  // steps in flight per wave
  __shared__ __attribute__((aligned(16))) v4i red[kSkWaves][CT][64];
  __shared__ uint32_t amax[16];
  __shared__ float sx[16];
  extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // [M][stride]
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int li = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * CT;
  const int K = (int)a.K, M = (int)a.M;
  // chunk i of a thread: of row row0 + (i / C) rows, 8 values from column 8 (col + (i % C) 64 G)
  const int rows = kSkWaves / G, row0 = wave / G, col = (wave % G) * 64 + lane;
  uint4 v[Q];
#pragma unroll
  for (int i = 0, r = row0, c = col, n = 0; i < Q; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < M && 8 * c < K) v[i] = *reinterpret_cast<const uint4*>(x + r * ldx + 8 * c);
    c += 64 * G;
    if (++n == C) n = 0, c = col, r += rows;
  }
  const int8_t* pb[CT];  // rows past the last one repeat it: their outputs are not stored
#pragma unroll
  for (int j = 0; j < CT; ++j) pb[j] = a.B + min(n0 + 16 * j + li, a.N - 1) * a.ldb;
  v4i fb[U][CT];
  // steps past the row's end read its last codes again, against zeros of X: no branch around a load
  const int last = (K - 1) & ~15;
  const auto load = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < CT; ++j) fb[u][j] = *reinterpret_cast<const v4i*>(pb[j] + min(s0 + u * kSkWaves * 64 + 16 * q, last));
  };
  load(wave * 64);
  if (t < 16) amax[t] = 0;
  __syncthreads();
  us2 m2 = {0, 0};
#pragma unroll
  for (int i = 0, r = row0, c = col, n = 0; i < Q; ++i) {
    if (8 * c + 8 > K) v[i] = keep_first(v[i], max(0, K - 8 * c));
    m2 = absmax_bits(m2, v[i]);
    c += 64 * G;
    if (++n == C || i == Q - 1) {
      const uint32_t m = wave_max_u32<true>(max((uint32_t)m2.x, (uint32_t)m2.y));
      if (lane == 0 && r < M) atomicMax(amax + r, m);
      m2 = (us2){0, 0};
      n = 0, c = col, r += rows;
    }
  }
  __syncthreads();
  if (t < M) sx[t] = make_scale(amax[t]).s;
#pragma unroll
  for (int i = 0, r = row0, c = col, n = 0; i < Q; ++i) {
    if (r < M && 8 * c < stride) {
      const GroupScale g = make_scale(__builtin_amdgcn_readfirstlane(amax[r]));
      const uint2 w = g.mode == 1 ? quantize_chunk<false, true, false, 1>(v[i], &g, 0, 0, 0)
                                  : quantize_chunk<false, true, false, -1>(v[i], &g, 0, 0, 0);
      *reinterpret_cast<uint2*>(codes + r * stride + 8 * c) = w;
    }
    c += 64 * G;
    if (++n == C) n = 0, c = col, r += rows;
  }
  __syncthreads();
  const int8_t* pa = codes + min(li, M - 1) * stride;
  v4i acc[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) acc[j] = (v4i){0, 0, 0, 0};
  const auto add = [&](const v4i(&w)[U][CT], int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = s0 + u * kSkWaves * 64 + 16 * q;
      v4i fa = *reinterpret_cast<const v4i*>(pa + min(k, last));
      if (k + 16 > K) fa = first_bytes(fa, K - k);
#pragma unroll
      for (int j = 0; j < CT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][j], fa, acc[j], 0, 0, 0);
    }
  };
  int s0 = wave * 64;
  for (; s0 + U * kSkWaves * 64 < K; s0 += U * kSkWaves * 64) {
    v4i w[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < CT; ++j) w[u][j] = fb[u][j];
    load(s0 + U * kSkWaves * 64);
    add(w, s0);
  }
  add(fb, s0);
#pragma unroll
  for (int j = 0; j < CT; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  write_outputs<1, CT>(a, red, sx, n0);
}

template <int MT>
void launch_skinny_tiles(const SkinnyArgs& a, hipStream_t stream) {
  if (a.N > kSkWideN)
    skinny_gemm<MT, 2><<<(unsigned)((a.N + 31) / 32), kSkThreads, 0, stream>>>(a);
  else
    skinny_gemm<MT, 1><<<(unsigned)((a.N + 15) / 16), kSkThreads, 0, stream>>>(a);
}

// G waves a row of X, and chunks of it a thread.
int skinny_group(int64_t M) { return M <= 1 ? 8 : M <= 2 ? 4 : M <= 4 ? 2 : 1; }
int skinny_chunks(int64_t M, int64_t K) { return (int)((K + 511) / 512 + skinny_group(M) - 1) / skinny_group(M); }

}  // namespace

hipError_t launch_skinny(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa, const int8_t* B,
                         int64_t ldb, const float* sb, uint16_t* C, int64_t ldc, const Epilogue& e, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  const SkinnyArgs a{A, B, sa, sb, C, M, N, K, lda, ldb, ldc, e};
  switch ((M + 15) / 16) {
    case 1: launch_skinny_tiles<1>(a, stream); break;
    case 2: launch_skinny_tiles<2>(a, stream); break;
    case 3: launch_skinny_tiles<3>(a, stream); break;
    default: launch_skinny_tiles<4>(a, stream);
  }
  return hipGetLastError();
}

// M rows in turns of kSkWaves / G, each of `chunks` chunks a thread: as many as registers hold.
bool skinny_takes_x(int64_t M, int64_t K) {
  if (M < 1 || M > 16 || K < 1) return false;
  const int turns = (int)(M * skinny_group(M) + kSkWaves - 1) / kSkWaves;
  return skinny_chunks(M, K) <= kSkChunks / turns;
}

hipError_t launch_skinny_raw(int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const int8_t* B, int64_t ldb,
                             const float* sb, uint16_t* C, int64_t ldc, const Epilogue& e, hipStream_t stream) {
  const SkinnyArgs a{nullptr, B, nullptr, sb, C, M, N, K, 0, ldb, ldc, e};
  const int G = skinny_group(M), per = skinny_chunks(M, K), turns = (int)(M * G + kSkWaves - 1) / kSkWaves;
  const int stride = (int)((K + 15) / 16 * 16 + 16);  // 16 more: rows start in different banks
  const size_t lds = (size_t)M * stride;
  const int held = per * turns <= 2 ? 2 : per * turns <= 4 ? 4 : kSkChunks;
  switch (held + (N > kSkWideN)) {
    case 2: skinny_raw<2, 1><<<(unsigned)((N + 15) / 16), kSkThreads, lds, stream>>>(a, X, ldx, G, per, stride); break;
    case 3: skinny_raw<2, 2><<<(unsigned)((N + 31) / 32), kSkThreads, lds, stream>>>(a, X, ldx, G, per, stride); break;
    case 4: skinny_raw<4, 1><<<(unsigned)((N + 15) / 16), kSkThreads, lds, stream>>>(a, X, ldx, G, per, stride); break;
    case 5: skinny_raw<4, 2><<<(unsigned)((N + 31) / 32), kSkThreads, lds, stream>>>(a, X, ldx, G, per, stride); break;
    case 8: skinny_raw<8, 1><<<(unsigned)((N + 15) / 16), kSkThreads, lds, stream>>>(a, X, ldx, G, per, stride); break;
    default: skinny_raw<8, 2><<<(unsigned)((N + 31) / 32), kSkThreads, lds, stream>>>(a, X, ldx, G, per, stride);
  }
  return hipGetLastError();
}

}  // namespace i8mp
