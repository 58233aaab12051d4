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
// LDS (exact in any order).
#include "activation.h"
#include "internal.h"

#include <algorithm>

namespace i8mp {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kSkWaves = 8, kSkThreads = 64 * kSkWaves;

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
  // one group of 4 adjacent outputs per thread and turn
  for (int o = threadIdx.x; o < MT * CT * 64; o += kSkThreads) {
    const int tile = o >> 6, l = o & 63;
    v4i s = red[0][tile][l];
#pragma unroll
    for (int w = 1; w < kSkWaves; ++w) s += red[w][tile][l];
    const int64_t m = 16 * (tile / CT) + (l & 15), n = n0 + 16 * (tile % CT) + 4 * (l >> 4);
    if (m >= a.M) continue;
    const float sam = a.sa[m];
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
void launch_skinny_tiles(const SkinnyArgs& a, hipStream_t stream) {
  skinny_gemm<MT, CT><<<(unsigned)((a.N + 16 * CT - 1) / (16 * CT)), kSkThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_skinny(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa, const int8_t* B,
                         int64_t ldb, const float* sb, uint16_t* C, int64_t ldc, const Epilogue& e, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  const SkinnyArgs a{A, B, sa, sb, C, M, N, K, lda, ldb, ldc, e};
  switch ((M + 15) / 16) {
    case 1: launch_skinny_tiles<1, 1>(a, stream); break;
    case 2: launch_skinny_tiles<2, 1>(a, stream); break;
    case 3: launch_skinny_tiles<3, 2>(a, stream); break;
    default: launch_skinny_tiles<4, 2>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace i8mp
