// A linear layer's INT8 GEMM (NT) with bias, activation and residual in its
// epilogue:
//   z[m,n] = float(acc) * sa[m] * sb[n] + bias[n],  y = act(z) + residual[m,n],
// all in fp32, y (and z, where it is kept for the backward) rounded once.
//
// The main loop is the pipelined GEMM's (gemm_pipelined.h).  As separate passes
// bias, activation and residual would read and write the M x N output up to three
// times more; here they cost the epilogue's arithmetic and the residual's one
// read.  The accumulators hold z between the two outputs, which go through the
// wave's own part of LDS one after the other to leave as whole row segments.  The
// residual's loads go out before anything else of the epilogue, in the
// accumulators' layout (8 bytes a lane; the four blocks of a row share its lines).
//
// Contractions that are no multiple of 16 are padded: whoever writes the first
// operand's codes fills the padding with zeros, and the second's padding may
// hold anything.
#include "activation.h"
#include "gemm_pipelined.h"

namespace i8mp {
namespace {

// Whole rows of a wave's WM x WN bf16 region of LDS (chunk c of row r at chunk
// c ^ (r mod chunks per row)) to memory.
template <int WM, int WN>
__device__ __forceinline__ void rows_out(const int8_t* mine, __bf16* __restrict__ C, int64_t ldc, int64_t mw, int64_t nw,
                                         int64_t M, int64_t N, int lane) {
  constexpr int CPR = WN / 8, PITCH = WN * 2, RPI = 64 / CPR;
  const int c = lane % CPR;
#pragma unroll 4
  for (int r0 = 0; r0 < WM; r0 += RPI) {
    const int r = r0 + lane / CPR;
    const uint4 v = *reinterpret_cast<const uint4*>(mine + r * PITCH + ((c ^ (r & (CPR - 1))) << 4));
    const int64_t m = mw + r, n = nw + 8 * c;
    if (m < M) {
      __bf16* dst = C + m * ldc + n;
      if (n + 8 <= N) {
        __builtin_nontemporal_store(__builtin_bit_cast(v4i, v), reinterpret_cast<v4i*>(dst));
      } else if (n < N) {
        const __bf16* hv = reinterpret_cast<const __bf16*>(&v);
        for (int e = 0; e < 8 && n + e < N; ++e) dst[e] = hv[e];
      }
    }
  }
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct ActEpilogue : Epilogue {
  template <int BM, int BN, int TM, int TN, bool VEC, int ACT, bool RES>
  __device__ __forceinline__ void run(v4i (&acc)[TM][TN], int64_t m0, int64_t n0, int wm, int wn, int64_t M, int64_t N,
                                      const float* s_lds, int8_t* stage, __bf16* __restrict__ C, int64_t ldc, int lane,
                                      int wave) const {
    constexpr int WM = 16 * TM, WN = 16 * TN, CPR = WN / 8, PITCH = WN * 2;
    int8_t* mine = stage + wave * (WM * PITCH);
    const int mr = lane & 15, q = lane >> 4;
    const int64_t mw = m0 + wm, nw = n0 + wn;
    uint2 res[RES ? TM : 1][RES ? TN : 1];
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int64_t m = mw + 16 * i + mr;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int64_t n4 = nw + 16 * j + 4 * q;
          res[i][j] = m < M && n4 < N ? *reinterpret_cast<const uint2*>(residual + m * ld_residual + n4) : make_uint2(0, 0);
        }
      }
    }
    // z in the accumulators' place
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const float4 sbq = *reinterpret_cast<const float4*>(s_lds + BM + wn + 16 * j + 4 * q);
      const float4 bq = *reinterpret_cast<const float4*>(s_lds + BM + BN + wn + 16 * j + 4 * q);
      const float sbv[4] = {sbq.x, sbq.y, sbq.z, sbq.w}, bv[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const float sam = s_lds[wm + 16 * i + mr];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = (float)acc[i][j][e] * sam;
          acc[i][j][e] = __float_as_int(__builtin_fmaf(y, sbv[e], bv[e]));
        }
      }
    }
    // one output: f(i, j, e) in the accumulators' layout
    auto out = [&](__bf16* __restrict__ dst, int64_t ld, auto f) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = 16 * i + mr;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          __bf16 h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = (__bf16)f(i, j, e);
          if constexpr (VEC) {
            const int chunk = 2 * j + (q >> 1);
            *reinterpret_cast<uint2*>(mine + r * PITCH + ((chunk ^ (r & (CPR - 1))) << 4) + 8 * (q & 1)) = __builtin_bit_cast(uint2, h);
          } else {
            const int64_t m = mw + r, n4 = nw + 16 * j + 4 * q;
            if (m < M) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n4 + e < N) dst[m * ld + n4 + e] = h[e];
            }
          }
        }
      }
      if constexpr (VEC) {  // the region is this wave's own, and its LDS operations stay in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        rows_out<WM, WN>(mine, dst, ld, mw, nw, M, N, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
    };
    if (z)
      out(reinterpret_cast<__bf16*>(z), ld_z, [&](int i, int j, int e) __attribute__((always_inline)) { return __int_as_float(acc[i][j][e]); });
    out(C, ldc, [&](int i, int j, int e) __attribute__((always_inline)) {
      float y = activation<ACT>(__int_as_float(acc[i][j][e]));
      if constexpr (RES) {
        const uint32_t w = e < 2 ? res[i][j].x : res[i][j].y;
        y += e & 1 ? hi_bf16(w) : lo_bf16(w);
      }
      return y;
    });
  }

  template <int BM, int BN, int TM, int TN, bool VEC>
  __device__ __forceinline__ void store(v4i (&acc)[TM][TN], int64_t m0, int64_t n0, int wm, int wn, int64_t M, int64_t N,
                                        const float* s_lds, int8_t* stage, __bf16* __restrict__ C, int64_t ldc, int lane,
                                        int wave) const {
#define I8MP_RUN(A)                                                                                                    \
  if (residual) run<BM, BN, TM, TN, VEC, A, true>(acc, m0, n0, wm, wn, M, N, s_lds, stage, C, ldc, lane, wave);        \
  else run<BM, BN, TM, TN, VEC, A, false>(acc, m0, n0, wm, wn, M, N, s_lds, stage, C, ldc, lane, wave);                \
  break
    switch (act) {
      case kActRelu: I8MP_RUN(kActRelu);
      case kActGelu: I8MP_RUN(kActGelu);
      case kActGeluTanh: I8MP_RUN(kActGeluTanh);
      case kActSilu: I8MP_RUN(kActSilu);
      default: I8MP_RUN(kActNone);
    }
#undef I8MP_RUN
  }
};

__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return activation<kActRelu>(z);
    case kActGelu: return activation<kActGelu>(z);
    case kActGeluTanh: return activation<kActGeluTanh>(z);
    case kActSilu: return activation<kActSilu>(z);
    default: return z;
  }
}

// The epilogue over the int32 partial planes of a split contraction (see
// splitk_reduce): one thread per 4 adjacent outputs of a row.
__global__ __launch_bounds__(256) void splitk_epilogue(const int32_t* __restrict__ P, int64_t ldp, int64_t plane, int splits,
                                                       int64_t M, int64_t N, const float* __restrict__ sa,
                                                       const float* __restrict__ sb, __bf16* __restrict__ C, int64_t ldc,
                                                       Epilogue epi) {
  const int64_t n = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (n >= N) return;
  const int left = (int)min(N - n, (int64_t)4);
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const int32_t* p = P + m * ldp + n;
    v4i acc = *reinterpret_cast<const v4i*>(p);
#pragma unroll 8
    for (int s = 1; s < splits; ++s) acc += *reinterpret_cast<const v4i*>(p + s * plane);
    const float sam = sa[m];
    uint2 res = make_uint2(0, 0);
    if (epi.residual) res = *reinterpret_cast<const uint2*>(epi.residual + m * epi.ld_residual + n);
    __bf16 h[4], hz[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float z = 0;
      if (e < left) z = __builtin_fmaf((float)acc[e] * sam, sb[n + e], epi.bias ? lo_bf16(epi.bias[n + e]) : 0.0f);
      hz[e] = (__bf16)z;
      float y = activate(epi.act, z);
      const uint32_t w = e < 2 ? res.x : res.y;
      if (epi.residual) y += e & 1 ? hi_bf16(w) : lo_bf16(w);
      h[e] = (__bf16)y;
    }
    for (int o = 0; o < 2; ++o) {
      __bf16* row = o ? reinterpret_cast<__bf16*>(epi.z) : C;
      if (!row) continue;
      const int64_t ld = o ? epi.ld_z : ldc;
      const bool vec = left == 4 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(row) % 8 == 0;
      row += m * ld + n;
      const __bf16* v = o ? hz : h;
      if (vec) *reinterpret_cast<uint2*>(row) = *reinterpret_cast<const uint2*>(v);
      else
        for (int e = 0; e < left; ++e) row[e] = v[e];
    }
  }
}

// Zeros into the padding of rows of codes: bytes [cols, ld) of each row, and
// whole rows [rows, rows_padded).
__global__ __launch_bounds__(256) void zero_padding(int8_t* __restrict__ q, int64_t rows, int64_t cols, int64_t ld) {
  const int64_t pad = ld - cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * pad; i += (int64_t)gridDim.x * 256)
    q[i / pad * ld + cols + i % pad] = 0;
}

template <int B, bool SIDE, bool VEC>
void launch_tiles(dim3 grid, int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa, const int8_t* Bp,
                  int64_t ldb, const float* sb, uint16_t* C, int64_t ldc, const ColmaxJob* side, const ActEpilogue& epi,
                  hipStream_t stream) {
  constexpr int WGN = B >= 256 ? 4 : 2;
  gemm_i8_pipelined<B, B, WGN, true, true, false, VEC, 0, SIDE, false, ActEpilogue><<<grid, 128 * WGN, 0, stream>>>(
      M, N, K, A, lda, sa, Bp, ldb, sb, C, ldc, K, 0, SIDE ? *side : ColmaxJob{}, epi);
}

template <int B>
hipError_t run_tiles(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa, const int8_t* Bp,
                     int64_t ldb, const float* sb, uint16_t* C, int64_t ldc, const ColmaxJob* side, const ActEpilogue& epi,
                     hipStream_t stream) {
  const int64_t tiles = ((M + B - 1) / B) * ((N + B - 1) / B);
  if (side && !side_fits(*side, tiles, B)) {
    const hipError_t e = launch_colmax_finalize(*side, stream);
    if (e != hipSuccess) return e;
    side = nullptr;
  }
  const auto rows16 = [](const void* p, int64_t ld) { return ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = rows16(C, ldc) && (!epi.z || rows16(epi.z, epi.ld_z));
  const dim3 grid((unsigned)tiles);
  if (side && vec) launch_tiles<B, true, true>(grid, M, N, K, A, lda, sa, Bp, ldb, sb, C, ldc, side, epi, stream);
  else if (side) launch_tiles<B, true, false>(grid, M, N, K, A, lda, sa, Bp, ldb, sb, C, ldc, side, epi, stream);
  else if (vec) launch_tiles<B, false, true>(grid, M, N, K, A, lda, sa, Bp, ldb, sb, C, ldc, side, epi, stream);
  else launch_tiles<B, false, false>(grid, M, N, K, A, lda, sa, Bp, ldb, sb, C, ldc, side, epi, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_zero_padding(int8_t* q, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
  const int64_t n = rows * (ld - cols);
  if (n <= 0) return hipSuccess;
  zero_padding<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0, stream>>>(q, rows, cols, ld);
  return hipGetLastError();
}

hipError_t launch_gemm_epilogue(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa,
                                const int8_t* B, int64_t ldb, const float* sb, uint16_t* C, int64_t ldc, const Epilogue& e,
                                void* ws, const ColmaxJob* side, hipStream_t stream) {
  if (side && side->n <= 0) side = nullptr;
  if (M == 0 || N == 0) return side ? launch_colmax_finalize(*side, stream) : hipSuccess;
  ActEpilogue epi;
  static_cast<Epilogue&>(epi) = e;
  const SplitPlan p = plan_split<true, true>(M, N, K, lda, ldb);
  if (p.splits < 2 || !ws)
    return big_tiles(M, N) >= kBigTileMin ? run_tiles<256>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, side, epi, stream)
                                          : run_tiles<128>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, side, epi, stream);
  const hipError_t err = launch_gemm_partials(M, N, K, A, lda, B, ldb, ws, side, stream);
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)((N + 1023) / 1024), (unsigned)std::min<int64_t>(M, 65535));
  splitk_epilogue<<<grid, 256, 0, stream>>>(static_cast<const int32_t*>(ws), p.ldp, M * p.ldp, p.splits, M, N, sa, sb,
                                            reinterpret_cast<__bf16*>(C), ldc, e);
  return hipGetLastError();
}

}  // namespace i8mp
