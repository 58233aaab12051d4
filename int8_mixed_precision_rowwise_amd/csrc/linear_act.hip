// A linear layer's INT8 GEMM (NT) with bias, activation and residual in its
// epilogue:
//   z[m,n] = float(acc) * sa[m] * sb[n] + bias[n],  y = act(z) + residual[m,n],
// all in fp32, y (and z, where it is kept for the backward) rounded once.
//
// The main loop is the pipelined GEMM's (gemm_pipelined.h).  As separate passes
// bias, activation and residual would read and write the M x N output up to three
// times more; here they cost the epilogue's arithmetic and the residual's one
// read.  Both outputs go through the wave's own part of LDS to leave as whole row
// segments, and the residual comes in the same way: its loads go out before
// anything else of the epilogue.
//
// Contractions that are no multiple of 16 are padded: whoever writes the first
// operand's codes fills the padding with zeros, and the second's padding may
// hold anything.
//
// Measured, this kernel alone, on several cards: 8192 x 5632 x 2048 with SiLU and the
// pre-activation kept 112 - 122 us, 8192 x 2048 x 5632 with the residual 79 - 86 us (1.6 and
// 2.3 Pop/s; 8192 cubed without an epilogue runs at 2.5, which would be 74 us for either).
// The first writes 185 MB behind its products, and one workgroup of 256 x 256 outputs fills
// a CU, so nothing overlaps them (smaller tiles, of which two fit, were not measured here).
#include "activation.h"
#include "gemm_pipelined.h"

namespace i8mp {
namespace {

// Rows of a wave's ROWS x WN bf16 region of LDS (16-byte chunk c of row r at
// chunk c ^ (r mod chunks per row)) to memory: 16 bytes a lane, or, for rows that
// start anywhere, one element a lane and row.
template <int ROWS, int WN, bool VEC>
__device__ __forceinline__ void rows_out(const int8_t* mine, __bf16* __restrict__ C, int64_t ldc, int64_t mw, int64_t nw,
                                         int64_t M, int64_t N, int lane) {
  constexpr int CPR = WN / 8, PITCH = WN * 2;
  if constexpr (VEC) {
    constexpr int RPI = 64 / CPR;
    const int c = lane % CPR;
    const int64_t n = nw + 8 * c;
    __bf16* dst = C + (mw + lane / CPR) * ldc + n;
#pragma unroll
    for (int r0 = 0; r0 < ROWS; r0 += RPI, dst += RPI * ldc) {
      const int r = r0 + lane / CPR;
      const uint4 v = *reinterpret_cast<const uint4*>(mine + r * PITCH + ((c ^ (r & (CPR - 1))) << 4));
      if (mw + r < M) {
        if (n + 8 <= N) {
          __builtin_nontemporal_store(__builtin_bit_cast(v4i, v), reinterpret_cast<v4i*>(dst));
        } else if (n < N) {
          const __bf16* hv = reinterpret_cast<const __bf16*>(mine + r * PITCH + ((c ^ (r & (CPR - 1))) << 4));
#pragma unroll 1
          for (int e = 0; n + e < N; ++e) dst[e] = hv[e];
        }
      }
    }
  } else {
    static_assert(WN == 64, "one column a lane");
    const int64_t n = nw + lane;
#pragma unroll 8
    for (int r = 0; r < ROWS; ++r) {
      const __bf16 v = *reinterpret_cast<const __bf16*>(mine + r * PITCH + (((lane >> 3) ^ (r & (CPR - 1))) << 4) + 2 * (lane & 7));
      if (mw + r < M && n < N) C[(mw + r) * ldc + n] = v;
    }
  }
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct ActEpilogue : Epilogue {
  // The wave's rows in two halves, so that its LDS holds both outputs of one:
  // y (where the residual's rows wait to be added) and z.
  template <int BM, int BN, int TM, int TN, bool VEC, int ACT, bool RES, bool KEEP>
  __device__ __forceinline__ void run(const v4i (&acc)[TM][TN], int64_t m0, int64_t n0, int wm, int wn, int64_t M, int64_t N,
                                      const float* s_lds, int8_t* stage, __bf16* __restrict__ C, int64_t ldc, int lane,
                                      int wave) const {
    constexpr int WM = 16 * TM, WN = 16 * TN, CPR = WN / 8, PITCH = WN * 2;
    constexpr int ROWS = WM / 2, RPI = 64 / CPR, LOADS = ROWS / RPI;
    int8_t* ybuf = stage + wave * (WM * PITCH);
    int8_t* zbuf = ybuf + ROWS * PITCH;
    const int mr = lane & 15, q = lane >> 4;
    const int64_t mw = m0 + wm, nw = n0 + wn;
    uint4 res[RES ? 2 * LOADS : 1];
    if constexpr (RES) {  // whole row segments, 16 bytes a lane; rows are padded to 16 bytes
      const int64_t n = nw + 8 * (lane % CPR);
      const uint16_t* src = residual + (mw + lane / CPR) * ld_residual + n;
#pragma unroll
      for (int k = 0; k < 2 * LOADS; ++k, src += RPI * ld_residual)
        res[k] = n < N && mw + k * RPI + lane / CPR < M ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (RES) {
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
          const int r = k * RPI + lane / CPR;
          *reinterpret_cast<uint4*>(ybuf + r * PITCH + (((lane % CPR) ^ (r & (CPR - 1))) << 4)) = res[h * LOADS + k];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const float4 sbq = *reinterpret_cast<const float4*>(s_lds + BM + wn + 16 * j + 4 * q);
        const float4 bq = *reinterpret_cast<const float4*>(s_lds + BM + BN + wn + 16 * j + 4 * q);
        const float sbv[4] = {sbq.x, sbq.y, sbq.z, sbq.w}, bv[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
        for (int ii = 0; ii < TM / 2; ++ii) {
          const int i = h * (TM / 2) + ii, r = 16 * ii + mr;
          const float sam = s_lds[wm + 16 * i + mr];
          const int off = r * PITCH + (((2 * j + (q >> 1)) ^ (r & (CPR - 1))) << 4) + 8 * (q & 1);
          float zv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) zv[e] = __builtin_fmaf((float)acc[i][j][e] * sam, sbv[e], bv[e]);
          if constexpr (KEEP) {
            const __bf16 hz[4] = {(__bf16)zv[0], (__bf16)zv[1], (__bf16)zv[2], (__bf16)zv[3]};
            *reinterpret_cast<uint2*>(zbuf + off) = __builtin_bit_cast(uint2, hz);
          }
          uint2 rv = make_uint2(0, 0);
          if constexpr (RES) rv = *reinterpret_cast<const uint2*>(ybuf + off);
          const float rf[4] = {lo_bf16(rv.x), hi_bf16(rv.x), lo_bf16(rv.y), hi_bf16(rv.y)};
          __bf16 hy[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = activation<ACT>(zv[e]);
            hy[e] = (__bf16)(RES ? y + rf[e] : y);
          }
          *reinterpret_cast<uint2*>(ybuf + off) = __builtin_bit_cast(uint2, hy);
        }
      }
      // the region is this wave's own, and its LDS operations stay in order
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      rows_out<ROWS, WN, VEC>(ybuf, C, ldc, mw + h * ROWS, nw, M, N, lane);
      if constexpr (KEEP) rows_out<ROWS, WN, VEC>(zbuf, reinterpret_cast<__bf16*>(z), ld_z, mw + h * ROWS, nw, M, N, lane);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }

  template <int BM, int BN, int TM, int TN, bool VEC>
  __device__ __forceinline__ void store(const v4i (&acc)[TM][TN], int64_t m0, int64_t n0, int wm, int wn, int64_t M, int64_t N,
                                        const float* s_lds, int8_t* stage, __bf16* __restrict__ C, int64_t ldc, int lane,
                                        int wave) const {
#define I8MP_RUN(A)                                                                                                    \
  if (residual) {                                                                                                      \
    if (z) run<BM, BN, TM, TN, VEC, A, true, true>(acc, m0, n0, wm, wn, M, N, s_lds, stage, C, ldc, lane, wave);       \
    else run<BM, BN, TM, TN, VEC, A, true, false>(acc, m0, n0, wm, wn, M, N, s_lds, stage, C, ldc, lane, wave);        \
  } else {                                                                                                             \
    if (z) run<BM, BN, TM, TN, VEC, A, false, true>(acc, m0, n0, wm, wn, M, N, s_lds, stage, C, ldc, lane, wave);      \
    else run<BM, BN, TM, TN, VEC, A, false, false>(acc, m0, n0, wm, wn, M, N, s_lds, stage, C, ldc, lane, wave);       \
  }                                                                                                                    \
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
  if (p.splits < 2 || !ws) {
    if (big_tiles(M, N) >= kBigTileMin && pipelined_ok<256, 256, true, true>(M, N, K, lda, ldb))
      return run_tiles<256>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, side, epi, stream);
    if (pipelined_ok<128, 128, true, true>(M, N, K, lda, ldb))
      return run_tiles<128>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, side, epi, stream);
    // rows too far apart for 32-bit offsets in a tile (a view of 16 MiB and more between
    // weight rows): the few-token kernel, whose addresses are whole, with the same bits
    if (side) {
      const hipError_t err = launch_colmax_finalize(*side, stream);
      if (err != hipSuccess) return err;
    }
    for (int64_t m = 0; m < M; m += kSkinnyRows) {
      Epilogue part = e;
      if (e.residual) part.residual = e.residual + m * e.ld_residual;
      if (e.z) part.z = e.z + m * e.ld_z;
      const hipError_t err = launch_skinny(std::min(M - m, kSkinnyRows), N, K, A + m * lda, lda, sa + m, B, ldb, sb, C + m * ldc, ldc,
                                           part, stream);
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  }
  const hipError_t err = launch_gemm_partials(M, N, K, A, lda, B, ldb, ws, side, stream);
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)((N + 1023) / 1024), (unsigned)std::min<int64_t>(M, 65535));
  splitk_epilogue<<<grid, 256, 0, stream>>>(static_cast<const int32_t*>(ws), p.ldp, M * p.ldp, p.splits, M, N, sa, sb,
                                            reinterpret_cast<__bf16*>(C), ldc, e);
  return hipGetLastError();
}

}  // namespace i8mp
