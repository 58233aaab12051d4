// Scaled INT8 GEMM for gfx950 in the three layouts of a linear layer's
// training step ("Quantized model training", section "Speed benchmarks >
// Matmul": A @ B.T, A @ B, A.T @ B; section "INT8 mixed precision training":
// scaled INT8 matmul after dynamic row-wise quantization):
//   acc[m,n] = sum_k A(m,k) B(k,n)   int8 x int8 -> int32 (exact)
//   C[m,n]   = bf16_RNE(RN32(RN32(float(acc)) * sa[m]) * sb[n])
// or the raw int32 accumulators.
//
// Structure: one workgroup per BM x BN output tile, K in slabs of 64 bytes
// through LDS.  Two kernels: a pipelined one (slabs loaded memory -> LDS by
// the buffer unit, several slabs in flight; v_mfma_i32_16x16x64_i8 on 16 x 16
// blocks; 8 waves for 256 x 256 tiles, 4 for 128 x 128) for contraction
// lengths that are multiples of 16, and a register-staged double-buffered one
// (4 waves, v_mfma_i32_32x32x32_i8 on 32 x 32 blocks) for every other shape.
// The linear chains may split a long contraction of a few-tile output over
// several copies of the tile grid (int32 partial planes, then splitk_reduce).
// An operand whose contraction dimension is contiguous in memory (A in NT and
// NN, B in NT) is staged K-major and fed to the MFMA with ds_read_b128; an
// operand whose contraction runs down its rows (B in NN and TN, A in TN) is
// staged in its storage orientation and transposed on the way out of LDS by
// ds_read_b64_tr_b8, so no transposed copy is ever written to memory.
//
// ds_read_b64_tr_b8: within each group of 16 lanes, lane i receives byte j
// from byte (i mod 8) of the 8 bytes addressed by lane 2j + i/8.  When lane
// 2j + h of a group addresses row k0 + j, columns n0 + 8h .. n0 + 8h + 7 of
// a [k][n] tile, lane i therefore receives column n0 + i at rows k0 .. k0+7.
//
// MFMA 32x32x32 i8 operand/result layout: lane l supplies row l % 32 of its
// first operand block and column l % 32 of its second with 16 contraction
// values in k order (k = 16 * (l / 32) + 0..15 of the 32-wide step); result
// register v of lane l holds row 8 * (v / 4) + 4 * (l / 32) + v % 4 (an index
// of the first operand), column l % 32 (of the second).
#include "gemm_pipelined.h"

#include <algorithm>

namespace i8mp {
namespace {

// Keep the first n (0..16) bytes of a 16-byte chunk.
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : ((1u << (8 * left)) - 1u);
    w[i] &= mask;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Global -> register staging of one BK-deep slab of an operand tile.
//   KMAJOR: R rows (output rows or columns) of BK contraction bytes, row r at
//           p[(mn0 + r) * ld + k0 ..]
//   else:   BK rows of R bytes, row k at p[(k0 + k) * ld + mn0 ..]
template <int R, bool KMAJOR>
struct Stager {
  static constexpr int kChunks = R * BK / 16 / kThreads;  // 16-byte chunks per thread
  uint4 v[kChunks];

  __device__ __forceinline__ void load(const int8_t* __restrict__ p, int64_t ld, int64_t mn0,
                                       int64_t MN, int64_t k0, int64_t K, int t) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * kThreads + t;
      if constexpr (KMAJOR) {
        const int r = id >> 2, c = id & 3;
        const int64_t kk = k0 + 16 * c;
        if (mn0 + r < MN && kk < K) {
          v[i] = *reinterpret_cast<const uint4*>(p + (mn0 + r) * ld + kk);
          if (kk + 16 > K) v[i] = keep_bytes(v[i], (int)(K - kk));
        } else {
          v[i] = make_uint4(0, 0, 0, 0);
        }
      } else {
        constexpr int CPR = R / 16;  // chunks per row
        const int k = id / CPR, c = id % CPR;
        const int64_t mm = mn0 + 16 * c;
        // bytes past MN inside a chunk only reach outputs that are never stored
        if (k0 + k < K && mm < MN)
          v[i] = *reinterpret_cast<const uint4*>(p + (k0 + k) * ld + mm);
        else
          v[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }

  __device__ __forceinline__ void store(int8_t* lds, int t) const {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * kThreads + t;
      int off;
      if constexpr (KMAJOR) {
        off = kmajor_off(id >> 2, id & 3);
      } else {
        constexpr int CPR = R / 16;
        off = mnmajor_off<R>(id / CPR, id % CPR);
      }
      *reinterpret_cast<uint4*>(lds + off) = v[i];
    }
  }
};

// MFMA operand (16 contraction bytes) for 32-row block `blk0` (row offset
// within the tile) at contraction step kk (0 or 1) of the slab.
template <int R, bool KMAJOR>
__device__ __forceinline__ v4i frag(const int8_t* lds, int blk0, int kk, int lane) {
  if constexpr (KMAJOR) {
    const int r = blk0 + (lane & 31);
    const int c = 2 * kk + (lane >> 5);
    return *reinterpret_cast<const v4i*>(lds + kmajor_off(r, c));
  } else {
    const int g = lane >> 4, li = lane & 15;
    const int n16 = blk0 + 16 * (g & 1);      // 16 output rows/cols of this lane group
    const int kb = 32 * kk + 16 * (g >> 1);   // 16 contraction rows of this lane group
    const int krow = kb + (li >> 1);
    const int c = n16 >> 4;
    const int half = (li & 1) << 3;
    const v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (lds_v2i*)(lds + mnmajor_off<R>(krow, c) + half));
    const v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (lds_v2i*)(lds + mnmajor_off<R>(krow + 8, c) + half));
    v4i out;
    out.x = lo.x;
    out.y = lo.y;
    out.z = hi.x;
    out.w = hi.y;
    return out;
  }
}

// Scales of the workgroup's BM rows and BN columns, staged in LDS once so
// the epilogue reads them with ds_read (global loads would have to wait
// behind the output stores, which share the vector-memory counter).
template <int BM, int BN, bool OUT_I32>
__device__ __forceinline__ void stage_scales(float* s_lds, int64_t m0, int64_t n0, int64_t M,
                                             int64_t N, const float* __restrict__ sa,
                                             const float* __restrict__ sb, int t) {
  if constexpr (!OUT_I32) {
    for (int i = t; i < BM + BN; i += kThreads) {
      float v = 0.0f;
      if (i < BM) {
        if (m0 + i < M) v = sa[m0 + i];
      } else if (n0 + (i - BM) < N) {
        v = sb[n0 + (i - BM)];
      }
      s_lds[i] = v;
    }
  }
  __syncthreads();
}

// Epilogue of one wave's TM x TN blocks of 32 x 32 accumulators whose
// top-left output is (mw, nw) = tile origin + (wm, wn).  The MFMAs take the
// B fragment as their first operand, so in block (i, j) lane l holds output
// row m = mw + 32i + l % 32 and register v holds column
// n = nw + 32j + 8(v / 4) + 4(l / 32) + v % 4: four consecutive registers
// are four adjacent outputs of one row, stored together (8 bytes of bf16 or
// 16 bytes of int32) when VEC.  y = RN(RN(float(acc) * sa[m]) * sb[n]).
// s_lds holds sa[tile rows] then sb[tile columns].
template <int BM, int TM, int TN, bool OUT_I32, bool VEC>
__device__ __forceinline__ void store_tile(const v16i (&acc)[TM][TN], int64_t m0, int64_t n0,
                                           int wm, int wn, int64_t M, int64_t N,
                                           const float* s_lds, void* __restrict__ Cv,
                                           int64_t ldc, int lane) {
  const int mr = lane & 31, nq = 4 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < TN; ++j) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + wm + 32 * i + mr;
      if (m >= M) continue;
      float sam = 0.0f;
      if constexpr (!OUT_I32) sam = s_lds[wm + 32 * i + mr];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int cn = wn + 32 * j + 8 * q + nq;  // column within the tile
        const int64_t n4 = n0 + cn;
        if (n4 >= N) continue;
        if constexpr (OUT_I32) {
          int32_t* row = static_cast<int32_t*>(Cv) + m * ldc;
          if (VEC && n4 + 4 <= N) {
            *reinterpret_cast<v4i*>(row + n4) =
                (v4i){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n4 + e < N) row[n4 + e] = acc[i][j][4 * q + e];
          }
        } else {
          const float4 sbq = *reinterpret_cast<const float4*>(s_lds + BM + cn);
          const float sbv[4] = {sbq.x, sbq.y, sbq.z, sbq.w};
          __bf16 h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = (float)acc[i][j][4 * q + e];
            y = y * sam;
            y = y * sbv[e];
            h[e] = (__bf16)y;  // round to nearest even
          }
          __bf16* row = static_cast<__bf16*>(Cv) + m * ldc;
          if (VEC && n4 + 4 <= N) {
            *reinterpret_cast<uint2*>(row + n4) = __builtin_bit_cast(uint2, h);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n4 + e < N) row[n4 + e] = h[e];
          }
        }
      }
    }
  }
}

template <int BM, int BN, bool A_KMAJOR, bool B_KMAJOR, bool OUT_I32, bool VEC>
__global__ __launch_bounds__(kThreads) void gemm_i8_general(int64_t M, int64_t N, int64_t K,
                                                    const int8_t* __restrict__ A, int64_t lda,
                                                    const float* __restrict__ sa,
                                                    const int8_t* __restrict__ B, int64_t ldb,
                                                    const float* __restrict__ sb,
                                                    void* __restrict__ Cv, int64_t ldc) {
  constexpr int WM = BM / 2, WN = BN / 2;  // 2 x 2 waves
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
  __shared__ __attribute__((aligned(16))) int8_t lds[2 * (A_BYTES + B_BYTES)];

  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + BN - 1) / BN);
  int tm, tn;
  tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wm0 = (wave >> 1) * WM, wn0 = (wave & 1) * WN;

  v16i acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = (v16i){};

  Stager<BM, A_KMAJOR> sa_stage;
  Stager<BN, B_KMAJOR> sb_stage;
  const int nk = (int)((K + BK - 1) / BK);
  if (nk > 0) {
    sa_stage.load(A, lda, m0, M, 0, K, t);
    sb_stage.load(B, ldb, n0, N, 0, K, t);
    sa_stage.store(lds, t);
    sb_stage.store(lds + A_BYTES, t);
  }
  __syncthreads();

  for (int kt = 0; kt < nk; ++kt) {
    int8_t* cur = lds + (kt & 1) * (A_BYTES + B_BYTES);
    int8_t* nxt = lds + ((kt & 1) ^ 1) * (A_BYTES + B_BYTES);
    const bool more = kt + 1 < nk;
    if (more) {
      sa_stage.load(A, lda, m0, M, (int64_t)(kt + 1) * BK, K, t);
      sb_stage.load(B, ldb, n0, N, (int64_t)(kt + 1) * BK, K, t);
    }
#pragma unroll
    for (int kk = 0; kk < BK / 32; ++kk) {
      v4i af[TM], bf[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) af[i] = frag<BM, A_KMAJOR>(cur, wm0 + 32 * i, kk, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) bf[j] = frag<BN, B_KMAJOR>(cur + A_BYTES, wn0 + 32 * j, kk, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[j], af[i], acc[i][j], 0, 0, 0);
    }
    if (more) {
      sa_stage.store(nxt, t);
      sb_stage.store(nxt + A_BYTES, t);
    }
    __syncthreads();
  }

  // every wave has passed its last LDS read of the slabs before any scale lands
  __syncthreads();
  float* s_lds = reinterpret_cast<float*>(lds);
  stage_scales<BM, BN, OUT_I32>(s_lds, m0, n0, M, N, sa, sb, t);
  store_tile<BM, TM, TN, OUT_I32, VEC>(acc, m0, n0, wm0, wn0, M, N, s_lds, Cv, ldc, lane);
}


// ---- matrix-core throughput probe ------------------------------------------
//
// The INT8 GEMM's matrix-core work with everything else taken away: the
// GEMM's launch shape (256 workgroups of 8 waves, two waves per SIMD) and its
// per-wave tile (8 x 4 blocks of 16 x 16, 128 accumulator registers), with the
// operands in registers.  Each wave loads two slabs' worth of fragments (real
// codes, so the operand bits toggle as in the GEMM) once, then issues
// `rounds` x 2 x 32 v_mfma_i32_16x16x64_i8, alternating the two fragment sets.
// Measures how fast the chip runs this work under its power limit.
__global__ __launch_bounds__(512) void mfma_rate_probe(const int8_t* __restrict__ codes, int64_t span,
                                                       int64_t rounds, int32_t* __restrict__ sink) {
  const int t = threadIdx.x, lane = t & 63;
  const int64_t wave = (int64_t)blockIdx.x * 8 + (t >> 6);
  // this wave's 24 fragments of 1 KiB, consecutive in the codes (wrapping)
  const int8_t* base = codes + (wave * 24 * 1024) % span;
  v4i a0[8], b0[4], a1[8], b1[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a0[i] = *reinterpret_cast<const v4i*>(base + i * 1024 + lane * 16);
    a1[i] = *reinterpret_cast<const v4i*>(base + (12 + i) * 1024 + lane * 16);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    b0[j] = *reinterpret_cast<const v4i*>(base + (8 + j) * 1024 + lane * 16);
    b1[j] = *reinterpret_cast<const v4i*>(base + (20 + j) * 1024 + lane * 16);
  }
  v4i acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
  for (int64_t r = 0; r < rounds; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0[j], a0[i], acc[i][j], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1[j], a1[i], acc[i][j], 0, 0, 0);
  }
  int32_t h = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) h ^= acc[i][j].x ^ acc[i][j].y ^ acc[i][j].z ^ acc[i][j].w;
  sink[(int64_t)blockIdx.x * 512 + t] = h;
}

template <int BM, int BN, bool AK, bool BKM, bool OUT_I32, bool VEC>
void launch(bool fast, bool rebase, dim3 grid, int64_t M, int64_t N, int64_t K, const int8_t* A,
            int64_t lda, const float* sa, const int8_t* B, int64_t ldb, const float* sb, void* C,
            int64_t ldc, const ColmaxJob* side, hipStream_t stream) {
  // 256 x 256 tiles: 8 waves (2 per SIMD, 128 x 64 each) so one wave's MFMAs
  // run while the other waits on its slab-load issue; 128 x 128: 4 waves.
  // side (pipelined kernel only) is a column-maxima reduction the caller has
  // checked fits (side_fits).  rebase: the pipelined kernel with per-slab
  // descriptors (rebase_ok; 256 x 256 tiles, packed bf16 output only).
  constexpr int WGN = BM >= 256 ? 4 : 2;
  if (fast && side)
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, OUT_I32, VEC, 0, true><<<grid, 128 * WGN, 0, stream>>>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, K, 0, *side, NoEpilogue{});
  else if (fast)
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, OUT_I32, VEC><<<grid, 128 * WGN, 0, stream>>>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, K, 0, ColmaxJob{}, NoEpilogue{});
  else if (rebase && BM == 256 && !OUT_I32 && VEC && !(AK && BKM)) {
    if constexpr (BM == 256 && !OUT_I32 && VEC && !(AK && BKM))
      gemm_i8_pipelined<BM, BN, WGN, AK, BKM, false, true, 0, false, true><<<grid, 128 * WGN, 0, stream>>>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, K, 0, ColmaxJob{}, NoEpilogue{});
  } else
    gemm_i8_general<BM, BN, AK, BKM, OUT_I32, VEC><<<grid, kThreads, 0, stream>>>(M, N, K, A, lda, sa, B, ldb, sb, C, ldc);
}

// Whether the pipelined kernel with per-slab descriptors (REBASE) takes a
// problem the plain form cannot because an operand read down its rows spans
// 2^31 bytes or more (e.g. a grad-weight GEMM over a wide output at many
// tokens): 256 x 256 tiles, the same shape rules, and each slab (BK rows of
// such an operand) within 32-bit offsets.
template <int BM, int BN, bool AK, bool BKM>
bool rebase_ok(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
  if (BM != 256 || (AK && BKM)) return false;
  const int64_t lim = int64_t(1) << 31;
  const int64_t a_ext = AK ? (int64_t)BM * lda : (int64_t)BK * lda;
  const int64_t b_ext = BKM ? (int64_t)BN * ldb : (int64_t)BK * ldb;
  const bool mn_ok = (AK || M % 4 == 0) && (BKM || N % 4 == 0);
  return K > 0 && K % 16 == 0 && a_ext < lim - 1024 && b_ext < lim - 1024 && mn_ok &&
         !pipelined_ok<BM, BN, AK, BKM>(M, N, K, lda, ldb);
}

template <int BM, int BN, bool AK, bool BKM>
hipError_t run(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa,
               const int8_t* B, int64_t ldb, const float* sb, uint16_t* Cb, int32_t* Ci,
               int64_t ldc, const ColmaxJob* side, hipStream_t stream) {
  const int64_t tiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  const dim3 grid((unsigned)tiles);
  const bool fast = pipelined_ok<BM, BN, AK, BKM>(M, N, K, lda, ldb);
  const bool rebase = rebase_ok<BM, BN, AK, BKM>(M, N, K, lda, ldb);
  if (side && (Ci || !(fast && side_fits(*side, tiles, BM)))) {  // as a launch of its own
    const hipError_t e = launch_colmax_finalize(*side, stream);
    if (e != hipSuccess) return e;
    side = nullptr;
  }
  // packed stores of adjacent outputs need 16-byte aligned rows
  const uintptr_t c = Ci ? reinterpret_cast<uintptr_t>(Ci) : reinterpret_cast<uintptr_t>(Cb);
  const bool vec = Ci ? (ldc % 4 == 0 && c % 16 == 0) : (ldc % 8 == 0 && c % 16 == 0);
  if (Ci) {  // the int32 hook: no column maxima ride along
    if (vec) launch<BM, BN, AK, BKM, true, true>(fast, rebase, grid, M, N, K, A, lda, sa, B, ldb, sb, Ci, ldc, nullptr, stream);
    else launch<BM, BN, AK, BKM, true, false>(fast, rebase, grid, M, N, K, A, lda, sa, B, ldb, sb, Ci, ldc, nullptr, stream);
  } else {
    if (vec) launch<BM, BN, AK, BKM, false, true>(fast, rebase, grid, M, N, K, A, lda, sa, B, ldb, sb, Cb, ldc, side, stream);
    else launch<BM, BN, AK, BKM, false, false>(fast, rebase, grid, M, N, K, A, lda, sa, B, ldb, sb, Cb, ldc, side, stream);
  }
  return hipGetLastError();
}

template <bool AK, bool BKM>
hipError_t pick(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa,
                const int8_t* B, int64_t ldb, const float* sb, uint16_t* Cb, int32_t* Ci,
                int64_t ldc, const ColmaxJob* side, hipStream_t stream) {
  if (big_tiles(M, N) >= kBigTileMin)
    return run<256, 256, AK, BKM>(M, N, K, A, lda, sa, B, ldb, sb, Cb, Ci, ldc, side, stream);
  return run<128, 128, AK, BKM>(M, N, K, A, lda, sa, B, ldb, sb, Cb, Ci, ldc, side, stream);
}

size_t plan_bytes(const SplitPlan& p, int64_t M) {
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)p.ldp * 4 : 0;
}

// C[m, n] = bf16_RNE(RN32(RN32(float(sum_s P[s][m][n]) * sa[m]) * sb[n]));
// one thread per 4 adjacent outputs of a row, rows over blockIdx.y.  T =
// int32_t: exact integer partial sums (INT8); T = float: fp32 partial sums
// (FP8), added in fp32 in plane order s = 0, 1, ... (a fixed order, so the
// result does not depend on scheduling).
template <typename T>
__global__ __launch_bounds__(256) void splitk_reduce(const T* __restrict__ P, int64_t ldp,
                                                     int64_t plane, int splits, int64_t M,
                                                     int64_t N, const float* __restrict__ sa,
                                                     const float* __restrict__ sb,
                                                     __bf16* __restrict__ C, int64_t ldc) {
  typedef T v4t __attribute__((ext_vector_type(4)));
  const int64_t n = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (n >= N) return;
  const bool vec = ldc % 4 == 0 && reinterpret_cast<uintptr_t>(C) % 8 == 0 && n + 4 <= N;
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const T* p = P + m * ldp + n;  // columns up to n + 3 < ldp: inside the plane
    v4t acc = *reinterpret_cast<const v4t*>(p);
#pragma unroll 8
    for (int s = 1; s < splits; ++s) acc += *reinterpret_cast<const v4t*>(p + s * plane);
    const float sam = sa[m];
    __bf16 h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y = (float)acc[e];
      y = y * sam;
      y = y * (n + e < N ? sb[n + e] : 0.0f);
      h[e] = (__bf16)y;  // round to nearest even
    }
    __bf16* row = C + m * ldc;
    if (vec) {
      *reinterpret_cast<uint2*>(row + n) = __builtin_bit_cast(uint2, h);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) row[n + e] = h[e];
    }
  }
}

// The partial planes of a split contraction: int32 sums (INT8) or raw fp32 sums
// (FP8), 4 bytes either way.
template <int FMT, bool AK, bool BKM>
hipError_t run_partials(const SplitPlan& p, int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                        const int8_t* B, int64_t ldb, void* P, const ColmaxJob* side, hipStream_t stream) {
  const int64_t tiles = big_tiles(M, N);
  const int64_t plane = M * p.ldp;
  const dim3 grid((unsigned)(tiles * p.splits));
  if (side && !side_fits(*side, tiles * p.splits, 256)) {  // as a launch of its own
    const hipError_t e = launch_colmax_finalize(*side, stream);
    if (e != hipSuccess) return e;
    side = nullptr;
  }
  if (side)
    gemm_i8_pipelined<256, 256, 4, AK, BKM, true, true, FMT, true><<<grid, 512, 0, stream>>>(
        M, N, K, A, lda, nullptr, B, ldb, nullptr, P, p.ldp, p.kchunk, plane, *side, NoEpilogue{});
  else
    gemm_i8_pipelined<256, 256, 4, AK, BKM, true, true, FMT><<<grid, 512, 0, stream>>>(
        M, N, K, A, lda, nullptr, B, ldb, nullptr, P, p.ldp, p.kchunk, plane, ColmaxJob{}, NoEpilogue{});
  return hipGetLastError();
}

template <int FMT, bool AK, bool BKM>
hipError_t run_split(const SplitPlan& p, int64_t M, int64_t N, int64_t K, const int8_t* A,
                     int64_t lda, const float* sa, const int8_t* B, int64_t ldb, const float* sb,
                     uint16_t* C, int64_t ldc, void* P, const ColmaxJob* side, hipStream_t stream) {
  const hipError_t e = run_partials<FMT, AK, BKM>(p, M, N, K, A, lda, B, ldb, P, side, stream);
  if (e != hipSuccess) return e;
  const int64_t plane = M * p.ldp;
  const dim3 rgrid((unsigned)((N + 1023) / 1024), (unsigned)std::min<int64_t>(M, 65535));
  if constexpr (FMT == 1)
    splitk_reduce<float><<<rgrid, 256, 0, stream>>>(static_cast<const float*>(P), p.ldp, plane, p.splits, M, N, sa, sb,
                                                   reinterpret_cast<__bf16*>(C), ldc);
  else
    splitk_reduce<int32_t><<<rgrid, 256, 0, stream>>>(static_cast<const int32_t*>(P), p.ldp, plane, p.splits, M, N, sa,
                                                     sb, reinterpret_cast<__bf16*>(C), ldc);
  return hipGetLastError();
}

// FP8 GEMM for any shape (the pipelined kernel needs K % 16 == 0, and
// output extents that are multiples of 4 where an operand is read down its
// rows).  The INT8 general kernel's structure (register-staged, byte-masked
// loads into the same swizzled LDS tiles, two slabs in LDS) with the
// pipelined FP8 kernel's fragments and instruction: each 64-deep slab is one
// v_mfma_scale_f32_32x32x64_f8f6f4 per 32 x 32 block with the operands placed
// exactly as there, and slabs are accumulated in the same order, so on shapes
// both kernels take the sums are bit-identical.  Contraction indices past K
// are zero in both operands (a product of two zeros has the smallest
// exponent sum, so it changes no group's truncation step).
template <int BM, int BN, bool A_KMAJOR, bool B_KMAJOR, bool OUT_F32, bool VEC>
__global__ __launch_bounds__(kThreads) void gemm_f8_general(int64_t M, int64_t N, int64_t K,
                                                            const int8_t* __restrict__ A, int64_t lda,
                                                            const float* __restrict__ sa,
                                                            const int8_t* __restrict__ B, int64_t ldb,
                                                            const float* __restrict__ sb,
                                                            void* __restrict__ Cv, int64_t ldc) {
  constexpr int WM = BM / 2, WN = BN / 2;  // 2 x 2 waves
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
  __shared__ __attribute__((aligned(16))) int8_t lds[2 * (A_BYTES + B_BYTES)];

  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + BN - 1) / BN);
  int tm, tn;
  tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wm0 = (wave >> 1) * WM, wn0 = (wave & 1) * WN;

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = Mma<1>::zero();

  Stager<BM, A_KMAJOR> sa_stage;
  Stager<BN, B_KMAJOR> sb_stage;
  const int nk = (int)((K + BK - 1) / BK);
  if (nk > 0) {
    sa_stage.load(A, lda, m0, M, 0, K, t);
    sb_stage.load(B, ldb, n0, N, 0, K, t);
    sa_stage.store(lds, t);
    sb_stage.store(lds + A_BYTES, t);
  }
  __syncthreads();

  for (int kt = 0; kt < nk; ++kt) {
    int8_t* cur = lds + (kt & 1) * (A_BYTES + B_BYTES);
    int8_t* nxt = lds + ((kt & 1) ^ 1) * (A_BYTES + B_BYTES);
    const bool more = kt + 1 < nk;
    if (more) {
      sa_stage.load(A, lda, m0, M, (int64_t)(kt + 1) * BK, K, t);
      sb_stage.load(B, ldb, n0, N, (int64_t)(kt + 1) * BK, K, t);
    }
    v8i af[TM], bf[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) af[i] = frag32f8<BM, A_KMAJOR>(cur, wm0 + 32 * i, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[j] = frag32f8<BN, B_KMAJOR>(cur + A_BYTES, wn0 + 32 * j, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = Mma<1>::mma(bf[j], af[i], acc[i][j]);
    if (more) {
      sa_stage.store(nxt, t);
      sb_stage.store(nxt + A_BYTES, t);
    }
    __syncthreads();
  }

  if constexpr (OUT_F32) {  // the raw fp32 sums (C holds floats)
    store32f_raw<TM, TN>(acc, m0, n0, wm0, wn0, M, N, static_cast<float*>(Cv), ldc, lane);
  } else {
    // every wave has passed its last LDS read of the slabs before any scale lands
    __syncthreads();
    float* s_lds = reinterpret_cast<float*>(lds);
    stage_scales<BM, BN, false>(s_lds, m0, n0, M, N, sa, sb, t);
    store32f_direct<BM, TM, TN>(acc, m0, n0, wm0, wn0, M, N, s_lds, static_cast<__bf16*>(Cv), ldc, lane);
  }
}

template <int BM, int BN, bool AK, bool BKM>
hipError_t run_fp8(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sa,
                   const uint8_t* B, int64_t ldb, const float* sb, uint16_t* C, float* Cf,
                   int64_t ldc, const ColmaxJob* side, hipStream_t stream) {
  const int64_t tiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  const dim3 grid((unsigned)tiles);
  constexpr int WGN = BM >= 256 ? 4 : 2;
  const bool vec = ldc % 8 == 0 && reinterpret_cast<uintptr_t>(C) % 16 == 0;
  const int8_t* a = reinterpret_cast<const int8_t*>(A);
  const int8_t* b = reinterpret_cast<const int8_t*>(B);
  const bool fast = pipelined_ok<BM, BN, AK, BKM>(M, N, K, lda, ldb);
  const bool rebase = !Cf && vec && rebase_ok<BM, BN, AK, BKM>(M, N, K, lda, ldb);
  if (side && (Cf || !(fast && side_fits(*side, tiles, BM)))) {  // as a launch of its own
    const hipError_t e = launch_colmax_finalize(*side, stream);
    if (e != hipSuccess) return e;
    side = nullptr;
  }
  if (rebase) {  // an operand read down its rows spans 2^31 bytes or more
    if constexpr (BM == 256 && !(AK && BKM))
      gemm_i8_pipelined<BM, BN, WGN, AK, BKM, false, true, 1, false, true><<<grid, 128 * WGN, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, C, ldc, K, 0, ColmaxJob{}, NoEpilogue{});
  } else if (side && vec) {
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, false, true, 1, true><<<grid, 128 * WGN, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, C, ldc, K, 0, *side, NoEpilogue{});
  } else if (side) {
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, false, false, 1, true><<<grid, 128 * WGN, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, C, ldc, K, 0, *side, NoEpilogue{});
  } else if (!fast) {
    if (Cf)
      gemm_f8_general<BM, BN, AK, BKM, true, false><<<grid, kThreads, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, Cf, ldc);
    else
      gemm_f8_general<BM, BN, AK, BKM, false, false><<<grid, kThreads, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, C, ldc);
  } else if (Cf) {
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, true, false, 1><<<grid, 128 * WGN, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, Cf, ldc, K, 0, ColmaxJob{}, NoEpilogue{});
  } else if (vec) {
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, false, true, 1><<<grid, 128 * WGN, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, C, ldc, K, 0, ColmaxJob{}, NoEpilogue{});
  } else {
    gemm_i8_pipelined<BM, BN, WGN, AK, BKM, false, false, 1><<<grid, 128 * WGN, 0, stream>>>(M, N, K, a, lda, sa, b, ldb, sb, C, ldc, K, 0, ColmaxJob{}, NoEpilogue{});
  }
  return hipGetLastError();
}

template <bool AK, bool BKM>
hipError_t pick_fp8(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sa,
                    const uint8_t* B, int64_t ldb, const float* sb, uint16_t* C, float* Cf,
                    int64_t ldc, const ColmaxJob* side, hipStream_t stream) {
  if (big_tiles(M, N) >= kBigTileMin)
    return run_fp8<256, 256, AK, BKM>(M, N, K, A, lda, sa, B, ldb, sb, C, Cf, ldc, side, stream);
  return run_fp8<128, 128, AK, BKM>(M, N, K, A, lda, sa, B, ldb, sb, C, Cf, ldc, side, stream);
}

}  // namespace

hipError_t launch_gemm_fp8(int layout, int64_t M, int64_t N, int64_t K, const uint8_t* A,
                           int64_t lda, const float* sa, const uint8_t* B, int64_t ldb,
                           const float* sb, uint16_t* C, float* C_f32, int64_t ldc,
                           hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  switch (layout) {
    case 0:
      return pick_fp8<true, true>(M, N, K, A, lda, sa, B, ldb, sb, C, C_f32, ldc, nullptr, stream);
    case 1:
      return pick_fp8<true, false>(M, N, K, A, lda, sa, B, ldb, sb, C, C_f32, ldc, nullptr, stream);
    default:
      return pick_fp8<false, false>(M, N, K, A, lda, sa, B, ldb, sb, C, C_f32, ldc, nullptr, stream);
  }
}

namespace {

SplitPlan plan_for(int layout, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
  switch (layout) {
    case 0: return plan_split<true, true>(M, N, K, lda, ldb);
    case 1: return plan_split<true, false>(M, N, K, lda, ldb);
    default: return plan_split<false, false>(M, N, K, lda, ldb);
  }
}

}  // namespace

size_t gemm_split_workspace_bytes(int layout, int64_t M, int64_t N, int64_t K, int64_t lda,
                                  int64_t ldb) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return plan_bytes(plan_for(layout, M, N, K, lda, ldb), M);
}

hipError_t launch_gemm_split(int layout, int64_t M, int64_t N, int64_t K, const int8_t* A,
                             int64_t lda, const float* sa, const int8_t* B, int64_t ldb,
                             const float* sb, uint16_t* C, int64_t ldc, void* ws,
                             const ColmaxJob* side, int fmt, hipStream_t stream) {
  if (side && side->n <= 0) side = nullptr;
  if (M == 0 || N == 0) return side ? launch_colmax_finalize(*side, stream) : hipSuccess;
  const SplitPlan p = K > 0 ? plan_for(layout, M, N, K, lda, ldb) : SplitPlan{1, K, 0};
  const uint8_t* a8 = reinterpret_cast<const uint8_t*>(A);
  const uint8_t* b8 = reinterpret_cast<const uint8_t*>(B);
  if (p.splits < 2 || !ws) {
    if (fmt == 1) {
      switch (layout) {
        case 0: return pick_fp8<true, true>(M, N, K, a8, lda, sa, b8, ldb, sb, C, nullptr, ldc, side, stream);
        case 1: return pick_fp8<true, false>(M, N, K, a8, lda, sa, b8, ldb, sb, C, nullptr, ldc, side, stream);
        default: return pick_fp8<false, false>(M, N, K, a8, lda, sa, b8, ldb, sb, C, nullptr, ldc, side, stream);
      }
    }
    switch (layout) {
      case 0: return pick<true, true>(M, N, K, A, lda, sa, B, ldb, sb, C, nullptr, ldc, side, stream);
      case 1: return pick<true, false>(M, N, K, A, lda, sa, B, ldb, sb, C, nullptr, ldc, side, stream);
      default: return pick<false, false>(M, N, K, A, lda, sa, B, ldb, sb, C, nullptr, ldc, side, stream);
    }
  }
  if (fmt == 1) {
    switch (layout) {
      case 0: return run_split<1, true, true>(p, M, N, K, A, lda, sa, B, ldb, sb, C, ldc, ws, side, stream);
      case 1: return run_split<1, true, false>(p, M, N, K, A, lda, sa, B, ldb, sb, C, ldc, ws, side, stream);
      default: return run_split<1, false, false>(p, M, N, K, A, lda, sa, B, ldb, sb, C, ldc, ws, side, stream);
    }
  }
  switch (layout) {
    case 0: return run_split<0, true, true>(p, M, N, K, A, lda, sa, B, ldb, sb, C, ldc, ws, side, stream);
    case 1: return run_split<0, true, false>(p, M, N, K, A, lda, sa, B, ldb, sb, C, ldc, ws, side, stream);
    default: return run_split<0, false, false>(p, M, N, K, A, lda, sa, B, ldb, sb, C, ldc, ws, side, stream);
  }
}

hipError_t launch_gemm_partials(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* B,
                                int64_t ldb, void* P, const ColmaxJob* side, hipStream_t stream) {
  return run_partials<0, true, true>(plan_split<true, true>(M, N, K, lda, ldb), M, N, K, A, lda, B, ldb, P, side, stream);
}

hipError_t launch_mfma_rate_probe(const int8_t* codes, int64_t bytes, int64_t rounds, int32_t* sink,
                                  hipStream_t stream) {
  const int64_t span = (bytes - 24 * 1024) / 1024 * 1024 + 1024;  // fragment origins a wave may take
  mfma_rate_probe<<<dim3(kMfmaProbeWorkgroups), 512, 0, stream>>>(codes, span, rounds, sink);
  return hipGetLastError();
}

hipError_t launch_gemm(int layout, int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                       const float* sa, const int8_t* B, int64_t ldb, const float* sb,
                       uint16_t* C_bf16, int32_t* C_i32, int64_t ldc, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  switch (layout) {
    case 0:
      return pick<true, true>(M, N, K, A, lda, sa, B, ldb, sb, C_bf16, C_i32, ldc, nullptr, stream);
    case 1:
      return pick<true, false>(M, N, K, A, lda, sa, B, ldb, sb, C_bf16, C_i32, ldc, nullptr, stream);
    default:
      return pick<false, false>(M, N, K, A, lda, sa, B, ldb, sb, C_bf16, C_i32, ldc, nullptr, stream);
  }
}

}  // namespace i8mp
