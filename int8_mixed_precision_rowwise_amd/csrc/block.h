// What the block-scaled FP8 kernels share: where an expert's rows lie, the exponent
// of a block's scale, and the launchers.
//
// Codes are E4M3 with one power-of-two scale for each 128 of the contraction.  A
// block's exponent is the least e >= -126 with amax <= 448 * 2^e, held as the byte
// e + 127 (E8M0), which the matrix instruction applies by itself while it
// multiplies: no scale costs a vector operation in the product, and x / 2^e is exact,
// so a code is rounded once.  A block that holds an infinity or NaN has the byte 255,
// the NaN of that format, and codes that are NaN.
#pragma once

#include "internal.h"

namespace i8mp {

constexpr int kBlock = 128;

// Rows of experts one after another: expert e has rows off[e] .. off[e + 1] - 1 of
// `rows` (offsets in device memory, 32 or 64 bits).  No offsets: one expert with all rows.
struct Ragged {
  const void* off;
  int bits;
  int64_t E, rows;
};

// Room that holds `rows` rows of E experts with each expert's first row at a multiple of
// `unit` (expert e's at unit * (off[e] / unit + e), which needs no sum over the experts
// before it), in units.
inline int64_t ragged_units(int64_t rows, int64_t E, int64_t unit) { return rows / unit + E; }

#ifdef __HIPCC__
namespace {

__device__ __forceinline__ int64_t offset_at(const Ragged& r, int64_t e) {
  const int64_t v = r.bits == 64 ? static_cast<const int64_t*>(r.off)[e] : (int64_t) static_cast<const int32_t*>(r.off)[e];
  return min(max(v, (int64_t)0), r.rows);  // whatever the offsets hold, rows stay within the tensors
}

// The rows that no expert has: those in front of the first one's and those behind the last one's.
struct OtherRows {
  int64_t front, end, count;
  __device__ __forceinline__ int64_t row(int64_t i) const { return i < front ? i : end + (i - front); }
};
__device__ __forceinline__ OtherRows other_rows(const Ragged& r) {
  if (!r.off) return {0, 0, 0};
  const int64_t front = offset_at(r, 0), end = offset_at(r, r.E);
  return {front, end, front + (r.rows - end)};
}

// Where a tile of an expert's rows lies: the expert (e), the tile's first row within it (local), the expert's first row and
// number of rows.
struct Place {
  int64_t e, local, first, count;
};

// First row and number of rows of this lane's expert e; no rows past the last expert.  What a wave needs of one of them
// it then reads from that lane, not from memory again: the way to a first load is a chain of such reads (the backward of
// 1551 rows of 13 experts 23.9 us, 24.7 with offsets read again).
struct LaneRows {
  int first, count;
};
__device__ __forceinline__ LaneRows lane_rows(const Ragged& r, int64_t e) {
  LaneRows l{(int)r.rows, 0};
  if (e < r.E) {
    l.first = (int)offset_at(r, e);
    l.count = max(0, (int)offset_at(r, e + 1) - l.first);
  }
  return l;
}
// Those of expert e0 + at, at the same in all lanes.
__device__ __forceinline__ void take_lane(const LaneRows& l, int64_t e0, int at, Place& p) {
  at = __builtin_amdgcn_readfirstlane(at);
  p.e = e0 + at;
  p.first = __builtin_amdgcn_readlane(l.first, at);
  p.count = __builtin_amdgcn_readlane(l.count, at);
}

// Block `s` of the room in units of UNIT rows.  false: no expert's.
template <int UNIT>
__device__ __forceinline__ bool locate(const Ragged& r, int64_t s, Place& p) {
  if (!r.off) {
    p.e = 0, p.first = 0, p.count = r.rows, p.local = s * UNIT;
    return p.local < p.count;
  }
  // the last expert whose first unit is at most s; a wave looks at 64 experts at a time
  const int lane = threadIdx.x & 63;
  bool some = false;
  for (int64_t e0 = 0; e0 < r.E; e0 += 64) {
    const LaneRows l = lane_rows(r, e0 + lane);
    const uint64_t m = __ballot(e0 + lane < r.E && l.first / UNIT + e0 + lane <= s);
    const int here = __popcll(m);
    if (here) take_lane(l, e0, here - 1, p), some = true;
    if (m != ~uint64_t(0)) break;
  }
  if (!some) return false;
  p.local = (s - (p.first / UNIT + p.e)) * UNIT;
  return p.local >= 0 && p.local < p.count;
}

// First unit of an expert in that room.
template <int UNIT>
__device__ __forceinline__ int64_t unit_of(const Place& p) {
  return p.first / UNIT + p.e;
}

// The exponent's byte of a block whose largest magnitude has the bf16 bits b:
// 448 = 1.75 * 2^8, so e is b's exponent less 8, and one more where its fraction is over 0.75.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t b) {
  const int byte = max((int)((b + 0x1F) >> 7) - 8, 1);
  return b >= 0x7F80u ? 255u : (uint32_t)byte;
}

// 2^-e; NaN for the byte 255.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (254u - byte) << 23);
}

// 2^e (infinity for the byte 255, which makes codes that do not matter).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Codes of four bf16 under one scale: the conversion divides by 2^e and rounds once (the same codes as x * 2^-e
// converted, over every bf16 pattern and exponent).
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, float scale) {
  typedef short s2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  s2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(b2, lo), scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(b2, hi), scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

}  // namespace
#endif

// Codes of a bf16 matrix x [rows of rag][cols], read through `index` (row r is x's row
// index[r], of n_src; a negative index or one past the end is a row of zeros) unless NULL.
// Along the rows: codes at rows 16 * unit_of<16> + local of q_row, exponents s_row[that row][block],
// rows of which lie ld_srow (a multiple of 4) apart.  Down the rows, blocks starting at the expert's first row: codes at the rows
// themselves of q_col, exponents s_col[unit_of<128> + block][column].  Pitch of codes: ldq
// = cols rounded up to 16, zeros behind cols.
struct BlockQuant {
  const uint16_t* x;
  int64_t ldx, cols, n_src;
  const int32_t* index;
  Ragged rag;
  uint8_t *q_row, *s_row, *q_col, *s_col;
  int64_t ldq, ld_srow, ld_scol;
};

// Exponents of weight blocks [E][ceil(N / 128)][ceil(K / 128)] spread to one byte for each
// row (along = 0: planes [E][K blocks][ld], byte n) or column (along = 1: [E][N blocks][ld],
// byte k) of the weight, as the products read them; ld a multiple of 16.
struct SpreadJob {
  const uint8_t* exps;
  int64_t E, nb, kb, ld;
  int along;
  uint8_t* planes;
  __host__ __device__ int64_t groups() const { return planes ? E * (along ? nb : kb) * (ld / 16) : 0; }
};

// rows / cols codes of `a`, column codes of `b` (NULL: none) and the spread exponents, in one launch.
hipError_t launch_block_quant(const BlockQuant& a, const BlockQuant* b, const SpreadJob& spread, hipStream_t stream);

hipError_t launch_block_quant_weight(const uint16_t* w, int64_t E, int64_t N, int64_t K, int64_t ldw, int64_t w_stride,
                                     uint8_t* codes, uint8_t* exps, hipStream_t stream);

// The products.  FORWARD: C[r][n] = sum_k A[r][k] B[e][n][k]; INPUT: C[r][k] = sum_n A[r][n]
// B[e][n][k]; WEIGHT: C[e][n][k] = sum_r A[r][n] B[r][k] over the expert's rows.
enum BlockProduct { kBlockForward = 0, kBlockInput = 1, kBlockWeight = 2 };
// Exponents: B's (and WEIGHT's A's) in planes [block][row or column], ldsb (ldsa) apart; the others' A's in rows
// [row][block], ldsa (a multiple of 4) apart.
struct BlockGemm {
  int64_t rows_out;      // C's rows (WEIGHT: N); others: rag's
  int64_t cols_out;      // C's columns
  int64_t contraction;   // FORWARD: K, INPUT: N; WEIGHT: the expert's rows
  const uint8_t *A, *sA; // codes and exponents
  int64_t lda, ldsa;
  // FORWARD: NULL, or row r of the experts' rows is A's row index[r], of n_src (another: a row of zeros); A then
  // lies row by row, and n_src * lda is below 2^31 - 1024.  Otherwise A has each expert's rows at 16 * unit_of<16>.
  const int32_t* index;
  int64_t n_src;
  const uint8_t *B, *sB;
  int64_t ldb, ldsb, b_stride, sb_stride;  // strides between experts (FORWARD, INPUT)
  uint16_t* C;
  int64_t ldc, c_stride;
  Ragged rag;
  int clear;  // rows that no expert has are written as zeros
  // set by the launcher from the plan
  uint32_t splits;
  int64_t kchunk, plane, plane_ld;
  float* planes;
};
// Tile size and, for one matrix, the parts of the contraction (of kchunk each, a multiple of 512) and the pitch of
// their planes.  rows, cols: C's; contraction as in BlockGemm (WEIGHT of one matrix: its rows); all_rows: ragged rows.
struct BlockPlan {
  bool big;
  int64_t splits, kchunk, plane_ld;
  size_t bytes(int64_t rows) const { return splits > 1 ? (size_t)(splits * rows * plane_ld) * 4 : 0; }
};
BlockPlan block_plan(BlockProduct what, int64_t rows, int64_t cols, int64_t contraction, int64_t E, int64_t all_rows);
hipError_t launch_block_gemm(BlockProduct what, const BlockGemm& g, const BlockPlan& plan, float* planes, hipStream_t stream);
hipError_t launch_block_gemms(const BlockGemm& dx, const BlockPlan& px, const BlockGemm& dw, const BlockPlan& pw, float* planes, hipStream_t stream);

// Few rows an expert against weight codes: bound by reading them, X quantized in the kernel.
struct BlockFew {
  const uint16_t* x;
  int64_t ldx, n_src;
  const int32_t* index;
  Ragged rag;
  int64_t N, K;
  const uint8_t *codes, *exps;
  uint16_t* Y;
  int64_t ldy;
  int clear;
};
hipError_t launch_block_few(const BlockFew& a, hipStream_t stream);
bool block_few_takes(int64_t rows, int64_t E, int64_t N, int64_t K);

}  // namespace i8mp
