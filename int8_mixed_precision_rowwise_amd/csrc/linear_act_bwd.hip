// The elementwise part of a linear layer's backward through its activation:
//   g = dY act'(Z),  dZ = bf16(g),  dbias = column sums of g (fp32),
// and dZ's codes along its rows (for dX = dZ W) and down its columns (for
// dW = dZ^T X).
//
// Both quantizations need maxima over the whole of a row and a column, so two
// passes are the least: the first reads dY and Z, writes dZ and leaves the maxima
// of every row's segment of 512 columns, the column maxima and the column sums of
// every band of rows; a short launch joins the bands; the second pass reads dZ once
// for both sets of codes.  6 and 4 bytes an element: both passes are bound by
// memory (GELU's derivative, some 40 operations, comes near).  A
// block is 8 waves; a lane owns 8 adjacent columns, a wave a 512-column segment of
// a row, so a row's maximum is one wave reduction and the columns' sums and maxima
// stay in the lane's registers over its rows.  Sums are joined in a fixed order:
// the same call gives the same bits.
//
// Measured at 8192 x 5632, GELU: first pass (276 MB) 50 us alone, with what it reads
// left in the last level, and 72 us in a whole backward; join 5 us; second pass (185 MB)
// 33 and 47 us.
#include "activation.h"
#include "quant_device.h"

#include <algorithm>

namespace i8mp {
namespace {

constexpr int kTile = 512, kWaves = 8, kBwdThreads = 64 * kWaves;
constexpr int kMaxBands = 256, kBandRows = 32;  // bands of rows in the first pass, at most, of so many rows at least
constexpr int kMaxBlockRows = 512;  // rows of a block of the second

__device__ __forceinline__ us2 max_us2(us2 a, uint32_t w) { return __builtin_elementwise_max(a, as_us2(w)); }
__device__ __forceinline__ void max_columns(us2 (&m)[4], uint4 v) {
  m[0] = max_us2(m[0], v.x & 0x7FFF7FFFu), m[1] = max_us2(m[1], v.y & 0x7FFF7FFFu);
  m[2] = max_us2(m[2], v.z & 0x7FFF7FFFu), m[3] = max_us2(m[3], v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint4 pack_columns(const us2 (&m)[4]) {
  return make_uint4(__builtin_bit_cast(uint32_t, m[0]), __builtin_bit_cast(uint32_t, m[1]),
                    __builtin_bit_cast(uint32_t, m[2]), __builtin_bit_cast(uint32_t, m[3]));
}

// First pass: grid (column tiles, bands).
template <int ACT>
__global__ __launch_bounds__(kBwdThreads) void act_grad_stats(ActBwdArgs a) {
  __shared__ uint4 red[kWaves][64];
  __shared__ float sums[kWaves][kTile];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * kTile + lane * 8;
  const int64_t r_begin = (int64_t)blockIdx.y * a.rows_per_band;
  const int64_t r_end = min(a.M, r_begin + a.rows_per_band);
  const int nvalid = (int)max((int64_t)0, min((int64_t)8, a.N - c0));
  const int64_t cl = nvalid > 0 ? c0 : 0;  // lanes past the last column read column 0, unused
  us2 cm[4] = {{0, 0}, {0, 0}, {0, 0}, {0, 0}};
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  constexpr int U = 4;
  for (int64_t r0 = r_begin + wave; r0 < r_end; r0 += U * kWaves) {
    uint4 y[U], z[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t r = min(r0 + k * kWaves, r_end - 1);
      y[k] = *reinterpret_cast<const uint4*>(a.dY + r * a.lddy + cl);
      if constexpr (ACT != kActNone) z[k] = *reinterpret_cast<const uint4*>(a.Z + r * a.ldz + cl);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t r = r0 + k * kWaves;
      if (r >= r_end) break;
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = elem(y[k], j);
        if constexpr (ACT != kActNone) g[j] *= activation_grad<ACT>(elem(z[k], j));
        if (j >= nvalid) g[j] = 0.0f;
        sum[j] += g[j];
      }
      uint4 d;
      if constexpr (ACT != kActNone) {
        __bf16 h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = (__bf16)g[j];
        d = __builtin_bit_cast(uint4, h);
        if (nvalid > 0) *reinterpret_cast<uint4*>(a.dZ + r * a.lddz + c0) = d;  // rows are padded to 16 bytes
      } else {
        d = nvalid == 8 ? y[k] : nvalid > 0 ? keep_first(y[k], nvalid) : make_uint4(0, 0, 0, 0);
      }
      if (a.row_codes) {
        const us2 m2 = absmax_bits(us2{0, 0}, d);
        const uint32_t m = wave_max_u32<true>(max((uint32_t)m2.x, (uint32_t)m2.y));
        if (lane == 0) a.segmax[r * a.tiles + blockIdx.x] = (uint16_t)m;
      }
      max_columns(cm, d);
    }
  }
  red[wave][lane] = pack_columns(cm);
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[wave][j * 64 + lane] = sum[j];  // column 8 lane + j
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) max_columns(cm, red[w][lane]);
    *reinterpret_cast<uint4*>(a.band_max + (int64_t)blockIdx.y * a.tiles * kTile + c0) = pack_columns(cm);
  }
  const int t = threadIdx.x;
  float s = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += sums[w][t];
  a.band_sum[((int64_t)blockIdx.y * a.tiles + blockIdx.x) * kTile + (t & 63) * 8 + (t >> 6)] = s;
}

// Column maxima (bf16 bits) and dbias of all the bands: 64
// columns a block, its 8 waves over the bands.
__global__ __launch_bounds__(kBwdThreads) void act_grad_join(ActBwdArgs a) {
  __shared__ uint32_t red_max[kWaves][64];
  __shared__ float red_sum[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane, pitch = (int64_t)a.tiles * kTile;  // pitch is a multiple of 64
  uint32_t m = 0;
  float s = 0;
#pragma unroll 8
  for (int b = wave; b < a.bands; b += kWaves) {
    m = max(m, (uint32_t)a.band_max[b * pitch + c]);
    s += a.band_sum[b * pitch + c];
  }
  red_max[wave][lane] = m, red_sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = max(m, red_max[w][lane]), s += red_sum[w][lane];
    a.col_max[c] = (uint16_t)m;
    if (a.dbias && c < a.N) a.dbias[c] = s;
  }
}

// Second pass: blocks of rows (up to M padded) by column tiles, the tiles of a
// row adjacent.  Columns N .. np of the row codes and rows M .. mp of the column
// codes become zero.
template <bool SR, bool ALIGNED4>
__global__ __launch_bounds__(kBwdThreads) void act_grad_quant(ActBwdArgs a) {
  __shared__ uint32_t row_max[kMaxBlockRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = (int)(blockIdx.x % a.tiles);
  const int64_t block = blockIdx.x / a.tiles;
  const int64_t c0 = (int64_t)tile * kTile + lane * 8;
  const int64_t r_begin = block * a.rows_per_block;
  const int64_t r_end = min(a.mp, r_begin + a.rows_per_block);
  const int nvalid = (int)max((int64_t)0, min((int64_t)8, a.N - c0));
  const int64_t cl = nvalid > 0 ? c0 : 0;
  if (a.row_codes && threadIdx.x < a.rows_per_block && r_begin + threadIdx.x < a.M) {
    const uint16_t* seg = a.segmax + (r_begin + threadIdx.x) * a.tiles;
    uint32_t m = 0;
    for (int s = 0; s < a.tiles; ++s) m = max(m, (uint32_t)seg[s]);
    row_max[threadIdx.x] = m;
  }
  const uint4 cb = *reinterpret_cast<const uint4*>(a.col_max + c0);
  const us2 cm[4] = {as_us2(cb.x), as_us2(cb.y), as_us2(cb.z), as_us2(cb.w)};
  __syncthreads();
  GroupScale g[8];
  bool mine = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = j & 1 ? cm[j >> 1].y : cm[j >> 1].x;
    g[j] = make_scale(j < nvalid ? bits : 0u);
    mine = mine && (j >= nvalid || g[j].mode == 1);
  }
  const bool all_fma = __all(mine);
  if (block == 0 && wave == 0 && a.col_codes) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < nvalid) a.col_scale[c0 + j] = g[j].s;
  }
  if (c0 >= a.np) return;
  constexpr int U = 4;
  for (int64_t r0 = r_begin + wave; r0 < r_end; r0 += U * kWaves) {
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t r = min(r0 + k * kWaves, a.M - 1);
      v[k] = *reinterpret_cast<const uint4*>(a.dZ + r * a.lddz + cl);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t r = r0 + k * kWaves;
      if (r >= r_end) break;
      if (nvalid < 8) v[k] = nvalid > 0 ? keep_first(v[k], nvalid) : make_uint4(0, 0, 0, 0);
      const uint64_t e0 = (uint64_t)(r * a.N + c0);
      if (a.row_codes && r < a.M) {
        const GroupScale row = make_scale(__builtin_amdgcn_readfirstlane(row_max[r - r_begin]));
        if (tile == 0 && lane == 0) a.row_scale[r] = row.s;
        *reinterpret_cast<uint2*>(a.row_codes + r * a.np + c0) =
            row.mode == 1 ? quantize_chunk<SR, ALIGNED4, false, 1>(v[k], &row, a.seed, a.row_offset, e0)
                          : quantize_chunk<SR, ALIGNED4, false, -1>(v[k], &row, a.seed, a.row_offset, e0);
      }
      if (a.col_codes) {
        uint2 codes = make_uint2(0, 0);
        if (r < a.M)
          codes = all_fma ? quantize_chunk<SR, ALIGNED4, true, 1>(v[k], g, a.seed, a.col_offset, e0)
                          : quantize_chunk<SR, ALIGNED4, true, -1>(v[k], g, a.seed, a.col_offset, e0);
        *reinterpret_cast<uint2*>(a.col_codes + r * a.np + c0) = codes;
      }
    }
  }
}

}  // namespace

void act_bwd_plan(ActBwdArgs& a) {
  a.np = (a.N + 15) / 16 * 16;
  a.mp = (a.M + 15) / 16 * 16;
  a.tiles = (int)std::max<int64_t>(1, (a.np + kTile - 1) / kTile);
  // about eight blocks a CU, in whole turns of a block's waves over the rows
  // (8192 x 5632, GELU: 50 us; 92 with fewer, which the second pass then joined)
  const int64_t want = std::min<int64_t>(kMaxBands, std::max<int64_t>(1, 2048 / a.tiles));
  a.rows_per_band = std::max<int64_t>(1, ((a.M + want - 1) / want + kBandRows - 1) / kBandRows) * kBandRows;
  a.bands = (int)((a.M + a.rows_per_band - 1) / a.rows_per_band);
  const int64_t blocks = std::max<int64_t>(1, 1024 / a.tiles);
  a.rows_per_block = std::max<int64_t>(32, (a.mp + blocks - 1) / blocks);
  a.rows_per_block = std::min<int64_t>(a.rows_per_block, kMaxBlockRows);
}

size_t act_bwd_segmax_bytes(const ActBwdArgs& a) { return (size_t)a.M * a.tiles * 2; }
size_t act_bwd_band_elems(const ActBwdArgs& a) { return (size_t)std::max(1, a.bands) * a.tiles * kTile; }
size_t act_bwd_columns(const ActBwdArgs& a) { return (size_t)a.tiles * kTile; }

hipError_t launch_act_bwd(const ActBwdArgs& a, int act, int round, hipStream_t stream) {
  if (a.bands > 0) {
    const dim3 grid((unsigned)a.tiles, (unsigned)a.bands);
    switch (act) {
      case kActRelu: act_grad_stats<kActRelu><<<grid, kBwdThreads, 0, stream>>>(a); break;
      case kActGelu: act_grad_stats<kActGelu><<<grid, kBwdThreads, 0, stream>>>(a); break;
      case kActGeluTanh: act_grad_stats<kActGeluTanh><<<grid, kBwdThreads, 0, stream>>>(a); break;
      case kActSilu: act_grad_stats<kActSilu><<<grid, kBwdThreads, 0, stream>>>(a); break;
      default: act_grad_stats<kActNone><<<grid, kBwdThreads, 0, stream>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  act_grad_join<<<(unsigned)(a.tiles * kTile / 64), kBwdThreads, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.row_codes && !a.col_codes)) return e;
  const dim3 grid((unsigned)(a.tiles * std::max<int64_t>(1, (a.mp + a.rows_per_block - 1) / a.rows_per_block)));
  if (round == 0) act_grad_quant<false, true><<<grid, kBwdThreads, 0, stream>>>(a);
  else if (a.N % 4 == 0) act_grad_quant<true, true><<<grid, kBwdThreads, 0, stream>>>(a);
  else act_grad_quant<true, false><<<grid, kBwdThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace i8mp
