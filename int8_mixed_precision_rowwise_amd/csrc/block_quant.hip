// Block-scaled FP8 codes of activations, gradients and weights (block.h has the format).
//
// A workgroup takes 128 rows (one block of one expert's) by 256 columns and holds them in
// registers: thread t has the 8 columns of chunk t % 32 in rows t / 32, t / 32 + 8, ...  So
// the source is read once whatever is wanted of it: the maxima along the rows come from the
// 16 lanes that share a row's block (DPP), those down the rows from a thread's 16 rows, joined
// across the workgroup in LDS.  Bound by memory: 2 bytes read and 1 (2 with both codes) written
// for each element.  8192 x 2048 along the rows 13 us (3.9 TB/s), a weight of 5632 x 2048 9.8, dY of 16384 x 5632 both ways
// and X of 16384 x 2048 down its rows 84 (5.6 TB/s, some of it from the last level); 1551 rows of 13 experts 11, which is a
// chain of dependent loads (offsets, index, rows) and one round of workgroups.
#include "block.h"
#include "quant_device.h"

namespace i8mp {
namespace {

constexpr int kTileRows = kBlock, kTileCols = 256, kLanes = kTileCols / 8, kGroups = kThreads / kLanes;
constexpr int kPer = kTileRows / kGroups;  // rows a thread holds

__device__ __forceinline__ us2 max_of_row16(us2 m) {  // over 16 lanes
  const auto step = [&](int moved) { m = __builtin_elementwise_max(m, as_us2((uint32_t)moved)); };
  step(__builtin_amdgcn_update_dpp(0, (int)__builtin_bit_cast(uint32_t, m), 0xB1, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, (int)__builtin_bit_cast(uint32_t, m), 0x4E, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, (int)__builtin_bit_cast(uint32_t, m), 0x141, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, (int)__builtin_bit_cast(uint32_t, m), 0x140, 0xF, 0xF, false));
  return m;
}

// Eight codes of a chunk under one scale.
__device__ __forceinline__ uint2 codes_of(const uint4& v, float scale) {
  return make_uint2(codes4(v.x, v.y, scale), codes4(v.z, v.w, scale));
}

// Eight codes of a chunk, each under a scale of its own (the conversion above takes one for two): inv is 2^-e.
__device__ __forceinline__ uint2 codes_of_columns(const uint4& v, const float* inv) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = elem(v, j) * inv[j];
  return make_uint2(pack_f8x4(f[0], f[1], f[2], f[3]), pack_f8x4(f[4], f[5], f[6], f[7]));
}

struct QuantLds {
  uint8_t byte[2][kTileRows];           // exponents along the rows
  uint4 colmax[kThreads / 64][kLanes];  // column maxima of each wave
};

__device__ __forceinline__ us2 max4(us2 a, us2 b) { return __builtin_elementwise_max(a, b); }

template <bool ROWS, bool COLS>
__device__ __forceinline__ void quant_tile(const BlockQuant& q, int64_t slot, int64_t ct, QuantLds& lds) {
  Place p;
  if (!locate<kTileRows>(q.rag, slot, p)) return;  // workgroup-uniform
  const int t = threadIdx.x, c = t % kLanes, g = t / kLanes;
  const int64_t col = ct * kTileCols + 8 * c;
  const int rows = (int)min((int64_t)kTileRows, p.count - p.local);
  const int64_t r0 = p.first + p.local;
  // Rows and columns past the tile's read its last row and first columns, and become zeros below: loads without
  // branches, so that all of a thread's are under way together.
  uint4 v[kPer];
  int64_t src[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) src[i] = r0 + min(g + kGroups * i, rows - 1);
  if (q.index) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) src[i] = q.index[src[i]];
  }
  const uint16_t* x = q.x + (col < q.cols ? col : 0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool there = !q.index || (src[i] >= 0 && src[i] < q.n_src);
    v[i] = *reinterpret_cast<const uint4*>(x + (there ? src[i] : 0) * q.ldx);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool there = !q.index || (src[i] >= 0 && src[i] < q.n_src);
    if (!there || g + kGroups * i >= rows) v[i] = make_uint4(0, 0, 0, 0);
  }
  if (col + 8 > q.cols) {
    const int keep = (int)max((int64_t)0, q.cols - col);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = keep_first(v[i], keep);
  }
  if constexpr (COLS) {
    us2 m[4] = {{0, 0}, {0, 0}, {0, 0}, {0, 0}};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      m[0] = max4(m[0], as_us2(v[i].x & 0x7FFF7FFFu)), m[1] = max4(m[1], as_us2(v[i].y & 0x7FFF7FFFu));
      m[2] = max4(m[2], as_us2(v[i].z & 0x7FFF7FFFu)), m[3] = max4(m[3], as_us2(v[i].w & 0x7FFF7FFFu));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = max4(m[j], as_us2((uint32_t)__shfl_xor((int)__builtin_bit_cast(uint32_t, m[j]), 32)));
    if ((t & 63) < kLanes)
      lds.colmax[t >> 6][c] = make_uint4(__builtin_bit_cast(uint32_t, m[0]), __builtin_bit_cast(uint32_t, m[1]),
                                         __builtin_bit_cast(uint32_t, m[2]), __builtin_bit_cast(uint32_t, m[3]));
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      // two rows' maxima in the halves of one word
      const us2 a = absmax_bits((us2){0, 0}, v[i]), b = absmax_bits((us2){0, 0}, v[i + 1]);
      const us2 m = max_of_row16(max4((us2){a.x, b.x}, (us2){a.y, b.y}));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = g + kGroups * (i + k);
        const uint32_t byte = exponent_byte(k ? m.y : m.x);
        if ((c & 15) == 0) lds.byte[c >> 4][r] = (uint8_t)byte;
        if (r < rows && col < q.ldq) {
          const uint2 w = codes_of(v[i + k], scale_of(byte));
          *reinterpret_cast<uint2*>(q.q_row + (16 * unit_of<16>(p) + p.local + r) * q.ldq + col) = w;
        }
      }
    }
  }
  __syncthreads();
  if constexpr (ROWS) {
    if (t < rows)  // both blocks' exponents; the second one's place is there even where its columns are not
      *reinterpret_cast<uint16_t*>(q.s_row + (16 * unit_of<16>(p) + p.local + t) * q.ld_srow + 2 * ct) =
          (uint16_t)(lds.byte[0][t] | lds.byte[1][t] << 8);
  }
  if constexpr (COLS) {
    if (col < q.ldq) {
      us2 m[4] = {{0, 0}, {0, 0}, {0, 0}, {0, 0}};
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) {
        const uint4 o = lds.colmax[w][c];
        m[0] = max4(m[0], as_us2(o.x)), m[1] = max4(m[1], as_us2(o.y)), m[2] = max4(m[2], as_us2(o.z)), m[3] = max4(m[3], as_us2(o.w));
      }
      float inv[8];
      uint32_t byte[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        byte[j] = exponent_byte(j & 1 ? m[j >> 1].y : m[j >> 1].x);
        inv[j] = inverse_scale(byte[j]);
      }
      if (g == 0)
        *reinterpret_cast<uint2*>(q.s_col + (unit_of<kTileRows>(p) + p.local / kTileRows) * q.ld_scol + col) =
            make_uint2(pack4(byte[0], byte[1], byte[2], byte[3]), pack4(byte[4], byte[5], byte[6], byte[7]));
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = g + kGroups * i;
        if (r < rows) *reinterpret_cast<uint2*>(q.q_col + (r0 + r) * q.ldq + col) = codes_of_columns(v[i], inv);
      }
    }
  }
}

__device__ __forceinline__ void spread(const SpreadJob& s, int64_t i) {  // 16 bytes
  const int64_t per = s.ld / 16, planes = s.along ? s.nb : s.kb;
  const int64_t at = i % per, plane = i / per % planes, e = i / (per * planes);
  const int64_t other = min(at * 16 / kBlock, (s.along ? s.kb : s.nb) - 1);
  const uint32_t b = s.exps[e * s.nb * s.kb + (s.along ? plane * s.kb + other : other * s.kb + plane)] * 0x01010101u;
  reinterpret_cast<uint4*>(s.planes)[i] = make_uint4(b, b, b, b);
}

// Workgroups: `na` of a, `nb` of b, the rest spreads exponents.
template <bool ROWS, bool COLS, bool SECOND>
__global__ __launch_bounds__(kThreads) void quant_blocks(BlockQuant a, BlockQuant b, SpreadJob s, int64_t na, int64_t nb) {
  __shared__ QuantLds lds;
  int64_t wg = blockIdx.x;
  if (wg < na) {
    const int64_t cts = (a.cols + kTileCols - 1) / kTileCols;
    quant_tile<ROWS, COLS>(a, wg / cts, wg % cts, lds);
    return;
  }
  wg -= na;
  if constexpr (SECOND) {
    if (wg < nb) {
      const int64_t cts = (b.cols + kTileCols - 1) / kTileCols;
      quant_tile<false, true>(b, wg / cts, wg % cts, lds);
      return;
    }
    wg -= nb;
  }
  const int64_t i = wg * kThreads + threadIdx.x;
  if (i < s.groups()) spread(s, i);
}

// Weights: one exponent for each 128 x 128.
__global__ __launch_bounds__(kThreads) void quant_weight(const uint16_t* __restrict__ w, int64_t N, int64_t K, int64_t ldw,
                                                         int64_t stride, uint8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  __shared__ uint32_t red[2][kThreads / 64];
  const int t = threadIdx.x, c = t % kLanes, g = t / kLanes;
  const int64_t cts = (K + kTileCols - 1) / kTileCols, rts = (N + kTileRows - 1) / kTileRows;
  const int64_t ct = blockIdx.x % cts, rt = blockIdx.x / cts % rts, e = blockIdx.x / (cts * rts);
  const int64_t col = ct * kTileCols + 8 * c, Kp = (K + 15) / 16 * 16, kb = (K + kBlock - 1) / kBlock;
  const int rows = (int)min((int64_t)kTileRows, N - rt * kTileRows);
  w += e * stride + rt * kTileRows * ldw + (col < K ? col : 0);
  uint4 v[kPer];
  us2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = *reinterpret_cast<const uint4*>(w + min(g + kGroups * i, rows - 1) * ldw);  // as in quant_tile
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (g + kGroups * i >= rows) v[i] = make_uint4(0, 0, 0, 0);
  if (col + 8 > K) {
    const int keep = (int)max((int64_t)0, K - col);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = keep_first(v[i], keep);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = absmax_bits(m, v[i]);
  m = max_of_row16(m);
  uint32_t a = max((uint32_t)m.x, (uint32_t)m.y);
  a = max(a, (uint32_t)__shfl_xor((int)a, 32));  // the wave's other row group
  if ((t & 47) == 0) red[(t >> 4) & 1][t >> 6] = a;
  __syncthreads();
  const int half = c >> 4;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) a = max(a, red[half][i]);
  const uint32_t byte = exponent_byte(a);
  const float scale = scale_of(byte);
  if (g == 0 && (c & 15) == 0 && col < K) exps[(e * rts + rt) * kb + 2 * ct + half] = (uint8_t)byte;
  if (col >= Kp) return;
  uint8_t* dst = codes + (e * N + rt * kTileRows) * Kp + col;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = g + kGroups * i;
    if (r < rows) *reinterpret_cast<uint2*>(dst + r * Kp) = codes_of(v[i], scale);
  }
}

int64_t tiles(const BlockQuant& q) {
  const int64_t slots = q.rag.off ? ragged_units(q.rag.rows, q.rag.E, kTileRows) : (q.rag.rows + kTileRows - 1) / kTileRows;
  return slots * ((q.cols + kTileCols - 1) / kTileCols);
}

}  // namespace

hipError_t launch_block_quant(const BlockQuant& a, const BlockQuant* b, const SpreadJob& s, hipStream_t stream) {
  const int64_t na = tiles(a), nb = b ? tiles(*b) : 0;
  const int64_t n = na + nb + (s.groups() + kThreads - 1) / kThreads;
  if (n == 0) return hipSuccess;
  const BlockQuant& second = b ? *b : a;
  const unsigned grid = (unsigned)n;
  if (b) {
    if (a.q_row)
      quant_blocks<true, true, true><<<grid, kThreads, 0, stream>>>(a, second, s, na, nb);
    else
      quant_blocks<false, true, true><<<grid, kThreads, 0, stream>>>(a, second, s, na, nb);
  } else {
    quant_blocks<true, false, false><<<grid, kThreads, 0, stream>>>(a, second, s, na, nb);
  }
  return hipGetLastError();
}

hipError_t launch_block_quant_weight(const uint16_t* w, int64_t E, int64_t N, int64_t K, int64_t ldw, int64_t stride,
                                     uint8_t* codes, uint8_t* exps, hipStream_t stream) {
  const int64_t n = E * ((N + kTileRows - 1) / kTileRows) * ((K + kTileCols - 1) / kTileCols);
  if (n == 0) return hipSuccess;
  quant_weight<<<(unsigned)n, kThreads, 0, stream>>>(w, N, K, ldw, stride, codes, exps);
  return hipGetLastError();
}

}  // namespace i8mp
