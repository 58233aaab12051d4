// A few rows of each expert (or of the one matrix) against weight codes: Y = X W^T.
//
// Bound by reading the codes, once, and everything else is small.  A workgroup takes 16 CT outputs of an
// expert; its 8 waves share the contraction, wave w taking every eighth block of 128, so that the workgroup
// reads 1 KiB of each weight row at a time.  Codes go from memory straight into the matrix instruction's
// registers (lane l holds 32 codes of row l % 16).  While the first are on their way the workgroup quantizes X
// into LDS, 32 / MT blocks of the contraction at a time: a block of a row lies in 16 lanes of one wave, so its
// maximum takes four DPP moves.  v_mfma_scale_f32_16x16x128_f8f6f4 multiplies a whole block and applies both
// scales; within a block the order of the contraction does not matter, so lane l takes the 16 bytes at
// 16 (l / 16) and those at 64 more, which reads whole 64-byte pieces of a row at once.  The waves' sums are
// joined in LDS in a fixed order.  One row against 14336 x 4096 takes 13.9 us (4.2 TB/s of 58.7 MB), 64 rows of 32
// experts of 1024 x 2048 14.5: the launch, the first codes' way and the join are some 3 of them.
#include "block.h"
#include "quant_device.h"

#include <algorithm>

namespace i8mp {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;

__device__ __forceinline__ v8i join(const v4i& lo, const v4i& hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

template <int MT, int CT, int U>
__global__ __launch_bounds__(kFewThreads, 4) void block_few(BlockFew a, uint32_t tiles) {
  constexpr int RT = 16 * MT, P = U * kFewWaves;               // rows; blocks of a phase, U of a wave
  constexpr int PITCH = P * kBlock + 16;                       // rows start in different banks
  constexpr int Q = 4;                                         // chunks of X that a thread has in flight
  extern __shared__ __attribute__((aligned(16))) int8_t lds[];  // codes of X, later the waves' sums
  __shared__ uint8_t byte[RT][P];
  const int t = threadIdx.x, lane = t & 63, li = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const uint32_t wg = blockIdx.x, e = wg / tiles, tile = wg - e * tiles;
  int64_t first = 0, count = a.rag.rows;
  if (a.rag.off) {
    first = offset_at(a.rag, e);
    count = offset_at(a.rag, e + 1) - first;
  }
  // Behind everything that is read: a store before would keep the offsets and the index out of scalar loads.
  const OtherRows other = a.clear ? other_rows(a.rag) : OtherRows{0, 0, 0};
  const auto clear = [&]() __attribute__((always_inline)) {
    for (int64_t i = wg; i < other.count; i += gridDim.x)
      for (int64_t c = t; c < a.N; c += kFewThreads) a.Y[other.row(i) * a.ldy + c] = 0;
  };
  if (count <= 0) return clear();  // workgroup-uniform
  const int64_t n0 = (int64_t)tile * (16 * CT);
  const int K = (int)a.K, Kp = (K + 15) & ~15, blocks = (K + kBlock - 1) / kBlock;
  const uint8_t* const w = a.codes + (e * a.N + n0) * Kp;
  const uint8_t* ex[CT];
  uint32_t row[CT];  // this lane's weight row; rows past the last one repeat it: their outputs are not stored
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    row[j] = (uint32_t)(min(n0 + 16 * j + li, a.N - 1) - n0) * Kp;
    ex[j] = a.exps + (e * ((a.N + kBlock - 1) / kBlock) + min(n0 + 16 * j, a.N - 1) / kBlock) * blocks;
  }
  v4i lo[U][CT], hi[U][CT];
  int ew[U][CT];
  // A wave's u-th block of the phase from block p0 on.  What lies behind the row's end reads its last chunk
  // or block again, against zeros of X: no load has a branch around it.
  const auto load = [&](int u, int p0) __attribute__((always_inline)) {
    const int b = min(p0 + wave + kFewWaves * u, blocks - 1), k = b * kBlock + 16 * q;
    const uint32_t k0 = min(k, Kp - 16), k1 = min(k + 64, Kp - 16);
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      lo[u][j] = *reinterpret_cast<const v4i*>(w + (row[j] + k0));
      hi[u][j] = *reinterpret_cast<const v4i*>(w + (row[j] + k1));
      ew[u][j] = ex[j][b];
    }
  };
  const int last = (K - 1) & ~7;  // X's last chunk
  for (int64_t r0 = 0; r0 < count; r0 += RT) {
    const int rows = (int)min((int64_t)RT, count - r0);
    v4f acc[MT][CT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = 0; p0 < blocks; p0 += P) {
      // X of this phase: 16 chunks of 8 values for each block; a wave's 64 lie in one row
      const int chunks = rows * P * 16;
      for (int c0 = 0; c0 < chunks; c0 += Q * kFewThreads) {
        // Every load first, and what has to be zeros cleared where it is used: a load whose value is looked at
        // here would be waited for here.
        uint4 v[Q];
        uint32_t keep[Q];
        int64_t src[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          const int c = c0 + i * kFewThreads + 64 * wave, r = min(c / (P * 16), rows - 1);
          src[i] = first + r0 + r;
          if (a.index) src[i] = a.index[src[i]];
        }
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          const int c = c0 + i * kFewThreads + 64 * wave, k = p0 * kBlock + 8 * (c % (P * 16) + lane);
          const bool some = !a.index || (src[i] >= 0 && src[i] < a.n_src);
          keep[i] = some && k < K ? ~0u : 0u;
          const int64_t at = some ? src[i] : 0;
          v[i] = *reinterpret_cast<const uint4*>(a.x + at * a.ldx + min(k, last));
        }
        // the weights' loads go out behind the first values of X, which are waited for first
        if (c0 == 0) {
#pragma unroll
          for (int u = 0; u < U; ++u) load(u, p0);
        }
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          const int c = c0 + i * kFewThreads + 64 * wave, r = c / (P * 16), in = c % (P * 16) + lane, k = p0 * kBlock + 8 * in;
          if (c >= chunks) break;
          v[i] = make_uint4(v[i].x & keep[i], v[i].y & keep[i], v[i].z & keep[i], v[i].w & keep[i]);
          if (k + 8 > K && k < K) v[i] = keep_first(v[i], K - k);
          const us2 m2 = absmax_bits((us2){0, 0}, v[i]);
          uint32_t m = max((uint32_t)m2.x, (uint32_t)m2.y);
          m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
          m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
          m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
          m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
          const uint32_t b = exponent_byte(m);
          const float scale = scale_of(b);
          *reinterpret_cast<uint2*>(lds + r * PITCH + 8 * in) = make_uint2(codes4(v[i].x, v[i].y, scale), codes4(v[i].z, v[i].w, scale));
          if ((lane & 15) == 0) byte[r][in >> 4] = (uint8_t)b;
        }
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = wave + kFewWaves * u;  // of this phase
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int r = min(16 * i + li, rows - 1);  // rows past the last one repeat it
          const int8_t* at = lds + r * PITCH + b * kBlock + 16 * q;
          const v8i fx = join(*reinterpret_cast<const v4i*>(at), *reinterpret_cast<const v4i*>(at + 64));
          // formats 0, 0: E4M3 for both; the weights first, so that a lane's results are adjacent in a row
#pragma unroll
          for (int j = 0; j < CT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(lo[u][j], hi[u][j]), fx, acc[i][j], 0, 0, 0, ew[u][j],
                                                                         0, (int)byte[r][b]);
        }
      }
      __syncthreads();
    }
    v4f(*red)[MT * CT][64] = reinterpret_cast<v4f(*)[MT * CT][64]>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) red[wave][i * CT + j][lane] = acc[i][j];
    __syncthreads();
    for (int o = t; o < MT * CT * 64; o += kFewThreads) {
      const int at = o >> 6, l = o & 63;
      v4f s = red[0][at][l];
#pragma unroll
      for (int v = 1; v < kFewWaves; ++v) s += red[v][at][l];
      const int64_t r = r0 + 16 * (at / CT) + (l & 15), n = n0 + 16 * (at % CT) + 4 * (l >> 4);
      if (r >= count) continue;
      __bf16* y = reinterpret_cast<__bf16*>(a.Y) + (first + r) * a.ldy + n;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n + c < a.N) y[c] = (__bf16)s[c];  // round to nearest even
    }
    __syncthreads();  // the sums have been read
  }
  clear();
}

template <int MT, int CT, int U>
void launch(const BlockFew& a, hipStream_t stream) {
  const int64_t tiles = (a.N + 16 * CT - 1) / (16 * CT), E = a.rag.off ? a.rag.E : 1;
  const int64_t rows = a.rag.off ? 16 * MT : std::min<int64_t>(16 * MT, a.rag.rows);
  const size_t codes = (size_t)(rows * (U * kFewWaves * kBlock + 16)), sums = (size_t)kFewWaves * MT * CT * 64 * 16;
  block_few<MT, CT, U><<<(unsigned)(tiles * E), kFewThreads, std::max(codes, sums), stream>>>(a, (uint32_t)tiles);
}

}  // namespace

// One tile of outputs a workgroup while each CU gets at most one workgroup, beyond that two, which share X.  Both
// sides, one and two: 1 row against 14336 x 4096 15.3 us and 14.2, 13 rows 24.9 and 19.3, 13 against 5003 x 2040 9.0
// and 8.0; 1 against 4096 x 14336 16.2 and 21.4, 4 against 4096 x 4096 6.6 and 9.6.
constexpr int64_t kFewWide = 16 * 256;

// Rows of one matrix, or of an expert on average, that this kernel takes: against the tiles' kernel and the quantization
// before it, 16 rows against 4096 x 14336 33.8 us and 64.3; 17 against 5632 x 2048 8.3 and 17.1; 32 against 14336 x 4096
// 28.4 and 25.9, 33 against 5632 x 2048 11.6 and 17.2 (64 rows 42.3 and 26.8 of 14336 x 4096).  The border moves with the
// codes' number, which the rule leaves out: near it the worse of the two is taken, at 2.5 us more for 32 rows of the
// larger weight and 5.6 for 33 of the smaller.
constexpr int64_t kFewRows = 32;

// Rows of all experts, which may lie unevenly: an expert's rows beyond 32 read its codes again.  This kernel's time and the
// tiles' over experts of 1024 x 2048, 8 of 2048 x 2048 or 128 of 768 x 2048: 64 rows of 8 10.3 us and 20.1, 128 of 8 17.4
// and 20.2 (22.3 and 19.9 with 34 of them in one), 128 of 32 17.7 and 21.5 (43 and 20 with all in one), 128 of 128 30.3 and
// 31.9, 256 of 32 20.0 and 21.9 (24.7 and 21.9 with 27 in one), 512 of 32 30 and 22 (52 and 23 with 111 in one).
constexpr int64_t kFewAll = 128;

bool block_few_takes(int64_t rows, int64_t E, int64_t N, int64_t K) {
  if (N < 1 || K < 1 || rows < 1) return false;
  const int64_t e = std::max<int64_t>(E, 1);
  return rows <= (E > 0 ? std::min(kFewRows * e, kFewAll) : kFewRows) && e * ((N + 15) / 16) < (int64_t(1) << 22);
}

// Blocks a wave has in flight: 2, or 4 where only one tile is held and the contraction is long enough for 4
// (1 row against 4096 x 4096: 7.1 us with 2, 6.2 with 4; against 5632 x 2048 with one tile 6.8 with 2, 8.0 with 4).
hipError_t launch_block_few(const BlockFew& a, hipStream_t stream) {
  const int64_t e = a.rag.off ? a.rag.E : 1, each = (a.rag.rows + e - 1) / e;
  const bool wide = a.N * e > kFewWide, long_k = a.K > 16 * kBlock;
  if (each > 16) {
    wide ? launch<2, 2, 2>(a, stream) : launch<2, 1, 2>(a, stream);
  } else if (wide) {
    launch<1, 2, 2>(a, stream);
  } else {
    long_k ? launch<1, 1, 4>(a, stream) : launch<1, 1, 2>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace i8mp
