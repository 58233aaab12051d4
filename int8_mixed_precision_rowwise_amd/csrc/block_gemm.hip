// Products of block-scaled FP8 codes, for one matrix or for the ragged rows of many experts.
//
// The pipeline is the FP8 GEMM's (gemm_pipelined.h): slabs of 64 of the contraction go from
// memory straight into LDS, four deep, and feed v_mfma_scale_f32_32x32x64_f8f6f4.  That
// instruction multiplies each lane's 32 contraction values by a power of two of its own, so the
// blocks' scales cost no vector operation: a lane needs the exponent's byte of its row (or
// column) of each 128, which lies in planes [block][row] and comes into LDS the same way as the
// codes, four blocks at a time (one more load a wave for every eight slabs).
#include "block.h"
#include "gemm_pipelined.h"

namespace i8mp {
namespace {

// The tile of a workgroup among the rows that the experts have: tiles of BM rows, expert after
// expert.  Every wave adds up the experts' tiles by itself (64 experts at a time).
struct RaggedTile {
  int64_t tiles;  // of all experts
  Place p;        // of tile `tm`, if tm < tiles
};

template <int BM>
__device__ __forceinline__ int64_t ragged_tiles(const Ragged& r) {
  if (!r.off) return (r.rows + BM - 1) / BM;
  int64_t n = 0;
  for (int64_t e = threadIdx.x & 63; e < r.E; e += 64) n += max((int64_t)0, offset_at(r, e + 1) - offset_at(r, e) + BM - 1) / BM;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  return n;
}

template <int BM>
__device__ __forceinline__ void ragged_place(const Ragged& r, int64_t tm, Place& p) {
  if (!r.off) {
    p.e = 0, p.first = 0, p.count = r.rows, p.local = tm * BM;
    return;
  }
  const int lane = threadIdx.x & 63;
  int64_t before = 0;  // tiles of the experts before this turn's 64
  for (int64_t e0 = 0; e0 < r.E; e0 += 64) {
    const int64_t e = e0 + lane;
    int64_t n = e < r.E ? max((int64_t)0, offset_at(r, e + 1) - offset_at(r, e) + BM - 1) / BM : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t up = __shfl_up(n, o);
      if (lane >= o) n += up;
    }
    const uint64_t past = __ballot(before + n > tm);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int64_t start = at ? before + __shfl(n, at - 1) : before;
      p.e = e0 + at;
      p.first = offset_at(r, p.e);
      p.count = offset_at(r, p.e + 1) - p.first;
      p.local = (tm - start) * BM;
      return;
    }
    before += __shfl(n, 63);
  }
  p.e = 0, p.first = 0, p.count = 0, p.local = 0;  // not reached: tm is one of the experts' tiles
}

// Consecutive workgroups go to the 8 XCDs in turn; each XCD gets a contiguous run of n tiles.
__device__ __forceinline__ int64_t xcd_run(int64_t wg, int64_t n) {
  const int64_t x = wg & 7;
  return x * (n >> 3) + min(x, n & 7) + (wg >> 3);
}

// bf16 of 32 x 32 accumulators through LDS, whole rows at a time (or element by element where
// C's rows do not start every 16 bytes).
template <int TM, int TN, bool VEC>
__device__ __forceinline__ void store_rows(const v16f (&acc)[TM][TN], int8_t* mine, uint16_t* __restrict__ C, int64_t ldc,
                                           int64_t rows, int64_t cols, int lane) {
  constexpr int WM = 32 * TM, WN = 32 * TN, CPR = WN / 8, PITCH = WN * 2, RPI = 64 / CPR;
  const int mr = lane & 31, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 32 * i + mr, chunk = 4 * j + q;
        __bf16 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (__bf16)acc[i][j][4 * q + e];  // round to nearest even
        *reinterpret_cast<uint2*>(mine + r * PITCH + ((chunk ^ (r & (CPR - 1))) << 4) + 8 * half) = __builtin_bit_cast(uint2, h);
      }
  __syncthreads();
  const int c = lane % CPR;
#pragma unroll 4
  for (int r0 = 0; r0 < WM; r0 += RPI) {
    const int r = r0 + lane / CPR;
    const uint4 v = *reinterpret_cast<const uint4*>(mine + r * PITCH + ((c ^ (r & (CPR - 1))) << 4));
    if (r >= rows || 8 * c >= cols) continue;
    uint16_t* dst = C + r * ldc + 8 * c;
    if (VEC && 8 * c + 8 <= cols) {
      __builtin_nontemporal_store(__builtin_bit_cast(v4i, v), reinterpret_cast<v4i*>(dst));
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * c + e < cols) dst[e] = h[e];
    }
  }
}

// Exponents of four blocks of one tile's rows and columns, (kind, block) at bytes
// (4 kind + block) * BM of the buffer: each wave loads 256 of its bytes.
template <int BM, int NW>
struct Exponents {
  const uint8_t* base;
  int64_t ld, left;  // plane pitch, bytes from base to the end of the planes
  int64_t first;     // of this lane within four planes
  __device__ __forceinline__ void init(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, int64_t a0, int64_t b0,
                                       int64_t blocks, int wave, int lane) {
    const bool is_b = wave >= NW / 2;
    const int k = NW == 8 ? wave & 3 : 2 * (wave & 1) + (lane >> 5);
    base = is_b ? b + b0 : a + a0;
    ld = is_b ? ldb : lda;
    left = blocks * ld - (is_b ? b0 : a0);
    first = k * ld + 4 * (NW == 8 ? lane : lane & 31);
  }
  __device__ __forceinline__ void issue(int8_t* buf, int64_t group, int wave) const {
    const int64_t skip = 4 * group * ld;
    const v4u r = Dma<64, true, NW>::make_rsrc(reinterpret_cast<const int8_t*>(base + skip),
                                               max((int64_t)0, min(left - skip, (int64_t)kOob)));
    const uint32_t o = (uint32_t)first;
    const uint32_t l = (uint32_t)__builtin_amdgcn_readfirstlane(
        (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)(buf + wave * 256)));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(l), "v"(o), "s"(r)
                 : "memory", "m0");
  }
};

template <int BM, int WGN, BlockProduct WHAT, bool REBASE, bool VEC>
__global__ __launch_bounds__(128 * WGN) void block_gemm(BlockGemm g) {
  constexpr int BN = BM, NW = 2 * WGN, NT = 64 * NW;
  constexpr int WM = BM / 2, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  constexpr bool AK = WHAT != kBlockWeight, BKM = WHAT == kBlockForward;
  constexpr int A_BYTES = BM * BK, SLAB = A_BYTES + BN * BK;
  constexpr int EXPS = 8 * BM;  // bytes of four blocks' exponents
  typedef Dma<BM, AK, NW, REBASE && !AK> DA;
  typedef Dma<BN, BKM, NW, REBASE && !BKM> DB;
  constexpr int NA = DA::kInst, PER = NA + DB::kInst;
  using S = SlabSchedule<TM, TN, PER>;
  static_assert(NW * WM * WN * 2 <= STAGES * SLAB, "the outputs fit where the slabs were");
  __shared__ __attribute__((aligned(1024))) int8_t lds[STAGES * SLAB + 2 * EXPS];
  int8_t* const exps = lds + STAGES * SLAB;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);

  const int64_t tiles_n = (g.cols_out + BN - 1) / BN;
  int64_t tiles_m, tm, tn, wg = blockIdx.x;
  Place p;
  if constexpr (WHAT == kBlockWeight) {
    tiles_m = (g.rows_out + BM - 1) / BM;
    const int64_t each = tiles_m * tiles_n;
    wg = xcd_run(wg, gridDim.x);
    p.e = wg / each;
    wg -= p.e * each;
    p.local = 0, p.first = 0, p.count = g.rag.rows;
    if (g.rag.off) {
      p.first = offset_at(g.rag, p.e);
      p.count = max((int64_t)0, offset_at(g.rag, p.e + 1) - p.first);
    }
  } else {
    tiles_m = ragged_tiles<BM>(g.rag);
    if (g.clear && g.rag.off) {
      for (int64_t r = offset_at(g.rag, g.rag.E) + wg; r < g.rag.rows; r += gridDim.x)
        for (int64_t c = t; c < g.cols_out; c += NT) g.C[r * g.ldc + c] = 0;
    }
    if (wg >= tiles_m * tiles_n) return;
    wg = xcd_run(wg, tiles_m * tiles_n);
  }
  {  // groups of 4 tile rows, so that the tiles of an XCD share panels in its L2
    const int64_t group = wg / (4 * tiles_n), first = 4 * group, rows = min(tiles_m - first, (int64_t)4);
    const int64_t in = wg - group * 4 * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
  }
  int64_t K = g.contraction, a_rows, c_rows;  // contraction; rows of A in this tile's operand; C's rows in this tile
  const int8_t *A = reinterpret_cast<const int8_t*>(g.A), *B = reinterpret_cast<const int8_t*>(g.B);
  const uint8_t *sA = g.sA, *sB = g.sB;
  int64_t m0 = tm * BM, n0 = tn * BN;
  uint16_t* C = g.C + n0;
  if constexpr (WHAT == kBlockWeight) {
    K = p.count;
    A += p.first * g.lda, B += p.first * g.ldb;
    sA += unit_of<kBlock>(p) * g.ldsa, sB += unit_of<kBlock>(p) * g.ldsb;
    a_rows = g.lda;
    c_rows = g.rows_out - m0;
    C += p.e * g.c_stride + m0 * g.ldc;
  } else {
    ragged_place<BM>(g.rag, tm, p);
    m0 = 16 * unit_of<16>(p) + p.local;
    a_rows = m0 + p.count - p.local;
    c_rows = p.count - p.local;
    B += p.e * g.b_stride, sB += p.e * g.sb_stride;
    C += (p.first + p.local) * g.ldc;
  }
  const int wm0 = (wave / WGN) * WM, wn0 = (wave % WGN) * WN;
  const int nk = (int)((K + BK - 1) / BK);
  const int64_t blocks = (K + kBlock - 1) / kBlock;

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = Mma<1>::zero();

  if (nk > 0) {  // an expert without rows: workgroup-uniform
    DA da;
    DB db;
    da.init(A, g.lda, m0, a_rows, K, wave, lane);
    db.init(B, g.ldb, n0, BKM ? g.cols_out : g.ldb, K, wave, lane);
    Exponents<BM, NW> ex;
    ex.init(sA, g.ldsa, sB, g.ldsb, m0, n0, blocks, wave, lane);

    v8i a[TM], b0[TN], b1[TN];
    int ea[TM], eb[TN], na[TM], nb[TN];  // exponents of this block and the next
    const auto read_exps = [&](int block) __attribute__((always_inline)) {
      const int8_t* at = exps + ((block >> 2) & 1) * EXPS + (block & 3) * BM + (lane & 31);
#pragma unroll
      for (int i = 0; i < TM; ++i) na[i] = *reinterpret_cast<const uint8_t*>(at + wm0 + 32 * i);
#pragma unroll
      for (int j = 0; j < TN; ++j) nb[j] = *reinterpret_cast<const uint8_t*>(at + 4 * BM + wn0 + 32 * j);
    };
    const auto next_exps = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TM; ++i) ea[i] = na[i];
#pragma unroll
      for (int j = 0; j < TN; ++j) eb[j] = nb[j];
    };
    const auto mma = [&](const v8i& bf, const v8i& af, int i, int j) __attribute__((always_inline)) {
      // formats 0, 0: E4M3 for both; the first operand is B, so that a lane's results are adjacent in a row
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf, af, acc[i][j], 0, 0, 0, eb[j], 0, ea[i]);
    };
    // A group of exponents goes out ahead of the slab that starts it, so it has landed whenever that
    // slab has; the waits below count slab loads and are at most stricter for the loads between them.
    ex.issue(exps, 0, wave);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      da.issue(lds + s * SLAB, s, K, wave);
      db.issue(lds + s * SLAB + A_BYTES, s, K, wave);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm((STAGES - 1) * PER));  // slab 0 has landed
    lds_barrier();
    read_exps(0);
    next_exps();
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = frag32f8<BM, AK>(lds, wm0 + 32 * i, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j) b0[j] = frag32f8<BN, BKM>(lds + A_BYTES, wn0 + 32 * j, lane);

    // One slab, as in gemm_pipelined.h: slab kt is multiplied from registers while slab kt + 1 is read
    // from LDS and slab kt + STAGES goes into slab kt's place.  ODD: the second half of a block, which
    // reads the next block's exponents.
    auto slab = [&](v8i(&bc)[TN], v8i(&bn)[TN], int kt, bool odd, bool tail) __attribute__((always_inline)) {
      const int8_t* nxt = lds + ((kt + 1) % STAGES) * SLAB;
      int8_t* dst = lds + (kt % STAGES) * SLAB;
      const int ns = kt + STAGES;
#pragma unroll
      for (int m = 0; m < S::HA; ++m) {
        mma(bc[m % TN], a[m / TN], m / TN, m % TN);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((STAGES - 2) * PER));  // slab kt + 1 has landed
      lds_barrier();
      if (odd) read_exps((kt + 1) >> 1);
      if (!tail && (ns & 7) == 0 && ns < nk) ex.issue(exps + ((ns >> 3) & 1) * EXPS, ns >> 3, wave);
#pragma unroll
      for (int m = S::HA; m < S::NM; ++m) {
        mma(bc[m % TN], a[m / TN], m / TN, m % TN);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          if (m == S::a_read(i)) a[i] = frag32f8<BM, AK>(nxt, wm0 + 32 * i, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (m == S::b_read(j)) bn[j] = frag32f8<BN, BKM>(nxt + A_BYTES, wn0 + 32 * j, lane);
#pragma unroll
        for (int d = 0; d < PER; ++d)
          if (m == S::dma_at(d)) {
            if (tail) {
              if (d < NA) da.issue_past_end(d, dst, wave);
              else db.issue_past_end(d - NA, dst + A_BYTES, wave);
            } else {
              if (d < NA) da.issue_one(d, dst, ns, K, wave);
              else db.issue_one(d - NA, dst + A_BYTES, ns, K, wave);
            }
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (odd) next_exps();
    };
    int kt = 0;
    for (; kt + 2 < nk; kt += 2) {
      slab(b0, b1, kt, false, false);
      slab(b1, b0, kt + 1, true, false);
    }
    if (kt + 1 < nk) {
      slab(b0, b1, kt, false, true);
      ++kt;
    }
    const bool odd = kt & 1;
#pragma unroll
    for (int m = 0; m < S::NM; ++m) mma(odd ? b1[m % TN] : b0[m % TN], a[m / TN], m / TN, m % TN);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));  // the trailing loads land before their place is used again
  }
  __syncthreads();
  store_rows<TM, TN, VEC>(acc, lds + wave * (WM * WN * 2), C + wm0 * g.ldc + wn0, g.ldc, c_rows - wm0, g.cols_out - n0 - wn0, lane);
}

template <int BM, int WGN, BlockProduct WHAT>
void launch(const BlockGemm& g, bool rebase, bool vec, unsigned grid, hipStream_t stream) {
  constexpr bool CAN = WHAT != kBlockForward;  // an operand read down its rows
  if (CAN && rebase) {
    if (vec)
      block_gemm<BM, WGN, WHAT, CAN, true><<<grid, 128 * WGN, 0, stream>>>(g);
    else
      block_gemm<BM, WGN, WHAT, CAN, false><<<grid, 128 * WGN, 0, stream>>>(g);
  } else if (vec) {
    block_gemm<BM, WGN, WHAT, false, true><<<grid, 128 * WGN, 0, stream>>>(g);
  } else {
    block_gemm<BM, WGN, WHAT, false, false><<<grid, 128 * WGN, 0, stream>>>(g);
  }
}

template <BlockProduct WHAT>
hipError_t launch_tiles(const BlockGemm& g, hipStream_t stream) {
  const bool ragged = g.rag.off != nullptr;
  const int64_t E = ragged ? g.rag.E : 1;
  const auto grid_of = [&](int64_t b) {
    const int64_t tn = (g.cols_out + b - 1) / b;
    if (WHAT == kBlockWeight) return E * ((g.rows_out + b - 1) / b) * tn;
    return (ragged ? ragged_units(g.rag.rows, E, b) : (g.rag.rows + b - 1) / b) * tn;
  };
  // bytes that an operand read down its rows spans
  const int64_t down = WHAT == kBlockForward ? 0 : WHAT == kBlockInput ? g.contraction * g.ldb : g.rag.rows * std::max(g.lda, g.ldb);
  const bool rebase = down >= (int64_t(1) << 31) - 1024;
  const bool vec = g.ldc % 8 == 0 && g.c_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(g.C) & 15) == 0;
  // the rows an expert's tiles are filled with, on average; see kBigTileMin for the tiles' sizes
  const bool full = WHAT == kBlockWeight || !ragged || g.rag.rows >= 192 * E;
  const bool big = grid_of(256) >= kBigTileMin && full;
  const int64_t n = grid_of(big ? 256 : 128);
  if (n == 0) return hipSuccess;
  if (big)
    launch<256, 4, WHAT>(g, rebase, vec, (unsigned)n, stream);
  else
    launch<128, 2, WHAT>(g, rebase, vec, (unsigned)n, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_gemm(BlockProduct what, const BlockGemm& g, hipStream_t stream) {
  switch (what) {
    case kBlockForward: return launch_tiles<kBlockForward>(g, stream);
    case kBlockInput: return launch_tiles<kBlockInput>(g, stream);
    default: return launch_tiles<kBlockWeight>(g, stream);
  }
}

}  // namespace i8mp
