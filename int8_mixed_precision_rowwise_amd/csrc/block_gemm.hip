// Products of block-scaled FP8 codes, for one matrix or for the ragged rows of many experts.
//
// The pipeline is the FP8 GEMM's (gemm_pipelined.h): slabs of 64 of the contraction go from
// memory straight into LDS, four deep, and feed v_mfma_scale_f32_32x32x64_f8f6f4.  That
// instruction multiplies each lane's 32 contraction values by a power of two of its own, so the
// blocks' scales cost no vector operation: a lane needs the exponent's byte of its row (or
// column) of each 128, which comes into LDS the same way as the codes, four blocks at a time.
//
// 8192 x 5632 x 2048 takes 90 us (2.1 PFLOP/s), 8192^3 415 to 465 (2.35 to 2.65; the library's row-wise FP8
// product 2.74).  Of the 90, 64 are 96 slabs (three rounds of tiles, the last three quarters full) of 0.67 us each, whose
// matrix instructions are 1024 cycles of each SIMD: 0.61 us at the 1.69 GHz that the card holds under this load (0.45 measured
// on zeros, at a higher clock).  They are busy 0.59 of the kernel's time.  A tile's end takes 5: its stores, and the next
// slabs' loads that queue behind them.  The kernel's start and end take 9.
//
// The big tiles' kernels take all 256 registers, half of them accumulators, and where a tile is opened or closed a few more
// vector and some tens of scalar ones, which go to memory and to lanes there (vector and scalar: forward 5 and 68, through an
// index 9 and 90, dX 17 and 79, dW 3 and 34); a tile's loop over its blocks has none of that.
#include "block.h"
#include "gemm_pipelined.h"

namespace i8mp {
namespace {

// The tiles of the experts' rows: tiles of BM rows, expert after expert.  Every wave adds up the
// experts' tiles by itself, 64 experts at a time.  Sums stop at the number that offsets which do not fall can make:
// others of many experts would take them past 32 bits, and tiles to rows that nobody has.
template <int BM>
__device__ __forceinline__ int most_tiles(const Ragged& r) {
  return (int)(r.rows / BM + r.E);
}
template <int BM>
__device__ __forceinline__ int ragged_tiles(const Ragged& r) {
  if (!r.off) return (int)((r.rows + BM - 1) / BM);
  const int most = most_tiles<BM>(r);
  int n = 0;
  for (int64_t e = threadIdx.x & 63; e < r.E; e += 64) n = min(n + (lane_rows(r, e).count + BM - 1) / BM, most);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n = min(n + __shfl_xor(n, o), most);
  return __builtin_amdgcn_readfirstlane(n);  // what loops over it then stays in scalar registers
}

// Where row tile tm lies.
template <int BM>
__device__ __forceinline__ void ragged_place(const Ragged& r, int tm, Place& p) {
  p.e = 0, p.first = 0, p.count = r.off ? 0 : r.rows, p.local = (int64_t)tm * BM;
  if (!r.off) return;
  const int lane = threadIdx.x & 63;
  const int most = most_tiles<BM>(r);
  int before = 0;  // tiles of the experts before this turn's 64
  for (int64_t e0 = 0; e0 < r.E; e0 += 64) {
    const LaneRows l = lane_rows(r, e0 + lane);
    int n = (l.count + BM - 1) / BM;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(n, o);
      if (lane >= o) n = min(n + up, most);
    }
    const uint64_t past = __ballot(before + n > tm);
    if (past) {  // always, in the end: tm is one of the experts' tiles
      const int at = __builtin_ctzll(past);
      const int start = at ? before + __shfl(n, at - 1) : before;
      if constexpr (BM == 128) {
        take_lane(l, e0, at, p);
      } else {  // registers are scarcer than time there (32768 rows of 32 experts through an index 93 us, 90 so)
        p.e = e0 + at;
        p.first = offset_at(r, p.e);
        p.count = max((int64_t)0, offset_at(r, p.e + 1) - p.first);
      }
      p.local = (int64_t)(tm - start) * BM;
      return;
    }
    before = min(before + __shfl(n, 63), most);
  }
}

// The i-th expert in falling order of rows (up to 64 experts; more: the i-th): the products that
// contract over an expert's rows start with the longest.
__device__ __forceinline__ void by_size(const Ragged& r, int64_t i, Place& p) {
  p.e = 0, p.first = 0, p.count = r.rows;
  if (!r.off) return;
  const int lane = threadIdx.x & 63;
  if (r.E > 64) return take_lane(lane_rows(r, i), i, 0, p);
  const LaneRows l = lane_rows(r, lane);
  int rank = 0;
  for (int k = 0; k < (int)r.E; ++k) {
    const int other = __builtin_amdgcn_readlane(l.count, k);
    rank += other > l.count || (other == l.count && k < lane);
  }
  take_lane(l, 0, __builtin_ctzll(__ballot(lane < r.E && rank == (int)i)), p);
}

// Consecutive workgroups go to the 8 XCDs in turn.  Runs of kRun tiles go to one XCD, so that they share
// panels in its L2; the XCDs take the runs in turn, so that experts of different sizes load them alike.
// (With an eighth of all tiles to each, the dW of 16384 rows of 8 experts took 346 us, and 222 so.)
constexpr uint32_t kRun = 32;
__device__ __forceinline__ uint32_t xcd_runs(uint32_t wg, uint32_t n) {
  const uint32_t whole = n / (8 * kRun) * (8 * kRun);
  if (wg < whole) {
    const uint32_t x = wg & 7, i = wg >> 3;
    return (i / kRun * 8 + x) * kRun + i % kRun;
  }
  // the rest: each XCD a run of what is left
  const uint32_t m = n - whole, k = wg - whole, x = k & 7;
  return whole + x * (m >> 3) + min(x, m & 7) + (k >> 3);
}

// Tiles of 256 x 256, one to a CU at a time; a last round with at most a quarter of the CUs' number is
// cut into quarter tiles, which together fill the CUs once (a quarter takes 0.42 to 0.47 of a whole one's
// time).
constexpr uint32_t kCUs = 256;
__host__ __device__ inline uint32_t whole_tiles(uint32_t n) { return n % kCUs <= kCUs / 4 ? n - n % kCUs : n; }

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

template <int BM>
constexpr int kLdsBytes = BM == 256 ? 4 * 512 * BK + 10240 : 4 * 256 * BK + 2048;  // of a workgroup of 8 waves, of 4

// Slab loads of one operand, as Dma (gemm_pipelined.h) with less state in registers: a lane's chunks of a
// slab's loads lie a fixed step apart.  Rows or columns past the operand are not looked at: a K-major operand's
// lie past the descriptor's end and arrive as zeros, the others' are the next row's bytes or zeros, and
// either only reach outputs that are not stored.
// GATHER (K-major): rows from anywhere in the operand, each at an offset of its own.
template <int R, bool KMAJOR, int NW, bool REBASE, bool GATHER = false>
struct Slabs {
  static constexpr int kInst = R * BK / 1024 / NW;
  static constexpr int CPR = R / 16, KR = 64 / CPR;               // [k][n] tiles: chunks a row, rows a load
  static_assert(KMAJOR || kInst == 1 || (NW * KR) % 32 == 0, "the swizzle repeats from load to load");
  v4u rsrc;
  uint32_t off[GATHER ? kInst : 1], at;  // this lane's chunk in slab 0; its contraction index within a slab
  uint32_t ld;
  const int8_t* base;
  int64_t bytes;

  __device__ __forceinline__ void init(const int8_t* p, int64_t ld_, int64_t mn0, int64_t MN, int64_t K, int wave, int lane) {
    ld = (uint32_t)ld_;
    if constexpr (KMAJOR) {
      base = p + mn0 * ld_;
      bytes = min((int64_t)R, MN - mn0) * ld_;
      const int c = (lane & 3) ^ ((lane >> 4) & 3);
      at = 16 * c;
      off[0] = (16 * wave + (lane >> 2)) * ld + at;
    } else {
      base = p + mn0;
      bytes = (K - 1) * ld_ + min((int64_t)R, MN - mn0);
      const int k = wave * KR + lane / CPR, c = (lane % CPR) ^ mnmajor_swz(R, k);
      at = k;
      off[0] = k * ld + 16 * c;
    }
    rsrc = Dma<64, true, NW>::make_rsrc(base, max((int64_t)0, min(bytes, (int64_t)kOob)));  // an empty contraction: nothing
  }
  // Row `row` of the tile for load j of this lane, and where it is: one outside [0, n) is a row of zeros.
  static __device__ __forceinline__ int row_of(int j, int wave, int lane) { return 16 * (wave + NW * j) + (lane >> 2); }
  __device__ __forceinline__ void init_rows(const int8_t* p, int64_t ld_, int64_t n, int lane) {
    ld = (uint32_t)ld_;
    base = p, bytes = n * ld_;
    at = 16 * ((lane & 3) ^ ((lane >> 4) & 3));
    rsrc = Dma<64, true, NW>::make_rsrc(base, bytes);
  }
  __device__ __forceinline__ void set_row(int j, int64_t src, int64_t n) {
    off[j] = src >= 0 && src < n ? (uint32_t)src * ld + at : kOob;
  }

  // Into byte `to` of LDS and the 1023 behind it.
  static __device__ __forceinline__ void load(uint32_t o, const v4u& r, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"((uint32_t)__builtin_amdgcn_readfirstlane(to)), "v"(o), "s"(r)
                 : "memory", "m0");
  }
  // Load j of the slab at contraction index k0, `ahead` = k0 (k0 ld in tiles read down their rows) bytes on, of
  // which `left` = K - k0 contraction indices are the operand's, into the operand's tile at byte `to` of LDS.
  __device__ __forceinline__ void issue_at(int j, uint32_t to, int k0, uint32_t ahead, int left, int wave) const {
    const int limit = min(left, BK) - (KMAJOR ? 0 : NW * KR * j);
    if constexpr (!GATHER) ahead += j * ((KMAJOR ? 16 * NW : NW * KR) * ld);
    v4u r = rsrc;
    if constexpr (REBASE && !KMAJOR) {
      const int64_t sh = (int64_t)k0 * ld;
      r = Dma<64, true, NW>::make_rsrc(base + sh, max((int64_t)0, min(bytes - sh, (int64_t)kOob)));
      ahead -= (uint32_t)sh;
    }
    // what is the same in all lanes is added up in scalar registers
    uint32_t o = off[GATHER ? j : 0] + (uint32_t)__builtin_amdgcn_readfirstlane(ahead);
    load((int)at < limit ? o : kOob, r, to + (wave + NW * j) * 1024);
  }
  __device__ __forceinline__ void issue_one(int j, uint32_t to, int slab, int K, int wave) const {
    const int k0 = BK * slab;
    issue_at(j, to, k0, (uint32_t)k0 * (KMAJOR ? 1u : ld), K - k0, wave);
  }
  __device__ __forceinline__ void issue(uint32_t to, int slab, int K, int wave) const {
#pragma unroll
    for (int j = 0; j < kInst; ++j) issue_one(j, to, slab, K, wave);
  }
  // For a slab past the contraction, so that it counts in the waits: zeros into a buffer nobody reads.
  __device__ __forceinline__ void issue_past_end(int j, uint32_t to, int wave) const { load(kOob, rsrc, to + (wave + NW * j) * 1024); }
};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_void*)const_cast<void*>(p)));
}

// Exponents of four blocks of one tile: A's 4 BM bytes, row after row (ROWS) or block after block, and B's 4 BN
// behind them, block after block; 256 bytes a load.
template <int BM, int BN, int NW, bool ROWS>
struct Exponents {
  static constexpr int kLoads = (BM + BN) / 64, kMine = (kLoads + NW - 1) / NW;  // of the workgroup, of a wave at most
  const uint8_t *a, *b;          // at the tile's first row and column
  int64_t lda, ldb, enda, endb;  // pitches, bytes to the end of the exponents
  uint32_t row[kMine];           // ROWS: this lane's row of A
  // a0, b0: the tile's first row and column; arows: ROWS: rows of A from there on
  __device__ __forceinline__ void init(const uint8_t* sa, int64_t la, const uint8_t* sb, int64_t lb, int64_t a0, int64_t b0,
                                       int64_t blocks, int64_t arows, int wave, int lane) {
    a = sa + (ROWS ? a0 * la : a0), b = sb + b0, lda = la, ldb = lb;
    enda = ROWS ? arows * la : blocks * la - a0, endb = blocks * lb - b0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) row[i] = (uint32_t)((64 * (wave + NW * i) + lane) * la);
  }
  // Row r of the tile for load i of this lane, if the load is one of A's.
  static __device__ __forceinline__ int row_of(int i, int wave, int lane) { return 64 * (wave + NW * i) + lane; }
  __device__ __forceinline__ void issue(int8_t* buf, int64_t group, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int load = wave + NW * i;
      if (load >= kLoads) break;
      const bool is_b = load >= BM / 64;
      const int R = is_b ? BN : BM, k = (is_b ? load - BM / 64 : load) * (256 / R) + lane / (R / 4);
      const int64_t ld = is_b ? ldb : lda, skip = 4 * group * (ROWS && !is_b ? 1 : ld), left = (is_b ? endb : enda) - skip;
      const v4u r = Dma<64, true, NW>::make_rsrc(reinterpret_cast<const int8_t*>((is_b ? b : a) + skip),
                                                 max((int64_t)0, min(left, (int64_t)kOob)));
      const uint32_t o = ROWS && !is_b ? row[i] : (uint32_t)(k * ld + 4 * (lane % (R / 4)));
      const uint32_t l = (uint32_t)__builtin_amdgcn_readfirstlane(
          (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)(buf + load * 256)));
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                   :
                   : "s"(l), "v"(o), "s"(r)
                   : "memory", "m0");
    }
  }
};

// The sums themselves, into a plane of partial sums (rows `ld` apart, a multiple of 4).
template <int TM, int TN>
__device__ __forceinline__ void store_sums(const v16f (&acc)[TM][TN], float* __restrict__ C, int64_t ld, int64_t rows, int64_t cols,
                                           int lane) {
  const int mr = lane & 31, nq = 4 * (lane >> 5);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (32 * i + mr >= rows) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = 32 * j + 8 * q + nq;  // columns up to the next multiple of 4 are the plane's
        if (n < cols)
          *reinterpret_cast<float4*>(C + (32 * i + mr) * ld + n) =
              make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
      }
  }
}

// What a tile reads and writes: rows p.local on of the expert (WEIGHT: columns p.local on of A), columns n0 on.
struct Operands {
  const int8_t *A, *B;
  const uint8_t *sA, *sB;
  int64_t K, m0, a_rows;  // contraction, first of A's rows (columns) and the end of them
  uint16_t* C;            // the tile's first output
  int64_t c_rows;         // rows of C from there on
};
template <BlockProduct WHAT>
__device__ __forceinline__ Operands operands(const BlockGemm& g, const Place& p, int64_t n0) {
  Operands o{reinterpret_cast<const int8_t*>(g.A), reinterpret_cast<const int8_t*>(g.B), g.sA, g.sB, g.contraction, 0, 0, g.C + n0, 0};
  if constexpr (WHAT == kBlockWeight) {
    o.K = p.count;
    o.A += p.first * g.lda, o.B += p.first * g.ldb;
    o.sA += unit_of<kBlock>(p) * g.ldsa, o.sB += unit_of<kBlock>(p) * g.ldsb;
    o.m0 = p.local, o.a_rows = g.lda;
    o.c_rows = g.rows_out - p.local;
    o.C += p.e * g.c_stride + p.local * g.ldc;
  } else {
    o.m0 = 16 * unit_of<16>(p) + p.local;
    o.c_rows = p.count - p.local;
    o.a_rows = o.m0 + o.c_rows;
    o.B += p.e * g.b_stride, o.sB += p.e * g.sb_stride;
    o.C += (p.first + p.local) * g.ldc;
  }
  return o;
}

// One tile: rows p.local on of the expert (WEIGHT: columns p.local on of A), columns n0 on; part `split` of the
// contraction.
template <int BM, int BN, int WR, int WGN, int STAGES, BlockProduct WHAT, bool REBASE, bool VEC, bool GATHER>
__device__ __forceinline__ void multiply(const BlockGemm& g, const Place& p, int64_t n0, uint32_t split, int8_t* lds) {
  constexpr int NW = WR * WGN;
  constexpr int WM = BM / WR, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  constexpr bool AK = WHAT != kBlockWeight, BKM = WHAT == kBlockForward;
  constexpr int A_BYTES = BM * BK, SLAB = A_BYTES + BN * BK;
  constexpr int EXPS = 4 * (BM + BN);  // bytes of four blocks' exponents
  typedef Slabs<BM, AK, NW, REBASE, GATHER> DA;
  typedef Slabs<BN, BKM, NW, REBASE> DB;
  constexpr int NA = DA::kInst, PER = NA + DB::kInst;
  using S = SlabSchedule<TM, TN, PER>;
  static_assert(NW * WM * WN * 2 <= STAGES * SLAB, "the outputs fit where the slabs were");
  static_assert(STAGES * SLAB + 2 * EXPS <= kLdsBytes<NW == 8 ? 256 : 128>, "room in LDS");
  int8_t* const exps = lds + STAGES * SLAB;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);

  Operands o(operands<WHAT>(g, p, n0));
  int64_t K = o.K;
  const int8_t *A = o.A, *B = o.B;
  const uint8_t *sA = o.sA, *sB = o.sB;
  const int64_t m0 = o.m0, a_rows = o.a_rows, c_rows = o.c_rows;
  uint16_t* const C = o.C;
  constexpr bool CAN_SPLIT = NW == 4;
  if (CAN_SPLIT && g.splits > 1) {  // one matrix
    const int64_t k0 = split * g.kchunk;
    K = min(g.kchunk, K - k0);
    A += AK ? k0 : k0 * g.lda;
    B += BKM ? k0 : k0 * g.ldb;
    sA += AK ? k0 / kBlock : k0 / kBlock * g.ldsa, sB += k0 / kBlock * g.ldsb;
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
    db.init(B, g.ldb, n0, BKM ? g.cols_out : g.ldb, K, wave, lane);
    Exponents<BM, BN, NW, AK> ex;
    if constexpr (GATHER) {
      da.init_rows(A, g.lda, g.n_src, lane);
      ex.init(sA, g.ldsa, sB, g.ldsb, 0, n0, blocks, g.n_src, wave, lane);
      const int32_t* index = g.index + p.first + p.local;
      const int last = (int)min(c_rows, (int64_t)BM) - 1;  // rows past it repeat it: their outputs are not stored
#pragma unroll
      for (int j = 0; j < NA; ++j) da.set_row(j, index[min(DA::row_of(j, wave, lane), last)], g.n_src);
#pragma unroll
      for (int i = 0; i < decltype(ex)::kMine; ++i) {
        const int64_t src = index[min(decltype(ex)::row_of(i, wave, lane), last)];
        ex.row[i] = src >= 0 && src < g.n_src ? (uint32_t)(src * g.ldsa) : kOob;
      }
    } else {
      da.init(A, g.lda, m0, a_rows, K, wave, lane);
      ex.init(sA, g.ldsa, sB, g.ldsb, m0, n0, blocks, a_rows - m0, wave, lane);
    }

    v8i a[TM], b0[TN], b1[TN];
    int ea[TM], eb[TN], na[TM], nb[TN];  // exponents of this block and the next
    const auto read_exps = [&](int block) __attribute__((always_inline)) {
      const int8_t* at = exps + ((block >> 2) & 1) * EXPS + (lane & 31);
#pragma unroll
      for (int i = 0; i < TM; ++i)
        na[i] = AK ? *reinterpret_cast<const uint8_t*>(exps + ((block >> 2) & 1) * EXPS + 4 * (wm0 + 32 * i + (lane & 31)) + (block & 3))
                   : *reinterpret_cast<const uint8_t*>(at + (block & 3) * BM + wm0 + 32 * i);
#pragma unroll
      for (int j = 0; j < TN; ++j) nb[j] = *reinterpret_cast<const uint8_t*>(at + 4 * BM + (block & 3) * BN + wn0 + 32 * j);
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
    const uint32_t lds0 = lds_address(lds);
    const int k = (int)K;
    ex.issue(exps, 0, wave, lane);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      da.issue(lds0 + s * SLAB, s, k, wave);
      db.issue(lds0 + s * SLAB + A_BYTES, s, k, wave);
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
    // reads the next block's exponents.  A slab's first instructions, up to the barrier, end the turn of the loop before
    // it: there nothing of LDS is under way, which the compiler would otherwise wait for at the loop's head.
    int stage = 0;  // slab kt's place
    const auto first_half = [&](v8i(&bc)[TN]) __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < S::HA; ++m) {
        mma(bc[m % TN], a[m / TN], m / TN, m % TN);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((STAGES - 2) * PER));  // slab kt + 1 has landed
      lds_barrier();
    };
    const auto second_half = [&](v8i(&bc)[TN], v8i(&bn)[TN], int kt, bool odd, bool tail) __attribute__((always_inline)) {
      const uint32_t dst = lds0 + stage * SLAB;
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      const int8_t* nxt = lds + stage * SLAB;
      const int ns = kt + STAGES;
      if (odd) read_exps((kt + 1) >> 1);
      if (!tail && (ns & 7) == 0 && ns < nk) ex.issue(exps + ((ns >> 3) & 1) * EXPS, ns >> 3, wave, lane);
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
              if (d < NA) da.issue_one(d, dst, ns, k, wave);
              else db.issue_one(d - NA, dst + A_BYTES, ns, k, wave);
            }
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (odd) next_exps();
    };
    int kt = 0;
    first_half(b0);
    for (; kt + 2 < nk; kt += 2) {
      second_half(b0, b1, kt, false, false);
      first_half(b1);
      second_half(b1, b0, kt + 1, true, false);
      first_half(b0);
    }
    if (kt + 1 < nk) {
      second_half(b0, b1, kt, false, true);
#pragma unroll
      for (int m = 0; m < S::NM; ++m) mma(b1[m % TN], a[m / TN], m / TN, m % TN);
    } else {
#pragma unroll
      for (int m = S::HA; m < S::NM; ++m) mma(b0[m % TN], a[m / TN], m / TN, m % TN);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));  // the trailing loads land before their place is used again
  }
  if (CAN_SPLIT && g.splits > 1) {
    const int64_t row = p.local + wm0, col = n0 + wn0;
    store_sums<TM, TN>(acc, g.planes + split * g.plane + row * g.plane_ld + col, g.plane_ld, c_rows - wm0, g.cols_out - col, lane);
    return;
  }
  __syncthreads();
  store_rows<TM, TN, VEC>(acc, lds + wave * (WM * WN * 2), C + wm0 * g.ldc + wn0, g.ldc, c_rows - wm0, g.cols_out - n0 - wn0, lane);
}

// What two lanes exchange in a transposition: b of the first and a of the second.
template <int QUAD_PERM>
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b, bool second) {
  const uint32_t t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(second ? a : b), QUAD_PERM, 0xF, 0xF, false);
  a = second ? t : a;
  b = second ? b : t;
}

// A wave's 128 x 64 outputs straight from its accumulators.  A lane has four adjacent columns of a row here and there, and
// the one 32 lanes on the next four; exchanging halves makes 32 columns in a row of one lane, four pieces of 16 bytes, and
// transposing these among four adjacent lanes puts 64 bytes of one row into them: a store takes a row's piece from four
// lanes at a time, or 16 bytes where they have different rows.  (8192 x 5632 x 2048 89.6 us, 92.6 with 16 bytes of a row each;
// 8192 x 8192 x 1024 with X's quantization 82 and 93, the backward of 32768 rows of 32 experts 278 and 292.)  What lies
// outside the tile falls outside the descriptor.
__device__ __forceinline__ void store_direct(const v16f (&acc)[4][2], uint16_t* C, uint32_t ldc, int rows, int cols, int lane) {
  const int mr = lane & 31, half = lane >> 5;
  rows = min(max(rows, 0), 128), cols = min(max(cols, 0), 64);
  const int bytes = __builtin_amdgcn_readfirstlane(rows > 0 && cols > 0 ? (int)(2 * ((rows - 1) * ldc + cols)) : 0);
  const uint64_t c = reinterpret_cast<uint64_t>(C);
  const uint64_t c0 = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(c >> 32)) << 32 |
                      (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)c);
  const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(c0), 0, bytes, 0x00020000);
  const int s = lane & 3;
  const bool odd = s & 1, high = s & 2;
  const uint32_t col = 32 * half + 8 * s;
  uint32_t at = (int)col < cols ? 2 * (4 * (mr >> 2) * ldc + col) : kOob;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v[4][4];  // chunk q of 8 columns of this lane's row and half
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        __bf16 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (__bf16)acc[i][j][4 * q + e];  // round to nearest even
        const uint2 u = __builtin_bit_cast(uint2, h);
        w[j][0] = u.x, w[j][1] = u.y;
      }
      const auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
      const auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
      v[q][0] = s0[0], v[q][1] = s1[0], v[q][2] = s0[1], v[q][3] = s1[1];
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      exchange<0xB1>(v[0][d], v[1][d], odd), exchange<0xB1>(v[2][d], v[3][d], odd);
      exchange<0x4E>(v[0][d], v[2][d], high), exchange<0x4E>(v[1][d], v[3][d], high);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const v4u c = {v[t][0], v[t][1], v[t][2], v[t][3]};
      __builtin_amdgcn_raw_buffer_store_b128(c, out, at == kOob ? kOob : at + 2 * t * ldc, 0, 0);
    }
    at = at == kOob ? kOob : at + 64 * ldc;  // rows past the last one lie past the descriptor's end
  }
}

constexpr int kBatch = 32;  // tiles whose places are worked out at a time

struct BigLds {
  int8_t slabs[4 * 512 * BK];
  int8_t exps[5][4 * 512];  // four groups, and one that nobody reads
  int info[kBatch][8];
  int index[2][256];  // of this tile's rows and the next one's
};

// Tiles info[0 .. n - 1] of 256 x 256, one after another without a pause: the pipeline's slab loads run on into
// the next tile while the last slabs of this one are multiplied, and its outputs leave while the next one's first
// slabs arrive.  A tile's contraction is taken in whole blocks of 128, two slabs, and at least two of them; the loads
// are two blocks ahead, so that they change to the next tile before the last two blocks, and the loop over a
// tile's blocks has no branch in it (one would let the compiler move matrix instructions past the loads and reads that they
// are to cover).
template <BlockProduct WHAT, bool REBASE, bool GATHER>
__device__ __forceinline__ void multiply_all(const BlockGemm& g, int n, BigLds& lds) {
  constexpr int BM = 256, BN = 256, WGN = 4, NW = 8, WM = 128, WN = 64, TM = 4, TN = 2;
  constexpr bool AK = WHAT != kBlockWeight, BKM = WHAT == kBlockForward;
  constexpr int A_BYTES = BM * BK, SLAB = A_BYTES + BN * BK;
  typedef Slabs<BM, AK, NW, REBASE, GATHER> DA;
  typedef Slabs<BN, BKM, NW, REBASE> DB;
  constexpr int NA = DA::kInst, PER = NA + DB::kInst;
  using S = SlabSchedule<TM, TN, PER>;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm0 = (wave / WGN) * WM, wn0 = (wave % WGN) * WN;
  const uint32_t slabs0 = lds_address(lds.slabs), exps0 = lds_address(lds.exps);

  const auto place = [&](int i, int64_t& n0) __attribute__((always_inline)) {
    const int* q = lds.info[i];
    Place p;
    p.e = __builtin_amdgcn_readfirstlane(q[0]);
    p.local = __builtin_amdgcn_readfirstlane(q[1]);
    p.first = __builtin_amdgcn_readfirstlane(q[2]);
    p.count = __builtin_amdgcn_readfirstlane(q[3]);
    n0 = __builtin_amdgcn_readfirstlane(q[4]);
    return p;
  };

  // What is being loaded: the slab at contraction index lk of a tile of K = lk + left, with the operands' bytes that
  // lie before it.
  DA da;
  DB db;
  int lk = 0, left = 0;
  uint32_t ahead_a = 0, ahead_b = 0;
  // Exponents of a group of four blocks: waves 0 .. 3 load A's, the others B's, of one block each; every block
  // counts one load, those that start no group one of zeros into a place of its own.
  const uint8_t* ex = nullptr;
  int64_t ex_left = 0;
  const bool ex_rows = AK && wave < 4;  // of 64 rows, four blocks each; otherwise of one block
  const uint32_t ex_ld = (uint32_t)(wave < 4 ? g.ldsa : g.ldsb), ex_step = ex_rows ? 4 : 4 * ex_ld;
  uint32_t ex_at = ex_rows ? (64 * wave + lane) * ex_ld : (wave & 3) * ex_ld + 4 * lane;
  int lgroup = 0;  // groups loaded so far
  // GATHER: the index of a tile's rows comes into LDS while the tile before it is multiplied (waves 0 .. 3, 64
  // rows each); at least four slabs are loaded and waited for before it is looked at.
  const auto fetch_index = [&](int i) __attribute__((always_inline)) {
    if constexpr (GATHER) {
      if (i >= n || wave >= 4) return;
      int64_t n0;
      const Place p = place(i, n0);
      const int64_t from = p.first + p.local;
      const v4u r = Dma<64, true, NW>::make_rsrc(reinterpret_cast<const int8_t*>(g.index + from), min((g.rag.rows - from) * 4, (int64_t)1024));
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                   :
                   : "s"(lds_address(lds.index[i & 1]) + wave * 256), "v"(256 * wave + 4 * lane), "s"(r)
                   : "memory", "m0");
    }
  };
  const auto open = [&](int i) __attribute__((always_inline)) {
    lk = 0, ahead_a = 0, ahead_b = 0;
    if (i < n) {
      int64_t n0;
      const Place p = place(i, n0);
      const Operands o = operands<WHAT>(g, p, n0);
      left = (int)o.K;
      db.init(o.B, g.ldb, n0, BKM ? g.cols_out : g.ldb, o.K, wave, lane);
      const int64_t planes = (o.K + kBlock - 1) / kBlock * ex_ld;
      if (wave >= 4) ex = o.sB + n0, ex_left = planes - n0;
      else if (!AK) ex = o.sA + o.m0, ex_left = planes - o.m0;
      if constexpr (GATHER) {
        da.init_rows(o.A, g.lda, g.n_src, lane);
        const int* index = lds.index[i & 1];
#pragma unroll
        for (int j = 0; j < NA; ++j) da.set_row(j, index[DA::row_of(j, wave, lane)], g.n_src);
        if (wave < 4) {
          const int src = index[64 * wave + lane];
          ex = o.sA, ex_left = g.n_src * g.ldsa;
          ex_at = src >= 0 && src < g.n_src ? (uint32_t)src * ex_ld : kOob;
        }
        fetch_index(i + 1);
      } else {
        da.init(o.A, g.lda, o.m0, o.a_rows, o.K, wave, lane);
        if (ex_rows) ex = o.sA + o.m0 * g.ldsa, ex_left = (o.a_rows - o.m0) * g.ldsa;
      }
    } else {
      left = 0, ex_left = 0;  // nothing but zeros
    }
  };
  const auto issue_exps = [&]() __attribute__((always_inline)) {  // before a block's slabs
    const bool starts = (lk & (4 * kBlock - 1)) == 0;
    const v4u r = Dma<64, true, NW>::make_rsrc(reinterpret_cast<const int8_t*>(ex), max((int64_t)0, min(ex_left, (int64_t)kOob)));
    const uint32_t to = exps0 + (starts ? lgroup & 3 : 4) * (uint32_t)sizeof(lds.exps[0]) + wave * 256;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"((uint32_t)__builtin_amdgcn_readfirstlane(to)), "v"(starts ? ex_at : kOob), "s"(r)
                 : "memory", "m0");
    ex += starts ? ex_step : 0;
    ex_left -= starts ? ex_step : 0;
    lgroup += starts;
  };
  const auto issue = [&](int d, uint32_t dst) __attribute__((always_inline)) {
    if (d < NA) da.issue_at(d, dst, lk, ahead_a, left, wave);
    else db.issue_at(d - NA, dst + A_BYTES, lk, ahead_b, left, wave);
  };
  const auto issued = [&]() __attribute__((always_inline)) {
    lk += BK, left -= BK;
    ahead_a += BK * (AK ? 1u : da.ld), ahead_b += BK * (BKM ? 1u : db.ld);
  };

  v16f acc[TM][TN];
  const auto clear_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = Mma<1>::zero();
  };
  v8i a[TM], b0[TN], b1[TN];
  int ea[TM], eb[TN], na[TM], nb[TN];  // exponents of this block and the next
  int rgroup = 0, rblock = 0;          // where they are read: group, block of it
  const auto read_exps = [&]() __attribute__((always_inline)) {
    const int8_t* at = lds.exps[rgroup & 3] + (lane & 31);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      na[i] = AK ? *reinterpret_cast<const uint8_t*>(lds.exps[rgroup & 3] + 4 * (wm0 + 32 * i + (lane & 31)) + rblock)
                 : *reinterpret_cast<const uint8_t*>(at + rblock * BM + wm0 + 32 * i);
#pragma unroll
    for (int j = 0; j < TN; ++j) nb[j] = *reinterpret_cast<const uint8_t*>(at + 4 * BM + rblock * BN + wn0 + 32 * j);
  };
  const auto next_exps = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i) ea[i] = na[i];
#pragma unroll
    for (int j = 0; j < TN; ++j) eb[j] = nb[j];
  };
  const auto mma = [&](const v8i& bf, const v8i& af, int i, int j) __attribute__((always_inline)) {
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf, af, acc[i][j], 0, 0, 0, eb[j], 0, ea[i]);
  };

  if constexpr (GATHER) {
    fetch_index(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    lds_barrier();
  }
  open(0);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if ((s & 1) == 0) issue_exps();
#pragma unroll
    for (int d = 0; d < PER; ++d) issue(d, slabs0 + s * SLAB);
    issued();
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 * PER));  // slab 0 has landed (and exponents a load for every block ahead of it)
  lds_barrier();
  read_exps();
  next_exps();
  clear_acc();
#pragma unroll
  for (int i = 0; i < TM; ++i) a[i] = frag32f8<BM, AK>(lds.slabs, wm0 + 32 * i, lane);
#pragma unroll
  for (int j = 0; j < TN; ++j) b0[j] = frag32f8<BN, BKM>(lds.slabs + A_BYTES, wn0 + 32 * j, lane);

  int stage = 0;  // this slab's place
  // One slab, both halves of multiply's; half: of the block.  The waits count slab loads and are at most stricter for the
  // exponents' loads and the last tile's stores among them.  (Waits that let a tile's stores go on for three more slabs, and
  // a loop head that waits for less of the last turn's reads, made no difference.)
  auto slab = [&](v8i(&bc)[TN], v8i(&bn)[TN], int half) __attribute__((always_inline)) {
    const uint32_t dst = slabs0 + stage * SLAB;
    stage = (stage + 1) & 3;
    const int8_t* nxt = lds.slabs + stage * SLAB;
#pragma unroll
    for (int m = 0; m < S::HA; ++m) {
      mma(bc[m % TN], a[m / TN], m / TN, m % TN);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * PER));  // the next slab has landed
    lds_barrier();
    if (half) read_exps();
    else issue_exps();
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
        if (m == S::dma_at(d)) issue(d, dst);
      __builtin_amdgcn_sched_barrier(0);
    }
    issued();
  };
#pragma unroll 1
  for (int ct = 0; ct < n; ++ct) {
    const int K = WHAT == kBlockWeight ? __builtin_amdgcn_readfirstlane(lds.info[ct][3]) : (int)g.contraction;
    const int blocks = max((K + kBlock - 1) / kBlock, 2);
    int b = 0;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      const int end = part ? blocks : blocks - 2;
      if (part) open(ct + 1);
#pragma unroll 1
      for (; b < end; ++b) {
        slab(b0, b1, 0);
        // the exponents of the next block: the next group's first after the group's fourth and after the tile's last
        const bool last = b + 1 == blocks || rblock == 3;
        rgroup += last;
        rblock = last ? 0 : rblock + 1;
        slab(b1, b0, 1);
        next_exps();
      }
    }
    int64_t n0;
    const Place p = place(ct, n0);
    const Operands o = operands<WHAT>(g, p, n0);
    store_direct(acc, o.C + wm0 * g.ldc + wn0, (uint32_t)g.ldc, (int)min(o.c_rows - wm0, (int64_t)WM), (int)min(g.cols_out - n0 - wn0, (int64_t)WN), lane);
    clear_acc();
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));  // the trailing loads land before their place is used again
  __syncthreads();
}

// The parts' sums added in order, rounded once.
__global__ __launch_bounds__(256) void add_planes(BlockGemm g, int64_t rows) {
  const uint32_t quads = (uint32_t)(g.plane_ld / 4);
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x, r = i / quads, n = (i - r * quads) * 4;
  if (r >= rows) return;
  const float* at = g.planes + r * g.plane_ld + n;
  float4 s = *reinterpret_cast<const float4*>(at);
  for (int64_t k = 1; k < g.splits; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(at + k * g.plane);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  __bf16* c = reinterpret_cast<__bf16*>(g.C) + r * g.ldc + n;
  const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < g.cols_out) c[e] = (__bf16)v[e];  // round to nearest even
}

// Where a tile lies, in groups of 4 tile rows (of an expert's tile rows), so that the tiles of an XCD share panels
// in its L2.  tiles_m: of all experts' rows (WEIGHT: of one expert's outputs).
template <int BM, BlockProduct WHAT>
__device__ __forceinline__ Place tile_place(const BlockGemm& g, uint32_t tile, uint32_t tiles_m, uint32_t tiles_n, int64_t& n0) {
  uint32_t e = 0;
  if constexpr (WHAT == kBlockWeight) {
    e = tile / (tiles_m * tiles_n);
    tile -= e * tiles_m * tiles_n;
  }
  const uint32_t group = tile / (4 * tiles_n), first = 4 * group, rows = min(tiles_m - first, 4u), in = tile - group * 4 * tiles_n;
  const uint32_t tm = first + in % rows, tn = in / rows;
  n0 = (int64_t)tn * BM;
  Place p;
  if constexpr (WHAT == kBlockWeight) {
    by_size(g.rag, e, p);
    p.local = (int64_t)tm * BM;
  } else {
    ragged_place<BM>(g.rag, tm, p);
  }
  return p;
}

template <int BM, BlockProduct WHAT>
__device__ __forceinline__ uint32_t tile_rows(const BlockGemm& g) {
  return WHAT == kBlockWeight ? (uint32_t)((g.rows_out + BM - 1) / BM) : ragged_tiles<BM>(g.rag);
}

// By workgroup wg of n.
template <BlockProduct WHAT>
__device__ __forceinline__ void clear_rows(const BlockGemm& g, uint32_t wg, uint32_t n) {
  if (WHAT == kBlockWeight || !g.clear) return;
  const OtherRows other = other_rows(g.rag);
  for (int64_t i = wg; i < other.count; i += n)
    for (int64_t c = threadIdx.x; c < g.cols_out; c += blockDim.x) g.C[other.row(i) * g.ldc + c] = 0;
}

// Tiles of 128 x 128, two workgroups a CU; this is workgroup wg of n.
template <BlockProduct WHAT, bool REBASE, bool VEC, bool GATHER>
__device__ __forceinline__ void small_tile(const BlockGemm& g, uint32_t wg, uint32_t n, int8_t* lds) {
  const uint32_t tiles_n = (uint32_t)((g.cols_out + 127) / 128), tiles_m = tile_rows<128, WHAT>(g);
  clear_rows<WHAT>(g, wg, n);
  const uint32_t each = tiles_m * tiles_n, all = each * (WHAT == kBlockWeight ? (uint32_t)g.rag.E : 1) * g.splits;
  if (wg >= all) return;
  uint32_t tile = xcd_runs(wg, all);
  // the parts of the contraction one after another: an XCD's run of tiles reads the same part
  const uint32_t split = g.splits > 1 ? tile / each : 0;
  int64_t n0;
  const Place p = tile_place<128, WHAT>(g, tile - split * each, tiles_m, tiles_n, n0);
  multiply<128, 128, 2, 2, 4, WHAT, REBASE, VEC, GATHER>(g, p, n0, split, lds);
}

template <BlockProduct WHAT, bool REBASE, bool VEC, bool GATHER>
__global__ __launch_bounds__(256, 2) void block_gemm_small(BlockGemm g) {
  __shared__ __attribute__((aligned(1024))) int8_t lds[kLdsBytes<128>];
  small_tile<WHAT, REBASE, VEC, GATHER>(g, blockIdx.x, gridDim.x, lds);
}

// Both products of a backward at once: nx workgroups (a multiple of 8, so that the XCDs' runs stay theirs) for dX, the
// rest for dW.
__global__ __launch_bounds__(256, 2) void block_gemm_both(BlockGemm dx, BlockGemm dw, uint32_t nx) {
  __shared__ __attribute__((aligned(1024))) int8_t lds[kLdsBytes<128>];
  if (blockIdx.x < nx)
    small_tile<kBlockInput, false, true, false>(dx, blockIdx.x, nx, lds);
  else
    small_tile<kBlockWeight, false, true, false>(dw, blockIdx.x - nx, gridDim.x - nx, lds);
}

// Tiles of 256 x 256: a workgroup for each CU takes every 256th of them, then at most one quarter of the last ones.
template <BlockProduct WHAT, bool REBASE, bool GATHER>
__global__ __launch_bounds__(512, 2) void block_gemm_big(BlockGemm g) {
  __shared__ __attribute__((aligned(1024))) BigLds lds;
  const uint32_t tiles_n = (uint32_t)((g.cols_out + 255) / 256), tiles_m = tile_rows<256, WHAT>(g);
  clear_rows<WHAT>(g, blockIdx.x, gridDim.x);
  const uint32_t all = tiles_m * tiles_n * (WHAT == kBlockWeight ? (uint32_t)g.rag.E : 1), whole = whole_tiles(all);
  const uint32_t wg = blockIdx.x, step = gridDim.x;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (uint32_t first = wg; first < whole; first += kBatch * step) {
    const int n = (int)min((whole - first + step - 1) / step, (uint32_t)kBatch);
    for (int i = wave; i < n; i += 8) {
      int64_t n0;
      const Place p = tile_place<256, WHAT>(g, xcd_runs(first + i * step, whole), tiles_m, tiles_n, n0);
      if (lane == 0) {
        int* q = lds.info[i];
        q[0] = (int)p.e, q[1] = (int)p.local, q[2] = (int)p.first, q[3] = (int)p.count, q[4] = (int)n0;
      }
    }
    __syncthreads();
    multiply_all<WHAT, REBASE, GATHER>(g, n, lds);
  }
  // the quarters of a tile to one XCD
  for (uint32_t i = wg; i < (all - whole + 7) / 8 * 32; i += step) {
    const uint32_t tile = whole + i / 32 * 8 + (i & 7), quarter = i / 8 & 3;
    if (tile >= all) continue;
    int64_t n0;
    Place p = tile_place<256, WHAT>(g, tile, tiles_m, tiles_n, n0);
    p.local += quarter & 1 ? 128 : 0;
    n0 += quarter & 2 ? 128 : 0;
    if (p.local >= (WHAT == kBlockWeight ? g.rows_out : p.count) || n0 >= g.cols_out) continue;
    multiply<128, 128, 2, 4, 8, WHAT, REBASE, true, GATHER>(g, p, n0, 0, lds.slabs);
    __syncthreads();  // the outputs have left LDS
  }
}

template <BlockProduct WHAT, bool REBASE, bool GATHER>
void launch(const BlockGemm& g, bool big, bool vec, unsigned grid, hipStream_t stream) {
  if (big)
    block_gemm_big<WHAT, REBASE, GATHER><<<grid, 512, 0, stream>>>(g);
  else if (vec)
    block_gemm_small<WHAT, REBASE, true, GATHER><<<grid, 256, 0, stream>>>(g);
  else
    block_gemm_small<WHAT, REBASE, false, GATHER><<<grid, 256, 0, stream>>>(g);
}

// At most: how many the experts' rows make, only the GPU knows.
int64_t tiles_of(BlockProduct what, int64_t rows, int64_t cols, int64_t E, bool ragged, int64_t b) {
  const int64_t tn = (cols + b - 1) / b;
  if (what == kBlockWeight) return E * ((rows + b - 1) / b) * tn;
  return (ragged ? ragged_units(rows, E, b) : (rows + b - 1) / b) * tn;
}

// An operand read down its rows that spans more bytes than a descriptor's offsets reach.
bool needs_rebase(BlockProduct what, const BlockGemm& g) {
  const int64_t down = what == kBlockForward ? 0 : what == kBlockInput ? g.contraction * g.ldb : g.rag.rows * std::max(g.lda, g.ldb);
  return down >= (int64_t(1) << 31) - 1024;
}
// Whole chunks of 8 columns can be written.
bool whole_chunks(const BlockGemm& g) {
  return g.ldc % 8 == 0 && g.c_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(g.C) & 15) == 0;
}
// The big tiles' kernel writes nothing else, and reads 256 rows of codes at offsets that stay below kOob, which stands
// for "nothing": the last chunk of rows 2^23 apart (contractions from 2^23 - 15 on) would be taken for it.
bool takes_big(const BlockGemm& g, const BlockPlan& plan) {
  return plan.big && whole_chunks(g) && g.cols_out % 8 == 0 && g.ldc < (int64_t(1) << 22) && 256 * std::max(g.lda, g.ldb) <= kOob;
}

template <BlockProduct WHAT>
hipError_t launch_tiles(const BlockGemm& g, const BlockPlan& plan, hipStream_t stream) {
  const bool ragged = g.rag.off != nullptr, rebase = needs_rebase(WHAT, g), vec = whole_chunks(g), big = takes_big(g, plan);
  const int64_t n = tiles_of(WHAT, g.rows_out, g.cols_out, ragged ? g.rag.E : 1, ragged, big ? 256 : 128) * plan.splits;
  if (n == 0) return hipSuccess;
  const bool cut = n > whole_tiles((uint32_t)n) || (ragged && WHAT != kBlockWeight);
  const unsigned grid = (unsigned)(big ? cut ? kCUs : std::min<int64_t>(n, kCUs) : n);
  if (WHAT != kBlockForward && rebase)
    launch<WHAT, WHAT != kBlockForward, false>(g, big, vec, grid, stream);
  else if (WHAT == kBlockForward && g.index)
    launch<WHAT, false, WHAT == kBlockForward>(g, big, vec, grid, stream);
  else
    launch<WHAT, false, false>(g, big, vec, grid, stream);
  return hipGetLastError();
}

BlockGemm with_plan(const BlockGemm& gemm, const BlockPlan& plan, float* planes) {
  BlockGemm g = gemm;
  g.splits = (uint32_t)plan.splits, g.kchunk = plan.kchunk;
  g.planes = planes, g.plane_ld = plan.plane_ld, g.plane = g.rows_out * plan.plane_ld;
  return g;
}

hipError_t join_parts(const BlockGemm& g, hipStream_t stream) {
  const int64_t quads = g.rows_out * (g.plane_ld / 4);
  if (g.splits == 1 || quads == 0) return hipSuccess;
  add_planes<<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(g, g.rows_out);
  return hipGetLastError();
}

}  // namespace

// Tiles of 256 x 256, or of 128 x 128, which start and end sooner, of which two share a CU, and by which a backward's
// two products go out together.  The bigger where they are more than half the CUs' number, the experts' rows fill
// them, and their number squared times the contraction reaches kBigWork.  Time of the small ones over that of the big: 128
// tiles 0.69 to 0.92 over contractions of 64 to 4096; 160 tiles 0.95 over 1024, 1.02 over 2048, 1.17 over 4096; 256
// tiles 0.91 over 512, 1.02 over 1024, 1.1 over 2048; 320 tiles 0.88 over 512, 1.00 over 1024; 512 tiles 0.9 over 128,
// 1.09 over 512; dW of 1024 tiles 1.2 over 64.
constexpr double kBigWork = 256.0 * 256.0 * 1024.0;

// One matrix with few tiles and a long contraction splits it, each part of at least
// 512 into a plane of fp32 sums that a second launch adds up.  Both sides, all the call's kernels: 64 rows against
// 4096 x 14336 65 us and 31, 128 rows 73 and 35, 64 against 4096 x 4096 25.5 and 20.0; dW of 32768 rows of 512 x 2048
// 152 us and 55, of 8192 of 256 x 2048 40 and 18.  With two parts only it does not pay (64 rows against 14336 x
// 4096 26.8 and 29.6), nor do parts over tiles of 256 x 256, whose planes are four times as many (the dW of
// 32768 rows of 512 x 2048 in 16 parts 54 us, of 4096 of 2048 x 2048 in 4 parts 43 us and 25 unsplit).
BlockPlan block_plan(BlockProduct what, int64_t rows, int64_t cols, int64_t contraction, int64_t E, int64_t all_rows) {
  BlockPlan p{false, 1, 0, 0};
  const bool ragged = E > 0;
  const int64_t e = std::max<int64_t>(E, 1), small = tiles_of(what, rows, cols, e, ragged, 128);
  const int64_t big = tiles_of(what, rows, cols, e, ragged, 256), depth = what == kBlockWeight ? all_rows / e : contraction;
  p.big = big > kCUs / 2 && (double)big * (double)big * (double)depth >= kBigWork && (what == kBlockWeight || !ragged || all_rows >= 192 * e);
  if (ragged || p.big || small == 0) return p;
  const int64_t s = std::min<int64_t>(kCUs / small, contraction / 512);
  if (s < 3) return p;
  p.kchunk = ((contraction + s - 1) / s + 4 * kBlock - 1) / (4 * kBlock) * (4 * kBlock);  // whole groups of exponents
  p.splits = (contraction + p.kchunk - 1) / p.kchunk;
  p.plane_ld = (cols + 3) / 4 * 4;
  return p;
}

hipError_t launch_block_gemm(BlockProduct what, const BlockGemm& gemm, const BlockPlan& plan, float* planes, hipStream_t stream) {
  const BlockGemm g = with_plan(gemm, plan, planes);
  const hipError_t e = what == kBlockForward ? launch_tiles<kBlockForward>(g, plan, stream)
                       : what == kBlockInput ? launch_tiles<kBlockInput>(g, plan, stream)
                                             : launch_tiles<kBlockWeight>(g, plan, stream);
  return e != hipSuccess ? e : join_parts(g, stream);
}

// In one launch where both take tiles of 128 x 128 and at most one has its contraction in parts (they share the
// planes).  The whole backward of 300 rows of 2048 x 2048 in 24.4 us, 29.2 with a launch each; of 1000 of 1000 x 1000
// 19.3 and 27.9; of 2048 of 4096 x 1024 39 and 49.
hipError_t launch_block_gemms(const BlockGemm& dx, const BlockPlan& px, const BlockGemm& dw, const BlockPlan& pw, float* planes,
                              hipStream_t stream) {
  const BlockGemm x = with_plan(dx, px, planes), w = with_plan(dw, pw, planes);
  const bool ragged = x.rag.off != nullptr;
  const int64_t e = ragged ? x.rag.E : 1;
  const int64_t nx = tiles_of(kBlockInput, x.rows_out, x.cols_out, e, ragged, 128) * px.splits;
  const int64_t nw = tiles_of(kBlockWeight, w.rows_out, w.cols_out, e, ragged, 128) * pw.splits;
  if (nx == 0 || nw == 0 || takes_big(x, px) || takes_big(w, pw) || !whole_chunks(x) || !whole_chunks(w) || (px.splits > 1 && pw.splits > 1) ||
      needs_rebase(kBlockInput, x) || needs_rebase(kBlockWeight, w)) {
    const hipError_t first = launch_block_gemm(kBlockInput, dx, px, planes, stream);
    return first != hipSuccess ? first : launch_block_gemm(kBlockWeight, dw, pw, planes, stream);
  }
  const int64_t nx8 = (nx + 7) / 8 * 8;
  block_gemm_both<<<(unsigned)(nx8 + nw), 256, 0, stream>>>(x, w, (uint32_t)nx8);
  hipError_t st = hipGetLastError();
  if (st == hipSuccess) st = join_parts(x, stream);
  return st != hipSuccess ? st : join_parts(w, stream);
}

}  // namespace i8mp
