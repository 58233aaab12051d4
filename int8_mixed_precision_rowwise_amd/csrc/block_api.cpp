// C ABI of the block-scaled FP8 linears and of the experts' routing (include/i8mp.h, last
// part).  Every argument is validated on the host before the first HIP call.
#include "block.h"
#include "checks.h"
#include "route.h"

#include <algorithm>
#include <initializer_list>

using namespace i8mp::checks;
using i8mp::kBlock;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 28, kMaxSide = int64_t(1) << 23, kMaxExperts = int64_t(1) << 16;

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Sizes whose launches have fewer than 2^32 work items and whose byte counts stay far from overflow.
bool block_dims_ok(int64_t M, int64_t N, int64_t K, int64_t E) {
  if (M < 0 || N < 0 || K < 0 || E < 0 || M >= kMaxRows || N >= kMaxSide || K >= kMaxSide || E >= kMaxExperts) return false;
  const int64_t e = std::max<int64_t>(E, 1);
  const int64_t sides = blocks_of(N) + blocks_of(K) + 2;
  const int64_t limit = int64_t(1) << 22;
  // tiles of rows by columns, tiles of weights, and the spread exponents
  return (M / kBlock + e + 1) * sides < limit && e * (blocks_of(N) + 1) * (blocks_of(K) + 1) < limit;
}

// Pitch of a row's exponents: whole words.
int64_t pitch4(int64_t K) { return (blocks_of(K) + 3) / 4 * 4; }

// Rows of the room in which each expert starts at a multiple of 16, and its blocks of 128.
int64_t room16(int64_t M, int64_t E) { return E ? 16 * i8mp::ragged_units(M, E, 16) : pad16(M); }
int64_t room128(int64_t M, int64_t E) { return E ? i8mp::ragged_units(M, E, kBlock) : blocks_of(M); }

i8mp::BlockPlan plan_fwd(int64_t M, int64_t N, int64_t K, int64_t E) { return i8mp::block_plan(i8mp::kBlockForward, M, N, K, E, M); }
i8mp::BlockPlan plan_dx(int64_t M, int64_t N, int64_t K, int64_t E) { return i8mp::block_plan(i8mp::kBlockInput, M, K, N, E, M); }
i8mp::BlockPlan plan_dw(int64_t M, int64_t N, int64_t K, int64_t E) { return i8mp::block_plan(i8mp::kBlockWeight, N, K, M, E, M); }

struct FwdWs {
  uint8_t *q, *s, *planes;
  float* sums;
};
size_t carve_fwd(void* ws, int64_t M, int64_t N, int64_t K, int64_t E, FwdWs* out) {
  Carver c{static_cast<char*>(ws)};
  FwdWs w{};
  w.q = static_cast<uint8_t*>(c.take((size_t)(room16(M, E) * pad16(K))));
  w.s = static_cast<uint8_t*>(c.take((size_t)(room16(M, E) * pitch4(K))));
  w.planes = static_cast<uint8_t*>(c.take((size_t)(std::max<int64_t>(E, 1) * blocks_of(K) * pad16(N))));
  w.sums = static_cast<float*>(c.take(plan_fwd(M, N, K, E).bytes(M)));
  if (out) *out = w;
  return c.used;
}

struct BwdWs {
  uint8_t *q, *s, *planes;        // dY along N, the weights' exponents
  uint8_t *qd, *sd, *qx, *sx;     // dY and X down the rows
  float* sums;                    // of one product after the other
};
size_t carve_bwd(void* ws, int64_t M, int64_t N, int64_t K, int64_t E, BwdWs* out) {
  Carver c{static_cast<char*>(ws)};
  BwdWs w{};
  w.q = static_cast<uint8_t*>(c.take((size_t)(room16(M, E) * pad16(N))));
  w.s = static_cast<uint8_t*>(c.take((size_t)(room16(M, E) * pitch4(N))));
  w.planes = static_cast<uint8_t*>(c.take((size_t)(std::max<int64_t>(E, 1) * blocks_of(N) * pad16(K))));
  w.qd = static_cast<uint8_t*>(c.take((size_t)(M * pad16(N))));
  w.sd = static_cast<uint8_t*>(c.take((size_t)(room128(M, E) * pad16(N))));
  w.qx = static_cast<uint8_t*>(c.take((size_t)(M * pad16(K))));
  w.sx = static_cast<uint8_t*>(c.take((size_t)(room128(M, E) * pad16(K))));
  w.sums = static_cast<float*>(c.take(std::max(plan_dx(M, N, K, E).bytes(M), plan_dw(M, N, K, E).bytes(N))));
  if (out) *out = w;
  return c.used;
}

struct BlockInputs {
  Range codes, exps, x, offsets, rows;
  bool reads(Range w) const {
    return overlap(w, codes) || overlap(w, exps) || overlap(w, x) || overlap(w, offsets) || overlap(w, rows);
  }
};

// need_w / need_x: whether the call reads the weights / X.
i8mp_status block_inputs(const i8mp_block* p, bool need_w, bool need_x, BlockInputs& in) {
  if (!p || !block_dims_ok(p->M, p->N, p->K, p->experts)) return I8MP_EINVAL;
  const int64_t M = p->M, N = p->N, K = p->K, E = std::max<int64_t>(p->experts, 1);
  if (p->experts > 0) {
    if (p->offset_bits != 32 && p->offset_bits != 64) return I8MP_EINVAL;
    if (!p->offsets || !aligned(p->offsets, (uintptr_t)p->offset_bits / 8)) return I8MP_EINVAL;
    in.offsets = vec_range(p->offsets, E + 1, p->offset_bits / 8);
  } else if (p->offsets) {
    return I8MP_EINVAL;
  }
  if (need_w && M > 0 && N > 0 && K > 0) {
    if (!p->codes || !p->exps || !aligned(p->codes, 16)) return I8MP_EINVAL;
    in.codes = vec_range(p->codes, E * N * pad16(K), 1);
    in.exps = vec_range(p->exps, E * blocks_of(N) * blocks_of(K), 1);
  }
  if (need_x && M > 0 && K > 0) {
    if (p->rows) {
      if (!aligned(p->rows, 4) || p->tokens < 1 || p->tokens >= kMaxRows) return I8MP_EINVAL;
      in.rows = vec_range(p->rows, M, 4);
    } else if (p->tokens != M) {
      return I8MP_EINVAL;
    }
    if (!chunked_ok(p->X, p->tokens, K, p->ldx, 2) || p->ldx > kMaxDim / std::max<int64_t>(p->tokens, 1)) return I8MP_EINVAL;
    in.x = mat_range(p->X, p->tokens, K, p->ldx, 2);
  }
  return I8MP_OK;
}

i8mp::Ragged ragged_of(const i8mp_block* p) {
  return {p->experts > 0 ? p->offsets : nullptr, p->offset_bits, std::max<int64_t>(p->experts, 1), p->M};
}

bool ws_ok(void* ws, size_t have, size_t need) { return need == 0 || (ws && aligned(ws, kAlign) && have >= need); }

int64_t dtype_bytes(int32_t dtype) { return dtype == I8MP_FP32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == I8MP_BF16 || dtype == I8MP_FP16 || dtype == I8MP_FP32; }

bool route_ok(const i8mp_route* p) {
  if (!p || !dtype_ok(p->dtype) || (p->score != I8MP_SOFTMAX && p->score != I8MP_SIGMOID)) return false;
  if (p->T < 0 || p->E < 1 || p->E > i8mp::kRouteMaxExperts || p->k < 1 || p->k > i8mp::kRouteMaxK || p->k > p->E) return false;
  if (p->T >= (int64_t(1) << 31) / p->k) return false;
  if (!elementwise_ok(p->logits, p->T, p->E, p->ld, dtype_bytes(p->dtype))) return false;
  return p->T == 0 || p->ld <= kMaxDim / p->T;
}

i8mp::RouteArgs route_args(const i8mp_route* p) {
  i8mp::RouteArgs a{};
  a.logits = p->logits, a.T = p->T, a.E = p->E, a.ld = p->ld;
  a.dtype = p->dtype, a.k = p->k, a.score = p->score, a.normalize = p->normalize != 0;
  return a;
}

bool none_overlap(std::initializer_list<Range> out, std::initializer_list<Range> in) {
  for (const Range* o = out.begin(); o != out.end(); ++o) {
    for (const Range& i : in)
      if (overlap(*o, i)) return false;
    for (const Range* other = out.begin(); other != o; ++other)
      if (overlap(*o, *other)) return false;
  }
  return true;
}

bool combine_ok(const i8mp_combine* p) {
  if (!p || !dtype_ok(p->dtype) || p->T < 0 || p->R < 0 || p->N < 0 || p->k < 1 || p->k > i8mp::kRouteMaxExperts) return false;
  if (p->T >= (int64_t(1) << 31) / p->k || p->R >= (int64_t(1) << 31) || p->N >= kMaxSide) return false;
  const int64_t elem = dtype_bytes(p->dtype);
  if (!elementwise_ok(p->Y, p->R, p->N, p->ldy, elem) || (p->R > 0 && p->ldy > kMaxDim / p->R)) return false;
  if (p->T > 0 && (!p->places || !aligned(p->places, 4) || !aligned(p->weights, 4))) return false;
  return true;
}

// Whether a matrix can be read and written 16 bytes at a time.
bool whole(const void* q, int64_t ld, int64_t elem) { return !q || (aligned(q, 16) && ld * elem % 16 == 0); }

i8mp::CombineArgs combine_args(const i8mp_combine* p) {
  i8mp::CombineArgs a{};
  a.T = p->T, a.R = p->R, a.N = p->N, a.k = p->k, a.dtype = p->dtype;
  a.Y = p->Y, a.ldy = p->ldy, a.places = p->places, a.weights = p->weights;
  return a;
}

}  // namespace

extern "C" {

i8mp_status i8mp_quantize_block_weight(const uint16_t* W, int64_t E, int64_t N, int64_t K, int64_t ldw, int64_t w_stride,
                                       uint8_t* codes, uint8_t* exps, void* stream) {
  if (E < 1 || !block_dims_ok(0, N, K, E)) return I8MP_EINVAL;
  if (!chunked_ok(W, N, K, ldw, 2) || w_stride < 0 || w_stride >= kMaxDim || ldw > kMaxDim / std::max<int64_t>(N, 1)) return I8MP_EINVAL;
  if (N == 0 || K == 0) return I8MP_OK;
  if (E > 1 && (w_stride % 8 != 0 || w_stride > kMaxDim / E)) return I8MP_EINVAL;
  if (!codes || !exps || !aligned(codes, 16)) return I8MP_EINVAL;
  Range in;
  in.b = reinterpret_cast<uintptr_t>(W);
  in.e = in.b + (uintptr_t)(2 * ((E - 1) * w_stride + (N - 1) * ldw + K));
  if (!none_overlap({vec_range(codes, E * N * pad16(K), 1), vec_range(exps, E * blocks_of(N) * blocks_of(K), 1)}, {in})) return I8MP_EINVAL;
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  return hip_status(i8mp::launch_block_quant_weight(W, E, N, K, ldw, w_stride, codes, exps, as_stream(stream)));
}

size_t i8mp_block_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t experts, int32_t backward) {
  if (!block_dims_ok(M, N, K, experts)) return 0;
  if (backward) return carve_bwd(nullptr, M, N, K, experts, nullptr);
  return i8mp::block_few_takes(M, experts, N, K) ? 0 : carve_fwd(nullptr, M, N, K, experts, nullptr);
}

i8mp_status i8mp_block_fwd(const i8mp_block* p, uint16_t* Y, int64_t ldy, int32_t clear, void* ws, size_t ws_bytes, void* stream) {
  BlockInputs in;
  const i8mp_status bad = block_inputs(p, true, true, in);
  if (bad != I8MP_OK) return bad;
  const int64_t M = p->M, N = p->N, K = p->K;
  if (!elementwise_ok(Y, M, N, ldy, 2) || (M > 0 && ldy > kMaxDim / M)) return I8MP_EINVAL;
  const Range ry = mat_range(Y, M, N, ldy, 2);
  if (in.reads(ry)) return I8MP_EINVAL;
  if (M == 0 || N == 0) return I8MP_OK;
  const size_t need = i8mp_block_workspace_bytes(M, N, K, p->experts, 0);
  if (!ws_ok(ws, ws_bytes, need)) return I8MP_EWORKSPACE;
  if (need) {
    const Range rw = vec_range(ws, (int64_t)need, 1);
    if (in.reads(rw) || overlap(rw, ry)) return I8MP_EINVAL;
  }
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  const hipStream_t s = as_stream(stream);
  const int64_t E = p->experts;
  const i8mp::Ragged rag = ragged_of(p);
  if (i8mp::block_few_takes(M, E, N, K)) {
    const i8mp::BlockFew f{p->X, p->ldx, p->tokens, p->rows, rag, N, K, p->codes, p->exps, Y, ldy, clear != 0};
    return hip_status(i8mp::launch_block_few(f, s));
  }
  FwdWs w;
  carve_fwd(ws, M, N, K, E, &w);
  // Where tokens are fewer than the rows that are read through an index, they are quantized once each, and the product
  // reads their codes through it (32768 rows of 8192 tokens of 2048: 12 us and the product's own time, 36 us for all
  // rows' codes).
  const bool gather = p->rows && p->tokens < M && p->tokens * pad16(K) < (int64_t(1) << 31) - 1024;
  const i8mp::Ragged tokens{nullptr, 0, 1, p->tokens};
  const i8mp::BlockQuant q{p->X, p->ldx, K, p->tokens, gather ? nullptr : p->rows, gather ? tokens : rag,
                           w.q, w.s, nullptr, nullptr, pad16(K), pitch4(K), 0};
  const i8mp::SpreadJob sp{p->exps, rag.E, blocks_of(N), blocks_of(K), pad16(N), 0, w.planes};
  const hipError_t e = i8mp::launch_block_quant(q, nullptr, sp, s);
  if (e != hipSuccess) return hip_status(e);
  i8mp::BlockGemm g{};
  g.rows_out = M, g.cols_out = N, g.contraction = K;
  g.A = w.q, g.sA = w.s, g.lda = pad16(K), g.ldsa = pitch4(K);
  g.index = gather ? p->rows : nullptr, g.n_src = p->tokens;
  g.B = p->codes, g.sB = w.planes, g.ldb = pad16(K), g.ldsb = pad16(N), g.b_stride = N * pad16(K), g.sb_stride = blocks_of(K) * pad16(N);
  g.C = Y, g.ldc = ldy, g.rag = rag, g.clear = clear != 0;
  return hip_status(i8mp::launch_block_gemm(i8mp::kBlockForward, g, plan_fwd(M, N, K, E), w.sums, s));
}

i8mp_status i8mp_block_bwd(const i8mp_block* p, const uint16_t* dY, int64_t lddy, uint16_t* dX, int64_t lddx, uint16_t* dW,
                           int64_t lddw, int32_t clear, void* ws, size_t ws_bytes, void* stream) {
  BlockInputs in;
  const i8mp_status bad = block_inputs(p, dX != nullptr, dW != nullptr, in);
  if (bad != I8MP_OK) return bad;
  const int64_t M = p->M, N = p->N, K = p->K, E = p->experts, Es = std::max<int64_t>(E, 1);
  if (!chunked_ok(dY, M, N, lddy, 2) || (M > 0 && lddy > kMaxDim / M)) return I8MP_EINVAL;
  if (dX && (!elementwise_ok(dX, M, K, lddx, 2) || (M > 0 && lddx > kMaxDim / M))) return I8MP_EINVAL;
  if (dW && (!elementwise_ok(dW, N, K, lddw, 2) || (N > 0 && lddw > kMaxDim / (Es * N)) || (E > 0 && lddw != K))) return I8MP_EINVAL;
  const Range rd = mat_range(dY, M, N, lddy, 2), rx = mat_range(dX, M, K, lddx, 2), rw = mat_range(dW, Es * N, K, lddw, 2);
  if (in.reads(rx) || in.reads(rw) || !none_overlap({rx, rw}, {rd})) return I8MP_EINVAL;
  const bool some_dx = dX && M > 0 && K > 0, some_dw = dW && N > 0 && K > 0;
  if (!some_dx && !some_dw) return I8MP_OK;
  const size_t need = i8mp_block_workspace_bytes(M, N, K, E, 1);
  if (!ws_ok(ws, ws_bytes, need)) return I8MP_EWORKSPACE;
  if (need) {
    const Range r = vec_range(ws, (int64_t)need, 1);
    if (in.reads(r) || !none_overlap({r}, {rx, rw, rd})) return I8MP_EINVAL;
  }
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  const hipStream_t s = as_stream(stream);
  const i8mp::Ragged rag = ragged_of(p);
  BwdWs w;
  carve_bwd(ws, M, N, K, E, &w);
  const int64_t np = pad16(N), kp = pad16(K);
  i8mp::BlockQuant d{dY, lddy, N, M, nullptr, rag, nullptr, nullptr, nullptr, nullptr, np, pitch4(N), np};
  const i8mp::BlockQuant x{p->X, p->ldx, K, p->tokens, p->rows, rag, nullptr, nullptr, w.qx, w.sx, kp, 0, kp};
  i8mp::SpreadJob sp{p->exps, rag.E, blocks_of(N), blocks_of(K), kp, 1, nullptr};
  if (some_dx) d.q_row = w.q, d.s_row = w.s, sp.planes = w.planes;
  if (some_dw) d.q_col = w.qd, d.s_col = w.sd;
  if (M > 0) {
    const hipError_t e = i8mp::launch_block_quant(d, some_dw ? &x : nullptr, sp, s);
    if (e != hipSuccess) return hip_status(e);
  }
  i8mp::BlockGemm gx{}, gw{};
  gx.cols_out = gw.cols_out = K, gx.rag = gw.rag = rag;
  gx.rows_out = M, gx.contraction = N;
  gx.A = w.q, gx.sA = w.s, gx.lda = np, gx.ldsa = pitch4(N);
  gx.B = p->codes, gx.sB = w.planes, gx.ldb = kp, gx.ldsb = kp, gx.b_stride = N * kp, gx.sb_stride = blocks_of(N) * kp;
  gx.C = dX, gx.ldc = lddx, gx.clear = clear != 0;
  gw.rows_out = N;
  gw.A = w.qd, gw.sA = w.sd, gw.lda = np, gw.ldsa = np;
  gw.B = w.qx, gw.sB = w.sx, gw.ldb = kp, gw.ldsb = kp;
  gw.C = dW, gw.ldc = lddw, gw.c_stride = N * lddw;
  const i8mp::BlockPlan px = plan_dx(M, N, K, E), pw = plan_dw(M, N, K, E);
  if (some_dx && some_dw) return hip_status(i8mp::launch_block_gemms(gx, px, gw, pw, w.sums, s));
  if (some_dx) return hip_status(i8mp::launch_block_gemm(i8mp::kBlockInput, gx, px, w.sums, s));
  return hip_status(i8mp::launch_block_gemm(i8mp::kBlockWeight, gw, pw, w.sums, s));
}

size_t i8mp_expert_route_workspace_bytes(int64_t T, int64_t E, int32_t k) {
  if (T < 0 || E < 1 || E > i8mp::kRouteMaxExperts) return 0;
  const int64_t per = i8mp::route_block_tokens(T, E, k);
  return T <= per ? 0 : up((size_t)((T + per - 1) / per * E * 4));
}

i8mp_status i8mp_expert_route(const i8mp_route* p, float* weights, int32_t* experts, int32_t* places, int32_t* rows,
                              int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
  if (!route_ok(p)) return I8MP_EINVAL;
  const int64_t n = p->T * p->k;
  if (!offsets || !aligned(offsets, 4)) return I8MP_EINVAL;
  for (const void* q : {(const void*)weights, (const void*)experts, (const void*)places, (const void*)rows})
    if (n > 0 && (!q || !aligned(q, 4))) return I8MP_EINVAL;
  const size_t need = i8mp_expert_route_workspace_bytes(p->T, p->E, p->k);
  if (!ws_ok(ws, ws_bytes, need)) return I8MP_EWORKSPACE;
  const Range rw = need ? vec_range(ws, (int64_t)need, 1) : Range{};
  if (!none_overlap({vec_range(weights, n, 4), vec_range(experts, n, 4), vec_range(places, n, 4), vec_range(rows, n, 4),
                     vec_range(offsets, p->E + 1, 4), rw},
                    {mat_range(p->logits, p->T, p->E, p->ld, dtype_bytes(p->dtype))}))
    return I8MP_EINVAL;
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  i8mp::RouteArgs a = route_args(p);
  a.weights = weights, a.experts = experts, a.places = places, a.rows = rows, a.offsets = offsets;
  a.hist = static_cast<int32_t*>(ws);
  return hip_status(i8mp::launch_route(a, as_stream(stream)));
}

i8mp_status i8mp_expert_route_bwd(const i8mp_route* p, const int32_t* experts, const float* dweights, void* dlogits, int64_t ld,
                                  void* stream) {
  if (!route_ok(p)) return I8MP_EINVAL;
  const int64_t n = p->T * p->k, elem = dtype_bytes(p->dtype);
  if (n > 0 && (!experts || !dweights || !aligned(experts, 4) || !aligned(dweights, 4))) return I8MP_EINVAL;
  if (!elementwise_ok(dlogits, p->T, p->E, ld, elem) || (p->T > 0 && ld > kMaxDim / p->T)) return I8MP_EINVAL;
  if (!none_overlap({mat_range(dlogits, p->T, p->E, ld, elem)},
                    {mat_range(p->logits, p->T, p->E, p->ld, elem), vec_range(experts, n, 4), vec_range(dweights, n, 4)}))
    return I8MP_EINVAL;
  if (p->T == 0) return I8MP_OK;
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  return hip_status(i8mp::launch_route_bwd(route_args(p), experts, dweights, dlogits, ld, as_stream(stream)));
}

i8mp_status i8mp_expert_combine(const i8mp_combine* p, const void* residual, int64_t ldr, void* out, int64_t ldo, void* stream) {
  if (!combine_ok(p)) return I8MP_EINVAL;
  const int64_t T = p->T, N = p->N, elem = dtype_bytes(p->dtype), n = T * p->k;
  if (!elementwise_ok(out, T, N, ldo, elem) || (T > 0 && ldo > kMaxDim / T)) return I8MP_EINVAL;
  if (residual && (!elementwise_ok(residual, T, N, ldr, elem) || (T > 0 && ldr > kMaxDim / T))) return I8MP_EINVAL;
  const Range ro = mat_range(out, T, N, ldo, elem), rr = mat_range(residual, T, N, ldr, elem);
  if (!none_overlap({ro}, {mat_range(p->Y, p->R, N, p->ldy, elem), vec_range(p->places, n, 4), vec_range(p->weights, n, 4)})) return I8MP_EINVAL;
  // the residual may be the output itself
  if (overlap(ro, rr) && !(residual == out && ldr == ldo)) return I8MP_EINVAL;
  if (T == 0 || N == 0) return I8MP_OK;
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  i8mp::CombineArgs a = combine_args(p);
  a.residual = residual, a.ldr = ldr, a.out = out, a.ldo = ldo;
  a.vec = N * elem % 16 == 0 && whole(p->Y, p->ldy, elem) && whole(residual, ldr, elem) && whole(out, ldo, elem);
  return hip_status(i8mp::launch_combine(a, as_stream(stream)));
}

i8mp_status i8mp_expert_combine_bwd(const i8mp_combine* p, const void* dout, int64_t ldd, const int32_t* rows, void* dY,
                                    int64_t ldg, float* dweights, void* stream) {
  if (!combine_ok(p)) return I8MP_EINVAL;
  const int64_t T = p->T, R = p->R, N = p->N, elem = dtype_bytes(p->dtype), n = T * p->k;
  if (!elementwise_ok(dout, T, N, ldd, elem) || (T > 0 && ldd > kMaxDim / T)) return I8MP_EINVAL;
  if (dY && (!elementwise_ok(dY, R, N, ldg, elem) || (R > 0 && ldg > kMaxDim / R))) return I8MP_EINVAL;
  if (!aligned(dweights, 4) || !aligned(rows, 4)) return I8MP_EINVAL;
  if (!none_overlap({mat_range(dY, R, N, ldg, elem), vec_range(dweights, n, 4)},
                    {mat_range(p->Y, R, N, p->ldy, elem), mat_range(dout, T, N, ldd, elem), vec_range(p->places, n, 4),
                     vec_range(p->weights, n, 4), vec_range(rows, R, 4)}))
    return I8MP_EINVAL;
  if ((T == 0 && (!rows || R == 0)) || (!dY && !dweights)) return I8MP_OK;
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  i8mp::CombineArgs a = combine_args(p);
  a.dout = dout, a.ldd = ldd, a.rows = rows, a.dY = dY, a.ldg = ldg, a.dweights = dweights;
  a.vec = N * elem % 16 == 0 && whole(p->Y, p->ldy, elem) && whole(dout, ldd, elem) && whole(dY, ldg, elem);
  return hip_status(i8mp::launch_combine_bwd(a, as_stream(stream)));
}

}  // extern "C"
