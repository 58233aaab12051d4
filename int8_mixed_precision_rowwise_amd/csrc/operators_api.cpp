// C ABI of the operators around the linears (include/i8mp.h, last part).
// Every argument is validated on the host before the first HIP call, so a
// rejected call launches nothing and writes nothing.
#include "checks.h"
#include "internal.h"

#include <algorithm>
#include <cmath>
#include <utility>

using namespace i8mp::checks;

namespace i8mp {

// Workgroups of at least this many over (segment, row) fill the chip twice.
constexpr int64_t kDistillFill = 1024;
constexpr int64_t kDistillSegMin = 512, kDistillSegMax = 4096;  // chunks of 16 bytes

static void distill_segments(int64_t T, int64_t chunks, int* segs, int* seg_chunks) {
  const int64_t want = (kDistillFill + T - 1) / T;
  int64_t per = (chunks + want - 1) / want;
  per = std::min(std::max((per + 1) / 2 * 2, kDistillSegMin), kDistillSegMax);  // even
  *segs = (int)((chunks + per - 1) / per);
  *seg_chunks = (int)per;
}

// 16-byte chunks that a row of V elements can touch at any alignment.
static int64_t distill_chunks(int64_t V, int elem) { return (V * elem + 15 + elem - 1) / 16 + 1; }

// A row in one workgroup's registers is read once; segments read it twice but
// spread few rows over the chip.  Both sides, loss and gradient of bf16 rows (a row a
// workgroup takes nearly the same time up to 256 rows): 32000 classes 10 us, in
// segments 13 for one row; 64000 classes 15 us, in segments 13 for 16 rows and 17
// for 32; 128256 classes 22 us, in segments 16 for 16 rows and 26 for 32.
static int distill_shape(int64_t T, int64_t V, int k, int elem) {
  const int64_t chunks = distill_chunks(V, elem);
  if (chunks > 16384 || (T < 24 && chunks > 4096)) return kSegments;
  // the least room that holds the row, with two kept entries a thread
  static const struct { int plan, threads, chunks; } kPlans[] = {
      {kRows64x2, 64, 2}, {kRows64x4, 64, 4}, {kRows64x8, 64, 8}, {kRows256x4, 256, 4}, {kRows256x8, 256, 8},
      {kRows512x8, 512, 8}, {kRows512x12, 512, 12}, {kRows512x16, 512, 16}, {kRows512x24, 512, 24}, {kRows512x32, 512, 32}};
  for (const auto& p : kPlans)
    if (chunks <= p.threads * p.chunks && k <= 2 * p.threads) return p.plan;
  return kSegments;
}

void distill_plan(DistillArgs& a, int elem) {
  a.plan = a.given ? kSegments : distill_shape(a.T, a.V, a.k, elem);
  distill_segments(a.T, distill_chunks(a.V, elem), &a.segs, &a.seg_chunks);
}

size_t distill_workspace_bytes(int64_t T, int64_t V, int k, int elem) {
  if (distill_shape(T, V, k, elem) != kSegments) return 0;
  int segs, per;
  distill_segments(T, distill_chunks(V, elem), &segs, &per);
  return (size_t)T * (size_t)segs * 16;
}

}  // namespace i8mp

namespace {

int64_t dtype_bytes(int32_t dtype) { return dtype == I8MP_FP32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == I8MP_BF16 || dtype == I8MP_FP16 || dtype == I8MP_FP32; }

// Heads [B][S][H][D] at p with the strides of the first three dimensions.
struct HeadsView {
  uintptr_t p = 0;
  int64_t b = 0, s = 0, h = 0, H = 0;
};

// Elements from the first to one past the last, over n values of a stride each.
int64_t heads_extent(const HeadsView& v, int64_t B, int64_t S, int64_t D) {
  return (B - 1) * v.b + (S - 1) * v.s + (v.H - 1) * v.h + D;
}

Range heads_range(const HeadsView& v, int64_t B, int64_t S, int64_t D, int64_t elem) {
  Range r;
  if (v.H == 0 || B == 0 || S == 0) return r;
  r.b = v.p;
  r.e = v.p + (uintptr_t)(heads_extent(v, B, S, D) * elem);
  return r;
}

// Whether no two elements of a view share their place: with the dimensions in
// the order of their strides, each stride spans all that lies within it.
bool heads_distinct(const HeadsView& v, int64_t B, int64_t S, int64_t D) {
  struct Dim { int64_t stride, n; } d[3] = {{v.b, B}, {v.s, S}, {v.h, v.H}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& c) { return a.stride < c.stride; });
  int64_t span = D;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    if (x.stride < span) return false;
    span += (x.n - 1) * x.stride;
  }
  return true;
}

// Whether two views share no element: disjoint byte ranges, or views with the same
// batch and token strides (of dimensions of one, any) whose heads lie in separate
// parts of a token, or are rows of one larger view that shares none.
bool heads_disjoint(const HeadsView& a, const HeadsView& c, int64_t B, int64_t S, int64_t D, int64_t elem) {
  if (!overlap(heads_range(a, B, S, D, elem), heads_range(c, B, S, D, elem))) return true;
  if ((S > 1 && a.s != c.s) || (B > 1 && a.b != c.b)) return false;
  const HeadsView& lo = a.p <= c.p ? a : c;
  const HeadsView& hi = a.p <= c.p ? c : a;
  if ((hi.p - lo.p) % (uintptr_t)elem) return false;
  const int64_t off = (int64_t)((hi.p - lo.p) / (uintptr_t)elem);
  // heads lo.H, lo.H + 1, ... of the larger view, `first` of them before hi's (heads before tokens in memory)
  const int64_t h = lo.H > 1 ? lo.h : hi.H > 1 ? hi.h : off;
  if (h > 0 && off % h == 0 && (hi.H == 1 || hi.h == h)) {
    const int64_t first = off / h;
    if (first >= lo.H && heads_distinct({lo.p, lo.b, lo.s, h, first + hi.H}, B, S, D)) return true;
  }
  int64_t period = S > 1 ? a.s : a.b;  // from one token to the next
  if (S > 1 && B > 1) {
    const bool s_inner = a.s <= a.b;
    period = s_inner ? a.s : a.b;
    if (s_inner ? a.b < S * a.s : a.s < B * a.b) return false;
  }
  const int64_t lo_ext = (lo.H - 1) * lo.h + D, hi_ext = (hi.H - 1) * hi.h + D;
  return off >= lo_ext && (B * S == 1 || off + hi_ext <= period);
}

bool act_ok(int32_t act) { return act >= I8MP_ACT_NONE && act <= I8MP_ACT_SILU; }
uint64_t pass_offset(uint64_t offset, int j) { return offset + ((uint64_t)j << 40); }
bool opts_ok(const i8mp_linear_opts* o) { return o && (o->round == I8MP_RNE || o->round == I8MP_SR); }
// Sizes whose buffers' byte counts stay far from overflow, and whose columns (16 work
// items each in the few-token kernel, 8 in the backward's join) fit a launch of fewer than 2^32.
bool linear_dims_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kArea = int64_t(1) << 50, kMaxColumns = int64_t(1) << 28;
  const int64_t m = M + 16, n = N + 16, k = K + 16;
  return dims_ok(M, N, K) && N < kMaxColumns && m <= kArea / n && m <= kArea / k && n <= kArea / k;
}

// The contraction a GEMM runs over: padded to whole 16-byte chunks.
int64_t padded_k(int64_t K) { return K > 0 ? pad16(K) : 16; }

struct ActFwdWs {
  int8_t *qx, *qw;
  float *sx, *sw;
  void *part_x, *part_w, *split;
};
size_t carve_act_fwd(void* ws, int64_t M, int64_t N, int64_t K, bool weights, ActFwdWs* out) {
  Carver c{static_cast<char*>(ws)};
  const int64_t kp = padded_k(K);
  ActFwdWs w{};
  w.qx = static_cast<int8_t*>(c.take((size_t)(M * kp)));
  w.sx = static_cast<float*>(c.take((size_t)M * 4));
  if (weights) {
    w.qw = static_cast<int8_t*>(c.take((size_t)(N * kp)));
    w.sw = static_cast<float*>(c.take((size_t)N * 4));
    w.part_x = c.take(i8mp::rowwise_colmax_workspace_bytes(M, K));
    w.part_w = c.take(i8mp::rowwise_colmax_workspace_bytes(N, K));
  }
  const size_t split = i8mp::gemm_split_workspace_bytes(I8MP_NT, M, N, kp, kp, kp);
  w.split = split ? c.take(split) : nullptr;
  if (out) *out = w;
  return c.used;
}

struct ActBwdWs {
  uint16_t* dz;
  int8_t *q_row, *q_col, *qw, *qx;
  float *s_row, *s_col, *sw, *sx, *band_sum;
  uint16_t *segmax, *band_max, *col_max;
  void *col, *split;
};
size_t carve_act_bwd(void* ws, int64_t M, int64_t N, int64_t K, ActBwdWs* out) {
  Carver c{static_cast<char*>(ws)};
  i8mp::ActBwdArgs a{};
  a.M = M, a.N = N;
  i8mp::act_bwd_plan(a);
  const int64_t kp = pad16(K);
  ActBwdWs w{};
  w.dz = static_cast<uint16_t*>(c.take((size_t)(M * a.np) * 2));
  w.q_row = static_cast<int8_t*>(c.take((size_t)(M * a.np)));
  w.q_col = static_cast<int8_t*>(c.take((size_t)(a.mp * a.np)));
  w.qw = static_cast<int8_t*>(c.take((size_t)(a.np * kp)));
  w.qx = static_cast<int8_t*>(c.take((size_t)(a.mp * kp)));
  w.s_row = static_cast<float*>(c.take((size_t)M * 4));
  w.s_col = static_cast<float*>(c.take((size_t)N * 4));
  w.sw = static_cast<float*>(c.take((size_t)K * 4));
  w.sx = static_cast<float*>(c.take((size_t)K * 4));
  w.segmax = static_cast<uint16_t*>(c.take(i8mp::act_bwd_segmax_bytes(a)));
  w.band_max = static_cast<uint16_t*>(c.take(i8mp::act_bwd_band_elems(a) * 2));
  w.band_sum = static_cast<float*>(c.take(i8mp::act_bwd_band_elems(a) * 4));
  w.col_max = static_cast<uint16_t*>(c.take(i8mp::act_bwd_columns(a) * 2));
  w.col = c.take(std::max(i8mp::colwise_workspace_bytes(N, K), i8mp::colwise_workspace_bytes(M, K)));
  const size_t split = std::max(i8mp::gemm_split_workspace_bytes(I8MP_NN, M, K, a.np, a.np, kp),
                                i8mp::gemm_split_workspace_bytes(I8MP_TN, N, K, a.mp, a.np, kp));
  w.split = split ? c.take(split) : nullptr;
  if (out) *out = w;
  return c.used;
}

// Checks of a forward's X, epilogue and outputs; its ranges for the overlap checks.
i8mp_status act_fwd_checks(const i8mp_linear_act* p, Range (&out)[2], Range (&in)[3]) {
  if (!p || !act_ok(p->activation) || !linear_dims_ok(p->M, p->N, p->K)) return I8MP_EINVAL;
  const int64_t M = p->M, N = p->N, K = p->K;
  if (K > I8MP_MAX_CONTRACTION) return I8MP_ERANGE;
  if (!chunked_ok(p->X, M, K, p->ldx, 2) || !elementwise_ok(p->Y, M, N, p->ldy, 2)) return I8MP_EINVAL;
  if (p->residual && !chunked_ok(p->residual, M, N, p->ld_residual, 2)) return I8MP_EINVAL;
  if (p->Z && !elementwise_ok(p->Z, M, N, p->ldz, 2)) return I8MP_EINVAL;
  if (p->bias && !aligned(p->bias, 2)) return I8MP_EINVAL;
  for (int64_t ld : {p->ldx, p->ldy, p->residual ? p->ld_residual : 0, p->Z ? p->ldz : 0})
    if (M > 0 && ld > kMaxDim / M) return I8MP_EINVAL;
  out[0] = mat_range(p->Y, M, N, p->ldy, 2);
  out[1] = mat_range(p->Z, M, N, p->ldz, 2);
  in[0] = mat_range(p->X, M, K, p->ldx, 2);
  in[1] = mat_range(p->residual, M, N, p->ld_residual, 2);
  in[2] = vec_range(p->bias, N, 2);
  return I8MP_OK;
}

i8mp::Epilogue epilogue_of(const i8mp_linear_act* p) {
  return {p->activation, p->bias, p->residual, p->ld_residual, p->Z, p->ldz};
}

// Codes of X (rounded as asked) times codes of W, with the epilogue.
hipError_t act_product(const i8mp_linear_act* p, int8_t* qx, const float* sx, const int8_t* qw, int64_t ldqw,
                       const float* sw, void* split, i8mp::ColmaxJob* side, hipStream_t s) {
  const int64_t M = p->M, N = p->N, K = p->K, kp = padded_k(K);
  if (M <= i8mp::kSkinnyRows) {
    const hipError_t e = side ? i8mp::launch_colmax_finalize(*side, s) : hipSuccess;
    return e != hipSuccess ? e : i8mp::launch_skinny(M, N, K, qx, kp, sx, qw, ldqw, sw, p->Y, p->ldy, epilogue_of(p), s);
  }
  const hipError_t e = i8mp::launch_zero_padding(qx, M, K, kp, s);
  if (e != hipSuccess) return e;
  return i8mp::launch_gemm_epilogue(M, N, kp, qx, kp, sx, qw, ldqw, sw, p->Y, p->ldy, epilogue_of(p), split, side, s);
}

// Checks of the loss's inputs; fills `a` (not its outputs).
i8mp_status distill_inputs(const i8mp_distill* p, i8mp::DistillArgs& a) {
  if (!p || !dtype_ok(p->dtype) || !dtype_ok(p->teacher_dtype)) return I8MP_EINVAL;
  if (!dims_ok(p->T, p->V) || p->T >= (int64_t(1) << 31) || p->V > (int64_t(1) << 30)) return I8MP_EINVAL;
  if (p->kept < 0 || p->kept > I8MP_DISTILL_MAX_KEPT) return I8MP_EINVAL;
  if (!(p->temperature > 0) || !std::isfinite(p->temperature) || !std::isfinite(p->ce_weight)) return I8MP_EINVAL;
  const int64_t elem = dtype_bytes(p->dtype), t_elem = dtype_bytes(p->teacher_dtype);
  if (!elementwise_ok(p->logits, p->T, p->V, p->ld, elem)) return I8MP_EINVAL;
  if (p->T > 0 && p->V > 0 && p->T > kMaxDim / (p->ld > 0 ? p->ld : 1)) return I8MP_EINVAL;
  const bool hard = p->labels && p->ce_weight != 0;
  if (p->T > 0 && p->kept > 0) {
    if (p->idx_bits != 32 && p->idx_bits != 64) return I8MP_EINVAL;
    if (!elementwise_ok(p->teacher, p->T, p->kept, p->teacher_ld, t_elem)) return I8MP_EINVAL;
    if (!elementwise_ok(p->idx, p->T, p->kept, p->idx_ld, p->idx_bits / 8)) return I8MP_EINVAL;
    if (p->teacher_ld > kMaxDim / p->T || p->idx_ld > kMaxDim / p->T) return I8MP_EINVAL;
  }
  if (p->lse && !vec_ok(p->lse, p->T)) return I8MP_EINVAL;
  if (hard && ((p->label_bits != 32 && p->label_bits != 64) || !aligned(p->labels, (uintptr_t)p->label_bits / 8))) return I8MP_EINVAL;
  a.logits = p->logits, a.teacher = p->teacher, a.idx = p->idx, a.lse = p->lse;
  a.labels = hard ? p->labels : nullptr;
  a.T = p->T, a.V = p->V, a.ld = p->ld, a.t_ld = p->teacher_ld, a.i_ld = p->idx_ld;
  a.ignore = p->ignore_index;
  a.tau = p->temperature, a.ce = p->ce_weight;
  const double log2e = 1.4426950408889634074;
  a.itau = 1.0 / (double)a.tau;
  a.cd = log2e * a.itau;
  a.c = (float)a.cd, a.c_lo = (float)(a.cd - (double)a.c);
  a.c1 = (float)log2e, a.c1_lo = (float)(log2e - (double)a.c1);
  a.k = p->kept, a.t_dtype = p->teacher_dtype;
  a.idx64 = p->idx_bits == 64, a.lab64 = p->label_bits == 64;
  return I8MP_OK;
}

// Whether the written range w overlaps anything the loss reads.
bool distill_reads(const i8mp_distill* p, Range w) {
  const int64_t T = p->T;
  return overlap(w, mat_range(p->logits, T, p->V, p->ld, dtype_bytes(p->dtype))) ||
         overlap(w, mat_range(p->teacher, T, p->kept, p->teacher_ld, dtype_bytes(p->teacher_dtype))) ||
         overlap(w, mat_range(p->idx, T, p->kept, p->idx_ld, p->idx_bits / 8)) || overlap(w, vec_range(p->lse, T, 4)) ||
         overlap(w, vec_range(p->labels, T, p->label_bits / 8));
}

i8mp_status distill_run(const i8mp_distill* p, i8mp::DistillArgs& a, void* stream) {
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  const int elem = (int)dtype_bytes(p->dtype);
  if (a.d)
    a.d_aligned = (reinterpret_cast<uintptr_t>(a.d) - reinterpret_cast<uintptr_t>(a.logits)) % 16 == 0 &&
                  (a.d_ld - a.ld) * elem % 16 == 0;
  i8mp::distill_plan(a, elem);
  const hipStream_t s = as_stream(stream);
  return hip_status(p->dtype == I8MP_BF16   ? i8mp::launch_distill_bf16(a, s)
                    : p->dtype == I8MP_FP16 ? i8mp::launch_distill_fp16(a, s)
                                            : i8mp::launch_distill_fp32(a, s));
}

i8mp_status distill_forward(const i8mp_distill* p, float* loss, double* stats, const float* grad, int64_t grad_s,
                            void* d, int64_t d_ld, void* ws, size_t ws_bytes, void* stream, bool step) {
  i8mp::DistillArgs a{};
  i8mp_status st = distill_inputs(p, a);
  if (st != I8MP_OK) return st;
  const int64_t elem = dtype_bytes(p->dtype);
  if (!vec_ok(loss, p->T) || (stats && !aligned(stats, 8))) return I8MP_EINVAL;
  const Range rl = vec_range(loss, p->T, 4), rs = vec_range(stats, p->T * I8MP_DISTILL_STATS, 8);
  Range rd, rg;
  if (step) {
    if (!elementwise_ok(d, p->T, p->V, d_ld, elem) || (p->T > 0 && d_ld > kMaxDim / p->T)) return I8MP_EINVAL;
    if (grad_s < 0 || grad_s >= kMaxDim || (p->T > 0 && (!grad || !aligned(grad, 4) || grad_s > kMaxDim / p->T))) return I8MP_EINVAL;
    rd = mat_range(d, p->T, p->V, d_ld, elem);
    rg = p->T > 0 ? vec_range(grad, (p->T - 1) * grad_s + 1, 4) : Range{};
  }
  if (p->T == 0) return I8MP_OK;
  if (p->V == 0) return I8MP_EINVAL;
  const size_t need = i8mp_distill_workspace_bytes(p->T, p->V, p->kept, p->dtype);
  if (need && (!ws || !aligned(ws, kAlign) || ws_bytes < need)) return I8MP_EWORKSPACE;
  const Range rw = need ? vec_range(ws, (int64_t)need, 1) : Range{};
  const Range out[4] = {rl, rs, rd, rw};
  for (int i = 0; i < 4; ++i) {
    if (distill_reads(p, out[i]) || overlap(out[i], rg)) return I8MP_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return I8MP_EINVAL;
  }
  a.loss = loss, a.stats = stats, a.grad = grad, a.grad_s = grad_s, a.d = d, a.d_ld = d_ld, a.partial = ws;
  return distill_run(p, a, stream);
}

}  // namespace

extern "C" {

size_t i8mp_linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t backward) {
  if (!linear_dims_ok(M, N, K)) return 0;
  return backward ? carve_act_bwd(nullptr, M, N, K, nullptr) : carve_act_fwd(nullptr, M, N, K, true, nullptr);
}

size_t i8mp_linear_wq_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return linear_dims_ok(M, N, K) && !i8mp::skinny_takes_x(M, K) ? carve_act_fwd(nullptr, M, N, K, false, nullptr) : 0;
}

i8mp_status i8mp_linear_act_fwd(const i8mp_linear_act* p, const i8mp_linear_opts* opts, float* colmax_x,
                                float* colmax_w, void* ws, size_t ws_bytes, void* stream) {
  Range out[4], in[4], o2[2], i3[3];
  if (!opts_ok(opts)) return I8MP_EINVAL;
  i8mp_status st = act_fwd_checks(p, o2, i3);
  if (st != I8MP_OK) return st;
  const int64_t M = p->M, N = p->N, K = p->K;
  if (!chunked_ok(p->W, N, K, p->ldw, 2) || (N > 0 && p->ldw > kMaxDim / N)) return I8MP_EINVAL;
  if ((colmax_x && !vec_ok(colmax_x, K)) || (colmax_w && !vec_ok(colmax_w, K))) return I8MP_EINVAL;
  out[0] = o2[0], out[1] = o2[1], out[2] = vec_range(colmax_x, K, 4), out[3] = vec_range(colmax_w, K, 4);
  in[0] = i3[0], in[1] = i3[1], in[2] = i3[2], in[3] = mat_range(p->W, N, K, p->ldw, 2);
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return I8MP_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return I8MP_EINVAL;
  }
  // without outputs there are still the column maxima: the other operand's, and 0 of the one without rows
  const bool empty = M == 0 || N == 0;
  if (empty && (K == 0 || (!colmax_x && !colmax_w))) return I8MP_OK;
  const size_t need = carve_act_fwd(nullptr, M, N, K, true, nullptr);
  if (!ws || !aligned(ws, kAlign) || ws_bytes < need) return I8MP_EWORKSPACE;
  const Range rw = vec_range(ws, (int64_t)need, 1);
  for (int i = 0; i < 4; ++i)
    if (overlap(rw, out[i]) || overlap(rw, in[i])) return I8MP_EINVAL;
  if ((st = device_check()) != I8MP_OK) return st;
  ActFwdWs w;
  carve_act_fwd(ws, M, N, K, true, &w);
  const hipStream_t s = as_stream(stream);
  const int64_t kp = padded_k(K);
  const int r = opts->round;
  const uint64_t ox = pass_offset(opts->offset, 0), ow = pass_offset(opts->offset, 1);
  hipError_t e;
  i8mp::ColmaxJob side{};  // X's and W's slab maxima, folded by the GEMM
  if (colmax_x && colmax_w && K > 0) {
    e = i8mp::launch_quantize_rowwise_colmax_pair(p->X, M, p->ldx, w.qx, kp, w.sx, colmax_x, ox, w.part_x, p->W, N, p->ldw,
                                                  w.qw, kp, w.sw, colmax_w, ow, w.part_w, K, r, opts->seed, false, 0, s);
    side.n = 2;
    side.cols = K;
    side.part[0] = static_cast<const uint16_t*>(w.part_x), side.part[1] = static_cast<const uint16_t*>(w.part_w);
    side.colmax[0] = colmax_x, side.colmax[1] = colmax_w;
    i8mp::rowwise_colmax_geometry(M, K, r, &side.slabs[0], &side.part_ld);
    i8mp::rowwise_colmax_geometry(N, K, r, &side.slabs[1], &side.part_ld);
  } else {
    e = colmax_x && K > 0
            ? i8mp::launch_quantize_rowwise_colmax(p->X, M, K, p->ldx, w.qx, kp, w.sx, colmax_x, r, opts->seed, ox, w.part_x, s)
            : i8mp::launch_quantize_rowwise(p->X, M, K, p->ldx, w.qx, kp, w.sx, r, opts->seed, ox, s);
    if (e == hipSuccess)
      e = colmax_w && K > 0
              ? i8mp::launch_quantize_rowwise_colmax(p->W, N, K, p->ldw, w.qw, kp, w.sw, colmax_w, r, opts->seed, ow, w.part_w, s)
              : i8mp::launch_quantize_rowwise(p->W, N, K, p->ldw, w.qw, kp, w.sw, r, opts->seed, ow, s);
  }
  if (e == hipSuccess)
    e = empty ? i8mp::launch_colmax_finalize(side, s)
              : act_product(p, w.qx, w.sx, w.qw, kp, w.sw, w.split, side.n ? &side : nullptr, s);
  return hip_status(e);
}

i8mp_status i8mp_linear_wq_fwd(const i8mp_linear_act* p, const int8_t* Wq, int64_t ldwq, const float* w_scale,
                               void* ws, size_t ws_bytes, void* stream) {
  Range out[2], in[3];
  i8mp_status st = act_fwd_checks(p, out, in);
  if (st != I8MP_OK) return st;
  const int64_t M = p->M, N = p->N, K = p->K;
  if (!chunked_ok(Wq, N, K, ldwq, 1) || (N > 0 && ldwq > kMaxDim / N) || !vec_ok(w_scale, N)) return I8MP_EINVAL;
  const Range all_in[5] = {in[0], in[1], in[2], mat_range(Wq, N, K, ldwq, 1), vec_range(w_scale, N, 4)};
  for (const Range& r : all_in)
    if (overlap(out[0], r) || overlap(out[1], r)) return I8MP_EINVAL;
  if (overlap(out[0], out[1])) return I8MP_EINVAL;
  if (M == 0 || N == 0) return I8MP_OK;
  const hipStream_t s = as_stream(stream);
  if (i8mp::skinny_takes_x(M, K)) {
    if ((st = device_check()) != I8MP_OK) return st;
    return hip_status(i8mp::launch_skinny_raw(M, N, K, static_cast<const uint16_t*>(p->X), p->ldx, Wq, ldwq, w_scale,
                                              p->Y, p->ldy, epilogue_of(p), s));
  }
  const size_t need = carve_act_fwd(nullptr, M, N, K, false, nullptr);
  if (!ws || !aligned(ws, kAlign) || ws_bytes < need) return I8MP_EWORKSPACE;
  const Range rw = vec_range(ws, (int64_t)need, 1);
  for (const Range& r : all_in)
    if (overlap(rw, r)) return I8MP_EINVAL;
  if (overlap(rw, out[0]) || overlap(rw, out[1])) return I8MP_EINVAL;
  if ((st = device_check()) != I8MP_OK) return st;
  ActFwdWs w;
  carve_act_fwd(ws, M, N, K, false, &w);
  // without a contraction the codes of X are the padding's zeros, and W's may be anything readable
  if (K == 0) Wq = w.qx, ldwq = 0;
  hipError_t e = i8mp::launch_quantize_rowwise(p->X, M, K, p->ldx, w.qx, padded_k(K), w.sx, I8MP_RNE, 0, 0, s);
  if (e == hipSuccess) e = act_product(p, w.qx, w.sx, Wq, ldwq, w_scale, w.split, nullptr, s);
  return hip_status(e);
}

i8mp_status i8mp_linear_act_bwd(const i8mp_linear_act_grad* p, const i8mp_linear_opts* opts, const float* colmax_x,
                                const float* colmax_w, void* ws, size_t ws_bytes, void* stream) {
  if (!p || !opts_ok(opts) || !act_ok(p->activation) || !linear_dims_ok(p->M, p->N, p->K)) return I8MP_EINVAL;
  const int64_t M = p->M, N = p->N, K = p->K;
  if (p->dX && N > I8MP_MAX_CONTRACTION) return I8MP_ERANGE;
  if (p->dW && M > I8MP_MAX_CONTRACTION) return I8MP_ERANGE;
  const bool act = p->activation != I8MP_ACT_NONE;
  if (!chunked_ok(p->dY, M, N, p->lddy, 2) || (act && !chunked_ok(p->Z, M, N, p->ldz, 2))) return I8MP_EINVAL;
  if (p->dX && (!chunked_ok(p->W, N, K, p->ldw, 2) || !elementwise_ok(p->dX, M, K, p->lddx, 2))) return I8MP_EINVAL;
  if (p->dW && (!chunked_ok(p->X, M, K, p->ldx, 2) || !elementwise_ok(p->dW, N, K, p->lddw, 2))) return I8MP_EINVAL;
  if ((p->dbias && !vec_ok(p->dbias, N)) || (colmax_x && !vec_ok(colmax_x, K)) || (colmax_w && !vec_ok(colmax_w, K))) return I8MP_EINVAL;
  for (int64_t ld : {p->lddy, act ? p->ldz : 0, p->dX ? p->lddx : 0, p->dW ? p->ldx : 0})
    if (M > 0 && ld > kMaxDim / M) return I8MP_EINVAL;
  for (int64_t ld : {p->dX ? p->ldw : 0, p->dW ? p->lddw : 0})
    if (N > 0 && ld > kMaxDim / N) return I8MP_EINVAL;
  const Range in[6] = {mat_range(p->dY, M, N, p->lddy, 2), act ? mat_range(p->Z, M, N, p->ldz, 2) : Range{},
                       p->dW ? mat_range(p->X, M, K, p->ldx, 2) : Range{}, p->dX ? mat_range(p->W, N, K, p->ldw, 2) : Range{},
                       vec_range(colmax_x, K, 4), vec_range(colmax_w, K, 4)};
  const Range out[3] = {mat_range(p->dX, M, K, p->lddx, 2), mat_range(p->dW, N, K, p->lddw, 2), vec_range(p->dbias, N, 4)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return I8MP_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return I8MP_EINVAL;
  }
  const bool want_dx = p->dX && M > 0 && K > 0, want_dw = p->dW && N > 0 && K > 0, want_db = p->dbias && N > 0;
  if (!want_dx && !want_dw && !want_db) return I8MP_OK;
  const size_t need = carve_act_bwd(nullptr, M, N, K, nullptr);
  if (!ws || !aligned(ws, kAlign) || ws_bytes < need) return I8MP_EWORKSPACE;
  const Range rw = vec_range(ws, (int64_t)need, 1);
  for (const Range& r : in)
    if (overlap(rw, r)) return I8MP_EINVAL;
  for (const Range& r : out)
    if (overlap(rw, r)) return I8MP_EINVAL;
  i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  ActBwdWs w;
  carve_act_bwd(ws, M, N, K, &w);
  const hipStream_t s = as_stream(stream);
  const int64_t kp = pad16(K);
  const int r = opts->round;
  const uint64_t seed = opts->seed, off = opts->offset;
  i8mp::ActBwdArgs a{};
  a.M = M, a.N = N;
  i8mp::act_bwd_plan(a);
  hipError_t e = hipSuccess;
  if (N > 0) {
    a.dY = p->dY, a.lddy = p->lddy, a.Z = p->Z, a.ldz = p->ldz;
    a.dZ = act ? w.dz : const_cast<uint16_t*>(p->dY);
    a.lddz = act ? a.np : p->lddy;
    a.row_codes = want_dx ? w.q_row : nullptr, a.row_scale = w.s_row;
    a.col_codes = want_dw ? w.q_col : nullptr, a.col_scale = w.s_col;
    a.dbias = want_db ? p->dbias : nullptr;
    a.segmax = w.segmax, a.band_max = w.band_max, a.band_sum = w.band_sum, a.col_max = w.col_max;
    a.seed = seed, a.row_offset = pass_offset(off, 2), a.col_offset = pass_offset(off, 4);
    e = i8mp::launch_act_bwd(a, p->activation, r, s);
  } else if (want_dx) {  // no columns: scales of zero
    e = i8mp::launch_quantize_rowwise(p->dY, M, 0, p->lddy, w.q_row, 16, w.s_row, I8MP_RNE, 0, 0, s);
  }
  // W and X down their columns, in one launch where both column maxima are given
  if (e == hipSuccess && want_dx && want_dw && colmax_x && colmax_w && M > 0) {
    e = i8mp::launch_quantize_colwise_given_pair(p->W, N, K, p->ldw, colmax_w, w.qw, kp, w.sw, pass_offset(off, 3), p->X, M, K,
                                                 p->ldx, colmax_x, w.qx, kp, w.sx, pass_offset(off, 5), r, seed, 0, s);
  } else {
    if (e == hipSuccess && want_dx)
      e = colmax_w ? i8mp::launch_quantize_colwise_given(p->W, N, K, p->ldw, colmax_w, w.qw, kp, w.sw, r, seed, pass_offset(off, 3), s)
                   : i8mp::launch_quantize_colwise(p->W, N, K, p->ldw, w.qw, kp, w.sw, r, seed, pass_offset(off, 3), w.col, s);
    if (e == hipSuccess && want_dw)
      e = colmax_x ? i8mp::launch_quantize_colwise_given(p->X, M, K, p->ldx, colmax_x, w.qx, kp, w.sx, r, seed, pass_offset(off, 5), s)
                   : i8mp::launch_quantize_colwise(p->X, M, K, p->ldx, w.qx, kp, w.sx, r, seed, pass_offset(off, 5), w.col, s);
  }
  // contractions over N and M padded to 16: dZ's codes are zero there
  if (e == hipSuccess && want_dx)
    e = i8mp::launch_gemm_split(I8MP_NN, M, K, a.np, w.q_row, a.np, w.s_row, w.qw, kp, w.sw, p->dX, p->lddx, w.split, nullptr, 0, s);
  if (e == hipSuccess && want_dw)
    e = i8mp::launch_gemm_split(I8MP_TN, N, K, a.mp, w.q_col, a.np, w.s_col, w.qx, kp, w.sx, p->dW, p->lddw, w.split, nullptr, 0, s);
  return hip_status(e);
}

size_t i8mp_distill_workspace_bytes(int64_t T, int64_t V, int32_t kept, int32_t dtype) {
  if (!dims_ok(T, V) || T == 0 || V == 0 || T >= (int64_t(1) << 31) || V > (int64_t(1) << 30) || kept < 0 || !dtype_ok(dtype)) return 0;
  return up(i8mp::distill_workspace_bytes(T, V, kept, (int)dtype_bytes(dtype)));
}

i8mp_status i8mp_distill_fwd(const i8mp_distill* p, float* loss, double* stats, void* ws, size_t ws_bytes,
                             void* stream) {
  return distill_forward(p, loss, stats, nullptr, 0, nullptr, 0, ws, ws_bytes, stream, false);
}

i8mp_status i8mp_distill_step(const i8mp_distill* p, const float* grad, int64_t grad_s, float* loss,
                              void* dlogits, int64_t d_ld, void* ws, size_t ws_bytes, void* stream) {
  return distill_forward(p, loss, nullptr, grad, grad_s, dlogits, d_ld, ws, ws_bytes, stream, true);
}

i8mp_status i8mp_distill_bwd(const i8mp_distill* p, const double* stats, const float* grad, int64_t grad_s,
                             void* dlogits, int64_t d_ld, void* stream) {
  i8mp::DistillArgs a{};
  i8mp_status st = distill_inputs(p, a);
  if (st != I8MP_OK) return st;
  const int64_t T = p->T, elem = dtype_bytes(p->dtype);
  if (!elementwise_ok(dlogits, T, p->V, d_ld, elem) || (T > 0 && d_ld > kMaxDim / T)) return I8MP_EINVAL;
  if (T > 0 && (!stats || !aligned(stats, 8))) return I8MP_EINVAL;
  if (grad_s < 0 || grad_s >= kMaxDim || (T > 0 && (!grad || !aligned(grad, 4) || grad_s > kMaxDim / T))) return I8MP_EINVAL;
  if (T == 0) return I8MP_OK;
  if (p->V == 0) return I8MP_EINVAL;
  const Range rd = mat_range(dlogits, T, p->V, d_ld, elem);
  if (distill_reads(p, rd) || overlap(rd, vec_range(grad, (T - 1) * grad_s + 1, 4)) ||
      overlap(rd, vec_range(stats, T * I8MP_DISTILL_STATS, 8)))
    return I8MP_EINVAL;
  a.stats = const_cast<double*>(stats), a.given = 1;
  a.grad = grad, a.grad_s = grad_s, a.d = dlogits, a.d_ld = d_ld;
  return distill_run(p, a, stream);
}

i8mp_status i8mp_rotary(const i8mp_heads* q, const i8mp_heads* k, int64_t B, int64_t S, int32_t D,
                        int32_t rot, int32_t dtype, int32_t pairs, int32_t inverse, const void* pos,
                        int32_t pos_bits, int64_t pos_b, int64_t pos_s, const double* freqs,
                        void* stream) {
  constexpr int64_t kMaxStride = kMaxDim, kMaxTokens = int64_t(1) << 30;
  if (!q || !dtype_ok(dtype) || (pairs != I8MP_PAIRS_HALF && pairs != I8MP_PAIRS_INTERLEAVED)) return I8MP_EINVAL;
  if (!dims_ok(B, S) || (B > 0 && S > kMaxTokens / B)) return I8MP_EINVAL;
  if (D < 2 || D > 4096 || D % 2 || rot < 2 || rot > D || rot % 2) return I8MP_EINVAL;
  if (pos_bits != 32 && pos_bits != 64) return I8MP_EINVAL;
  const int64_t elem = dtype_bytes(dtype), pos_elem = pos_bits / 8;
  i8mp_heads t[2] = {*q, k ? *k : i8mp_heads{}};
  HeadsView x[2], y[2];
  for (int i = 0; i < 2; ++i) {
    if (t[i].heads < 0 || t[i].heads > 65535) return I8MP_EINVAL;
    for (int64_t s : {t[i].x_b, t[i].x_s, t[i].x_h, t[i].y_b, t[i].y_s, t[i].y_h})
      if (s < 0 || s >= kMaxStride) return I8MP_EINVAL;
    if (t[i].heads == 0 || B == 0 || S == 0) continue;
    for (const auto& v : {std::pair<int64_t, int64_t>{t[i].x_b, t[i].x_s}, {t[i].y_b, t[i].y_s}})
      if ((B > 1 && v.first > kMaxDim / B) || (S > 1 && v.second > kMaxDim / S)) return I8MP_EINVAL;
    if (t[i].x_h > kMaxDim / t[i].heads || t[i].y_h > kMaxDim / t[i].heads) return I8MP_EINVAL;
    x[i] = {reinterpret_cast<uintptr_t>(t[i].x), t[i].x_b, t[i].x_s, t[i].x_h, t[i].heads};
    y[i] = {reinterpret_cast<uintptr_t>(t[i].y), t[i].y_b, t[i].y_s, t[i].y_h, t[i].heads};
  }
  if (t[0].heads + t[1].heads > 65535) return I8MP_EINVAL;
  if (t[0].heads + t[1].heads == 0 || B == 0 || S == 0) return I8MP_OK;
  if (pos_b < 0 || pos_s < 0 || pos_b >= kMaxStride || pos_s >= kMaxStride) return I8MP_EINVAL;
  if (!pos || !aligned(pos, (uintptr_t)pos_elem) || !freqs || !aligned(freqs, 8)) return I8MP_EINVAL;
  const Range rp = vec_range(pos, (B - 1) * pos_b + (S - 1) * pos_s + 1, pos_elem), rf = vec_range(freqs, rot / 2, 8);
  for (int i = 0; i < 2; ++i) {
    if (t[i].heads == 0) continue;
    if (!t[i].x || !t[i].y || !aligned(t[i].x, (uintptr_t)elem) || !aligned(t[i].y, (uintptr_t)elem)) return I8MP_EINVAL;
    if (!heads_distinct(y[i], B, S, D)) return I8MP_EINVAL;
    const Range ry = heads_range(y[i], B, S, D, elem);
    if (overlap(ry, rp) || overlap(ry, rf)) return I8MP_EINVAL;
    for (int j = 0; j < 2; ++j) {
      if (t[j].heads == 0) continue;
      const bool in_place = i == j && x[i].p == y[i].p && x[i].b == y[i].b && x[i].s == y[i].s && x[i].h == y[i].h;
      if (!in_place && !heads_disjoint(y[i], x[j], B, S, D, elem)) return I8MP_EINVAL;
    }
  }
  if (t[0].heads && t[1].heads && !heads_disjoint(y[0], y[1], B, S, D, elem)) return I8MP_EINVAL;
  const i8mp_status st = device_check();
  if (st != I8MP_OK) return st;
  return hip_status(i8mp::launch_rotary(t[0], t[1], B, S, D, rot, dtype, pairs == I8MP_PAIRS_HALF, inverse != 0, pos,
                                        pos_bits == 32, pos_b, pos_s, freqs, as_stream(stream)));
}

}  // extern "C"
