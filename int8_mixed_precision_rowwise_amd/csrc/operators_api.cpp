// C ABI of the operators around the linears (include/i8mp.h, last part).
// Every argument is validated on the host before the first HIP call, so a
// rejected call launches nothing and writes nothing.
#include "checks.h"
#include "internal.h"

#include <algorithm>
#include <utility>

using namespace i8mp::checks;

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

// Whether two views share no element: disjoint byte ranges, or the same batch
// and token strides with the two views' heads in separate parts of a token.
bool heads_disjoint(const HeadsView& a, const HeadsView& c, int64_t B, int64_t S, int64_t D, int64_t elem) {
  if (!overlap(heads_range(a, B, S, D, elem), heads_range(c, B, S, D, elem))) return true;
  if (a.s != c.s || a.b != c.b) return false;
  int64_t period = S > 1 ? a.s : a.b;  // from one token to the next
  if (S > 1 && B > 1) {
    const bool s_inner = a.s <= a.b;
    period = s_inner ? a.s : a.b;
    if (s_inner ? a.b < S * a.s : a.s < B * a.b) return false;
  }
  const HeadsView& lo = a.p <= c.p ? a : c;
  const HeadsView& hi = a.p <= c.p ? c : a;
  if ((hi.p - lo.p) % (uintptr_t)elem) return false;
  const int64_t off = (int64_t)((hi.p - lo.p) / (uintptr_t)elem);
  const int64_t lo_ext = (lo.H - 1) * lo.h + D, hi_ext = (hi.H - 1) * hi.h + D;
  return off >= lo_ext && (B * S == 1 || off + hi_ext <= period);
}

}  // namespace

extern "C" {

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
