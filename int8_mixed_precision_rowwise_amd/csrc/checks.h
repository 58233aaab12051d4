// Argument checks and workspace carving shared by the C ABI's sources: every
// argument is validated on the host before the first HIP call.
#pragma once

#include "../../include/i8mp.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

namespace i8mp {
namespace checks {

constexpr int64_t kMaxDim = int64_t(1) << 40;  // rejects sizes whose products could overflow

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [begin, end) byte range of a rows x cols matrix with leading dim ld.
struct Range {
  uintptr_t b = 0, e = 0;
};

inline Range mat_range(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  Range r;
  if (!p || rows <= 0 || cols <= 0) return r;
  r.b = reinterpret_cast<uintptr_t>(p);
  r.e = r.b + (uintptr_t)(((rows - 1) * ld + cols) * elem);
  return r;
}

inline Range vec_range(const void* p, int64_t n, int64_t elem) { return mat_range(p, 1, n, n, elem); }

inline bool overlap(Range a, Range b) { return a.b < a.e && b.b < b.e && a.b < b.e && b.b < a.e; }

inline bool dims_ok(int64_t a, int64_t b = 0, int64_t c = 0) {
  return a >= 0 && b >= 0 && c >= 0 && a < kMaxDim && b < kMaxDim && c < kMaxDim;
}

// Input or output matrix of `elem`-byte elements read/written in 16-byte
// chunks: base 16-aligned, rows 16-aligned, ld >= cols.  A matrix with no
// elements may be NULL.
inline bool chunked_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  if (rows == 0 || cols == 0) return ld >= 0 && ld < kMaxDim;
  return p && aligned(p, 16) && ld >= cols && ld < kMaxDim && (ld * elem) % 16 == 0;
}

// Output matrix written element by element: natural alignment, ld >= cols.
inline bool elementwise_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  if (rows == 0 || cols == 0) return ld >= 0 && ld < kMaxDim;
  return p && aligned(p, (uintptr_t)elem) && ld >= cols && ld < kMaxDim;
}

inline bool vec_ok(const void* p, int64_t n) { return n == 0 || (p && aligned(p, 4)); }

// gfx950 check, cached per device: 0 unknown, 1 ok, 2 not gfx950.
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_device_state[kMaxDevices];

inline i8mp_status device_check() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return I8MP_EDEVICE;
  }
  if (dev < kMaxDevices) {
    const int s = g_device_state[dev].load(std::memory_order_relaxed);
    if (s == 1) return I8MP_OK;
    if (s == 2) return I8MP_EDEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    (void)hipGetLastError();
    return I8MP_EDEVICE;
  }
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) g_device_state[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? I8MP_OK : I8MP_EDEVICE;
}

inline i8mp_status hip_status(hipError_t e) { return e == hipSuccess ? I8MP_OK : I8MP_EHIP; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr size_t kAlign = 256;
inline size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }
inline int64_t pad16(int64_t n) { return (n + 15) / 16 * 16; }

// Workspace carving: regions in a fixed order, each 256-byte aligned.
struct Carver {
  char* base;
  size_t used = 0;
  void* take(size_t n) {
    void* p = base ? base + used : nullptr;
    used += up(n);
    return p;
  }
};

}  // namespace checks
}  // namespace i8mp
