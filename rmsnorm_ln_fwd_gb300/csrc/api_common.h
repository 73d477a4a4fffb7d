// Argument checks shared by the C entry points (norm_api.cu, stream_api.cu):
// dtype, size and stride validation and the byte ranges of the overlap rules.
// Everything here runs on the host and touches no device memory.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "launch.h"
#include "norm.h"

namespace normk {
// Defined in norm_api.cu (not part of the C ABI).
bool device_info_for(int dev, DeviceInfo* out);     // attributes only; no error word
bool current_device_info(DeviceInfo* out);          // the current device, error word and policies included
norm_status launch_result(const char* where, cudaError_t e);
}  // namespace normk

namespace normapi {

constexpr int64_t kMaxH = int64_t(1) << 24;  // counts stay exact in fp32

inline size_t elem_size(norm_dtype d) { return d == NORM_F32 ? 4 : 2; }

inline norm_status check_dtypes(norm_dtype x, norm_dtype w) {
  const bool xv = x == NORM_F32 || x == NORM_BF16 || x == NORM_F16;
  const bool wv = w == NORM_F32 || w == NORM_BF16 || w == NORM_F16;
  if (!xv || !wv) return NORM_ERR_UNSUPPORTED;
  if (w != x && w != NORM_F32) return NORM_ERR_UNSUPPORTED;
  return NORM_OK;
}

inline bool shape_ok(int64_t N, int64_t H) { return N >= 0 && H >= 1 && H <= kMaxH; }

inline bool eps_ok(float eps) { return std::isfinite(eps) && eps > 0.f; }

// The byte range [lo, hi) touched by N rows of H elements, `ld` apart.
struct Span {
  uintptr_t lo, hi;
};

// ld >= H and the extent (N-1)*ld + H elements fits comfortably in 63 bits.
inline bool ld_ok(int64_t ld, int64_t N, int64_t H, size_t es) {
  if (ld < H) return false;
  if (N <= 1) return true;
  const int64_t limit = (INT64_MAX / 8) / (int64_t)es;
  return (N - 1) <= (limit - H) / ld;
}

inline Span rows_span(const void* p, int64_t N, int64_t ld, int64_t H, size_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const uint64_t n = N == 0 ? 0 : (uint64_t)((N - 1) * ld + H) * es;
  return Span{lo, lo + n};
}

inline Span vec_span(const void* p, int64_t n, size_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + (uint64_t)n * es};
}

inline bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// Whether any span of `a` overlaps any span of `b` (empty spans never do).
template <size_t NA, size_t NB>
inline bool any_overlap(const Span (&a)[NA], const Span (&b)[NB]) {
  for (const Span& p : a)
    for (const Span& q : b)
      if (overlap(p, q)) return true;
  return false;
}

// Whether every pointer is a multiple of its element size (null is).
template <size_t N>
inline bool elements_aligned(const void* const (&p)[N], size_t es) {
  for (const void* q : p)
    if (reinterpret_cast<uintptr_t>(q) % es != 0) return false;
  return true;
}

constexpr Span kNoSpan{0, 0};

// Two row tensors may be the same buffer (same pointer and stride) or
// disjoint; anything in between is a partial overlap.
inline bool same_or_disjoint(const void* p, int64_t ldp, const void* q, int64_t ldq, int64_t N, int64_t H, size_t es) {
  if (p == q && ldp == ldq) return true;
  return !overlap(rows_span(p, N, ldp, H, es), rows_span(q, N, ldq, H, es));
}

inline bool disjoint_rows(const void* p, int64_t ldp, const void* q, int64_t ldq, int64_t N, int64_t H, size_t es) {
  return !overlap(rows_span(p, N, ldp, H, es), rows_span(q, N, ldq, H, es));
}

inline normk::Dtype to_dt(norm_dtype d) {
  return d == NORM_BF16 ? normk::DT_BF16 : (d == NORM_F16 ? normk::DT_F16 : normk::DT_F32);
}

// Each compute entry point is an NVTX range named after it, so a profiler
// (ncu --nvtx, nsys) can attribute kernels to the call that launched them; with
// no tool attached a range costs a few nanoseconds.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace normapi
