// layer_checks.hpp -- the argument checks that layer_api.cpp and block_api.cpp share.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/ssd_layer.h"
#include "layer_host.hpp"

namespace ssd {
ssd_status report(ssd_status st, const char* msg);   // ssd_api.cpp: the thread's last error

inline ssd_status fail(ssd_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline ssd_status fail(ssd_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report(st, buf);
}
inline ssd_status ok() { return report(SSD_OK, ""); }
inline ssd_status launched(hipError_t e, const char* what) {
  return e == hipSuccess ? ok() : fail(SSD_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

template <typename F>
inline ssd_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return report(SSD_ERR_INTERNAL, "unexpected exception");
  }
}

// Whether the product of the sizes, in elements of 8 bytes, fits int64.
template <typename... I>
inline bool fits(I... sizes) {
  int64_t room = INT64_MAX / 8;
  for (int64_t s : {(int64_t)sizes...}) {
    if (s < 1) return false;
    room /= s;
  }
  return room > 0;
}

inline bool is_aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
template <typename... P>
inline bool aligned16(P... ps) {
  for (const void* p : {static_cast<const void*>(ps)...})
    if (!is_aligned(p, 16)) return false;
  return true;
}

// A strided operand's strides (contiguous ones for NULL).
inline void strides_of(const ssd_strides* s, int64_t L, int64_t width, int64_t out[2]) {
  out[0] = s ? s->batch : L * width;
  out[1] = s ? s->token : width;
}
inline ssd_status check_strides(const char* name, const int64_t s[2], int64_t batch, int64_t L,
                         int64_t width, bool output) {
  if (s[0] < 0 || s[1] < 0) return fail(SSD_ERR_BAD_VALUE, "%s: strides must not be negative", name);
  // the offset of the last element, in bytes, has to fit int64
  const __int128 last = (__int128)(batch - 1) * s[0] + (__int128)(L - 1) * s[1] + width;
  if (last > INT64_MAX / 8) return fail(SSD_ERR_BAD_SHAPE, "%s: strides overflow int64", name);
  if (output) {
    const bool rows = L == 1 || s[1] >= width;
    const bool outer = batch == 1 || (L == 1 ? s[0] >= width : s[0] >= (L - 1) * s[1] + width);
    const bool inner = batch == 1 || (s[0] >= width && (L == 1 || s[1] >= (batch - 1) * s[0] + width));
    if (!rows || !(outer || inner))
      return fail(SSD_ERR_BAD_VALUE, "%s: the rows of an output must not overlap", name);
  }
  return SSD_OK;
}
// Accesses of `per` elements of `size` bytes to every row of a strided operand.
inline bool row_vectors(const void* p, const int64_t s[2], int per, size_t size) {
  return is_aligned(p, per * size) && s[0] % per == 0 && s[1] % per == 0;
}
// Whether two buffers of `bytes` share memory (neither does where one is absent).
inline bool overlap(const void* a, const void* b, int64_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p && q && (p < q ? q - p : p - q) < (uintptr_t)bytes;
}

inline ssd_status check_io(int32_t io_dtype, int64_t reserved) {
  if (io_dtype != SSD_BF16 && io_dtype != SSD_F32)
    return fail(SSD_ERR_BAD_DTYPE, "io_dtype must be SSD_BF16 or SSD_F32 (got %d)", io_dtype);
  if (reserved != 0) return fail(SSD_ERR_BAD_DTYPE, "reserved field must be 0");
  return SSD_OK;
}
inline size_t element(int32_t io_dtype) { return io_dtype == SSD_BF16 ? 2 : 4; }

// ---- gated norm ----

inline ssd_status norm_shape(const ssd_gated_norm_problem& p) {
  if (p.batch <= 0 || p.seqlen <= 0 || p.channels <= 0 || p.ngroups <= 0)
    return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  if (p.channels % p.ngroups != 0)
    return fail(SSD_ERR_BAD_SHAPE, "channels (%lld) must be a multiple of ngroups (%lld)",
                (long long)p.channels, (long long)p.ngroups);
  if (!fits(p.batch, p.seqlen, p.channels))
    return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  ssd_status st = check_io(p.io_dtype, p.reserved);
  if (st != SSD_OK) return st;
  if (!(p.eps >= 0.0f) || std::isinf(p.eps)) return fail(SSD_ERR_BAD_VALUE, "eps must be finite and >= 0");
  if (p.norm_before_gate != 0 && p.norm_before_gate != 1)
    return fail(SSD_ERR_BAD_VALUE, "norm_before_gate must be 0 or 1 (got %d)", p.norm_before_gate);
  return SSD_OK;
}
inline ssd_status norm_supported(const ssd_gated_norm_problem& p) {
  if (p.channels / p.ngroups > norm_group_limit())
    return fail(SSD_ERR_UNSUPPORTED, "at most %lld channels per group (got %lld)",
                (long long)norm_group_limit(), (long long)(p.channels / p.ngroups));
  if (!norm_grid_ok(p.batch, p.seqlen, p.channels, p.ngroups))
    return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
  return SSD_OK;
}
}  // namespace ssd
