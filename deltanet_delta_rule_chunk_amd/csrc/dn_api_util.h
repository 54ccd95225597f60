// dn_api_util.h -- argument checks and the workspace that the C ABI's source
// files share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "deltanet.h"

namespace dn {
namespace api {

// Keeps the error for deltanet_last_hip_error; DN_ERR_HIP.
int hip_fail(hipError_t e);

inline bool dtype_ok(int t) { return t == DN_F32 || t == DN_BF16; }
inline size_t dtype_size(int t) { return t == DN_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  const void* p;
  size_t n;  // bytes
};

inline bool overlap(Span a, Span b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

template <int N>
bool any_misaligned(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return true;
  return false;
}

// Whether any output overlaps an input, another output or the workspace, or
// the workspace an input.
template <int NI, int NO>
bool any_overlap(const Span (&in)[NI], const Span (&out)[NO], Span ws) {
  for (int i = 0; i < NO; ++i) {
    for (const Span& x : in)
      if (overlap(out[i], x)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(out[i], out[j])) return true;
    if (overlap(ws, out[i])) return true;
  }
  for (const Span& x : in)
    if (overlap(ws, x)) return true;
  return false;
}

// The caller's workspace, or one allocated and freed on the stream.
class Workspace {
 public:
  Workspace(void* given, size_t need, hipStream_t stream) : p_(given), stream_(stream) {
    if (!given && need > 0) {
      error_ = hipMallocAsync(&p_, need, stream);
      own_ = error_ == hipSuccess;
    }
  }
  Workspace(const Workspace&) = delete;
  Workspace& operator=(const Workspace&) = delete;
  ~Workspace() {
    if (own_) (void)hipFreeAsync(p_, stream_);
  }
  hipError_t error() const { return error_; }
  void* get() const { return p_; }
  // Frees it; the first error of the call.
  hipError_t done(hipError_t e) {
    if (own_) {
      own_ = false;
      const hipError_t f = hipFreeAsync(p_, stream_);
      if (e == hipSuccess) e = f;
    }
    return e;
  }

 private:
  void* p_;
  hipStream_t stream_;
  hipError_t error_ = hipSuccess;
  bool own_ = false;
};

}  // namespace api
}  // namespace dn
