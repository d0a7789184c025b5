// Host-side helpers shared by the sources of the C ABI: the error message of
// the calling thread, launch timing, workspace carving and pointer checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <exception>
#include <string>

#include "../../include/prism.h"

namespace prism {

// Stores the message prism_last_error() returns on this thread.
prism_status fail(prism_status st, const std::string& msg);

// Launch timing (prism_timing_begin .. prism_timing_end).
bool timing_on();
hipEvent_t timing_event();                                   // from a pool; nullptr if none
void timing_add(const char* name, hipEvent_t a, hipEvent_t b);

template <typename F>
hipError_t timed(const char* name, hipStream_t s, F&& f) {
  if (!timing_on()) return f();
  hipEvent_t a = timing_event(), b = timing_event();
  if (a) (void)hipEventRecord(a, s);
  hipError_t err = f();
  if (b) (void)hipEventRecord(b, s);
  if (a && b) timing_add(name, a, b);
  return err;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Carve {
  size_t off = 0;
  char* base = nullptr;
  template <typename P>
  P* take(size_t bytes) {
    P* p = base ? reinterpret_cast<P*>(base + off) : nullptr;
    off += align256(bytes);
    return p;
  }
};

inline prism_status check_ptr(const void* p, const char* name, bool required) {
  if (!p) return required ? fail(PRISM_ERR_NULL, std::string(name) + " is NULL") : PRISM_OK;
  if (reinterpret_cast<uintptr_t>(p) & 15u)
    return fail(PRISM_ERR_ALIGN, std::string(name) + " is not 16-byte aligned");
  return PRISM_OK;
}

// A caller's workspace or kept buffer against the size it needs.
inline prism_status check_buffer(const void* p, size_t have, size_t need, const char* what) {
  if (!p) return fail(PRISM_ERR_WORKSPACE, std::string(what) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) & 255u)
    return fail(PRISM_ERR_ALIGN, std::string(what) + " is not 256-byte aligned");
  if (have < need)
    return fail(PRISM_ERR_WORKSPACE, std::string(what) + " has " + std::to_string(have) +
                                         " bytes, needs " + std::to_string(need));
  return PRISM_OK;
}

// Runs an entry point's body so that no C++ exception (a failed allocation of
// a message) leaves it.
template <typename F>
prism_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return PRISM_ERR_HIP;
  }
}

}  // namespace prism

#define CHECK_PTR(p, req)                                  \
  do {                                                     \
    prism_status st_ = prism::check_ptr((p), #p, (req));   \
    if (st_ != PRISM_OK) return st_;                       \
  } while (0)

#define HIP_TRY(name, stream, expr)                                                        \
  do {                                                                                    \
    hipError_t e_ = prism::timed((name), (stream), [&]() { return (expr); });             \
    if (e_ != hipSuccess)                                                                 \
      return prism::fail(PRISM_ERR_HIP, std::string(name) + ": " + hipGetErrorString(e_)); \
  } while (0)
