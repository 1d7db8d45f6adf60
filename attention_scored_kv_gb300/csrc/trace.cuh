// NVTX ranges around every ABI call, for profiler timelines (Nsight Systems, ncu's
// range filters): on when the environment variable KVS_NVTX is set to anything but
// "0" when the library is first used.  Without an attached tool the calls do nothing.
#pragma once
#include <nvtx3/nvToolsExt.h>

#include <cstdlib>
#include <cstring>

namespace kvs {

inline bool tracing_on() {
  static const bool on = [] {
    const char* v = std::getenv("KVS_NVTX");
    return v && *v && std::strcmp(v, "0") != 0;
  }();
  return on;
}

struct Trace {
  explicit Trace(const char* name) : on(tracing_on()) {
    if (on) nvtxRangePushA(name);
  }
  ~Trace() {
    if (on) nvtxRangePop();
  }
  Trace(const Trace&) = delete;
  Trace& operator=(const Trace&) = delete;
  bool on;
};

}  // namespace kvs
