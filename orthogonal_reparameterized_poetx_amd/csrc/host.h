// Host-side services of api.hip for the entry points defined in other files:
// the thread's error message and the optional per-launch timing record.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace poetx {

constexpr size_t kWsAlign = 256;   // alignment of a workspace and of its parts

// sets poetx_last_error() (printf format) and returns code
int host_fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// POETX_EHIP with the runtime's message if the last launch failed
int host_check_launch(const char* what);
// POETX_EWORKSPACE unless ws is 256-byte aligned and holds `need` bytes
int host_check_ws(void* ws, size_t have, size_t need);

// records an event pair around the launches issued during its lifetime, if
// poetx_timing_enable(1) is in force
class HostTimer {
 public:
  HostTimer(hipStream_t s, const char* name, double flops, double bytes);
  ~HostTimer();
  HostTimer(const HostTimer&) = delete;
  HostTimer& operator=(const HostTimer&) = delete;

 private:
  void* t_;
};

}  // namespace poetx
