// fa_host.h -- host-side helpers of fa_api.cu that other host translation
// units of the library use (internal; no device code).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/fa.h"

namespace fa {

// The argument checks of fa_fwd and the current device's support check
// (compute capability 10.3, the library's static arrays reachable), in that
// order; launches and allocates nothing.
fa_status_t check_call(const void* q, const void* k, const void* v, const void* o,
                       const void* lse, int B, int H, int Sq, int Skv, int D,
                       float scale, int dtype);

// The argument checks alone (no device call).
fa_status_t check_args(const void* q, const void* k, const void* v, const void* o,
                       const void* lse, int B, int H, int Sq, int Skv, int D, float scale,
                       int dtype);

// A tanh cap is off (0) or within the range that the kernels' fp32 terms cover.
inline bool softcap_ok(float c) { return c == 0.f || (c >= 1e-6f && c <= 1e6f); }

// The current device's support check alone (compute capability 10.3).
fa_status_t check_device();

// Process-unique id of the calling thread's current CUDA context; a thread that
// has none yet gets its device's (0 when that fails).  Device addresses of the library's static __device__
// arrays belong to the context that loaded the module: after
// cudaDeviceReset the primary context is a new one, with a new id, and every
// cached address must be looked up again.
unsigned long long context_id();

// What a launch on the current device needs, after its support check.
struct LaunchEnv {
  int sm_count;
  unsigned* status;               // device status word
  unsigned long long timeout_ns;  // watchdog limit
  bool captured;                  // the stream is being captured
  unsigned long long* sched;      // the scheduler slots
};
fa_status_t launch_env(cudaStream_t stream, LaunchEnv* out);

// A scheduler slot for one persistent launch (PrefillParams::sched).
unsigned long long* take_sched_slot(const LaunchEnv& env);

// The library's workspace for the score and cache calls on `stream` of the
// current device, grown to `need` bytes.  Not for captured calls.  `hold` is
// locked (the device's lock): keep it until the call's launches are all in the
// stream, so that no other thread's call comes between them or grows the workspace
// under them.
fa_status_t library_workspace(cudaStream_t stream, size_t need, void** out,
                              std::unique_lock<std::mutex>* hold);

// The current device's multiprocessors; 0 without a supported device.
int device_sms();

// TMA descriptor of a [heads, rows, D] 16-bit tensor, boxes of 64 columns x
// box_rows.
fa_status_t encode_rows(CUtensorMap* m, const void* base, int D, int rows, int heads,
                        int box_rows, bool bf16);

}  // namespace fa
