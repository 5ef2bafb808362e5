// The handle's contents and the helpers that every C entry point shares: error records, the
// device guard, pointer alignment.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "vla.h"
#include "vla_internal.cuh"

constexpr int kHostSlots = 3;   // staging slots of the host-buffer path (copy in / scan / copy out)

struct vla_handle_s {
  int device = 0;
  int sm_count = 0;
  vla::DevStatus* status = nullptr;
  std::string last_error;
  unsigned long long wait_limit = vla::kWaitLimitNs;   // of the products' waits, in ns; 0: their self-test
  // Host-buffer path (vla_scan_fwd_host), made on its first use: a device workspace with
  // the state and kHostSlots staging slots, a copy-in and a copy-out stream, and events.
  bool host_ready = false;
  int last_gathered = -1;       // copy-in path and window of the last vla_scan_fwd_host call
  long long last_seg = 0;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  cudaStream_t s_in = nullptr, s_out = nullptr;
  cudaEvent_t ev_start = nullptr, ev_end = nullptr;
  cudaEvent_t ev_in[kHostSlots] = {}, ev_run[kHostSlots] = {}, ev_out[kHostSlots] = {};
};

namespace vla {
namespace api {

// Records the message on the handle (the calling thread's when h is NULL); returns `code`.
vla_err_t fail(vla_handle_t h, vla_err_t code, const std::string& msg);

inline std::string cuda_msg(const char* what, cudaError_t e) {
  return std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")";
}

// Runs `fn` with `device` current and restores the caller's device.
template <typename F>
cudaError_t on_device(int device, F fn) {
  int prev = -1;
  cudaError_t e = cudaGetDevice(&prev);
  if (e != cudaSuccess) return e;
  if (prev != device) {
    e = cudaSetDevice(device);
    if (e != cudaSuccess) return e;
  }
  cudaError_t r = fn();
  if (prev != device) {
    cudaError_t e2 = cudaSetDevice(prev);
    if (r == cudaSuccess) r = e2;
  }
  return r;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace api
}  // namespace vla
