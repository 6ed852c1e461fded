// Pieces of the C interface that every entry point needs: errors without
// exceptions, the status of a launch, alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string>

#include "../../include/mlora.h"

namespace mlora {

// The message mlora_last_error() returns on this thread (api.cpp).
void set_last_error(const std::string& msg);

// No exception leaves a C entry, not even from building a message.
inline mlora_status api_fail(mlora_status st, const char* msg) noexcept {
  try {
    set_last_error(msg);
  } catch (...) {
  }
  return st;
}

inline mlora_status api_launched() noexcept {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return MLORA_OK;
  try {
    set_last_error(std::string("kernel launch: ") + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")");
  } catch (...) {
  }
  return MLORA_ERR_HIP;
}

inline bool api_aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace mlora
