// fa_host.h — host-side state and checks shared by the translation units of
// the C ABI (defined in fa_fwd.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

namespace fa {

struct DeviceState {
  bool ready = false;
  bool supported = false;
  int device = 0;
  int sm_count = 0;
  int* status = nullptr;  // device address of g_device_status
  int* debug_record = nullptr;  // device address of g_debug_record
};

// The current device's state, set up on first use: FA_OK, FA_ERR_UNSUPPORTED
// (not sm_103) or FA_ERR_CUDA.  The launch fault hook (FA_FAULT_INJECT=launch)
// answers FA_ERR_CUDA here.
int current_device(DeviceState** out);

// The driver's tensor-map encoder (valid once current_device succeeded).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

bool ranges_overlap(const void* a, size_t abytes, const void* b, size_t bbytes);
bool aligned16(const void* p);
unsigned long long timeout_ns_from_env();

}  // namespace fa
