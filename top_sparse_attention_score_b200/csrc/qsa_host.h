// qsa_host.h -- host helpers shared by the translation units of the C ABI: error text,
// launch accounting, device set-up and the tensor-map encoder.  Defined in qsa_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>
#include <utility>

#include "qsa.h"

namespace qsa {
namespace host {

// Record the calling thread's error text and return `code`.
int fail(int code, const char* fmt, ...);
// Clear it and return QSA_OK.
int ok();
// Count a launch and turn the error its launch call returned into QSA_ERR_CUDA.
int launched(const char* what, cudaError_t e);
// Kernel attributes, SM count and status word of the current device, once per device.
int prepare_device();
// The current device's status word (after prepare_device).
uint32_t* device_status();
int sm_count();
int tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while its predecessor on the stream drains; every kernel here waits on
// griddepcontrol.wait before touching memory its predecessors use.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace host
}  // namespace qsa
