// Host helpers shared by the translation units of libfa_fwd.so (defined in
// fa_fwd.cu), and the bits of the device status word.
#pragma once
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>
#include <cstring>
#include <utility>

namespace fa_host {

constexpr int kStatusRange = 2;   // a value outside what its format holds
constexpr int kStatusIndex = 4;   // a page id, length or position out of range met by a paged call

int* status_ptr();                                        // device status word of the current device
int cuda_fail(cudaError_t e);                             // records e, returns FA_ERR_CUDA
void* scratch_alloc(size_t bytes, cudaStream_t st);       // stream-ordered scratch (null on failure)
int sm_count();                                           // SMs of the current device (0 on failure)
long long wait_timeout_ns();                              // limit of the bounded on-chip waits
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // null where the driver has none

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while the previous kernel on the stream drains; it waits for that kernel
// (griddepcontrol.wait) before it writes or reads global memory.  Ahead of that
// wait it may read only what was final before the previous kernel let it go, so
// that kernel has to wait for those before it first (fa_decode_join_kernel and
// fa_select_kernel read the lengths early: their predecessors wait, then trigger).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace fa_host
