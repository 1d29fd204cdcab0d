// strata_host.h -- what the library's host files share: the per-thread error message, and what the
// calls without a context know of the current device.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace strata {

// Stores a one-line message for strata_last_error() and returns `code`.
__attribute__((visibility("hidden"), format(printf, 2, 3))) int host_fail(int code, const char* fmt, ...);

// The current device's word of STRATA_DEVERR_* bits and its number of SMs.
__attribute__((visibility("hidden"))) int tail_device(uint32_t** errors, int* sms);

// A launch that may be set up while the kernel before it on the stream still runs: the kernel waits for that one
// (griddepcontrol.wait) before it reads or writes anything of the caller's, or of the workspace.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[2];
  Launch(unsigned grid, unsigned block, size_t smem, void* stream, unsigned cluster = 1) {
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
      attrs[1].id = cudaLaunchAttributeClusterDimension;
      attrs[1].val.clusterDim.x = cluster;
      attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
    }
    cfg.attrs = attrs;
  }
  Launch(const Launch&) = delete;
  template <typename... P, typename... A>
  cudaError_t operator()(void (*kernel)(P...), A... args) const {
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  }
};

}  // namespace strata
