// strata_host.h -- what the library's host files share: the per-thread error message, and what the
// calls without a context know of the current device.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace strata {

// Stores a one-line message for strata_last_error() and returns `code`.
__attribute__((visibility("hidden"), format(printf, 2, 3))) int host_fail(int code, const char* fmt, ...);

// The current device, its word of STRATA_DEVERR_* bits and its number of SMs.
__attribute__((visibility("hidden"))) int tail_device(int* device, uint32_t** errors, int* sms);

// SMs of a GB300, which sizes that are asked for without a device go by.
constexpr int GB300_SMS = 152;

// A launch.  One that overlaps may be set up while the kernel before it on the stream still runs: the kernel waits
// for that one (griddepcontrol.wait) before it reads or writes anything of the caller's, or of the workspace.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[3];
  Launch(unsigned grid, unsigned block, size_t smem, void* stream, bool overlaps, unsigned cluster = 1, bool together = false) {
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    if (cluster > 1) {
      attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attrs[cfg.numAttrs].val.clusterDim.x = cluster;
      attrs[cfg.numAttrs].val.clusterDim.y = attrs[cfg.numAttrs].val.clusterDim.z = 1;
      ++cfg.numAttrs;
    }
    if (overlaps) {
      attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attrs[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
      ++cfg.numAttrs;
    }
    if (together) {  // blocks wait on one another: all of them run at the same time
      attrs[cfg.numAttrs].id = cudaLaunchAttributeCooperative;
      attrs[cfg.numAttrs].val.cooperative = 1;
      ++cfg.numAttrs;
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
