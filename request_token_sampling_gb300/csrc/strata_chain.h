// strata_chain.h -- which launches of a stream may be set up while the kernel before them still runs.
//
// A kernel launched that way (programmatic dependent launch) waits on the GPU for the end of the one kernel before
// it.  That this implies the end of all earlier ones holds as long as every kernel waited for its own
// predecessor before it ended, or before it let the next one start.  Two kinds of kernels do not:
//   a sampling call with STRATA_FLAG_OWN_OUTPUTS waits for nothing;
//   the operators of strata_tail.h, and what they follow, still run when the next kernel starts, and a sampling
//   call with early loads lets the one after it start before it has waited itself.
// So an operator behind a call with own outputs, and a call with early loads behind an operator, is launched as an
// ordinary kernel, which starts when all work of the stream has ended.  One such launch is enough: what comes
// after it can rely on it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <memory>
#include <mutex>
#include <unordered_map>

namespace strata {

// What the launches on a stream so far leave open.
struct ChainState {
  bool waitless = false;  // the end of the newest kernel says nothing of those before it
  bool early = false;     // an operator may still run when the kernel after the newest one starts

  // May the next operator's first kernel overlap?  Its later ones follow a kernel that has waited.
  bool operator_overlaps() const { return !waitless; }
  void operator_launched(bool overlapped) {
    if (!overlapped) waitless = false;
    early = true;
  }
  // `early_load`: the call reads its inputs, and lets the next kernel start, before it waits (if it waits at all).
  bool sampling_overlaps(bool early_load) const { return !(early_load && early); }
  void sampling_launched(bool overlapped, bool early_load, bool own_outputs) {
    if (!overlapped) waitless = early = false;
    if (!early_load) early = false;  // it waited before it let anything start
    if (overlapped && own_outputs) waitless = true;
  }
};

// Set by the first operator and by the first overlapping call with own outputs of the process.  Each side sets
// its own and then looks at the other's, so that of two at the same time one sees the other.
inline std::atomic<bool>& operators_used() {
  static std::atomic<bool> used{false};
  return used;
}
inline std::atomic<bool>& waitless_used() {
  static std::atomic<bool> used{false};
  return used;
}

// The state of one stream, and of the capture that goes through it.
struct StreamChain {
  std::mutex lock;
  ChainState eager, captured;
  unsigned long long capture = 0;
};

inline StreamChain& chain_of(int device, cudaStream_t stream) {
  static thread_local char here;  // the per-thread default stream is another one in each thread
  static std::mutex lock;
  static std::unordered_map<uint64_t, std::unique_ptr<StreamChain>> chains;  // entries are never taken out
  const uint64_t handle = reinterpret_cast<uint64_t>(stream == cudaStreamPerThread ? reinterpret_cast<cudaStream_t>(&here)
                                                     : stream == cudaStreamLegacy  ? nullptr
                                                                                   : stream);
  const uint64_t key = handle ^ static_cast<uint64_t>(device) << 56;
  static thread_local uint64_t last_key = 0;
  static thread_local StreamChain* last = nullptr;
  if (last != nullptr && key == last_key) return *last;
  std::lock_guard<std::mutex> hold(lock);
  std::unique_ptr<StreamChain>& c = chains[key];
  if (!c) {
    c = std::make_unique<StreamChain>();
    c->eager.waitless = waitless_used().load();  // calls before the first operator were not noted by stream
  }
  last_key = key;
  last = c.get();
  return *c;
}

// The state of the stream that a call launches on, held from the decision to the launch.
class Chain {
 public:
  Chain(int device, cudaStream_t stream) : chain_(chain_of(device, stream)), hold_(chain_.lock) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(stream, &status, &id) != cudaSuccess) {
      (void)cudaGetLastError();  // the launch itself will say
      status = cudaStreamCaptureStatusNone;
    }
    state_ = &chain_.eager;
    if (status == cudaStreamCaptureStatusActive) {
      if (id != chain_.capture) {
        chain_.capture = id;
        chain_.captured = ChainState{};
        chain_.captured.waitless = waitless_used().load();
      }
      state_ = &chain_.captured;
    }
  }
  ChainState* operator->() { return state_; }

 private:
  StreamChain& chain_;
  std::unique_lock<std::mutex> hold_;
  ChainState* state_;
};

// Runs launch(overlaps), which launches an operator's kernels: the first one with that, later ones overlapping.
template <typename F>
cudaError_t launch_operator(int device, void* stream, F launch) {
  try {
    operators_used().store(true);
    Chain chain(device, static_cast<cudaStream_t>(stream));
    const bool overlaps = chain->operator_overlaps();
    const cudaError_t e = launch(overlaps);
    if (e == cudaSuccess)
      chain->operator_launched(overlaps);
    else
      chain->early = true;  // one of its kernels may run
    return e;
  } catch (...) {  // no exception leaves a C call
    return cudaErrorMemoryAllocation;
  }
}

}  // namespace strata
