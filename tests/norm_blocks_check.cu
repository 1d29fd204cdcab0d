// Host-side check of layer norm's launches on devices with any number of SMs: blocks that go through many rows by turns are no more than
// run at a time, a multiple of eight of them (their rows are cut alike), and the workspace has a group for each.  The library's
// source is compiled in with its CUDA calls replaced; nothing runs on a GPU.  Exit status 1 on a violation.
#include <cuda_runtime.h>

#include <cstdio>

static int device_sms = 0;
static cudaError_t fake_attributes(cudaFuncAttributes* a) { return a->numRegs = 64, cudaSuccess; }
static cudaError_t fake_capture(cudaStreamCaptureStatus* status) { return *status = cudaStreamCaptureStatusNone, cudaSuccess; }
template <typename K, typename A>
static cudaError_t fake_launch(const cudaLaunchConfig_t* cfg, K kernel, A args);
#define cudaFuncGetAttributes(a, kernel) fake_attributes(a)
#define cudaFuncSetAttribute(f, which, v) cudaSuccess
#define cudaStreamGetCaptureInfo(stream, status, id) fake_capture(status)
#define cudaLaunchKernelEx(cfg, kernel, ...) fake_launch(cfg, kernel, __VA_ARGS__)
#include "../request_token_sampling_gb300/csrc/strata_layer_norm.cu"

static long long rings = 0, bad = 0;
static int depth_of(const strata::LayerNormArgs& a) { return a.depth; }
static int depth_of(const strata::LayerNormGradArgs& a) { return a.depth; }
static int groups_of(const strata::LayerNormArgs&) { return 1; }
static int groups_of(const strata::LayerNormGradArgs& a) { return a.groups; }
template <typename K, typename A>
static cudaError_t fake_launch(const cudaLaunchConfig_t* cfg, K, A args) {
  if (depth_of(args) == 0 || cfg->dynamicSmemBytes == 0) return cudaSuccess;  // not a ring's
  const int threads = static_cast<int>(cfg->blockDim.x), blocks = static_cast<int>(cfg->gridDim.x);
  const int at_a_time = std::min({65536 / (64 * threads), 2048 / threads, static_cast<int>(233472 / (cfg->dynamicSmemBytes + 1024))});
  const bool ok = args.T <= 152 ? blocks == args.T : blocks >= 8 && blocks % 8 == 0 && blocks <= std::max(8, device_sms * std::max(1, at_a_time));
  ++rings;
  if ((!ok || groups_of(args) > grad_groups(args.T, args.H)) && ++bad <= 5)
    std::printf("sms %d T %d H %d: %d blocks, %d at a time on an SM\n", device_sms, args.T, args.H, blocks, at_a_time);
  return cudaSuccess;
}

namespace strata {
int host_fail(int code, const char*, ...) { return code; }
int tail_device(int* device, uint32_t** errors, int* sms) {
  static uint32_t word;
  *device = 0;
  *errors = &word;
  *sms = device_sms;
  return STRATA_OK;
}
}  // namespace strata

int main() {
  char* const p = reinterpret_cast<char*>(1 << 20);  // never read
  float* const f = reinterpret_cast<float*>(p);
  for (int sms : {1, 2, 64, 131, 132, 148, 152, 160})
    for (int T : {5, 153, 700, 2000, 8192, 100000})
      for (int H : {520, 1135, 5003, 8192})
        for (int dtype : {STRATA_DTYPE_F32, STRATA_DTYPE_BF16}) {
          device_sms = sms;
          strata_layer_norm_rows(p, H, nullptr, 0, p, p, dtype, T, H, 1e-5f, nullptr, 0, p, H, f, f, nullptr);
          strata_layer_norm_grad(p, H, p, H, p, f, f, nullptr, 0, dtype, T, H, p, H, p, p, p, int64_t{1} << 50, nullptr);
        }
  std::printf("%lld launches, %lld bad\n", rings, bad);
  return bad != 0 || rings < 300;
}
