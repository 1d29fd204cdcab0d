// Host-side check of the losses' launches on devices with any number of SMs: their tiles are cut by the blocks, which have an SM each, so
// there are no more of them than SMs; and the two kernels that work out the parts of dx agree on how many ran at a time.  The
// library's source is compiled in with its CUDA calls replaced; nothing runs on a GPU.  Exit status 1 on a violation.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <type_traits>
#include <vector>

static int calls = 0, device_sms = 0;
static CUresult fake_encode() { return CUDA_SUCCESS; }
static cudaError_t fake_entry(void** p, cudaDriverEntryPointQueryResult* found) {
  *p = reinterpret_cast<void*>(&fake_encode);
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
static cudaError_t fake_capture(cudaStreamCaptureStatus* status) { return *status = cudaStreamCaptureStatusNone, cudaSuccess; }
template <typename K, typename... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t* cfg, K kernel, A... args);
#define cudaGetDriverEntryPointByVersion(name, p, version, flags, found) fake_entry(p, found)
#define cudaFuncSetAttribute(f, which, v) (++calls, cudaSuccess)
#define cudaStreamGetCaptureInfo(stream, status, id) fake_capture(status)
#define cudaLaunchKernelEx(cfg, kernel, ...) fake_launch(cfg, kernel, __VA_ARGS__)
#include "../request_token_sampling_gb300/csrc/strata_loss.cu"

struct Seen {
  unsigned blocks = 0, cluster = 1;
  bool products = false;
  std::vector<int> units;     // of LOSS_DX, and of the kernel that joins its parts
  std::vector<int> numbers;   // dx_blocks
};
static std::vector<Seen> seen;
static void look(Seen& s, const strata::LossArgs& a) { s.units.push_back(a.units); }
static void look(Seen& s, const strata::LossDxArgs& a) { s.units.push_back(a.units); }
static void look(Seen& s, int n) { s.numbers.push_back(n); }
template <typename T>
static void look(Seen&, const T&) {}
template <typename K, typename... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t* cfg, K, A... args) {
  Seen s;
  s.blocks = cfg->gridDim.x;
  s.products = cfg->blockDim.x == strata::LOSS_THREADS;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) s.cluster = cfg->attrs[i].val.clusterDim.x;
  (look(s, args), ...);
  seen.push_back(s);
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
  long long n = 0, bad = 0;
  char* const p = reinterpret_cast<char*>(1 << 20);  // never read
  float* const f = reinterpret_cast<float*>(p);
  int32_t* const ids = reinterpret_cast<int32_t*>(p);
  const int64_t big = int64_t{1} << 50;
  for (int sms : {2, 3, 64, 131, 132, 148, 150, 151, 152, 160})
    for (int T : {1, 33, 128, 129, 300, 1024, 4096, 9000})
      for (int V : {300, 32000, 151001})
        for (int H : {64, 1024, 4096})
          for (int way = 0; way < 4; ++way) {
            device_sms = sms;
            seen.clear();
            const int rc = way == 0 ? strata_cross_entropy_rows(p, H, p, H, T, V, H, ids, f, f, p, big, nullptr)
                                    : strata_cross_entropy_grad(p, H, p, H, T, V, H, ids, f, f, way == 1 ? nullptr : p, H, way == 2 ? nullptr : p, H, p, big, nullptr);
            bool ok = rc == STRATA_OK && !seen.empty();
            int units = -1, products = 0;
            for (const Seen& s : seen) {
              if (!s.products) continue;
              ++products;
              ok = ok && s.blocks >= 1 && s.blocks <= static_cast<unsigned>(sms < 152 ? sms : 152) && s.blocks % s.cluster == 0;
              for (int dx : s.numbers) ok = ok && dx == (way == 1 ? 0 : way == 2 ? static_cast<int>(s.blocks) : dx) && (way != 3 || (dx >= 1 && dx < static_cast<int>(s.blocks)));
              for (int dx : s.numbers) units = dx;  // both products in one launch
              if (s.numbers.empty() && s.cluster == 2 && way >= 2) units = s.units.back();
            }
            ok = ok && products > 0;
            if (way >= 2)  // what LOSS_DX had is what its parts are joined by
              ok = ok && seen.back().units.size() == 1 && seen.back().units[0] == units && units >= 1 && units <= sms;
            ++n;
            if (!ok && ++bad <= 5) std::printf("sms %d T %d V %d H %d way %d: rc %d, %zu launches, units %d\n", sms, T, V, H, way, rc, seen.size(), units);
          }
  std::printf("%lld calls, %lld bad\n", n, bad);
  return bad != 0;
}
