// A draw whose waits for a row's copies run out: each such row gets id -1 and NaN and the error bit is raised; the
// kernel ends, and the same call with the usual limit is right.  Needs a GPU.  Exit status 1 where that is not so.
#include "../request_token_sampling_gb300/csrc/strata_tail.cu"

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <vector>

// What strata_tail.cu takes from the library's other files.
int strata::host_fail(int code, const char* fmt, ...) {
  std::printf("failed: %d %s\n", code, fmt);
  return code;
}
__device__ uint32_t g_errors;
int strata::tail_device(int* device, uint32_t** errors, int* sms) {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_errors) != cudaSuccess) return STRATA_ECUDA;
  *errors = static_cast<uint32_t*>(p);
  *sms = 152;
  return cudaGetDevice(device) == cudaSuccess ? STRATA_OK : STRATA_ECUDA;
}

int main() {
  constexpr int B = 24, V = 200000, LARGEST = 777;
  std::vector<float> row(V), us(B, 0.5f);
  for (int i = 0; i < V; ++i) row[i] = static_cast<float>(i % 1000) * 1e-3f;
  row[LARGEST] = 90.0f;
  float *logits = nullptr, *u = nullptr, *lps = nullptr;
  int32_t* ids = nullptr;
  if (cudaMalloc(&logits, sizeof(float) * B * V) != cudaSuccess || cudaMalloc(&u, 4 * B) != cudaSuccess || cudaMalloc(&lps, 4 * B) != cudaSuccess ||
      cudaMalloc(&ids, 4 * B) != cudaSuccess || cudaMemcpy(u, us.data(), 4 * B, cudaMemcpyHostToDevice) != cudaSuccess)
    return 2;
  for (int b = 0; b < B; ++b)
    if (cudaMemcpy(logits + static_cast<size_t>(b) * V, row.data(), 4 * V, cudaMemcpyHostToDevice) != cudaSuccess) return 2;
  uint32_t *errors = nullptr, bits = 0;
  int device = 0, sms = 0;
  if (strata::tail_device(&device, &errors, &sms) != STRATA_OK) return 2;

  // the call's own launch with a limit of no look: a look can wait until the copy is there
  constexpr int RANKS = 16, CHUNK = ((V + RANKS - 1) / RANKS + 15) / 16 * 16;
  const size_t smem = (sizeof(strata::DrawShared) + 15) / 16 * 16 + sizeof(float) * CHUNK;
  void (*kernel)(strata::DrawArgs) = strata::draw_kernel<float, 0>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return 2;
  strata::DrawArgs A{logits, V, V, CHUNK, B, false, u, nullptr, nullptr, nullptr, nullptr, ids, lps, errors};
  const strata::Launch launch(B * RANKS, strata::DRAW_THREADS, smem, nullptr, false, RANKS);
  std::vector<int32_t> got(B);
  std::vector<float> lp(B);
  auto read = [&] {
    return cudaDeviceSynchronize() == cudaSuccess && cudaMemcpy(got.data(), ids, 4 * B, cudaMemcpyDeviceToHost) == cudaSuccess &&
           cudaMemcpy(lp.data(), lps, 4 * B, cudaMemcpyDeviceToHost) == cudaSuccess &&
           cudaMemcpyFromSymbol(&bits, g_errors, 4) == cudaSuccess;
  };
  int lost = 0, bad = 0;
  for (int i = 0; i < 20; ++i) {
    if (cudaMemset(ids, 0x55, 4 * B) != cudaSuccess || launch(kernel, A) != cudaSuccess || !read()) return 2;
    for (int b = 0; b < B; ++b) {
      lost += got[b] == -1;
      bad += !((got[b] == -1 && std::isnan(lp[b])) || (got[b] == LARGEST && lp[b] <= 0.0f));
    }
  }
  bad += lost != 20 * B || bits != STRATA_DEVERR_TIMEOUT;
  bits = 0;
  if (cudaMemcpyToSymbol(g_errors, &bits, 4) != cudaSuccess) return 2;
  if (strata_draw_rows(logits, STRATA_DTYPE_F32, B, V, V, u, nullptr, nullptr, nullptr, nullptr, ids, lps, nullptr) != STRATA_OK || !read()) return 2;
  for (int b = 0; b < B; ++b) bad += got[b] != LARGEST;
  bad += bits != 0;
  std::printf("%d rows lost, %d bad\n", lost, bad);
  return bad == 0 ? 0 : 1;
}
