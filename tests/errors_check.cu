// strata_tail_errors against kernels of another stream that raise a bit all the while: every time that the bit goes
// up, one call has to tell it.  The library's source is compiled in, so that the test can raise bits.  Needs a GPU.
// Exit status 1 where a bit was lost.
#include "../request_token_sampling_gb300/csrc/strata_project.cu"

#include <cstdio>
#include <thread>

// What strata_project.cu takes from the library's other files.
int strata::host_fail(int code, const char* fmt, ...) {
  std::printf("failed: %d %s\n", code, fmt);
  return code;
}

__global__ void raise_bits(unsigned long long* raised) {
  for (int i = 0; i < 100; ++i) {
    if ((atomicOr(&g_tail_errors, 0x08u) & 0x08u) == 0u) ++*raised;
    __nanosleep(500);
  }
}

int main() {
  cudaStream_t mine, other;
  unsigned long long* raised = nullptr;
  if (cudaStreamCreateWithFlags(&mine, cudaStreamNonBlocking) != cudaSuccess ||
      cudaStreamCreateWithFlags(&other, cudaStreamNonBlocking) != cudaSuccess || cudaMalloc(&raised, 8) != cudaSuccess ||
      cudaMemset(raised, 0, 8) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
    return 2;
  unsigned long long told = 0, all = 0;
  uint32_t bits = 0;
  // both kernels are on the GPU before the counting begins
  raise_bits<<<1, 1, 0, other>>>(raised);
  if (cudaDeviceSynchronize() != cudaSuccess || strata_tail_errors(&bits, mine) != STRATA_OK || cudaMemset(raised, 0, 8) != cudaSuccess)
    return 2;
  std::atomic<bool> done{false};
  std::thread raising([&] {
    for (int i = 0; i < 400; ++i) raise_bits<<<1, 1, 0, other>>>(raised);
    (void)cudaStreamSynchronize(other);
    done = true;
  });
  while (!done) {
    if (strata_tail_errors(&bits, mine) != STRATA_OK) return 2;
    told += bits != 0;
  }
  raising.join();
  if (cudaDeviceSynchronize() != cudaSuccess || strata_tail_errors(&bits, mine) != STRATA_OK) return 2;
  told += bits != 0;
  if (cudaMemcpy(&all, raised, 8, cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
  std::printf("raised %llu told %llu\n", all, told);
  return all == told && all > 20 ? 0 : 1;
}
