// strata_project.cu -- host side of strata_project_rows (include/strata_tail.h).
#include <cuda_runtime.h>

#include "../../include/strata_tail.h"
#include "strata_host.h"
#include "strata_project.cuh"

using strata::host_fail;

namespace {

// Bits of STRATA_DEVERR_* that kernels of these calls raise (one word on each device).
__device__ uint32_t g_tail_errors;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int cuda_fail(cudaError_t e, const char* what) {
  return host_fail(STRATA_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

template <typename E>
void launch_simple(const strata::ProjectArgs& A, cudaStream_t s) {
  if (A.S > 0) {
    const int64_t warps = static_cast<int64_t>(A.T) * A.R;
    strata::shrink_kernel<E><<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(A);
  }
  const dim3 grid(static_cast<unsigned>((A.N + 7) / 8), static_cast<unsigned>((A.T + strata::PROJ_ROWS - 1) / strata::PROJ_ROWS));
  strata::project_kernel<E><<<grid, 256, 0, s>>>(A);
}

}  // namespace

extern "C" int64_t strata_project_workspace(int T, int S, int R) {
  if (T <= 0 || S <= 0 || R <= 0) return 0;
  return static_cast<int64_t>(T) * R * 4;
}

extern "C" int strata_project_rows(const void* x, int64_t ldx, const float* x_scale, const void* w, int64_t ldw,
                                   const float* w_scale, int dtype, int T, int N, int K, const void* a, const void* b,
                                   int S, int R, const int32_t* row_adapter, const float* adapter_scale, void* y,
                                   int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream) {
  if (dtype != STRATA_DTYPE_BF16 && dtype != STRATA_DTYPE_F8) return host_fail(STRATA_EINVAL, "dtype %d", dtype);
  if (T < 0 || N < 1) return host_fail(STRATA_EINVAL, "T=%d N=%d", T, N);
  if (T > 65535 * strata::PROJ_ROWS) return host_fail(STRATA_ERANGE, "T=%d", T);
  if (K < 1 || K > STRATA_TAIL_MAX_WIDTH) return host_fail(STRATA_ERANGE, "K=%d outside 1..%d", K, STRATA_TAIL_MAX_WIDTH);
  if (S < 0 || S > STRATA_TAIL_MAX_ADAPTERS) return host_fail(STRATA_ERANGE, "S=%d outside 0..%d", S, STRATA_TAIL_MAX_ADAPTERS);
  if (S > 0 && (R < 16 || R > STRATA_TAIL_MAX_RANK || R % 16 != 0))
    return host_fail(STRATA_ERANGE, "R=%d is not a multiple of 16 up to %d", R, STRATA_TAIL_MAX_RANK);
  if (ldx < K || ldw < K || ldy < N) return host_fail(STRATA_EINVAL, "a row stride below its row");
  const bool f8 = dtype == STRATA_DTYPE_F8;
  if ((x_scale != nullptr) != f8 || (w_scale != nullptr) != f8)
    return host_fail(STRATA_EINVAL, "x_scale and w_scale go with 8-bit rows, and only with them");
  if (T == 0) return STRATA_OK;
  if (x == nullptr || w == nullptr || y == nullptr) return host_fail(STRATA_EINVAL, "null x, w or y");
  if (S > 0 && (a == nullptr || b == nullptr || row_adapter == nullptr || adapter_scale == nullptr))
    return host_fail(STRATA_EINVAL, "null a, b, row_adapter or adapter_scale");
  const int64_t esz = f8 ? 1 : 2;
  if (misaligned(x, 16) || misaligned(w, 16) || (S > 0 && (misaligned(a, 16) || misaligned(b, 16))))
    return host_fail(STRATA_EALIGN, "x, w, a or b not 16-byte aligned");
  if (K * esz % 16 != 0 || ldx * esz % 16 != 0 || ldw * esz % 16 != 0 || (S > 0 && K % 8 != 0))
    return host_fail(STRATA_EALIGN, "K or a row stride is not a multiple of 16 bytes");
  if (misaligned(y, 2) || misaligned(x_scale, 4) || misaligned(w_scale, 4) || misaligned(row_adapter, 4) ||
      misaligned(adapter_scale, 4))
    return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  const int64_t need = strata_project_workspace(T, S, R);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || misaligned(workspace, 256)))
    return host_fail(STRATA_EINVAL, "the workspace needs %lld bytes on 256 bytes of alignment", static_cast<long long>(need));
  strata::ProjectArgs A{x, w, x_scale, w_scale, adapter_scale, static_cast<const __nv_bfloat16*>(a),
                        static_cast<const __nv_bfloat16*>(b), row_adapter, static_cast<__nv_bfloat16*>(y),
                        static_cast<float*>(workspace), ldx, ldw, ldy, T, N, K, S, R};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (f8)
    launch_simple<__nv_fp8_e4m3>(A, s);
  else
    launch_simple<__nv_bfloat16>(A, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? STRATA_OK : cuda_fail(e, "strata_project_rows");
}

extern "C" int strata_tail_errors(uint32_t* bits, void* stream) {
  if (bits == nullptr) return host_fail(STRATA_EINVAL, "null bits");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_tail_errors, sizeof(*bits), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_tail_errors, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? STRATA_OK : cuda_fail(e, "strata_tail_errors");
}
