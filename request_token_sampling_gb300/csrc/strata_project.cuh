// strata_project.cuh -- a projection shared by all rows plus each row's own low-rank adapter.
//
//   y[t] = sx[t] sw (x[t] w^T) + h[t] b_c^T,   h[t] = g_c sx[t] (x[t] a_c^T),   c = row_adapter[t]
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace strata {

struct ProjectArgs {
  const void *x, *w;
  const float *x_scale, *w_scale, *adapter_scale;
  const __nv_bfloat16 *a, *b;
  const int32_t* row_adapter;
  __nv_bfloat16* y;
  float* h;  // workspace, [T][R]
  int64_t ldx, ldw, ldy;
  int T, N, K, S, R;
};

__device__ __forceinline__ float proj_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float proj_f32(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

__device__ __forceinline__ float proj_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// h: one warp per row and rank.
template <typename E>
__global__ void __launch_bounds__(256) shrink_kernel(ProjectArgs A) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int t = static_cast<int>(at / A.R), r = static_cast<int>(at % A.R), lane = threadIdx.x & 31;
  if (t >= A.T) return;
  const int c = A.row_adapter[t];
  if (c < 0 || c >= A.S) return;
  const E* x = static_cast<const E*>(A.x) + t * A.ldx;
  const __nv_bfloat16* a = A.a + (static_cast<int64_t>(c) * A.R + r) * A.K;
  float s = 0.0f;
  for (int k = lane; k < A.K; k += 32) s = fmaf(proj_f32(x[k]), proj_f32(a[k]), s);
  s = proj_warp_sum(s);
  if (lane == 0) A.h[at] = A.adapter_scale[c] * ((A.x_scale != nullptr ? A.x_scale[t] : 1.0f) * s);
}

// One warp per output of PROJ_ROWS rows: w is read once for them, x from L1.
constexpr int PROJ_ROWS = 8;
template <typename E>
__global__ void __launch_bounds__(256) project_kernel(ProjectArgs A) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (n >= A.N) return;
  const E* w = static_cast<const E*>(A.w) + n * A.ldw;
  const int t0 = blockIdx.y * PROJ_ROWS, rows = min(PROJ_ROWS, A.T - t0);
  float s[PROJ_ROWS] = {};
  for (int k = lane; k < A.K; k += 32) {
    const float wk = proj_f32(w[k]);
#pragma unroll
    for (int i = 0; i < PROJ_ROWS; ++i)
      if (i < rows) s[i] = fmaf(proj_f32(static_cast<const E*>(A.x)[(t0 + i) * A.ldx + k]), wk, s[i]);
  }
#pragma unroll
  for (int i = 0; i < PROJ_ROWS; ++i) {
    if (i >= rows) break;
    const int t = t0 + i, c = A.S > 0 ? A.row_adapter[t] : -1;
    float v = proj_warp_sum(s[i]), d = 0.0f;
    if (A.x_scale != nullptr) v *= A.x_scale[t] * A.w_scale[n];
    if (c >= 0 && c < A.S) {
      const __nv_bfloat16* b = A.b + (static_cast<int64_t>(c) * A.N + n) * A.R;
      for (int r = lane; r < A.R; r += 32) d = fmaf(A.h[static_cast<int64_t>(t) * A.R + r], proj_f32(b[r]), d);
      v += proj_warp_sum(d);
    }
    if (lane == 0) A.y[t * A.ldy + n] = __float2bfloat16_rn(v);
  }
}

}  // namespace strata
