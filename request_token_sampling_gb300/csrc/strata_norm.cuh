// strata_norm.cuh -- root-mean-square norm of rows with the residual's addition and an 8-bit output.
//
//   h = x + residual;  y = h * rsqrt(mean(h^2) + eps) * weight;  scale = max(max|y| / 448, 2^-100);
//   q = e4m3(y / scale)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace strata {

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *y, *q;
  float* scale;
  int64_t ldx, ldr, ldro, ldy, ldq;
  int T, H;
  float eps;
};

constexpr int NORM_THREADS = 256;
constexpr float F8_MAX = 448.0f;
constexpr float F8_SCALE_MIN = 0x1p-100f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// max that keeps a NaN of either side: a NaN in a row makes its scale NaN.
__device__ __forceinline__ float max_nan(float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); }

template <bool MAX>
__device__ __forceinline__ float norm_join(float v) {
  __shared__ float part[NORM_THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < NORM_THREADS / 32; ++i) v = MAX ? max_nan(v, part[i]) : v + part[i];
  return v;
}

// One block per row; the row is read again for each of the three steps (sum of squares, largest
// output, write), the second and third time from L2.
template <typename E>
__global__ void __launch_bounds__(NORM_THREADS) norm_kernel(NormArgs A) {
  const int64_t t = blockIdx.x;
  const E* x = static_cast<const E*>(A.x) + t * A.ldx;
  const E* r = A.residual != nullptr ? static_cast<const E*>(A.residual) + t * A.ldr : nullptr;
  const E* w = static_cast<const E*>(A.weight);
  auto at = [&](int j) { return to_f32(x[j]) + (r != nullptr ? to_f32(r[j]) : 0.0f); };
  float ss = 0.0f;
  for (int j = threadIdx.x; j < A.H; j += NORM_THREADS) {
    const float h = at(j);
    ss += h * h;
  }
  const float inv = rsqrtf(norm_join<false>(ss) / static_cast<float>(A.H) + A.eps);
  float scale = 0.0f;
  if (A.q != nullptr) {
    float big = 0.0f;
    for (int j = threadIdx.x; j < A.H; j += NORM_THREADS) big = max_nan(big, fabsf(at(j) * inv * to_f32(w[j])));
    scale = max_nan(norm_join<true>(big) / F8_MAX, F8_SCALE_MIN);
    if (threadIdx.x == 0) A.scale[t] = scale;
  }
  for (int j = threadIdx.x; j < A.H; j += NORM_THREADS) {
    const float h = at(j), y = h * inv * to_f32(w[j]);
    if (A.residual_out != nullptr) from_f32(h, static_cast<E*>(A.residual_out) + t * A.ldro + j);
    if (A.y != nullptr) from_f32(y, static_cast<E*>(A.y) + t * A.ldy + j);
    if (A.q != nullptr) static_cast<__nv_fp8_e4m3*>(A.q)[t * A.ldq + j] = __nv_fp8_e4m3(y / scale);
  }
}

}  // namespace strata
