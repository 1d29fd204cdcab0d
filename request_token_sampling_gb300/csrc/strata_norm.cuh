// strata_norm.cuh -- root-mean-square norm of rows with the residual's addition and an 8-bit output.
//
//   h = x + residual;  y = h * rsqrt(mean(h^2) + eps) * weight;  scale = max(max|y| / 448, 2^-100);
//   q = e4m3(y * (1 / scale))
//
// Bound by HBM from about 100 rows on, by the launch below.  Each element is read and written once: a row
// stays in registers between the two joins (sum of squares, largest output).  What the SMs execute is close
// behind: conversions go two at a time, and q is a product by 1/scale, where a division and conversions one
// by one took twice the time.  Measured (one GB300, us on the GPU): 8192 x 8192 bfloat16 with residual 77
// (6.9 TB/s), 1021 x 5003 float32 with both outputs 11 (4.2 TB/s), 64 x 5120 with 8-bit output 2.1.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "strata_device.cuh"

namespace strata {

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *y, *q;
  float* scale;
  int64_t ldx, ldr, ldro, ldy, ldq;
  int T, H;
  float eps;
};

constexpr float F8_MAX = 448.0f;
constexpr float F8_SCALE_MIN = 0x1p-100f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// max that keeps a NaN of either side: a NaN in a row makes its scale NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// N elements by one access where N of them are 16 bytes (their 8-bit outputs N bytes), or one by one.
template <typename E, int N>
struct alignas(sizeof(E) * N) Pack {
  E v[N];
};

// Two bfloat16 at a time: a word's halves are floats but for 16 zero bits, and one instruction rounds two.
template <typename E, int N>
__device__ __forceinline__ void unpack(const Pack<E, N>& p, float (&f)[N]) {
  if constexpr (sizeof(E) == 2 && N % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(p.v[i]);
  }
}
template <typename E, int N>
__device__ __forceinline__ Pack<E, N> pack(const float (&f)[N]) {
  Pack<E, N> p;
  if constexpr (sizeof(E) == 2 && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) reinterpret_cast<__nv_bfloat162*>(&p)[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) from_f32(f[i], &p.v[i]);
  }
  return p;
}
template <int N>
__device__ __forceinline__ Pack<__nv_fp8_e4m3, N> pack_f8(const float (&f)[N], float by) {
  Pack<__nv_fp8_e4m3, N> p;
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      reinterpret_cast<__nv_fp8x2_storage_t*>(&p)[i] =
          __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * by, f[2 * i + 1] * by), __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p.v[i] = __nv_fp8_e4m3(f[i] * by);
  }
  return p;
}

// Joins a value over the threads of a row: a warp, or the whole block.
template <bool MAX, bool BLOCK>
__device__ __forceinline__ float norm_join(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  if constexpr (BLOCK) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    v = lane < warps ? part[lane] : 0.0f;  // both joins are over values of 0 or more
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
      v = MAX ? max_nan(v, w) : v + w;
    }
  }
  return v;
}

// Stores N bytes of each lane, in a row at `to` + N * lane, by whole words wherever `to` lies: a lane's words
// end where words do in memory and begin with the last bytes of the lane before it.  Lanes without a
// pack follow those with one; `last`: no pack follows this lane's in the row.
template <int N>
__device__ __forceinline__ void store_bytes(uint8_t* to, const Pack<__nv_fp8_e4m3, N>& bytes, bool has, bool last) {
  static_assert(N % 4 == 0, "words");
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&bytes);
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to) & 3u);  // the same in all lanes
  const uint32_t lane = threadIdx.x & 31;
  uint32_t before = __shfl_up_sync(0xFFFFFFFFu, w[N / 4 - 1], 1);
  if (!has) return;
  uint32_t* at = reinterpret_cast<uint32_t*>(to - off);
  if (off == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) at[i] = w[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    if (i == 0 && lane == 0) {
      for (uint32_t b = off; b < 4; ++b) to[b - off] = static_cast<uint8_t>(w[0] >> (8 * (b - off)));
    } else {
      at[i] = __funnelshift_l(before, w[i], 8 * off);
    }
    before = w[i];
  }
  if (lane == 31 || last)
    for (uint32_t b = 0; b < off; ++b) to[N - off + b] = static_cast<uint8_t>(before >> (8 * (4 - off + b)));
}

// The row stays in registers between its sum of squares, its largest output and its outputs: PER packs
// of N elements in each thread of a warp (BLOCK false: a row for each warp) or of the block.  SHIFT: rows
// start anywhere, all tensors of type E at the same distance from a 16-byte boundary.  Packs lie on the
// boundaries, the up to 2 (N - 1) elements before the first and after the last go to as many threads, one
// to each, and the weight and the 8-bit output, which lie otherwise, go element by element.
__host__ __device__ constexpr int norm_most_threads(int n, int per) { return n * per > 8 ? 512 : 1024; }  // by registers
template <typename E, int N, int PER, bool BLOCK, bool SHIFT>
__global__ void __launch_bounds__(BLOCK ? norm_most_threads(N, PER) : 128) norm_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float part[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int threads = BLOCK ? blockDim.x : 32, me = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int64_t t = BLOCK ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (!BLOCK && t >= A.T) return;
  using P = Pack<E, N>;
  const E* x = static_cast<const E*>(A.x) + t * A.ldx;
  const E* r = static_cast<const E*>(A.residual) + t * A.ldr;
  const E* w = static_cast<const E*>(A.weight);
  E* ro = static_cast<E*>(A.residual_out) + t * A.ldro;
  E* y = static_cast<E*>(A.y) + t * A.ldy;
  __nv_fp8_e4m3* q = static_cast<__nv_fp8_e4m3*>(A.q) + t * A.ldq;
  const int head = SHIFT ? min(A.H, static_cast<int>(-(reinterpret_cast<uintptr_t>(x) / sizeof(E)) & (N - 1))) : 0;
  const int packs = (A.H - head) / N;
  int edge = -1;  // this thread's element outside the packs
  if (SHIFT) {
    const int tail = A.H - head - packs * N;
    if (me < head + tail) edge = me < head ? me : packs * N + me;
  }
  auto has = [&](int i) { return i * threads + me < packs; };
  auto at = [&](int i) { return head + (i * threads + me) * N; };
  P px[PER], pr[PER], pw[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (has(i)) {
      px[i] = *reinterpret_cast<const P*>(x + at(i));
      if (A.residual != nullptr) pr[i] = *reinterpret_cast<const P*>(r + at(i));
    }
  }
  float he = 0.0f, we = 0.0f;
  if (SHIFT && edge >= 0) {
    he = to_f32(x[edge]) + (A.residual != nullptr ? to_f32(r[edge]) : 0.0f);
    we = to_f32(w[edge]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!has(i)) continue;
    if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < N; ++e) pw[i].v[e] = w[at(i) + e];
    } else {
      pw[i] = *reinterpret_cast<const P*>(w + at(i));
    }
  }
  float h[PER][N] = {}, ss = he * he;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!has(i)) continue;
    unpack(px[i], h[i]);
    if (A.residual != nullptr) {
      float b[N];
      unpack(pr[i], b);
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] += b[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    if (A.residual_out != nullptr) *reinterpret_cast<P*>(ro + at(i)) = pack<E>(h[i]);
  }
  if (SHIFT && edge >= 0 && A.residual_out != nullptr) from_f32(he, ro + edge);
  const float inv = rsqrtf(norm_join<false, BLOCK>(ss, part[0]) / static_cast<float>(A.H) + A.eps);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!has(i)) continue;
    float b[N];
    unpack(pw[i], b);
#pragma unroll
    for (int e = 0; e < N; ++e) h[i][e] = h[i][e] * inv * b[e];
    if (A.y != nullptr) *reinterpret_cast<P*>(y + at(i)) = pack<E>(h[i]);
  }
  if (SHIFT && edge >= 0) {
    he = he * inv * we;
    if (A.y != nullptr) from_f32(he, y + edge);
  }
  if (A.q == nullptr) return;
  float big = fabsf(he);
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) big = max_nan(big, fabsf(h[i][e]));  // absent packs are zeros
  const float scale = max_nan(norm_join<true, BLOCK>(big, part[1]) / F8_MAX, F8_SCALE_MIN), by = 1.0f / scale;
  if (me == 0) A.scale[t] = scale;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const Pack<__nv_fp8_e4m3, N> out = pack_f8(h[i], by);
    if constexpr (SHIFT) {
      store_bytes<N>(reinterpret_cast<uint8_t*>(q + at(i)), out, has(i), i * threads + me + 1 == packs);
    } else {
      if (has(i)) *reinterpret_cast<Pack<__nv_fp8_e4m3, N>*>(q + at(i)) = out;
    }
  }
  if (SHIFT && edge >= 0) q[edge] = __nv_fp8_e4m3(he * by);
}

// Rows too wide for a block's registers: read again for each step, the second and third time from L2.
template <typename E>
__global__ void __launch_bounds__(1024) norm_wide_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float part[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const E* x = static_cast<const E*>(A.x) + t * A.ldx;
  const E* r = A.residual != nullptr ? static_cast<const E*>(A.residual) + t * A.ldr : nullptr;
  const E* w = static_cast<const E*>(A.weight);
  auto at = [&](int j) { return to_f32(x[j]) + (r != nullptr ? to_f32(r[j]) : 0.0f); };
  float ss = 0.0f;
  for (int j = threadIdx.x; j < A.H; j += 1024) {
    const float h = at(j);
    ss = fmaf(h, h, ss);
  }
  const float inv = rsqrtf(norm_join<false, true>(ss, part[0]) / static_cast<float>(A.H) + A.eps);
  float scale = 0.0f;
  if (A.q != nullptr) {
    float big = 0.0f;
    for (int j = threadIdx.x; j < A.H; j += 1024) big = max_nan(big, fabsf(at(j) * inv * to_f32(w[j])));
    scale = max_nan(norm_join<true, true>(big, part[1]) / F8_MAX, F8_SCALE_MIN);
    if (threadIdx.x == 0) A.scale[t] = scale;
  }
  const float by = 1.0f / scale;
  for (int j = threadIdx.x; j < A.H; j += 1024) {
    const float h = at(j), y = h * inv * to_f32(w[j]);
    if (A.residual_out != nullptr) from_f32(h, static_cast<E*>(A.residual_out) + t * A.ldro + j);
    if (A.y != nullptr) from_f32(y, static_cast<E*>(A.y) + t * A.ldy + j);
    if (A.q != nullptr) static_cast<__nv_fp8_e4m3*>(A.q)[t * A.ldq + j] = __nv_fp8_e4m3(y * by);
  }
}

}  // namespace strata
