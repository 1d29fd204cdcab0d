// strata_layer_norm.cuh -- layer norm of rows, with the residual's addition, and its way back.
//
//   h = x + residual;  v = (h - mean(h)) rstd, rstd = 1 / sqrt(mean((h - mean)^2) + eps);  y = v weight + bias
//   a = dy weight;  dx = rstd (a - mean(a) - v mean(a v)) + dresidual;  dweight = sum_t dy v;  dbias = sum_t dy
//
// Bound by HBM: every element is read and written once.  A row stays in registers between its joins, so the variance
// is a second sum over differences from the mean, not a difference of large sums.
#pragma once

#include "strata_norm.cuh"

namespace strata {

struct LayerNormArgs {
  const void *x, *residual, *weight, *bias;
  void *residual_out, *y;
  float *mean, *rstd;
  int64_t ldx, ldr, ldro, ldy;
  int T, H;
  float eps;
};

__host__ __device__ constexpr int layer_norm_most_threads(int n, int per) { return n * per > 8 ? 512 : 1024; }  // by registers

// The joins of a row's sum and of its squared differences.  Each warp takes both about its own mean, by shuffles, and the
// warps' come together behind one barrier: the squares about the row's mean are the warps' and, for each warp, its elements times
// the square of what the means differ by.  `mine`: this warp's elements.
template <bool BLOCK>
__device__ __forceinline__ float layer_norm_mean(float s, int mine) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return mine > 0 ? s / static_cast<float>(mine) : 0.0f;
}
template <bool BLOCK>
__device__ __forceinline__ void layer_norm_join(float& mean, float& squares, int mine, int H, float (*part)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(0xFFFFFFFFu, squares, o);
  if constexpr (BLOCK) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
      part[0][threadIdx.x >> 5] = mean;
      part[1][threadIdx.x >> 5] = squares;
      part[2][threadIdx.x >> 5] = static_cast<float>(mine);
    }
    __syncthreads();
    const float m = lane < warps ? part[0][lane] : 0.0f, n = lane < warps ? part[2][lane] : 0.0f;
    mean = m * n;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mean += __shfl_xor_sync(0xFFFFFFFFu, mean, o);
    mean /= static_cast<float>(H);
    const float d = m - mean;
    squares = lane < warps ? fmaf(n * d, d, part[1][lane]) : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(0xFFFFFFFFu, squares, o);
  }
}

// PER packs of N elements in each thread of a warp (BLOCK false: a row for each warp) or of the block.
template <typename E, int N, int PER, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? layer_norm_most_threads(N, PER) : 128) layer_norm_kernel(const __grid_constant__ LayerNormArgs A) {
  __shared__ float part[3][32];
  grid_dep_wait();
  grid_dep_launch();
  const int threads = BLOCK ? blockDim.x : 32, me = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int64_t t = BLOCK ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (!BLOCK && t >= A.T) return;
  using P = Pack<E, N>;
  const P* x = reinterpret_cast<const P*>(static_cast<const E*>(A.x) + t * A.ldx);
  const P* r = reinterpret_cast<const P*>(static_cast<const E*>(A.residual) + t * A.ldr);
  const P *w = static_cast<const P*>(A.weight), *b = static_cast<const P*>(A.bias);
  P* ro = reinterpret_cast<P*>(static_cast<E*>(A.residual_out) + t * A.ldro);
  P* y = reinterpret_cast<P*>(static_cast<E*>(A.y) + t * A.ldy);
  const int packs = A.H / N;
  auto at = [&](int i) { return i * threads + me; };
  P px[PER], pr[PER], pw[PER], pb[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (at(i) < packs) {
      px[i] = x[at(i)];
      if (A.residual != nullptr) pr[i] = r[at(i)];
    }
  }
  // few rows ask for the weight at once; many find it in the caches when they need it, and their registers hold more rows on an SM
  constexpr bool EARLY = PER == 1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (EARLY && at(i) < packs && A.y != nullptr) {
      pw[i] = w[at(i)];
      if (A.bias != nullptr) pb[i] = b[at(i)];
    }
  }
  float h[PER][N] = {}, s = 0.0f;
  int mine = 0;  // elements of this warp
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    mine += max(0, min(32, packs - (at(i) - (me & 31)))) * N;
    if (at(i) >= packs) continue;
    unpack(px[i], h[i]);
    if (A.residual != nullptr) {
      float f[N];
      unpack(pr[i], f);
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] += f[e];
      if (A.residual_out != nullptr) ro[at(i)] = pack<E>(h[i]);
    } else if (A.residual_out != nullptr) {
      ro[at(i)] = px[i];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) s += h[i][e];
  }
  float mean = layer_norm_mean<BLOCK>(s, mine), ss = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (at(i) >= packs) continue;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = h[i][e] - mean;
      ss = fmaf(d, d, ss);
    }
  }
  layer_norm_join<BLOCK>(mean, ss, mine, A.H, part);
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(A.H) + A.eps);
  if (me == 0) {
    if (A.mean != nullptr) A.mean[t] = mean;
    if (A.rstd != nullptr) A.rstd[t] = rstd;
  }
  if (A.y == nullptr) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (at(i) >= packs) continue;
    float f[N], c[N] = {};
    unpack(EARLY ? pw[i] : w[at(i)], f);
    if (A.bias != nullptr) unpack(EARLY ? pb[i] : b[at(i)], c);
#pragma unroll
    for (int e = 0; e < N; ++e) h[i][e] = fmaf((h[i][e] - mean) * rstd, f[e], c[e]);
    y[at(i)] = pack<E>(h[i]);
  }
}

// Rows too wide for a block's registers: read again for each step, the second and third time from L2.
template <typename E>
__global__ void __launch_bounds__(1024) layer_norm_wide_kernel(const __grid_constant__ LayerNormArgs A) {
  __shared__ float part[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const E* x = static_cast<const E*>(A.x) + t * A.ldx;
  const E* r = A.residual != nullptr ? static_cast<const E*>(A.residual) + t * A.ldr : nullptr;
  auto at = [&](int j) { return to_f32(x[j]) + (r != nullptr ? to_f32(r[j]) : 0.0f); };
  float s = 0.0f, ss = 0.0f;
  for (int j = threadIdx.x; j < A.H; j += 1024) s += at(j);
  const float mean = norm_join<false, true>(s, part[0]) / static_cast<float>(A.H);
  for (int j = threadIdx.x; j < A.H; j += 1024) {
    const float d = at(j) - mean;
    ss = fmaf(d, d, ss);
  }
  const float rstd = 1.0f / sqrtf(norm_join<false, true>(ss, part[1]) / static_cast<float>(A.H) + A.eps);
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[t] = mean;
    if (A.rstd != nullptr) A.rstd[t] = rstd;
  }
  for (int j = threadIdx.x; j < A.H; j += 1024) {
    const float h = at(j);
    if (A.y != nullptr) {
      const float w = to_f32(static_cast<const E*>(A.weight)[j]), b = A.bias != nullptr ? to_f32(static_cast<const E*>(A.bias)[j]) : 0.0f;
      from_f32(fmaf((h - mean) * rstd, w, b), static_cast<E*>(A.y) + t * A.ldy + j);
    }
    if (A.residual_out != nullptr) from_f32(h, static_cast<E*>(A.residual_out) + t * A.ldro + j);
  }
}

// ------------------------------------------------------------------------------ the way back
struct LayerNormGradArgs {
  const void *dy, *x, *weight, *dresidual;
  const float *mean, *rstd;
  void *dx, *dweight, *dbias;
  float* part;  // [groups][2][H]: sums of dy v and of dy over a group of rows
  uint32_t* errors;
  int64_t lddy, ldx, lddr, lddx;
  int T, H, groups, depth;  // depth: rows on their way at a time (layer_norm_ring_kernel)
};

// Joins two sums over the threads of a row.  `part` holds two floats for each warp; rows take turns with two of them, so
// that one barrier a row is enough.
template <bool BLOCK>
__device__ __forceinline__ void layer_norm_join2(float& a, float& b, float2* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if constexpr (BLOCK) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    const float2 v = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
    a = v.x;
    b = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
  }
}

constexpr int LAYER_NORM_GRAD_THREADS = 512, LAYER_NORM_GRAD_WARPS = 8;
__host__ __device__ constexpr int layer_norm_grad_most_threads(int n, int per) { return n * per > 8 ? LAYER_NORM_GRAD_THREADS : 704; }  // by registers

// Rows b, b + groups, ... of a block (BLOCK), or of its warps one after another (eight rows of it at a time): a
// thread has the same columns of all of them, so the sums over rows stay in its registers, in 32 bits.  The
// next row is on its way while this one's sums are joined.
template <typename E, int N, int PER, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? layer_norm_grad_most_threads(N, PER) : 32 * LAYER_NORM_GRAD_WARPS) layer_norm_grad_kernel(const __grid_constant__ LayerNormGradArgs A) {
  __shared__ float2 part[2][32];
  extern __shared__ float sums[];  // warps alone: [2][H]
  grid_dep_wait();
  grid_dep_launch();
  using P = Pack<E, N>;
  const int threads = BLOCK ? blockDim.x : 32, me = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int packs = A.H / N, warp = threadIdx.x >> 5;
  const int first = BLOCK ? blockIdx.x : blockIdx.x * LAYER_NORM_GRAD_WARPS + warp, step = BLOCK ? gridDim.x : gridDim.x * LAYER_NORM_GRAD_WARPS;
  auto at = [&](int i) { return i * threads + me; };
  auto row = [&](const void* p, int64_t ld, int64_t t) { return reinterpret_cast<const P*>(static_cast<const E*>(p) + t * ld); };
  P pdy[PER], px[PER], pdr[PER];
  float dw[PER][N] = {}, db[PER][N] = {}, mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= packs) continue;
      pdy[i] = row(A.dy, A.lddy, t)[at(i)];
      px[i] = row(A.x, A.ldx, t)[at(i)];
      if (A.dresidual != nullptr) pdr[i] = row(A.dresidual, A.lddr, t)[at(i)];
    }
    mean = A.mean[t];
    rstd = A.rstd[t];
  };
  if (first < A.T) load(first);
  int turn = 0;
  for (int64_t t = first; t < A.T; t += step, turn ^= 1) {
    float a[PER][N], v[PER][N], sa = 0.0f, sav = 0.0f;
    P dr[PER];
    const float scale = rstd;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= packs) continue;
      float w[N];
      unpack(static_cast<const P*>(A.weight)[at(i)], w);  // from the nearest cache, for the registers' sake
      unpack(pdy[i], a[i]);
      unpack(px[i], v[i]);
      dr[i] = pdr[i];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[i][e] = (v[i][e] - mean) * rstd;
        dw[i][e] = fmaf(a[i][e], v[i][e], dw[i][e]);
        db[i][e] += a[i][e];
        a[i][e] *= w[e];
        sa += a[i][e];
        sav = fmaf(a[i][e], v[i][e], sav);
      }
    }
    if (t + step < A.T) load(t + step);
    layer_norm_join2<BLOCK>(sa, sav, part[turn]);
    sa /= static_cast<float>(A.H);
    sav /= static_cast<float>(A.H);
    if (A.dx == nullptr) continue;
    P* dx = reinterpret_cast<P*>(static_cast<E*>(A.dx) + t * A.lddx);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= packs) continue;
      float c[N] = {};
      if (A.dresidual != nullptr) unpack(dr[i], c);
#pragma unroll
      for (int e = 0; e < N; ++e) c[e] = fmaf(scale, a[i][e] - sa - v[i][e] * sav, c[e]);
      dx[at(i)] = pack<E>(c);
    }
  }
  if (A.part == nullptr) return;
  float* out = A.part + static_cast<int64_t>(blockIdx.x) * 2 * A.H;
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= packs) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        out[at(i) * N + e] = dw[i][e];
        out[A.H + at(i) * N + e] = db[i][e];
      }
    }
  } else {  // one warp after another: always the same order
    for (int turn = 0; turn < LAYER_NORM_GRAD_WARPS; ++turn) {
      if (warp == turn) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (at(i) >= packs) continue;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int c = at(i) * N + e;
            sums[c] = (turn > 0 ? sums[c] : 0.0f) + dw[i][e];
            sums[A.H + c] = (turn > 0 ? sums[A.H + c] : 0.0f) + db[i][e];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * A.H; c += blockDim.x) out[c] = sums[c];
  }
}

// Rows on 16 bytes, too wide for a warp: as above, by a block, but the rows to come are on their way to shared memory, as bulk
// copies, `depth` of them ahead.  A row's copies start when every thread has read the one that had its place, which the
// join's barrier tells.
constexpr int LAYER_NORM_RING = 16;
constexpr uint32_t LAYER_NORM_SPINS = 1u << 22;
template <typename E, int PER>
__global__ void __launch_bounds__(LAYER_NORM_GRAD_THREADS) layer_norm_ring_kernel(const __grid_constant__ LayerNormGradArgs A) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  __shared__ float2 part[2][32];
  __shared__ uint64_t full[LAYER_NORM_RING];
  extern __shared__ __align__(16) uint8_t rows[];  // [depth][dy, x, dresidual][H]
  using P = Pack<E, N>;
  const int packs = A.H / N, me = threadIdx.x, threads = blockDim.x, step = gridDim.x;
  const uint32_t bytes = static_cast<uint32_t>(A.H) * sizeof(E), tensors = A.dresidual != nullptr ? 3 : 2;
  if (me == 0) {
    for (int i = 0; i < A.depth; ++i) mbar_init(&full[i], 1);
    fence_proxy_async_smem();
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  auto fetch = [&](int64_t t, int slot) {
    uint8_t* to = rows + static_cast<size_t>(slot) * tensors * bytes;
    mbar_arrive_expect_tx(&full[slot], tensors * bytes);
    bulk_g2s(to, static_cast<const E*>(A.dy) + t * A.lddy, bytes, &full[slot]);
    bulk_g2s(to + bytes, static_cast<const E*>(A.x) + t * A.ldx, bytes, &full[slot]);
    if (A.dresidual != nullptr) bulk_g2s(to + 2 * bytes, static_cast<const E*>(A.dresidual) + t * A.lddr, bytes, &full[slot]);
  };
  if (me == 0)
    for (int i = 0; i < A.depth && blockIdx.x + static_cast<int64_t>(i) * step < A.T; ++i) fetch(blockIdx.x + static_cast<int64_t>(i) * step, i);
  auto at = [&](int i) { return i * threads + me; };
  P pw[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (at(i) < packs) pw[i] = static_cast<const P*>(A.weight)[at(i)];
  float dw[PER][N] = {}, db[PER][N] = {};
  int slot = 0, turn = 0;
  uint32_t phase = 0;
  float mean = blockIdx.x < A.T ? A.mean[blockIdx.x] : 0.0f, rstd = blockIdx.x < A.T ? A.rstd[blockIdx.x] : 0.0f;
  for (int64_t t = blockIdx.x; t < A.T; t += step, turn ^= 1) {
    // copies that do not arrive leave the results without meaning; all waits end, and so does the kernel
    uint32_t spin = 0;
    while (!mbar_try_wait(&full[slot], phase) && ++spin < LAYER_NORM_SPINS) {
    }
    if (spin >= LAYER_NORM_SPINS) atomicOr(A.errors, 0x08u);  // STRATA_DEVERR_TIMEOUT
    const P* in = reinterpret_cast<const P*>(rows + static_cast<size_t>(slot) * tensors * bytes);
    float a[PER][N], v[PER][N], sa = 0.0f, sav = 0.0f;
    P dr[PER];
    const float scale = rstd;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= packs) continue;
      float w[N];
      unpack(pw[i], w);
      unpack(in[at(i)], a[i]);
      unpack(in[packs + at(i)], v[i]);
      if (A.dresidual != nullptr) dr[i] = in[2 * packs + at(i)];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[i][e] = (v[i][e] - mean) * rstd;
        dw[i][e] = fmaf(a[i][e], v[i][e], dw[i][e]);
        db[i][e] += a[i][e];
        a[i][e] *= w[e];
        sa += a[i][e];
        sav = fmaf(a[i][e], v[i][e], sav);
      }
    }
    if (t + step < A.T) {
      mean = A.mean[t + step];
      rstd = A.rstd[t + step];
    }
    layer_norm_join2<true>(sa, sav, part[turn]);
    if (me == 0 && t + static_cast<int64_t>(A.depth) * step < A.T) fetch(t + static_cast<int64_t>(A.depth) * step, slot);
    if (++slot == A.depth) {
      slot = 0;
      phase ^= 1u;
    }
    if (A.dx == nullptr) continue;
    sa /= static_cast<float>(A.H);
    sav /= static_cast<float>(A.H);
    P* dx = reinterpret_cast<P*>(static_cast<E*>(A.dx) + t * A.lddx);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= packs) continue;
      float c[N] = {};
      if (A.dresidual != nullptr) unpack(dr[i], c);
#pragma unroll
      for (int e = 0; e < N; ++e) c[e] = fmaf(scale, a[i][e] - sa - v[i][e] * sav, c[e]);
      dx[at(i)] = pack<E>(c);
    }
  }
  if (A.part == nullptr) return;
  float* out = A.part + static_cast<int64_t>(blockIdx.x) * 2 * A.H;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (at(i) >= packs) continue;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      out[at(i) * N + e] = dw[i][e];
      out[A.H + at(i) * N + e] = db[i][e];
    }
  }
}

// Rows too wide for that: dx by a block for each row, which reads it twice, ...
template <typename E>
__global__ void __launch_bounds__(1024) layer_norm_grad_wide_kernel(const __grid_constant__ LayerNormGradArgs A) {
  __shared__ float2 part[32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const E *dy = static_cast<const E*>(A.dy) + t * A.lddy, *x = static_cast<const E*>(A.x) + t * A.ldx, *w = static_cast<const E*>(A.weight);
  const E* dr = A.dresidual != nullptr ? static_cast<const E*>(A.dresidual) + t * A.lddr : nullptr;
  const float mean = A.mean[t], rstd = A.rstd[t];
  float sa = 0.0f, sav = 0.0f;
  for (int j = threadIdx.x; j < A.H; j += 1024) {
    const float a = to_f32(dy[j]) * to_f32(w[j]);
    sa += a;
    sav = fmaf(a, (to_f32(x[j]) - mean) * rstd, sav);
  }
  layer_norm_join2<true>(sa, sav, part);
  sa /= static_cast<float>(A.H);
  sav /= static_cast<float>(A.H);
  for (int j = threadIdx.x; j < A.H; j += 1024) {
    const float a = to_f32(dy[j]) * to_f32(w[j]), v = (to_f32(x[j]) - mean) * rstd;
    from_f32(fmaf(rstd, a - sa - v * sav, dr != nullptr ? to_f32(dr[j]) : 0.0f), static_cast<E*>(A.dx) + t * A.lddx + j);
  }
}
// ... and the sums over rows by a thread for each column and group of rows.
template <typename E>
__global__ void __launch_bounds__(256) layer_norm_grad_columns_kernel(const __grid_constant__ LayerNormGradArgs A) {
  grid_dep_wait();
  grid_dep_launch();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= A.H) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t t = blockIdx.y; t < A.T; t += A.groups) {
    const float d = to_f32(static_cast<const E*>(A.dy)[t * A.lddy + c]);
    dw = fmaf(d, (to_f32(static_cast<const E*>(A.x)[t * A.ldx + c]) - A.mean[t]) * A.rstd[t], dw);
    db += d;
  }
  float* out = A.part + static_cast<int64_t>(blockIdx.y) * 2 * A.H;
  out[c] = dw;
  out[A.H + c] = db;
}

// The groups' sums of 32 columns: 32 warps take every 32nd group, and are added up in order.
template <typename E>
__global__ void __launch_bounds__(1024) layer_norm_sum_kernel(const __grid_constant__ LayerNormGradArgs A) {
  __shared__ float2 of[32][33];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  float dw = 0.0f, db = 0.0f;
  if (c < A.H) {
#pragma unroll 4
    for (int g = warp; g < A.groups; g += 32) {
      dw += A.part[static_cast<int64_t>(g) * 2 * A.H + c];
      db += A.part[static_cast<int64_t>(g) * 2 * A.H + A.H + c];
    }
  }
  of[warp][lane] = make_float2(dw, db);
  __syncthreads();
  const float2 v = of[lane][warp];  // warp w: column w, a lane for each of the 32
  dw = v.x;
  db = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    dw += __shfl_xor_sync(0xFFFFFFFFu, dw, o);
    db += __shfl_xor_sync(0xFFFFFFFFu, db, o);
  }
  const int column = blockIdx.x * 32 + warp;
  if (lane > 0 || column >= A.H) return;
  if (A.dweight != nullptr) from_f32(dw, static_cast<E*>(A.dweight) + column);
  if (A.dbias != nullptr) from_f32(db, static_cast<E*>(A.dbias) + column);
}

}  // namespace strata
