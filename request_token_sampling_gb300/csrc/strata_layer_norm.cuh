// strata_layer_norm.cuh -- layer norm of rows, with the residual's addition, and its way back.
//
//   h = x + residual;  v = (h - mean(h)) rstd, rstd = 1 / sqrt(mean((h - mean)^2) + eps);  y = v weight + bias
//   a = dy weight;  dx = rstd (a - mean(a) - v mean(a v)) + dresidual;  dweight = sum_t dy v;  dbias = sum_t dy
//
// Bound by HBM: every element is read and written once.  A row stays in registers between its joins, so the variance
// is a second sum over differences from the mean, not a difference of large sums.  Measured (one GB300, us in a stream of
// calls): 8192 x 8192 bfloat16 with residual 81 (6.6 TB/s), back 97 (88 and the second kernel); 8192 x 5003, whose rows start
// anywhere, 62 and 97; 1021 x 5003 float32 15 and 22; 8192 x 1135 25 and 31.  A row's chain through a block (two
// joins of shuffles, a barrier) takes 1.6 us, so narrow rows want several blocks to an SM.
#pragma once

#include "strata_norm.cuh"

namespace strata {

// How a row that starts anywhere is cut: packs of N elements on the 16-byte boundaries, and up to 2 (N - 1) elements before the
// first and behind the last, which go one to a thread (`edge`: this one's column, or -1).  SHIFT false: it starts on 16 bytes
// and ends with a pack.  Rows that are a multiple of eight apart are cut alike, so that a thread that goes through such
// rows keeps its columns.
template <typename E, int N, bool SHIFT>
struct RowCut {
  int head = 0, packs, edge = -1, edges = 0;
  __device__ __forceinline__ RowCut(const E* row, int H, int me) {
    if constexpr (SHIFT) {
      head = min(H, static_cast<int>(-(reinterpret_cast<uintptr_t>(row) / sizeof(E)) & (N - 1)));
      packs = (H - head) / N;
      edges = H - packs * N;
      if (me < edges) edge = me < head ? me : packs * N + me;
    } else {
      packs = H / N;
    }
  }
};
// The weight, or the bias, of a pack's columns.
template <typename E, int N, bool SHIFT>
__device__ __forceinline__ Pack<E, N> column_pack(const E* w, int column) {
  Pack<E, N> p;
  if constexpr (SHIFT) {
#pragma unroll
    for (int e = 0; e < N; ++e) p.v[e] = w[column + e];
  } else {
    p = *reinterpret_cast<const Pack<E, N>*>(w + column);
  }
  return p;
}

struct LayerNormArgs {
  const void *x, *residual, *weight, *bias;
  void *residual_out, *y;
  float *mean, *rstd;
  int64_t ldx, ldr, ldro, ldy;
  uint32_t* errors;
  int T, H;
  float eps;
  int depth;  // rows on their way at a time (layer_norm_ring_kernel)
};

__host__ __device__ constexpr int layer_norm_most_threads(int n, int per) { return n * per > 8 ? 512 : 1024; }  // by registers

// The joins of a row's sum and of its squared differences.  Each warp takes both about its own mean, by shuffles, and the
// warps' come together behind one barrier: the squares about the row's mean are the warps' and, for each warp, its elements times
// the square of what the means differ by.  `mine`: this warp's elements.
__device__ __forceinline__ float layer_norm_mean(float& sum, int mine) {
  sum = warp_sum(sum);
  return mine > 0 ? sum / static_cast<float>(mine) : 0.0f;
}
template <bool BLOCK>
__device__ __forceinline__ void layer_norm_join(float& mean, float& squares, float sum, int mine, int H, float (*part)[32]) {
  squares = warp_sum(squares);
  if constexpr (BLOCK) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
      part[0][threadIdx.x >> 5] = sum;
      part[1][threadIdx.x >> 5] = squares;
      part[2][threadIdx.x >> 5] = static_cast<float>(mine);
    }
    __syncthreads();
    const float s = lane < warps ? part[0][lane] : 0.0f, n = lane < warps ? part[2][lane] : 0.0f;
    mean = warp_sum(s) / static_cast<float>(H);
    const float d = n > 0.0f ? s / n - mean : 0.0f;
    squares = warp_sum(lane < warps ? fmaf(n * d, d, part[1][lane]) : 0.0f);
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
  float mean = layer_norm_mean(s, mine), ss = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (at(i) >= packs) continue;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = h[i][e] - mean;
      ss = fmaf(d, d, ss);
    }
  }
  layer_norm_join<BLOCK>(mean, ss, s, mine, A.H, part);
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

// Rows that come as bulk copies into a ring of shared memory, `depth` of them (two at least).  A row's place is free when all
// threads are past the next row's join; a warp that has nothing else to do starts the copies (thread 0 of the others took
// 0.3 us a row for it).  Each row's packs alone are copied: what lies before and behind them is read by the threads that
// have it.
constexpr int LAYER_NORM_RING = 16, LAYER_NORM_RING_THREADS = 512;  // and a warp that starts the copies
constexpr uint32_t LAYER_NORM_SPINS = 1u << 22;
template <typename E, int TENSORS>
struct RowRing {
  uint64_t* full;
  uint8_t* rows;
  const E* from[TENSORS];
  int64_t ld[TENSORS];
  uint32_t bytes, place;  // of a row's packs; of a row in the ring
  int tensors, depth, slot = 0, before = -1;
  uint32_t phase = 0;
  __device__ __forceinline__ void fetch(int64_t t, int to) {
    mbar_arrive_expect_tx(&full[to], static_cast<uint32_t>(tensors) * bytes);
#pragma unroll
    for (int i = 0; i < TENSORS; ++i)
      if (i < tensors) bulk_g2s(rows + (static_cast<size_t>(to) * tensors + i) * place, from[i] + t * ld[i], bytes, &full[to]);
  }
  __device__ __forceinline__ void start(int64_t first, int64_t step, int64_t T) {
    for (int i = 0; i < depth && first + i * step < T; ++i) fetch(first + i * step, i);
  }
  // Behind the join of row `t`: the place of the row before it is free.
  __device__ __forceinline__ void refill(int64_t t, int64_t step, int64_t T) {
    if (before >= 0 && t + (depth - 1) * step < T) fetch(t + (depth - 1) * step, before);
  }
  // Copies that do not arrive leave the results without meaning; all waits end, and so does the kernel.
  __device__ __forceinline__ void wait(uint32_t* errors) {
    uint32_t spin = 0;
    while (!mbar_try_wait(&full[slot], phase) && ++spin < LAYER_NORM_SPINS) {
    }
    if (spin >= LAYER_NORM_SPINS) atomicOr(errors, 0x08u);  // STRATA_DEVERR_TIMEOUT
  }
  template <int N>
  __device__ __forceinline__ const Pack<E, N>& pack_of(int i, int at) const {
    return reinterpret_cast<const Pack<E, N>*>(rows + (static_cast<size_t>(slot) * tensors + i) * place)[at];
  }
  __device__ __forceinline__ void next() {
    before = slot;
    if (++slot == depth) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// Many rows that start anywhere: a block goes through rows that are cut alike, the weight's packs beside the ring.  (Rows that all
// start on 16 bytes are faster a block each: 8192 x 8192 bfloat16 81 us against 85, 8192 x 2048 24 against 26; of those that do
// not, 8192 x 5003 takes 62 here, element by element 160, 8192 x 1135 25 and 27.)
template <typename E, int PER>
__global__ void __launch_bounds__(LAYER_NORM_RING_THREADS + 32, 1) layer_norm_ring_kernel(const __grid_constant__ LayerNormArgs A) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  __shared__ float part[2][3][32];
  __shared__ uint64_t full[LAYER_NORM_RING];
  extern __shared__ __align__(16) uint8_t ring_rows[];  // [depth][x, residual][H], weight, bias
  using P = Pack<E, N>;
  const int me = threadIdx.x, threads = blockDim.x - 32, step = gridDim.x;
  const int64_t first = blockIdx.x;
  if (me == 0) {
    for (int i = 0; i < A.depth; ++i) mbar_init(&full[i], 1);
    fence_proxy_async_smem();
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  const E *x = static_cast<const E*>(A.x), *r = static_cast<const E*>(A.residual), *w = static_cast<const E*>(A.weight), *b = static_cast<const E*>(A.bias);
  const RowCut<E, N, true> cut(x + first * A.ldx, A.H, me);
  const uint32_t place = (static_cast<uint32_t>(A.H) * static_cast<uint32_t>(sizeof(E)) + 15) / 16 * 16;
  RowRing<E, 2> ring{full, ring_rows, {x + cut.head, r + cut.head}, {A.ldx, A.ldr}, static_cast<uint32_t>(cut.packs) * 16, place, r != nullptr ? 2 : 1, A.depth};
  if (me >= threads) {
    if (me == threads) ring.start(first, step, A.T);
    for (int64_t t = first, turn = 0; t < A.T; t += step, turn ^= 1) {
      float none = 0.0f, nothing = 0.0f;
      layer_norm_join<true>(none, nothing, 0.0f, 0, A.H, part[turn]);
      if (me == threads) ring.refill(t, step, A.T);
      ring.next();
    }
    return;
  }
  P* sw = reinterpret_cast<P*>(ring_rows + static_cast<size_t>(A.depth) * ring.tensors * place);
  P* sb = reinterpret_cast<P*>(reinterpret_cast<uint8_t*>(sw) + place);
  auto at = [&](int i) { return i * threads + me; };  // the pack, of column head + N at(i)
  int mine = me < 32 ? cut.edges : 0;  // elements of this warp
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    mine += max(0, min(32, cut.packs - (i * threads + (me & ~31)))) * N;
    if (at(i) >= cut.packs) continue;
    sw[at(i)] = column_pack<E, N, true>(w, cut.head + at(i) * N);  // read by this thread alone
    if (A.bias != nullptr) sb[at(i)] = column_pack<E, N, true>(b, cut.head + at(i) * N);
  }
  float xe = 0.0f, re = 0.0f, we = 0.0f, be = 0.0f;
  auto load_edge = [&](int64_t t) {
    if (cut.edge >= 0) {
      xe = to_f32(x[t * A.ldx + cut.edge]);
      if (r != nullptr) re = to_f32(r[t * A.ldr + cut.edge]);
    }
  };
  load_edge(first);
  if (cut.edge >= 0) {
    we = to_f32(w[cut.edge]);
    if (A.bias != nullptr) be = to_f32(b[cut.edge]);
  }
  const float over = 1.0f / static_cast<float>(A.H);
  int turn = 0;
  for (int64_t t = first; t < A.T; t += step, turn ^= 1) {
    E *ro = static_cast<E*>(A.residual_out) + t * A.ldro, *y = static_cast<E*>(A.y) + t * A.ldy;
    float h[PER][N] = {}, s = 0.0f;
    const float he = xe + re;
    ring.wait(A.errors);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= cut.packs) continue;
      unpack(ring.template pack_of<N>(0, at(i)), h[i]);
      if (r != nullptr) {
        float f[N];
        unpack(ring.template pack_of<N>(1, at(i)), f);
#pragma unroll
        for (int e = 0; e < N; ++e) h[i][e] += f[e];
      }
      if (A.residual_out != nullptr) *reinterpret_cast<P*>(ro + cut.head + at(i) * N) = pack<E>(h[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) s += h[i][e];
    }
    if (cut.edge >= 0) {
      s += he;
      if (A.residual_out != nullptr) from_f32(he, ro + cut.edge);
    }
    if (t + step < A.T) load_edge(t + step);
    float mean = layer_norm_mean(s, mine), ss = cut.edge >= 0 ? (he - mean) * (he - mean) : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= cut.packs) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = h[i][e] - mean;
        ss = fmaf(d, d, ss);
      }
    }
    layer_norm_join<true>(mean, ss, s, mine, A.H, part[turn]);
    ring.next();
    const float rstd = rsqrtf(fmaf(ss, over, A.eps));
    if (me == 0) {
      if (A.mean != nullptr) A.mean[t] = mean;
      if (A.rstd != nullptr) A.rstd[t] = rstd;
    }
    if (A.y == nullptr) continue;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= cut.packs) continue;
      float f[N], c[N] = {};
      unpack(sw[at(i)], f);
      if (A.bias != nullptr) unpack(sb[at(i)], c);
#pragma unroll
      for (int e = 0; e < N; ++e) c[e] = fmaf((h[i][e] - mean) * rstd, f[e], c[e]);
      *reinterpret_cast<P*>(y + cut.head + at(i) * N) = pack<E>(c);
    }
    if (cut.edge >= 0) from_f32(fmaf((he - mean) * rstd, we, be), y + cut.edge);
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
template <typename E, int N, int PER, bool BLOCK, bool SHIFT>
__global__ void __launch_bounds__(BLOCK ? layer_norm_grad_most_threads(N, PER) : 32 * LAYER_NORM_GRAD_WARPS, BLOCK ? 1 : 2) layer_norm_grad_kernel(const __grid_constant__ LayerNormGradArgs A) {
  __shared__ float2 part[2][32];
  extern __shared__ float sums[];  // warps alone: [2][H to whole packs]
  grid_dep_wait();
  grid_dep_launch();
  using P = Pack<E, N>;
  const int threads = BLOCK ? blockDim.x : 32, me = BLOCK ? threadIdx.x : threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = BLOCK ? blockIdx.x : blockIdx.x * LAYER_NORM_GRAD_WARPS + warp, step = BLOCK ? gridDim.x : gridDim.x * LAYER_NORM_GRAD_WARPS;
  auto row = [&](const void* p, int64_t ld, int64_t t) { return static_cast<const E*>(p) + t * ld; };
  const RowCut<E, N, SHIFT> cut(row(A.x, A.ldx, first), A.H, me);
  auto has = [&](int i) { return i * threads + me < cut.packs; };
  auto at = [&](int i) { return cut.head + (i * threads + me) * N; };
  P pdy[PER], px[PER], pdr[PER];
  float dw[PER][N] = {}, db[PER][N] = {}, mean = 0.0f, rstd = 0.0f;
  float dye = 0.0f, xe = 0.0f, dre = 0.0f, dwe = 0.0f, dbe = 0.0f;
  const float we = SHIFT && cut.edge >= 0 ? to_f32(static_cast<const E*>(A.weight)[cut.edge]) : 0.0f;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!has(i)) continue;
      pdy[i] = *reinterpret_cast<const P*>(row(A.dy, A.lddy, t) + at(i));
      px[i] = *reinterpret_cast<const P*>(row(A.x, A.ldx, t) + at(i));
      if (A.dresidual != nullptr) pdr[i] = *reinterpret_cast<const P*>(row(A.dresidual, A.lddr, t) + at(i));
    }
    if (SHIFT && cut.edge >= 0) {
      dye = to_f32(row(A.dy, A.lddy, t)[cut.edge]);
      xe = to_f32(row(A.x, A.ldx, t)[cut.edge]);
      if (A.dresidual != nullptr) dre = to_f32(row(A.dresidual, A.lddr, t)[cut.edge]);
    }
    mean = A.mean[t];
    rstd = A.rstd[t];
  };
  if (first < A.T) load(first);
  int turn = 0;
  for (int64_t t = first; t < A.T; t += step, turn ^= 1) {
    float a[PER][N], v[PER][N], sa = 0.0f, sav = 0.0f;
    P dr[PER];
    const float scale = rstd, ce = dre;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!has(i)) continue;
      float w[N];
      unpack(column_pack<E, N, SHIFT>(static_cast<const E*>(A.weight), at(i)), w);  // from the nearest cache, for the registers' sake
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
    const float ve = (xe - mean) * rstd, ae = dye * we;
    if (SHIFT && cut.edge >= 0) {
      dwe = fmaf(dye, ve, dwe);
      dbe += dye;
      sa += ae;
      sav = fmaf(ae, ve, sav);
    }
    if (t + step < A.T) load(t + step);
    layer_norm_join2<BLOCK>(sa, sav, part[turn]);
    sa /= static_cast<float>(A.H);
    sav /= static_cast<float>(A.H);
    if (A.dx == nullptr) continue;
    E* dx = static_cast<E*>(A.dx) + t * A.lddx;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!has(i)) continue;
      float c[N] = {};
      if (A.dresidual != nullptr) unpack(dr[i], c);
#pragma unroll
      for (int e = 0; e < N; ++e) c[e] = fmaf(scale, a[i][e] - sa - v[i][e] * sav, c[e]);
      *reinterpret_cast<P*>(dx + at(i)) = pack<E>(c);
    }
    if (SHIFT && cut.edge >= 0) from_f32(fmaf(scale, ae - sa - ve * sav, ce), dx + cut.edge);
  }
  if (A.part == nullptr) return;
  float* out = A.part + static_cast<int64_t>(blockIdx.x) * 2 * A.H;
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!has(i)) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        out[at(i) + e] = dw[i][e];
        out[A.H + at(i) + e] = db[i][e];
      }
    }
  } else {  // one warp after another: always the same order; columns of neighbouring lanes lie beside one another
    const int eighth = (A.H + N - 1) / N, half = N * eighth;
    auto spread = [&](int c) { return c % N * eighth + c / N; };
    for (int turn = 0; turn < LAYER_NORM_GRAD_WARPS; ++turn) {
      if (warp == turn) {
        auto add = [&](int c, float w, float b) {
          sums[spread(c)] = (turn > 0 ? sums[spread(c)] : 0.0f) + w;
          sums[half + spread(c)] = (turn > 0 ? sums[half + spread(c)] : 0.0f) + b;
        };
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (!has(i)) continue;
#pragma unroll
          for (int e = 0; e < N; ++e) add(at(i) + e, dw[i][e], db[i][e]);
        }
        if (SHIFT && cut.edge >= 0) add(cut.edge, dwe, dbe);
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < A.H; c += blockDim.x) {
      out[c] = sums[spread(c)];
      out[A.H + c] = sums[half + spread(c)];
    }
  }
}

// Wider rows: as above, by a block, through a ring.  Threads with 16 elements need the registers that a further warp would
// take: there thread 0 starts the copies.
__host__ __device__ constexpr int layer_norm_grad_ring_threads(int n, int per) { return n * per > 8 ? 512 : 704; }
__host__ __device__ constexpr int layer_norm_copier(int n, int per) { return n * per > 8 ? 0 : 32; }
template <typename E, int PER, bool SHIFT>
__global__ void __launch_bounds__(layer_norm_grad_ring_threads(16 / static_cast<int>(sizeof(E)), PER) + layer_norm_copier(16 / static_cast<int>(sizeof(E)), PER), 1) layer_norm_grad_ring_kernel(const __grid_constant__ LayerNormGradArgs A) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  __shared__ float2 part[2][32];
  __shared__ uint64_t full[LAYER_NORM_RING];
  extern __shared__ __align__(16) uint8_t ring_rows[];  // [depth][dy, x, dresidual][H], weight
  using P = Pack<E, N>;
  constexpr int COPIER = layer_norm_copier(N, PER);
  const int me = threadIdx.x, threads = blockDim.x - COPIER, step = gridDim.x;
  const int64_t first = blockIdx.x;
  if (me == 0) {
    for (int i = 0; i < A.depth; ++i) mbar_init(&full[i], 1);
    fence_proxy_async_smem();
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  const E *dy = static_cast<const E*>(A.dy), *x = static_cast<const E*>(A.x), *r = static_cast<const E*>(A.dresidual), *w = static_cast<const E*>(A.weight);
  const RowCut<E, N, SHIFT> cut(x + first * A.ldx, A.H, me);
  const uint32_t place = (static_cast<uint32_t>(A.H) * static_cast<uint32_t>(sizeof(E)) + 15) / 16 * 16;
  RowRing<E, 3> ring{full, ring_rows, {dy + cut.head, x + cut.head, r + cut.head}, {A.lddy, A.ldx, A.lddr}, static_cast<uint32_t>(cut.packs) * 16, place,
                     r != nullptr ? 3 : 2, A.depth};
  if (COPIER == 0 && me == 0) ring.start(first, step, A.T);
  if (me >= threads) {
    if (me == threads) ring.start(first, step, A.T);
    for (int64_t t = first, turn = 0; t < A.T; t += step, turn ^= 1) {
      float none = 0.0f, nothing = 0.0f;
      layer_norm_join2<true>(none, nothing, part[turn]);
      if (me == threads) ring.refill(t, step, A.T);
      ring.next();
    }
    return;
  }
  P* sw = reinterpret_cast<P*>(ring_rows + static_cast<size_t>(A.depth) * ring.tensors * place);
  auto at = [&](int i) { return i * threads + me; };  // the pack, of column head + N at(i)
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (at(i) < cut.packs) sw[at(i)] = column_pack<E, N, SHIFT>(w, cut.head + at(i) * N);  // read by this thread alone
  float dw[PER][N] = {}, db[PER][N] = {};
  float dye = 0.0f, xe = 0.0f, dre = 0.0f, dwe = 0.0f, dbe = 0.0f;
  const float we = SHIFT && cut.edge >= 0 ? to_f32(w[cut.edge]) : 0.0f, over = 1.0f / static_cast<float>(A.H);
  auto load_edge = [&](int64_t t) {
    if (SHIFT && cut.edge >= 0) {
      dye = to_f32(dy[t * A.lddy + cut.edge]);
      xe = to_f32(x[t * A.ldx + cut.edge]);
      if (r != nullptr) dre = to_f32(r[t * A.lddr + cut.edge]);
    }
  };
  load_edge(first);
  int turn = 0;
  float next_mean = A.mean[first], next_rstd = A.rstd[first];
  for (int64_t t = first; t < A.T; t += step, turn ^= 1) {
    const float mean = next_mean, rstd = next_rstd, ve = (xe - mean) * rstd, ae = dye * we, ce = dre;
    float a[PER][N], v[PER][N], sa = 0.0f, sav = 0.0f;
    ring.wait(A.errors);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= cut.packs) continue;
      float f[N];
      unpack(sw[at(i)], f);
      unpack(ring.template pack_of<N>(0, at(i)), a[i]);
      unpack(ring.template pack_of<N>(1, at(i)), v[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[i][e] = (v[i][e] - mean) * rstd;
        dw[i][e] = fmaf(a[i][e], v[i][e], dw[i][e]);
        db[i][e] += a[i][e];
        a[i][e] *= f[e];
        sa += a[i][e];
        sav = fmaf(a[i][e], v[i][e], sav);
      }
    }
    if (SHIFT && cut.edge >= 0) {
      dwe = fmaf(dye, ve, dwe);
      dbe += dye;
      sa += ae;
      sav = fmaf(ae, ve, sav);
    }
    if (t + step < A.T) {
      next_mean = A.mean[t + step];
      next_rstd = A.rstd[t + step];
      load_edge(t + step);
    }
    layer_norm_join2<true>(sa, sav, part[turn]);
    if (COPIER == 0 && me == 0) ring.refill(t, step, A.T);
    if (A.dx != nullptr) {
      sa *= over;
      sav *= over;
      E* dx = static_cast<E*>(A.dx) + t * A.lddx;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (at(i) >= cut.packs) continue;
        float c[N] = {};
        if (r != nullptr) unpack(ring.template pack_of<N>(2, at(i)), c);
#pragma unroll
        for (int e = 0; e < N; ++e) c[e] = fmaf(rstd, a[i][e] - sa - v[i][e] * sav, c[e]);
        *reinterpret_cast<P*>(dx + cut.head + at(i) * N) = pack<E>(c);
      }
      if (SHIFT && cut.edge >= 0) from_f32(fmaf(rstd, ae - sa - ve * sav, ce), dx + cut.edge);
    }
    ring.next();
  }
  if (A.part == nullptr) return;
  float* out = A.part + static_cast<int64_t>(blockIdx.x) * 2 * A.H;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (at(i) >= cut.packs) continue;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      out[cut.head + at(i) * N + e] = dw[i][e];
      out[A.H + cut.head + at(i) * N + e] = db[i][e];
    }
  }
  if (SHIFT && cut.edge >= 0) {
    out[cut.edge] = dwe;
    out[A.H + cut.edge] = dbe;
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

// The groups' sums of 32 columns, of dweight (blockIdx.y 0) or of dbias: 32 warps take every 32nd group, and are added up in order.
template <typename E>
__global__ void __launch_bounds__(1024) layer_norm_sum_kernel(const __grid_constant__ LayerNormGradArgs A) {
  __shared__ float of[32][33];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  E* to = static_cast<E*>(blockIdx.y == 0 ? A.dweight : A.dbias);
  if (to == nullptr) return;
  float s = 0.0f;
  if (c < A.H) {
    const float* from = A.part + static_cast<int64_t>(blockIdx.y) * A.H + c;
#pragma unroll 8
    for (int g = warp; g < A.groups; g += 32) s += from[static_cast<int64_t>(g) * 2 * A.H];
  }
  of[warp][lane] = s;
  __syncthreads();
  s = warp_sum(of[lane][warp]);  // warp w: column w, a lane for each of the 32
  const int column = blockIdx.x * 32 + warp;
  if (lane == 0 && column < A.H) from_f32(s, to + column);
}

}  // namespace strata
