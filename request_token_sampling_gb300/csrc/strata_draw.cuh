// strata_draw.cuh -- one id per logit row from the caller's random numbers: top_k, min_p, top_p,
// temperature, with no limit on top_k.
//
// Every cut of the chain is a threshold in one order (logit descending, lowest index first), so what
// is left of a row is always {key > K} and, of the entries with key == K, those up to an index I.
// top_k finds K by counts, top_p by weights.  Weights are whole numbers (floor(exp(.) * 2^43)), so a
// sum of them is exact in 64 bits: it does not depend on the order or the split it was made in.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace strata {

struct DrawArgs {
  const void* logits;
  int64_t ld;
  int V;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* ids;
  float* lps;
};

using u64 = unsigned long long;

constexpr int DRAW_THREADS = 1024;
constexpr int DRAW_WARPS = DRAW_THREADS / 32;
constexpr float DRAW_ONE = 0x1p43f;     // V <= 2^19 weights of at most 2^43 sum below 2^63
constexpr uint32_t NO_KEY = 0u;         // NaN and -inf: below every key that can be chosen

__device__ __forceinline__ float draw_f32(float v) { return v; }
__device__ __forceinline__ float draw_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Order-preserving key; -0.0 and +0.0 share one.  -inf maps to 0x007FFFFF, NaN is taken out first.
__device__ __forceinline__ uint32_t draw_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (x == x && k > 0x007FFFFFu) ? k : NO_KEY;
}
__device__ __forceinline__ float draw_val(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// The whole-number weight of an entry `d` = logit - largest logit away from the top, tempered by
// `inv` = 1 / temperature.  d == 0 is the top itself (also where both are +inf, or inv is inf).
__device__ __forceinline__ float draw_dist(uint32_t key, uint32_t top) {
  return key == top ? 0.0f : draw_val(key) - draw_val(top);
}
__device__ __forceinline__ u64 draw_weight(float dt) {
  const float e = expf(dt);
  return e == e ? __float2ull_rz(e * DRAW_ONE) : 0ull;
}
// floor(of * total / 2^24) for of <= 2^24 and total < 2^63
__device__ __forceinline__ u64 draw_share(u64 of, u64 total) {
  return of * (total >> 24) + ((of * (total & 0xFFFFFFu)) >> 24);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

struct DrawShared {
  u64 warp[DRAW_WARPS];
  u64 bins[256];
  u64 found_sum;
  uint32_t found;
};

template <typename E>
struct DrawRow {
  const E* row;
  int V;
  DrawShared* sh;

  __device__ uint32_t key(int i) const { return draw_key(draw_f32(row[i])); }

  // The largest key of the row.
  __device__ uint32_t top() {
    uint32_t k = NO_KEY;
    for (int i = threadIdx.x; i < V; i += DRAW_THREADS) k = max(k, key(i));
    k = __reduce_max_sync(0xFFFFFFFFu, k);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh->warp[threadIdx.x >> 5] = k;
    __syncthreads();
    for (int w = 0; w < DRAW_WARPS; ++w) k = max(k, static_cast<uint32_t>(sh->warp[w]));
    return k;
  }

  template <typename F>
  __device__ u64 total(F f) {
    u64 s = 0;
    for (int i = threadIdx.x; i < V; i += DRAW_THREADS) s += f(i, key(i));
    s = warp_sum(s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh->warp[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0;
    for (int w = 0; w < DRAW_WARPS; ++w) s += sh->warp[w];
    return s;
  }

  // The key K with sum(key > K) < target <= sum(key >= K) of f over the row, for 1 <= target <= the
  // whole sum: eight bits of it at a time.  `above` = sum(key > K).
  template <typename F>
  __device__ uint32_t select(F f, u64 target, u64* above) {
    uint32_t prefix = 0, mask = 0;
    u64 over = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int b = threadIdx.x; b < 256; b += DRAW_THREADS) sh->bins[b] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < V; i += DRAW_THREADS) {
        const uint32_t k = key(i);
        if ((k & mask) != prefix) continue;
        const u64 v = f(i, k);
        if (v) atomicAdd(&sh->bins[(k >> shift) & 255u], v);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        u64 sum = over;
        int b = 255;
        while (b > 0 && sum + sh->bins[b] < target) sum += sh->bins[b--];
        sh->found = static_cast<uint32_t>(b);
        sh->found_sum = sum;
      }
      __syncthreads();
      over = sh->found_sum;
      prefix |= sh->found << shift;
      mask |= 255u << shift;
    }
    *above = over;
    return prefix;
  }

  // The first index whose running sum of f, in index order, exceeds `target` (< the whole sum).
  template <typename F>
  __device__ int locate(F f, u64 target) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = (V + DRAW_WARPS - 1) / DRAW_WARPS;
    const int from = min(V, warp * part), to = min(V, from + part);
    u64 s = 0;
    for (int i = from + lane; i < to; i += 32) s += f(i, key(i));
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) sh->warp[warp] = s;
    __syncthreads();
    u64 before = 0;
    for (int w = 0; w < warp; ++w) before += sh->warp[w];
    if (before <= target && target < before + s) {
      for (int base = from; base < to; base += 32) {
        u64 run = base + lane < to ? f(base + lane, key(base + lane)) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 up = __shfl_up_sync(0xFFFFFFFFu, run, o);
          if (lane >= o) run += up;
        }
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, before + run > target);
        if (over) {
          if (lane == 0) sh->found = static_cast<uint32_t>(base + __ffs(over) - 1);
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, run, 31);
      }
    }
    __syncthreads();
    return static_cast<int>(sh->found);
  }
};

// One block per row; every step reads the row again (the first time from HBM, then from L2).
template <typename E>
__global__ void __launch_bounds__(DRAW_THREADS) draw_kernel(DrawArgs A) {
  __shared__ DrawShared shared;
  const int b = blockIdx.x;
  DrawRow<E> R{static_cast<const E*>(A.logits) + static_cast<int64_t>(b) * A.ld, A.V, &shared};
  const float T = A.temperature != nullptr ? A.temperature[b] : 1.0f;
  const float P = A.top_p != nullptr ? A.top_p[b] : 1.0f, m = A.min_p != nullptr ? A.min_p[b] : 0.0f;
  const int k = A.top_k != nullptr ? A.top_k[b] : 0;

  const uint32_t top = R.top();
  if (top == NO_KEY) {
    if (threadIdx.x == 0) {
      A.ids[b] = -1;
      if (A.lps != nullptr) A.lps[b] = __int_as_float(0x7FC00000);
    }
    return;
  }
  // what is left: keys above K, and of the keys equal to K the indices up to I
  uint32_t K = 1;
  int I = A.V - 1;
  auto left = [&](int i, uint32_t key) { return key > K || (key == K && i <= I); };
  auto cut = [&](uint32_t key, u64 ties) {   // keeps the first `ties` (>= 1) of what is left at `key`
    const uint32_t k0 = K;
    const int i0 = I;
    I = R.locate([&](int i, uint32_t kk) -> u64 { return kk == key && (kk > k0 || i <= i0); }, ties - 1);
    K = key;
  };
  bool head = !(T > 0.0f);
  if (!head && k > 0 && k < A.V) {
    const u64 n = R.total([&](int, uint32_t kk) -> u64 { return kk != NO_KEY; });
    if (static_cast<u64>(k) < n) {
      u64 above;
      const uint32_t key = R.select([](int, uint32_t kk) -> u64 { return kk != NO_KEY; }, k, &above);
      cut(key, k - above);
    }
  }
  if (!head && !(m <= 0.0f)) {
    const float least = draw_val(top) + logf(m);
    if (!(draw_val(top) >= least)) {
      head = true;
    } else {
      const uint32_t key = draw_key(least);
      if (key > K) {
        K = key;
        I = A.V - 1;
      }
    }
  }
  if (!head && !(P >= 1.0f)) {
    auto w = [&](int i, uint32_t kk) -> u64 { return left(i, kk) ? draw_weight(draw_dist(kk, top)) : 0ull; };
    const u64 all = R.total(w);
    const u64 target = draw_share(P > 0.0f ? static_cast<u64>(P * 0x1p24f) : 0ull, all);
    if (target == 0) {
      head = true;
    } else {
      u64 above;
      const uint32_t key = R.select(w, target, &above);
      const u64 each = draw_weight(draw_dist(key, top));
      cut(key, (target - above + each - 1) / each);
    }
  }
  if (head) {
    const int i = R.locate([&](int, uint32_t kk) -> u64 { return kk == top; }, 0);
    if (threadIdx.x == 0) {
      A.ids[b] = i;
      if (A.lps != nullptr) A.lps[b] = 0.0f;
    }
    return;
  }
  const float inv = 1.0f / T;
  auto dist = [&](uint32_t kk) {
    const float d = draw_dist(kk, top);
    return d == 0.0f ? 0.0f : d * inv;
  };
  auto w = [&](int i, uint32_t kk) -> u64 { return left(i, kk) ? draw_weight(dist(kk)) : 0ull; };
  const u64 all = R.total(w);
  const float u = A.u[b];
  const u64 U = u > 0.0f ? static_cast<u64>(fminf(u, 1.0f - 0x1p-24f) * 0x1p24f) : 0ull;
  const int i = R.locate(w, draw_share(U, all));
  if (threadIdx.x == 0) {
    A.ids[b] = i;
    if (A.lps != nullptr) A.lps[b] = dist(R.key(i)) - logf(static_cast<float>(all) * (1.0f / DRAW_ONE));
  }
}

}  // namespace strata
