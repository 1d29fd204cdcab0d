// strata_draw.cuh -- one id per logit row from the caller's random numbers: top_k, min_p, top_p,
// temperature, with no limit on top_k.
//
// Every cut of the chain is a threshold in one order (logit descending, lowest index first), so what
// is left of a row is always {key > K} and, of the entries with key == K, those up to an index I.
// Weights are whole numbers (floor(exp(.) * 2^43)), so a sum of them is exact in 64 bits: it does not
// depend on the order or the split it was made in.
//
// A cluster of blocks holds one row in its shared memory, so the row is read from HBM once and every
// further step runs on chip.  Its blocks count the row into 2048 equal steps of distance from the
// largest logit.  Where the counts show that what the cuts leave is among at most DRAW_LIST entries
// (the usual case), those go to the first block, which orders them and finishes alone.  Otherwise the
// cluster narrows K down by counts (top_k) or weights (top_p), a range of keys at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "strata_device.cuh"

namespace strata {

struct DrawArgs {
  const void* logits;
  int64_t ld;
  int V, chunk;  // chunk: ids of a block, a multiple of 16
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* ids;
  float* lps;
  uint32_t* errors;
};

using u64 = unsigned long long;

constexpr int DRAW_THREADS = 512;
constexpr int DRAW_WARPS = DRAW_THREADS / 32;
constexpr int DRAW_BINS = 2048;
constexpr int DRAW_PER_THREAD = DRAW_BINS / DRAW_THREADS;
constexpr float DRAW_STEPS = 64.0f;     // bins per unit of logit: 32 units, beyond which a weight is 0
constexpr int DRAW_LIST = 2048;
constexpr int DRAW_PIECES = 4;          // parts a block's ids arrive in
constexpr int DRAW_MAX_CLUSTER = 16;
constexpr float DRAW_ONE = 0x1p43f;     // V <= 2^19 weights of at most 2^43 sum below 2^63
constexpr uint32_t NO_KEY = 0u;         // NaN and -inf: below every key that can be chosen
constexpr uint32_t DRAW_SPINS = 1u << 24;

// Order-preserving key; -0.0 and +0.0 share one.  -inf maps to 0x007FFFFF, NaN is taken out first.
__device__ __forceinline__ uint32_t draw_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (x == x && k > 0x007FFFFFu) ? k : NO_KEY;
}
__device__ __forceinline__ float draw_val(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// The whole-number weight of a (tempered) distance from the largest logit.
__device__ __forceinline__ u64 draw_weight(float dt) {
  const float e = expf(dt);
  return e == e ? __float2ull_rz(e * DRAW_ONE) : 0ull;
}
// floor(of * total / 2^24) for of <= 2^24 and total < 2^63
__device__ __forceinline__ u64 draw_share(u64 of, u64 total) {
  return of * (total >> 24) + ((of * (total & 0xFFFFFFu)) >> 24);
}
__device__ __forceinline__ u64 draw_warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ T draw_warp_scan(T v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}
__device__ __forceinline__ uint32_t draw_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ u64 draw_ld_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

struct DrawShared {
  uint64_t bars[DRAW_PIECES];
  u64 slot[2][2];            // what this block tells the others: two values, two turns
  u64 warp[DRAW_WARPS];
  u64 found;
  uint32_t listed;           // entries in the first block's list
  uint32_t lo[DRAW_BINS];    // counts, or the lower and upper halves of 64-bit sums
  uint32_t hi[DRAW_BINS];
  u64 list[DRAW_LIST];       // key << 32 | ~index: the order of the chain, descending
};

template <typename E>
struct DrawRow {
  static constexpr int VEC = 16 / static_cast<int>(sizeof(E));
  DrawShared* sh;
  const E* ids;        // this block's part of the row in shared memory, NaN beyond its end
  int vecs, base;      // 16-byte vectors of it, its first index
  uint32_t rank, ranks, turn;
  int warp, lane;

  template <typename F>
  __device__ __forceinline__ void vec(int v, F f) const {
    const uint4 raw = reinterpret_cast<const uint4*>(ids)[v];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float x;
      if constexpr (sizeof(E) == 4)
        x = __uint_as_float(w[i]);
      else
        x = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      f(v * VEC + i, x);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = threadIdx.x; v < vecs; v += DRAW_THREADS) vec(v, f);
  }

  // Every block's pair of values to every block: `sum` and the sum over lower ranks, or the maximum.
  __device__ void tell(u64 a, u64 b) {  // called by one thread, before meet()
    sh->slot[turn & 1][0] = a;
    sh->slot[turn & 1][1] = b;
  }
  __device__ void meet() {
    cluster_arrive();
    cluster_wait();
    ++turn;
  }
  __device__ u64 heard(int which, uint32_t from) const {
    return draw_ld_u64(dsmem_addr(smem_u32(&sh->slot[(turn + 1) & 1][which]), from));
  }
  __device__ u64 heard_sum(int which, u64* before = nullptr) const {
    const u64 v = static_cast<uint32_t>(lane) < ranks ? heard(which, lane) : 0;
    if (before != nullptr) *before = draw_warp_sum(static_cast<uint32_t>(lane) < rank ? v : 0);
    return draw_warp_sum(v);
  }

  // Sums f over the row by contiguous parts, one to a warp (sh->warp holds this block's): the row's
  // sum and what comes before this block.
  template <typename F>
  __device__ u64 parts(F f, u64* before) {
    const int part = (vecs + DRAW_WARPS - 1) / DRAW_WARPS;
    const int to = min(vecs, (warp + 1) * part);
    u64 s = 0;
    for (int v = warp * part + lane; v < to; v += 32) vec(v, [&](int i, float x) { s += f(base + i, x); });
    s = draw_warp_sum(s);
    __syncthreads();
    if (lane == 0) sh->warp[warp] = s;
    __syncthreads();
    if (warp == 0) {
      s = draw_warp_sum(lane < DRAW_WARPS ? sh->warp[lane] : 0);
      if (lane == 0) tell(s, 0);
    }
    meet();
    return heard_sum(0, before);
  }
  // After parts(f): the first index whose running sum exceeds `target` (< the row's sum), to all blocks.
  template <typename F>
  __device__ int find(F f, u64 target, u64 before) {
    if (threadIdx.x == 0) tell(0, 0);
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += sh->warp[w];
    if (before <= target && target - before < sh->warp[warp]) {
      const int part = (vecs + DRAW_WARPS - 1) / DRAW_WARPS;
      const int to = min(vecs, (warp + 1) * part);
      for (int v0 = warp * part; v0 < to; v0 += 32) {
        u64 own = 0;
        if (v0 + lane < to) vec(v0 + lane, [&](int i, float x) { own += f(base + i, x); });
        const u64 upto = draw_warp_scan(own, lane);
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, before + upto > target);
        if (over != 0) {
          if (lane == __ffs(over) - 1) {
            u64 run = before + upto - own;
            int at = -1;
            vec(v0 + lane, [&](int i, float x) {
              run += f(base + i, x);
              if (at < 0 && run > target) at = base + i;
            });
            tell(static_cast<u64>(at) + 1, 0);
          }
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
    }
    meet();
    return static_cast<int>(heard_sum(0)) - 1;
  }

  __device__ void clear_bins() {
    for (int b = threadIdx.x; b < DRAW_BINS; b += DRAW_THREADS) sh->lo[b] = sh->hi[b] = 0;
    __syncthreads();
  }
  // 64-bit addition from two 32-bit ones: the carry is known from the old lower half, whatever the order.
  __device__ __forceinline__ void add_bin(int b, u64 v) {
    const uint32_t l = static_cast<uint32_t>(v);
    uint32_t h = static_cast<uint32_t>(v >> 32);
    const uint32_t old = atomicAdd(&sh->lo[b], l);
    h += (old + l < old);
    if (h) atomicAdd(&sh->hi[b], h);
  }
  // After a meet(): the cluster's sums of this thread's bins, and over all lower bins.
  __device__ u64 all_bins(u64 (&v)[DRAW_PER_THREAD], bool wide) {
#pragma unroll
    for (int i = 0; i < DRAW_PER_THREAD; ++i) v[i] = 0;
    for (uint32_t q = 0; q < ranks; ++q) {
      const uint32_t l = dsmem_addr(smem_u32(&sh->lo[threadIdx.x * DRAW_PER_THREAD]), q);
      const uint32_t h = dsmem_addr(smem_u32(&sh->hi[threadIdx.x * DRAW_PER_THREAD]), q);
#pragma unroll
      for (int i = 0; i < DRAW_PER_THREAD; ++i) {
        v[i] += draw_ld_u32(l + 4 * i);
        if (wide) v[i] += static_cast<u64>(draw_ld_u32(h + 4 * i)) << 32;
      }
    }
    u64 s = 0;
#pragma unroll
    for (int i = 0; i < DRAW_PER_THREAD; ++i) s += v[i];
    return block_scan(s) - s;
  }
  // Inclusive sum over the block's threads.
  __device__ u64 block_scan(u64 s) {
    const u64 upto = draw_warp_scan(s, lane);
    __syncthreads();
    if (lane == 31) sh->warp[warp] = upto;
    __syncthreads();
    u64 below = 0;
    for (int w = 0; w < warp; ++w) below += sh->warp[w];
    return below + upto;
  }
  // The first of all bins whose inclusive sum reaches `target` >= 1 (DRAW_BINS: none), and the sum
  // below it.  `below` and `v` as all_bins gave them.
  __device__ int cross(const u64 (&v)[DRAW_PER_THREAD], u64 below, u64 target, u64* under) {
    __syncthreads();
    if (threadIdx.x == 0) sh->found = DRAW_BINS;
    __syncthreads();
    u64 run = below;
    for (int i = 0; i < DRAW_PER_THREAD; ++i) {
      if (run < target && run + v[i] >= target) {
        sh->found = threadIdx.x * DRAW_PER_THREAD + i;
        sh->warp[0] = run;
      }
      run += v[i];
    }
    __syncthreads();
    if (under != nullptr) *under = sh->warp[0];
    return static_cast<int>(sh->found);
  }

  // The key K with sum(key > K) < target <= sum(key >= K) of f over the row, 1 <= target <= the row's
  // sum, by ever finer equal ranges of keys.  `above` = sum(key > K).
  template <typename F>
  __device__ uint32_t select(F f, float top, u64 target, u64* above) {
    u64 over = 0, v[DRAW_PER_THREAD];
    // ranges of distance first, which spread a row's logits evenly
    meet();
    clear_bins();
    each([&](int i, float x) {
      const u64 w = f(base + i, x);
      if (w) add_bin(bin(x, top), w);
    });
    __syncthreads();
    meet();
    u64 below = all_bins(v, true), under;
    int b = cross(v, below, target, &under);
    over += under;
    // the least and the greatest key in there
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    each([&](int i, float x) {
      if (f(base + i, x) && bin(x, top) == b) {
        const uint32_t k = draw_key(x);
        lo = min(lo, k);
        hi = max(hi, k);
      }
    });
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    __syncthreads();
    if (lane == 0) sh->warp[warp] = static_cast<u64>(lo) << 32 | hi;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < DRAW_WARPS; ++w) {
        lo = min(lo, static_cast<uint32_t>(sh->warp[w] >> 32));
        hi = max(hi, static_cast<uint32_t>(sh->warp[w]));
      }
      tell(lo, hi);
    }
    meet();
    lo = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(lane) < ranks ? static_cast<uint32_t>(heard(0, lane)) : 0xFFFFFFFFu);
    hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(lane) < ranks ? static_cast<uint32_t>(heard(1, lane)) : 0u);
    while (lo < hi) {
      int shift = 0;
      while (((hi - lo) >> shift) >= DRAW_BINS) ++shift;
      clear_bins();
      each([&](int i, float x) {
        const uint32_t k = draw_key(x);
        if (k < lo || k > hi) return;
        const u64 w = f(base + i, x);
        if (w) add_bin((hi - k) >> shift, w);
      });
      __syncthreads();
      meet();
      below = all_bins(v, true);
      b = cross(v, below, target - over, &under);
      over += under;
      const uint32_t width = 1u << shift, from = hi - (static_cast<uint32_t>(b) << shift);
      lo = from - lo < width ? lo : from - width + 1;
      hi = from;
      meet();
    }
    *above = over;
    return hi;
  }

  static __device__ __forceinline__ int bin(float x, float top) {
    return x == top ? 0 : min(DRAW_BINS - 1, static_cast<int>((top - x) * DRAW_STEPS));
  }

  // Orders list[0, n) descending; what is beyond n up to a power of two is filled with zeros.
  __device__ void sort(int n) {
    int size = 32;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += DRAW_THREADS) sh->list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2) {
      for (int j = k / 2; j > 0; j /= 2) {
        for (int p = threadIdx.x; p < size / 2; p += DRAW_THREADS) {
          const int i = (p & ~(j - 1)) * 2 + (p & (j - 1));
          const u64 a = sh->list[i], b = sh->list[i + j];
          if ((a < b) == ((i & k) == 0)) {
            sh->list[i] = b;
            sh->list[i + j] = a;
          }
        }
        __syncthreads();
      }
    }
  }
};

template <typename E>
__global__ void __launch_bounds__(DRAW_THREADS, 2) draw_kernel(const __grid_constant__ DrawArgs A) {
  extern __shared__ __align__(16) uint8_t raw[];
  DrawShared* sh = reinterpret_cast<DrawShared*>(raw);
  E* ids = reinterpret_cast<E*>(raw + (sizeof(DrawShared) + 15) / 16 * 16);
  DrawRow<E> R;
  R.sh = sh;
  R.ids = ids;
  R.rank = cluster_ctarank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(R.ranks));
  R.turn = 0;
  R.warp = threadIdx.x >> 5;
  R.lane = threadIdx.x & 31;
  const int row = blockIdx.x / R.ranks;
  R.base = static_cast<int>(R.rank) * A.chunk;
  const int n = max(0, min(A.chunk, A.V - R.base));
  constexpr int VEC = DrawRow<E>::VEC;
  R.vecs = (n + VEC - 1) / VEC;
  const E* from = static_cast<const E*>(A.logits) + row * A.ld + R.base;

  // The block's part of the row, in pieces; what does not fill 16 bytes by plain loads.
  const int whole = n / VEC, piece = (whole + DRAW_PIECES - 1) / DRAW_PIECES;
  if (threadIdx.x == 0) {
    for (int p = 0; p < DRAW_PIECES; ++p) mbar_init(&sh->bars[p], 1);
    fence_proxy_async_smem();
    sh->listed = 0;
    for (int p = 0; p < DRAW_PIECES; ++p) {
      const int v0 = min(whole, p * piece), bytes = (min(whole, v0 + piece) - v0) * 16;
      if (bytes > 0) {
        mbar_arrive_expect_tx(&sh->bars[p], bytes);
        bulk_g2s(ids + v0 * VEC, from + v0 * VEC, bytes, &sh->bars[p]);
      }
    }
  }
  if (threadIdx.x < VEC && whole < R.vecs) {
    const int i = whole * VEC + threadIdx.x;
    if constexpr (sizeof(E) == 4)
      ids[i] = i < n ? from[i] : __int_as_float(0x7FC00000);
    else
      ids[i] = i < n ? from[i] : __ushort_as_bfloat16(0x7FC0);
  }
  const float T = A.temperature != nullptr ? A.temperature[row] : 1.0f;
  const float P = A.top_p != nullptr ? A.top_p[row] : 1.0f, m = A.min_p != nullptr ? A.min_p[row] : 0.0f;
  const int k = A.top_k != nullptr ? A.top_k[row] : 0;
  __syncthreads();

  // The largest logit and its lowest index.
  u64 best = 0;
  auto look = [&](int i, float x) {
    const u64 e = static_cast<u64>(draw_key(x)) << 32 | static_cast<uint32_t>(~(R.base + i));
    best = best < e ? e : best;
  };
  for (int p = 0; p < DRAW_PIECES; ++p) {
    const int v0 = min(whole, p * piece), v1 = min(whole, v0 + piece);
    if (v1 > v0) {
      uint32_t spin = 0;
      while (!mbar_try_wait(&sh->bars[p], 0))
        if (++spin >= DRAW_SPINS) {
          atomicOr(A.errors, 0x08u);  // STRATA_DEVERR_TIMEOUT
          break;
        }
      for (int v = v0 + threadIdx.x; v < v1; v += DRAW_THREADS) R.vec(v, look);
    }
  }
  if (threadIdx.x == 0 && whole < R.vecs) R.vec(whole, look);
  best = warp_max_u64(best);
  if (R.lane == 0) sh->warp[R.warp] = best;
  __syncthreads();
  if (R.warp == 0) {
    best = warp_max_u64(R.lane < DRAW_WARPS ? sh->warp[R.lane] : 0);
    if (R.lane == 0) R.tell(best, 0);
  }
  R.meet();
  best = warp_max_u64(static_cast<uint32_t>(R.lane) < R.ranks ? R.heard(0, R.lane) : 0);

  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  const float top = draw_val(top_key);
  const bool lead = R.rank == 0;
  auto answer = [&](int id, float lp) {  // by one thread of the cluster
    A.ids[row] = id;
    if (A.lps != nullptr) A.lps[row] = lp;
  };
  const float least = !(m <= 0.0f) ? top + logf(m) : -INFINITY;  // min_p's threshold
  const bool k_on = k > 0 && k < A.V, p_on = !(P >= 1.0f);
  const u64 p24 = P > 0.0f ? static_cast<u64>(fminf(P, 1.0f) * 0x1p24f) : 0ull;
  if (top_key == NO_KEY || !(T > 0.0f) || (!(m <= 0.0f) && !(top >= least)) || (p_on && p24 == 0)) {
    if (lead && threadIdx.x == 0)
      answer(top_key == NO_KEY ? -1 : static_cast<int>(~static_cast<uint32_t>(best)),
             top_key == NO_KEY ? __int_as_float(0x7FC00000) : 0.0f);
    R.meet();  // nobody leaves while another block may still read its values
    return;
  }
  const float inv = 1.0f / T, u = A.u[row];
  const u64 u24 = u > 0.0f ? static_cast<u64>(fminf(u, 1.0f - 0x1p-24f) * 0x1p24f) : 0ull;
  auto tempered = [&](float x) { return x == top ? 0.0f : (x - top) * inv; };

  // what is left: keys above K, and of the keys equal to K the indices up to I
  uint32_t K = max(1u, m <= 0.0f ? 1u : draw_key(least));
  int I = A.V - 1;
  auto left = [&](int i, uint32_t key) { return key > K || (key == K && i <= I); };

  if (k_on || p_on) {
    R.clear_bins();
    u64 mass = 0;
    const bool need_mass = p_on && !k_on;
    const bool all = !k_on;  // top_k counts every entry, top_p those that min_p left
    R.each([&](int, float x) {
      if (!(x > -INFINITY) || (all && !(x >= least))) return;
      atomicAdd(&sh->lo[DrawRow<E>::bin(x, top)], 1u);
      if (need_mass) mass += draw_weight(x == top ? 0.0f : x - top);
    });
    mass = draw_warp_sum(mass);
    __syncthreads();
    if (R.lane == 0) sh->warp[R.warp] = mass;
    __syncthreads();
    if (R.warp == 0) {
      mass = draw_warp_sum(R.lane < DRAW_WARPS ? sh->warp[R.lane] : 0);
      if (R.lane == 0) R.tell(mass, 0);
    }
    R.meet();
    mass = R.heard_sum(0);
    u64 v[DRAW_PER_THREAD];
    const u64 below = R.all_bins(v, false);
    // the last bin that the cuts can reach into
    int cut = DRAW_BINS - 1;
    bool whole_set = true;  // the bins up to `cut` hold all that top_k and min_p leave
    if (k_on) {
      const int b = R.cross(v, below, k, nullptr);
      if (b < DRAW_BINS) cut = b;
    }
    if (!(m <= 0.0f)) cut = min(cut, DrawRow<E>::bin(least, top));
    auto count_to = [&](int b) {
      __syncthreads();
      u64 run = below;
      for (int i = 0; i < DRAW_PER_THREAD; ++i) {
        run += v[i];
        if (static_cast<int>(threadIdx.x) * DRAW_PER_THREAD + i == b) sh->found = run;
      }
      __syncthreads();
      return sh->found;
    };
    u64 entries = count_to(cut);
    const u64 target_all = draw_share(p24, mass);
    if (entries > DRAW_LIST && need_mass) {
      // a lower bound of the bins' weights: enough of them to reach top_p's share for certain
      u64 lower[DRAW_PER_THREAD], s = 0;
      for (int i = 0; i < DRAW_PER_THREAD; ++i) {
        const float edge = -static_cast<float>(threadIdx.x * DRAW_PER_THREAD + i + 1) / DRAW_STEPS;
        lower[i] = v[i] * __float2ull_rz(expf(edge) * (DRAW_ONE * (1.0f - 0x1p-18f)));
        s += lower[i];
      }
      const u64 under = R.block_scan(s) - s;
      const int b = R.cross(lower, under, target_all, nullptr);
      if (b < cut) {
        cut = b;
        whole_set = false;
        entries = count_to(cut);
      }
    }
    if (entries <= DRAW_LIST) {
      // to the first block's list, in any order
      const uint32_t there = dsmem_addr(smem_u32(&sh->list[0]), 0), counter = dsmem_addr(smem_u32(&sh->listed), 0);
      R.each([&](int i, float x) {
        if (x > -INFINITY && DrawRow<E>::bin(x, top) <= cut && (!all || x >= least)) {
          const uint32_t here = __activemask(), first = __ffs(here) - 1;  // one addition for these lanes
          uint32_t at = 0;
          if (static_cast<uint32_t>(R.lane) == first) at = dsmem_atomic_add(counter, __popc(here));
          at = __shfl_sync(here, at, first) + __popc(here & ((1u << R.lane) - 1u));
          if (at < DRAW_LIST) dsmem_st_v2(there + 8 * at, ~static_cast<uint32_t>(R.base + i), draw_key(x));
        }
      });
      R.meet();
      if (!lead) return;
      const int listed = min(static_cast<int>(sh->listed), DRAW_LIST);
      R.sort(listed);
      // top_k is the list's length now, min_p a key, top_p a running sum
      int kept = k_on ? min(k, listed) : listed;
      {
        int mine = 0;
        for (int i = threadIdx.x; i < kept; i += DRAW_THREADS) mine += draw_val(sh->list[i] >> 32) >= least;
        mine = __reduce_add_sync(0xFFFFFFFFu, mine);
        __syncthreads();
        if (R.lane == 0) sh->warp[R.warp] = mine;
        __syncthreads();
        kept = 0;
        for (int w = 0; w < DRAW_WARPS; ++w) kept += static_cast<int>(sh->warp[w]);
      }
      constexpr int PER = DRAW_LIST / DRAW_THREADS;
      auto sums = [&](int count, auto weight, u64 (&w)[PER], u64* sum) {  // each thread PER entries in a row
        u64 s = 0;
        for (int i = 0; i < PER; ++i) {
          const int at = static_cast<int>(threadIdx.x) * PER + i;
          w[i] = at < count ? weight(sh->list[at]) : 0;
          s += w[i];
        }
        const u64 upto = R.block_scan(s);
        u64 whole = 0;
        for (int q = 0; q < DRAW_WARPS; ++q) whole += sh->warp[q];
        *sum = whole;
        return upto - s;
      };
      u64 w[PER], sum;
      if (p_on) {
        u64 run = sums(kept, [&](u64 e) { const float x = draw_val(e >> 32); return draw_weight(x == top ? 0.0f : x - top); }, w, &sum);
        const u64 target = whole_set ? draw_share(p24, sum) : target_all;
        int mine = 0;
        for (int i = 0; i < PER; ++i) {
          const int at = static_cast<int>(threadIdx.x) * PER + i;
          mine += at < kept && (at == 0 || run < target);
          run += w[i];
        }
        mine = __reduce_add_sync(0xFFFFFFFFu, mine);
        __syncthreads();
        if (R.lane == 0) sh->warp[R.warp] = mine;
        __syncthreads();
        kept = 0;
        for (int q = 0; q < DRAW_WARPS; ++q) kept += static_cast<int>(sh->warp[q]);
      }
      // index order: swap the halves, so that the greatest ~index comes first
      __syncthreads();
      for (int i = threadIdx.x; i < kept; i += DRAW_THREADS) sh->list[i] = sh->list[i] << 32 | sh->list[i] >> 32;
      __syncthreads();
      R.sort(kept);
      u64 run = sums(kept, [&](u64 e) { return draw_weight(tempered(draw_val(static_cast<uint32_t>(e)))); }, w, &sum);
      const u64 target = draw_share(u24, sum);
      for (int i = 0; i < PER; ++i) {
        if (run <= target && run + w[i] > target) {
          const u64 e = sh->list[threadIdx.x * PER + i];
          answer(static_cast<int>(~static_cast<uint32_t>(e >> 32)),
                 tempered(draw_val(static_cast<uint32_t>(e))) - logf(static_cast<float>(sum) * (1.0f / DRAW_ONE)));
        }
        run += w[i];
      }
      return;
    }
    // Too many: narrow K down over the whole row.
    auto keep_first = [&](uint32_t key, u64 ties) {  // keeps the first `ties` (>= 1) of what is left at `key`
      const uint32_t k0 = K;
      const int i0 = I;
      auto f = [&](int i, float x) -> u64 {
        const uint32_t kk = draw_key(x);
        return kk == key && (kk > k0 || i <= i0);
      };
      u64 before;
      R.parts(f, &before);
      I = R.find(f, ties - 1, before);
      K = key;
    };
    if (k_on) {
      const uint32_t least_key = K;
      K = 1;
      auto f = [&](int, float x) -> u64 { return x > -INFINITY; };
      u64 before;
      if (static_cast<u64>(k) < R.parts(f, &before)) {
        u64 above;
        const uint32_t key = R.select(f, top, k, &above);
        keep_first(key, k - above);
      }
      if (least_key > K) {
        K = least_key;
        I = A.V - 1;
      }
    }
    if (p_on) {
      auto f = [&](int i, float x) -> u64 {
        return left(i, draw_key(x)) ? draw_weight(x == top ? 0.0f : x - top) : 0ull;
      };
      u64 before;
      const u64 target = draw_share(p24, R.parts(f, &before));
      u64 above;
      const uint32_t key = R.select(f, top, target, &above);
      const u64 one = draw_weight(key == top_key ? 0.0f : draw_val(key) - top);
      keep_first(key, (target - above + one - 1) / one);
    }
  }
  auto f = [&](int i, float x) -> u64 { return left(i, draw_key(x)) ? draw_weight(tempered(x)) : 0ull; };
  u64 before;
  const u64 all = R.parts(f, &before);
  const int at = R.find(f, draw_share(u24, all), before);
  if (at >= R.base && at < R.base + n && threadIdx.x == 0) {
    float x;
    if constexpr (sizeof(E) == 4)
      x = ids[at - R.base];
    else
      x = __bfloat162float(ids[at - R.base]);
    answer(at, tempered(x) - logf(static_cast<float>(all) * (1.0f / DRAW_ONE)));
  }
  R.meet();
}

}  // namespace strata
