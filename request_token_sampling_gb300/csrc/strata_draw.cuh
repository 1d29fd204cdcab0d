// strata_draw.cuh -- one id per logit row from the caller's random numbers: top_k, min_p, top_p,
// temperature, with no limit on top_k.
//
// Every cut of the chain is a threshold in one order (logit descending, lowest index first), so what
// is left of a row is always {key > K} and, of the entries with key == K, those up to an index I.
// Weights are whole numbers (floor(exp(.) * 2^43)), so a sum of them is exact in 64 bits: it does not
// depend on the order or the split it was made in.
//
// A cluster of blocks holds one row in its shared memory, so the row is read from HBM once and every
// further step runs on chip.  The usual cuts leave few entries.  Each thread's largest logit shows where
// they end: the bin in which the threads' maxima are k, or weigh top_p's share, has all that the cuts can
// reach above it.  The entries up to there (a list of at most DRAW_LIST) go to the first block, which
// orders them and finishes alone.  Where they are more, the cluster counts or weighs the whole row into
// 2048 equal steps of distance from the largest logit, and orders the entries of the step that a cut
// falls into.
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
constexpr int DRAW_COARSE = DRAW_THREADS;  // bins of the threads' maxima, a quarter as fine
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
__device__ __forceinline__ void draw_ld_v4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void dsmem_st_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct DrawShared {
  uint64_t bars[DRAW_PIECES];
  u64 slot[2][2][DRAW_MAX_CLUSTER];  // what each block told: two turns of two values
  u64 warp[DRAW_WARPS];
  u64 found;
  uint32_t listed;           // entries in the first block's list
  alignas(16) uint32_t lo[DRAW_BINS];  // the lower and upper halves of the bins' sums
  alignas(16) uint32_t hi[DRAW_BINS];
  uint32_t count[DRAW_COARSE];
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

  // Two values of each block to all blocks of the row: tell() by one warp, meet(), heard().  A block reads
  // its own shared memory only, so the others may end.
  __device__ void tell(u64 a, u64 b) {
    if (static_cast<uint32_t>(lane) < ranks) {
      dsmem_st_u64(dsmem_addr(smem_u32(&sh->slot[turn & 1][0][rank]), lane), a);
      dsmem_st_u64(dsmem_addr(smem_u32(&sh->slot[turn & 1][1][rank]), lane), b);
    }
  }
  __device__ void meet() {
    cluster_arrive();
    cluster_wait();
    ++turn;
  }
  __device__ u64 heard(int which, uint32_t from) const { return sh->slot[(turn + 1) & 1][which][from]; }
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
      tell(s, 0);
    }
    meet();
    return heard_sum(0, before);
  }
  // After parts(f): the first index whose running sum exceeds `target` (< the row's sum), to all blocks.
  template <typename F>
  __device__ int find(F f, u64 target, u64 before) {
    if (threadIdx.x == 0) sh->found = 0;
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
            sh->found = static_cast<u64>(at) + 1;
          }
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
    }
    __syncthreads();
    if (warp == 0) tell(sh->found, 0);
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
  __device__ u64 all_bins(u64 (&v)[DRAW_PER_THREAD]) {
    static_assert(DRAW_PER_THREAD == 4, "16-byte loads");
#pragma unroll
    for (int i = 0; i < DRAW_PER_THREAD; ++i) v[i] = 0;
    for (uint32_t q = 0; q < ranks; ++q) {
      uint32_t l[4], h[4];
      draw_ld_v4(dsmem_addr(smem_u32(&sh->lo[threadIdx.x * 4]), q), l);
      draw_ld_v4(dsmem_addr(smem_u32(&sh->hi[threadIdx.x * 4]), q), h);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += static_cast<u64>(h[i]) << 32 | l[i];
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
    u64 below = all_bins(v), under;
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
    if (warp == 0) {
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
      below = all_bins(v);
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

  // Appends an entry to the first block's list (with the others of this warp that are here).
  __device__ __forceinline__ void append(int i, float x) {
    const uint32_t here = __activemask(), first = __ffs(here) - 1;
    uint32_t at = 0;
    if (static_cast<uint32_t>(lane) == first) at = dsmem_atomic_add(dsmem_addr(smem_u32(&sh->listed), 0), __popc(here));
    at = __shfl_sync(here, at, first) + __popc(here & ((1u << lane) - 1u));
    if (at < DRAW_LIST)
      dsmem_st_v2(dsmem_addr(smem_u32(&sh->list[0]), 0) + 8 * at, ~static_cast<uint32_t>(base + i), draw_key(x));
  }
  // The block's sum of one value per thread, to thread 0 of warp 0 at least.
  __device__ u64 block_sum(u64 v) {
    v = draw_warp_sum(v);
    __syncthreads();
    if (lane == 0) sh->warp[warp] = v;
    __syncthreads();
    return draw_warp_sum(lane < DRAW_WARPS ? sh->warp[lane] : 0);
  }

  // The cut that leaves sum(f) >= target, 1 <= target <= the row's sum, with as few entries as can be:
  // the last of them.  f is 0 for what earlier cuts took.
  template <typename F>
  __device__ void narrow(F f, float top, u64 target, uint32_t* K, int* I) {
    meet();  // the bins and the list of the step before are read
    if (threadIdx.x == 0) sh->listed = 0;
    clear_bins();
    each([&](int i, float x) {
      const u64 w = f(base + i, x);
      if (w) add_bin(bin(x, top), w);
    });
    __syncthreads();
    meet();
    u64 v[DRAW_PER_THREAD], under;
    const u64 below = all_bins(v);
    const int b = cross(v, below, target, &under);
    u64 mine = 0;
    each([&](int i, float x) {
      if (bin(x, top) == b && f(base + i, x)) {
        append(i, x);
        ++mine;
      }
    });
    mine = block_sum(mine);
    if (warp == 0) tell(mine, 0);
    meet();
    const u64 entries = heard_sum(0);
    if (entries > DRAW_LIST) {  // a great many alike
      u64 above;
      const uint32_t key = select(f, top, target, &above);
      const u64 one = f(-1, draw_val(key));
      auto same = [&](int i, float x) -> u64 { return draw_key(x) == key && f(i, x); };
      u64 before;
      parts(same, &before);
      *I = find(same, (target - above + one - 1) / one - 1, before);
      *K = key;
      return;
    }
    if (rank == 0) {
      sort(static_cast<int>(entries));
      constexpr int PER = DRAW_LIST / DRAW_THREADS;
      u64 w[PER], s = 0;
      for (int i = 0; i < PER; ++i) {
        const int at = static_cast<int>(threadIdx.x) * PER + i;
        const u64 e = at < static_cast<int>(entries) ? sh->list[at] : 0;
        w[i] = e ? f(static_cast<int>(~static_cast<uint32_t>(e)), draw_val(static_cast<uint32_t>(e >> 32))) : 0;
        s += w[i];
      }
      u64 run = under + block_scan(s) - s;
      for (int i = 0; i < PER; ++i) {
        if (run < target && run + w[i] >= target) sh->found = sh->list[threadIdx.x * PER + i];
        run += w[i];
      }
      __syncthreads();
      if (warp == 0) tell(sh->found, 0);
    }
    meet();
    const u64 e = heard(0, 0);
    *K = static_cast<uint32_t>(e >> 32);
    *I = static_cast<int>(~static_cast<uint32_t>(e));
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

  cluster_arrive_relaxed();  // this block runs: its shared memory may be written by the others

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
  for (int i = threadIdx.x; i < DRAW_COARSE; i += DRAW_THREADS) sh->count[i] = sh->lo[i] = sh->hi[i] = 0;
  const float T = A.temperature != nullptr ? A.temperature[row] : 1.0f;
  const float P = A.top_p != nullptr ? A.top_p[row] : 1.0f, m = A.min_p != nullptr ? A.min_p[row] : 0.0f;
  const int k = A.top_k != nullptr ? A.top_k[row] : 0;
  __syncthreads();

  // The thread's largest logit and its lowest index, then the row's.
  float most = -INFINITY;
  int most_at = -1;
  auto look = [&](int i, float x) {
    if (x > most) {  // not for NaN and -inf
      most = x;
      most_at = i;
    }
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
  u64 best = most_at < 0 ? 0 : static_cast<u64>(draw_key(most)) << 32 | static_cast<uint32_t>(~(R.base + most_at));
  best = warp_max_u64(best);
  if (R.lane == 0) sh->warp[R.warp] = best;
  __syncthreads();
  if (R.warp == 0) {
    best = warp_max_u64(R.lane < DRAW_WARPS ? sh->warp[R.lane] : 0);
  }
  cluster_wait();
  if (R.warp == 0) {
    R.tell(best, 0);
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
    return;
  }
  const float inv = 1.0f / T, u = A.u[row];
  const u64 u24 = u > 0.0f ? static_cast<u64>(fminf(u, 1.0f - 0x1p-24f) * 0x1p24f) : 0ull;
  auto tempered = [&](float x) { return x == top ? 0.0f : (x - top) * inv; };

  // what is left: keys above K, and of the keys equal to K the indices up to I
  uint32_t K = max(1u, m <= 0.0f ? 1u : draw_key(least));
  int I = A.V - 1;
  auto left = [&](int i, uint32_t key) { return key > K || (key == K && i <= I); };

  auto flat = [&](float x) { return draw_weight(x == top ? 0.0f : x - top); };  // at temperature 1
  bool try_list = k_on ? k <= DRAW_LIST / 2 : p_on;
  if (try_list) {
    // What top_k alone leaves, or (without it) what min_p leaves and top_p weighs, from the threads' maxima.
    u64 mass = 0;
    if (!k_on) {
      R.each([&](int, float x) { mass += x >= least && x > -INFINITY ? flat(x) : 0; });
      mass = R.block_sum(mass);
      if (R.warp == 0) R.tell(mass, 0);
    }
    if (most_at >= 0) {
      const int b = DrawRow<E>::bin(most, top) / (DRAW_BINS / DRAW_COARSE);
      atomicAdd(&sh->count[b], 1u);
      if (!k_on && most >= least) R.add_bin(b, flat(most));
    }
    R.meet();
    u64 v = 0, w = 0;
    for (uint32_t q = 0; q < R.ranks; ++q) {
      v += draw_ld_u32(dsmem_addr(smem_u32(&sh->count[threadIdx.x]), q));
      if (!k_on)
        w += static_cast<u64>(draw_ld_u32(dsmem_addr(smem_u32(&sh->hi[threadIdx.x]), q))) << 32 |
             draw_ld_u32(dsmem_addr(smem_u32(&sh->lo[threadIdx.x]), q));
    }
    // the first bin by which the maxima are k or weigh the share; without one, the last with few maxima
    const u64 target = k_on ? static_cast<u64>(k) : draw_share(p24, mass = R.heard_sum(0));
    const u64 upto = R.block_scan(v), reach = k_on ? upto : R.block_scan(w);
    __syncthreads();
    if (threadIdx.x == 0) sh->found = 0;
    __syncthreads();
    if (reach - (k_on ? v : w) < target && reach >= target) sh->found = static_cast<u64>(threadIdx.x) + 1;
    __syncthreads();
    int cut = static_cast<int>(sh->found) - 1;
    if (cut < 0) cut = __syncthreads_count(upto <= DRAW_LIST / 4) - 1;
    const float width = static_cast<float>(cut + 1) * (DRAW_BINS / DRAW_COARSE) / DRAW_STEPS;
    const bool rest = cut >= DRAW_COARSE - 1;  // the last bin holds everything further away
    u64 mine = 0, listed_mass = 0;
    R.each([&](int i, float x) {
      if (x > -INFINITY && x >= least && (rest || x == top || top - x < width)) {
        R.append(i, x);
        ++mine;
        if (!k_on) listed_mass += flat(x);
      }
    });
    mine = R.block_sum(mine);
    if (!k_on) listed_mass = R.block_sum(listed_mass);
    if (R.warp == 0) R.tell(mine, listed_mass);
    R.meet();
    const u64 entries = R.heard_sum(0);
    // top_k needs the bin of the k-th maximum, top_p its share: else the row is narrowed down as a whole
    try_list = entries <= DRAW_LIST && (k_on ? sh->found != 0 || rest : R.heard_sum(1) >= target);
    if (try_list) {
      if (!lead) return;
      const int listed = static_cast<int>(entries);
      R.sort(listed);
      int kept = k_on ? min(k, listed) : listed;
      constexpr int PER = DRAW_LIST / DRAW_THREADS;
      u64 ws[PER], sum;
      auto sums = [&](int count, auto weight) {  // each thread PER entries in a row; what comes before them
        u64 s = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int at = static_cast<int>(threadIdx.x) * PER + i;
          ws[i] = at < count ? weight(sh->list[at]) : 0;
          s += ws[i];
        }
        const u64 upto = R.block_scan(s);
        sum = 0;
        for (int q = 0; q < DRAW_WARPS; ++q) sum = sh->warp[q] + sum;
        return upto - s;
      };
      if (p_on) {
        u64 run = sums(kept, [&](u64 e) { return flat(draw_val(static_cast<uint32_t>(e >> 32))); });
        const u64 share = k_on ? draw_share(p24, sum) : target;
        u64 under = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int at = static_cast<int>(threadIdx.x) * PER + i;
          under += at < kept && (at == 0 || run < share);
          run += ws[i];
        }
        kept = static_cast<int>(R.block_sum(under));
      }
      // index order: swap the halves, so that the greatest ~index comes first
      __syncthreads();
      for (int i = threadIdx.x; i < kept; i += DRAW_THREADS) sh->list[i] = sh->list[i] << 32 | sh->list[i] >> 32;
      __syncthreads();
      R.sort(kept);
      u64 run = sums(kept, [&](u64 e) { return draw_weight(tempered(draw_val(static_cast<uint32_t>(e)))); });
      const u64 draw = draw_share(u24, sum);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (run <= draw && run + ws[i] > draw) {
          const u64 e = sh->list[threadIdx.x * PER + i];
          answer(static_cast<int>(~static_cast<uint32_t>(e >> 32)),
                 tempered(draw_val(static_cast<uint32_t>(e))) - logf(static_cast<float>(sum) * (1.0f / DRAW_ONE)));
        }
        run += ws[i];
      }
      return;
    }
  }
  if (k_on) {
    auto f = [&](int, float x) -> u64 { return x > -INFINITY; };
    u64 before;
    const uint32_t least_key = K;
    if (static_cast<u64>(k) < R.parts(f, &before)) {
      R.narrow(f, top, k, &K, &I);
      if (least_key > K) {
        K = least_key;
        I = A.V - 1;
      }
    }
  }
  if (p_on) {
    const uint32_t K0 = K;
    const int I0 = I;
    auto f = [&](int i, float x) -> u64 {
      const uint32_t key = draw_key(x);
      return key > K0 || (key == K0 && i <= I0) ? flat(x) : 0ull;
    };
    u64 before;
    const u64 target = draw_share(p24, R.parts(f, &before));
    R.narrow(f, top, target, &K, &I);
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
}

}  // namespace strata
