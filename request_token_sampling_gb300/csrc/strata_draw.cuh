// strata_draw.cuh -- one id per logit row from the caller's random numbers: top_k, min_p, top_p,
// temperature, with no limit on top_k.
//
// Every cut of the chain is a threshold in one order (logit descending, lowest index first), so what
// is left of a row is always {key > K} and, of the entries with key == K, those up to an index I.
// Weights are whole numbers (floor(exp(.) * 2^43)), so a sum of them is exact in 64 bits: it does not
// depend on the order or the split it was made in.
//
// A cluster of blocks holds one row in its shared memory, so the row is read from HBM once and every
// further step runs on chip.
//   top_k of up to DRAW_LIST / 2: the bin in which the threads' largest logits are k has all of the
//     top_k at or above it.  The entries up to there (the list) go to the first block, which orders
//     them and finishes alone.
//   top_p alone: the row is weighed into DRAW_BINS equal steps of distance from the largest logit.  Few
//     entries up to the step that top_p falls into: a list, as above.  Many: only that step's entries
//     are listed and ordered, which gives K and I.
//   a larger top_k: K and I the same way, from counts.
// What K and I leave is summed by contiguous parts, and the part that the random number falls into is
// summed again entry by entry.
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
constexpr int DRAW_COARSE = DRAW_THREADS;  // bins of the threads' maxima, a quarter as fine
constexpr int DRAW_LIST = 2048;
constexpr int DRAW_PIECES = 4;          // parts a block's ids arrive in
constexpr int DRAW_MAX_CLUSTER = 16;
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
// The whole-number weight floor(exp(dt) * 2^43) of a (tempered) distance dt <= 0 from the largest logit:
// the float's 24 bits, shifted (the conversion instruction to 64 bits runs at a small part of this
// rate).  2^19 weights of at most 2^43 sum below 2^63.
__device__ __forceinline__ u64 draw_weight(float dt) {
  const uint32_t e = __float_as_uint(expf(dt));
  const int s = static_cast<int>(e >> 23) - 107;  // of a unit in the last place of the 24 bits
  const uint32_t up = static_cast<uint32_t>(max(s, 0)), down = static_cast<uint32_t>(min(max(-s, 0), 31));
  const uint32_t m = ((e & 0x7FFFFFu) | 0x800000u) >> down;
  return static_cast<u64>(__funnelshift_l(m, 0u, up)) << 32 | (m << up);
}
constexpr float DRAW_UNIT = 0x1p-43f;
// floor(of * total / 2^24) for of <= 2^24 and total < 2^63
__device__ __forceinline__ u64 draw_share(u64 of, u64 total) {
  return of * (total >> 24) + ((of * (total & 0xFFFFFFu)) >> 24);
}
__device__ __forceinline__ u64 draw_warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ u64 draw_warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xFFFFFFFFu, v, o);
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
  u64 slot[2][2][DRAW_MAX_CLUSTER];    // what each block told: two turns of two values
  u64 warp[DRAW_WARPS];
  u64 found, found_sum;
  uint32_t listed;                     // entries in the first block's list
  alignas(16) uint32_t lo[DRAW_BINS];  // the lower and upper halves of the bins' sums
  alignas(16) uint32_t hi[DRAW_BINS];
  uint32_t count[DRAW_COARSE];         // threads' maxima
  u64 list[DRAW_LIST];                 // key << 32 | ~index: the order of the chain, descending
};

template <typename E>
struct DrawRow {
  static constexpr int VEC = 16 / static_cast<int>(sizeof(E));
  DrawShared* sh;
  const E* ids;        // this block's part of the row in shared memory, NaN beyond its end
  int vecs, base;      // 16-byte vectors of it, its first index
  uint32_t rank, ranks, turn;
  int warp, lane;
  float top;           // the row's largest logit

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

  // The block's sum of one value per thread, to all threads.
  __device__ u64 block_sum(u64 v) {
    v = draw_warp_sum(v);
    __syncthreads();
    if (lane == 0) sh->warp[warp] = v;
    __syncthreads();
    return draw_warp_sum(lane < DRAW_WARPS ? sh->warp[lane] : 0);
  }
  // Inclusive sum over the block's threads, and the whole sum.
  __device__ u64 block_scan(u64 s, u64* all = nullptr) {
    const u64 upto = draw_warp_scan(s, lane);
    __syncthreads();
    if (lane == 31) sh->warp[warp] = upto;
    __syncthreads();
    const u64 w = lane < DRAW_WARPS ? sh->warp[lane] : 0;
    if (all != nullptr) *all = draw_warp_sum(w);
    return draw_warp_sum(lane < warp ? w : 0) + upto;
  }

  // Sums f over the row by contiguous parts, one to a warp (sh->warp holds this block's): the row's
  // sum and what comes before this block.
  template <typename F>
  __device__ u64 parts(F f, u64* before) {
    const int part = (vecs + DRAW_WARPS - 1) / DRAW_WARPS;
    const int to = min(vecs, (warp + 1) * part);
    u64 s = 0;
    for (int v = warp * part + lane; v < to; v += 32) vec(v, [&](int i, float x) { s += f(base + i, x); });
    s = block_sum(s);
    if (warp == 0) tell(s, 0);
    meet();
    return heard_sum(0, before);
  }
  // After parts(f): the first index whose running sum exceeds `target` (< the row's sum), to all blocks.
  // The whole block sums the part again, a vector to a thread.
  template <typename F>
  __device__ int find(F f, u64 target, u64 before) {
    if (threadIdx.x == 0) sh->found = 0;
    const u64 mine = lane < DRAW_WARPS ? sh->warp[lane] : 0;
    const u64 upto = before + draw_warp_scan(mine, lane);
    const uint32_t over = __ballot_sync(0xFFFFFFFFu, lane < DRAW_WARPS && upto - mine <= target && target < upto);
    if (over != 0) {  // in this block
      const int hit = __ffs(over) - 1;
      u64 run = __shfl_sync(0xFFFFFFFFu, upto - mine, hit);
      const int part = (vecs + DRAW_WARPS - 1) / DRAW_WARPS;
      const int to = min(vecs, (hit + 1) * part);
      for (int v0 = hit * part; v0 < to; v0 += DRAW_THREADS) {
        const int v = v0 + static_cast<int>(threadIdx.x);
        u64 own = 0, all;
        if (v < to) vec(v, [&](int i, float x) { own += f(base + i, x); });
        const u64 here = run + block_scan(own, &all);
        if (here - own <= target && target < here) {
          u64 sum = here - own;
          int at = -1;
          vec(v, [&](int i, float x) {
            sum += f(base + i, x);
            if (at < 0 && sum > target) at = base + i;
          });
          sh->found = static_cast<u64>(at) + 1;
        }
        run += all;
      }
    }
    __syncthreads();
    if (warp == 0) tell(sh->found, 0);
    meet();
    return static_cast<int>(heard_sum(0)) - 1;
  }

  __device__ __forceinline__ int bin(float x) const {
    return x == top ? 0 : min(DRAW_BINS - 1, static_cast<int>((top - x) * DRAW_STEPS));
  }
  // A logit at or below every entry of the bins before `b`, and above -inf.
  __device__ __forceinline__ float floor_of(int b) const {
    return b >= DRAW_BINS ? -3.402823466e38f : fmaxf(-3.402823466e38f, top - b * (1.0001f / DRAW_STEPS));
  }

  __device__ void clear_bins() {
    for (int b = threadIdx.x; b < DRAW_BINS / 4; b += DRAW_THREADS)
      reinterpret_cast<uint4*>(sh->lo)[b] = reinterpret_cast<uint4*>(sh->hi)[b] = make_uint4(0, 0, 0, 0);
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
  // After a meet(): the cluster's sums of this thread's bins, over all lower bins, and over all.
  __device__ u64 all_bins(u64 (&v)[DRAW_PER_THREAD], u64* all) {
    static_assert(DRAW_PER_THREAD == 4, "16-byte loads");
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0;
    const uint32_t lo = smem_u32(&sh->lo[threadIdx.x * 4]), hi = smem_u32(&sh->hi[threadIdx.x * 4]);
    for (uint32_t q0 = 0; q0 < ranks; q0 += 4) {
      uint32_t l[4][4], h[4][4];
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) {  // the loads of four blocks on their way at once
        draw_ld_v4(dsmem_addr(lo, min(q0 + q, ranks - 1)), l[q]);
        draw_ld_v4(dsmem_addr(hi, min(q0 + q, ranks - 1)), h[q]);
      }
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q)
        if (q0 + q < ranks)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += static_cast<u64>(h[q][i]) << 32 | l[q][i];
    }
    const u64 s = v[0] + v[1] + v[2] + v[3];
    return block_scan(s, all) - s;
  }
  // The cluster's number of maxima in coarse bin `b`.
  __device__ uint32_t all_maxima(int b) {
    const uint32_t at = smem_u32(&sh->count[b]);
    uint32_t s = 0;
#pragma unroll
    for (uint32_t q = 0; q < DRAW_MAX_CLUSTER; ++q) {
      const uint32_t v = draw_ld_u32(dsmem_addr(at, min(q, ranks - 1)));
      s += q < ranks ? v : 0;
    }
    return s;
  }
  // The first of all bins whose inclusive sum reaches `target` >= 1 (DRAW_BINS: none), and the sum
  // below it.  `below` and `v` as all_bins gave them.
  __device__ int cross(const u64 (&v)[DRAW_PER_THREAD], u64 below, u64 target, u64* under) {
    __syncthreads();
    if (threadIdx.x == 0) sh->found = DRAW_BINS;
    __syncthreads();
    u64 run = below;
#pragma unroll
    for (int i = 0; i < DRAW_PER_THREAD; ++i) {
      if (run < target && run + v[i] >= target) {
        sh->found = threadIdx.x * DRAW_PER_THREAD + i;
        sh->found_sum = run;
      }
      run += v[i];
    }
    __syncthreads();
    *under = sh->found_sum;
    return static_cast<int>(sh->found);
  }

  // The key K with sum(key > K) < target <= sum(key >= K) of f over the row's bin `b`, of which `over`
  // lies above, by ever finer equal ranges of keys: for bins of any number of equal logits.
  template <typename F>
  __device__ uint32_t select(F f, int b, u64 over, u64 target, u64* above) {
    u64 v[DRAW_PER_THREAD], under, all;
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    each([&](int i, float x) {
      if (f(base + i, x) && bin(x) == b) {
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
      const u64 below = all_bins(v, &all);
      const int at = cross(v, below, target - over, &under);
      over += under;
      const uint32_t width = 1u << shift, from = hi - (static_cast<uint32_t>(at) << shift);
      lo = from - lo < width ? lo : from - width + 1;
      hi = from;
      meet();
    }
    *above = over;
    return hi;
  }

  // Orders list[0, n) descending; what is beyond n up to a power of two is filled with zeros.
  __device__ void sort(int n) {
    int size = 32;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += DRAW_THREADS) sh->list[i] = 0;
    __syncthreads();
    if (size <= DRAW_THREADS) {
      // an entry to a thread: steps of less than a warp go from lane to lane
      u64 a = static_cast<int>(threadIdx.x) < size ? sh->list[threadIdx.x] : 0;
      for (int k = 2; k <= size; k *= 2) {
        for (int j = k / 2; j > 0; j /= 2) {
          u64 b;
          if (j >= 32) {
            __syncthreads();
            if (static_cast<int>(threadIdx.x) < size) sh->list[threadIdx.x] = a;
            __syncthreads();
            b = static_cast<int>(threadIdx.x) < size ? sh->list[threadIdx.x ^ j] : 0;
          } else {
            b = __shfl_xor_sync(0xFFFFFFFFu, a, j);
          }
          const bool larger = ((threadIdx.x & k) == 0) == ((threadIdx.x & j) == 0);  // of the two, this thread keeps it
          a = larger == (a < b) ? b : a;
        }
      }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < size) sh->list[threadIdx.x] = a;
      __syncthreads();
      return;
    }
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
  // Lists the entries from `least` to `most` that take(index, x) wants, in any order; the row's number
  // of them (the list has the first DRAW_LIST).  A vector without any costs a comparison an entry.
  template <typename F>
  __device__ u64 gather(float least, float most, F take) {
    uint32_t mine = 0;
    for (int v = threadIdx.x; v < vecs; v += DRAW_THREADS) {
      bool any = false;
      vec(v, [&](int, float x) { any |= x >= least && x <= most; });
      if (!any) continue;
      vec(v, [&](int i, float x) {
        if (x >= least && x <= most && take(base + i, x)) {
          append(i, x);
          ++mine;
        }
      });
    }
    const u64 s = block_sum(mine);
    if (warp == 0) tell(s, 0);
    meet();
    return heard_sum(0);
  }

  // The last entry that a cut leaves: with as few as can be, sum(f) reaches `target`, 1 <= target <= the row's
  // sum.  It is in bin `b`, and `under` is the sum of the bins before.  f is 0 for what earlier cuts took.
  // The list is empty.
  template <typename F>
  __device__ void pin(F f, int b, u64 under, u64 target, uint32_t* K, int* I) {
    const float most = b == 0 ? top : fminf(top, top - b * (0.9999f / DRAW_STEPS));
    const u64 entries = gather(floor_of(b + 1), most, [&](int i, float x) { return bin(x) == b && f(i, x) != 0; });
    if (entries > DRAW_LIST) {  // a great many alike
      u64 above;
      const uint32_t key = select(f, b, under, target, &above);
      const u64 one = f(-1, draw_val(key));
      auto same = [&](int i, float x) -> u64 { return draw_key(x) == key && f(i, x) != 0; };
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
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = static_cast<int>(threadIdx.x) * PER + i;
        const u64 e = at < static_cast<int>(entries) ? sh->list[at] : 0;
        w[i] = e ? f(static_cast<int>(~static_cast<uint32_t>(e)), draw_val(static_cast<uint32_t>(e >> 32))) : 0;
        s += w[i];
      }
      u64 run = under + block_scan(s) - s;
#pragma unroll
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
  const float T = A.temperature != nullptr ? A.temperature[row] : 1.0f;
  const float P = A.top_p != nullptr ? A.top_p[row] : 1.0f, m = A.min_p != nullptr ? A.min_p[row] : 0.0f;
  const int k = A.top_k != nullptr ? A.top_k[row] : 0;
  const float u = A.u[row];
  if (threadIdx.x < VEC && whole < R.vecs) {
    const int i = whole * VEC + threadIdx.x;
    if constexpr (sizeof(E) == 4)
      ids[i] = i < n ? from[i] : __int_as_float(0x7FC00000);
    else
      ids[i] = i < n ? from[i] : __ushort_as_bfloat16(0x7FC0);
  }
  sh->count[threadIdx.x] = 0;
  R.clear_bins();

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
  cluster_wait();
  if (R.warp == 0) {
    best = warp_max_u64(R.lane < DRAW_WARPS ? sh->warp[R.lane] : 0);
    R.tell(best, 0);
  }
  R.meet();
  best = warp_max_u64(static_cast<uint32_t>(R.lane) < R.ranks ? R.heard(0, R.lane) : 0);

  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  const float top = draw_val(top_key);
  R.top = top;
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
  const float inv = 1.0f / T;
  const u64 u24 = u > 0.0f ? static_cast<u64>(fminf(u, 1.0f - 0x1p-24f) * 0x1p24f) : 0ull;
  // fmaxf: an infinite distance by an infinite temperature is no number, and weighs nothing
  auto tempered = [&](float x) { return x == top ? 0.0f : fmaxf((x - top) * inv, -1000.0f); };
  auto flat = [&](float x) { return draw_weight(x == top ? 0.0f : x - top); };  // at temperature 1

  // what is left: keys above K, and of the keys equal to K the indices up to I
  uint32_t K = max(1u, m <= 0.0f ? 1u : draw_key(least));
  int I = A.V - 1;

  // The first block's list holds all that the cuts leave, and maybe more below: it finishes alone.
  // `share`: top_p's part of the weight, 0 where it is of the list after top_k.
  auto finish = [&](int listed, u64 share) {
    R.sort(listed);
    constexpr int PER = DRAW_LIST / DRAW_THREADS;
    int kept = k_on ? min(k, listed) : listed;
    const int per = listed <= DRAW_THREADS ? 1 : PER;  // entries of a thread, in a row
    u64 ws[PER], sum;
    auto sums = [&](int count, auto weight) {  // what comes before a thread's entries
      u64 s = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = static_cast<int>(threadIdx.x) * per + i;
        ws[i] = i < per && at < count ? weight(sh->list[at]) : 0;
        s += ws[i];
      }
      return R.block_scan(s, &sum) - s;
    };
    if (p_on) {
      u64 run = sums(kept, [&](u64 e) { return flat(draw_val(static_cast<uint32_t>(e >> 32))); });
      if (share == 0) share = draw_share(p24, sum);
      u64 under = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = static_cast<int>(threadIdx.x) * per + i;
        under += i < per && at < kept && (at == 0 || run < share);
        run += ws[i];
      }
      kept = static_cast<int>(R.block_sum(under));
    }
    // index order: swap the halves, so that the greatest ~index comes first
    __syncthreads();
    for (int i = threadIdx.x; i < kept; i += DRAW_THREADS) sh->list[i] = sh->list[i] << 32 | sh->list[i] >> 32;
    R.sort(kept);
    u64 run = sums(kept, [&](u64 e) { return draw_weight(tempered(draw_val(static_cast<uint32_t>(e)))); });
    const u64 draw = draw_share(u24, sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (run <= draw && run + ws[i] > draw) {
        const u64 e = sh->list[threadIdx.x * per + i];
        answer(static_cast<int>(~static_cast<uint32_t>(e >> 32)),
               tempered(draw_val(static_cast<uint32_t>(e))) - logf(static_cast<float>(sum) * DRAW_UNIT));
      }
      run += ws[i];
    }
  };
  auto count_maximum = [&]() {
    if (most_at >= 0) atomicAdd(&sh->count[R.bin(most) / (DRAW_BINS / DRAW_COARSE)], 1u);
  };
  auto all = [](int, float) { return true; };
  bool listed_before = false;
  auto new_list = [&]() {  // with at least one meet() before the next entry
    if (threadIdx.x == 0) sh->listed = 0;
    listed_before = false;
  };

  u64 v[DRAW_PER_THREAD], under, sum, before;
  if (k_on && k <= DRAW_LIST / 2) {
    count_maximum();
    R.meet();
    const u64 here = R.all_maxima(threadIdx.x), upto = R.block_scan(here);
    __syncthreads();
    if (threadIdx.x == 0) sh->found = DRAW_COARSE;
    __syncthreads();
    if (upto - here < static_cast<u64>(k) && upto >= static_cast<u64>(k)) sh->found = threadIdx.x;
    __syncthreads();
    // fewer maxima than k: every entry
    const int last = (static_cast<int>(sh->found) + 1) * (DRAW_BINS / DRAW_COARSE);
    const u64 entries = R.gather(fmaxf(least, R.floor_of(last)), top, all);
    if (entries <= DRAW_LIST) {
      if (lead) finish(static_cast<int>(entries), 0);
      return;
    }
    listed_before = true;
  }
  if (k_on) {
    if (listed_before) new_list();
    auto one = [&](int, float x) -> u64 { return x > -INFINITY; };
    R.each([&](int, float x) {
      if (x > -INFINITY) atomicAdd(&sh->lo[R.bin(x)], 1u);
    });
    __syncthreads();
    R.meet();
    const u64 below = R.all_bins(v, &sum);
    if (static_cast<u64>(k) < sum) {
      const uint32_t least_key = K;
      const int b = R.cross(v, below, k, &under);
      R.pin(one, b, under, k, &K, &I);
      listed_before = true;
      if (least_key > K) {
        K = least_key;
        I = A.V - 1;
      }
    }
  }
  if (p_on) {
    const uint32_t K0 = K;
    const int I0 = I;
    auto weight = [&](int i, float x) -> u64 {
      const uint32_t key = draw_key(x);
      return key > K0 || (key == K0 && i <= I0) ? flat(x) : 0ull;
    };
    if (k_on) {
      R.meet();  // the bins and the list of the step before are read
      if (listed_before) new_list();
      R.clear_bins();
    } else {
      count_maximum();
    }
    R.each([&](int i, float x) {
      const u64 w = weight(R.base + i, x);
      if (w) R.add_bin(R.bin(x), w);
    });
    __syncthreads();
    R.meet();
    const u64 below = R.all_bins(v, &sum), share = draw_share(p24, sum);
    const int b = R.cross(v, below, share, &under);
    bool few = false;
    if (!k_on) {  // how many entries there are up to b: about as many as maxima, where they are few
      const int last = b / (DRAW_BINS / DRAW_COARSE);
      few = R.block_sum(static_cast<int>(threadIdx.x) <= last ? R.all_maxima(threadIdx.x) : 0) <= DRAW_LIST / 4;
    }
    if (few) {
      const u64 entries = R.gather(fmaxf(least, R.floor_of(b + 1)), top, all);
      if (entries <= DRAW_LIST) {
        if (lead) finish(static_cast<int>(entries), share);
        return;
      }
      R.meet();
      new_list();
      R.meet();
    }
    R.pin(weight, b, under, share, &K, &I);
  }
  auto left = [&](int i, float x) -> u64 {
    const uint32_t key = draw_key(x);
    return key > K || (key == K && i <= I) ? draw_weight(tempered(x)) : 0ull;
  };
  const u64 total = R.parts(left, &before);
  const int at = R.find(left, draw_share(u24, total), before);
  if (at >= R.base && at < R.base + n && threadIdx.x == 0) {
    float x;
    if constexpr (sizeof(E) == 4)
      x = ids[at - R.base];
    else
      x = __bfloat162float(ids[at - R.base]);
    answer(at, tempered(x) - logf(static_cast<float>(total) * DRAW_UNIT));
  }
}

}  // namespace strata
