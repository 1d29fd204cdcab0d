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
//   A small top_k: four threads' largest logit, from all blocks, show a threshold that has all of the top_k
//     at or above it.  The entries up to there (the list) go to the first block, which orders them and
//     finishes alone.
//   top_p alone: the row is weighed into DRAW_BINS equal steps of distance from the largest logit.  Few
//     entries up to the step that top_p falls into: a list, as above.  Many: only that step's entries
//     are listed and ordered, which gives K and I.
//   a larger top_k: K and I the same way, from counts.
// What K and I leave is summed by contiguous parts, and the part that the random number falls into is
// summed again entry by entry.
//
// Bound by latency: a step that runs once a row costs its barriers, exchanges and first instructions, and a row of
// 248,320 has ten to thirty of them.  Measured (one GB300, us on the GPU): one row of 32,000 with all cuts
// 7.5 to 8.1, 5 rows of 248,320 10.6 to 11.0, 19 rows of 151,001 with nothing cut 13.7, 64 bfloat16 rows of 248,320 with keys of
// every kind 56 (a large top_k with top_p is the longest), with nothing cut 29.
//
// Reading another block's shared memory runs at about 16 bytes a cycle for an SM and an exchange of two
// values takes about 700 cycles (measured), so the blocks' bins are summed by shares and what all need
// to know is pushed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "strata_device.cuh"

namespace strata {

struct DrawArgs {
  const void* logits;
  int64_t ld;
  int V, chunk;  // chunk: ids of a block, a multiple of 16
  int B;
  bool sorted;   // rows that may take long first (B <= DRAW_SORT_MOST)
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
constexpr float DRAW_STEPS = 64.0f;     // bins per unit of logit: 32 units, beyond which a weight is 0
constexpr int DRAW_COARSE = DRAW_THREADS;  // bins of the maxima, a quarter as fine
constexpr int DRAW_MAXIMA = DRAW_THREADS / 4;  // of a block: the largest logit of each four threads, or (a row in one or
                                               // two blocks) of each thread
constexpr int DRAW_LIST = 2048;
constexpr int DRAW_SORT_MOST = 2048;    // rows whose order every block finds for itself
constexpr int DRAW_PICKED = 512;        // of a warp's part of at most 2048 logits
constexpr int DRAW_PIECES = 4;          // parts a block's ids arrive in
constexpr int DRAW_MAX_CLUSTER = 16;
constexpr float DRAW_REACH = 0.75f;     // below the smallest maximum, of its distance to their mean
constexpr uint32_t NO_KEY = 0u;         // NaN and -inf: below every key that can be chosen
constexpr uint32_t DRAW_DEAD = 0xFFFFFFFFu;  // above every logit's key: a wait for a part of the row ran out
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
  const uint32_t s = (e >> 23) - 107u;  // of a unit in the last place of the 24 bits; negative: downwards
  const uint32_t m = (e & 0x7FFFFFu) | 0x800000u;
  uint32_t up, down, hi;  // a shift by 32 or more (a negative one too) gives 0
  asm("shl.b32 %0, %1, %2;" : "=r"(up) : "r"(m), "r"(s));
  asm("shr.u32 %0, %1, %2;" : "=r"(down) : "r"(m), "r"(0u - s));
  asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(m), "r"(32u - s));
  return static_cast<u64>(hi) << 32 | (up | down);
}
// Sums of such weights, of up to 2^9 of them, in six instructions each: e = A 2^-20 + r, where an addition of 8
// rounded towards zero leaves A in the low bits of the float, and one of 2^-20 does so for r 2^43.
struct DrawSum {
  uint32_t a = 0, b = 0, n = 0;
  __device__ __forceinline__ void add(float dt, uint32_t* top20 = nullptr, uint32_t* low23 = nullptr) {
    const float e = expf(dt), t = __fadd_rz(e, 8.0f);
    const uint32_t ta = __float_as_uint(t), tb = __float_as_uint(__fadd_rz(e - (t - 8.0f), 0x1p-20f));
    a += ta;
    b += tb;
    ++n;
    if (top20 != nullptr) *top20 = ta - 0x41000000u;
    if (low23 != nullptr) *low23 = tb - 0x35800000u;
  }
  __device__ __forceinline__ u64 sum() const {
    return (static_cast<u64>(a - n * 0x41000000u) << 23) + (b - n * 0x35800000u);
  }
};
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
__device__ __forceinline__ void dsmem_st_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct DrawShared {
  uint64_t bars[DRAW_PIECES];
  u64 slot[2][2][DRAW_MAX_CLUSTER];  // what each block told: two turns of two values
  u64 warp[DRAW_WARPS];
  u64 found, found_sum;
  uint32_t listed;                   // entries in the first block's list
  uint32_t local;                    // entries in this block's own
  // Sums of bins in three parts of 15, 15 and 14 bits, so that 2^15 weights add up without a carry.
  // Before: the maxima of all blocks (part 0) and their counts (part 2).  After: this block's own list.
  union alignas(16) {
    uint32_t part[3][DRAW_BINS];
    u64 own[DRAW_LIST];
  };
  // key << 32 | ~index, the order of the chain, descending: the first block's list.  Or, of every block, each
  // warp's part of the row without the logits that no cut reaches: places in it, ascending.
  union {
    alignas(16) u64 list[DRAW_LIST];
    uint16_t picked[DRAW_WARPS][DRAW_PICKED];
  };
  u64 few[DRAW_THREADS];             // entries of one bin, likewise; scratch of the bins' sums before
};
static_assert(offsetof(DrawShared, part) % 16 == 0 && offsetof(DrawShared, list) % 16 == 0, "16-byte accesses");
static_assert(DRAW_MAXIMA * DRAW_MAX_CLUSTER <= DRAW_BINS, "the maxima fit part 0");
static_assert(DRAW_PICKED <= DRAW_THREADS, "find() takes an entry to a thread");

template <typename E>
struct DrawRow {
  static constexpr int VEC = 16 / static_cast<int>(sizeof(E));
  DrawShared* sh;
  const E* ids;        // this block's part of the row in shared memory, NaN beyond its end
  int vecs, base;      // 16-byte vectors of it, its first index
  uint32_t rank, ranks, turn;
  int warp, lane;
  float top;           // the row's largest logit
  bool compact = false;  // this block goes through what it picked, else through all of its part of the row
  int picked = 0;        // of this warp

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
  // The largest of a vector, -inf where it has none; a NaN is passed over.
  __device__ __forceinline__ float vec_max(int v) const {
    const uint4 raw = reinterpret_cast<const uint4*>(ids)[v];
    if constexpr (sizeof(E) == 4) {
      return fmaxf(fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)), fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w))),
                   -INFINITY);
    } else {
      auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
      const __nv_bfloat162 m = __hmax2(__hmax2(two(raw.x), two(raw.y)), __hmax2(two(raw.z), two(raw.w)));
      return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(E) == 4)
      return ids[i];
    else
      return __bfloat162float(ids[i]);
  }
  // f(place in the block's part, logit) of this warp's contiguous part of that (or of what was picked of it).
  __device__ __forceinline__ int part_vecs() const { return (vecs + DRAW_WARPS - 1) / DRAW_WARPS; }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (compact) {
      for (int i = lane; i < picked; i += 32) {
        const int at = sh->picked[warp][i];
        f(at, value(at));
      }
    } else {
      const int to = min(vecs, (warp + 1) * part_vecs());
      for (int v = warp * part_vecs() + lane; v < to; v += 32) vec(v, f);
    }
  }
  // Goes through the warp's part once with f, and picks the logits from `least` (above -inf) on, in their order.
  template <typename F>
  __device__ void pick(float least, F f) {
    const int to = min(vecs, (warp + 1) * part_vecs());
    int n = 0;
    bool fits = true;
    for (int v0 = warp * part_vecs(); v0 < to; v0 += 32) {
      const int v = v0 + lane;
      uint32_t mask = 0;
      if (v < to)
        vec(v, [&](int i, float x) {
          f(i, x);
          mask |= (x >= least ? 1u : 0u) << (i % VEC);
        });
      const int own = __popc(mask), upto = draw_warp_scan(own, lane);
      const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
      fits = fits && n + all <= DRAW_PICKED;
      if (fits)
        for (int at = n + upto - own; mask != 0; mask &= mask - 1) sh->picked[warp][at++] = static_cast<uint16_t>(v * VEC + __ffs(mask) - 1);
      n += all;
    }
    picked = n;
    compact = __syncthreads_and(fits);
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
  template <typename T>
  __device__ T block_scan(T s, T* all = nullptr) {
    const T upto = draw_warp_scan(s, lane);
    T* to = reinterpret_cast<T*>(sh->warp);
    __syncthreads();
    if (lane == 31) to[warp] = upto;
    __syncthreads();
    const T w = draw_warp_scan(lane < DRAW_WARPS ? to[lane] : T(0), lane);
    const T below = __shfl_sync(0xFFFFFFFFu, w, max(warp - 1, 0));
    if (all != nullptr) *all = __shfl_sync(0xFFFFFFFFu, w, DRAW_WARPS - 1);
    return upto + (warp > 0 ? below : T(0));
  }

  // Sums f over the row by contiguous parts, one to a warp (sh->warp holds this block's): the row's
  // sum and what comes before this block.
  template <typename F>
  __device__ u64 parts(F f, u64* before) {
    u64 s = 0;
    each([&](int i, float x) { s += f(base + i, x); });
    return told(s, before);
  }
  // The same of the weights of the distances dist(index, x).
  template <typename F>
  __device__ u64 weight_parts(F dist, u64* before) {
    DrawSum s;  // at most 2^9 logits to a lane
    each([&](int i, float x) { s.add(dist(base + i, x)); });
    return told(s.sum(), before);
  }
  __device__ u64 told(u64 s, u64* before) {
    s = block_sum(s);
    if (warp == 0) tell(s, 0);
    meet();
    return heard_sum(0, before);
  }
  // After parts(f): the first index whose running sum exceeds `target` (< the row's sum); -1 in all threads of
  // the cluster but the one that finds it.  The whole block sums the part again, a vector or an entry to a thread.
  template <typename F>
  __device__ int locate(F f, u64 target, u64 before) {
    int found = -1;
    const u64 mine = lane < DRAW_WARPS ? sh->warp[lane] : 0;
    const u64 upto = before + draw_warp_scan(mine, lane);
    const uint32_t over = __ballot_sync(0xFFFFFFFFu, lane < DRAW_WARPS && upto - mine <= target && target < upto);
    if (over != 0) {  // in this block
      const int hit = __ffs(over) - 1;
      u64 run = __shfl_sync(0xFFFFFFFFu, upto - mine, hit);
      if (compact) {
        // an entry to a thread; entries that were not picked are at the end of a warp's places, and weigh nothing
        if (warp == hit && lane == 0) sh->local = static_cast<uint32_t>(picked);
        __syncthreads();
        const int at = threadIdx.x < sh->local ? sh->picked[hit][threadIdx.x] : -1;
        const u64 own = at >= 0 ? f(base + at, value(at)) : 0;
        const u64 here = run + block_scan(own);
        if (here - own <= target && target < here) found = base + at;
      } else {
        const int to = min(vecs, (hit + 1) * part_vecs());
        for (int v0 = hit * part_vecs(); v0 < to; v0 += DRAW_THREADS) {
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
            found = at;
          }
          run += all;
        }
      }
    }
    return found;
  }
  // The same to all threads of the cluster.
  template <typename F>
  __device__ int find(F f, u64 target, u64 before) {
    __syncthreads();
    if (threadIdx.x == 0) sh->found = 0;
    const int at = locate(f, target, before);
    __syncthreads();
    if (at >= 0) sh->found = static_cast<u64>(at) + 1;
    __syncthreads();
    if (warp == 0) tell(sh->found, 0);
    meet();
    return static_cast<int>(heard_sum(0)) - 1;
  }

  // Distances count from here, so that an infinite largest logit shares step 0 with the greatest finite ones.
  __device__ __forceinline__ float finite_top() const { return fminf(top, 3.402823466e38f); }
  // The step of distance that a logit is in.  Truncated by an addition of 2^23 rounded towards zero: a conversion
  // would share its unit with the exponential.
  __device__ __forceinline__ int bin(float x) const {
    const float d = fminf(fmaxf(finite_top() - x, 0.0f), (DRAW_BINS - 0.5f) / DRAW_STEPS);
    return __float_as_int(__fmaf_rz(d, DRAW_STEPS, 8388608.0f)) & (2 * DRAW_BINS - 1);
  }
  // A logit at or below every entry of the bins before `b`, and above -inf.
  __device__ __forceinline__ float floor_of(int b) const {
    return b >= DRAW_BINS ? -3.402823466e38f : fmaxf(-3.402823466e38f, finite_top() - b * (1.0001f / DRAW_STEPS));
  }

  // Sums f over the row into bins at(x), of the logits from `least` on, and adds the blocks' bins up, each block
  // a share of them: the sum of the whole row, and that of the bins.  cross() then finds the first bin whose
  // inclusive sum reaches `target` >= 1 (one does), and the sum below it.
  struct Bins {
    u64 v[4], below;  // this thread's bins (one to four in a row) and what lies before them
  };
  template <typename F, typename At>
  __device__ u64 weigh(F f, At at, float least, Bins* bins, u64* binned) {
    clear_bins();
    u64 row = 0;
    each([&](int i, float x) {
      const u64 w = f(base + i, x);
      row += w;
      add_if(w != 0 && x >= least, at(x), static_cast<uint32_t>(w) & 0x7FFFu, static_cast<uint32_t>(w >> 15) & 0x7FFFu,
             static_cast<uint32_t>(w >> 30));
    });
    return join(row, bins, binned);
  }
  // The same of the weights of the distances dist(index, x), by distance; `row` is what they sum to in the block,
  // or it is taken of what each() goes through.
  template <typename F>
  __device__ u64 weigh_distances(F dist, float least, const DrawSum* row, Bins* bins, u64* binned) {
    clear_bins();
    DrawSum mine;
    each([&](int i, float x) {
      uint32_t a, b;  // the weight is a 2^23 + b
      mine.add(dist(base + i, x), &a, &b);
      add_if((a | b) != 0 && x >= least, bin(x), b & 0x7FFFu, (b >> 15) | (a & 0x7Fu) << 8, a >> 7);
    });
    return join((row != nullptr ? *row : mine).sum(), bins, binned);
  }
  // And of a count of logits, of which this thread saw `row` in all.
  __device__ u64 count(float least, uint32_t row, Bins* bins, u64* binned) {
    clear_bins();
    each([&](int, float x) { red_if(x >= least && x > -INFINITY, &sh->part[0][bin(x)], 1u); });
    return join(row, bins, binned);
  }
  __device__ __forceinline__ void clear_bins() {
    __syncthreads();
    for (int b = threadIdx.x; b < 3 * DRAW_BINS / 4; b += DRAW_THREADS)
      reinterpret_cast<uint4*>(sh->part)[b] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  // Without a branch, so that a vector's logits go through side by side.
  __device__ __forceinline__ void red_if(bool on, uint32_t* to, uint32_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared.add.u32 [%1], %2;\n\t}" ::"r"(
                     static_cast<uint32_t>(on)),
                 "r"(smem_u32(to)), "r"(v)
                 : "memory");
  }
  __device__ __forceinline__ void add_if(bool on, int b, uint32_t w0, uint32_t w1, uint32_t w2) {
    red_if(on, &sh->part[0][b], w0);
    red_if(on && w1 != 0, &sh->part[1][b], w1);
    red_if(on && w2 != 0, &sh->part[2][b], w2);
  }
  __device__ u64 join(u64 row, Bins* bins, u64* binned) {
    __syncthreads();
    meet();
    const int share = DRAW_BINS / static_cast<int>(ranks);  // 128 to 2048 bins
    const int per = max(1, share / DRAW_THREADS), first = static_cast<int>(rank) * share;
    u64 s = 0;
    if (share >= DRAW_THREADS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bins->v[i] = 0;
        if (i < per)
          for (uint32_t q = 0; q < ranks; ++q) bins->v[i] += bin_of(first + threadIdx.x * per + i, q);
        s += bins->v[i];
      }
    } else {
      // several threads to a bin, four blocks to each
      const int b = threadIdx.x % share, group = threadIdx.x / share, groups = DRAW_THREADS / share;
#pragma unroll
      for (int q = 0; q < 4; ++q) s += bin_of(first + b, min(group * 4 + q, static_cast<int>(ranks) - 1));
      __syncthreads();
      sh->few[threadIdx.x] = s;
      __syncthreads();
      s = 0;
      if (group == 0)
        for (int g = 0; g < groups; ++g) s += sh->few[g * share + b];
      bins->v[0] = s;
      bins->v[1] = bins->v[2] = bins->v[3] = 0;
    }
    u64 here, before;
    const u64 upto = block_scan(s, &here);
    row = block_sum(row);
    if (warp == 0) tell(here, row);
    meet();
    *binned = heard_sum(0, &before);
    bins->below = before + upto - s;
    return heard_sum(1);
  }
  __device__ __forceinline__ u64 bin_of(int b, uint32_t q) const {
    const uint32_t at = dsmem_addr(smem_u32(&sh->part[0][b]), q);
    return static_cast<u64>(draw_ld_u32(at)) + (static_cast<u64>(draw_ld_u32(at + 4 * DRAW_BINS)) << 15) +
           (static_cast<u64>(draw_ld_u32(at + 8 * DRAW_BINS)) << 30);
  }
  __device__ int cross(const Bins& bins, u64 target, u64* under) {
    __syncthreads();
    if (threadIdx.x == 0) sh->found = sh->found_sum = 0;
    __syncthreads();
    const int share = DRAW_BINS / static_cast<int>(ranks), per = max(1, share / DRAW_THREADS);
    u64 run = bins.below;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (run < target && run + bins.v[i] >= target) {
        sh->found = static_cast<u64>(rank * share + threadIdx.x * per + i) + 1;
        sh->found_sum = run;
      }
      run += bins.v[i];
    }
    __syncthreads();
    if (warp == 0) tell(sh->found, sh->found_sum);
    meet();
    *under = heard_sum(1);
    return static_cast<int>(heard_sum(0)) - 1;
  }

  // The key K with sum(key > K) < target <= sum(key >= K) of f, between the keys lo and hi, above which lies
  // `over`, by ever finer equal ranges of keys.
  template <typename F>
  __device__ uint32_t select(F f, uint32_t lo, uint32_t hi, u64 over, u64 target, u64* above) {
    while (lo < hi) {
      int shift = 0;
      while (((hi - lo) >> shift) >= DRAW_BINS) ++shift;
      Bins bins;
      u64 under;
      weigh([&](int i, float x) -> u64 { const uint32_t k = draw_key(x); return k >= lo && k <= hi ? f(i, x) : 0; },
            [&](float x) { return (hi - draw_key(x)) >> shift; }, -INFINITY, &bins, &under);
      const int at = cross(bins, target - over, &under);
      over += under;
      const uint32_t width = 1u << shift, from = hi - (static_cast<uint32_t>(at) << shift);
      lo = from - lo < width ? lo : from - width + 1;
      hi = from;
    }
    *above = over;
    return hi;
  }

  // A barrier of the first `threads` threads (whole warps).
  __device__ __forceinline__ void some_sync(int threads) const { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); }

  // Orders a[0, n) descending; what is beyond n up to a power of two is filled with zeros.
  __device__ void sort(u64* list, int n) {
    int size = 32;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += DRAW_THREADS) list[i] = 0;
    __syncthreads();
    if (size <= DRAW_THREADS) {
      // an entry to a thread: steps of less than a warp go from lane to lane
      if (static_cast<int>(threadIdx.x) < size) {
        u64 a = list[threadIdx.x];
        for (int k = 2; k <= size; k *= 2) {
          for (int j = k / 2; j > 0; j /= 2) {
            u64 b;
            if (j >= 32) {
              some_sync(size);
              list[threadIdx.x] = a;
              some_sync(size);
              b = list[threadIdx.x ^ j];
            } else {
              b = __shfl_xor_sync(0xFFFFFFFFu, a, j);
            }
            const bool larger = ((threadIdx.x & k) == 0) == ((threadIdx.x & j) == 0);  // of the two, this thread keeps it
            a = larger == (a < b) ? b : a;
          }
        }
        some_sync(size);
        list[threadIdx.x] = a;
      }
      __syncthreads();
      return;
    }
    for (int k = 2; k <= size; k *= 2) {
      for (int j = k / 2; j > 0; j /= 2) {
        for (int p = threadIdx.x; p < size / 2; p += DRAW_THREADS) {
          const int i = (p & ~(j - 1)) * 2 + (p & (j - 1));
          const u64 a = list[i], b = list[i + j];
          if ((a < b) == ((i & k) == 0)) {
            list[i] = b;
            list[i + j] = a;
          }
        }
        __syncthreads();
      }
    }
  }

  // Lists the entries from `least` (above -inf) on, in any order, in the first block (the list has the first
  // DRAW_LIST); the row's number of them.  A vector without any costs little more than its largest.  A block lists its own first: an addition in another block's memory takes as long as meet().  Once a
  // row: the list's counter starts at 0.
  __device__ u64 gather(float least) {
    __syncthreads();
    if (threadIdx.x == 0) sh->local = 0;
    __syncthreads();
    for (int v = threadIdx.x; v < vecs; v += DRAW_THREADS) {
      if (!(vec_max(v) >= least)) continue;
      vec(v, [&](int i, float x) {
        if (x >= least) {
          const uint32_t at = atomicAdd(&sh->local, 1u);
          if (at < DRAW_LIST) sh->own[at] = static_cast<u64>(draw_key(x)) << 32 | static_cast<uint32_t>(~(base + i));
        }
      });
    }
    __syncthreads();
    const uint32_t here = sh->local;
    if (here > 0) {  // the same in all threads
      if (threadIdx.x == 0) sh->found = dsmem_atomic_add(dsmem_addr(smem_u32(&sh->listed), 0), here);
      __syncthreads();
      const uint32_t from = static_cast<uint32_t>(sh->found), there = dsmem_addr(smem_u32(&sh->list[0]), 0);
      for (uint32_t i = threadIdx.x; i < min(here, static_cast<uint32_t>(DRAW_LIST)); i += DRAW_THREADS)
        if (from + i < DRAW_LIST) dsmem_st_u64(there + 8 * (from + i), sh->own[i]);
    }
    if (warp == 0) tell(here, 0);
    meet();
    return heard_sum(0);
  }

  // The last entry that a cut leaves: with as few as can be, sum(f) reaches `target`, 1 <= target <= the row's
  // sum.  It is in bin `b`, and `under` is the sum of the bins before.  f is 0 for what earlier cuts took.
  template <typename F>
  __device__ void pin(F f, int b, u64 under, u64 target, uint32_t* K, int* I) {
    const float least = floor_of(b + 1), most = b == 0 ? top : finite_top() - b * (0.9999f / DRAW_STEPS);
    __syncthreads();
    if (threadIdx.x == 0) sh->local = 0;
    __syncthreads();
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    each([&](int i, float x) {
      if (x >= least && x <= most && bin(x) == b && f(base + i, x) != 0) {
        const uint32_t at = atomicAdd(&sh->local, 1u), key = draw_key(x);
        if (at < DRAW_LIST) sh->own[at] = static_cast<u64>(key) << 32 | static_cast<uint32_t>(~(base + i));
        lo = min(lo, key);
        hi = max(hi, key);
      }
    });
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) sh->warp[warp] = static_cast<u64>(lo) << 32 | hi;
    __syncthreads();
    if (warp == 0) {
      const u64 w = lane < DRAW_WARPS ? sh->warp[lane] : 0xFFFFFFFF00000000ull;
      lo = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(w >> 32));
      hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(w));
      tell(sh->local, static_cast<u64>(lo) << 32 | hi);
    }
    meet();
    u64 ahead;
    const u64 entries = heard_sum(0, &ahead);
    const u64 told_keys = static_cast<uint32_t>(lane) < ranks ? heard(1, lane) : 0xFFFFFFFF00000000ull;
    lo = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(told_keys >> 32));
    hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(told_keys));
    if (lo < hi && entries <= DRAW_THREADS) {  // the first block orders them
      const uint32_t there = dsmem_addr(smem_u32(&sh->few[0]), 0) + 8 * static_cast<uint32_t>(ahead), here = sh->local;
      for (uint32_t i = threadIdx.x; i < here; i += DRAW_THREADS) dsmem_st_u64(there + 8 * i, sh->own[i]);
      meet();
      if (rank == 0) {
        sort(sh->few, static_cast<int>(entries));
        const u64 e = threadIdx.x < entries ? sh->few[threadIdx.x] : 0;
        const u64 w = e ? f(static_cast<int>(~static_cast<uint32_t>(e)), draw_val(static_cast<uint32_t>(e >> 32))) : 0;
        const u64 upto = under + block_scan(w);
        if (upto - w < target && upto >= target) sh->found = e;
        __syncthreads();
        if (warp == 0) tell(sh->found, 0);
      }
      meet();
      const u64 e = heard(0, 0);
      *K = static_cast<uint32_t>(e >> 32);
      *I = static_cast<int>(~static_cast<uint32_t>(e));
      return;
    }
    // one logit many times over, or too many: the logit, then how many of it
    u64 above = under;
    const uint32_t key = select(f, lo, hi, under, target, &above);
    const float val = draw_val(key);
    const u64 one = f(-1, val);
    auto same = [&](int i, float x) -> u64 { return x == val && f(i, x) != 0; };
    u64 before;
    parts(same, &before);
    *I = find(same, (target - above + one - 1) / one - 1, before);
    *K = key;
  }
};

// Where rows are more than run at once, those whose keys may take long (a large top_k, top_p without top_k) come
// first, so that the last to start are short: the row that is `at`-th in that order.
__device__ __forceinline__ bool draw_long(const DrawArgs& A, int row, int list_k) {
  const float T = A.temperature != nullptr ? A.temperature[row] : 1.0f, P = A.top_p != nullptr ? A.top_p[row] : 1.0f;
  const int k = A.top_k != nullptr ? A.top_k[row] : 0;
  const bool k_on = k > 0 && k < A.V;
  return T > 0.0f && (k_on ? k > list_k : !(P >= 1.0f));
}
__device__ __forceinline__ int row_in_order(const DrawArgs& A, int at, uint32_t* words) {
  uint32_t ranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int list_k = static_cast<int>(ranks) * (ranks <= 2 ? DRAW_THREADS : DRAW_MAXIMA) / 2, groups = (A.B + 31) / 32;
  for (int g = threadIdx.x >> 5; g < groups; g += DRAW_WARPS) {
    const int row = g * 32 + (threadIdx.x & 31);
    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, row < A.B && draw_long(A, row, list_k));
    if ((threadIdx.x & 31) == 0) words[g] = bits;
  }
  __syncthreads();
  int all = 0;
  for (int g = 0; g < groups; ++g) all += __popc(words[g]);
  const bool is_long = at < all;
  int left = is_long ? at : at - all, row = 0;
  for (int g = 0; g < groups; ++g) {
    uint32_t bits = is_long ? words[g] : ~words[g];
    const int n = __popc(bits);
    if (left >= n) {
      left -= n;
      continue;
    }
    while (left-- > 0) bits &= bits - 1;
    row = g * 32 + __ffs(bits) - 1;
    break;
  }
  __syncthreads();
  return row;
}

// SPINS: looks at a copy before it counts as lost.  A row that lost one gets id -1 and NaN, once its copies are over.
template <typename E, uint32_t SPINS = DRAW_SPINS>
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
  grid_dep_wait();
  grid_dep_launch();
  const int row = A.sorted ? row_in_order(A, blockIdx.x / R.ranks, reinterpret_cast<uint32_t*>(sh->part)) : blockIdx.x / R.ranks;
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
  sh->part[2][threadIdx.x] = 0;  // DRAW_COARSE counts
  __syncthreads();

  // The thread's largest logit and the first vector that has it, then the row's.
  float most = -INFINITY;
  int most_in = -1;
  auto look = [&](int v) {
    const float m = R.vec_max(v);
    if (m > most) {  // not for a vector of NaN and -inf
      most = m;
      most_in = v;
    }
  };
  bool lost = false;
  for (int p = 0; p < DRAW_PIECES && !lost; ++p) {
    const int v0 = min(whole, p * piece), v1 = min(whole, v0 + piece);
    if (v1 > v0) {
      uint32_t spin = 0;
      while (spin < SPINS && !mbar_try_wait(&sh->bars[p], 0)) ++spin;
      lost = spin >= SPINS;
      if (lost) {
        atomicOr(A.errors, 0x08u);  // STRATA_DEVERR_TIMEOUT
        break;
      }
      for (int v = v0 + threadIdx.x; v < v1; v += DRAW_THREADS) look(v);
    }
  }
  if (threadIdx.x == 0 && whole < R.vecs) look(whole);
  // The largest of four threads to all blocks: to each block by 32 threads, four to a store.  Or each thread's own.
  const uint32_t own_key = lost ? DRAW_DEAD : draw_key(most);
  const bool fine = R.ranks <= 2;
  const int row_maxima = static_cast<int>(R.ranks) * (fine ? DRAW_THREADS : DRAW_MAXIMA);
  if (!fine) {
    uint32_t four = max(own_key, __shfl_xor_sync(0xFFFFFFFFu, own_key, 1));
    four = max(four, __shfl_xor_sync(0xFFFFFFFFu, four, 2));
    uint32_t* mine = reinterpret_cast<uint32_t*>(sh->list);
    if ((R.lane & 3) == 0) mine[threadIdx.x / 4] = four;
  }
  __syncthreads();
  cluster_wait();
  if (fine) {
    for (uint32_t q = 0; q < R.ranks; ++q)
      dsmem_st_u32(dsmem_addr(smem_u32(&sh->part[0][R.rank * DRAW_THREADS + threadIdx.x]), q), own_key);
  } else if (static_cast<uint32_t>(R.warp) < R.ranks) {
    const uint4 keys = reinterpret_cast<const uint4*>(sh->list)[R.lane];
    dsmem_st_v4(dsmem_addr(smem_u32(&sh->part[0][R.rank * DRAW_MAXIMA + R.lane * 4]), R.warp), keys.x, keys.y, keys.z, keys.w);
  }
  R.meet();
  uint32_t maxima[DRAW_MAXIMA * DRAW_MAX_CLUSTER / DRAW_THREADS], top_key = NO_KEY;
#pragma unroll
  for (int i = 0; i < DRAW_MAXIMA * DRAW_MAX_CLUSTER / DRAW_THREADS; ++i) {
    const int at = i * DRAW_THREADS + threadIdx.x;
    maxima[i] = at < row_maxima ? sh->part[0][at] : NO_KEY;
    top_key = max(top_key, maxima[i]);
  }
  top_key = __reduce_max_sync(0xFFFFFFFFu, top_key);
  if (R.lane == 0) sh->warp[R.warp] = top_key;
  __syncthreads();
  top_key = __reduce_max_sync(0xFFFFFFFFu, R.lane < DRAW_WARPS ? static_cast<uint32_t>(sh->warp[R.lane]) : NO_KEY);

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
  if (top_key == NO_KEY || top_key == DRAW_DEAD) {
    if (lead && threadIdx.x == 0) answer(-1, __int_as_float(0x7FC00000));
    if (top_key == DRAW_DEAD) {  // no copy of a block may be in flight when it ends
      uint32_t spin = 0;
      for (int p = 0; p < DRAW_PIECES; ++p)
        if (min(whole, (p + 1) * piece) > min(whole, p * piece))
          while (spin < DRAW_SPINS && !mbar_try_wait(&sh->bars[p], 0)) ++spin;
    }
    return;
  }
  if (!(T > 0.0f) || (!(m <= 0.0f) && !(top >= least)) || (p_on && p24 == 0)) {  // the first in order
    uint32_t first = 0xFFFFFFFFu;
    if (own_key == top_key)
      R.vec(most_in, [&](int i, float x) {
        if (x == top) first = min(first, static_cast<uint32_t>(R.base + i));
      });
    first = __reduce_min_sync(0xFFFFFFFFu, first);
    __syncthreads();
    if (R.lane == 0) sh->warp[R.warp] = first;
    __syncthreads();
    if (R.warp == 0) {
      first = __reduce_min_sync(0xFFFFFFFFu, R.lane < DRAW_WARPS ? static_cast<uint32_t>(sh->warp[R.lane]) : 0xFFFFFFFFu);
      R.tell(first, 0);
    }
    R.meet();
    first = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(R.lane) < R.ranks ? static_cast<uint32_t>(R.heard(0, R.lane)) : 0xFFFFFFFFu);
    if (lead && threadIdx.x == 0) answer(static_cast<int>(first), 0.0f);
    return;
  }
  const float inv = 1.0f / T;
  const u64 u24 = u > 0.0f ? static_cast<u64>(fminf(u, 1.0f - 0x1p-24f) * 0x1p24f) : 0ull;
  // fmaxf: an infinite distance by an infinite temperature is no number, and weighs nothing
  auto tempered = [&](float x) { return x == top ? 0.0f : fmaxf((x - top) * inv, -1000.0f); };
  auto flat = [&](float x) { return draw_weight(x == top ? 0.0f : x - top); };  // at temperature 1

  // what is left: logits above `edge`, and of the logits equal to it the indices up to I
  float edge = fmaxf(least, -3.402823466e38f);
  int I = A.V - 1;

  // The first block's list holds all that the cuts leave, and maybe more below: it finishes alone.
  // `share`: top_p's part of the weight, 0 where it is of the list after top_k.
  auto finish = [&](int listed, u64 share) {
    R.sort(sh->list, listed);
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
      kept = per == 1 ? __syncthreads_count(static_cast<int>(under)) : static_cast<int>(R.block_sum(under));
    }
    if (kept <= DRAW_THREADS / 4) {
      // Few: four threads to an entry add up the weights of the entries with lower indices, and all weights,
      // which takes half the time of ordering them.
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < kept) sh->few[threadIdx.x] = draw_weight(tempered(draw_val(static_cast<uint32_t>(sh->list[threadIdx.x] >> 32))));
      __syncthreads();
      const int e = threadIdx.x % (DRAW_THREADS / 4), group = threadIdx.x / (DRAW_THREADS / 4);
      const u64 mine = e < kept ? sh->list[e] : 0;
      u64 lower = 0, whole_sum = 0;
#pragma unroll 4
      for (int j = group; j < kept; j += 4) {
        const u64 w = sh->few[j];
        whole_sum += w;
        lower += static_cast<uint32_t>(sh->list[j]) > static_cast<uint32_t>(mine) ? w : 0;  // ~index
      }
      u64(*part)[2] = reinterpret_cast<u64(*)[2]>(sh->part);
      part[threadIdx.x][0] = lower;
      part[threadIdx.x][1] = whole_sum;
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < kept) {
        for (int g = 1; g < 4; ++g) {
          lower += part[g * (DRAW_THREADS / 4) + e][0];
          whole_sum += part[g * (DRAW_THREADS / 4) + e][1];
        }
        const u64 draw = draw_share(u24, whole_sum);
        if (lower <= draw && lower + sh->few[e] > draw)
          answer(static_cast<int>(~static_cast<uint32_t>(mine)),
                 tempered(draw_val(static_cast<uint32_t>(mine >> 32))) - logf(static_cast<float>(whole_sum) * DRAW_UNIT));
      }
      return;
    }
    // index order: swap the halves, so that the greatest ~index comes first
    __syncthreads();
    for (int i = threadIdx.x; i < kept; i += DRAW_THREADS) sh->list[i] = sh->list[i] << 32 | sh->list[i] >> 32;
    R.sort(sh->list, kept);
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
  auto pinned = [&](uint32_t key, int i) {
    edge = draw_val(key);
    I = i;
  };

  typename DrawRow<E>::Bins bins;
  u64 under, before, binned;
  if (k_on && (A.V <= DRAW_LIST || k <= row_maxima / 2)) {
    float from = edge;
    if (k <= row_maxima / 2) {
      // the bin in which the maxima are k
#pragma unroll
      for (int i = 0; i < DRAW_MAXIMA * DRAW_MAX_CLUSTER / DRAW_THREADS; ++i)
        if (maxima[i] != NO_KEY) atomicAdd(&sh->part[2][R.bin(draw_val(maxima[i])) / (DRAW_BINS / DRAW_COARSE)], 1u);
      if (threadIdx.x == 0) sh->found = DRAW_COARSE;
      __syncthreads();
      const uint32_t here = sh->part[2][threadIdx.x], upto = R.block_scan(here);
      if (upto - here < static_cast<uint32_t>(k) && upto >= static_cast<uint32_t>(k)) sh->found = threadIdx.x;
      __syncthreads();
      // fewer maxima than k: every entry
      from = fmaxf(from, R.floor_of((static_cast<int>(sh->found) + 1) * (DRAW_BINS / DRAW_COARSE)));
    }
    const u64 entries = R.gather(from);
    if (entries <= DRAW_LIST) {
      if (lead) finish(static_cast<int>(entries), 0);
      return;
    }
  }
  // Cuts that leave many mostly leave a small part of the row all the same: it is gone through once, and what
  // is out of their reach is left out from then on.  Where a cut turns out to lie further down, the row is taken
  // whole.  top_p reaches below the smallest of the maxima by DRAW_REACH of its distance to their mean (a
  // twelfth of a normal distribution is left).
  float start = 0.0f;
  if (!k_on && p_on) {
    uint32_t low = 0xFFFFFFFFu;
    float sum = 0.0f, some = 0.0f;
#pragma unroll
    for (int i = 0; i < DRAW_MAXIMA * DRAW_MAX_CLUSTER / DRAW_THREADS; ++i) {
      low = min(low, maxima[i] - 1u);  // NO_KEY: the greatest
      sum += maxima[i] != NO_KEY ? draw_val(maxima[i]) : 0.0f;
      some += maxima[i] != NO_KEY ? 1.0f : 0.0f;
    }
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    sum = warp_sum(sum);
    some = warp_sum(some);
    __syncthreads();
    float* to = reinterpret_cast<float*>(sh->part[2]);
    if (R.lane == 0) {
      sh->warp[R.warp] = low;
      to[R.warp] = sum;
      to[DRAW_WARPS + R.warp] = some;
    }
    __syncthreads();
    low = __reduce_min_sync(0xFFFFFFFFu, R.lane < DRAW_WARPS ? static_cast<uint32_t>(sh->warp[R.lane]) : 0xFFFFFFFFu);
    sum = warp_sum(R.lane < DRAW_WARPS ? to[R.lane] : 0.0f);
    some = warp_sum(R.lane < DRAW_WARPS ? to[DRAW_WARPS + R.lane] : 0.0f);
    const float least_maximum = draw_val(low + 1u);
    start = fmaxf(least_maximum - DRAW_REACH * (sum / some - least_maximum), -3.402823466e38f);
    __syncthreads();
  }
  if (k_on) {
    // The reach of a large top_k, from a sample: each thread's first vector, counted in coarse bins.  It is set a few
    // standard deviations further than the sample's k-th, and to the furthest of the blocks'.
    __syncthreads();
    sh->part[2][threadIdx.x] = 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < R.vecs)
      R.vec(threadIdx.x, [&](int, float x) { R.red_if(x > -INFINITY, &sh->part[2][R.bin(x) / (DRAW_BINS / DRAW_COARSE)], 1u); });
    if (threadIdx.x == 0) sh->found = DRAW_COARSE;
    __syncthreads();
    uint32_t sample;
    const uint32_t here = sh->part[2][threadIdx.x], upto = R.block_scan(here, &sample);
    const float share = static_cast<float>(k) / static_cast<float>(A.V) * static_cast<float>(sample);
    const uint32_t want = static_cast<uint32_t>(share + 3.0f * sqrtf(share) + 3.0f);
    if (upto - here < want && upto >= want) sh->found = threadIdx.x;
    __syncthreads();
    start = R.floor_of((static_cast<int>(sh->found) + 1) * (DRAW_BINS / DRAW_COARSE));
    if (R.warp == 0) R.tell(draw_key(start), 0);
    R.meet();
    start = draw_val(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(R.lane) < R.ranks ? static_cast<uint32_t>(R.heard(0, R.lane)) : 0xFFFFFFFFu));
  }
  if (k_on) {
    auto one = [&](int, float x) -> u64 { return x > -INFINITY; };
    uint32_t row = 0;
    R.pick(start, [&](int, float x) { row += x > -INFINITY; });
    if (static_cast<u64>(k) < R.count(start, row, &bins, &binned)) {
      if (static_cast<u64>(k) > binned) {
        R.compact = false;
        R.count(-INFINITY, row, &bins, &binned);
      }
      const int b = R.cross(bins, k, &under);
      uint32_t key;
      int i;
      R.pin(one, b, under, k, &key, &i);
      if (draw_val(key) >= edge) pinned(key, i);
    } else {
      R.compact = false;
    }
  }
  if (p_on) {
    const float edge0 = edge;
    const int I0 = I;
    auto weight = [&](int i, float x) -> u64 { return x > edge0 || (x == edge0 && i <= I0) ? flat(x) : 0ull; };
    auto distance = [&](int i, float x) {
      const float d = x == top ? 0.0f : x - top;
      return x > edge0 || (x == edge0 && i <= I0) ? d : -1000.0f;
    };
    DrawSum row;
    if (!k_on) {
      if (top <= 3.402823466e38f)
        R.pick(start, [&](int, float x) { row.add(x >= edge0 ? x - top : -1000.0f); });
      else
        R.pick(start, [&](int i, float x) { row.add(distance(R.base + i, x)); });
    }
    const u64 share = draw_share(p24, R.weigh_distances(distance, k_on ? -INFINITY : start, k_on ? nullptr : &row, &bins, &binned));
    if (share > binned) {  // not after a top_k: what it leaves is all there
      R.compact = false;
      R.weigh_distances(distance, -INFINITY, nullptr, &bins, &binned);
    }
    const int b = R.cross(bins, share, &under);
    if (!k_on) {
      // how many entries there are up to b: about as many as maxima, where they are few
      uint32_t few = 0;
#pragma unroll
      for (int i = 0; i < DRAW_MAXIMA * DRAW_MAX_CLUSTER / DRAW_THREADS; ++i)
        few += maxima[i] != NO_KEY && R.bin(draw_val(maxima[i])) <= b;
      if (R.block_sum(few) <= row_maxima / 2) {
        const u64 entries = R.gather(fmaxf(edge, R.floor_of(b + 1)));
        if (entries <= DRAW_LIST) {
          if (lead) finish(static_cast<int>(entries), share);
          return;
        }
        R.compact = false;  // the list lies where the picked were
      }
    }
    uint32_t key;
    int i;
    R.pin(weight, b, under, share, &key, &i);
    pinned(key, i);
  }
  auto left = [&](int i, float x) -> u64 {
    const u64 w = draw_weight(tempered(x));
    return x > edge || (x == edge && i <= I) ? w : 0ull;
  };
  // the same as distances: without infinities a product alone, and without a cut through equal logits one comparison
  auto finite = [&](float x) { return fmaxf((x - top) * inv, -1000.0f); };
  const bool usual = top <= 3.402823466e38f && inv <= 3.402823466e38f;
  const u64 total =
      usual && I == A.V - 1 ? R.weight_parts([&](int, float x) { return x >= edge ? finite(x) : -1000.0f; }, &before)
      : usual ? R.weight_parts([&](int i, float x) { return x > edge || (x == edge && i <= I) ? finite(x) : -1000.0f; }, &before)
              : R.weight_parts([&](int i, float x) { return x > edge || (x == edge && i <= I) ? tempered(x) : -1000.0f; }, &before);
  const int at = R.locate(left, draw_share(u24, total), before);
  if (at >= 0) answer(at, tempered(R.value(at - R.base)) - logf(static_cast<float>(total) * DRAW_UNIT));
}

}  // namespace strata
