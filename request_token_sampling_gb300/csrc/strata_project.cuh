// strata_project.cuh -- a projection shared by all rows plus each row's own low-rank adapter.
//
//   y[t] = sx[t] sw (x[t] w^T) + h[t] b_c^T,   h[t] = g_c sx[t] (x[t] a_c^T),   c = row_adapter[t]
//
// Two kernels.  shrink_kernel (few rows) or inner_kernel (many) computes the inner rows h in 32 bits and writes them, as
// two bfloat16 each, spread out: for each tile of rows and each adapter of the tile a block [tile rows][R] that holds h
// where the row uses that adapter and zeros elsewhere.  project_kernel then treats b of the tile's adapters as
// more of the sum's length: for a tile of 128 outputs and up to 128 rows,
//   base += w[128][64] x[rows][64]^T  over K,     delta += b_j[128][R] spread_j[rows][R]^T  over the adapters j, both parts
// with tcgen05.mma (outputs are its M, rows its N: a tile of w is read once for all rows).  base and delta
// are separate accumulators: 8-bit rows scale base alone, and a product 0 * inf of a broken adapter,
// which falls on other requests' rows in delta, is found there and taken back.  More than 128 rows of
// bfloat16 go to pair_kernel, below.
//
// Few rows are bound by reading w and b from HBM: w comes by TMA through up to 11 stages of shared memory, 112 to 176 KB
// of it on their way to an SM.  Measured (one GB300, us on the GPU, sizes rows x outputs x width):
// 8 x 248,320 x 2,048 bfloat16 with 8 adapters of rank 16 163 to 166 (6.5 TB/s), 64 rows of 8 bits with 32 adapters of
// rank 32 155 (6.8 TB/s), 1 x 32,000 x 1,024 16.6 (4 TB/s: 250 tiles on 152 SMs, and the start).  128 x 32,000 x 2,048
// with 64 adapters of rank 64 takes 96: zeros of the spread inner rows are what L2 has to bring.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "strata_device.cuh"
#include "strata_mma.cuh"

namespace strata {

struct ProjectArgs {
  const void* x;
  const float *x_scale, *w_scale, *adapter_scale;
  const __nv_bfloat16 *a, *b;
  const int32_t* row_adapter;
  __nv_bfloat16* y;
  __nv_bfloat16* spread;  // [tiles][most][upper, lower part][tile rows][R], or the parts outermost (parts_beside())
  int64_t low;            // the lower parts' distance from the upper ones
  int block_rows;         // of one adapter of a tile: its rows, twice where the parts are beside one another
  int32_t* lists;         // per tile: how many adapters, then their ids in ascending order ([1 + tile rows])
  uint32_t* ready;        // per tile: warps that have written their part of its inner rows (pair_kernel)
  uint32_t* errors;
  int64_t ldx, ldy;
  int T, N, K, S, R;
  int most;               // adapters that a tile can have: min(S, T, tile rows)
  int rank_block;         // R is cut into blocks of 64, 32 or 16 (one swizzle line of shared memory)
  int n_tiles, t_tiles, tile_rows;
};

constexpr int PROJ_M = 128;        // outputs of a tile: the accumulator's lanes
constexpr int PROJ_LINE = 128;     // bytes of a row that one stage holds (64 bfloat16 or 128 8-bit elements)
constexpr int PROJ_THREADS = 192;  // warp 0 loads, warp 1 issues the products, warps 2-5 write the tile

// Both parts of up to 64 inner rows are one operand of twice the rows, for the same products' price; 128 would not fit tensor
// memory so, nor would the stages be many.
__host__ __device__ constexpr bool parts_beside(int bn) { return bn <= 64; }
__host__ __device__ constexpr int proj_stage_bytes(int bn) { return (PROJ_M + (parts_beside(bn) ? 2 : 1) * bn) * PROJ_LINE; }
__host__ __device__ constexpr int proj_stages(int bn) { return bn <= 16 ? 11 : bn <= 32 ? 9 : 7; }
// Else: stages of adapters whose inner rows' lower parts share one stage before them, as many as have room there.
__host__ __device__ constexpr int proj_group(int bn) { return proj_stage_bytes(bn) / (bn * PROJ_LINE); }
__host__ __device__ constexpr int proj_smem(int bn) { return proj_stages(bn) * proj_stage_bytes(bn) + 1024 + 512; }

// Instruction descriptor: 32-bit sums, both operands K-major, M = 128 outputs, N = `bn` rows.
// Operand format 1 is bfloat16 in kind::f16, 0 is e4m3 in kind::f8f6f4.
__device__ constexpr uint32_t mma_idesc(bool f8, int bn) {
  return (1u << 4) | (f8 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(bn >> 3) << 17) |
         (static_cast<uint32_t>(PROJ_M >> 4) << 24);
}

// ------------------------------------------------------------------------------ the inner rows
__device__ __forceinline__ float proj_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float proj_f32(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

__device__ __forceinline__ float proj_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// An inner product as two bfloat16 for the tensor cores, 16 of its 24 bits: with one of them alone its rounding
// was a tenth of y's error.  What is not finite is all in the upper part.
__device__ __forceinline__ void proj_split(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float rest = v - __bfloat162float(hi);
  lo = __float2bfloat16_rn(fabsf(rest) < __int_as_float(0x7F800000) ? rest : 0.0f);
}

// The adapters of a tile of rows, as the bits of 32 words, and whether a row has none; the whole block.
struct TileAdapters {
  uint32_t bits[32], none;
};
__device__ __forceinline__ void tile_adapters(const ProjectArgs& A, int t0, int rows, TileAdapters* used) {
  if (threadIdx.x < 32) used->bits[threadIdx.x] = 0;
  if (threadIdx.x == 0) used->none = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < rows; i += blockDim.x) {
    const int c = A.row_adapter[t0 + i];
    if (c >= 0 && c < A.S)
      atomicOr(&used->bits[c >> 5], 1u << (c & 31));
    else
      used->none = 1;
  }
  __syncthreads();
}
// A tile's list: how many adapters it has (and whether its rows differ in them), then their ids.
constexpr int32_t LIST_COUNT = 0xFFFF, LIST_MIXED = 1 << 30;
__device__ __forceinline__ void write_list(const ProjectArgs& A, int tile, int tile_rows, const TileAdapters& used) {
  int32_t* list = A.lists + static_cast<int64_t>(tile) * (tile_rows + 1);
  int n = 0;
  for (int w = 0; w < 32; ++w)
    for (uint32_t bits = used.bits[w]; bits; bits &= bits - 1) list[1 + n++] = w * 32 + __ffs(bits) - 1;
  list[0] = n | (n > 1 || (n == 1 && used.none) ? LIST_MIXED : 0);
}

// Eight warps: the block of row t takes eight of its inner products, one to a warp.  Bound by a few loads one after
// another (8 rows x 2,048, 8 adapters of rank 16: 9.6 us cold and alone, most of it beside the first tiles).
template <typename E>
__global__ void __launch_bounds__(256) shrink_kernel(ProjectArgs A, int tile_rows) {
  grid_dep_wait();    // first: the next kernel relies on what was before this one being done
  grid_dep_launch();
  __shared__ TileAdapters used;
  const int t = blockIdx.x, tile = t / tile_rows, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + warp;
  const int t0 = tile * tile_rows;
  tile_adapters(A, t0, min(tile_rows, A.T - t0), &used);
  const int c = A.row_adapter[t];
  const bool mine = c >= 0 && c < A.S;
  int count = 0, at = -1;
  for (int w = 0; w < 32; ++w) {
    if (mine && w == c >> 5) at = count + __popc(used.bits[w] & ((1u << (c & 31)) - 1u));
    count += __popc(used.bits[w]);
  }
  if (t == t0 && blockIdx.y == 0 && threadIdx.x == 0) write_list(A, tile, tile_rows, used);
  float s = 0.0f;
  if (mine) {
    const E* x = static_cast<const E*>(A.x) + t * A.ldx;
    const __nv_bfloat16* a = A.a + (static_cast<int64_t>(c) * A.R + r) * A.K;
    for (int k = lane * 8; k < A.K; k += 256) {
      __align__(16) __nv_bfloat16 av[8];
      __align__(16) E xv[8];
      *reinterpret_cast<uint4*>(av) = *reinterpret_cast<const uint4*>(a + k);
      if constexpr (sizeof(E) == 2)
        *reinterpret_cast<uint4*>(xv) = *reinterpret_cast<const uint4*>(x + k);
      else
        *reinterpret_cast<uint2*>(xv) = *reinterpret_cast<const uint2*>(x + k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(proj_f32(xv[i]), proj_f32(av[i]), s);
    }
    s = proj_warp_sum(s);
    s = A.adapter_scale[c] * ((A.x_scale != nullptr ? A.x_scale[t] : 1.0f) * s);
  }
  __nv_bfloat16 hi, lo;
  proj_split(s, hi, lo);
  const __nv_bfloat16 zero = __float2bfloat16_rn(0.0f);
  for (int j = lane; j < count; j += 32) {
    __nv_bfloat16* h = A.spread + ((static_cast<int64_t>(tile) * A.most + j) * A.block_rows + (t - t0)) * A.R + r;
    h[0] = j == at ? hi : zero;
    h[A.low] = j == at ? lo : zero;
  }
}

// Many rows: the same inner rows on the tensor cores.  A cluster of INNER_SPLIT blocks takes 128 of the
// inner products (the matrices a of a tile's adapters one below another) for all rows of a tile, each
// block a part of K, and adds the parts up in rank order (few tiles have work, so K is split eight ways).  8-bit rows
// are widened to bfloat16 (exactly) on their way to the operand by the four warps that later write the result.
// Bound by latency: start, a short loop, two cluster barriers (cold, us: 64 8-bit rows x 2,048 with 32 adapters of rank 32
// 13.6, 2,180 x 1,776 with 8 22.4).
constexpr int INNER_SPLIT = 8, INNER_ROWS = 128;
constexpr int INNER_A = PROJ_M * PROJ_LINE;
__host__ __device__ constexpr int inner_stages(bool f8) { return f8 ? 3 : 4; }
__host__ __device__ constexpr int inner_stage_bytes(bool f8) { return INNER_A + INNER_ROWS * PROJ_LINE * (f8 ? 3 : 2) / 2; }
__host__ __device__ constexpr int inner_smem(bool f8) { return inner_stages(f8) * inner_stage_bytes(f8) + 1024 + 512; }

struct InnerBars {
  uint64_t full[4], wide[4], empty[4], done, drained;
  uint32_t tmem, dead;
  TileAdapters used;
};

template <bool F8>
__global__ void __launch_bounds__(PROJ_THREADS, 1)
    inner_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mx,
                 const __grid_constant__ ProjectArgs A, int groups, int box_rows) {
  constexpr int STAGES = inner_stages(F8), STAGE = inner_stage_bytes(F8), X = INNER_A, RAW = INNER_A + INNER_ROWS * PROJ_LINE;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  InnerBars* B = reinterpret_cast<InnerBars*>(smem + STAGES * STAGE);
  const int warp = warp_index(), lane = threadIdx.x & 31, rows_max = A.tile_rows;
  const uint32_t rank = cluster_ctarank();
  const int unit = blockIdx.x / INNER_SPLIT, tile = unit / groups, first = unit % groups;
  volatile uint32_t* dead = &B->dead;
  const uint32_t bit = 0x08u;  // STRATA_DEVERR_TIMEOUT
  grid_dep_wait();    // first: the next kernel relies on what was before this one being done
  grid_dep_launch();

  const int t0 = tile * rows_max, rows = min(rows_max, A.T - t0);
  tile_adapters(A, t0, rows, &B->used);
  int count = 0;
  for (int w = 0; w < 32; ++w) count += __popc(B->used.bits[w]);
  auto adapter = [&](int j) {  // the j-th of them
    for (int w = 0; w < 32; ++w) {
      uint32_t bits = B->used.bits[w];
      const int n = __popc(bits);
      if (j >= n) {
        j -= n;
        continue;
      }
      while (j-- > 0) bits &= bits - 1;
      return w * 32 + __ffs(bits) - 1;
    }
    return 0;
  };
  if (first == 0 && rank == 0 && threadIdx.x == 0) write_list(A, tile, rows_max, B->used);
  const int stack = count * A.R;               // the adapters' matrices one below another
  if (first * PROJ_M >= stack) return;         // the whole cluster

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->wide[i], 128);
      mbar_init(&B->empty[i], 1);
    }
    mbar_init(&B->done, 1);
    mbar_init(&B->drained, 1);
    B->dead = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B->tmem)), "r"(static_cast<uint32_t>(INNER_ROWS)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;
  const int k_stages = (A.K + 63) / 64;
  const int from = static_cast<int>(static_cast<int64_t>(k_stages) * rank / INNER_SPLIT);
  const int to = static_cast<int>(static_cast<int64_t>(k_stages) * (rank + 1) / INNER_SPLIT);
  uint32_t begun = 0, turn = 0;  // stages before this group
  Ring<STAGES> ring;             // of the loading and of the issuing warp

  for (int q0 = first * PROJ_M; q0 < stack; q0 += groups * PROJ_M, begun += to - from, ++turn) {
    const int mine = min(PROJ_M, stack - q0);
    if (warp == 0) {
      const int boxes = (mine + box_rows - 1) / box_rows;
      int at_row[PROJ_M / 16];
      for (int i = 0; i < boxes; ++i) {
        const int q = q0 + i * box_rows;
        at_row[i] = adapter(q / A.R) * A.R + q % A.R;
      }
      const uint32_t bytes = static_cast<uint32_t>(boxes * box_rows * PROJ_LINE + rows_max * (F8 ? 64 : PROJ_LINE));
      bool alive = true;
      for (int s = from; s < to; ++s, ring.next()) {
        if (ring.begun >= STAGES && !proj_wait(&B->empty[ring.slot], ring.phase ^ 1u, dead, A.errors, bit)) {
          alive = false;
          break;
        }
        const uint32_t at = smem_u32(smem + ring.slot * STAGE), bar = smem_u32(&B->full[ring.slot]);
        if (elect_one()) {
          mbar_arrive_expect_tx(&B->full[ring.slot], bytes);
          for (int i = 0; i < boxes; ++i) tma_2d(at + i * box_rows * PROJ_LINE, &ma, s * 64, at_row[i], bar);
          tma_2d(at + (F8 ? RAW : X), &mx, s * 64, t0, bar);
        }
      }
      if (!alive) ring.drain(B->full);
    } else if (warp == 1) {
      bool alive = true, add = false;
      const uint32_t idesc = mma_idesc(false, rows_max);
      for (int s = from; s < to; ++s, ring.next()) {
        if (!proj_wait(&B->full[ring.slot], ring.phase, dead, A.errors, bit) ||
            (F8 && !proj_wait(&B->wide[ring.slot], ring.phase, dead, A.errors, bit))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = smem_u32(smem + ring.slot * STAGE);
        const uint64_t da = mma_desc(at, PROJ_LINE), db = mma_desc(at + X, PROJ_LINE);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mma<false>(tmem, da + 2 * i, db + 2 * i, idesc, add || i > 0);
          mma_commit(&B->empty[ring.slot]);
        }
        add = true;
      }
      if (elect_one()) mma_commit(alive ? &B->done : &B->drained);
      if (!alive)
        for (uint32_t spin = 0; spin < PROJ_SPINS && !mbar_try_wait(&B->drained, 0); ++spin) {
        }
    } else if (warp >= 2) {
      if constexpr (F8) {
        uint32_t it = begun;
        for (int s = from; s < to; ++s, ++it) {
          const uint32_t slot = it % STAGES;
          if (!proj_wait(&B->full[slot], (it / STAGES) & 1, dead, A.errors, bit)) break;
          uint8_t* stage = smem + slot * STAGE;
          for (int r = threadIdx.x - 64; r < rows_max; r += 128) {
            const uint4* in = reinterpret_cast<const uint4*>(stage + RAW + r * 64);
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 16 elements: two 16-byte pieces of the operand's line
              const uint4 v = in[c];
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
                const __nv_bfloat162 b = __float22bfloat162_rn(__half22float2(__half2(h)));
                o[i] = *reinterpret_cast<const uint32_t*>(&b);
              }
              uint8_t* to_line = stage + X + r * PROJ_LINE;
              *reinterpret_cast<uint4*>(to_line + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(to_line + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&B->wide[slot]);
        }
      }
      const uint32_t quarter = warp & 3;
      const bool ok = proj_wait(&B->done, turn & 1, dead, A.errors, bit);
      if (ok) {
        tc_fence_after();
        float* sums = reinterpret_cast<float*>(smem);  // [row][product]: every stage is free by now
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
          float v[16] = {};
          if (to > from) tmem_ld16(tmem + (quarter << 21) + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) sums[(c + i) * PROJ_M + quarter * 32 + lane] = v[i];
        }
        tc_fence_before();
      }
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (*dead == 0u) {
      // four products of a row to a thread, the same four for all its rows; a row's sums of other adapters
      // are not looked at
      constexpr int FOURS = PROJ_M / 4, GO = INNER_SPLIT * PROJ_THREADS / FOURS;
      const uint32_t own = smem_u32(smem);
      const int id = static_cast<int>(rank) * PROJ_THREADS + threadIdx.x, m = id % FOURS * 4, q = q0 + m, j = q / A.R;
      if (q < stack) {
        const int c = adapter(j);
        const float by = A.adapter_scale[c];
        __nv_bfloat16* to_row = A.spread + (static_cast<int64_t>(tile) * A.most + j) * A.block_rows * A.R + q % A.R;
        for (int t = id / FOURS; t < rows; t += GO) {
          __align__(8) __nv_bfloat16 hi[4], lo[4];
          *reinterpret_cast<uint2*>(hi) = *reinterpret_cast<uint2*>(lo) = make_uint2(0, 0);
          if (A.row_adapter[t0 + t] == c) {
            float4 v[INNER_SPLIT];
#pragma unroll
            for (uint32_t i = 0; i < INNER_SPLIT; ++i) v[i] = dsmem_ld_v4(dsmem_addr(own, i) + (t * PROJ_M + m) * 4);
            float4 sum = v[0];
#pragma unroll
            for (uint32_t i = 1; i < INNER_SPLIT; ++i) {
              sum.x += v[i].x;
              sum.y += v[i].y;
              sum.z += v[i].z;
              sum.w += v[i].w;
            }
            const float sx = A.x_scale != nullptr ? A.x_scale[t0 + t] : 1.0f;
            const float four[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) proj_split(by * (sx * four[i]), hi[i], lo[i]);
          }
          *reinterpret_cast<uint2*>(to_row + t * A.R) = *reinterpret_cast<const uint2*>(hi);
          *reinterpret_cast<uint2*>(to_row + t * A.R + A.low) = *reinterpret_cast<const uint2*>(lo);
        }
      }
    }
    // the next group's copies overwrite the sums that generic stores wrote and the others read
    fence_proxy_async_smem();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
  }
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(INNER_ROWS)) : "memory");
  }
}

// ------------------------------------------------------------------------------ the products
template <int BN>
struct ProjBars {
  uint64_t full[proj_stages(BN)], empty[proj_stages(BN)], done[2], freed[2], drained;
  uint32_t tmem, dead;
};

// Where a row's inner row lies in the spread of its tile, or -1 for a row without an adapter.
__device__ __forceinline__ int64_t proj_place(const ProjectArgs& A, int tile, int tile_rows, int t) {
  const int c = A.row_adapter[t];
  if (c < 0 || c >= A.S) return -1;
  const int32_t* list = A.lists + static_cast<int64_t>(tile) * (tile_rows + 1);
  int j = 0;  // its adapter's place among the list's ascending ids
  for (int to = (list[0] & LIST_COUNT) - 1; j < to;) {
    const int at = (j + to) / 2;
    if (list[1 + at] < c)
      j = at + 1;
    else
      to = at;
  }
  return ((static_cast<int64_t>(tile) * A.most + j) * A.block_rows + (t - tile * tile_rows)) * A.R;
}
// d + sum of eight (h + l) b
__device__ __forceinline__ void proj_add8(const uint4& h, const uint4& l, const uint4& b, float& d) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    d = fmaf(__uint_as_float(hw[e] << 16) + __uint_as_float(lw[e] << 16), __uint_as_float(bw[e] << 16), d);
    d = fmaf(__uint_as_float(hw[e] & 0xFFFF0000u) + __uint_as_float(lw[e] & 0xFFFF0000u), __uint_as_float(bw[e] & 0xFFFF0000u), d);
  }
}
// delta for one output and row from its own adapter alone, where the tile's sum is not finite.
__device__ __noinline__ float proj_own_delta(const ProjectArgs& A, int64_t place, int t, int n) {
  const uint4 *h = reinterpret_cast<const uint4*>(A.spread + place), *l = reinterpret_cast<const uint4*>(A.spread + A.low + place);
  const uint4* b = reinterpret_cast<const uint4*>(A.b + (static_cast<int64_t>(A.row_adapter[t]) * A.N + n) * A.R);
  float d = 0.0f;
#pragma unroll 4
  for (int i = 0; i < A.R / 8; ++i) {
    proj_add8(__ldcg(h + i), __ldcg(l + i), b[i], d);
  }
  return d;
}

// The same of the rows t .. t + 3, where `bad` has their bits; `some`: of any lane.  The rows go side by side, so that
// their loads do not wait for one another: one row after another took 1.3 us each.
__device__ __forceinline__ void proj_own_deltas(const ProjectArgs& A, int tile, int tile_rows, int t, int n, uint32_t bad,
                                                uint32_t some, float* d) {
  const int lane = threadIdx.x & 31;
  const int64_t place = lane < 4 && (some >> lane & 1u) ? proj_place(A, tile, tile_rows, t + lane) : -1;  // of row t + lane
  const int c = place >= 0 ? A.row_adapter[t + lane] : -1;
  const uint4 *h[4], *b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t its = __shfl_sync(0xFFFFFFFFu, place, i);
    const int ci = __shfl_sync(0xFFFFFFFFu, c, i);
    if (bad >> i & 1u) d[i] = 0.0f;
    if (ci < 0) bad &= ~(1u << i);
    h[i] = reinterpret_cast<const uint4*>(A.spread + max(its, static_cast<int64_t>(0)));
    b[i] = reinterpret_cast<const uint4*>(A.b + (static_cast<int64_t>(max(ci, 0)) * A.N + n) * A.R);
  }
#pragma unroll 1
  for (int r = 0; r < A.R / 8; ++r) {
    uint4 hv[4], lv[4], bv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (bad >> i & 1u) {
        hv[i] = __ldcg(h[i] + r);
        lv[i] = __ldcg(h[i] + A.low / 8 + r);
        bv[i] = b[i][r];
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (bad >> i & 1u) proj_add8(hv[i], lv[i], bv[i], d[i]);
  }
  __syncwarp();
}

template <int BN, bool F8>
__device__ __forceinline__ void proj_write(const ProjectArgs& A, int t_tile, int t, int n, float sw, float base, float delta,
                                           bool adapters) {
  float v = base;
  if constexpr (F8) v *= A.x_scale[t] * sw;
  if (adapters) {
    if (!(fabsf(delta) < __int_as_float(0x7F800000))) {
      const int64_t place = proj_place(A, t_tile, BN, t);
      delta = place < 0 ? 0.0f : proj_own_delta(A, place, t, n);
    }
    v += delta;
  }
  A.y[t * A.ldy + n] = __float2bfloat16_rn(v);
}

// A block per SM goes through tiles (SPLIT false), or a cluster's blocks share one tile's stages and
// join their sums through shared memory in rank order (SPLIT: few tiles, all of the GPU to be kept busy).
template <int BN, bool F8, bool SPLIT>
__global__ void __launch_bounds__(PROJ_THREADS, 1)
    project_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                   const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mh,
                   const __grid_constant__ ProjectArgs A) {
  constexpr int STAGES = proj_stages(BN), STAGE = proj_stage_bytes(BN);
  constexpr int ELEMS = F8 ? 128 : 64;  // of the sum's length in one stage
  constexpr bool BESIDE = parts_beside(BN);
  constexpr int H_ROWS = BESIDE ? 2 * BN : BN, GROUP = proj_group(BN);
  constexpr uint32_t BUF_COLS = BN + H_ROWS;  // a tile's base and delta; there are two
  constexpr uint32_t TMEM_COLS = BN == 16 ? 128 : BN == 32 ? 256 : 512;
  static_assert(2 * BUF_COLS <= TMEM_COLS, "two tiles in tensor memory");
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  ProjBars<BN>* B = reinterpret_cast<ProjBars<BN>*>(smem + STAGES * STAGE);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  volatile uint32_t* dead = &B->dead;
  const uint32_t bit = 0x08u;  // STRATA_DEVERR_TIMEOUT

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->done[i], 1);
      mbar_init(&B->freed[i], 4);
    }
    mbar_init(&B->drained, 1);
    B->dead = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B->tmem)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  if (A.S == 0) grid_dep_wait();  // nothing ran before it in this call
  grid_dep_launch();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;

  const int k_stages = (A.K + ELEMS - 1) / ELEMS;
  const int blocks = A.S > 0 ? A.R / A.rank_block : 0;          // rank blocks of an adapter
  const int per_stage = A.S > 0 ? 64 / A.rank_block : 1;        // rank blocks in a stage
  const uint32_t line = static_cast<uint32_t>(A.rank_block) * 2;
  uint32_t rank = 0, ranks = 1;
  if constexpr (SPLIT) {
    rank = cluster_ctarank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  }
  const int first = SPLIT ? blockIdx.x / ranks : blockIdx.x;
  const int step = SPLIT ? A.n_tiles * A.t_tiles : gridDim.x;
  const int tiles = A.n_tiles * A.t_tiles;
  auto adapters_of = [&](int t_tile) {
    return A.S > 0 ? *(A.lists + static_cast<int64_t>(t_tile) * (BN + 1)) & LIST_COUNT : 0;
  };
  // what a block takes of `all` stages: of the base's and, on its own, of the adapters' (whose number is known
  // only when the previous kernel is done: `lists` and `spread` are its outputs)
  auto share = [&](int all, uint32_t of, int& from, int& to) {
    from = SPLIT ? static_cast<int>(static_cast<int64_t>(all) * of / ranks) : 0;
    to = SPLIT ? static_cast<int>(static_cast<int64_t>(all) * (of + 1) / ranks) : all;
  };
  auto stages_of = [&](int subs) { return (subs + per_stage - 1) / per_stage; };
  auto wait_shrink = [&]() {
    if (A.S > 0) grid_dep_wait();
  };

  if (warp == 0) {
    Ring<STAGES> ring;
    bool alive = true, waited = false;
    auto room = [&]() {  // in the next stage
      if (ring.begun >= STAGES && !proj_wait(&B->empty[ring.slot], ring.phase ^ 1u, dead, A.errors, bit)) alive = false;
      return alive;
    };
    for (int tile = first; tile < tiles && alive; tile += step) {
      const int n0 = tile / A.t_tiles * PROJ_M, t_tile = tile % A.t_tiles;
      int from, to;
      share(k_stages, rank, from, to);
      for (int s = from; s < to && room(); ++s, ring.next()) {
        const uint32_t at = smem_u32(smem + ring.slot * STAGE), bar = smem_u32(&B->full[ring.slot]);
        if (elect_one()) {
          mbar_arrive_expect_tx(&B->full[ring.slot], (PROJ_M + BN) * PROJ_LINE);
          tma_2d(at, &mw, s * ELEMS, n0, bar);
          tma_2d(at + PROJ_M * PROJ_LINE, &mx, s * ELEMS, t_tile * BN, bar);
        }
      }
      if (A.S == 0 || !alive) continue;
      if (!waited) wait_shrink(), waited = true;  // now what the adapters add
      const int subs = adapters_of(t_tile) * blocks;
      share(stages_of(subs), rank, from, to);
      const int32_t* ids = A.lists + static_cast<int64_t>(t_tile) * (BN + 1) + 1;
      for (int s = from; s < to && room(); ++s, ring.next()) {
        if (!BESIDE && (s - from) % GROUP == 0) {  // the lower parts of the next stages' inner rows
          const uint32_t at = smem_u32(smem + ring.slot * STAGE), bar = smem_u32(&B->full[ring.slot]);
          const int sub0 = s * per_stage, n = min(min(GROUP, to - s) * per_stage, subs - sub0);
          if (elect_one()) {
            mbar_arrive_expect_tx(&B->full[ring.slot], static_cast<uint32_t>(n) * BN * line);
            for (int i = 0; i < n; ++i) {
              const int j = (sub0 + i) / blocks, rb = (sub0 + i) % blocks;
              tma_2d(at + i * BN * line, &mh, rb * A.rank_block, ((A.t_tiles + t_tile) * A.most + j) * BN, bar);
            }
          }
          ring.next();
          if (!room()) break;
        }
        const uint32_t at = smem_u32(smem + ring.slot * STAGE), bar = smem_u32(&B->full[ring.slot]);
        const int sub0 = s * per_stage, n = min(per_stage, subs - sub0);
        if (elect_one()) {
          mbar_arrive_expect_tx(&B->full[ring.slot], static_cast<uint32_t>(n) * (PROJ_M + H_ROWS) * line);
          for (int i = 0; i < n; ++i) {
            const int j = (sub0 + i) / blocks, rb = (sub0 + i) % blocks;
            tma_3d(at + i * PROJ_M * line, &mb, rb * A.rank_block, n0, ids[j], bar);
            tma_2d(at + PROJ_M * PROJ_LINE + i * H_ROWS * line, &mh, rb * A.rank_block, (t_tile * A.most + j) * H_ROWS, bar);
          }
        }
      }
    }
    if (!alive) ring.drain(B->full);
  } else if (warp == 1) {
    Ring<STAGES> ring;
    uint32_t turn = 0;
    bool alive = true, waited = false;
    auto landed = [&]() {  // the next stage
      if (!proj_wait(&B->full[ring.slot], ring.phase, dead, A.errors, bit)) alive = false;
      tc_fence_after();
      return alive;
    };
    for (int tile = first; tile < tiles && alive; tile += step, ++turn) {
      const int t_tile = tile % A.t_tiles;
      const uint32_t buf = turn & 1, base = tmem + buf * BUF_COLS, delta = base + BN;
      if (turn >= 2 && !proj_wait(&B->freed[buf], (turn / 2 + 1) & 1, dead, A.errors, bit)) {
        alive = false;
        break;
      }
      tc_fence_after();
      int from, to;
      share(k_stages, rank, from, to);
      for (int s = from; s < to && landed(); ++s, ring.next()) {
        const uint32_t at = smem_u32(smem + ring.slot * STAGE);
        const uint64_t da = mma_desc(at, PROJ_LINE), db = mma_desc(at + PROJ_M * PROJ_LINE, PROJ_LINE);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)  // 32 bytes of each row at a time
            mma<F8>(base, da + 2 * i, db + 2 * i, mma_idesc(F8, BN), s > from || i > 0);
          mma_commit(&B->empty[ring.slot]);
        }
      }
      if (A.S > 0 && alive) {
        if (!waited) wait_shrink(), waited = true;
        const int subs = adapters_of(t_tile) * blocks;
        share(stages_of(subs), rank, from, to);
        bool add = false;
        uint32_t low = 0;
        for (int s = from; s < to && landed(); ++s, ring.next()) {
          if (!BESIDE && (s - from) % GROUP == 0) {
            low = ring.slot;
            ring.next();
            if (!landed()) break;
          }
          const uint32_t at = smem_u32(smem + ring.slot * STAGE), at_h = at + PROJ_M * PROJ_LINE;
          const uint32_t at_low = smem_u32(smem + low * STAGE) + (s - from) % GROUP * per_stage * BN * line;
          const int n = min(per_stage, subs - s * per_stage);
          if (elect_one()) {
            for (int i = 0; i < n; ++i) {
              const uint64_t da = mma_desc(at + i * PROJ_M * line, line);
              const uint64_t db = mma_desc(at_h + i * H_ROWS * line, line), dl = mma_desc(at_low + i * BN * line, line);
              for (int q = 0; q < A.rank_block / 16; ++q) {
                mma<false>(delta, da + 2 * q, db + 2 * q, mma_idesc(false, H_ROWS), add || i > 0 || q > 0);
                if constexpr (!BESIDE) mma<false>(delta, da + 2 * q, dl + 2 * q, mma_idesc(false, BN), true);
              }
            }
            mma_commit(&B->empty[ring.slot]);
            if (!BESIDE && ((s - from) % GROUP == GROUP - 1 || s + 1 == to)) mma_commit(&B->empty[low]);
          }
          add = true;
        }
      }
      if (alive && elect_one()) mma_commit(&B->done[buf]);
    }
    if (!alive) {  // the products in flight end before the block gives its tensor memory back
      if (elect_one()) mma_commit(&B->drained);
      for (uint32_t spin = 0; spin < PROJ_SPINS && !mbar_try_wait(&B->drained, 0); ++spin) {
      }
    }
  } else if (warp >= 2) {
    const uint32_t quarter = warp & 3;  // the 32 lanes of tensor memory that this warp may read
    uint32_t turn = 0;
    wait_shrink();
    for (int tile = first; tile < tiles; tile += step, ++turn) {
      const int t_tile = tile % A.t_tiles, t0 = t_tile * BN, n = tile / A.t_tiles * PROJ_M + quarter * 32 + lane;
      const uint32_t buf = turn & 1;
      const int adapters = adapters_of(t_tile);
      const bool ok = proj_wait(&B->done[buf], (turn / 2) & 1, dead, A.errors, bit);
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + buf * BUF_COLS + (quarter << 21);
      // a delta's columns, both parts
      auto load_delta = [&](int c, float(&v)[16]) {
        tmem_ld16(base + BN + c, v);
        if constexpr (BESIDE) {
          float low[16];
          tmem_ld16(base + 2 * BN + c, low);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += low[i];
        }
      };
      const int rows = min(BN, A.T - t0);
      if constexpr (!SPLIT) {
        // few instructions an output: a warp writes its 32 outputs of all rows while the next tile is summed, and
        // the last tile's writing is waited for
        const float sw = F8 && n < A.N ? A.w_scale[n] : 1.0f;
        __nv_bfloat16* y = A.y + t0 * A.ldy + n;
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
          float vb[16], vd[16] = {};
          tmem_ld16(base + c, vb);
          if (adapters > 0) load_delta(c, vd);
          const float scale = F8 && lane < 16 && c + lane < rows ? A.x_scale[t0 + c + lane] : 0.0f;  // of row c + lane
          tmem_wait_ld();
          if (adapters > 0) {
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) bad |= fabsf(vd[i]) < __int_as_float(0x7F800000) ? 0u : 1u << i;
            if (n >= A.N) bad = 0;
            if (rows - c < 16) bad &= (1u << (rows - c)) - 1u;
            if (const uint32_t some = __reduce_or_sync(0xFFFFFFFFu, bad); some != 0) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                if (some >> i & 15u) proj_own_deltas(A, t_tile, BN, t0 + c + i, n, bad >> i & 15u, some >> i & 15u, vd + i);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if constexpr (F8) vb[i] *= __shfl_sync(0xFFFFFFFFu, scale, i) * sw;
            vb[i] += vd[i];
          }
          if (n < A.N) {
            if (rows - c >= 16) {
#pragma unroll
              for (int i = 0; i < 16; ++i, y += A.ldy) *y = __float2bfloat16_rn(vb[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i, y += A.ldy)
                if (c + i < rows) *y = __float2bfloat16_rn(vb[i]);
            }
          }
        }
      } else {
        // this block's sums to its own shared memory: [base, delta][row][output]
        int from, to;
        share(k_stages, rank, from, to);
        const bool has_base = to > from;
        share(stages_of(adapters * blocks), rank, from, to);
        const bool has_delta = to > from;
        float* mine = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
          float vb[16] = {}, vd[16] = {};
          if (has_base) tmem_ld16(base + c, vb);
          if (has_delta) load_delta(c, vd);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            mine[(c + i) * PROJ_M + quarter * 32 + lane] = vb[i];
            if (has_delta) mine[(BN + c + i) * PROJ_M + quarter * 32 + lane] = vd[i];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->freed[buf]);
    }
  }
  __syncthreads();
  if constexpr (SPLIT) {
    cluster_arrive();
    cluster_wait();
    if (*dead == 0u) {
      const int tile = first, t_tile = tile % A.t_tiles, t0 = t_tile * BN, n0 = tile / A.t_tiles * PROJ_M;
      const int rows = min(BN, A.T - t0), adapters = adapters_of(t_tile);
      // four outputs of a row to a thread; delta lies with the ranks that had stages of it
      constexpr int FOURS = PROJ_M / 4, MOST = 8;
      const uint32_t own = smem_u32(smem);
      const int m = threadIdx.x % FOURS * 4, n = n0 + m, d_stages = stages_of(adapters * blocks);
      const int outs = min(4, A.N - n);
      float sw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[i] = F8 && i < outs ? A.w_scale[n + i] : 1.0f;
      for (int t = (static_cast<int>(rank) * PROJ_THREADS + threadIdx.x) / FOURS; t < rows && outs > 0;
           t += static_cast<int>(ranks) * PROJ_THREADS / FOURS) {
        float4 vb[MOST], vd[MOST];
#pragma unroll
        for (uint32_t q = 0; q < MOST; ++q) {
          vb[q] = vd[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (q >= ranks) continue;
          const uint32_t at = dsmem_addr(own, q) + (t * PROJ_M + m) * 4;
          vb[q] = dsmem_ld_v4(at);
          int from, to;
          share(d_stages, q, from, to);
          if (to > from) vd[q] = dsmem_ld_v4(at + BN * PROJ_M * 4);
        }
#pragma unroll
        for (uint32_t q = 1; q < MOST; ++q) {
          vb[0].x += vb[q].x, vb[0].y += vb[q].y, vb[0].z += vb[q].z, vb[0].w += vb[q].w;
          vd[0].x += vd[q].x, vd[0].y += vd[q].y, vd[0].z += vd[q].z, vd[0].w += vd[q].w;
        }
        const float b4[4] = {vb[0].x, vb[0].y, vb[0].z, vb[0].w}, d4[4] = {vd[0].x, vd[0].y, vd[0].z, vd[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < outs) proj_write<BN, F8>(A, t_tile, t0 + t, n + i, sw[i], b4[i], d4[i], adapters > 0);
      }
    }
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// ------------------------------------------------------------------------------ prompts
// Many rows of bfloat16: two blocks of a cluster, one on each of two SMs, share a tile of 256 outputs and up
// to 256 rows (A.tile_rows, a multiple of 16).  Each holds its 128 outputs of w and half of the rows, and
// the pair's products read the other half from the other SM, so that an SM takes in 64 bytes a cycle
// where a tile of 128 x 128 on one SM would need 128.  base and delta are one accumulator here, and two
// tiles have room in tensor memory: a tile is written while the next is summed.  What a broken adapter
// spoils in other requests' rows is therefore found in the sums: where one is not finite and an adapter of the tile
// has an infinity or a NaN for that output, the pair goes through such tiles again at the end, with base in one
// accumulator and the sound adapters, then each broken one alone, in the other, and writes such outputs anew
// (4,099 x 4,096 x 4,096, us: sound 106, one infinity in an adapter 174, an adapter of NaN 204, 400 rows of NaN 116).
// The inner rows are tiles of the same kind, before all others: 256 of a tile's stacked products a unit, with
// the matrices a in w's place.  A tile of outputs adds its adapters last, and waits before that until its
// rows' units are done.  They are the lowest tiles, so they are taken first and wait for nothing; the launch is
// cooperative, so the pairs that have them run.
//
// Bound by the tensor cores (and their power) in the loop: 4,099 x 4,096 x 4,096 without adapters takes 72 us (1.9 PFLOP/s).
// With 8 adapters of rank 64 it takes 100: their units, the first tiles' wait for them, the lower parts' products, and tiles
// that do not come out even on 76 pairs are the rest.
constexpr int PAIR_STAGES = 7, PAIR_STAGE = 2 * PROJ_M * PROJ_LINE;
__host__ __device__ constexpr int pair_smem() { return PAIR_STAGES * PAIR_STAGE + 1024 + 512; }

struct PairBars {
  uint64_t full[PAIR_STAGES], empty[PAIR_STAGES], done[2], freed[2], drained;
  uint32_t tmem, dead, again;
  uint32_t which[8];  // of a tile's list: adapters with an infinity or a NaN for one of the pair's 256 outputs
};

__device__ __forceinline__ void dsmem_or_u32(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// For which of the outputs n .. n + 31 a tile's adapters have an infinity or a NaN, as bits; the whole warp.  With `which`
// (a shared address), the bits of such adapters' places in the list are set there, in both blocks of the pair.
__device__ __noinline__ uint32_t proj_broken(const ProjectArgs& A, const int32_t* list, int n, uint32_t which) {
  const int count = list[0] & LIST_COUNT, pieces = A.R / 8, lane = threadIdx.x & 31;  // pieces of 16 bytes to an output
  uint32_t broken = 0;
  for (int k = lane; k < 32 * pieces; k += 32) {
    const int of = k / pieces;
    if (n + of >= A.N) break;
    bool any = false;
    for (int j0 = 0; j0 < count; j0 += 16) {  // sixteen loads on their way
      uint4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = reinterpret_cast<const uint4*>(A.b + (static_cast<int64_t>(list[1 + min(j0 + i, count - 1)]) * A.N + n) * A.R)[k];
      uint32_t found = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        for (const uint32_t w : {v[i].x, v[i].y, v[i].z, v[i].w})
          if ((w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u) found |= 1u << min(i, count - 1 - j0);
      any |= found != 0;
      if (found != 0 && which != 0u)
        for (uint32_t q = 0; q < 2; ++q) dsmem_or_u32(dsmem_addr(which + 4 * (j0 >> 5), q), found << (j0 & 31));
    }
    broken |= static_cast<uint32_t>(any) << of;
  }
  __syncwarp();
  return __reduce_or_sync(0xFFFFFFFFu, broken);
}

// The lists of a call's tiles; no unit is done.
__global__ void __launch_bounds__(256) plan_kernel(const __grid_constant__ ProjectArgs A) {
  __shared__ TileAdapters used;
  grid_dep_wait();    // first: the next kernel relies on what was before this one being done
  grid_dep_launch();
  const int tile = blockIdx.x, t0 = tile * A.tile_rows;
  tile_adapters(A, t0, min(A.tile_rows, A.T - t0), &used);
  if (threadIdx.x == 0) {
    write_list(A, tile, A.tile_rows, used);
    A.ready[tile] = 0;
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PROJ_THREADS, 1)
    pair_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mh,
                const __grid_constant__ CUtensorMap ma, const __grid_constant__ ProjectArgs A, int box_rows) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  PairBars* B = reinterpret_cast<PairBars*>(smem + PAIR_STAGES * PAIR_STAGE);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool lead = rank == 0;
  volatile uint32_t* dead = &B->dead;
  const uint32_t bit = 0x08u;  // STRATA_DEVERR_TIMEOUT
  constexpr uint32_t TMEM_COLS = 512;

  if (threadIdx.x == 0) {
    for (int i = 0; i < PAIR_STAGES; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->done[i], 1);
      mbar_init(&B->freed[i], 8);  // the first block's: four warps of each
    }
    mbar_init(&B->drained, 1);
    B->dead = B->again = 0;
    for (uint32_t& w : B->which) w = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B->tmem)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  if (A.S == 0) grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = B->tmem;

  const int rows_max = A.tile_rows, half = rows_max / 2;
  const int k_stages = (A.K + 63) / 64;
  const int blocks = A.S > 0 ? A.R / A.rank_block : 0, per_stage = A.S > 0 ? 64 / A.rank_block : 1;
  const uint32_t line = static_cast<uint32_t>(A.rank_block) * 2;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  auto list_of = [&](int t_tile) { return A.lists + static_cast<int64_t>(t_tile) * (rows_max + 1); };
  auto stack_of = [&](int t_tile) { return (list_of(t_tile)[0] & LIST_COUNT) * A.R; };  // inner products
  auto units_of = [&](int t_tile) { return (stack_of(t_tile) + 2 * PROJ_M - 1) / (2 * PROJ_M); };
  int units = 0;
  if (A.S > 0) {
    grid_dep_wait();
    for (int t = lane; t < A.t_tiles; t += 32) units += units_of(t);
    units = __reduce_add_sync(0xFFFFFFFFu, units);
  }
  const int tiles = units + A.n_tiles * A.t_tiles;
  // The rows and, of a unit, the first inner product (else -1) of tile `tile`, asked for in ascending order.
  struct Place {
    int t_tile = 0, before = 0;
  };
  auto unit_of = [&](int tile, Place& at) {
    if (tile >= units) {
      at.t_tile = (tile - units) % A.t_tiles;
      return -1;
    }
    for (int n; tile >= at.before + (n = units_of(at.t_tile)); ++at.t_tile) at.before += n;
    return (tile - at.before) * 2 * PROJ_M;
  };

  Ring<PAIR_STAGES> ring;  // of the loading and of the issuing warp
  bool alive = true;
  uint32_t turn = 0;       // tiles so far, of the issuing warp and of those that write
  auto room = [&]() {      // in the next stage
    if (ring.begun >= PAIR_STAGES && !proj_wait(&B->empty[ring.slot], ring.phase ^ 1u, dead, A.errors, bit)) alive = false;
    return alive;
  };
  auto landed = [&]() {  // the next stage
    if (!proj_wait(&B->full[ring.slot], ring.phase, dead, A.errors, bit)) alive = false;
    tc_fence_after();
    return alive;
  };
  // 256 outputs: M counts in sixteens
  const uint32_t idesc = (mma_idesc(false, rows_max) & 0x00FFFFFFu) | (16u << 24);
  // Rank blocks from rank block 0 of the list's adapter `j` on, `subs` of them: for every two stages of b with the upper parts
  // of the inner rows, one stage before them with the lower parts.
  auto load_blocks = [&](int t_tile, int n0, int j, int subs) {
    auto load_rows = [&](uint32_t at, uint32_t bar, int part, int sub0, int n) {
      for (int i = 0; i < n; ++i) {
        const int jj = j + (sub0 + i) / blocks, rb = (sub0 + i) % blocks;
        pair_tma_2d(at + i * half * line, &mh, rb * A.rank_block, ((part * A.t_tiles + t_tile) * A.most + jj) * rows_max + rank * half, bar);
      }
    };
    for (int s = 0; s * per_stage < subs && alive && room(); ++s, ring.next()) {
      const int sub0 = s * per_stage, n = min(per_stage, subs - sub0);
      if (s % 2 == 0) {
        const uint32_t at = smem_u32(smem + ring.slot * PAIR_STAGE), bar = dsmem_addr(smem_u32(&B->full[ring.slot]), 0);
        const int both = min(2 * per_stage, subs - sub0);
        if (elect_one()) {
          if (lead) mbar_arrive_expect_tx(&B->full[ring.slot], static_cast<uint32_t>(2 * both * half) * line);
          load_rows(at, bar, 1, sub0, both);
        }
        ring.next();
        if (!room()) break;
      }
      const uint32_t at = smem_u32(smem + ring.slot * PAIR_STAGE), bar = dsmem_addr(smem_u32(&B->full[ring.slot]), 0);
      if (elect_one()) {
        if (lead) mbar_arrive_expect_tx(&B->full[ring.slot], static_cast<uint32_t>(2 * n * (PROJ_M + half)) * line);
        for (int i = 0; i < n; ++i)
          pair_tma_3d(at + i * PROJ_M * line, &mb, (sub0 + i) % blocks * A.rank_block, n0, list_of(t_tile)[1 + j + (sub0 + i) / blocks], bar);
        load_rows(at + PROJ_M * PROJ_LINE, bar, 0, sub0, n);
      }
    }
  };
  auto add_blocks = [&](uint32_t sum, int subs, bool add) {
    uint32_t low = 0;
    for (int s = 0; s * per_stage < subs && alive && landed(); ++s, ring.next()) {
      if (s % 2 == 0) {
        low = ring.slot;
        ring.next();
        if (!landed()) break;
      }
      const int n = min(per_stage, subs - s * per_stage);
      const uint32_t at = smem_u32(smem + ring.slot * PAIR_STAGE), at_h = at + PROJ_M * PROJ_LINE;
      const uint32_t at_low = smem_u32(smem + low * PAIR_STAGE) + s % 2 * per_stage * half * line;
      if (elect_one()) {
        for (int i = 0; i < n; ++i) {
          const uint64_t da = mma_desc(at + i * PROJ_M * line, line);
          const uint64_t db = mma_desc(at_h + i * half * line, line), dl = mma_desc(at_low + i * half * line, line);
          for (int q = 0; q < A.rank_block / 16; ++q) {
            pair_mma(sum, da + 2 * q, db + 2 * q, idesc, add || s > 0 || i > 0 || q > 0);
            pair_mma(sum, da + 2 * q, dl + 2 * q, idesc, true);
          }
        }
        pair_commit(&B->empty[ring.slot]);
        if (s % 2 == 1 || (s + 1) * per_stage >= subs) pair_commit(&B->empty[low]);
      }
    }
  };
  auto load_base = [&](int t0, int n0) {
    for (int s = 0; s < k_stages && room(); ++s, ring.next()) {
      const uint32_t at = smem_u32(smem + ring.slot * PAIR_STAGE), bar = dsmem_addr(smem_u32(&B->full[ring.slot]), 0);
      if (elect_one()) {
        if (lead) mbar_arrive_expect_tx(&B->full[ring.slot], static_cast<uint32_t>(2 * (PROJ_M + half) * PROJ_LINE));
        pair_tma_2d(at, &mw, s * 64, n0, bar);
        pair_tma_2d(at + PROJ_M * PROJ_LINE, &mx, s * 64, t0, bar);
      }
    }
  };
  auto add_base = [&](uint32_t sum) {
    for (int s = 0; s < k_stages && landed(); ++s, ring.next()) {
      const uint32_t at = smem_u32(smem + ring.slot * PAIR_STAGE);
      const uint64_t da = mma_desc(at, PROJ_LINE), db = mma_desc(at + PROJ_M * PROJ_LINE, PROJ_LINE);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pair_mma(sum, da + 2 * i, db + 2 * i, idesc, s > 0 || i > 0);
        pair_commit(&B->empty[ring.slot]);
      }
    }
  };
  auto freed_all = [&]() {  // the products in flight end before the blocks give their tensor memory back
    if (elect_one()) pair_commit(&B->drained);
    for (uint32_t spin = 0; spin < PROJ_SPINS && !mbar_try_wait(&B->drained, 0); ++spin) {
    }
  };

  if (warp == 0) {
    Place place;
    for (int tile = first; tile < tiles && alive; tile += step) {
      const int q0 = unit_of(tile, place), t_tile = place.t_tile, t0 = t_tile * rows_max + rank * half;
      if (q0 >= 0) {
        const int stack = stack_of(t_tile);
        auto boxes_of = [&](int r) { return (max(0, min(PROJ_M, stack - q0 - r * PROJ_M)) + box_rows - 1) / box_rows; };
        const int boxes = boxes_of(rank);
        const uint32_t bytes = static_cast<uint32_t>(((boxes_of(0) + boxes_of(1)) * box_rows + rows_max) * PROJ_LINE);
        for (int s = 0; s < k_stages && room(); ++s, ring.next()) {
          const uint32_t at = smem_u32(smem + ring.slot * PAIR_STAGE), bar = dsmem_addr(smem_u32(&B->full[ring.slot]), 0);
          if (elect_one()) {
            if (lead) mbar_arrive_expect_tx(&B->full[ring.slot], bytes);
            for (int i = 0; i < boxes; ++i) {
              const int q = q0 + rank * PROJ_M + i * box_rows;
              pair_tma_2d(at + i * box_rows * PROJ_LINE, &ma, s * 64, list_of(t_tile)[1 + q / A.R] * A.R + q % A.R, bar);
            }
            pair_tma_2d(at + PROJ_M * PROJ_LINE, &mx, s * 64, t0, bar);
          }
        }
        continue;
      }
      const int n0 = ((tile - units) / A.t_tiles * 2 + rank) * PROJ_M;
      load_base(t0, n0);
      if (A.S == 0 || !alive) continue;
      {  // its rows' units: eight warps of a pair write each
        const uint32_t need = static_cast<uint32_t>(units_of(t_tile)) * 8;
        uint32_t spin = 0, seen;
        do {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(A.ready + t_tile) : "memory");
          if (!__any_sync(0xFFFFFFFFu, seen != need)) break;
          if (__any_sync(0xFFFFFFFFu, *dead != 0u)) alive = false;
        } while (alive && ++spin < PROJ_SPINS);
        if (alive && spin >= PROJ_SPINS) {
          *dead = 1u;
          atomicOr(A.errors, bit);
          alive = false;
        }
        asm volatile("fence.proxy.async;" ::: "memory");
      }
      load_blocks(t_tile, n0, 0, (list_of(t_tile)[0] & LIST_COUNT) * blocks);
    }
    if (!alive && lead) ring.drain(B->full);
  } else if (warp == 1 && lead) {
    Place place;
    for (int tile = first; tile < tiles && alive; tile += step, ++turn) {
      const int q0 = unit_of(tile, place);
      const uint32_t buf = turn & 1, sum = tmem + buf * 256;
      if (turn >= 2 && !proj_wait(&B->freed[buf], (turn / 2 + 1) & 1, dead, A.errors, bit)) {
        alive = false;
        break;
      }
      tc_fence_after();
      add_base(sum);
      if (A.S > 0 && q0 < 0) add_blocks(sum, (list_of(place.t_tile)[0] & LIST_COUNT) * blocks, true);
      if (alive && elect_one()) pair_commit(&B->done[buf]);
    }
    if (!alive) freed_all();
  } else if (warp >= 2) {
    const uint32_t quarter = warp & 3;
    Place place;
    for (int tile = first; tile < tiles; tile += step, ++turn) {
      const int q0 = unit_of(tile, place), t_tile = place.t_tile, t0 = t_tile * rows_max;
      const int rows = min(rows_max, A.T - t0), lane_at = static_cast<int>(rank * PROJ_M + quarter * 32) + lane;
      const uint32_t buf = turn & 1, sum = tmem + buf * 256 + (quarter << 21);
      // A unit: the lane's adapter is the same for sixteen lanes, and lane k has for its sixteen which of the rows
      // 32 (k & 15) .. have it.  (Row after row, with the second part, took 2.5 us more before the first tiles.)
      uint32_t masks = 0;
      float by = 0.0f;
      const int stack = q0 >= 0 ? stack_of(t_tile) : 0;
      if (q0 >= 0) {
        const int q = q0 + lane_at, c = q < stack ? list_of(t_tile)[1 + q / A.R] : -2;
        if (c >= 0) by = A.adapter_scale[c];
        const int c_lo = __shfl_sync(0xFFFFFFFFu, c, 0), c_hi = __shfl_sync(0xFFFFFFFFu, c, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int of = i * 32 + lane < rows ? A.row_adapter[t0 + i * 32 + lane] : -1;
          const uint32_t lo = __ballot_sync(0xFFFFFFFFu, of == c_lo), hi = __ballot_sync(0xFFFFFFFFu, of == c_hi);
          if ((lane & 15) == i) masks = lane < 16 ? lo : hi;
        }
      }
      if (!proj_wait(&B->done[buf], (turn / 2) & 1, dead, A.errors, bit)) {
        alive = false;
        break;
      }
      tc_fence_after();
      if (q0 >= 0) {
        // inner rows, zeros where a row has another adapter
#pragma unroll 1
        for (int c0 = 0; c0 < rows; c0 += 32) {
          const uint32_t mine = __shfl_sync(0xFFFFFFFFu, masks, c0 / 32 + (lane & 16));
          float v[32];
          tmem_ld32(sum + c0, v);
          tmem_wait_ld();
          const int q = q0 + lane_at;
          // two rows at a time: of both lanes of a pair the even one stores the first row, four bytes, and the odd one the second
          const int odd = lane & 1;
          __nv_bfloat16* h = A.spread + ((static_cast<int64_t>(t_tile) * A.most + q / A.R) * rows_max + c0 + odd) * A.R + (q - odd) % A.R;
          const int upto = q < stack ? rows - c0 - odd : 0;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            __nv_bfloat162 hi, lo;
            proj_split(mine >> i & 1u ? by * v[i] : 0.0f, hi.x, lo.x);
            proj_split(mine >> (i + 1) & 1u ? by * v[i + 1] : 0.0f, hi.y, lo.y);
            const uint32_t hw = *reinterpret_cast<const uint32_t*>(&hi), lw = *reinterpret_cast<const uint32_t*>(&lo);
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, __byte_perm(hw, lw, odd ? 0x5410 : 0x7632), 1);
            if (i < upto) {
              *reinterpret_cast<uint32_t*>(h + i * A.R) = __byte_perm(hw, other, odd ? 0x3254 : 0x5410);
              *reinterpret_cast<uint32_t*>(h + i * A.R + A.low) = __byte_perm(lw, other, odd ? 0x3276 : 0x7610);
            }
          }
        }
        tc_fence_before();
        asm volatile("fence.proxy.async;" ::: "memory");
        __threadfence();
        __syncwarp();
        if (lane == 0) {
          atomicAdd(A.ready + t_tile, 1u);
          mbar_arrive_remote(dsmem_addr(smem_u32(&B->freed[buf]), 0));
        }
        continue;
      }
      const int n = (tile - units) / A.t_tiles * 2 * PROJ_M + lane_at;
      const bool mixed = A.S > 0 && (list_of(t_tile)[0] & LIST_MIXED) != 0;
      bool looked = false;  // at what the adapters have for the warp's outputs
      __nv_bfloat16* y = A.y + t0 * A.ldy + n;
#pragma unroll 1
      for (int c = 0; c < rows; c += 32) {  // the last columns of a buffer's 256 may be stale: they are not used
        float v[32];
        tmem_ld32(sum + c, v);
        tmem_wait_ld();
        if (mixed) {
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) bad |= fabsf(v[i]) < __int_as_float(0x7F800000) ? 0u : 1u << i;
          if (rows - c < 32) bad &= (1u << (rows - c)) - 1u;
          // a row's own operands may be the reason: then its sum stands
          if (!looked && __any_sync(0xFFFFFFFFu, bad != 0 && n < A.N)) {
            looked = true;
            const uint32_t again = *static_cast<volatile uint32_t*>(&B->again);
            if (__all_sync(0xFFFFFFFFu, again == 0u) && proj_broken(A, list_of(t_tile), n - lane, 0u) != 0u && lane < 2)
              dsmem_st_u32(dsmem_addr(smem_u32(&B->again), lane), 1u);
            __syncwarp();
          }
        }
        if (n < A.N) {
          if (rows - c >= 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i, y += A.ldy) *y = __float2bfloat16_rn(v[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i, y += A.ldy)
              if (c + i < rows) *y = __float2bfloat16_rn(v[i]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(dsmem_addr(smem_u32(&B->freed[buf]), 0));
    }
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  if (B->again != 0u) {  // the same in both blocks
    // Base in the first buffer, adapters in the second.  Both are free; what waits for them counts on with the first
    // one's barriers.
    tc_fence_after();
    const bool died = !alive;
    const uint32_t quarter = warp & 3, base = tmem, delta = tmem + 256;
    uint32_t round = (turn + 1) / 2;  // of done[0] and freed[0]
#pragma unroll 1
    for (int tile = first; tile < tiles; tile += step) {
      const int t_tile = tile < units ? 0 : (tile - units) % A.t_tiles, t0 = t_tile * rows_max;
      const int32_t* list = list_of(t_tile);
      if (tile < units || (list[0] & LIST_MIXED) == 0) continue;
      const int n0 = ((tile - units) / A.t_tiles * 2 + rank) * PROJ_M, count = list[0] & LIST_COUNT;
      const int rows = min(rows_max, A.T - t0), n = n0 + quarter * 32 + lane;
      uint32_t columns = 0;  // of this warp's, those to write
      if (warp >= 2) columns = proj_broken(A, list, n - lane, smem_u32(B->which));
      __syncthreads();
      cluster_arrive();
      cluster_wait();
      uint32_t some = 0;
      for (int i = 0; i < 8; ++i) some |= B->which[i];
      auto is_broken = [&](int j) { return (B->which[j >> 5] >> (j & 31) & 1u) != 0u; };
      // a round for the sound ones (-1), then one for each broken one
      auto next_broken = [&](int j) {
        for (++j; j < count && !is_broken(j); ++j) {
        }
        return j;
      };
      if (some != 0u) {
        if (warp == 0) {
          if (alive) load_base(t0 + rank * half, n0);
          for (int own = -1; own < count && alive; own = next_broken(own))
            for (int j = max(own, 0); j < (own < 0 ? count : own + 1); ++j) {
              if (own < 0 && is_broken(j)) continue;
              load_blocks(t_tile, n0, j, blocks);
            }
        } else if (warp == 1 && lead) {
          uint32_t in_tile = 0;
          for (int own = -1; own < count && alive; own = next_broken(own), ++round, ++in_tile) {
            // the round before has been written (the last tile's last one before the barrier)
            if (in_tile > 0 && !proj_wait(&B->freed[0], (round + 1) & 1, dead, A.errors, bit)) {
              alive = false;
              break;
            }
            tc_fence_after();
            if (own < 0) add_base(base);
            bool add = false;
            for (int j = max(own, 0); j < (own < 0 ? count : own + 1); ++j) {
              if (own < 0 && is_broken(j)) continue;
              add_blocks(delta, blocks, add);
              add = true;
            }
            if (alive && elect_one()) pair_commit(&B->done[0]);
          }
        } else if (warp >= 2) {
          const bool mine = columns >> lane & 1u;
          for (int own = -1; own < count && alive; own = next_broken(own), ++round) {
            if (!proj_wait(&B->done[0], round & 1, dead, A.errors, bit)) {
              alive = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < rows && columns != 0; c0 += 32) {
              const int of = c0 + lane < rows ? A.row_adapter[t0 + c0 + lane] : -1;
              const bool has = of >= 0 && of < A.S;
              bool now = own < 0 ? c0 + lane < rows : of == list[1 + own];
              if (own < 0)
                for (int j = next_broken(-1); j < count; j = next_broken(j)) now = now && of != list[1 + j];
              const uint32_t writes = __ballot_sync(0xFFFFFFFFu, now), adds = __ballot_sync(0xFFFFFFFFu, now && has);
              if (writes == 0) continue;
              float v[32], d[32];
              tmem_ld32(base + (quarter << 21) + c0, v);
              tmem_ld32(delta + (quarter << 21) + c0, d);
              tmem_wait_ld();
              if (mine) {
                __nv_bfloat16* y = A.y + (t0 + c0) * A.ldy + n;
#pragma unroll
                for (int i = 0; i < 32; ++i, y += A.ldy)
                  if (writes >> i & 1u) *y = __float2bfloat16_rn(adds >> i & 1u ? v[i] + d[i] : v[i]);
              }
              __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(dsmem_addr(smem_u32(&B->freed[0]), 0));
          }
        }
      }
      __syncthreads();
      if (threadIdx.x < 8) B->which[threadIdx.x] = 0;
      cluster_arrive();
      cluster_wait();
      tc_fence_after();
    }
    if (!alive && !died && lead) {
      if (warp == 0) ring.drain(B->full);
      if (warp == 1) freed_all();
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
  // neither block's shared or tensor memory is given back while the other's products use it: both are past a barrier
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

}  // namespace strata
