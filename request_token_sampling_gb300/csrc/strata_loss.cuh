// strata_loss.cuh -- losses over a whole vocabulary straight from the rows and the head, and their gradients.
//
//   z = x w^T / s;  lse = log sum exp z;  loss = s^2 sum_k q_k (log q_k - (z_k - lse));  dz = g s (exp(z - lse) - q)
//   dx = dz w;  dw = dz^T x            (a cross entropy has one k with q = 1, and s = 1)
//
// The logits exist as tiles of tensor memory only.  One kernel makes all four kinds of products on the tensor cores:
//   LOSS_SUMS   z of up to 256 rows and 256 ids: a maximum and a sum of exponentials for each row, and z of the row's ids
//   LOSS_DIFFS  z again, and d = exp(z - lse) - q in bfloat16 to the workspace, for a piece of the vocabulary
//   LOSS_DW     dw of the piece: d^T xs over the rows (both operands with the sum's index outermost in memory)
//   LOSS_DX     parts of dx: d w over the piece's ids (w with the sum's index outermost), in 32 bits, or dx where one is all
// Between d and its products stands one rounding to bfloat16, the type of w and x, which the tensor cores ask for: at most 2^-8 of
// each term, as far off as the results' own rounding (together 1.1 to 1.5 times that, as a rule; up to 2.3 times of one to four
// rows, where one d is most of a result).  g stays out of d: dx is scaled in 32 bits at the end, and
// x of a row is scaled by g / max|g| in xs, which changes nothing where all g are equal (a mean).
//
// Rows that are left out do not take part: the others are copied one after another first (loss_gather_kernel), but for scores
// that take less than the copy would save.
//
// Many rows are bound by the tensor cores: tiles of 256 x 256 on two SMs, half of the columns brought by each (64 bytes a cycle
// where a tile on one SM takes 96), six or seven stages of 32 KB on their way, and two accumulators, which four writing warps each
// empty by turns.  Measured (one GB300, rows x ids x width): the sums of 2,048 x 32,000 x 2,048 144 us (1.87 PFLOP/s, a library
// product's rate), differences, dw and dx 154, 150 and 151; a whole step of 4,096 x 32,000 x 4,096, an eighth of the rows left
// out, 2,190 us in a stream of steps, which the power limit sets (1,990 alone).  Few rows are bound by HBM: tiles of 128 rows on one
// SM, whose rows past the last one are neither loaded nor looked at: the sums of 64 x 248,320 x 2,048 150 us (6.8 TB/s); the step
// of 96 such rows 661, of which w's three readings and dw's writing take 600 at the copy's rate.
#pragma once

#include <cuda_bf16.h>

#include "strata_mma.cuh"
#include "strata_norm.cuh"

namespace strata {

enum LossMode { LOSS_SUMS, LOSS_DIFFS, LOSS_DW, LOSS_DX };

constexpr int LOSS_LINE = 128;        // bytes of a row that one stage holds: 64 bfloat16
constexpr int LOSS_THREADS = 320;     // warp 0 loads, warp 1 issues the products, warps 2-9 write the tile
constexpr int LOSS_WRITERS = 8;       // four for each of the two accumulators: they write one tile after another by turns
constexpr int LOSS_BAND = 16;         // tiles of the inner index that a band has: what its operands take stays in L2
constexpr int LOSS_RUNS = 4;          // steps of 64 rows up to which dw's tiles go in runs (below, where they are)
constexpr int LOSS_NO_ID = 0x7FFFFFFF;
// The tensor cores cut their sums off to 32 bits after every 16 products, always towards zero: lse of rows 1,024 wide is off by
// 5e-7 of itself, of rows 4,096 wide by 2.4e-6.  So the scores' sums of wider rows (LONG) are taken out of tensor memory and added up
// in registers, rounded, every 16 steps of 64 (up to 8e-7, for 1 % of a step's time; every 8 steps 3e-7, for 2 to 11 %).  Up to twice that
// width few rows, where it takes 4 %, have narrow tiles instead, with two sums in tensor memory, one of each half of the width.
// The differences take z in the same runs (LossArgs::run), and so the same bits of it that lse was made of: what is left of a row that
// is all but sure of its token is z - lse, which an error in only one of the two would drown (2.4e-6 of a z of 20 is as
// much as a 1 - p of 5e-5).
constexpr int LOSS_LONG = 16;
// Two SMs share a tile: 128 rows and half of the columns each; one SM alone has 128 rows and all columns.  What is left of
// shared memory holds results on their way out, a piece of 32 rows for each writing warp.
constexpr int LOSS_PIECE = 4096;
constexpr int LOSS_MOST_STAGES = 8;
__host__ __device__ constexpr int loss_ring_bytes(int mode, bool pair) { return (!pair || mode != LOSS_SUMS ? 192 : 224) * 1024; }
__host__ __device__ constexpr int loss_smem(int mode, bool pair) {
  return loss_ring_bytes(mode, pair) + (mode == LOSS_SUMS ? 0 : LOSS_WRITERS * LOSS_PIECE) + 1024 + 512;
}
// Where B lies in a stage, and a stage's bytes.  A's products read 128 rows wherever they end: the rows behind `a_rows` are some
// of B's, and of what they give nothing is looked at.
__host__ __device__ constexpr int loss_b_place(int a_rows) { return a_rows * LOSS_LINE; }
__host__ __device__ constexpr int loss_stage_bytes(int a_rows, int b_rows) { return (a_rows + b_rows) * LOSS_LINE; }
__host__ __device__ constexpr int loss_stages(int ring, int stage) {
  const int n = (ring - 128 * LOSS_LINE) / stage + 1, m = ring / stage;  // the last one's 128 rows lie in the ring, too
  const int least = n < m ? n : m;
  return least < LOSS_MOST_STAGES ? least : LOSS_MOST_STAGES;
}

struct LossArgs {
  const int32_t* count;   // rows that take part, as the plan found them; NULL: all T
  const int32_t* rows;    // which they are; NULL: row r itself
  const int32_t* ids;     // [T][K], ascending where K > 1, those that are not there last as LOSS_NO_ID
  const float* q;         // [T][K] beside them; NULL: 1
  const float* lse;       // of row t, for LOSS_DIFFS
  const float* by;        // scale of LOSS_DW's results
  const int32_t* same;    // LOSS_DW: not 0 where all rows' scales are equal, and the rows need no scaled copy
  float2* parts;          // [rows][n_tiles], or two of each tile (LONG): exponent and sum of the columns, for LOSS_SUMS
  float* picks;           // [rows][K]: z of the row's ids
  __nv_bfloat16* out;     // d or dw
  int64_t ldo;
  int wide;               // dw's rows start on 32 bytes and are so many times as wide
  uint32_t* errors;
  float scale;            // log2(e) / s
  float dw_scale;         // s
  int T, V, H, K;
  int row0, rows_most;    // rows row0 .. of this launch
  int v0, columns;        // the piece of the vocabulary
  int bn, n_tiles;        // columns of a tile, and tiles of them
  int a_rows;             // rows that one SM's tile brings where they are A; the accumulator's other rows are not looked at
  int d_rows;             // rows that d has
  int run;                // LOSS_SUMS, LOSS_DIFFS: steps of 64 that one sum in tensor memory has
  int splits, rows_pad;   // LOSS_DX: parts that a piece may be cut into, and rows of each
  int k_piece, units;     // steps of 64 ids in a piece, and tiles that run at a time
  int add;                // LOSS_DX: onto what is there
  __nv_bfloat16* dx;      // LOSS_DX: where one part is all, the results themselves, scaled by g; NULL: there are more pieces
  int64_t lddx;
  const float* g;
};

struct LossBars {
  uint64_t full[LOSS_MOST_STAGES], empty[LOSS_MOST_STAGES], done[2], freed[2], drained;
  uint32_t tmem, dead;
};

// Shared-memory operand descriptor of an operand whose index of the sum is outermost: blocks of 64 rows or columns, each
// 64 lines (one for each step of the sum) of 128 bytes, a block 8,192 bytes from the next; eight lines make a swizzle group.
__device__ __forceinline__ uint64_t loss_desc_outer(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// 32-bit sums of bfloat16; A and B with the sum's index innermost, or outermost (bits 15 and 16).
__device__ __forceinline__ uint32_t loss_idesc(int m, int n, bool a_outer, bool b_outer) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_outer ? 1u << 15 : 0u) | (b_outer ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]),
      "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* m, int x, int y, uint32_t src) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Few tiles of dx leave SMs idle in the last turn, so the sum over a piece's ids is cut into parts; the whole warp.  In
// eighths of a stage's time (0.33 us): turns of so many stages and three to start and end with, and each part's way
// to memory and back (4 bytes each way and element: 0.23 stages for a pair's tile).
__device__ __forceinline__ int loss_splits(int tiles, int k, int most, int units, bool pair) {
  const int s = static_cast<int>(threadIdx.x & 31) + 1;
  uint32_t cost = 0x07FFFFFFu;
  if (s <= most && (s == 1 || k >= 4 * s)) cost = min(cost, static_cast<uint32_t>((tiles * s + units - 1) / units * ((k + s - 1) / s + 3) * 8 + s * tiles * (pair ? 2 : 1)));
  return static_cast<int>(__reduce_min_sync(FULL_MASK, cost << 5 | static_cast<uint32_t>(s - 1)) & 31u) + 1;
}

// The stages' ring as one warp goes through it.
struct LossRing {
  uint32_t stages, slot = 0, phase = 0, begun = 0;
  __device__ __forceinline__ void next() {
    ++begun;
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // Waits until the copies of the newest stages have landed: no copy of a block may be in flight when it ends.
  __device__ __forceinline__ void drain(uint64_t* full) {
    for (uint32_t i = 0; i < stages && begun > 0; ++i, --begun) {
      phase ^= slot == 0;
      slot = slot == 0 ? stages - 1 : slot - 1;
      for (uint32_t spin = 0; spin < PROJ_SPINS && !mbar_try_wait(&full[slot], phase); ++spin) {
      }
    }
  }
};

// Tile `tile` of `outer` x `inner`: bands of LOSS_BAND inner ones, which go fastest.
__device__ __forceinline__ void loss_place(int tile, int outer, int inner, int& o, int& i) {
  if (inner <= LOSS_BAND) {
    o = tile / inner;
    i = tile - o * inner;
    return;
  }
  const int band = tile / (LOSS_BAND * outer), width = min(LOSS_BAND, inner - band * LOSS_BAND), rest = tile - band * LOSS_BAND * outer;
  o = rest / width;
  i = band * LOSS_BAND + rest - o * width;
}

// The next of a row's ids from `from` on, in ascending order.
struct LossIds {
  const int32_t* ids;
  const float* q;
  int at, K, next;
  __device__ __forceinline__ void start(const LossArgs& A, int64_t t, int from) {
    K = t < 0 ? 0 : A.K;
    ids = A.ids + (t < 0 ? 0 : t) * A.K;
    q = A.q != nullptr ? A.q + (t < 0 ? 0 : t) * A.K : nullptr;
    at = 0;
    if (K == 1) {
      if (ids[0] < from) at = 1;
    } else {
      for (int upto = K; at < upto;) {
        const int mid = (at + upto) / 2;
        if (ids[mid] < from)
          at = mid + 1;
        else
          upto = mid;
      }
    }
    next = at < K ? ids[at] : LOSS_NO_ID;
  }
  __device__ __forceinline__ float weight() const { return q != nullptr ? q[at] : 1.0f; }
  __device__ __forceinline__ void advance() { next = ++at < K ? ids[at] : LOSS_NO_ID; }
};

// As block `block` of `blocks`.  Maps: A, B, B of scaled rows (LOSS_DW), results (LOSS_DX).
template <int MODE, bool PAIR, bool LONG>
__device__ __forceinline__ void loss_products(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const CUtensorMap& mo, const LossArgs& A,
                                              int block, int blocks) {
  constexpr int RING = loss_ring_bytes(MODE, PAIR), TILE_M = PAIR ? 256 : 128;
  constexpr bool A_OUTER = MODE == LOSS_DW, B_OUTER = MODE == LOSS_DW || MODE == LOSS_DX;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* staging = smem + RING;
  LossBars* B = reinterpret_cast<LossBars*>(staging + (MODE == LOSS_SUMS ? 0 : LOSS_WRITERS * LOSS_PIECE));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool lead = rank == 0;
  volatile uint32_t* dead = &B->dead;
  const uint32_t bit = 0x08u;  // STRATA_DEVERR_TIMEOUT
  constexpr uint32_t TMEM_COLS = 512;

  if (threadIdx.x == 0) {
    for (int i = 0; i < LOSS_MOST_STAGES; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->done[i], 1);
      mbar_init(&B->freed[i], LOSS_WRITERS / (PAIR ? 1 : 2) * (LONG ? 2 : 1));  // the first block's: four warps of each, or all
    }
    mbar_init(&B->drained, 1);
    B->dead = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B->tmem)), "r"(TMEM_COLS) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B->tmem)), "r"(TMEM_COLS) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  if constexpr (PAIR) {
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  const uint32_t tmem = B->tmem;

  // this launch's rows and tiles
  const int live = max(0, min((A.count != nullptr ? *A.count : A.T) - A.row0, A.rows_most));
  const int row_tiles = (live + TILE_M - 1) / TILE_M;
  int outer, inner, k_all, splits = 1;
  if constexpr (MODE == LOSS_SUMS || MODE == LOSS_DIFFS) {
    outer = A.n_tiles, inner = row_tiles, k_all = (A.H + 63) / 64;
  } else if constexpr (MODE == LOSS_DW) {
    outer = (A.columns + TILE_M - 1) / TILE_M, inner = A.n_tiles, k_all = (live + 63) / 64;
  } else {
    outer = A.n_tiles, inner = row_tiles, k_all = (A.columns + 63) / 64;
    splits = loss_splits(outer * inner, A.k_piece, A.splits, A.units, PAIR);
  }
  const int per_split = outer * inner;
  int tiles = per_split * splits, first = PAIR ? block / 2 : block, step = PAIR ? blocks / 2 : blocks;
  // Few rows: dw is bound by its writing, and blocks that write one tile after another of the same ids leave memory fuller
  // pages (96 rows, 1 GB: 262 us, by turns 283; with 32 bytes a store 247).  With more rows the blocks' parts of d would
  // not fit in L2 together.
  if (MODE == LOSS_DW && k_all <= LOSS_RUNS) {
    const int64_t all = tiles;
    tiles = static_cast<int>(all * (first + 1) / step);
    first = static_cast<int>(all * first / step);
    step = 1;
  }
  const int half = PAIR ? A.bn / 2 : A.bn;  // columns that this block brings
  auto stages_of = [&](int split, int& from, int& to) {
    if constexpr (MODE == LOSS_DX) {  // 8,192 steps and 32 parts at most
      from = k_all * split / splits;
      to = k_all * (split + 1) / splits;
    } else {
      from = 0;
      to = k_all;
    }
  };

  // two sums of a narrow tile of logits
  const bool halves = MODE == LOSS_SUMS && !LONG && A.run < k_all;

  // rows that a stage holds: a pair's always as many, so that the numbers are known; of rows as B all that the tile has
  const int a_rows = PAIR || MODE == LOSS_DW ? 128 : A.a_rows, b_place = loss_b_place(a_rows);
  const int stage_bytes = PAIR ? loss_stage_bytes(128, 128) : loss_stage_bytes(a_rows, A.bn);
  LossRing ring{static_cast<uint32_t>(PAIR ? RING / loss_stage_bytes(128, 128) : loss_stages(RING, stage_bytes))};  // of the loading and of the issuing warp
  bool alive = true;
  uint32_t turn = 0;  // accumulators so far, of the issuing warp and of those that write
  if (warp == 0) {
    asm volatile("fence.proxy.async;" ::: "memory");  // rows and d were written by ordinary stores of kernels before
    const uint32_t bytes = static_cast<uint32_t>((PAIR ? 2 : 1) * (a_rows + half)) * LOSS_LINE;
    const CUtensorMap* mx = MODE == LOSS_DW && *A.same == 0 ? &mc : &mb;
    for (int tile = first; tile < tiles && alive; tile += step) {
      int o, i, from, to;
      const int split = MODE == LOSS_DX ? tile / per_split : 0;
      loss_place(tile - split * per_split, outer, inner, o, i);
      stages_of(split, from, to);
      for (int s = from; s < to; ++s, ring.next()) {
        if (ring.begun >= ring.stages && !proj_wait(&B->empty[ring.slot], ring.phase ^ 1u, dead, A.errors, bit)) {
          alive = false;
          break;
        }
        const uint32_t at = smem_u32(smem + ring.slot * stage_bytes), at_b = at + b_place;
        const uint32_t bar = PAIR ? dsmem_addr(smem_u32(&B->full[ring.slot]), 0) : smem_u32(&B->full[ring.slot]);
        auto load = [&](uint32_t to_, const CUtensorMap* m, int x, int y) {
          if constexpr (PAIR)
            pair_tma_2d(to_, m, x, y, bar);
          else
            tma_2d(to_, m, x, y, bar);
        };
        if (elect_one()) {
          if (lead) mbar_arrive_expect_tx(&B->full[ring.slot], bytes);
          if constexpr (MODE == LOSS_SUMS || MODE == LOSS_DIFFS) {
            load(at, &ma, s * 64, A.row0 + i * TILE_M + rank * 128);
            load(at_b, &mb, s * 64, A.v0 + o * A.bn + rank * half);
          } else if constexpr (MODE == LOSS_DW) {
            for (int b = 0; b < 2; ++b) load(at + b * 8192, &ma, o * TILE_M + rank * 128 + b * 64, s * 64);
            for (int b = 0; b < half / 64; ++b) load(at_b + b * 8192, mx, i * A.bn + rank * half + b * 64, s * 64);
          } else {
            load(at, &ma, s * 64, i * TILE_M + rank * 128);
            for (int b = 0; b < half / 64; ++b) load(at_b + b * 8192, &mb, o * A.bn + rank * half + b * 64, A.v0 + s * 64);
          }
        }
      }
    }
    if (!alive && lead) ring.drain(B->full);
  } else if (warp == 1 && lead) {
    const uint32_t idesc = loss_idesc(TILE_M, A.bn, A_OUTER, B_OUTER);
    constexpr uint32_t STEP_A = A_OUTER ? 128 : 2, STEP_B = B_OUTER ? 128 : 2;  // 16 steps of the sum, in 16 bytes
    for (int tile = first; tile < tiles && alive; tile += step) {
      int from, to;
      stages_of(MODE == LOSS_DX ? tile / per_split : 0, from, to);
      // one accumulator for a tile, or for each run of its steps
      for (int begin = from; alive; begin += A.run, ++turn) {
        const int end = LONG ? min(begin + A.run, to) : to;
        const uint32_t buf = turn & 1, sum = tmem + buf * 256;
        if (turn >= 2 && !proj_wait(&B->freed[buf], (turn / 2 + 1) & 1, dead, A.errors, bit)) {
          alive = false;
          break;
        }
        tc_fence_after();
        for (int s = begin; s < end; ++s, ring.next()) {
          if (!proj_wait(&B->full[ring.slot], ring.phase, dead, A.errors, bit)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = smem_u32(smem + ring.slot * stage_bytes), at_b = at + b_place;
          const uint64_t da = A_OUTER ? loss_desc_outer(at) : mma_desc(at, LOSS_LINE), db = B_OUTER ? loss_desc_outer(at_b) : mma_desc(at_b, LOSS_LINE);
          const bool later = halves && s >= A.run;
          const uint32_t to_sum = later ? sum + 128 : sum;
          const bool adds = s > (later ? A.run : begin);
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (PAIR)
                pair_mma(to_sum, da + STEP_A * i, db + STEP_B * i, idesc, adds || i > 0);
              else
                mma<false>(to_sum, da + STEP_A * i, db + STEP_B * i, idesc, adds || i > 0);
            }
            if constexpr (PAIR)
              pair_commit(&B->empty[ring.slot]);
            else
              mma_commit(&B->empty[ring.slot]);
          }
        }
        if (alive && elect_one()) {
          if constexpr (PAIR)
            pair_commit(&B->done[buf]);
          else
            mma_commit(&B->done[buf]);
        }
        if (end >= to) {
          ++turn;
          break;
        }
      }
    }
    if (!alive) {  // the products in flight end before the blocks give their tensor memory back
      if (elect_one()) {
        if constexpr (PAIR)
          pair_commit(&B->drained);
        else
          mma_commit(&B->drained);
      }
      for (uint32_t spin = 0; spin < PROJ_SPINS && !mbar_try_wait(&B->drained, 0); ++spin) {
      }
    }
  } else if (warp >= 2) {
    const uint32_t quarter = warp & 3;
    const uint32_t group = (warp - 2) / 4;
    uint32_t buf = group;  // the accumulator that this warp empties: always the same one, but for LONG, where both groups share each
    const int from_c = LONG ? static_cast<int>(group) * 128 : 0;  // and have half of the columns
    const uint32_t mine = smem_u32(staging) + (warp - 2) * LOSS_PIECE;  // this warp's piece
    // A lane fills the line of its row, 16 bytes at a time, swizzled so that lines and columns both go without bank conflicts
    // (and as a tensor copy expects it).
    auto put = [&](int piece, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + lane * 128 + ((piece ^ (lane & 7)) << 4)), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    };
    auto put32 = [&](int column, const float (&v)[32]) {  // as bfloat16
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 two = __floats2bfloat162_rn(v[8 * p + 2 * e], v[8 * p + 2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&two);
        }
        put(column / 8 + p, w[0], w[1], w[2], w[3]);
      }
    };
    // Whole lines of 128 bytes to memory: rows y .., columns x .. of A.out, 32 bytes a lane where they lie on that, else 16.
    // (Tensor copies want a fence between the proxies for each piece, in which the warps spent a third of their time.)
    auto line_piece = [&](int row, int piece) {
      uint4 v;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(mine + row * 128 + ((piece ^ (row & 7)) << 4)) : "memory");
      return v;
    };
    auto write_lines = [&](int64_t y, int x, int rows, int columns) {
      __syncwarp();
      if (MODE == LOSS_DIFFS || A.wide != 0) {
        const int row = lane >> 2, piece = (lane & 3) * 2;
        __nv_bfloat16* to = A.out + (y + row) * A.ldo + x + piece * 8;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint4 v = line_piece(n * 8 + row, piece), u = line_piece(n * 8 + row, piece + 1);
          if (n * 8 + row < rows && piece * 8 < columns)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + n * 8 * A.ldo), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
        }
      } else {
        const int row = lane >> 3, piece = lane & 7;
        __nv_bfloat16* to = A.out + (y + row) * A.ldo + x + piece * 8;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const uint4 v = line_piece(n * 4 + row, piece);
          if (n * 4 + row < rows && piece * 8 < columns) *reinterpret_cast<uint4*>(to + n * 4 * A.ldo) = v;
        }
      }
      __syncwarp();
    };
    // 32 bits: by a tensor copy, which also adds
    auto open = [&]() {
      if (lane == 0) tma_store_wait_read();
      __syncwarp();
    };
    auto send = [&](int x, int y, bool add) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (add)
          tma_add_2d(&mo, x, y, mine);
        else
          tma_store_2d(&mo, x, y, mine);
        tma_store_commit();
      }
    };
    [[maybe_unused]] const float by = MODE == LOSS_DW ? *A.by * A.dw_scale : 1.0f;
    const uint32_t lanes = quarter << 21;
    auto empties = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_remote(dsmem_addr(smem_u32(&B->freed[b]), 0));
        else
          mbar_arrive(&B->freed[b]);
      }
    };
    const int step_w = LONG ? step : 2 * step;
    for (int tile = first + (LONG ? 0 : static_cast<int>(group) * step); tile < tiles; tile += step_w) {
      int o, i, from, to;
      const int split = MODE == LOSS_DX ? tile / per_split : 0;
      loss_place(tile - split * per_split, outer, inner, o, i);
      stages_of(split, from, to);
      const int in_tile = static_cast<int>(rank * 128 + quarter * 32);  // this warp's first lane
      const int r = i * TILE_M + in_tile + lane;                         // of SUMS and DIFFS: the row of this launch
      // of these 32 rows none takes part (those of d that the products for dw read are zeros)
      const bool idle = MODE != LOSS_DW && r - lane >= (MODE == LOSS_DIFFS ? min(A.d_rows, (live + 63) / 64 * 64) : live);
      [[maybe_unused]] int64_t t = -1;
      [[maybe_unused]] LossIds ids{};
      [[maybe_unused]] int n0 = 0;
      [[maybe_unused]] float lse = 0.0f, lse2 = 0.0f;
      if constexpr (MODE == LOSS_SUMS || MODE == LOSS_DIFFS) {
        if (r < live) t = A.rows != nullptr ? A.rows[A.row0 + r] : A.row0 + r;
        n0 = A.v0 + o * A.bn;
        ids.start(A, t, n0 + from_c);
        if (MODE == LOSS_DIFFS && t >= 0) {
          lse = A.lse[t];
          lse2 = lse * 1.44269504088896340736f;
        }
      }
      const int columns = min(A.bn, A.v0 + A.columns - n0);  // of LOSS_SUMS
      [[maybe_unused]] float top = -INFINITY, base = 0.0f, total = 0.0f;
      // 32 logits of the row, of columns c ..
      [[maybe_unused]] auto add_logits = [&](float (&v)[32], int c) {
        if (columns - c < 32) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = c + e < columns ? v[e] : -INFINITY;
        }
        const int end = n0 + min(c + 32, columns);
        while (__any_sync(FULL_MASK, ids.next < end)) {
          if (ids.next < end) {
            float z = 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const bool it = ids.next == n0 + c + e;
              z = it ? v[e] : z;
              if (A.q == nullptr) v[e] = it ? -INFINITY : v[e];  // a cross entropy: the sum is that of the other ids
            }
            A.picks[static_cast<int64_t>(r) * A.K + ids.at] = z;
            ids.advance();
          }
        }
        float m = v[0];
#pragma unroll
        for (int e = 1; e < 32; ++e) m = fmaxf(m, v[e]);
        top = fmaxf(top, m);
        const float now = fabsf(top) < INFINITY ? top * A.scale : 0.0f;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          s0 += ex2_approx(fmaf(v[e], A.scale, -now));
          s1 += ex2_approx(fmaf(v[e + 1], A.scale, -now));
        }
        total = (total > 0.0f ? total * ex2_approx(base - now) : total) + (s0 + s1);
        base = now;
      };
      if constexpr (LONG) {
        // this warp's 128 columns: what the accumulators had is added up, and put back into the last one
        float z[8][16] = {};
        for (int begin = from; begin < to; begin += A.run, ++turn) {
          buf = turn & 1;
          if (!proj_wait(&B->done[buf], (turn / 2) & 1, dead, A.errors, bit)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const bool last = begin + A.run >= to;
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // columns beyond the tile's are there, and not looked at
            if (idle) break;
            float v[16];
            const uint32_t at = tmem + buf * 256 + lanes + from_c + j * 16;
            tmem_ld16(at, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) z[j][e] += v[e];
            if (last) tmem_st16(at, z[j]);
          }
          if (!last) empties(buf);
        }
        if (!alive) break;
        tmem_wait_st();
      } else {
        if (!proj_wait(&B->done[buf], turn & 1, dead, A.errors, bit)) {
          alive = false;
          break;
        }
        ++turn;
        tc_fence_after();
      }
      const uint32_t sum = tmem + buf * 256 + lanes;
      if (idle) {
      } else if constexpr (MODE == LOSS_SUMS) {
#pragma unroll 1
        for (int c = from_c; c < (LONG ? min(columns, from_c + 128) : columns); c += 32) {
          float v[32];
          tmem_ld32(sum + c, v);
          if (halves) {
            float u[32];
            tmem_ld32(sum + 128 + c, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] += u[e];
          } else {
            tmem_wait_ld();
          }
          add_logits(v, c);
        }
        if (t >= 0) A.parts[(static_cast<int64_t>(r) * A.n_tiles + o) * (LONG ? 2 : 1) + (LONG ? group : 0)] = make_float2(base, total);
      } else if constexpr (MODE == LOSS_DIFFS) {
        const int upto = t < 0 ? 0 : A.v0 + A.columns - n0;  // zeros beyond the rows and the vocabulary
#pragma unroll 1
        for (int c = from_c; c < (LONG ? min(A.bn, from_c + 128) : A.bn); c += 32) {
          float v[32];
          tmem_ld32(sum + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = ex2_approx(fmaf(v[e], A.scale, -lse2));
          // p - q of the row's ids, from z again: near 1 both are 1 - exp(z - lse) and 1 - q away from it, which keeps the digits
          if (__any_sync(FULL_MASK, ids.next < n0 + c + 32)) {
            float z[32];
            tmem_ld32(sum + c, z);
            tmem_wait_ld();
            do {
              if (ids.next < n0 + c + 32) {
                const int at = ids.next - n0 - c;
                float q = 0.0f, d = 0.0f;
                do {  // one that comes twice counts twice
                  q += ids.weight();
                  ids.advance();
                } while (ids.next == n0 + c + at);
#pragma unroll
                for (int e = 0; e < 32; ++e) d = at == e ? z[e] : d;
                d = d / A.dw_scale - lse;
                d = d > -0.5f ? expm1f(d) + (1.0f - q) : expf(d) - q;
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = at == e ? d : v[e];
              }
            } while (__any_sync(FULL_MASK, ids.next < n0 + c + 32));
          }
          if (upto - c < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = c + e < upto ? v[e] : 0.0f;
          }
          put32(c & 32, v);
          if ((c & 32) != 0 || c + 32 >= A.bn) write_lines(i * TILE_M + in_tile, o * A.bn + (c & ~32), A.d_rows - i * TILE_M - in_tile, (c & 32) + 32);
        }
      } else if (MODE == LOSS_DX && splits == 1 && A.dx != nullptr) {
        if (r < live) t = A.rows[r];
        const float scale = t >= 0 ? A.g[t] * A.dw_scale : 0.0f;
#pragma unroll 1
        for (int c = 0; c < A.bn; c += 64) {
          const int x = o * A.bn + c;
          if (x >= A.H) break;
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            float v[32];
            tmem_ld32(sum + c + h, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= scale;
            put32(h, v);
          }
          __syncwarp();
#pragma unroll
          for (int n = 0; n < 8; ++n) {  // rows wherever they belong, four lines at a time
            const int row = n * 4 + (lane >> 3), piece = lane & 7, to = __shfl_sync(FULL_MASK, static_cast<int>(t), row);
            const uint4 v = line_piece(row, piece);
            if (to >= 0 && piece * 8 < A.H - x) *reinterpret_cast<uint4*>(A.dx + to * A.lddx + x + piece * 8) = v;
          }
        }
      } else {
        const bool none = from == to;  // no rows, or a part without ids: nothing was added up
        constexpr int COLUMNS = MODE == LOSS_DX ? 32 : 64;  // 128 bytes of results
#pragma unroll 1
        for (int c = 0; c < A.bn; c += COLUMNS) {
          const int x = (MODE == LOSS_DX ? o : i) * A.bn + c;
          if (x >= A.H) break;
          float v[COLUMNS];
#pragma unroll
          for (int h = 0; h < COLUMNS; h += 32) tmem_ld32(sum + c + h, *reinterpret_cast<float(*)[32]>(v + h));
          tmem_wait_ld();
          if (none) {
#pragma unroll
            for (int e = 0; e < COLUMNS; ++e) v[e] = 0.0f;
          }
          if constexpr (MODE == LOSS_DW) {
#pragma unroll
            for (int h = 0; h < COLUMNS; h += 32) {
#pragma unroll
              for (int e = h; e < h + 32; ++e) v[e] *= by;
              put32(h, *reinterpret_cast<float(*)[32]>(v + h));
            }
            const int y = o * TILE_M + in_tile;
            write_lines(A.v0 + y, x, A.columns - y, A.H - x);
          } else {
            open();
#pragma unroll
            for (int p = 0; p < 8; ++p)
              put(p, __float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]), __float_as_uint(v[4 * p + 2]), __float_as_uint(v[4 * p + 3]));
            send(x, split * A.rows_pad + i * TILE_M + in_tile, A.add != 0);
          }
        }
      }
      empties(buf);
    }
    if (MODE == LOSS_DX && lane == 0) tma_store_wait_all();
  }
  __syncthreads();
  if constexpr (PAIR) {  // neither block's shared or tensor memory is given back while the other's products use it
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

template <int MODE, bool PAIR, bool LONG>
__global__ void __launch_bounds__(LOSS_THREADS, 1)
    loss_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mc,
                const __grid_constant__ CUtensorMap mo, const __grid_constant__ LossArgs A) {
  loss_products<MODE, PAIR, LONG>(ma, mb, mc, mo, A, blockIdx.x, gridDim.x);
}

// Both products of few rows: dw is bound by writing to memory, dx by reading w, so blocks of both kinds (`dx_blocks` of dx,
// spread evenly) keep memory busy both ways at once.
__global__ void __launch_bounds__(LOSS_THREADS, 1)
    loss_both_kernel(const __grid_constant__ CUtensorMap wa, const __grid_constant__ CUtensorMap wb, const __grid_constant__ CUtensorMap wc,
                     const __grid_constant__ CUtensorMap xa, const __grid_constant__ CUtensorMap xb, const __grid_constant__ CUtensorMap xo,
                     const __grid_constant__ LossArgs W, const __grid_constant__ LossArgs X, int dx_blocks) {
  const int block = static_cast<int>(blockIdx.x), blocks = static_cast<int>(gridDim.x), before = block * dx_blocks / blocks;
  if ((block + 1) * dx_blocks / blocks > before)
    loss_products<LOSS_DX, false, false>(xa, xb, xb, xo, X, before, dx_blocks);
  else
    loss_products<LOSS_DW, false, false>(wa, wb, wc, wc, W, block - before, blocks - dx_blocks);
}

// ------------------------------------------------------------------------------ a teacher's tokens
struct LossListArgs {
  const int32_t* ids;
  const float* teacher;
  int32_t* sorted;      // [T][K], ascending, those that are not there last
  float *q, *logq;      // [T][K] in that order
  int32_t* state;       // [T]: 1 takes part, 0 left out, -1 has an id of V or more
  float over;           // 1 / s
  int T, V, K;
};

// A warp for each row: up to four tokens a lane, ranked by comparison with all others (equal ids by their place).
__global__ void __launch_bounds__(128) loss_list_kernel(const __grid_constant__ LossListArgs A) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= A.T) return;
  int id[4], rank[4] = {};
  float l[4], top = -INFINITY;
  bool beyond = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i * 32 + lane;
    id[i] = k < A.K ? A.ids[t * A.K + k] : -1;
    l[i] = k < A.K ? A.teacher[t * A.K + k] : -INFINITY;
    if (id[i] < 0 || l[i] == -INFINITY) {
      id[i] = LOSS_NO_ID;
    } else {
      beyond |= id[i] >= A.V;
      top = max_nan(top, l[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, o));
  // the largest first, then the temperature: finite values of any size stay so, or have no share
  float p[4], total = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l[i] = (l[i] - top) * A.over;
    p[i] = id[i] != LOSS_NO_ID ? expf(l[i]) : 0.0f;
    total += p[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL_MASK, total, o);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j * 32 >= A.K) break;
    for (int from = 0; from < 32; ++from) {
      const int other = __shfl_sync(FULL_MASK, id[j], from), place = j * 32 + from;
#pragma unroll
      for (int i = 0; i < 4; ++i) rank[i] += other < id[i] || (other == id[i] && place < i * 32 + lane);
    }
  }
  const float log_total = logf(total);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i * 32 + lane >= A.K) continue;
    A.sorted[t * A.K + rank[i]] = id[i];
    A.q[t * A.K + rank[i]] = id[i] != LOSS_NO_ID ? p[i] / total : 0.0f;
    A.logq[t * A.K + rank[i]] = l[i] - log_total;
  }
  const bool any = __any_sync(FULL_MASK, id[0] != LOSS_NO_ID || id[1] != LOSS_NO_ID || id[2] != LOSS_NO_ID || id[3] != LOSS_NO_ID);
  beyond = __any_sync(FULL_MASK, beyond);
  if (lane == 0) A.state[t] = beyond ? -1 : any ? 1 : 0;
}

// ------------------------------------------------------------------------------ rows that take part
struct LossPlanArgs {
  const int32_t *ids, *state;  // state NULL: by the row's one id
  const float* g;              // NULL: no gradient
  const __nv_bfloat16* x;
  int64_t ldx;
  int32_t *rows, *place, *count;  // [T] both ways (place -1 and -2: left out, id of V or more), and how many
  float* by;                      // max |g|, or g where all rows have the same ...
  int32_t* same;                  // ... which this tells
  __nv_bfloat16 *copy, *scaled;   // the rows, and with unequal g also scaled by g / max |g|
  float *loss, *lse;              // of rows that do not take part
  __nv_bfloat16* dx;
  int64_t lddx;
  int T, V, H, tile_rows;
};

__device__ __forceinline__ int loss_state(const int32_t* ids, const int32_t* state, int64_t t, int V) {
  if (state != nullptr) return state[t];
  return ids[t] < 0 ? 0 : ids[t] < V ? 1 : -1;
}

// What all rows together say: where row `mine` goes among those that take part, how many there are, and their scale.  By the
// whole block, each thread a run of rows; `A.place` and `A.rows` are filled in where `writes`.
struct LossPlan {
  int place, count;
  float by;
  bool same;
};
template <int THREADS>
__device__ __forceinline__ LossPlan loss_plan(const LossPlanArgs& A, int mine, bool writes) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int sums[WARPS], found;
  __shared__ float tops[WARPS], lows[WARPS], highs[WARPS];
  const int each = (A.T + THREADS - 1) / THREADS, from = min(A.T, static_cast<int>(threadIdx.x) * each), to = min(A.T, from + each);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto takes_part = [&](int t) { return loss_state(A.ids, A.state, t, A.V) == 1 && (A.g == nullptr || A.g[t] != 0.0f); };
  int own = 0;
  float top = 0.0f, low = INFINITY, high = -INFINITY;  // of |g| where it is finite, and of g
  for (int t = from; t < to; ++t) {
    if (!takes_part(t)) continue;
    ++own;
    if (A.g == nullptr) continue;
    const float g = A.g[t];
    if (fabsf(g) < INFINITY) top = fmaxf(top, fabsf(g));
    low = g == g ? fminf(low, g) : -INFINITY;
    high = fmaxf(high, g);
  }
  int before = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL_MASK, before, o);
    if (lane >= o) before += v;
    top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
    low = fminf(low, __shfl_xor_sync(FULL_MASK, low, o));
    high = fmaxf(high, __shfl_xor_sync(FULL_MASK, high, o));
  }
  if (lane == 31) sums[warp] = before;
  if (lane == 0) tops[warp] = top, lows[warp] = low, highs[warp] = high;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  int all = 0, r = before - own;
  for (int w = 0; w < WARPS; ++w) {
    r += w < warp ? sums[w] : 0;
    all += sums[w];
    top = fmaxf(top, tops[w]);
    low = fminf(low, lows[w]);
    high = fmaxf(high, highs[w]);
  }
  for (int t = from; t < to; ++t) {
    const bool part = takes_part(t);
    const int place = part ? r++ : loss_state(A.ids, A.state, t, A.V) < 0 ? -2 : -1;
    if (t == mine) found = place;
    if (writes) {
      if (part) A.rows[place] = t;
      A.place[t] = place;
    }
  }
  __syncthreads();
  const bool same = low == high && fabsf(low) < INFINITY;
  return {found, all, same ? low : top > 0.0f ? top : 1.0f, same};
}
__device__ __forceinline__ void loss_plan_told(const LossPlanArgs& A, const LossPlan& p) {
  *A.count = p.count;
  *A.same = p.same;
  *A.by = p.by;
}

// One block numbers the rows that take part in ascending order.
__global__ void __launch_bounds__(1024) loss_plan_kernel(const __grid_constant__ LossPlanArgs A) {
  grid_dep_wait();
  grid_dep_launch();
  const LossPlan p = loss_plan<1024>(A, -1, true);
  if (threadIdx.x == 0) loss_plan_told(A, p);
}

// A block for each row: copies of those that take part, results of the others.  The last `tile_rows` blocks write the rows
// of zeros behind the last one, up to the end of its tile.  PLANS: there was no plan, and each block makes it for itself, which
// for up to LOSS_PLAN_ROWS rows takes less than a kernel before this one (128 rows: 1 us against 4).
constexpr int LOSS_PLAN_ROWS = 1024;
template <bool PLANS>
__global__ void __launch_bounds__(128) loss_gather_kernel(const __grid_constant__ LossPlanArgs A) {
  grid_dep_wait();
  grid_dep_launch();
  const int packs = A.H / 8, t = static_cast<int>(blockIdx.x);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  LossPlan p{};
  if constexpr (PLANS) {
    p = loss_plan<128>(A, t, t == 0);
    if (t == 0 && threadIdx.x == 0) loss_plan_told(A, p);
  } else {
    p = {t < A.T ? A.place[t] : -1, *A.count, *A.by, *A.same != 0};
  }
  const bool scales = A.scaled != nullptr && !p.same;
  int64_t r = p.place;
  if (t >= A.T) {
    r = static_cast<int64_t>(p.count) + t - A.T;
    if (r >= (p.count + A.tile_rows - 1) / A.tile_rows * A.tile_rows) return;
    for (int i = threadIdx.x; i < packs; i += 128) {
      reinterpret_cast<uint4*>(A.copy + r * A.H)[i] = zero;
      if (scales) reinterpret_cast<uint4*>(A.scaled + r * A.H)[i] = zero;
    }
    return;
  }
  if (r < 0) {
    if (threadIdx.x == 0 && A.loss != nullptr) A.loss[t] = r == -2 ? NAN : 0.0f;
    if (threadIdx.x == 0 && A.lse != nullptr) A.lse[t] = r == -2 ? NAN : 0.0f;
    if (A.dx != nullptr)
      for (int i = threadIdx.x; i < packs; i += 128) reinterpret_cast<uint4*>(A.dx + t * A.lddx)[i] = zero;
    return;
  }
  const float by = scales ? A.g[t] / p.by : 1.0f;
  for (int i = threadIdx.x; i < packs; i += 128) {
    const Pack<__nv_bfloat16, 8> v = reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(A.x + t * A.ldx)[i];
    reinterpret_cast<Pack<__nv_bfloat16, 8>*>(A.copy + r * A.H)[i] = v;
    if (scales) {
      float f[8];
      unpack(v, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= by;
      reinterpret_cast<Pack<__nv_bfloat16, 8>*>(A.scaled + r * A.H)[i] = pack<__nv_bfloat16>(f);
    }
  }
}

// ------------------------------------------------------------------------------ results
struct LossJoinArgs {
  const int32_t *count, *rows, *ids, *state;
  const float *q, *logq, *picks;
  const float2* parts;
  float *loss, *lse;
  float s;
  int T, V, K, row0, n_tiles;
};

// A block for each row: the tiles' sums together (of a cross entropy those of the other ids), and the loss.
__global__ void __launch_bounds__(128) loss_join_kernel(const __grid_constant__ LossJoinArgs A) {
  __shared__ float joined[4][2];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t r = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (A.count != nullptr && A.row0 + r >= *A.count) return;
  const int64_t t = A.rows != nullptr ? A.rows[A.row0 + r] : A.row0 + r;
  const int state = loss_state(A.ids, A.state, t, A.V);
  if (state != 1) {
    if (threadIdx.x == 0) A.loss[t] = A.lse[t] = state < 0 ? NAN : 0.0f;
    return;
  }
  // sums of nothing but exp(-inf) say nothing of their exponent
  const float2* parts = A.parts + r * A.n_tiles;
  float top = -INFINITY;
  for (int i = threadIdx.x; i < A.n_tiles; i += 128)
    if (parts[i].y != 0.0f) top = fmaxf(top, parts[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
  if (lane == 0) joined[warp][0] = top;
  __syncthreads();
  top = fmaxf(fmaxf(joined[0][0], joined[1][0]), fmaxf(joined[2][0], joined[3][0]));
  float total = 0.0f;
  for (int i = threadIdx.x; i < A.n_tiles; i += 128)
    if (parts[i].y != 0.0f) total += parts[i].y < INFINITY ? parts[i].y * ex2_approx(parts[i].x - top) : parts[i].y;
  total = warp_sum(total);
  if (lane == 0) joined[warp][1] = total;
  __syncthreads();
  if (warp > 0) return;
  total = (joined[0][1] + joined[1][1]) + (joined[2][1] + joined[3][1]);
  float lse = total > 0.0f || total != total ? top * 0.693147180559945309417f + logf(total) : -INFINITY, loss = 0.0f;
  if (A.q == nullptr) {
    // log(1 + exp(d)), d = the others' lse - z: a loss near 0 keeps its digits
    const float z = A.picks[r], d = lse - z, more = log1pf(expf(-fabsf(d)));
    const bool infinite = z == INFINITY || lse == INFINITY;
    loss = z == INFINITY ? NAN : fmaxf(d, 0.0f) + (d != d ? d : more);
    lse = infinite && z == z && lse == lse ? INFINITY : (d > 0.0f ? lse : z) + (d != d ? d : more);
  } else {
    for (int k = lane; k < A.K; k += 32) {
      const float q = A.q[t * A.K + k];
      if (q != 0.0f) loss += q * (A.logq[t * A.K + k] - (A.picks[r * A.K + k] / A.s - lse));
    }
    loss = warp_sum(loss) * A.s * A.s;
  }
  if (lane == 0) {
    A.loss[t] = loss;
    A.lse[t] = lse;
  }
}

struct LossDxArgs {
  const int32_t *count, *rows;
  const float *parts, *g;
  __nv_bfloat16* dx;
  int64_t lddx, part;  // elements from one part to the next
  float s;
  int H, splits, k_piece, units, width, tile_rows;  // as LOSS_DX had them
  bool whole;                                       // one piece: one part of it has been written already
};

// dx from its parts, added up in order: 512 columns of a row a block, four a thread.
__global__ void __launch_bounds__(128) loss_dx_kernel(const __grid_constant__ LossDxArgs A) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t r = blockIdx.x;
  const int count = *A.count, c = (blockIdx.y * 128 + threadIdx.x) * 4;
  if (r >= count) return;
  const int tiles = (count + A.tile_rows - 1) / A.tile_rows * ((A.H + A.width - 1) / A.width);
  const int splits = loss_splits(tiles, A.k_piece, A.splits, A.units, A.tile_rows == 256);
  if (c >= A.H || (A.whole && splits == 1)) return;
  const int64_t t = A.rows[r];
  const float by = A.g[t] * A.s;
  const float* at = A.parts + r * A.H + c;
  float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int p = 0; p < splits; ++p, at += A.part) {
    const float4 v = *reinterpret_cast<const float4*>(at);
    f.x += v.x, f.y += v.y, f.z += v.z, f.w += v.w;
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(f.x * by, f.y * by), hi = __floats2bfloat162_rn(f.z * by, f.w * by);
  *reinterpret_cast<uint2*>(A.dx + t * A.lddx + c) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// dw of no rows.
__global__ void __launch_bounds__(256) loss_zero_kernel(__nv_bfloat16* dw, int64_t lddw, int H) {
  grid_dep_wait();
  grid_dep_launch();
  uint4* to = reinterpret_cast<uint4*>(dw + blockIdx.x * lddw);
  for (int i = threadIdx.x; i < H / 8; i += 256) to[i] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace strata
