// strata_loss.cu -- host side of the losses over a vocabulary and their gradients (include/strata_train.h).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/strata_train.h"
#include "strata_chain.h"
#include "strata_host.h"
#include "strata_loss.cuh"

using strata::host_fail;

namespace {

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int cuda_fail(cudaError_t e, const char* what) { return host_fail(STRATA_ECUDA, "%s: %s", what, cudaGetErrorString(e)); }

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;
using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, strata::LossArgs);
Kernel sums_kernel(bool pair, bool is_long) {
  return pair ? (is_long ? strata::loss_kernel<strata::LOSS_SUMS, true, true> : strata::loss_kernel<strata::LOSS_SUMS, true, false>)
              : (is_long ? strata::loss_kernel<strata::LOSS_SUMS, false, true> : strata::loss_kernel<strata::LOSS_SUMS, false, false>);
}
Kernel diffs_kernel(bool pair, bool is_long) {
  return pair ? (is_long ? strata::loss_kernel<strata::LOSS_DIFFS, true, true> : strata::loss_kernel<strata::LOSS_DIFFS, true, false>)
              : (is_long ? strata::loss_kernel<strata::LOSS_DIFFS, false, true> : strata::loss_kernel<strata::LOSS_DIFFS, false, false>);
}

// What the calls need of a device, found at the first call on it.  A failure is not kept: the next call tries again.
struct Device {
  std::mutex lock;
  std::atomic<bool> known{false};
  EncodeFn encode = nullptr;
};

cudaError_t find_device(Device& d) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
  if (e == cudaSuccess && (found != cudaDriverEntryPointSuccess || p == nullptr)) e = cudaErrorNotSupported;
  d.encode = reinterpret_cast<EncodeFn>(p);
  auto shared = [&](Kernel kernel, int mode, bool pair) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, strata::loss_smem(mode, pair));
  };
  for (bool pair : {false, true}) {
    for (bool is_long : {false, true}) {
      shared(sums_kernel(pair, is_long), strata::LOSS_SUMS, pair);
      shared(diffs_kernel(pair, is_long), strata::LOSS_DIFFS, pair);
    }
  }
  shared(strata::loss_kernel<strata::LOSS_DW, true, false>, strata::LOSS_DW, true);
  shared(strata::loss_kernel<strata::LOSS_DX, true, false>, strata::LOSS_DX, true);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(strata::loss_both_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, strata::loss_smem(strata::LOSS_DW, false));
  return e;
}

int device_entry(int id, const Device** dev) {
  static Device devices[64];
  if (id < 0 || id >= 64) return host_fail(STRATA_ERANGE, "device %d", id);
  Device& d = devices[id];
  if (!d.known.load(std::memory_order_acquire)) {
    try {
      std::lock_guard<std::mutex> hold(d.lock);
      if (!d.known.load()) {
        if (const cudaError_t e = find_device(d); e != cudaSuccess) return cuda_fail(e, "device setup");
        d.known.store(true, std::memory_order_release);
      }
    } catch (...) {  // no exception leaves a C call
      return host_fail(STRATA_ECUDA, "device setup");
    }
  }
  *dev = &d;
  return STRATA_OK;
}

// A map of `rows` rows of `width` elements (bfloat16, or float32), cut into boxes of 128 bytes by `box_rows`.
bool map_rows(const Device& dev, CUtensorMap* m, bool f32, const void* p, int64_t width, int64_t rows, int64_t ld, int box_rows) {
  const cuuint64_t esz = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(ld) * esz};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(strata::LOSS_LINE / esz), static_cast<cuuint32_t>(box_rows)}, ones[2] = {1, 1};
  return dev.encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------------------ a call's plan
// It goes by the sizes alone, so that the workspace's size can be asked for without a device.  Its tiles are for as many SMs; on a device
// with fewer as many blocks are launched as that one has, since each goes through the tiles by its number and has an SM alone.
constexpr int SMS = strata::GB300_SMS, PAIRS = SMS / 2;
// Blocks of dx's product where few rows have both in one launch, dw's in the others.  dx's bring d's rows beside w, dw's write.  Which
// share is better goes by the width, hardly by the rows (the way back of 5, 32 and 96 rows, us, 54 blocks and 64: x 177,128 x 480 106, 108,
// 117 and 113, 114, 117; x 150,000 x 744 148, 153, 159 and 155, 160, 165; x 84,656 x 984 112, 115, 118 and 118, 122, 126; x 150,000 x 1,024
// 164, 165, 180 and 161, 161, 176; x 150,000 x 1,280 205, 209, 231 and 196, 197, 214; 32 and 96 rows x 248,320 x 2,048 494, 539 and 482, 511;
// x 32,000 x 4,096 145, 158 and 141, 155.  Of 64 rows 64 blocks are better for narrow ones too, 111 and 107 at a width of 480.)
int dx_blocks_for(int H) { return H < 1024 ? 54 : 64; }
constexpr int ALONE_ROWS = 128;           // a call with more may work by pairs of SMs
// A score that takes longer works on a copy of the rows that take part.  The copy costs 4 us and rows that are left out save their
// share: with a quarter of them it pays from here on (ns).
constexpr double MOVE_COST = 30000;
constexpr int SLAB_ROWS = 8192;           // whose tiles' sums are held at a time
// Of differences held at a time: pieces that would stay in L2 have more turns that leave SMs idle (distillation of 1,024 rows x
// 248,320 x 2,048, us: 64 MB 2,694, 128 MB 2,633, 512 MB 2,559, 2 GB 2,564).  And of parts of dx.
constexpr int64_t PIECE_BYTES = int64_t{512} << 20, PARTS_BYTES = int64_t{256} << 20;

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

// Whether a score's sums are taken out of tensor memory on the way.  Of few rows from twice the width on: up to there narrow tiles'
// two sums cost less, beyond they are too long.  (Narrow tiles and these, us: 64 rows x 248,320 x 2,048 153.0 and 158.2, x 2,056
// 185.6 and 173.6; 96 x 64,000 x 4,096 81.6 and 84.7; 16 x 8,000 x 8,192 28.9 and 30.0, and lse off by 1.8e-6 and 4e-7.)
bool sums_long(int rows, int H) { return H > 64 * strata::LOSS_LONG * (rows <= ALONE_ROWS ? 2 : 1); }

// Tiles of the logits: of two SMs or of one, and how many columns, by what their turns cost.  In ns, as measured: a step of 64
// of a pair's tile (columns + 80), and each turn 900 beside it; tiles of one SM cost 20 % more a step and 600, but bring fewer
// rows that are none, and start and hand their tiles over 4 us sooner.  (Score of 300 rows x 32,000 x 1,024, us: one SM 20, two
// 28; 512 x 128,000 x 1,024: 98 and 82; the gradients of 300 x 8,000 x 2,048: 51 and 59, of 1,024 x 32,000 x 1,024: 168 and
// 152.)  On the way back two more products follow, in which pairs gain another tenth.
struct Tiles {
  bool pair;
  int columns;
  double cost;
};
Tiles tiles_for(int rows, int64_t columns, int H, bool grad) {
  Tiles best{false, 256, 1e30};
  const double steps = static_cast<double>(tiles_of(H, 64));
  for (bool pair : {false, true}) {
    if (pair && rows <= ALONE_ROWS) break;
    const int64_t row_tiles = tiles_of(rows, pair ? 256 : 128);
    const int step = pair || grad ? 32 : 16;
    // few rows are bound by reading w whatever the tiles: scores of wider ones take narrow tiles, which have two sums
    for (int bn = rows <= ALONE_ROWS && !grad && H > 512 && !sums_long(rows, H) ? 128 : 256; bn >= (grad ? 64 : pair ? 128 : 16); bn -= step) {
      const double turns = static_cast<double>(tiles_of(row_tiles * tiles_of(columns, bn), pair ? PAIRS : SMS));
      double cost = pair ? turns * (steps * (bn + 80) + 900) + 4000 : rows <= ALONE_ROWS ? turns * (bn + 16) : turns * (steps * (bn + 80) * 1.2 + 600);
      if (grad && !pair) cost *= 1.1;
      if (cost < best.cost) best = {pair, bn, cost};
    }
  }
  return best;
}

struct Plan {
  int T, V, H, K;
  bool lists, grad, pair, moved;    // a teacher's tokens; for a gradient; tiles of two SMs; works on a copy of the rows
  int tile_rows = 0, rows_pad = 0, d_rows = 0, slab = 0, bn = 0;  // slab: rows whose tiles' sums are held at a time; bn: columns of a tile of logits
  int run = 0;                                // steps of 64 whose products one sum of a logit has in tensor memory
  int piece = 0, splits = 1, width = 0;       // ids of a piece; most parts of dx; columns of a tile of dw and dx
  int64_t sorted = 0, q = 0, logq = 0, state = 0, rows = 0, place = 0, count = 0, by = 0, same = 0, copy = 0, scaled = 0, parts = 0, picks = 0,
          d = 0, dx = 0, bytes = 0;           // places in the workspace

  Plan(int T, int V, int H, int K, bool grad)
      : T(T), V(V), H(H), K(std::max(K, 1)), lists(K > 0), grad(grad), pair(false), moved(grad) {
    slab = std::min(T, SLAB_ROWS);
    // a piece of the vocabulary whose differences are held at a time: 2,048 ids of the most rows
    const int64_t most = PIECE_BYTES / (tiles_of(T, 256) * 512);
    const Tiles scores = tiles_for(slab, V, H, false), tiles = grad ? tiles_for(T, std::min<int64_t>(most, V), H, true) : scores;
    // a gradient's logits are added up as its score's were, whatever its tiles
    const int steps = static_cast<int>(tiles_of(H, 64));
    run = is_long() ? strata::LOSS_LONG : scores.columns <= 128 ? (steps + 1) / 2 : steps;
    pair = tiles.pair;
    moved = grad || (T > ALONE_ROWS && (tiles.cost > MOVE_COST || T > slab));
    bn = tiles.columns;
    tile_rows = pair ? 256 : 128;
    auto take = [&](int64_t n) {
      const int64_t at = bytes;
      bytes += (n + 255) / 256 * 256;
      return at;
    };
    const int64_t t = T, words = t * this->K * 4;
    rows_pad = static_cast<int>(tiles_of(T, tile_rows) * tile_rows);
    if (lists) {
      sorted = take(words);
      q = take(words);
      logq = take(words);
      state = take(t * 4);
    }
    if (moved) {
      rows = take(t * 4);
      place = take(t * 4);
      count = take(4);
      by = take(4);
      same = take(4);
      copy = take(static_cast<int64_t>(rows_pad) * H * 2);
    }
    if (!grad) {
      parts = take(slab * tiles_of(V, bn) * (is_long() ? 16 : 8));
      picks = take(static_cast<int64_t>(slab) * this->K * 4);
      return;
    }
    scaled = take(static_cast<int64_t>(rows_pad) * H * 2);
    piece = static_cast<int>((V <= most ? tiles_of(V, 2 * bn) : most / (2 * bn)) * 2 * bn);  // whole tiles, and steps of 64
    d_rows = T <= ALONE_ROWS ? (T + 7) / 8 * 8 : rows_pad;  // few rows: no more than they have; beyond, copies bring zeros
    d = take(static_cast<int64_t>(d_rows) * piece * 2);
    width = H <= 128 ? 128 : 256;
    const int64_t one = static_cast<int64_t>(rows_pad) * H * 4;
    splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(32, PARTS_BYTES / one)));
    dx = take(splits * one);
  }
  bool is_long() const { return sums_long(T, H); }
  bool in_runs() const { return run < tiles_of(H, 64); }  // of a gradient, whose tiles may be too wide for two sums
};

struct Loss {
  const void *x, *w;
  int64_t ldx, ldw;
  int T, V, H, K;
  const int32_t* ids;
  const float* teacher;  // NULL: a cross entropy
  float temperature;
  void* workspace;
  int64_t workspace_bytes;
  void* stream;
};

// What both directions check.
int check(const Loss& C, bool grad) {
  if (C.T < 0 || C.V < 1) return host_fail(STRATA_EINVAL, "T=%d V=%d", C.T, C.V);
  if (C.T > STRATA_LOSS_MAX_ROWS) return host_fail(STRATA_ERANGE, "T=%d above %d", C.T, STRATA_LOSS_MAX_ROWS);
  if (C.V > STRATA_MAX_VOCAB) return host_fail(STRATA_ERANGE, "V=%d above %d", C.V, STRATA_MAX_VOCAB);
  if (C.H < 1 || C.H > STRATA_LOSS_MAX_WIDTH) return host_fail(STRATA_ERANGE, "H=%d outside 1..%d", C.H, STRATA_LOSS_MAX_WIDTH);
  if (C.K < 0 || C.K > STRATA_DISTILL_MAX_TOKENS) return host_fail(STRATA_ERANGE, "K=%d outside 1..%d", C.K, STRATA_DISTILL_MAX_TOKENS);
  if (C.ldx < C.H || C.ldw < C.H) return host_fail(STRATA_EINVAL, "a row stride below H=%d", C.H);
  if (!(C.temperature >= 0.001f && C.temperature <= 1000.0f))
    return host_fail(STRATA_EINVAL, "temperature=%g outside 0.001..1000", static_cast<double>(C.temperature));
  if (C.H % 8 != 0 || C.ldx % 8 != 0 || C.ldw % 8 != 0) return host_fail(STRATA_EALIGN, "H or a row stride is not a multiple of 8");
  if (C.T == 0) return STRATA_OK;
  if (C.x == nullptr || C.w == nullptr || C.ids == nullptr || (C.K > 0 && C.teacher == nullptr))
    return host_fail(STRATA_EINVAL, "null x, w, ids or teacher");
  if (misaligned(C.x, 16) || misaligned(C.w, 16)) return host_fail(STRATA_EALIGN, "x or w not 16-byte aligned");
  if (misaligned(C.ids, 4) || misaligned(C.teacher, 4)) return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  const int64_t need = strata_loss_workspace(C.T, C.V, C.H, C.K, grad);
  if (C.workspace == nullptr || C.workspace_bytes < need || misaligned(C.workspace, 256))
    return host_fail(STRATA_EINVAL, "the workspace needs %lld bytes on 256 bytes of alignment", static_cast<long long>(need));
  return STRATA_OK;
}

template <typename T>
T* at(const Loss& C, int64_t place) {
  return reinterpret_cast<T*>(static_cast<char*>(C.workspace) + place);
}

// Launches one kernel after another, the first as the chain of its stream says.
struct Run {
  void* stream;
  bool overlaps;
  int sms;  // that the products' blocks have
  cudaError_t e = cudaSuccess;
  template <typename K, typename... A>
  void operator()(K kernel, unsigned grid, unsigned block, size_t smem, unsigned cluster, A... args) {
    if (e != cudaSuccess) return;
    e = strata::Launch(grid, block, smem, stream, overlaps, cluster)(kernel, args...);
    overlaps = true;
  }
  template <int MODE>
  void products(Kernel kernel, bool pair, int64_t tiles, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const CUtensorMap& o,
                const strata::LossArgs& A) {
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(tiles, pair ? sms / 2 : sms)) * (pair ? 2 : 1);
    (*this)(kernel, blocks, strata::LOSS_THREADS, strata::loss_smem(MODE, pair), pair ? 2 : 1, a, b, c, o, A);
  }
};

// A teacher's tokens in order, and the copies of the rows that take part.
void launch_plan(Run& run, const Loss& C, const Plan& P, const float* g, float* loss, float* lse, void* dx, int64_t lddx) {
  if (P.lists) {
    const strata::LossListArgs A{C.ids, C.teacher, at<int32_t>(C, P.sorted), at<float>(C, P.q), at<float>(C, P.logq), at<int32_t>(C, P.state),
                                 1.0f / C.temperature, C.T, C.V, P.K};
    run(strata::loss_list_kernel, static_cast<unsigned>((C.T + 3) / 4), 128, 0, 1, A);
  }
  if (!P.moved) return;
  strata::LossPlanArgs A{};
  A.ids = C.ids;
  A.state = P.lists ? at<int32_t>(C, P.state) : nullptr;
  A.g = g;
  A.x = static_cast<const __nv_bfloat16*>(C.x);
  A.ldx = C.ldx;
  A.rows = at<int32_t>(C, P.rows);
  A.place = at<int32_t>(C, P.place);
  A.count = at<int32_t>(C, P.count);
  A.by = at<float>(C, P.by);
  A.same = at<int32_t>(C, P.same);
  A.copy = at<__nv_bfloat16>(C, P.copy);
  A.scaled = P.grad ? at<__nv_bfloat16>(C, P.scaled) : nullptr;
  A.loss = loss;
  A.lse = lse;
  A.dx = static_cast<__nv_bfloat16*>(dx);
  A.lddx = lddx;
  A.T = C.T;
  A.V = C.V;
  A.H = C.H;
  A.tile_rows = P.tile_rows;
  const bool plans = C.T <= strata::LOSS_PLAN_ROWS;
  if (!plans) run(strata::loss_plan_kernel, 1, 1024, 0, 1, A);
  run(plans ? strata::loss_gather_kernel<true> : strata::loss_gather_kernel<false>, static_cast<unsigned>(C.T + P.tile_rows), 128, 0, 1, A);
}

strata::LossArgs products_args(const Loss& C, const Plan& P, uint32_t* errors) {
  strata::LossArgs A{};
  A.count = P.moved ? at<int32_t>(C, P.count) : nullptr;
  A.rows = P.moved ? at<int32_t>(C, P.rows) : nullptr;
  A.ids = P.lists ? at<int32_t>(C, P.sorted) : C.ids;
  A.q = P.lists ? at<float>(C, P.q) : nullptr;
  A.errors = errors;
  A.scale = static_cast<float>(1.4426950408889634 / static_cast<double>(C.temperature));
  A.dw_scale = C.temperature;
  A.T = C.T;
  A.V = C.V;
  A.H = C.H;
  A.K = P.K;
  A.rows_most = P.rows_pad;
  A.rows_pad = P.rows_pad;
  A.a_rows = std::min(128, (C.T + 7) / 8 * 8);
  A.d_rows = P.d_rows;
  A.run = P.run;
  A.splits = P.splits;
  A.k_piece = P.piece / 64;
  return A;
}

int forward(const Loss& C, float* loss, float* lse, const char* name) {
  if (const int rc = check(C, false); rc != STRATA_OK) return rc;
  if (C.T == 0) return STRATA_OK;
  if (loss == nullptr || lse == nullptr) return host_fail(STRATA_EINVAL, "null loss or lse");
  if (misaligned(loss, 4) || misaligned(lse, 4)) return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  uint32_t* errors = nullptr;
  int device = 0, sms = 0;
  if (const int rc = strata::tail_device(&device, &errors, &sms); rc != STRATA_OK) return rc;
  sms = std::max(2, std::min(SMS, sms));
  const Device* dev = nullptr;
  if (const int rc = device_entry(device, &dev); rc != STRATA_OK) return rc;
  const Plan P(C.T, C.V, C.H, C.K, false);
  CUtensorMap mx, mw;
  if (!(P.moved ? map_rows(*dev, &mx, false, at<void>(C, P.copy), C.H, P.rows_pad, C.H, 128)
                : map_rows(*dev, &mx, false, C.x, C.H, C.T, C.ldx, P.pair ? 128 : std::min(128, (C.T + 7) / 8 * 8))))
    return host_fail(STRATA_EINVAL, "x cannot be mapped");
  if (!map_rows(*dev, &mw, false, C.w, C.H, C.V, C.ldw, P.pair ? P.bn / 2 : P.bn)) return host_fail(STRATA_EINVAL, "w cannot be mapped");
  const cudaError_t e = strata::launch_operator(device, C.stream, [&](bool overlaps) {
    Run run{C.stream, overlaps, sms};
    launch_plan(run, C, P, nullptr, loss, lse, nullptr, 0);
    strata::LossArgs A = products_args(C, P, errors);
    A.columns = C.V;
    A.bn = P.bn;
    A.n_tiles = static_cast<int>(tiles_of(C.V, P.bn));
    A.parts = at<float2>(C, P.parts);
    A.picks = at<float>(C, P.picks);
    strata::LossJoinArgs J{A.count, A.rows, A.ids, P.lists ? at<int32_t>(C, P.state) : nullptr, A.q, P.lists ? at<float>(C, P.logq) : nullptr,
                           A.picks, A.parts, loss, lse, C.temperature, C.T, C.V, P.K, 0, A.n_tiles * (P.is_long() ? 2 : 1)};
    for (int row0 = 0; row0 < C.T; row0 += P.slab) {
      A.row0 = J.row0 = row0;
      A.rows_most = std::min(P.slab, C.T - row0);
      run.products<strata::LOSS_SUMS>(sums_kernel(P.pair, P.is_long()), P.pair, tiles_of(A.rows_most, P.tile_rows) * A.n_tiles, mx, mw, mw, mw, A);
      run(strata::loss_join_kernel, static_cast<unsigned>(A.rows_most), 128, 0, 1, J);
    }
    return run.e;
  });
  return e == cudaSuccess ? STRATA_OK : cuda_fail(e, name);
}

int backward(const Loss& C, const float* lse, const float* g, void* dx, int64_t lddx, void* dw, int64_t lddw, const char* name) {
  if (dx == nullptr && dw == nullptr && C.T != 0) return host_fail(STRATA_EINVAL, "no output");  // an empty dx may have no address
  if (const int rc = check(C, true); rc != STRATA_OK) return rc;
  if ((dx != nullptr && lddx < C.H) || (dw != nullptr && lddw < C.H)) return host_fail(STRATA_EINVAL, "a row stride below H=%d", C.H);
  if (misaligned(dx, 16) || misaligned(dw, 16)) return host_fail(STRATA_EALIGN, "dx or dw not 16-byte aligned");
  if ((dx != nullptr && lddx % 8 != 0) || (dw != nullptr && lddw % 8 != 0)) return host_fail(STRATA_EALIGN, "a row stride is not a multiple of 8");
  if (C.T == 0 && dw == nullptr) return STRATA_OK;
  if (C.T > 0 && (lse == nullptr || g == nullptr)) return host_fail(STRATA_EINVAL, "null lse or g");
  if (misaligned(lse, 4) || misaligned(g, 4)) return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  uint32_t* errors = nullptr;
  int device = 0, sms = 0;
  if (const int rc = strata::tail_device(&device, &errors, &sms); rc != STRATA_OK) return rc;
  sms = std::max(2, std::min(SMS, sms));
  cudaError_t e;
  if (C.T == 0) {
    e = strata::launch_operator(device, C.stream, [&](bool overlaps) {
      return strata::Launch(static_cast<unsigned>(C.V), 256, 0, C.stream, overlaps)(strata::loss_zero_kernel, static_cast<__nv_bfloat16*>(dw), lddw, C.H);
    });
    return e == cudaSuccess ? STRATA_OK : cuda_fail(e, name);
  }
  const Device* dev = nullptr;
  if (const int rc = device_entry(device, &dev); rc != STRATA_OK) return rc;
  const Plan P(C.T, C.V, C.H, C.K, true);
  CUtensorMap mx, mw, mxo, mxs, mwo, md, mds, mdx;
  const int a_rows = P.pair ? 128 : std::min(128, (C.T + 7) / 8 * 8);
  if (!map_rows(*dev, &mx, false, at<void>(C, P.copy), C.H, P.rows_pad, C.H, a_rows) ||
      !map_rows(*dev, &mxo, false, at<void>(C, P.copy), C.H, P.d_rows, C.H, 64) ||
      !map_rows(*dev, &mxs, false, at<void>(C, P.scaled), C.H, P.d_rows, C.H, 64) ||
      !map_rows(*dev, &mdx, true, at<void>(C, P.dx), C.H, static_cast<int64_t>(P.splits) * P.rows_pad, C.H, 32))
    return host_fail(STRATA_EINVAL, "the workspace cannot be mapped");
  if (!map_rows(*dev, &mw, false, C.w, C.H, C.V, C.ldw, P.pair ? P.bn / 2 : P.bn) || !map_rows(*dev, &mwo, false, C.w, C.H, C.V, C.ldw, 64))
    return host_fail(STRATA_EINVAL, "w cannot be mapped");
  e = strata::launch_operator(device, C.stream, [&](bool overlaps) {
    Run run{C.stream, overlaps, sms};
    launch_plan(run, C, P, g, nullptr, nullptr, dx, lddx);
    strata::LossArgs A = products_args(C, P, errors);
    const int dx_share = C.T <= ALONE_ROWS ? dx_blocks_for(C.H) : SMS / 2;  // of many rows both products cost the same
    const int dx_blocks = dx == nullptr ? 0 : dw == nullptr ? sms : std::max(1, dx_share * sms / SMS);
    A.units = P.pair ? sms / 2 : dx_blocks;
    A.lse = lse;
    A.wide = !misaligned(dw, 32) && lddw % 16 == 0 && C.H % 16 == 0;
    A.by = at<float>(C, P.by);
    A.same = at<int32_t>(C, P.same);
    const bool whole = P.piece >= C.V;
    A.dx = whole ? static_cast<__nv_bfloat16*>(dx) : nullptr;
    A.lddx = lddx;
    A.g = g;
    const int64_t row_tiles = P.rows_pad / P.tile_rows, across = tiles_of(C.H, P.width);
    for (int v0 = 0; v0 < C.V; v0 += P.piece) {
      A.v0 = v0;
      A.columns = std::min(P.piece, C.V - v0);
      // what lies beyond the piece's ids is not looked at, but read as zeros
      if (!map_rows(*dev, &md, false, at<void>(C, P.d), A.columns, P.d_rows, P.piece, a_rows) ||
          !map_rows(*dev, &mds, false, at<void>(C, P.d), A.columns, P.d_rows, P.piece, 64))
        return cudaErrorInvalidValue;
      A.bn = P.bn;
      A.n_tiles = static_cast<int>(tiles_of(A.columns, P.bn));
      A.out = at<__nv_bfloat16>(C, P.d);
      A.ldo = P.piece;
      run.products<strata::LOSS_DIFFS>(diffs_kernel(P.pair, P.in_runs()), P.pair, row_tiles * A.n_tiles, mx, mw, mw, mw, A);
      A.bn = P.width;
      A.n_tiles = static_cast<int>(across);
      A.out = static_cast<__nv_bfloat16*>(dw);
      A.ldo = lddw;
      A.add = v0 > 0;
      if (!P.pair) {
        run(strata::loss_both_kernel, static_cast<unsigned>(sms), strata::LOSS_THREADS, strata::loss_smem(strata::LOSS_DW, false), 1, mds, mxo, mxs, md, mwo, mdx, A, A, dx_blocks);
        continue;
      }
      if (dw != nullptr)
        run.products<strata::LOSS_DW>(strata::loss_kernel<strata::LOSS_DW, true, false>, true, tiles_of(A.columns, 256) * across, mds, mxo, mxs, mxs, A);
      if (dx != nullptr)
        run.products<strata::LOSS_DX>(strata::loss_kernel<strata::LOSS_DX, true, false>, true, row_tiles * across * P.splits, md, mwo, mwo, mdx, A);
    }
    if (dx != nullptr) {
      const strata::LossDxArgs D{A.count, A.rows, at<float>(C, P.dx), g, static_cast<__nv_bfloat16*>(dx), lddx, static_cast<int64_t>(P.rows_pad) * C.H,
                                 C.temperature, C.H, P.splits, A.k_piece, A.units, P.width, P.tile_rows, whole};
      if (run.e == cudaSuccess) {
        strata::Launch launch(static_cast<unsigned>(C.T), 128, 0, C.stream, run.overlaps);
        launch.cfg.gridDim.y = static_cast<unsigned>((C.H + 511) / 512);
        run.e = launch(strata::loss_dx_kernel, D);
      }
    }
    return run.e;
  });
  return e == cudaSuccess ? STRATA_OK : cuda_fail(e, name);
}

}  // namespace

extern "C" int64_t strata_loss_workspace(int T, int V, int H, int K, int grad) {
  if (T <= 0 || V <= 0 || H <= 0 || K < 0) return 0;
  if (T > STRATA_LOSS_MAX_ROWS || V > STRATA_MAX_VOCAB || H > STRATA_LOSS_MAX_WIDTH || K > STRATA_DISTILL_MAX_TOKENS) return 0;  // calls that are refused
  return Plan(T, V, H, K, grad != 0).bytes;
}

extern "C" int strata_cross_entropy_rows(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H, const int32_t* ids,
                                         float* loss, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  return forward(Loss{x, w, ldx, ldw, T, V, H, 0, ids, nullptr, 1.0f, workspace, workspace_bytes, stream}, loss, lse, "strata_cross_entropy_rows");
}

extern "C" int strata_cross_entropy_grad(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H, const int32_t* ids,
                                         const float* lse, const float* g, void* dx, int64_t lddx, void* dw, int64_t lddw, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
  return backward(Loss{x, w, ldx, ldw, T, V, H, 0, ids, nullptr, 1.0f, workspace, workspace_bytes, stream}, lse, g, dx, lddx, dw, lddw,
                  "strata_cross_entropy_grad");
}

extern "C" int strata_distill_rows(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H, int K, const int32_t* ids,
                                   const float* teacher, float temperature, float* loss, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  if (K < 1) return host_fail(STRATA_ERANGE, "K=%d outside 1..%d", K, STRATA_DISTILL_MAX_TOKENS);
  return forward(Loss{x, w, ldx, ldw, T, V, H, K, ids, teacher, temperature, workspace, workspace_bytes, stream}, loss, lse, "strata_distill_rows");
}

extern "C" int strata_distill_grad(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H, int K, const int32_t* ids,
                                   const float* teacher, float temperature, const float* lse, const float* g, void* dx, int64_t lddx, void* dw,
                                   int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream) {
  if (K < 1) return host_fail(STRATA_ERANGE, "K=%d outside 1..%d", K, STRATA_DISTILL_MAX_TOKENS);
  return backward(Loss{x, w, ldx, ldw, T, V, H, K, ids, teacher, temperature, workspace, workspace_bytes, stream}, lse, g, dx, lddx, dw, lddw,
                  "strata_distill_grad");
}
