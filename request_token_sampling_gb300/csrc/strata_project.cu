// strata_project.cu -- host side of strata_project_rows (include/strata_tail.h).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/strata_tail.h"
#include "strata_chain.h"
#include "strata_host.h"
#include "strata_project.cuh"

using strata::host_fail;

namespace {

// Bits of STRATA_DEVERR_* that kernels of these calls raise (one word on each device).
__device__ uint32_t g_tail_errors;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int cuda_fail(cudaError_t e, const char* what) {
  return host_fail(STRATA_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;
using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, strata::ProjectArgs);

constexpr int MAX_ROWS = 1 << 19;  // rows times adapters of a tile count in 31 bits
constexpr int MAX_OUTPUTS = INT32_MAX - 2 * strata::PROJ_M;  // outputs of the last tile, and beyond N, too
constexpr int SHRINK_ROWS = 32;     // a call with more takes its inner rows from the tensor cores
constexpr int BN_SIZES[4] = {16, 32, 64, 128};

template <int BN>
Kernel pick(bool f8, bool split) {
  return f8 ? (split ? strata::project_kernel<BN, true, true> : strata::project_kernel<BN, true, false>)
            : (split ? strata::project_kernel<BN, false, true> : strata::project_kernel<BN, false, false>);
}

Kernel kernel_for(int bn, bool f8, bool split) {
  return bn == 16 ? pick<16>(f8, split) : bn == 32 ? pick<32>(f8, split) : bn == 64 ? pick<64>(f8, split) : pick<128>(f8, split);
}

// What the calls need to know of a device, found at the first call on it that needs it.  A failure is not kept: the
// next call tries again.
struct Device {
  std::mutex lock;
  std::atomic<bool> known{false}, projects{false};
  int sms = 0;
  uint32_t* errors = nullptr;
  EncodeFn encode = nullptr;  // this and the kernels' attributes: for projections
};

cudaError_t find_device(Device& d, int id) {
  void* p = nullptr;
  cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, id);
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&p, g_tail_errors);
  d.errors = static_cast<uint32_t*>(p);
  return e;
}

cudaError_t find_projects(Device& d) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
  if (e == cudaSuccess && (found != cudaDriverEntryPointSuccess || p == nullptr)) e = cudaErrorNotSupported;
  d.encode = reinterpret_cast<EncodeFn>(p);
  auto shared = [&](const void* kernel, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  for (int bn : BN_SIZES)
    for (int i = 0; i < 4; ++i) shared(reinterpret_cast<const void*>(kernel_for(bn, i & 1, i & 2)), strata::proj_smem(bn));
  shared(reinterpret_cast<const void*>(strata::pair_kernel), strata::pair_smem());
  shared(reinterpret_cast<const void*>(strata::inner_kernel<false>), strata::inner_smem(false));
  shared(reinterpret_cast<const void*>(strata::inner_kernel<true>), strata::inner_smem(true));
  return e;
}

// A map of `dims` (innermost first; strides in bytes of the outer ones) cut into boxes of `box`.
bool encode(EncodeFn fn, CUtensorMap* m, bool bytes, int rank, const void* p, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, int line) {
  const cuuint32_t ones[3] = {1, 1, 1};
  return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims,
            strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            line == 0   ? CU_TENSOR_MAP_SWIZZLE_NONE
            : line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B 
            : line == 64  ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_32B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a tile on one SM: the fewest that hold the call's rows, 128 for more.  The products' cost grows
// with them, and w is read once for each tile of rows.
int tile_rows(int T) {
  for (int bn : BN_SIZES)
    if (T <= bn) return bn;
  return 128;
}

// Few tiles leave most of the GPU idle: then a cluster of blocks shares a tile, as many as still fit beside
// one another and have two stages each.
int split_ranks(int64_t tiles, int k_stages, int sms) {
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= sms && k_stages >= ranks * 4) ranks *= 2;
  return ranks;
}

// Rows of a tile of the pair kernel, or 0 where tiles on one SM take less time.  A 64-deep stage of a pair's tile
// of r rows was measured at about 1.02 (80 + r) ns (193 ns for 128 rows, 265 for 192, 342 for 256), one of 128 x 128 on
// one SM at 220 ns: the cost of a choice is its tiles one after another on an SM times that.
int pair_rows(int T, int N, int k_stages, bool adapters, int sms) {
  const int64_t n_pairs = (N + 2 * strata::PROJ_M - 1) / (2 * strata::PROJ_M), n_tiles = (N + strata::PROJ_M - 1) / strata::PROJ_M;
  auto waves = [](int64_t tiles, int64_t at_once) { return (tiles + at_once - 1) / at_once; };
  const int64_t tiles = n_tiles * ((T + 127) / 128);
  int64_t best = waves(tiles, sms) * 215 / split_ranks(tiles, k_stages, sms);
  int rows = 0;
  for (int r = 256; r >= 64; r -= 16) {
    const int64_t t_tiles = (T + r - 1) / r;
    const int64_t cost = waves(n_pairs * t_tiles + (adapters ? t_tiles : 0), sms / 2) * (80 + r);  // mostly one unit a tile of rows
    if (cost < best) {
      best = cost;
      rows = r;
    }
  }
  return rows;
}

// The current device's entry, with what projections need or without, or an error code.
int current_device(const Device** dev, int* device, bool projects) {
  static Device devices[64];
  int id = -1;
  cudaError_t e = cudaGetDevice(&id);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (id >= 64) return host_fail(STRATA_ERANGE, "device %d", id);
  Device& d = devices[id];
  if (!(projects ? d.projects : d.known).load(std::memory_order_acquire)) {
    try {
      std::lock_guard<std::mutex> hold(d.lock);
      if (!d.known.load()) {
        if ((e = find_device(d, id)) != cudaSuccess) return cuda_fail(e, "device setup");
        d.known.store(true, std::memory_order_release);
      }
      if (projects && !d.projects.load()) {
        if ((e = find_projects(d)) != cudaSuccess) return cuda_fail(e, "device setup");
        d.projects.store(true, std::memory_order_release);
      }
    } catch (...) {  // no exception leaves a C call
      return host_fail(STRATA_ECUDA, "device setup");
    }
  }
  *dev = &d;
  *device = id;
  return STRATA_OK;
}

// The lists and the words beside them.
int64_t lists_bytes(int t_tiles, int bn) { return (static_cast<int64_t>(t_tiles) * (bn + 2) * 4 + 255) / 256 * 256; }

}  // namespace

int strata::tail_device(int* device, uint32_t** errors, int* sms) {
  const Device* dev = nullptr;
  const int rc = current_device(&dev, device, false);
  if (rc != STRATA_OK) return rc;
  *errors = dev->errors;
  *sms = dev->sms;
  return STRATA_OK;
}

namespace {

// The inner rows are spread out over a tile's adapters, so the workspace grows with rows times adapters.  Calls that
// would take more than 256 MB go through their rows in slabs that use it one after another, of 2,048 rows at least (a layer of
// 4,096 outputs keeps the GPU busy for two waves).
int slab_rows(int S, int R) {
  const int64_t rows = (int64_t{256} << 20) / (static_cast<int64_t>(std::min(S, 256)) * R * 4) / 256 * 256;
  return static_cast<int>(std::min<int64_t>(MAX_ROWS, std::max<int64_t>(2048, rows)));
}

}  // namespace

extern "C" int64_t strata_project_workspace(int T, int S, int R) {
  if (T <= 0 || S <= 0 || R <= 0) return 0;
  if (T <= 128) return lists_bytes(1, 128) + static_cast<int64_t>(std::min(S, T)) * tile_rows(T) * R * 4;
  // whatever tiles the call takes: 64 to 256 rows each
  const int rows = std::min(T, slab_rows(S, R));
  return lists_bytes((rows + 63) / 64, 256) + (static_cast<int64_t>(rows) + 256) * std::min(S, 256) * R * 4;
}

// One slab of rows, its arguments checked.
static int project_slab(const Device& dev, int device, const void* x, int64_t ldx, const float* x_scale, const void* w, int64_t ldw,
                        const float* w_scale, bool f8, int T, int N, int K, const void* a, const void* b, int S, int R,
                        const int32_t* row_adapter, const float* adapter_scale, __nv_bfloat16* y, int64_t ldy, void* workspace,
                        void* stream) {
  const int64_t esz = f8 ? 1 : 2;
  const cuuint32_t elems = f8 ? 128 : 64;
  const int k_stages = (K + static_cast<int>(elems) - 1) / static_cast<int>(elems);
  const int pair = T > 128 && !f8 ? pair_rows(T, N, k_stages, S > 0, dev.sms) : 0;  // tiles of two SMs
  const int bn = pair > 0 ? pair : tile_rows(T), t_tiles = (T + bn - 1) / bn;
  const int n_tiles = pair > 0 ? (N + 2 * strata::PROJ_M - 1) / (2 * strata::PROJ_M) : (N + strata::PROJ_M - 1) / strata::PROJ_M;
  const int64_t tiles = static_cast<int64_t>(t_tiles) * n_tiles;
  const int most = std::min(S, std::min(T, bn));
  // tiles of inner products before the pairs' others
  const int64_t units = pair > 0 && S > 0 ? static_cast<int64_t>(t_tiles) * ((most * R + 2 * strata::PROJ_M - 1) / (2 * strata::PROJ_M)) : 0;
  if (tiles + units > INT32_MAX - dev.sms) return host_fail(STRATA_ERANGE, "T=%d N=%d", T, N);  // they are counted in steps of the grid
  strata::ProjectArgs A{};
  A.x = x;
  A.x_scale = x_scale;
  A.w_scale = w_scale;
  A.adapter_scale = adapter_scale;
  A.a = static_cast<const __nv_bfloat16*>(a);
  A.b = static_cast<const __nv_bfloat16*>(b);
  A.row_adapter = row_adapter;
  A.y = y;
  A.lists = static_cast<int32_t*>(workspace);
  A.ready = static_cast<uint32_t*>(workspace) + static_cast<int64_t>(t_tiles) * (bn + 1);
  A.spread = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(workspace) + lists_bytes(t_tiles, bn));
  const bool beside = pair == 0 && strata::parts_beside(bn);
  A.low = beside ? static_cast<int64_t>(bn) * R : static_cast<int64_t>(t_tiles) * most * bn * R;
  A.block_rows = beside ? 2 * bn : bn;
  A.errors = dev.errors;
  A.ldx = ldx;
  A.ldy = ldy;
  A.T = T;
  A.N = N;
  A.K = K;
  A.S = S;
  A.R = R;
  A.most = most;
  A.rank_block = R % 64 == 0 ? 64 : R % 32 == 0 ? 32 : 16;
  A.n_tiles = n_tiles;
  A.t_tiles = t_tiles;
  A.tile_rows = bn;

  CUtensorMap mw, mx, mb{}, mh{}, ma{}, mt{};
  const int box_rows = R % 128 == 0 ? 128 : R % 64 == 0 ? 64 : R % 32 == 0 ? 32 : 16;  // of a, in one copy
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldw * esz)};
    const cuuint32_t box[2] = {elems, strata::PROJ_M};
    if (!encode(dev.encode, &mw, f8, 2, w, dims, strides, box, 128)) return host_fail(STRATA_EINVAL, "w cannot be mapped");
  }
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldx * esz)};
    const cuuint32_t box[2] = {elems, static_cast<cuuint32_t>(pair > 0 ? bn / 2 : bn)};
    if (!encode(dev.encode, &mx, f8, 2, x, dims, strides, box, 128)) return host_fail(STRATA_EINVAL, "x cannot be mapped");
  }
  if (S > 0) {
    const cuuint64_t r = static_cast<cuuint64_t>(R), bytes = r * 2;
    const cuuint64_t dims[3] = {r, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(S)};
    const cuuint64_t strides[2] = {bytes, bytes * static_cast<cuuint64_t>(N)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(A.rank_block), strata::PROJ_M, 1};
    if (!encode(dev.encode, &mb, false, 3, b, dims, strides, box, A.rank_block * 2)) return host_fail(STRATA_EINVAL, "b cannot be mapped");
    const cuuint64_t hdims[2] = {r, 2 * static_cast<cuuint64_t>(t_tiles) * most * bn};
    const cuuint32_t hbox[2] = {static_cast<cuuint32_t>(A.rank_block), static_cast<cuuint32_t>(pair > 0 ? bn / 2 : A.block_rows)};
    if (!encode(dev.encode, &mh, false, 2, A.spread, hdims, strides, hbox, A.rank_block * 2))
      return host_fail(STRATA_EINVAL, "the workspace cannot be mapped");
    if (T > SHRINK_ROWS) {
      const cuuint64_t adims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(S) * R};
      const cuuint64_t astrides[1] = {static_cast<cuuint64_t>(K) * 2};
      const cuuint32_t abox[2] = {64, static_cast<cuuint32_t>(box_rows)};
      if (!encode(dev.encode, &ma, false, 2, a, adims, astrides, abox, 128)) return host_fail(STRATA_EINVAL, "a cannot be mapped");
    }
    if (T > SHRINK_ROWS && pair == 0) {
      const cuuint64_t xdims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(T)};
      const cuuint64_t xstrides[1] = {static_cast<cuuint64_t>(ldx * esz)};
      const cuuint32_t xbox[2] = {64, static_cast<cuuint32_t>(bn)};
      if (!encode(dev.encode, &mt, f8, 2, x, xdims, xstrides, xbox, f8 ? 0 : 128)) return host_fail(STRATA_EINVAL, "x cannot be mapped");
    }
  }
  // the inner rows (or, for pairs, the lists alone)
  auto launch_inner = [&](bool overlaps) {
    if (T <= SHRINK_ROWS) {
      strata::Launch launch(static_cast<unsigned>(T), 256, 0, stream, overlaps);
      launch.cfg.gridDim.y = static_cast<unsigned>(R / 8);
      return f8 ? launch(strata::shrink_kernel<__nv_fp8_e4m3>, A, bn) : launch(strata::shrink_kernel<__nv_bfloat16>, A, bn);
    }
    if (pair > 0) return strata::Launch(static_cast<unsigned>(t_tiles), 256, 0, stream, overlaps)(strata::plan_kernel, A);
    // clusters of a tile: one where the tiles fill the GPU, as many as there can be work for where they do not
    const int groups = std::min((most * R + strata::PROJ_M - 1) / strata::PROJ_M,
                                std::max(1, dev.sms / strata::INNER_SPLIT / t_tiles));
    const strata::Launch launch(static_cast<unsigned>(t_tiles) * groups * strata::INNER_SPLIT, strata::PROJ_THREADS,
                                strata::inner_smem(f8), stream, overlaps, strata::INNER_SPLIT);
    return launch(f8 ? strata::inner_kernel<true> : strata::inner_kernel<false>, ma, mt, A, groups, box_rows);
  };
  // set up while the inner rows' kernel runs, and waits for it before what it wrote; up to 32 rows its blocks also run beside
  // that one's, above they start on the SMs that it leaves free
  auto launch_products = [&](bool overlaps) {
    if (pair > 0) {
      const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(tiles + units, dev.sms / 2));
      return strata::Launch(2 * pairs, strata::PROJ_THREADS, strata::pair_smem(), stream, overlaps, 1, S > 0)(
          strata::pair_kernel, mw, mx, mb, mh, ma, A, box_rows);
    }
    const int ranks = split_ranks(tiles, k_stages, dev.sms);
    const unsigned grid = static_cast<unsigned>(ranks > 1 ? tiles * ranks : std::min<int64_t>(tiles, dev.sms));
    return strata::Launch(grid, strata::PROJ_THREADS, strata::proj_smem(bn), stream, overlaps, static_cast<unsigned>(ranks))(
        kernel_for(bn, f8, ranks > 1), mw, mx, mb, mh, A);
  };
  const cudaError_t e = strata::launch_operator(device, stream, [&](bool overlaps) {
    if (S == 0) return launch_products(overlaps);
    const cudaError_t first = launch_inner(overlaps);
    return first == cudaSuccess ? launch_products(true) : first;
  });
  return e == cudaSuccess ? STRATA_OK : cuda_fail(e, "strata_project_rows");
}

extern "C" int strata_project_rows(const void* x, int64_t ldx, const float* x_scale, const void* w, int64_t ldw,
                                   const float* w_scale, int dtype, int T, int N, int K, const void* a, const void* b,
                                   int S, int R, const int32_t* row_adapter, const float* adapter_scale, void* y,
                                   int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream) {
  if (dtype != STRATA_DTYPE_BF16 && dtype != STRATA_DTYPE_F8) return host_fail(STRATA_EINVAL, "dtype %d", dtype);
  if (T < 0 || N < 1) return host_fail(STRATA_EINVAL, "T=%d N=%d", T, N);
  if (T > MAX_ROWS) return host_fail(STRATA_ERANGE, "T=%d above %d", T, MAX_ROWS);
  if (N > MAX_OUTPUTS) return host_fail(STRATA_ERANGE, "N=%d above %d", N, MAX_OUTPUTS);
  if (K < 1 || K > STRATA_TAIL_MAX_WIDTH) return host_fail(STRATA_ERANGE, "K=%d outside 1..%d", K, STRATA_TAIL_MAX_WIDTH);
  if (S < 0 || S > STRATA_TAIL_MAX_ADAPTERS) return host_fail(STRATA_ERANGE, "S=%d outside 0..%d", S, STRATA_TAIL_MAX_ADAPTERS);
  if (S > 0 && (R < 16 || R > STRATA_TAIL_MAX_RANK || R % 16 != 0))
    return host_fail(STRATA_ERANGE, "R=%d is not a multiple of 16 up to %d", R, STRATA_TAIL_MAX_RANK);
  if (ldx < K || ldw < K || ldy < N) return host_fail(STRATA_EINVAL, "a row stride below its row");
  const bool f8 = dtype == STRATA_DTYPE_F8;
  if ((x_scale != nullptr) != f8 || (w_scale != nullptr) != f8)
    return host_fail(STRATA_EINVAL, "x_scale and w_scale go with 8-bit rows, and only with them");
  if (T == 0) return STRATA_OK;
  if (x == nullptr || w == nullptr || y == nullptr) return host_fail(STRATA_EINVAL, "null x, w or y");
  if (S > 0 && (a == nullptr || b == nullptr || row_adapter == nullptr || adapter_scale == nullptr))
    return host_fail(STRATA_EINVAL, "null a, b, row_adapter or adapter_scale");
  const int64_t esz = f8 ? 1 : 2;
  if (misaligned(x, 16) || misaligned(w, 16) || (S > 0 && (misaligned(a, 16) || misaligned(b, 16))))
    return host_fail(STRATA_EALIGN, "x, w, a or b not 16-byte aligned");
  if (K * esz % 16 != 0 || ldx * esz % 16 != 0 || ldw * esz % 16 != 0 || (S > 0 && K % 8 != 0))
    return host_fail(STRATA_EALIGN, "K or a row stride is not a multiple of 16 bytes");
  if (misaligned(y, 2) || misaligned(x_scale, 4) || misaligned(w_scale, 4) || misaligned(row_adapter, 4) ||
      misaligned(adapter_scale, 4))
    return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  const int64_t need = strata_project_workspace(T, S, R);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || misaligned(workspace, 256)))
    return host_fail(STRATA_EINVAL, "the workspace needs %lld bytes on 256 bytes of alignment", static_cast<long long>(need));
  const Device* found = nullptr;
  int device = 0;
  if (const int rc = current_device(&found, &device, true); rc != STRATA_OK) return rc;
  const int slab = S > 0 ? slab_rows(S, R) : T;
  for (int t = 0; t < T; t += slab) {
    const int rc = project_slab(*found, device, static_cast<const char*>(x) + t * ldx * esz, ldx, f8 ? x_scale + t : nullptr, w, ldw, w_scale, f8,
                                std::min(slab, T - t), N, K, a, b, S, R, S > 0 ? row_adapter + t : nullptr, adapter_scale,
                                static_cast<__nv_bfloat16*>(y) + t * ldy, ldy, workspace, stream);
    if (rc != STRATA_OK) return rc;
  }
  return STRATA_OK;
}

// The bits and their clearing in one step, which no kernel of another stream comes between.  A call has a word of its
// own for the answer while it waits.
constexpr unsigned ERROR_CALLS = 64;
__device__ uint32_t g_told[ERROR_CALLS];
__global__ void take_errors(unsigned call) { g_told[call] = atomicExch(&g_tail_errors, 0u); }

extern "C" int strata_tail_errors(uint32_t* bits, void* stream) {
  if (bits == nullptr) return host_fail(STRATA_EINVAL, "null bits");
  static std::atomic<unsigned> calls{0};
  static std::mutex busy[ERROR_CALLS];
  try {
    const unsigned call = calls.fetch_add(1) % ERROR_CALLS;
    std::lock_guard<std::mutex> hold(busy[call]);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    take_errors<<<1, 1, 0, s>>>(call);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(bits, g_told, sizeof(*bits), call * sizeof(*bits), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? STRATA_OK : cuda_fail(e, "strata_tail_errors");
  } catch (...) {  // no exception leaves a C call
    return host_fail(STRATA_ECUDA, "strata_tail_errors");
  }
}
