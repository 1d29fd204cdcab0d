// strata_layer_norm.cu -- host side of strata_layer_norm_rows and strata_layer_norm_grad (include/strata_train.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "../../include/strata_train.h"
#include "strata_chain.h"
#include "strata_host.h"
#include "strata_layer_norm.cuh"

using strata::host_fail;

namespace {

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// How a call's rows lie: all on 16 bytes, with a width of whole packs (`packed`); or anywhere, but in all tensors the same way
// (`alike`: packs on the boundaries).
struct Lie {
  const void* first = nullptr;
  int64_t ld = 0;
  int T, n;
  bool packed, alike = true;
  Lie(const void* x, int64_t ldx, int T, int H, int esz) : first(x), ld(ldx), T(T), n(16 / esz), packed(H % (16 / esz) == 0) { look(x, ldx); }
  void look(const void* p, int64_t ldp) {
    if (p == nullptr) return;
    packed = packed && !misaligned(p, 16) && (T == 1 || ldp % n == 0);
    alike = alike && (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(first)) % 16 == 0 && (T == 1 || (ldp - ld) % n == 0);
  }
  void look_column(const void* p) { packed = packed && !misaligned(p, 16); }
};

constexpr int SMS = strata::GB300_SMS, SM_BYTES = 224 * 1024;          // shared memory of an SM for rows on their way
constexpr int BLOCK_WIDTH = 512 * 16, WARP_WIDTH = 32 * 16;

// Registers of a kernel's thread, for the number of its blocks on an SM; found once.
template <typename K>
int registers(K kernel) {
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, kernel) == cudaSuccess ? a.numRegs : 128;
}

// Lets a kernel have an SM's shared memory, once on each device.
template <typename K>
cudaError_t allow_shared(K kernel, std::atomic<uint64_t>& done, int device) {
  const uint64_t bit = uint64_t{1} << (device & 63);
  if ((done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_BYTES);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// How rows go through rings: a block's threads (PER packs each, and the warp of the copies), blocks of an SM (as many as its
// registers, threads and shared memory hold, with two rows on their way at least), and rows on their way.  `ring`: bytes of a
// row in it, `beside`: of the weight.
struct RingShape {
  int threads, blocks, depth;
  size_t smem;
  RingShape(int packs, int per, int copier, int ring, int beside, int regs) {
    threads = ((packs + per - 1) / per + 31) / 32 * 32 + copier;
    blocks = std::max(1, std::min({8, 65536 / ((regs + 7) / 8 * 8 * threads), 2048 / threads, SM_BYTES / (2 * ring + beside + 1024)}));
    depth = std::max(2, std::min(strata::LAYER_NORM_RING, (SM_BYTES / blocks - 1024 - beside) / ring));
    smem = static_cast<size_t>(depth) * ring + beside;
  }
};
// A multiple of eight that leaves each block some rows, or a block for each row.  On a device with fewer SMs there are no more than run
// at a time: one that starts when others end would have its share of the rows still to go through.
int ring_grid(int T, int blocks, int sms = SMS) {
  return T <= SMS ? T : std::max(8, std::min(std::min(sms, SMS) * blocks / 8 * 8, std::max(SMS, T / 8 / 8 * 8)));
}

// The shape of a call, as the root-mean-square norm's: many rows are bound by HBM, a thread takes up to 16
// elements, so that enough bytes are on their way; few rows are bound by latency: a row goes to as many threads as it has packs.
template <typename E, int N, int PER>
cudaError_t launch_forward(const strata::LayerNormArgs& A, int least, bool overlaps, int device, int sms, void* stream) {
  if constexpr (N * PER <= 32 && PER <= 16) {
    const int packs = (A.H + N - 1) / N, need = (packs + PER - 1) / PER;
    if (PER < least || need > strata::layer_norm_most_threads(N, PER)) return launch_forward<E, N, PER * 2>(A, least, overlaps, device, sms, stream);
    constexpr int ROWS = 4;
    if (need <= 32)
      return strata::Launch((static_cast<unsigned>(A.T) + ROWS - 1) / ROWS, 32 * ROWS, 0, stream, overlaps)(strata::layer_norm_kernel<E, N, PER, false>, A);
    return strata::Launch(A.T, (need + 31) / 32 * 32, 0, stream, overlaps)(strata::layer_norm_kernel<E, N, PER, true>, A);
  } else {
    return strata::Launch(A.T, 1024, 0, stream, overlaps)(strata::layer_norm_wide_kernel<E>, A);
  }
}
// Many rows that start anywhere (the boundary is that of rows up to some 2,000 wide: 600 rows x 2,049, us, 6.1 element by element and 6.8
// here, x 1,135 4.4 and 6.3; x 5,003 11.6 and 8.2; 8,192 rows x 1,135 27 and 25).
template <typename E, int PER>
cudaError_t launch_ring(strata::LayerNormArgs A, bool overlaps, int device, int sms, void* stream) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  if constexpr (N * PER <= 16) {
    if ((A.H / N + PER - 1) / PER > strata::LAYER_NORM_RING_THREADS) return launch_ring<E, PER * 2>(A, overlaps, device, sms, stream);
    const int row = (A.H * static_cast<int>(sizeof(E)) + 15) / 16 * 16;
    const auto kernel = strata::layer_norm_ring_kernel<E, PER>;
    static const int regs = registers(kernel);
    const RingShape ring(A.H / N, PER, 32, row * (A.residual != nullptr ? 2 : 1), 2 * row, regs);
    A.depth = ring.depth;
    static std::atomic<uint64_t> allowed{0};
    if (const cudaError_t e = allow_shared(kernel, allowed, device); e != cudaSuccess) return e;
    return strata::Launch(ring_grid(A.T, ring.blocks, sms), ring.threads, ring.smem, stream, overlaps)(kernel, A);
  } else {
    return cudaErrorInvalidValue;  // not reached: wider rows have their own kernels
  }
}
template <typename E>
cudaError_t launch_forward(const strata::LayerNormArgs& A, const Lie& lie, bool overlaps, int device, int sms, void* stream) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  if (A.T >= 4 * SMS && A.H > WARP_WIDTH && A.H <= BLOCK_WIDTH && lie.alike && !lie.packed) return launch_ring<E, 1>(A, overlaps, device, sms, stream);
  const int packs = A.H / (lie.packed ? N : 1);
  const int least = A.T < 2 * SMS ? 1 : packs > 64 ? 4 : packs > 32 ? 2 : 1;
  return lie.packed ? launch_forward<E, N, 1>(A, least, overlaps, device, sms, stream) : launch_forward<E, 1, 1>(A, least, overlaps, device, sms, stream);
}

// Groups of rows whose sums over rows are kept apart, until the last kernel adds them up: those of a block.  Rows too wide for a
// ring have few, for the sake of the workspace.
constexpr int WIDE_GROUPS = 16;
int grad_groups(int T, int H) {
  if (H > BLOCK_WIDTH) return std::min(T, WIDE_GROUPS);
  if (H > WARP_WIDTH) return ring_grid(T, 4);
  return std::min((T - 1) / strata::LAYER_NORM_GRAD_WARPS + 1, SMS * 2);
}

// Narrow rows by warps; wider ones that lie in no common way by a block, element by element.
template <typename E, int N, int PER, bool SHIFT>
cudaError_t launch_rows(const strata::LayerNormGradArgs& A, bool overlaps, int device, int sms, void* stream) {
  if constexpr (N * PER <= 16) {
    const int need = (A.H / N + PER - 1) / PER;
    if (A.H <= WARP_WIDTH) {
      if (need > 32) return launch_rows<E, N, PER * 2, SHIFT>(A, overlaps, device, sms, stream);
      return strata::Launch(A.groups, 32 * strata::LAYER_NORM_GRAD_WARPS, static_cast<size_t>((A.H + N - 1) / N * N) * 8, stream, overlaps)(
          strata::layer_norm_grad_kernel<E, N, PER, false, SHIFT>, A);
    }
    if (need > strata::layer_norm_grad_most_threads(N, PER)) return launch_rows<E, N, PER * 2, SHIFT>(A, overlaps, device, sms, stream);
    if constexpr (N == 1)
      return strata::Launch(A.groups, (need + 31) / 32 * 32, 0, stream, overlaps)(strata::layer_norm_grad_kernel<E, N, PER, true, false>, A);
  }
  return cudaErrorInvalidValue;  // not reached: wider rows have their own kernels
}

// Rows through a ring: as many on their way as an SM's shared memory has room for beside its other blocks.
template <typename E, int PER, bool SHIFT>
cudaError_t launch_ring(strata::LayerNormGradArgs& A, bool overlaps, int device, int sms, void* stream) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  if constexpr (N * PER <= 16) {
    const int need = (A.H / N + PER - 1) / PER;
    if (need > strata::layer_norm_grad_ring_threads(N, PER)) return launch_ring<E, PER * 2, SHIFT>(A, overlaps, device, sms, stream);
    const int row = (A.H * static_cast<int>(sizeof(E)) + 15) / 16 * 16;
    const auto kernel = strata::layer_norm_grad_ring_kernel<E, PER, SHIFT>;
    static const int regs = registers(kernel);
    const RingShape ring(A.H / N, PER, strata::layer_norm_copier(N, PER), row * (A.dresidual != nullptr ? 3 : 2), row, regs);
    A.depth = ring.depth;
    A.groups = std::min(A.groups, ring_grid(A.T, ring.blocks, sms));
    static std::atomic<uint64_t> allowed{0};
    if (const cudaError_t e = allow_shared(kernel, allowed, device); e != cudaSuccess) return e;
    return strata::Launch(A.groups, ring.threads, ring.smem, stream, overlaps)(kernel, A);
  } else {
    return cudaErrorInvalidValue;  // not reached: wider rows have their own kernels
  }
}

template <typename E>
cudaError_t launch_grad(strata::LayerNormGradArgs A, const Lie& lie, bool overlaps, int device, int sms, void* stream) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  cudaError_t e = cudaSuccess;
  if (A.T > 0) {
    if (A.H <= BLOCK_WIDTH) {
      const bool warps = A.H <= WARP_WIDTH;
      e = lie.packed  ? (warps ? launch_rows<E, N, 1, false>(A, overlaps, device, sms, stream) : launch_ring<E, 1, false>(A, overlaps, device, sms, stream))
          : lie.alike ? (warps ? launch_rows<E, N, 1, true>(A, overlaps, device, sms, stream) : launch_ring<E, 1, true>(A, overlaps, device, sms, stream))
                      : launch_rows<E, 1, 1, false>(A, overlaps, device, sms, stream);
      overlaps = true;
    } else {  // the sums first: dx may be dy or x
      if (A.part != nullptr) {
        strata::Launch launch((A.H + 255) / 256, 256, 0, stream, overlaps);
        launch.cfg.gridDim.y = static_cast<unsigned>(A.groups);
        e = launch(strata::layer_norm_grad_columns_kernel<E>, A);
        overlaps = true;
      }
      if (e == cudaSuccess && A.dx != nullptr) {
        e = strata::Launch(A.T, 1024, 0, stream, overlaps)(strata::layer_norm_grad_wide_kernel<E>, A);
        overlaps = true;
      }
    }
  }
  if (e != cudaSuccess || A.part == nullptr) return e;
  strata::Launch launch((A.H + 31) / 32, 1024, 0, stream, overlaps);
  launch.cfg.gridDim.y = 2;
  return launch(strata::layer_norm_sum_kernel<E>, A);
}

}  // namespace

extern "C" int strata_layer_norm_rows(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                      const void* bias, int dtype, int T, int H, float eps, void* residual_out, int64_t ldro,
                                      void* y, int64_t ldy, float* mean, float* rstd, void* stream) {
  if (dtype != STRATA_DTYPE_F32 && dtype != STRATA_DTYPE_BF16) return host_fail(STRATA_EINVAL, "dtype %d", dtype);
  if (T < 0) return host_fail(STRATA_EINVAL, "T=%d", T);
  if (H < 1 || H > STRATA_TAIL_MAX_WIDTH) return host_fail(STRATA_ERANGE, "H=%d outside 1..%d", H, STRATA_TAIL_MAX_WIDTH);
  if (!(eps >= 0.0f)) return host_fail(STRATA_EINVAL, "eps=%g is not a number of 0 or more", static_cast<double>(eps));
  if (ldx < H || (residual != nullptr && ldr < H) || (residual_out != nullptr && ldro < H) || (y != nullptr && ldy < H))
    return host_fail(STRATA_EINVAL, "a row stride below H=%d", H);
  if (T == 0) return STRATA_OK;
  if (residual_out == nullptr && y == nullptr && mean == nullptr && rstd == nullptr) return host_fail(STRATA_EINVAL, "no output");
  if (x == nullptr || weight == nullptr) return host_fail(STRATA_EINVAL, "null x or weight");
  const uintptr_t esz = dtype == STRATA_DTYPE_F32 ? 4 : 2;
  if (misaligned(x, esz) || misaligned(residual, esz) || misaligned(weight, esz) || misaligned(bias, esz) || misaligned(residual_out, esz) ||
      misaligned(y, esz) || misaligned(mean, 4) || misaligned(rstd, 4))
    return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  strata::LayerNormArgs A{x, residual, weight, bias, residual_out, y, mean, rstd, ldx, ldr, ldro, ldy, nullptr, T, H, eps, 0};
  int device = 0, sms = 0;
  if (const int rc = strata::tail_device(&device, &A.errors, &sms); rc != STRATA_OK) return rc;
  Lie lie(x, ldx, T, H, static_cast<int>(esz));
  lie.look(residual, ldr);
  lie.look(residual_out, ldro);
  lie.look(y, ldy);
  lie.look_column(weight);
  lie.look_column(bias);
  const cudaError_t e = strata::launch_operator(device, stream, [&](bool overlaps) {
    return dtype == STRATA_DTYPE_F32 ? launch_forward<float>(A, lie, overlaps, device, sms, stream) : launch_forward<__nv_bfloat16>(A, lie, overlaps, device, sms, stream);
  });
  return e == cudaSuccess ? STRATA_OK : host_fail(STRATA_ECUDA, "strata_layer_norm_rows: %s", cudaGetErrorString(e));
}

extern "C" int64_t strata_layer_norm_workspace(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return static_cast<int64_t>(grad_groups(T, H)) * 2 * H * 4;
}

extern "C" int strata_layer_norm_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight, const float* mean,
                                      const float* rstd, const void* dresidual, int64_t lddr, int dtype, int T, int H, void* dx,
                                      int64_t lddx, void* dweight, void* dbias, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
  if (dtype != STRATA_DTYPE_F32 && dtype != STRATA_DTYPE_BF16) return host_fail(STRATA_EINVAL, "dtype %d", dtype);
  if (T < 0) return host_fail(STRATA_EINVAL, "T=%d", T);
  if (H < 1 || H > STRATA_TAIL_MAX_WIDTH) return host_fail(STRATA_ERANGE, "H=%d outside 1..%d", H, STRATA_TAIL_MAX_WIDTH);
  if (lddy < H || ldx < H || (dresidual != nullptr && lddr < H) || (dx != nullptr && lddx < H))
    return host_fail(STRATA_EINVAL, "a row stride below H=%d", H);
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (T == 0 && !sums) return STRATA_OK;  // an empty dx may have no address
  if (!sums && dx == nullptr) return host_fail(STRATA_EINVAL, "no output");
  const uintptr_t esz = dtype == STRATA_DTYPE_F32 ? 4 : 2;
  if (misaligned(dweight, esz) || misaligned(dbias, esz)) return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  if (T > 0) {
    if (dy == nullptr || x == nullptr || weight == nullptr || mean == nullptr || rstd == nullptr)
      return host_fail(STRATA_EINVAL, "null dy, x, weight, mean or rstd");
    if (misaligned(dy, esz) || misaligned(x, esz) || misaligned(weight, esz) || misaligned(dresidual, esz) || misaligned(dx, esz) ||
        misaligned(mean, 4) || misaligned(rstd, 4))
      return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
    const int64_t need = strata_layer_norm_workspace(T, H);
    if (sums && (workspace == nullptr || workspace_bytes < need || misaligned(workspace, 256)))
      return host_fail(STRATA_EINVAL, "the workspace needs %lld bytes on 256 bytes of alignment", static_cast<long long>(need));
  }
  uint32_t* errors = nullptr;
  int device = 0, sms = 0;
  if (const int rc = strata::tail_device(&device, &errors, &sms); rc != STRATA_OK) return rc;
  Lie lie(x, ldx, T, H, static_cast<int>(esz));
  lie.look(dy, lddy);
  lie.look(dresidual, lddr);
  lie.look(dx, lddx);
  lie.look_column(weight);
  // without rows the sums are those of no groups; the workspace is not touched
  float* part = !sums ? nullptr : T > 0 ? static_cast<float*>(workspace) : static_cast<float*>(dweight != nullptr ? dweight : dbias);
  const strata::LayerNormGradArgs A{dy, x, weight, dresidual, mean, rstd, dx, dweight, dbias, part, errors, lddy, ldx, lddr, lddx, T, H,
                                    T > 0 ? grad_groups(T, H) : 0, 0};
  const cudaError_t e = strata::launch_operator(device, stream, [&](bool overlaps) {
    return dtype == STRATA_DTYPE_F32 ? launch_grad<float>(A, lie, overlaps, device, sms, stream)
                                     : launch_grad<__nv_bfloat16>(A, lie, overlaps, device, sms, stream);
  });
  return e == cudaSuccess ? STRATA_OK : host_fail(STRATA_ECUDA, "strata_layer_norm_grad: %s", cudaGetErrorString(e));
}
