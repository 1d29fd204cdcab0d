// strata_tail.cu -- host side of strata_norm_rows and strata_draw_rows (include/strata_tail.h).
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/strata_tail.h"
#include "strata_chain.h"
#include "strata_draw.cuh"
#include "strata_host.h"
#include "strata_norm.cuh"

using strata::host_fail;

namespace {

constexpr int64_t DRAW_BYTES = 64 * 1024;   // of a row in one block: two such blocks fit an SM
constexpr int DRAW_LEAST = 4096;            // ids of a block below which splitting a row further costs more than it saves
constexpr int64_t DRAW_SMEM = 200 * 1024;   // 2^19 float32 ids in 16 blocks and the block's own part
static_assert(STRATA_MAX_VOCAB * 4 / strata::DRAW_MAX_CLUSTER + sizeof(strata::DrawShared) + 64 <= DRAW_SMEM, "a row fits a cluster");

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// The shape of a call.  Many rows are bound by HBM: a thread takes up to four packs, so that enough
// bytes are on their way, but no more than put the row into one warp (T=8000, H=301: two packs and a warp
// to a row 6.3 us, four 8.7, one and two warps 7.8).  Few rows are bound by
// latency: a row goes to as many threads as it has packs.
template <typename E, int N, int PER, bool SHIFT>
cudaError_t launch_norm(const strata::NormArgs& A, int least, bool overlaps, void* stream) {
  if constexpr (PER <= (N == 1 ? 16 : 4)) {
    const int packs = (A.H + N - 1) / N, need = std::max((packs + PER - 1) / PER, SHIFT ? 2 * (N - 1) : 1);
    if (PER < least || need > strata::norm_most_threads(N, PER)) return launch_norm<E, N, PER * 2, SHIFT>(A, least, overlaps, stream);
    constexpr int ROWS = 4;
    if (need <= 32)
      return strata::Launch((static_cast<unsigned>(A.T) + ROWS - 1) / ROWS, 32 * ROWS, 0, stream, overlaps)(strata::norm_kernel<E, N, PER, false, SHIFT>, A);
    return strata::Launch(A.T, (need + 31) / 32 * 32, 0, stream, overlaps)(strata::norm_kernel<E, N, PER, true, SHIFT>, A);
  } else {
    return strata::Launch(A.T, 1024, 0, stream, overlaps)(strata::norm_wide_kernel<E>, A);
  }
}

// `packed`: all rows lie on 16 bytes; `alike`: they lie anywhere, but all tensors the same way.
template <typename E>
cudaError_t launch_norm(const strata::NormArgs& A, bool packed, bool alike, int sms, bool overlaps, void* stream) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  const int packs = A.H / (packed || alike ? N : 1);
  const int least = A.T < 2 * sms ? 1 : packs > 64 ? 4 : packs > 32 ? 2 : 1;
  return packed  ? launch_norm<E, N, 1, false>(A, least, overlaps, stream)
         : alike ? launch_norm<E, N, 1, true>(A, least, overlaps, stream)
                 : launch_norm<E, 1, 1, false>(A, least, overlaps, stream);
}

}  // namespace

extern "C" int strata_norm_rows(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                int dtype, int T, int H, float eps, void* residual_out, int64_t ldro, void* y,
                                int64_t ldy, void* q, int64_t ldq, float* scale, void* stream) {
  if (dtype != STRATA_DTYPE_F32 && dtype != STRATA_DTYPE_BF16) return host_fail(STRATA_EINVAL, "dtype %d", dtype);
  if (T < 0) return host_fail(STRATA_EINVAL, "T=%d", T);
  if (H < 1 || H > STRATA_TAIL_MAX_WIDTH) return host_fail(STRATA_ERANGE, "H=%d outside 1..%d", H, STRATA_TAIL_MAX_WIDTH);
  if (!(eps >= 0.0f)) return host_fail(STRATA_EINVAL, "eps=%g is not a number of 0 or more", static_cast<double>(eps));
  if (ldx < H || (residual != nullptr && ldr < H) || (residual_out != nullptr && ldro < H) || (y != nullptr && ldy < H) ||
      (q != nullptr && ldq < H))
    return host_fail(STRATA_EINVAL, "a row stride below H=%d", H);
  if (T == 0) return STRATA_OK;
  if (residual_out == nullptr && y == nullptr && q == nullptr) return host_fail(STRATA_EINVAL, "no output");
  if ((q == nullptr) != (scale == nullptr)) return host_fail(STRATA_EINVAL, "q and scale must be given together");
  if (x == nullptr || weight == nullptr) return host_fail(STRATA_EINVAL, "null x or weight");
  const uintptr_t esz = dtype == STRATA_DTYPE_F32 ? 4 : 2;
  if (misaligned(x, esz) || misaligned(residual, esz) || misaligned(weight, esz) || misaligned(residual_out, esz) ||
      misaligned(y, esz) || misaligned(scale, 4))
    return host_fail(STRATA_EALIGN, "a pointer is not aligned to its element");
  strata::NormArgs A{x, residual, weight, residual_out, y, q, scale, ldx, ldr, ldro, ldy, ldq, T, H, eps};
  uint32_t* errors = nullptr;
  int device = 0, sms = 0;
  if (const int rc = strata::tail_device(&device, &errors, &sms); rc != STRATA_OK) return rc;
  // 16 bytes at a time where the width, every stride and every address allow it
  const int64_t n = 16 / static_cast<int64_t>(esz);
  auto fits = [&](const void* p, int64_t ld, int64_t size) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % (n * size)) == 0 && (T == 1 || ld % n == 0));
  };
  const bool packed = H % n == 0 && fits(x, ldx, esz) && fits(residual, ldr, esz) && fits(weight, 0, esz) &&
                      fits(residual_out, ldro, esz) && fits(y, ldy, esz) && fits(q, ldq, 1);
  auto like_x = [&](const void* p, int64_t ld) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(x)) % 16 == 0 && (T == 1 || (ld - ldx) % n == 0));
  };
  const bool alike = like_x(residual, ldr) && like_x(residual_out, ldro) && like_x(y, ldy);
  const cudaError_t e = strata::launch_operator(device, stream, [&](bool overlaps) {
    return dtype == STRATA_DTYPE_F32 ? launch_norm<float>(A, packed, alike, sms, overlaps, stream)
                                     : launch_norm<__nv_bfloat16>(A, packed, alike, sms, overlaps, stream);
  });
  return e == cudaSuccess ? STRATA_OK : host_fail(STRATA_ECUDA, "strata_norm_rows: %s", cudaGetErrorString(e));
}

extern "C" int strata_draw_rows(const void* logits, int dtype, int B, int V, int64_t ld, const float* u,
                                const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                                int32_t* out_ids, float* out_lps, void* stream) {
  if (dtype != STRATA_DTYPE_F32 && dtype != STRATA_DTYPE_BF16) return host_fail(STRATA_EINVAL, "dtype %d", dtype);
  if (B < 0) return host_fail(STRATA_EINVAL, "B=%d", B);
  if (V < 1 || V > STRATA_MAX_VOCAB) return host_fail(STRATA_ERANGE, "V=%d outside 1..%d", V, STRATA_MAX_VOCAB);
  if (ld < V) return host_fail(STRATA_EINVAL, "ld=%lld below V=%d", static_cast<long long>(ld), V);
  if (B == 0) return STRATA_OK;
  if (logits == nullptr || u == nullptr || out_ids == nullptr) return host_fail(STRATA_EINVAL, "null logits, u or out_ids");
  const int64_t esz = dtype == STRATA_DTYPE_F32 ? 4 : 2;
  if (misaligned(logits, 16)) return host_fail(STRATA_EALIGN, "logits not 16-byte aligned");
  if (ld * esz % 16 != 0)
    return host_fail(STRATA_EALIGN, "row stride of %lld bytes not a multiple of 16", static_cast<long long>(ld * esz));
  if (misaligned(u, 4) || misaligned(temperature, 4) || misaligned(top_k, 4) || misaligned(top_p, 4) ||
      misaligned(min_p, 4) || misaligned(out_ids, 4) || misaligned(out_lps, 4))
    return host_fail(STRATA_EALIGN, "a per-row array is not 4-byte aligned");
  uint32_t* errors = nullptr;
  int device = 0, sms = 0;
  if (const int rc = strata::tail_device(&device, &errors, &sms); rc != STRATA_OK) return rc;
  const bool f32 = dtype == STRATA_DTYPE_F32;
  const void* kernel = f32 ? reinterpret_cast<const void*>(strata::draw_kernel<float>)
                           : reinterpret_cast<const void*>(strata::draw_kernel<__nv_bfloat16>);
  // Blocks of a row: as few as hold it with two blocks to an SM, but four where that gives each 2048 ids
  // (a top_k of up to 64 a block takes the short way: 64 rows of 32,000 with a top_k around 100 take 11.6 us,
  // with two blocks to a row 27.8), more where few rows would leave the GPU idle and a block still has
  // DRAW_LEAST ids.
  int ranks = 1;
  while (ranks < strata::DRAW_MAX_CLUSTER &&
         (V * esz > static_cast<int64_t>(ranks) * DRAW_BYTES || (ranks < 4 && V >= 4 * 2048) ||
          (static_cast<int64_t>(B) * ranks * 2 <= sms && V >= ranks * 2 * DRAW_LEAST)))
    ranks *= 2;
  const int chunk = ((V + ranks - 1) / ranks + 15) / 16 * 16;
  const size_t smem = (sizeof(strata::DrawShared) + 15) / 16 * 16 + static_cast<size_t>(chunk) * esz;
  const bool sorted = static_cast<int64_t>(B) * ranks > 2 * sms && B <= strata::DRAW_SORT_MOST && (top_k != nullptr || top_p != nullptr);
  strata::DrawArgs A{logits, ld, V, chunk, B, sorted, u, temperature, top_p, min_p, top_k, out_ids, out_lps, errors};
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(DRAW_SMEM));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return host_fail(STRATA_ECUDA, "strata_draw_rows: %s", cudaGetErrorString(e));
  e = strata::launch_operator(device, stream, [&](bool overlaps) {
    const strata::Launch launch(static_cast<unsigned>(B) * ranks, strata::DRAW_THREADS, smem, stream, overlaps, static_cast<unsigned>(ranks));
    return f32 ? launch(strata::draw_kernel<float>, A) : launch(strata::draw_kernel<__nv_bfloat16>, A);
  });
  return e == cudaSuccess ? STRATA_OK : host_fail(STRATA_ECUDA, "strata_draw_rows: %s", cudaGetErrorString(e));
}
