// The sizes that strata_layer_norm_grad goes by, up to the largest call that it accepts.  Built so that an overflow of a signed number ends
// the program.  The library's host code is compiled into this program; nothing runs on a GPU.
#include <cstdarg>
#include <cstdio>

#include "../request_token_sampling_gb300/csrc/strata_layer_norm.cu"

namespace strata {
int host_fail(int code, const char*, ...) { return code; }
int tail_device(int*, uint32_t**, int*) { return STRATA_ECUDA; }
}  // namespace strata

int main() {
  long long bad = 0;
  const int Ts[] = {1, 7, 8, 9, 152, 153, 2431, 2432, 2433, 1 << 20, 2147483639, 2147483640, 2147483641, 2147483646, 2147483647};
  const int Hs[] = {1, 2, 511, 512, 513, 8192, 8193, STRATA_TAIL_MAX_WIDTH};
  for (int T : Ts)
    for (int H : Hs) {
      const int groups = grad_groups(T, H);
      // each group has a row, at least
      const long long rows = H > BLOCK_WIDTH || H > WARP_WIDTH ? 1 : strata::LAYER_NORM_GRAD_WARPS;
      const bool ok = groups >= 1 && (groups - 1LL) * rows < T && groups <= 4 * SMS && strata_layer_norm_workspace(T, H) == groups * 8LL * H;
      if (!ok && ++bad <= 5) std::printf("T %d H %d: %d groups\n", T, H, groups);
    }
  std::printf("%lld bad\n", bad);
  return bad != 0;
}
