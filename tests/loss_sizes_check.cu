// The sizes that the losses and their gradients go by, over the calls that they accept.  The library's host code is compiled into this
// program; nothing runs on a GPU.
#include <cstdarg>
#include <cstdio>

#include "../request_token_sampling_gb300/csrc/strata_loss.cu"

namespace strata {
int host_fail(int code, const char*, ...) { return code; }
int tail_device(int*, uint32_t**, int*) { return STRATA_ECUDA; }
}  // namespace strata

int main() {
  long long n = 0, bad = 0;
  const int Ts[] = {1, 5, 8, 64, 127, 128, 129, 300, 1024, 2049, 4096, 8192, 8193, 40000, 94312, 115585, 131071, 131072};
  const int Vs[] = {1, 255, 257, 1000, 32000, 70001, 151001, 248320, 262143, 524288};
  const int Hs[] = {8, 64, 128, 136, 512, 520, 1024, 1032, 2048, 2056, 4096, 8192, 32768};
  for (int T : Ts)
    for (int V : Vs)
      for (int H : Hs) {
        const Plan there(T, V, H, 0, false), back(T, V, H, 0, true);
        const int64_t d = static_cast<int64_t>(back.d_rows) * back.piece * 2;
        ++n;
        // a piece: whole tiles and steps of 64; up to 512 MB, or one round of tiles more where that holds all ids
        bool ok = back.piece % (2 * back.bn) == 0 && back.piece % 64 == 0 && back.bn <= 256;
        ok = ok && (back.piece < V ? d <= PIECE_BYTES : d <= PIECE_BYTES + back.d_rows * 511LL * 2 && back.piece - V < 512);
        // both ways add a logit up in the same runs, which their tiles have room for
        ok = ok && there.run == back.run && there.run >= 1;
        ok = ok && (there.is_long() ? there.run == strata::LOSS_LONG : there.bn > 128 || tiles_of(H, 64) <= 2 * there.run);
        ok = ok && there.bytes == strata_loss_workspace(T, V, H, 0, 0) && back.bytes == strata_loss_workspace(T, V, H, 0, 1);
        if (!ok && ++bad <= 5)
          std::printf("T %d V %d H %d: piece %d of tiles of %d, %lld bytes, runs %d and %d\n", T, V, H, back.piece, back.bn, static_cast<long long>(d), there.run, back.run);
      }
  std::printf("%lld plans, %lld bad\n", n, bad);
  return bad != 0;
}
