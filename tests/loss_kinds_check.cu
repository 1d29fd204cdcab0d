// Which kernels the sizes in tests/test_gpu_train_edges.py go through, so that they stay the kinds they are there for.  The library's
// host code is compiled into this program; nothing runs on a GPU.
#include <cstdarg>
#include <cstdio>

#include "../request_token_sampling_gb300/csrc/strata_loss.cu"

namespace strata {
int host_fail(int code, const char*, ...) { return code; }
int tail_device(int*, uint32_t**, int*) { return STRATA_ECUDA; }
}  // namespace strata

struct Kind {
  int T, V, H;
  bool pair;  // tiles of two SMs
  int runs;   // of a logit's sum: 1, 2 in a narrow tile (of a score up to 128 rows), or runs added up in registers
  bool taken_out;
};
int main() {
  int bad = 0;
  const Kind kinds[] = {{400, 90000, 1088, true, 2, true},   {500, 50000, 2056, true, 3, true},   {600, 40000, 1032, false, 2, true},
                        {100, 60000, 2056, false, 3, true},  {64, 90000, 576, false, 2, false},   {100, 90000, 1536, false, 2, false},
                        {90, 120000, 264, false, 1, false},  {2000, 40000, 520, true, 1, false}};
  for (const Kind& k : kinds)
    for (bool grad : {false, true}) {
      const Plan P(k.T, k.V, k.H, 0, grad);
      const int64_t tiles = tiles_of(k.T, P.tile_rows) * tiles_of(k.V, P.bn), runs = tiles_of(tiles_of(k.H, 64), P.run);
      if (P.pair == k.pair && runs == k.runs && P.is_long() == k.taken_out && tiles > (P.pair ? PAIRS : SMS) && (!grad || P.piece >= k.V)) continue;
      ++bad;
      std::printf("%d x %d x %d, grad %d: pair %d, %lld runs, %lld tiles, piece %d\n", k.T, k.V, k.H, grad, P.pair, static_cast<long long>(runs),
                  static_cast<long long>(tiles), P.piece);
    }
  std::printf("%d bad\n", bad);
  return bad != 0;
}
