// Host-side check of the rule by which sampling calls and the operators of strata_tail.h overlap on one stream
// (ChainState of strata_chain.h): random streams of calls go through it and an event model of programmatic
// dependent launch.  What a call reads after its wait, or is told to be complete before the call in front of it, has
// to be complete.  The same model has to find fault with the rules that leave one of the two conditions out.  The
// library's host code is compiled in; nothing runs on a GPU.  Exit status 1 on a violation.
#include "../request_token_sampling_gb300/csrc/strata_sample.cu"
#include <random>

enum Kind { OTHER, OPERATOR, TWO_KERNELS, SAMPLE, SAMPLE_PDL, SAMPLE_EARLY, SAMPLE_OWN, KINDS };

struct Calls {
  long long bad = 0, operators = 0, overlapped = 0;
  // `fence_operators`, `fence_sampling`: the two conditions.
  void run(std::mt19937& rng, bool fence_operators, bool fence_sampling) {
    strata::ChainState chain;
    bool pending = false;
    // Of the stream so far: when the newest kernel started, let the next one start, and ended; when all had ended.
    long long start = 0, trigger = 0, end = 0, all_end = 0;
    struct Done { Kind kind; long long end; } calls[16];
    const int n = 3 + static_cast<int>(rng() % 13);
    for (int i = 0; i < n; ++i) {
      const Kind kind = static_cast<Kind>(rng() % KINDS);
      auto work = [&] { return 1 + static_cast<long long>(rng() % (rng() % 8 == 0 ? 1000 : 30)); };
      // One kernel: overlapping or not; it waits for the one before it at once, at its end, or never; it lets the next one start at
      // its start, after that wait, or at its end.  Returns when it reads what it reads.
      enum Wait { FIRST, LAST, NEVER };
      enum Let { AT_START, AFTER_WAIT, AT_END };
      auto kernel = [&](bool overlaps, Wait wait, Let let) {
        const long long from = overlaps ? std::max(start, trigger) + static_cast<long long>(rng() % 5) : all_end;
        const long long before = overlaps ? end : all_end;
        const long long waited = wait == FIRST ? std::max(from, before) : from;
        long long until = waited + work();
        if (wait == LAST) until = std::max(until, before) + 1;
        start = from;
        trigger = let == AT_START ? from + 1 : let == AFTER_WAIT ? waited + 1 : until;
        end = until;
        all_end = std::max(all_end, until);
        return waited;
      };
      long long read = 0;
      int told = i;  // calls before this one are complete by `read`
      if (kind == OTHER) {
        read = kernel(false, FIRST, AT_END);
      } else if (kind == OPERATOR || kind == TWO_KERNELS) {
        const bool overlaps = !fence_operators || chain.operator_overlaps();
        read = kernel(overlaps, FIRST, AFTER_WAIT);
        if (kind == TWO_KERNELS) kernel(true, FIRST, AT_START);
        chain.operator_launched(overlaps);
        ++operators;
        overlapped += overlaps;
      } else {
        uint32_t flags = kind == SAMPLE ? 0u : STRATA_FLAG_PDL;
        if (kind == SAMPLE_EARLY || kind == SAMPLE_OWN) flags |= STRATA_FLAG_EARLY_LOAD;
        if (kind == SAMPLE_OWN) flags |= STRATA_FLAG_OWN_OUTPUTS;
        flags = launch_flags(flags, pending);
        const bool early = (flags & STRATA_FLAG_EARLY_LOAD) != 0u, own = early && (flags & STRATA_FLAG_OWN_OUTPUTS) != 0u;
        bool overlaps = (flags & STRATA_FLAG_PDL) != 0u;
        if (fence_sampling) overlaps = overlaps && chain.sampling_overlaps(early);
        read = kernel(overlaps, own ? NEVER : early ? LAST : FIRST, early ? AT_START : AFTER_WAIT);
        chain.sampling_launched(overlaps, early, own);
        pending = pending_after(pending, flags, true);
        if (early) told = i - 1;
      }
      // An operator may read what any call wrote.  A sampling call's logits come from anything but a sampling call.
      for (int j = 0; j < told; ++j)
        if (calls[j].end > read && (kind <= TWO_KERNELS || calls[j].kind <= TWO_KERNELS)) {
          ++bad;
          break;
        }
      calls[i] = {kind, end};
    }
  }
};

int main() {
  std::mt19937 rng(11);
  Calls rule, no_operators, no_sampling;
  for (int i = 0; i < 300000; ++i) {
    rule.run(rng, true, true);
    no_operators.run(rng, false, true);
    no_sampling.run(rng, true, false);
  }
  const bool seen = no_operators.bad > 1000 && no_sampling.bad > 1000;
  // most operators still overlap: one ordinary launch behind calls with own outputs is enough
  const bool kept = rule.overlapped * 10 > rule.operators * 7;
  std::printf("%lld bad; without the operators' condition %lld, without the sampling calls' %lld; %lld of %lld operators overlap\n",
              rule.bad, no_operators.bad, no_sampling.bad, rule.overlapped, rule.operators);
  return rule.bad == 0 && seen && kept ? 0 : 1;
}
