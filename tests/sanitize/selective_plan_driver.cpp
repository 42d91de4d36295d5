// How a selective scan cuts packed sequences of unequal lengths (scan_grid of
// ssd_selective_plan.h), built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "ssd_selective_plan.h"

namespace {

int failures = 0;
#define CHECK(cond)                                                      \
  do {                                                                   \
    if (!(cond)) {                                                       \
      ++failures;                                                        \
      std::printf("%s:%d: failed: %s\n", __FILE__, __LINE__, #cond);     \
    }                                                                    \
  } while (0)

using Bounds = std::vector<int32_t>;

// The run that a workgroup finds at place `at`.
ssd::Run run_at(const ssd::RunGrid& g, int at) {
  if (g.cu == nullptr) return ssd::equal_run(g, at);
  if (!ssd::firsts_lead(g)) {
    int last = 0;
    for (int i = 1; i < g.nseq; ++i)
      if (ssd::first_slot(g, ssd::seq_bound(g, g.cu[i]), i) <= at) last = i;
    return ssd::packed_run(g, at, last, ssd::seq_bound(g, g.cu[last]),
                           ssd::seq_bound(g, g.cu[last + 1]));
  }
  int seq = at < g.nseq ? at : 0;
  if (at >= g.nseq)
    for (int i = 0; i < g.nseq; ++i)
      if (ssd::seq_bound(g, g.cu[i]) / g.run <= at - g.nseq) seq = i;
  const int begin = ssd::seq_bound(g, g.cu[seq]);
  return ssd::packed_run(g, ssd::slot_at(g, at, seq, begin), seq, begin,
                         ssd::seq_bound(g, g.cu[seq + 1]));
}

// Every token lies in one run of its own sequence, short sequences in one run and longer ones
// in as many as they need, inside the slots and marks that workspaces hold.
void check_runs(const ssd::ScanShape& s, bool back, const Bounds& cu, bool packed) {
  const ssd::RunGrid g = ssd::scan_grid(packed ? cu.data() : nullptr, s, back);
  const int64_t slots = ssd::run_slots(g);
  CHECK(g.run >= 1 && g.whole >= g.run && slots <= ssd::scan_most_slots(s, back));
  if (!back && (packed ? g.tokens > g.whole : g.per_seq > 1))
    CHECK(sizeof(float) * slots * s.dim * (s.n + 1) <= ssd::scan_fwd_bytes(s));
  std::vector<int> seen(g.tokens, 0), runs(g.nseq, 0);
  std::vector<ssd::Run> at_slot(slots);
  std::vector<int> there(slots, 0);
  for (int at = 0; at < slots; ++at) {
    const ssd::Run r = run_at(g, at);
    CHECK(r.slot >= 0 && r.slot < slots);
    at_slot[r.slot] = r;
    ++there[r.slot];
  }
  int64_t mark = 0;
  for (int slot = 0; slot < slots; ++slot) {
    CHECK(there[slot] == 1);           // the order has every slot, once
    const ssd::Run r = at_slot[slot];
    if (!r.on) continue;
    CHECK(r.seq >= 0 && r.seq < g.nseq && r.seq_begin == cu[r.seq] && r.seq_end == cu[r.seq + 1]);
    CHECK(r.first + r.index == slot && r.first >= 0 && r.first + r.count <= slots);
    CHECK(r.begin >= r.seq_begin && r.begin <= r.end && r.end <= r.seq_end);
    CHECK(r.end - r.begin <= (r.count == 1 ? g.whole : g.run));
    CHECK(r.index == runs[r.seq] && r.index < r.count);
    ++runs[r.seq];
    for (int t = r.begin; t < r.end; ++t) ++seen[t];
    if (back) {
      const int64_t first = ssd::first_mark(r, slot);
      CHECK(first >= mark && (r.begin - r.seq_begin) % ssd::kMark == 0);
      mark = first + (r.end - r.begin + ssd::kMark - 1) / ssd::kMark;
      CHECK(mark <= ssd::scan_marks(s));
    }
  }
  for (int t = 0; t < g.tokens; ++t) CHECK(seen[t] == (t >= cu.front() && t < cu.back()));
  for (int i = 0; i < g.nseq; ++i) {
    const int len = cu[i + 1] - cu[i];
    CHECK(runs[i] == (len > g.whole ? (len + g.run - 1) / g.run : 1));
    // a sequence that is cut is never walked without what joins its runs, or a few at most
    if (runs[i] > 1) CHECK(ssd::joins(g) || runs[i] <= ssd::kFoldRuns + 1);
  }
  if (!packed) return;
  // bounds that descend or lie outside give runs inside the tokens, slots and marks all the same
  std::mt19937 rng(g.tokens + g.nseq);
  Bounds wild(g.nseq + 1);
  for (auto& v : wild) v = (int32_t)(rng() >> 1) % (3 * g.tokens) - g.tokens;
  wild[rng() % wild.size()] = back ? INT32_MIN : INT32_MAX;
  for (int at = 0; at < slots; ++at)
    for (int seq = 0; seq < g.nseq; ++seq) {
      if (ssd::firsts_lead(g) && at < g.nseq && seq != at) continue;
      const int begin = ssd::seq_bound(g, wild[seq]);
      const int slot = ssd::firsts_lead(g) ? ssd::slot_at(g, at, seq, begin) : at;
      CHECK(slot >= 0 && slot < slots);
      const ssd::Run r =
          ssd::packed_run(g, slot, seq, begin, ssd::seq_bound(g, wild[seq + 1]));
      if (!r.on) continue;
      CHECK(r.begin >= 0 && r.begin <= r.end && r.end <= g.tokens && r.end - r.begin <= g.whole);
      CHECK(r.first >= 0 && r.first + r.count <= slots);
      if (back)
        CHECK(ssd::first_mark(r, slot) + (r.end - r.begin + 7) / 8 <= ssd::scan_marks(s));
    }
}

void partitions() {
  std::mt19937 rng(5);
  auto below = [&](int n) { return (int)(rng() % (unsigned)n); };
  for (int i = 0; i < 300; ++i) {
    const int nseq = 1 + below(i % 3 ? 100 : 6), tokens = 1 + below(i % 2 ? 6000 : 200);
    Bounds cu(nseq + 1);
    for (auto& v : cu) v = below(tokens + 1);
    if (i % 4 == 0)                     // one long sequence among tiny ones
      for (auto& v : cu) v = v < tokens / 2 ? v % (nseq + 1) : tokens - v % (nseq + 1);
    for (auto& v : cu) v = std::min(std::max(v, 0), tokens);
    std::sort(cu.begin(), cu.end());
    if (i % 5) cu.front() = 0, cu.back() = tokens;
    const int64_t dim = 64 * (1 + below(100));
    const int len = 1 + below(200);
    Bounds even(nseq + 1);
    for (int j = 0; j <= nseq; ++j) even[j] = j * len;
    for (bool back : {false, true}) {
      check_runs({tokens, nseq, dim, 16, 1, 0, 0, 0, 0, 0}, back, cu, true);
      check_runs({(int64_t)nseq * len, nseq, dim, 16, 1, 0, 0, 0, 0, 0}, back, even, false);
      check_runs({(int64_t)nseq * len, nseq, dim, 16, 1, 0, 0, 0, 0, 0}, back, even, true);
    }
  }
}

// One sequence that holds almost all tokens, beside others of one token or none, is cut the
// same however many the others are: into runs that spread over the chip.
void one_long_sequence() {
  for (bool back : {false, true})
    for (int64_t tokens : {1000, 3000, 16384, 32768, 65536})
      for (int64_t dim : {768, 1536, 2560, 5120, 8192}) {
        int64_t longest = 0;
        for (int nseq : {2, 12, 13, 25, 26, 52, 64, 200, 1000}) {
          const ssd::ScanShape s{tokens, nseq, dim, 16, 1, 0, 0, 0, 0, 0};
          Bounds cu(nseq + 1, 0);
          cu.back() = (int32_t)tokens - (nseq > 1000 ? 0 : nseq / 2);
          const ssd::RunGrid g = ssd::scan_grid(cu.data(), s, back);
          const int len = cu.back() - cu[nseq - 1];
          const int64_t run = len > g.whole ? g.run : len;
          if (nseq == 2) longest = run;
          if (run > 2 * longest)
            std::printf("%s %d tokens of %d channels: runs of %d beside %d others, of %d beside 1\n",
                        back ? "gradients" : "forward", (int)tokens, (int)dim, (int)run, nseq - 1,
                        (int)longest);
          CHECK(run <= 2 * longest);
        }
      }
}

// And no sequence that stays whole is a chain that outlasts the call's other work: it has no more
// tokens than a wave for every SIMD would, or than a few runs.
void whole_sequences() {
  for (bool back : {false, true})
    for (int64_t tokens : {1000, 16384, 65536, 1 << 20})
      for (int64_t dim : {768, 2560, 5120})
        for (int nseq : {1, 12, 13, 26, 64, 200, 1000, 4096}) {
          const ssd::ScanShape s{tokens, nseq, dim, 16, 1, 0, 0, 0, 0, 0};
          const int64_t whole = ssd::scan_whole(s, back), cut = ssd::scan_cut(s, back);
          CHECK(whole >= cut);
          CHECK(whole == cut || whole <= 128 + 8 ||
                whole * 1024 <= tokens * ssd::channel_blocks(s) + 8 * 1024);
        }
}

}  // namespace

int main() {
  partitions();
  one_long_sequence();
  whole_sequences();
  if (failures != 0) return 1;
  std::printf("all checks passed\n");
  return 0;
}
