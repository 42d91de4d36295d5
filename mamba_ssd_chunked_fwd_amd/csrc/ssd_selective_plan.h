// ssd_selective_plan.h -- how the selective operators cut their work (internal to
// libssd; plain C++, so that the host layer's tests compile it without a GPU): runs of
// tokens, the slots that hold them, and the layouts of the scan's workspaces.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd_selective_launch.h"

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define SSD_BOTH __host__ __device__ __forceinline__
#else
#define SSD_BOTH inline
#endif

namespace ssd {

// Division of n < 2^31 by a number that the host knows (Granlund and Montgomery, "Division by
// invariant integers using multiplication"): with l = ceil(log2 d) and M = floor(2^32
// (2^l - d) / d) + 1, n / d = (n + floor(M n / 2^32)) >> l.  A wave's start would spend
// microseconds in divisions.
struct Divide {
  uint32_t d, m, shift;
  Divide() = default;
  explicit Divide(int64_t by) : d((uint32_t)by), m(0), shift(0) {
    while (((uint64_t)1 << shift) < d) ++shift;
    m = (uint32_t)((((((uint64_t)1 << shift) - d) << 32) / d) + 1);
  }
  SSD_BOTH uint32_t of(uint32_t n) const {
    return (uint32_t)(n + (uint32_t)(((uint64_t)m * n) >> 32)) >> shift;
  }
};

// Every sequence of more than `whole` tokens is cut into runs of at most `run`, counted by
// slots: sequence i owns the slots from cu[i] / run + i on.  Since
// ceil(len / run) <= floor(cu[i+1] / run) - floor(cu[i] / run) + 1, these never meet those
// of sequence i + 1, and tokens / run + nseq slots hold all sequences of any
// lengths: the host needs none of them to size a launch (up to nseq slots
// stay empty).  Without cu all lengths are equal and no slot is.  (Tokens, sequences and
// slots are fewer than 2^31.)
struct RunGrid {
  const int32_t* cu;
  int tokens, nseq, run, len;   // len: of a sequence, without cu
  int whole;                    // the longest sequence that is one run (`run` tokens or more)
  int per_seq;                  // slots of a sequence, without cu
  Divide by_run, by_per_seq;
};

inline RunGrid make_run_grid(const int32_t* cu, int64_t tokens, int64_t nseq, int64_t run,
                             int64_t whole = 0) {
  RunGrid g{};
  g.cu = cu;
  g.tokens = (int)tokens;
  g.nseq = (int)nseq;
  g.run = (int)run;
  g.len = (int)(tokens / nseq);
  g.whole = (int)(whole > run ? whole : run);
  g.per_seq = g.len > g.whole ? (g.len + g.run - 1) / g.run : 1;
  g.by_run = Divide(g.run);
  g.by_per_seq = Divide(g.per_seq);
  return g;
}
inline int64_t run_slots(const RunGrid& g) {
  return g.cu != nullptr ? (int64_t)(g.tokens / g.run) + g.nseq : (int64_t)g.nseq * g.per_seq;
}

struct Run {
  int seq, seq_begin, seq_end;   // the sequence and its tokens
  int begin, end;                // the run's tokens
  int slot, first;               // its slot, and that of the sequence's first run
  int index, count;              // this run and how many the sequence has
  bool on;                       // whether the slot holds a run (an empty sequence has one)
};

// An entry of cu, as the nearest token or end.
SSD_BOTH int seq_bound(const RunGrid& g, int v) { return v < 0 ? 0 : (v > g.tokens ? g.tokens : v); }
// The slot of the first run of a sequence that begins at `begin`.
SSD_BOTH int first_slot(const RunGrid& g, int begin, int seq) {
  return (int)g.by_run.of((uint32_t)begin) + seq;
}
SSD_BOTH int run_count(const RunGrid& g, int len) {
  return len > g.whole ? (int)g.by_run.of((uint32_t)(len - 1)) + 1 : 1;
}
SSD_BOTH Run place_run(const RunGrid& g, int slot, Run r) {
  const int len = r.seq_end > r.seq_begin ? r.seq_end - r.seq_begin : 0;
  r.seq_end = r.seq_begin + len;
  r.slot = slot;
  r.index = slot - r.first;
  r.count = run_count(g, len);
  r.on = r.index >= 0 && r.index < r.count;
  r.begin = r.on ? r.seq_begin + r.index * g.run : 0;
  r.end = r.on && r.index + 1 < r.count ? r.begin + g.run : r.seq_end;
  return r;
}
// The run of `slot` where the sequences are equally long, and where they are packed: `seq`, from
// `begin` to `end`, is the last sequence whose first slot is not behind `slot`.  Where cu
// descends that is some sequence, and the result some run of tokens in [0, tokens), or none.
SSD_BOTH Run equal_run(const RunGrid& g, int slot) {
  Run r;
  r.seq = (int)g.by_per_seq.of((uint32_t)slot);
  r.seq_begin = r.seq * g.len;
  r.seq_end = r.seq_begin + g.len;
  r.first = r.seq * g.per_seq;
  return place_run(g, slot, r);
}
SSD_BOTH Run packed_run(const RunGrid& g, int slot, int seq, int begin, int end) {
  Run r;
  r.seq = seq;
  r.seq_begin = begin;
  r.seq_end = end;
  r.first = first_slot(g, begin, seq);
  return place_run(g, slot, r);
}

// Where some sequences stay whole and others are cut, a scan's workgroups take the first slots of
// all sequences first, then the others: the whole ones are long workgroups among many whose slot
// holds no run, and in the slots' order gathered on some of the SIMDs (16 sequences of 2048 tokens
// of 5120 channels 1726 us, in this order 985).  Place `at` < nseq is the first slot of sequence
// `at`; place nseq + e is slot e + (the number of sequences that begin before the end of the
// tokens' e'th `run`), of which `seq` is the last (0 if there is none).
SSD_BOTH bool firsts_lead(const RunGrid& g) { return g.whole > g.run; }
SSD_BOTH int slot_at(const RunGrid& g, int at, int seq, int begin) {
  if (at < g.nseq) return first_slot(g, begin, seq);
  const int e = at - g.nseq;
  return e + seq + ((int)g.by_run.of((uint32_t)begin) <= e ? 1 : 0);
}

// ---- the scan
constexpr int kScanLanes = 64;     // channels of a wave
// Tokens whose states a wave of the gradients' second walk holds in registers at once; states
// are marked in memory at this distance by the first walk.
constexpr int kMark = 8;
constexpr int kBwdWaves = 4;       // waves of a workgroup of the second walk

inline int64_t channel_blocks(const ScanShape& s) {
  return s.ngroups * ((s.dim / s.ngroups + kScanLanes - 1) / kScanLanes);
}

// A channel block of a sequence is a chain that one wave walks, and fewer than 1024 chains leave
// SIMDs idle.  Runs that start from the states of those before them fill the chip, but cost a
// second walk over all but each sequence's last one (forward), or longer joins (backward, where
// two walks are made in any case).  The lengths of packed sequences are not known here: one of
// them may hold almost all tokens, and any number be empty.  So a sequence is cut or not by its
// own length.

// The tokens of a run of a sequence that is cut.
inline int64_t scan_cut(const ScanShape& s, bool backward) {
  const int64_t blocks = channel_blocks(s), unit = backward ? kMark : 4;
  const int64_t chains = s.nseq * blocks;
  // (8192 waves are what the chip holds at once.  The gradients' second walk takes a few rounds
  // of longer workgroups, into which the sequences' last, shorter runs have to fit: 648 us
  // without room for them, 622 with it; forward it makes no difference)
  const int64_t waves = backward ? (chains < 2048 ? 4096 - chains : 2048) : 8192;
  int64_t run = (s.tokens * blocks + waves - 1) / waves;
  // More rounds of shorter runs even out the shorter ones: gradients at 16384 x 5120 in 1 to 5
  // sequences 1427 to 1562 us with runs of 344, 1415 to 1440 with 144; 16384 x 2560 763 to 797
  // with 144 to 168.  Forward 32768 tokens in 3 sequences 978 with 320, 955 with 144, in one 976
  // and 965; one of 65536 x 2560 1013 and 977, of 16384 x 5120 506 with 160 and 520.
  if (run > 144) run = 144;
  // (very many sequences: gradients of 3000 x 2560 in 400, one of them of 2600 tokens, 343 us with
  // runs of 32, 362 with 64)
  const int64_t mean = (s.tokens + s.nseq - 1) / s.nseq;
  if (run > 4 * mean) run = 4 * mean;
  int64_t least = 24;
  if (!backward) {
    // Where there are waves for every SIMD in any case, a run's walk (0.36 us a token, twice)
    // is weighed against the join (0.07 us a run): their sum is least near the root of a tenth
    // of the tokens (643 tokens of 1536 channels: 28 us with runs of 12, 43 with runs of 32).
    least = 8;
    while (10 * least * least < s.tokens) least += unit;
  }
  if (run < least) run = least;
  return (run + unit - 1) / unit * unit;
}

// The longest sequence that is walked whole: one whose chain ends about when all tokens do, as
// equal sequences' do from 1280 chains on (gradients 2560).  Measured at 32768 tokens of 5120
// channels of 16 states in bf16, in 13, 16, 20, 26 and 52 equal sequences: whole 1209, 982, 802,
// 851 and 668 us, cut 960, 963, 957, 941 and 969; gradients in 26, 32, 52 and 64: whole 3650,
// 2984, 3092 and 2769, cut 2920, 2969, 3001 and 3003; at 16384 x 2560 in 52 and 64 956 and 775
// whole, 916 and 902 cut.  One sequence with 90% of the tokens beside 12 to 127 others is cut: 900
// to 980 us and 2800 to 2970.  (Runs of four times the mean length, whatever that is, took it up
// to 5880 and 6070.)
inline int64_t scan_whole(const ScanShape& s, bool backward) {
  const int64_t blocks = channel_blocks(s), unit = backward ? kMark : 4;
  const int64_t cut = scan_cut(s, backward), mean = (s.tokens + s.nseq - 1) / s.nseq;
  if (s.nseq * blocks < (backward ? 2560 : 1024)) return cut;
  int64_t run = s.tokens * blocks / (backward ? 2560 : 1280);
  // (few tokens: the join counts too.  3000 tokens of 2560 channels in 26 sequences 71 us whole,
  // 84 cut)
  const int64_t least = mean < 128 ? mean : 128;
  if (run > 4 * mean) run = 4 * mean;
  if (run < least) run = least;
  if (run < cut) run = cut;
  const int64_t most = INT32_MAX / unit * unit;
  run = (run + unit - 1) / unit * unit;
  return run > most ? most : run;
}

// The tokens of a run where all sequences are equally long: all of them whole, or cut.
inline int64_t scan_run(const ScanShape& s, bool backward) {
  const int64_t unit = backward ? kMark : 4, mean = (s.tokens + s.nseq - 1) / s.nseq;
  const int64_t cut = scan_cut(s, backward);
  if (mean > scan_whole(s, backward) || 4 * mean < cut) return cut;
  const int64_t most = INT32_MAX / unit * unit, run = (4 * mean + unit - 1) / unit * unit;
  return run > most ? most : run;
}
// Slots of such runs.
inline int64_t scan_slots(const ScanShape& s, bool backward) {
  return s.tokens / scan_run(s, backward) + s.nseq;
}
// The runs of a call.
inline RunGrid scan_grid(const int32_t* cu, const ScanShape& s, bool backward) {
  if (cu == nullptr) return make_run_grid(cu, s.tokens, s.nseq, scan_run(s, backward));
  return make_run_grid(cu, s.tokens, s.nseq, scan_cut(s, backward), scan_whole(s, backward));
}
// Slots that hold them, however the sequences are given.
inline int64_t scan_most_slots(const ScanShape& s, bool backward) {
  const int64_t equal = scan_slots(s, backward);
  const int64_t packed = s.tokens / scan_cut(s, backward) + s.nseq;
  return equal > packed ? equal : packed;
}
// Marks: each run's own from begin / kMark + slot on (as slots from cu).
inline int64_t scan_marks(const ScanShape& s) {
  return s.tokens / kMark + scan_most_slots(s, true) + 1;
}
SSD_BOTH int64_t first_mark(const Run& r, int64_t slot) { return r.begin / kMark + slot; }

// Blocks of a group's channels that the second walk's workgroups take: a lane has four
// states of two channels.
inline int64_t wide_blocks(const ScanShape& s) {
  const int64_t channels = kBwdWaves * (2 * kScanLanes * 4 / s.n);
  return (s.dim / s.ngroups + channels - 1) / channels;
}

// Few runs: each goes through those before it itself.  Many: a launch of their own joins them.
constexpr int kFoldRuns = 4;       // runs that a sequence may have for the first form
inline bool joins(const RunGrid& g) {
  return g.cu != nullptr ? g.tokens > g.whole && g.tokens / g.run > kFoldRuns
                         : g.per_seq > kFoldRuns;
}

// The forward call's workspace: states [slots, N, dim], then totals [slots, dim].
inline size_t scan_fwd_bytes(const ScanShape& s) {
  if (s.tokens <= scan_whole(s, false)) return 16;     // (nor are equal sequences cut)
  return sizeof(float) * (size_t)scan_most_slots(s, false) * (size_t)(s.dim * (s.n + 1));
}

// The gradients', in bytes from its start.
struct BwdLayout {
  size_t states, totals, back, marks, mark_totals, dA, bc, all;
};
inline BwdLayout bwd_layout(const ScanShape& s) {
  const size_t slots = (size_t)scan_most_slots(s, true), marks = (size_t)scan_marks(s);
  const size_t D = (size_t)s.dim, N = (size_t)s.n;
  size_t at = 0;
  const auto take = [&at](size_t floats) {
    const size_t p = at;
    at += (floats * sizeof(float) + 15) & ~(size_t)15;
    return p;
  };
  BwdLayout l;
  l.states = take(slots * N * D);
  l.totals = take(slots * D);
  l.back = take(slots * N * D);
  l.marks = take(marks * N * D);
  l.mark_totals = take(marks * D);
  l.dA = take(slots * (N + 2) * D);
  l.bc = take((size_t)wide_blocks(s) * (size_t)(s.tokens * s.ngroups) * 2 * N);
  l.all = at;
  return l;
}

// Whether the launches' grids hold a shape: a launch has fewer than 2^32 threads.
inline bool scan_grid_fits(const ScanShape& s, bool backward) {
  constexpr int64_t kBlocks = (int64_t)1 << 26;     // of 64 threads
  const int64_t slots = scan_most_slots(s, backward);
  if (slots >= kBlocks / channel_blocks(s)) return false;
  if (!backward) return true;
  // the second walk's workgroups have 256 threads, and so have the sums' over rows of B and C
  return slots < kBlocks / kBwdWaves / (s.ngroups * wide_blocks(s)) &&
         s.tokens <= (kBlocks / 4 - 1) * 256 / (2 * s.n * s.ngroups);
}
inline bool scan_step_grid_fits(const ScanShape& s) {
  return s.tokens < ((int64_t)1 << 32) / (s.dim * (s.n / 4) + 256);
}

// ---- the convolution
// Tokens of a run: enough runs to fill the chip, and no more than 64 tokens, from where on rows
// read twice no longer count.  The gradients' runs, which go past their ends and leave a row of
// partial sums each, are longer.  `units` of 512 channels are two waves each forward and four in
// the gradients (eight where rows do not start on whole vectors).  Measured in bf16, calls one
// behind the other: forward 16384 x 5376 80 us with runs of 44, 81 of 32, 83 of 64, 87 of 16; 8192
// x 2560 18.7 of 10, 17.5 of 16 to 32, 20.5 of 64.  Gradients 16384 x 5376 128 with 64, 129 of 32,
// 131 of 96, 152 of 16; 8192 x 2560 33 with 32, 38 of 16, 37 of 64; 2048 x 2560 21 with 8 to 32,
// 27 of 64.
inline int64_t conv_run(const ConvShape& s, bool backward) {
  const int64_t units = (s.dim + 511) / 512;
  int64_t run = s.tokens * units / (backward ? 1400 : 4096);
  if (backward) run = (run + 4) / 8 * 8;
  return run < 8 ? 8 : (run > 64 ? 64 : run);
}
inline int64_t conv_slots(const ConvShape& s, bool backward) {
  return s.tokens / conv_run(s, backward) + s.nseq;
}
// A launch has fewer than 2^32 threads: up to 256 more than channels for each slot.
inline bool conv_grid_fits(const ConvShape& s, bool backward, bool step) {
  const int64_t slots = step ? s.tokens : conv_slots(s, backward);
  return slots < ((int64_t)1 << 32) / (s.dim + 256);
}
inline size_t conv_bwd_bytes(const ConvShape& s) {
  return sizeof(float) * (size_t)conv_slots(s, true) * (size_t)((s.width + 1) * s.dim);
}

}  // namespace ssd
