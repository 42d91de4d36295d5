// ssd_selective_device.h -- device-side parts that the short convolution and
// the selective scan share (internal to libssd): where a workgroup's run of
// tokens lies in the packed sequences, and the activations.
#pragma once

#include "ssd_device.h"

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
  __device__ __forceinline__ uint32_t of(uint32_t n) const {
    return (uint32_t)(n + (uint32_t)(((uint64_t)m * n) >> 32)) >> shift;
  }
};

// Every sequence is cut into runs of at most `run` tokens, counted by slots:
// sequence i owns the slots from cu[i] / run + i on.  Since
// ceil(len / run) <= floor(cu[i+1] / run) - floor(cu[i] / run) + 1, these never meet those
// of sequence i + 1, and tokens / run + nseq slots hold all sequences of any
// lengths: the host needs none of them to size a launch (up to nseq slots
// stay empty).  Without cu all lengths are equal and no slot is.  (Tokens, sequences and
// slots are fewer than 2^31.)
struct RunGrid {
  const int32_t* cu;
  int tokens, nseq, run, len;   // len: of a sequence, without cu
  int per_seq;                  // slots of a sequence, without cu
  Divide by_run, by_per_seq;
};

inline RunGrid make_run_grid(const int32_t* cu, int64_t tokens, int64_t nseq, int64_t run) {
  RunGrid g{};
  g.cu = cu;
  g.tokens = (int)tokens;
  g.nseq = (int)nseq;
  g.run = (int)run;
  g.len = (int)(tokens / nseq);
  g.per_seq = g.len > g.run ? (g.len + g.run - 1) / g.run : 1;
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
  int first;                     // the slot of the sequence's first run
  int index, count;              // this run and how many the sequence has
  bool on;                       // whether the slot holds a run (an empty sequence has one)
};

__device__ __forceinline__ int seq_bound(const RunGrid& g, int i) {
  const int v = g.cu[i];
  return v < 0 ? 0 : (v > g.tokens ? g.tokens : v);
}

// The run of `slot`: a 64-way search by the lanes of each wave.  Where cu
// descends the result is some run of some tokens in [0, tokens), or none.
__device__ __forceinline__ Run find_run(const RunGrid& g, int slot) {
  Run r;
  if (g.cu == nullptr) {
    r.seq = (int)g.by_per_seq.of(slot);
    r.seq_begin = r.seq * g.len;
    r.seq_end = r.seq_begin + g.len;
    r.first = r.seq * g.per_seq;
  } else {
    int lo = 0, hi = g.nseq;
    while (hi - lo > 1) {
      const int step = (hi - lo + kWave - 1) / kWave;
      const int64_t at = lo + (int64_t)step * (threadIdx.x % kWave);
      const int p = at < hi ? (int)at : hi - 1;
      const bool reached = at < hi && (int)g.by_run.of(seq_bound(g, p)) + p <= slot;
      int n = __popcll(__ballot(reached));
      n = __builtin_amdgcn_readfirstlane(n < 1 ? 1 : n);
      lo += step * (n - 1);
      if (lo > g.nseq - 1) lo = g.nseq - 1;
      hi = lo + step < hi ? lo + step : hi;
    }
    r.seq = lo;
    r.seq_begin = seq_bound(g, lo);
    r.seq_end = seq_bound(g, lo + 1);
    r.first = (int)g.by_run.of(r.seq_begin) + lo;
  }
  const int len = r.seq_end > r.seq_begin ? r.seq_end - r.seq_begin : 0;
  r.seq_end = r.seq_begin + len;
  r.index = slot - r.first;
  r.count = len > g.run ? (int)g.by_run.of(len - 1) + 1 : 1;
  r.on = r.index >= 0 && r.index < r.count;
  r.begin = r.on ? r.seq_begin + r.index * g.run : 0;
  r.end = r.on && r.seq_end - r.begin > g.run ? r.begin + g.run : r.seq_end;
  return r;
}

__device__ __forceinline__ float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }

// 1 / (1 + exp(-v)); exp(-v) may overflow, to a result of 0 that is below 2^-127.
__device__ __forceinline__ float sigmoid_f(float v) {
  return rcp_hw(1.0f + exp2_hw(-kLog2e * v));
}

// ln(1 + exp(v)) = max(v, 0) + ln(1 + e) with e = exp(-|v|), and
// ln(1 + e) = 2 artanh(s) with s = e / (2 + e) <= 1/3: good to a few roundings of the
// result for every v, also where it is small (1 + e would lose e's digits).  The
// polynomial is artanh(s) / s in s^2, fitted to 4e-9 of it by weighted least squares.
__device__ __forceinline__ float softplus_f(float v) {
  const float e = exp2_hw(-kLog2e * __builtin_fabsf(v));
  const float s = e * rcp_hw(2.0f + e), q = s * s;
  float p = 0.14089166f;
  p = __builtin_fmaf(p, q, 0.13980302f);
  p = __builtin_fmaf(p, q, 0.20012455f);
  p = __builtin_fmaf(p, q, 0.33333157f);
  p = __builtin_fmaf(p, q, 1.0f);
  // (a NaN comes through e)
  return __builtin_fmaf(s + s, p, __builtin_fmaxf(v, 0.0f));
}

// `yes` where `on`, formed in any case: a branch for every token would cut the walks into
// blocks, across which the compiler moves work to where it fills the registers.
__device__ __forceinline__ float pick(bool on, float yes, float no) {
  asm volatile("" : "+v"(yes));
  return on ? yes : no;
}

// One element of an array of fp32 or bf16, and back (rounded once).
template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  else
    return ((const float*)p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (BF16)
    ((uint16_t*)p)[i] = (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu);
  else
    ((float*)p)[i] = v;
}

}  // namespace ssd
