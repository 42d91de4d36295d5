// ssd_selective_device.h -- device-side parts that the short convolution and
// the selective scan share (internal to libssd): where a workgroup's run of
// tokens lies in the packed sequences, and the activations.
#pragma once

#include "ssd_device.h"

namespace ssd {

// Every sequence is cut into runs of at most `run` tokens, counted by slots:
// sequence i owns the slots from cu[i] / run + i on.  Since
// ceil(len / run) <= floor(cu[i+1] / run) - floor(cu[i] / run) + 1, these never meet those
// of sequence i + 1, and tokens / run + nseq slots hold all sequences of any
// lengths: the host needs none of them to size a launch (up to nseq slots
// stay empty).  Without cu all lengths are equal and no slot is.
struct RunGrid {
  const int32_t* cu;
  int64_t tokens, nseq, run;
  int64_t per_seq;       // slots of a sequence (without cu)
};

inline RunGrid make_run_grid(const int32_t* cu, int64_t tokens, int64_t nseq, int64_t run) {
  const int64_t len = tokens / nseq;
  return RunGrid{cu, tokens, nseq, run, len > run ? (len + run - 1) / run : 1};
}
inline int64_t run_slots(const RunGrid& g) {
  return g.cu != nullptr ? g.tokens / g.run + g.nseq : g.nseq * g.per_seq;
}

struct Run {
  int64_t seq, seq_begin, seq_end;   // the sequence and its tokens
  int64_t begin, end;                // the run's tokens
  int64_t first;                     // the slot of the sequence's first run
  int64_t index, count;              // this run and how many the sequence has
  bool on;                           // whether the slot holds a run (an empty sequence has one)
};

__device__ __forceinline__ int64_t seq_bound(const RunGrid& g, int64_t i) {
  const int64_t v = g.cu[i];
  return v < 0 ? 0 : (v > g.tokens ? g.tokens : v);
}

// The run of `slot`: a 64-way search by the lanes of each wave.  Where cu
// descends the result is some run of some tokens in [0, tokens), or none.
__device__ __forceinline__ Run find_run(const RunGrid& g, int64_t slot) {
  Run r;
  if (g.cu == nullptr) {
    const int64_t len = g.tokens / g.nseq;
    r.seq = slot / g.per_seq;
    r.seq_begin = r.seq * len;
    r.seq_end = r.seq_begin + len;
    r.first = r.seq * g.per_seq;
  } else {
    int64_t lo = 0, hi = g.nseq;
    while (hi - lo > 1) {
      const int64_t step = (hi - lo + kWave - 1) / kWave;
      const int64_t p = lo + step * (threadIdx.x % kWave);
      const bool reached = p < hi && seq_bound(g, p) / g.run + p <= slot;
      int n = __popcll(__ballot(reached));
      n = __builtin_amdgcn_readfirstlane(n < 1 ? 1 : n);
      lo += step * (n - 1);
      if (lo > g.nseq - 1) lo = g.nseq - 1;
      hi = lo + step < hi ? lo + step : hi;
    }
    r.seq = lo;
    r.seq_begin = seq_bound(g, lo);
    r.seq_end = seq_bound(g, lo + 1);
    r.first = r.seq_begin / g.run + lo;
  }
  const int64_t len = r.seq_end > r.seq_begin ? r.seq_end - r.seq_begin : 0;
  r.seq_end = r.seq_begin + len;
  r.index = slot - r.first;
  r.count = len > g.run ? (len + g.run - 1) / g.run : 1;
  r.on = r.index >= 0 && r.index < r.count;
  r.begin = r.seq_begin + r.index * g.run;
  r.end = r.begin + g.run < r.seq_end ? r.begin + g.run : r.seq_end;
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
