// ssd_selective_device.h -- device-side parts that the short convolution and
// the selective scan share (internal to libssd): where a workgroup's run of
// tokens lies in the packed sequences, and the activations.
#pragma once

#include "ssd_device.h"
#include "ssd_selective_plan.h"

namespace ssd {

// The last sequence of which `reached(begin, sequence)` holds (0 if there is none), where it holds
// of all before one: a 64-way search by the lanes of each wave.
template <class Reached>
__device__ __forceinline__ int last_sequence(const RunGrid& g, Reached reached) {
  int lo = 0, hi = g.nseq;
  while (hi - lo > 1) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int64_t at = lo + (int64_t)step * (threadIdx.x % kWave);
    const int p = at < hi ? (int)at : hi - 1;
    int n = __popcll(__ballot(at < hi && reached(seq_bound(g, g.cu[p]), p)));
    n = __builtin_amdgcn_readfirstlane(n < 1 ? 1 : n);
    lo += step * (n - 1);
    if (lo > g.nseq - 1) lo = g.nseq - 1;
    hi = lo + step < hi ? lo + step : hi;
  }
  return lo;
}
// The run of `slot`.
__device__ __forceinline__ Run find_run(const RunGrid& g, int slot) {
  if (g.cu == nullptr) return equal_run(g, slot);
  const int seq = last_sequence(
      g, [&](int begin, int i) { return first_slot(g, begin, i) <= slot; });
  return packed_run(g, slot, seq, seq_bound(g, g.cu[seq]), seq_bound(g, g.cu[seq + 1]));
}
// The run that a scan's workgroups take at place `at`.
__device__ __forceinline__ Run find_ordered_run(const RunGrid& g, int at) {
  if (g.cu == nullptr || !firsts_lead(g)) return find_run(g, at);
  int seq = at;
  if (at >= g.nseq)
    seq = last_sequence(
        g, [&](int begin, int) { return (int)g.by_run.of((uint32_t)begin) <= at - g.nseq; });
  const int begin = seq_bound(g, g.cu[seq]);
  return packed_run(g, slot_at(g, at, seq, begin), seq, begin, seq_bound(g, g.cu[seq + 1]));
}

__device__ __forceinline__ float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }

// 1 / (1 + exp(-v)); exp(-v) may overflow, to a result of 0 that is below 2^-127.
__device__ __forceinline__ float sigmoid_f(float v) {
  return rcp_hw(1.0f + exp2_hw(-kLog2e * v));
}

// ln(1 + exp(v)) = max(v, 0) + ln(1 + e) with e = exp(-|v|), and ln(1 + e) = 2 artanh(s) with s =
// e / (2 + e) <= 1/3: good to a few roundings of the result and of the exponent, |v| 2^-24 of it,
// which count where v is far below zero (1 + e would lose all of e's digits there).  The
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
