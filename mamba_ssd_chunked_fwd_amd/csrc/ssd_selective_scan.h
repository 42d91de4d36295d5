// ssd_selective_scan.h -- what the selective scan's forward and backward
// kernels share (internal to libssd).
//
// A lane owns a channel and its N states; a wave owns 64 channels of one group,
// so B_t and C_t are the same for all its lanes and come through scalar loads
// into scalar registers, and rows of x, dt, z and y are read and written 64
// channels at a time.
#pragma once

#include <cfloat>

#include "ssd_selective_device.h"
#include "ssd_selective_launch.h"

namespace ssd {

struct ScanArgs {
  ScanInputs in;
  const float* init;
  void* y;
  float* fin;
  RunGrid runs;
  int64_t dim, ngroups;
  int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;
  int group_dim;       // channels of a group
  int group_blocks;    // blocks of 64 channels of a group
  Divide by_blocks, by_slot;   // by it, and by the blocks of all groups
  int softplus;
  int paired;          // whether two channels' elements are read and written at once
  int joined;          // whether scan_join_kernel has been through the states
  // Of a split call, for each slot: the state that the run leaves [slots, N, dim] (in the
  // forward call the slot of a sequence's last run, whose state nobody asks for, holds the
  // initial state instead, so that final_state may be init_state's buffer), and the sum of
  // its time steps [slots, dim].
  float *states, *totals;
};

inline ScanArgs make_scan_args(const ScanInputs& in, const float* init, const ScanShape& s,
                               bool softplus) {
  ScanArgs a{};
  a.in = in;
  a.init = init;
  a.dim = s.dim;
  a.ngroups = s.ngroups;
  a.x_stride = s.x_stride;
  a.dt_stride = s.dt_stride;
  a.z_stride = s.z_stride;
  a.b_stride = s.b_stride;
  a.c_stride = s.c_stride;
  a.group_dim = (int)(s.dim / s.ngroups);
  a.group_blocks = (a.group_dim + kWave - 1) / kWave;
  a.by_blocks = Divide(a.group_blocks);
  a.by_slot = Divide(a.group_blocks * s.ngroups);
  a.softplus = softplus;
  // every pair of a group's channels there, and on 4 bytes in every row
  const auto even = [](const void* p, int64_t stride) {
    return (uintptr_t)p % 4 == 0 && stride % 2 == 0;
  };
  a.paired = a.group_dim % 2 == 0 && even(in.x, s.x_stride) && even(in.dt, s.dt_stride) &&
             (in.z == nullptr || even(in.z, s.z_stride));
  return a;
}

// The workgroup's 64 channels and its place in the order of the slots.
struct ScanPlace {
  int at, group, lanes;
  int64_t channel;
  __device__ __forceinline__ explicit ScanPlace(const ScanArgs& a) {
    at = (int)a.by_slot.of(blockIdx.x);
    const uint32_t rest = blockIdx.x - (uint32_t)at * a.by_slot.d;
    group = (int)a.by_blocks.of(rest);
    const int first = (int)(rest - (uint32_t)group * a.by_blocks.d) * kWave;
    channel = (int64_t)group * a.group_dim + first;
    lanes = a.group_dim - first < kWave ? a.group_dim - first : kWave;
  }
};

template <int N>
__device__ __forceinline__ void load_states(const float* p, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const f32x4 q = *(const f32x4*)(p + 4 * k);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * k + e] = q[e];
  }
}
template <int N>
__device__ __forceinline__ void store_states(float* p, const float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k)
    *(f32x4*)(p + 4 * k) = (f32x4){v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
}

// A in powers of two: exp(delta A) = exp2(delta A2).  Kept finite where A is, so that no time (a
// token past a run's end has none) decays nothing.
__device__ __forceinline__ float in_powers_of_two(float A) {
  const float v = A * kLog2e;
  return v < -FLT_MAX ? -FLT_MAX : (v > FLT_MAX ? FLT_MAX : v);
}

// N values of B or C of one token, the same for all lanes.
template <int N, bool BF16>
struct States {
  static constexpr int kWords = BF16 ? N / 2 : N;
  uint32_t w[kWords];
  States() = default;
  __device__ __forceinline__ explicit States(const void* p) {
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(4)));
    typedef const __attribute__((address_space(4))) words* scalar;
    const scalar q = (scalar)(uintptr_t)p;
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) {
      const words v = q[k];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * k + e] = v[e];
    }
  }
  __device__ __forceinline__ float operator[](int n) const {
    if constexpr (BF16) return n & 1 ? bf16_hi(w[n / 2]) : bf16_lo(w[n / 2]);
    return __uint_as_float(w[n]);
  }
};

// B and C (or B alone) of the tokens of a run, one after the other, in pieces of 32 bytes,
// each piece read while the one before it is worked on: more would not leave enough scalar
// registers.
template <int NS, bool BF16, bool BOTH>
struct StateRows {
  static constexpr int kMost = BF16 ? 16 : 8;
  static constexpr int kPiece = NS < kMost ? NS : kMost, kPieces = NS / kPiece;
  static constexpr int kBytes = kPiece * (BF16 ? 2 : 4);
  typedef States<kPiece, BF16> S;
  const char *b, *c;
  int64_t b_step, c_step;
  int left;
  S nb, nc;
  __device__ __forceinline__ StateRows(const char* b_, const char* c_, int64_t bs, int64_t cs,
                                       int tokens)
      : b(b_), c(c_), b_step(bs), c_step(cs), left(tokens) {
    if (tokens > 0) read(0);
  }
  __device__ __forceinline__ void read(int k) {
    // (keeps the reads of many tokens from gathering and filling the scalar registers)
    asm volatile("" : "+s"(b));
    if (BOTH) asm volatile("" : "+s"(c));
    nb = S(b + k * kBytes);
    if (BOTH) nc = S(c + k * kBytes);
  }
  // Piece k of the present token; behind the last one comes the next token.
  __device__ __forceinline__ void next(int k, S& B, S& C) {
    B = nb;
    C = nc;
    if (k + 1 < kPieces) {
      read(k + 1);
    } else {
      if (--left > 0) {       // (the row behind the last one need not exist)
        b += b_step;
        c += c_step;
      }
      read(0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
};

// The rows of a wave's inputs from some token on: uniform pointers, which move from row to
// row (multiples of the steps would fill the scalar registers), and the lane's place.
template <bool BF16>
struct Rows {
  const char *x, *dt, *z, *B, *C;
  int64_t x_step, dt_step, z_step, b_step, c_step;   // bytes between rows
  uint32_t lane;
  // n: states of a group, from which the n0'th on are wanted
  __device__ __forceinline__ Rows(const ScanArgs& a, const ScanPlace& pl, int64_t t, int own,
                                  int n, int n0) {
    constexpr int el = BF16 ? 2 : 4;
    x_step = a.x_stride * el;
    dt_step = a.dt_stride * el;
    z_step = (a.in.z ? a.z_stride : a.x_stride) * el;
    b_step = a.b_stride * el;
    c_step = a.c_stride * el;
    x = (const char*)a.in.x + pl.channel * el + t * x_step;
    dt = (const char*)a.in.dt + pl.channel * el + t * dt_step;
    // (without a gate rows of x are read in the place of z's, and not used)
    z = (const char*)(a.in.z ? a.in.z : a.in.x) + pl.channel * el + t * z_step;
    B = (const char*)a.in.B + ((int64_t)pl.group * n + n0) * el + t * b_step;
    C = (const char*)a.in.C + ((int64_t)pl.group * n + n0) * el + t * c_step;
    lane = (uint32_t)own * el;
  }
};

// The element `lane` bytes into a row, as it lies in memory, and as a float.
template <bool BF16>
struct Raw {
  typedef uint16_t type;
  static __device__ __forceinline__ float get(type v) { return __uint_as_float((uint32_t)v << 16); }
};
template <>
struct Raw<false> {
  typedef float type;
  static __device__ __forceinline__ float get(type v) { return v; }
};
// A uniform row and a lane's place in it, as a buffer access: no 64-bit address for each
// lane is formed.
__device__ __forceinline__ rsrc_t row_rsrc(const void* row) { return make_rsrc(row, 0x7FFFFFFF); }
template <bool BF16>
__device__ __forceinline__ typename Raw<BF16>::type load_raw(const char* row, uint32_t lane) {
  if constexpr (BF16)
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row_rsrc(row), (int)lane, 0, 0);
  else
    return load_f32(row_rsrc(row), lane);
}
template <bool BF16>
__device__ __forceinline__ void store_raw(char* row, uint32_t lane, float v) {
  if constexpr (BF16)
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu), row_rsrc(row),
                                          (int)lane, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), row_rsrc(row), (int)lane, 0, 0);
}

// NS of the N states of a channel in a slot's record, from the n0'th on.
template <int N, int NS>
__device__ __forceinline__ void store_run(float* to, const ScanArgs& a, int64_t slot, int64_t d,
                                          int n0, const float (&h)[NS]) {
#pragma unroll
  for (int n = 0; n < NS; ++n) to[(slot * N + n0 + n) * a.dim + d] = h[n];
}
template <int N>
__device__ __forceinline__ void load_run(const ScanArgs& a, int64_t slot, int64_t d,
                                         float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = a.states[(slot * N + n) * a.dim + d];
}

// ---- the states at the runs' starts
// Few runs: each goes through those before it itself (no launch).  Many: a launch of their
// own (scan_join_kernel) replaces what the runs leave by what they start from.
// The first form, for some of a channel's states: `left(s, n)` is what run s leaves of
// state n (the first run's includes the initial state).
template <int N, class Left>
__device__ __forceinline__ void fold_runs(const ScanArgs& a, int64_t first, int64_t slot,
                                          int64_t d, const float (&A2)[N], float (&h)[N],
                                          Left left) {
  for (int64_t s = first; s < slot; ++s) {
    const float total = a.totals[s * a.dim + d];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float v = left(s, n);
      h[n] = s == first ? v : __builtin_fmaf(exp2_hw(total * A2[n]), h[n], v);
    }
  }
}

// The second form's launch (in ssd_selective_scan.hip).  With `back` it also replaces the
// gradients at the runs' starts by those at their ends.
void launch_scan_join(const ScanArgs& a, int64_t n, float* back, const float* dfinal,
                      hipStream_t st);

}  // namespace ssd
