// ssd_selective_scan.h -- what the selective scan's forward and backward
// kernels share (internal to libssd).
//
// A lane owns a channel and its N states; a wave owns 64 channels of one group,
// so B_t and C_t are the same for all its lanes and come through scalar loads
// into scalar registers, and rows of x, dt, z and y are read and written 64
// channels at a time.
#pragma once

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
  int softplus;
  // Of a split call, for each slot: the state that the run leaves [slots, N, dim]
  // (the slot of a sequence's last run, whose state nobody asks for, holds the initial
  // state instead, so that final_state may be init_state's buffer), and the sum of
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
  a.softplus = softplus;
  return a;
}

// The workgroup's 64 channels and its slot.
struct ScanPlace {
  int64_t slot, channel;
  int group, lanes;
  __device__ __forceinline__ explicit ScanPlace(const ScanArgs& a)
      : ScanPlace(a, blockIdx.x, a.group_blocks) {}
  __device__ __forceinline__ ScanPlace(const ScanArgs& a, int64_t item, int blocks) {
    const int64_t per_slot = a.ngroups * blocks;
    slot = item / per_slot;
    const int rest = (int)(item % per_slot);
    group = rest / blocks;
    const int at = rest % blocks * kWave;
    channel = (int64_t)group * a.group_dim + at;
    lanes = a.group_dim - at < kWave ? a.group_dim - at : kWave;
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

// N values of B or C of one token, the same for all lanes.
template <int N, bool BF16>
struct States {
  static constexpr int kWords = BF16 ? N / 2 : N;
  uint32_t w[kWords];
  // p: the first token's; `at`: bytes to the token's
  __device__ __forceinline__ States(const void* p, int64_t at) {
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(4)));
    typedef const __attribute__((address_space(4))) words* scalar;
    const scalar q = (scalar)(uintptr_t)((const char*)p + at);
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

// Tokens read at a time, one such block ahead of the arithmetic.
constexpr int kBlock = 4;

// The rows of a wave's inputs: uniform bases and a lane's place in them.
template <bool BF16>
struct Rows {
  const char *x, *dt, *z, *B, *C;
  int64_t x_step, dt_step, z_step, b_step, c_step;   // bytes between rows
  uint32_t lane;
  __device__ __forceinline__ Rows(const ScanArgs& a, const ScanPlace& pl, uint32_t lane_, int n) {
    constexpr int el = BF16 ? 2 : 4;
    x = (const char*)a.in.x + pl.channel * el;
    dt = (const char*)a.in.dt + pl.channel * el;
    z = (const char*)a.in.z + pl.channel * el;
    B = (const char*)a.in.B + (int64_t)pl.group * n * el;
    C = (const char*)a.in.C + (int64_t)pl.group * n * el;
    x_step = a.x_stride * el;
    dt_step = a.dt_stride * el;
    z_step = a.z_stride * el;
    b_step = a.b_stride * el;
    c_step = a.c_stride * el;
    lane = lane_;
  }
};

// The state at the start of a run: those that the runs before it leave, each decayed
// by the runs between, from the first on.
template <int N>
__device__ __forceinline__ void fold_runs(const ScanArgs& a, int64_t first, int64_t slot,
                                          int64_t d, const float (&A2)[N], float (&h)[N]) {
  for (int64_t s = first; s < slot; ++s) {
    const float total = a.totals[s * a.dim + d];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float left = a.states[(s * N + n) * a.dim + d];
      // (the first run's state includes the initial one)
      h[n] = s == first ? left : __builtin_fmaf(exp2_hw(total * A2[n]), h[n], left);
    }
  }
}

template <int N>
__device__ __forceinline__ void store_run(const ScanArgs& a, int64_t slot, int64_t d,
                                          const float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) a.states[(slot * N + n) * a.dim + d] = h[n];
}
template <int N>
__device__ __forceinline__ void load_run(const ScanArgs& a, int64_t slot, int64_t d,
                                         float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = a.states[(slot * N + n) * a.dim + d];
}

}  // namespace ssd
