// The recurrent form of the selective scan: one token for every sequence b, the state updated in
// place.  Per channel d and state n,
//   h = exp(delta A) h + delta x B,   y = (sum_n C h + D x) silu(z)
//
// MI355X design.  The state is read and written once (8 N bytes per channel) and little else: an
// HBM stream.  A lane holds a 16-byte unit, four states of one channel; the N/4 lanes of a
// channel lie side by side, form the channel's time step each for itself and meet in u by lane
// exchanges.  All of it is fp32.
//
// Measured: 200 sequences of 5120 channels of 16 states (131 MB of states, 139 in all) 25.4 us =
// 5.5 TB/s, where part of the state still lies in the last-level cache (a device copy moves
// 5.15); one sequence of 2560 channels 2.9 us, of which a launch is the most.
#include "ssd_host.h"
#include "ssd_selective_scan.h"

namespace ssd {
namespace {

// Four values of B or C (which start on 4 bytes).
template <bool BF16>
__device__ __forceinline__ f32x4 load_four(const void* p, int64_t i) {
  typedef u32x2 u32x2_4 __attribute__((aligned(4)));
  typedef f32x4 f32x4_4 __attribute__((aligned(4)));
  if constexpr (BF16) {
    const u32x2 u = *(const u32x2_4*)((const uint16_t*)p + i);
    return (f32x4){bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
  } else {
    return *(const f32x4_4*)((const float*)p + i);
  }
}

template <int N, bool BF16>
__global__ __launch_bounds__(256) void selective_step_kernel(const ScanArgs a, Divide by_blocks,
                                                             Divide by_group) {
  constexpr int L = N / 4;              // lanes of a channel
  const int64_t b = by_blocks.of(blockIdx.x);
  const int unit = (int)(blockIdx.x - (uint32_t)b * by_blocks.d) * 256 + (int)threadIdx.x;
  const bool on = unit < (int)a.dim * L;
  const int64_t d = on ? unit / L : a.dim - 1;
  const int n = unit % L * 4;
  const int64_t g = by_group.of((uint32_t)d);

  float* hp = a.fin + (b * a.dim + d) * N + n;
  f32x4 h = *(const f32x4*)hp;
  const f32x4 A = *(const f32x4*)(a.in.A + d * N + n);
  const f32x4 B = load_four<BF16>(a.in.B, b * a.b_stride + g * N + n);
  const f32x4 C = load_four<BF16>(a.in.C, b * a.c_stride + g * N + n);
  const float x = load_one<BF16>(a.in.x, b * a.x_stride + d);
  float delta = load_one<BF16>(a.in.dt, b * a.dt_stride + d);
  const float z = a.in.z ? load_one<BF16>(a.in.z, b * a.z_stride + d) : 0.0f;
  if (a.in.dt_bias) delta += a.in.dt_bias[d];
  if (a.softplus) delta = softplus_f(delta);
  const float dx = delta * x, step = delta * kLog2e;
  float u = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = __builtin_fmaf(exp2_hw(step * A[e]), h[e], dx * B[e]);
    u = __builtin_fmaf(C[e], h[e], u);
  }
#pragma unroll
  for (int off = 1; off < L; off <<= 1) u += __shfl_xor(u, off, kWave);
  if (!on) return;
  *(f32x4*)hp = h;
  if (n != 0) return;
  if (a.in.D) u = __builtin_fmaf(a.in.D[d], x, u);
  if (a.in.z) u *= z * sigmoid_f(z);
  store_one<BF16>(a.y, b * a.dim + d, u);
}

}  // namespace

int launch_scan_step(const ScanInputs& in, float* state, void* y, bool softplus, bool bf16,
                     const ScanShape& s, void* stream) {
  clear_launch_error();
  ScanArgs a = make_scan_args(in, nullptr, s, softplus);
  a.y = y;
  a.fin = state;
  const int blocks = (int)((s.dim * (s.n / 4) + 255) / 256);
  const dim3 grid((unsigned)(s.tokens * blocks));
  const Divide by_blocks(blocks), by_group(a.group_dim);
  hipStream_t st = (hipStream_t)stream;
#define SSD_STEP(N)                                                                              \
  case N:                                                                                        \
    if (bf16)                                                                                    \
      hipLaunchKernelGGL((selective_step_kernel<N, true>), grid, dim3(256), 0, st, a, by_blocks, \
                         by_group);                                                              \
    else                                                                                         \
      hipLaunchKernelGGL((selective_step_kernel<N, false>), grid, dim3(256), 0, st, a,           \
                         by_blocks, by_group);                                                   \
    break
  switch (s.n) {
    SSD_STEP(8);
    SSD_STEP(16);
    SSD_STEP(32);
    default:
      SSD_STEP(64);
  }
#undef SSD_STEP
  return (int)hipGetLastError();
}

}  // namespace ssd
