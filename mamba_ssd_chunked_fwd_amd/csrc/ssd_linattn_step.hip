// The recurrent form of linear attention with a decay for each head: one
// token for every (sequence b, head h), the state updated in place:
//   S = exp(log_decay_h) S + k v^T;   o = scale q^T S
// S is K x V, fp32; head h uses q and k of group h / (H/G).
//
// MI355X design.  The step reads and writes the state once (8 K V bytes per
// head) and little else, so it is HBM-bound: a coalesced stream over the
// state.  A workgroup of 256 threads owns V/CB columns of one (b, h), all K
// rows: a thread's 16-byte unit holds 4 columns of one row, the units of a row
// lie on consecutive threads, and the thread steps down the rows, so its
// columns, its four values of v and its part of o stay the same.  The
// columns are what is split for small batches (they are independent; rows meet
// in o): CB = 8, 4, 2 or 1, the smallest that gives every CU a workgroup.
//
// Measured on MI355X: 200 sequences of 32 heads of 128 x 64 (422 MB) 62 us under the
// profiler, where half the state still lies in the last-level cache, 80 us over
// rotating states (5.3 TB/s; a device copy moves 5.1); one sequence of 32 heads of
// 128 x 128 4 us, of which a launch is the most.
#include "ssd_block_launch.h"
#include "ssd_device.h"
#include "ssd_host.h"

#include <type_traits>

namespace ssd {
namespace {

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  else
    return ((const float*)p)[i];
}

template <int K, int V, int CB, bool BF16>
__global__ __launch_bounds__(256) void linattn_step_kernel(
    const void* __restrict__ q, const void* __restrict__ k, const void* __restrict__ v,
    const float* __restrict__ log_decay, float* __restrict__ state, void* __restrict__ o,
    float scale, int H, int G) {
  constexpr int UPR = V / 4 / CB;        // 16-byte units of a row
  constexpr int RP = 256 / UPR;          // rows at a time
  constexpr int IT = K / RP;             // rows of a thread
  constexpr int RW = kWave / UPR;        // rows of a wave at a time
  static_assert(UPR >= 1 && K % RP == 0 && UPR <= kWave, "unit split");
  __shared__ float qk[2][K];
  __shared__ f32x4 part[4][UPR];

  const int64_t bh = blockIdx.x / CB;
  const int cb = blockIdx.x % CB;
  const int64_t b = bh / H;
  const int h = (int)(bh % H), g = h / (H / G);
  const int tid = threadIdx.x, unit = tid % UPR, row = tid / UPR;
  const int col = (cb * UPR + unit) * 4;

  float* S = state + bh * K * V + col;
  f32x4 s[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) s[i] = *(const f32x4*)(S + (int64_t)(row + RP * i) * V);
  if (tid < K) qk[0][tid] = load1<BF16>(q, (b * G + g) * K + tid) * scale;
  else if (tid - K < K) qk[1][tid - K] = load1<BF16>(k, (b * G + g) * K + tid - K);
  f32x4 vv;
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = load1<BF16>(v, bh * V + col + e);
  const float lam = expf(log_decay[h]);
  __syncthreads();

  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const float qv = qk[0][row + RP * i], kv = qk[1][row + RP * i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = __builtin_fmaf(kv, vv[e], lam * s[i][e]);
      acc[e] = __builtin_fmaf(qv, s[i][e], acc[e]);
    }
    *(f32x4*)(S + (int64_t)(row + RP * i) * V) = s[i];
  }
  // Sum over the rows: within the wave, then over the four waves.
#pragma unroll
  for (int off = UPR; off < UPR * RW; off <<= 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], off, kWave);
  }
  if (tid % kWave < UPR) part[tid / kWave][unit] = acc;
  __syncthreads();
  if (tid < UPR) {
    acc = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    if constexpr (BF16) {
      *(u32x2*)((uint16_t*)o + bh * V + col) =
          (u32x2){pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3])};
    } else {
      *(f32x4*)((float*)o + bh * V + col) = acc;
    }
  }
}

template <int K, int V, bool BF16>
int launch_kv(const void* q, const void* k, const void* v, const float* ld, float* state, void* o,
              float scale, const LinattnShape& s, hipStream_t st) {
  const int64_t heads = s.tokens * s.nheads;
  const int H = (int)s.nheads, G = (int)s.ngroups;
#define SSD_STEP(CB)                                                                             \
  hipLaunchKernelGGL((linattn_step_kernel<K, V, CB, BF16>), dim3((unsigned)(heads * CB)),        \
                     dim3(256), 0, st, q, k, v, ld, state, o, scale, H, G)
  if (heads >= 256)
    SSD_STEP(1);
  else if (heads >= 128)
    SSD_STEP(2);
  else if (heads >= 64)
    SSD_STEP(4);
  else
    SSD_STEP((K * V / 1024 < 8 ? K * V / 1024 : 8));   // a unit per thread at least
#undef SSD_STEP
  return (int)hipGetLastError();
}

}  // namespace

int launch_linattn_step(const void* q, const void* k, const void* v, const float* log_decay,
                        float* state, void* o, float scale, bool bf16, const LinattnShape& s,
                        void* stream) {
  clear_launch_error();
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto kk, auto vv) {
    constexpr int K = decltype(kk)::value, V = decltype(vv)::value;
    return bf16 ? launch_kv<K, V, true>(q, k, v, log_decay, state, o, scale, s, st)
                : launch_kv<K, V, false>(q, k, v, log_decay, state, o, scale, s, st);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  if (s.dk == 64) return s.dv == 64 ? go(I64{}, I64{}) : go(I64{}, I128{});
  return s.dv == 64 ? go(I128{}, I64{}) : go(I128{}, I128{});
}

}  // namespace ssd
