// Gradients of the selective scan (ssd_selective_scan.hip).
#include "ssd_selective_scan.h"

#include "ssd_host.h"

namespace ssd {
namespace {

// Tokens whose states a wave holds in registers at once; states are marked in memory
// at this distance by the first walk.
constexpr int kMark = 8;
constexpr int kWaves = 4;
constexpr float kLn2 = 0.6931471805599453f;

struct BwdArgs {
  ScanArgs f;            // (states and totals: those that the runs leave)
  const void* dy;
  const float* dfinal;
  ScanGradients out;
  float* back;           // [slots, N, dim]: the gradient at a run's start, from zeros at its end
  float* marks;          // [marks, N, dim]: states inside the runs, from zeros at their start
  float* mark_totals;    // [marks, dim]: the time steps' sums from the runs' starts to there
  float* dA_part;        // [slots, N + 2, dim]: of dA, dD and ddt_bias
  float* bc_part;        // [blocks of a group, tokens, groups, 2, N]: of dB and dC
  int64_t slots;
};

__device__ __forceinline__ int64_t first_mark(const Run& r, int64_t slot) {
  return r.begin / kMark + slot;
}

// The first walk, up the tokens: of each run the state that it leaves, the states inside
// it, and the gradient that its outputs give the state at its start,
//   sum_t (prod_{s<=t} exp(delta_s A)) C_t du_t
template <int N, bool BF16>
__global__ __launch_bounds__(kWave) void scan_local_kernel(const BwdArgs b) {
  const ScanArgs& a = b.f;
  const ScanPlace pl(a);
  const Run r = find_run(a.runs, pl.slot);
  if (!r.on) return;
  const int lane = threadIdx.x;
  const bool mine = lane < pl.lanes;
  const int own = mine ? lane : pl.lanes - 1;
  const int64_t d = pl.channel + own;

  float A2[N], h[N], decay[N], back[N];
  load_states<N>(a.in.A + d * N, A2);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A2[n] *= kLog2e;
    h[n] = 0.0f;
    decay[n] = 1.0f;
    back[n] = 0.0f;
  }
  if (r.index == 0 && a.init != nullptr) load_states<N>(a.init + (r.seq * a.dim + d) * N, h);
  const float bias = a.in.dt_bias ? a.in.dt_bias[d] : 0.0f;
  const Rows<BF16> rows(a, pl, own, N);
  const char* dy = (const char*)b.dy + pl.channel * (BF16 ? 2 : 4);
  const int64_t dy_step = a.dim * (BF16 ? 2 : 4);
  int64_t mark = first_mark(r, pl.slot);
  double total = 0.0;
  for (int64_t t0 = r.begin; t0 < r.end; t0 += kMark, ++mark) {
    if (t0 > r.begin && mine) {
#pragma unroll
      for (int n = 0; n < N; ++n) b.marks[(mark * N + n) * a.dim + d] = h[n];
      b.mark_totals[mark * a.dim + d] = (float)total;
    }
    float x[kMark], dt[kMark], g[kMark];
#pragma unroll
    for (int j = 0; j < kMark; ++j) {
      const int64_t t = t0 + j < r.end ? t0 + j : r.end - 1;
      x[j] = load_one<BF16>(rows.x + t * rows.x_step, own);
      dt[j] = load_one<BF16>(rows.dt + t * rows.dt_step, own);
      g[j] = load_one<BF16>(dy + t * dy_step, own);
      if (a.in.z != nullptr) {
        const float z = load_one<BF16>(rows.z + t * rows.z_step, own);
        g[j] *= z * sigmoid_f(z);
      }
    }
#pragma unroll
    for (int j = 0; j < kMark; ++j) {
      if (t0 + j >= r.end) break;
      const States<N, BF16> B(rows.B, (t0 + j) * rows.b_step);
      const States<N, BF16> C(rows.C, (t0 + j) * rows.c_step);
      const float v = dt[j] + bias;
      const float delta = a.softplus ? softplus_f(v) : v;
      const float dx = delta * x[j];
      total += delta;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float e = exp2_hw(delta * A2[n]);
        h[n] = __builtin_fmaf(e, h[n], dx * B[n]);
        decay[n] *= e;
        back[n] = __builtin_fmaf(decay[n], C[n] * g[j], back[n]);
      }
    }
  }
  if (!mine) return;
  store_run<N>(a, pl.slot, d, h);
  a.totals[pl.slot * a.dim + d] = (float)total;
#pragma unroll
  for (int n = 0; n < N; ++n) b.back[(pl.slot * N + n) * a.dim + d] = back[n];
}

// ---- sums over a wave's lanes, several values at once
// Two values' sums over pairs of lanes that differ in one bit of their number: the
// lanes without that bit hold a's, those with it b's.
__device__ __forceinline__ float merge32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float merge16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
constexpr int kRowRor8 = 0x128, kHalfMirror = 0x141, kQuadXor2 = 0x4E, kQuadXor1 = 0xB1;
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ float merge_dpp(float a, float b, bool upper) {
  return (upper ? b : a) + moved<CTRL>(upper ? a : b);
}

// Sums of M (8 or 16) values, taken in one by one: in the end `sum` holds, in the lanes whose
// bits 5, 4, 3 (and 2) are n's bits 0, 1, 2 (and 3), value n's sum over the lanes that
// differ in those bits.
template <int M>
struct LaneSums {
  float l0, l1, l2, l3, sum;
  __device__ __forceinline__ void add(int n, float v) {
    const int lane = threadIdx.x;
    if ((n & 1) == 0) {
      l0 = v;
      return;
    }
    v = merge32(l0, v);
    if ((n & 2) == 0) {
      l1 = v;
      return;
    }
    v = merge16(l1, v);
    if ((n & 4) == 0) {
      l2 = v;
      return;
    }
    v = merge_dpp<kRowRor8>(l2, v, lane & 8);
    if (M == 8) {
      sum = v;
      return;
    }
    if ((n & 8) == 0) {
      l3 = v;
      return;
    }
    sum = merge_dpp<kHalfMirror>(l3, v, lane & 4);
  }
};

// The sums over all lanes of dB's and dC's M values, from what LaneSums has of each: a
// lane holds that of value value_of(lane).
template <int M>
__device__ __forceinline__ float lane_total(float dB, float dC) {
  const int lane = threadIdx.x;
  if constexpr (M == 16) {
    const float v = merge_dpp<kQuadXor2>(dB, dC, lane & 2);
    return v + moved<kQuadXor1>(v);
  } else {
    float v = merge_dpp<kHalfMirror>(dB, dC, lane & 4);
    v += moved<kQuadXor2>(v);
    return v + moved<kQuadXor1>(v);
  }
}
// Which of the 2 M values (dB's first) a lane holds.
template <int M>
__device__ __forceinline__ int value_of(int lane) {
  const int n = (lane >> 5 & 1) | (lane >> 4 & 1) << 1 | (lane >> 3 & 1) << 2;
  return M == 16 ? n | (lane >> 2 & 1) << 3 | (lane >> 1 & 1) << 4 : n | (lane >> 2 & 1) << 3;
}

// The second walk, down the tokens.  A wave holds NS of the N states of 64 channels;
// SL = N / NS waves share the channels, and the waves of a workgroup add up
// what dB and dC get from their channels.
template <int NS, int SL, bool BF16>
__global__ __launch_bounds__(kWave * kWaves) void scan_bwd_kernel(const BwdArgs b) {
  constexpr int N = NS * SL;
  constexpr int kMaxChannels = kWaves / SL;     // channel blocks of a workgroup
  __shared__ float bc[2][kMaxChannels][SL][kMark][2 * NS];
  // of several slices: their parts of x's and the time step's gradients, and of u
  __shared__ float parts[SL > 1 ? kMaxChannels : 1][SL > 1 ? SL : 1][SL > 1 ? kMark : 1][3]
                        [SL > 1 ? kWave : 1];
  __shared__ float start[kWaves][NS][kWave];

  const ScanArgs& a = b.f;
  const int waves = (int)blockDim.x / kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int slice = wave % SL, cw = wave / SL, nchan = waves / SL;
  const int lane = threadIdx.x % kWave;
  // the workgroup's block of nchan * 64 channels, and the wave's 64 of them
  const int wide = (a.group_dim + nchan * kWave - 1) / (nchan * kWave);
  const int64_t per_slot = a.ngroups * wide;
  const int64_t slot = blockIdx.x / per_slot;
  const int rest = (int)(blockIdx.x % per_slot);
  const int group = rest / wide, block = rest % wide;
  const int at = (block * nchan + cw) * kWave;
  const int lanes = a.group_dim - at < kWave ? a.group_dim - at : kWave;   // may be <= 0
  const bool mine = lane < lanes;
  const int own = mine ? lane : (lanes > 0 ? lanes - 1 : 0);
  ScanPlace pl(a, 0, 1);
  pl.slot = slot;
  pl.group = group;
  pl.channel = (int64_t)group * a.group_dim + (lanes > 0 ? at : 0);
  pl.lanes = lanes;
  const int64_t d = pl.channel + own;
  const int n0 = slice * NS;

  float* dA_row = b.dA_part + slot * (N + 2) * a.dim + d;
  const Run r = find_run(a.runs, slot);
  if (!r.on || r.begin >= r.end) {
    if (mine) {
#pragma unroll
      for (int n = 0; n < NS; ++n) dA_row[(n0 + n) * a.dim] = 0.0f;
      if (slice == 0) dA_row[N * a.dim] = dA_row[(N + 1) * a.dim] = 0.0f;
      // an empty sequence passes its final state's gradient on
      if (r.on && b.out.dinit != nullptr) {
        float v[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) v[n] = 0.0f;
        if (b.dfinal) load_states<NS>(b.dfinal + (r.seq * a.dim + d) * N + n0, v);
        store_states<NS>(b.out.dinit + (r.seq * a.dim + d) * N + n0, v);
      }
    }
    return;
  }

  float A2[NS], R[NS], dA[NS];
  load_states<NS>(a.in.A + d * N + n0, A2);
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    A2[n] *= kLog2e;
    R[n] = 0.0f;
    dA[n] = 0.0f;
  }
  // the state at the run's start
  {
    float h[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = 0.0f;
    if (r.index == 0) {
      if (a.init != nullptr) load_states<NS>(a.init + (r.seq * a.dim + d) * N + n0, h);
    } else {
      for (int64_t s = r.first; s < slot; ++s) {
        const float total = a.totals[s * a.dim + d];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float left = a.states[(s * N + n0 + n) * a.dim + d];
          h[n] = s == r.first ? left : __builtin_fmaf(exp2_hw(total * A2[n]), h[n], left);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) start[wave][n][lane] = h[n];
  }
  // the gradient of the state at its end
  if (b.dfinal != nullptr) load_states<NS>(b.dfinal + (r.seq * a.dim + d) * N + n0, R);
  for (int64_t s = r.first + r.count - 1; s > slot; --s) {
    const float total = a.totals[s * a.dim + d];
#pragma unroll
    for (int n = 0; n < NS; ++n)
      R[n] = __builtin_fmaf(exp2_hw(total * A2[n]), R[n],
                            b.back[(s * N + n0 + n) * a.dim + d]);
  }

  const float bias = a.in.dt_bias ? a.in.dt_bias[d] : 0.0f;
  const float skip = a.in.D ? a.in.D[d] : 0.0f;
  const bool gated = a.in.z != nullptr;
  const Rows<BF16> rows(a, pl, own, N);
  constexpr int el = BF16 ? 2 : 4;
  const int64_t out_step = a.dim * el;
  const char* dy = (const char*)b.dy + pl.channel * el;
  char* dx_out = (char*)b.out.dx + pl.channel * el;
  char* ddt_out = (char*)b.out.ddt + pl.channel * el;
  char* dz_out = gated ? (char*)b.out.dz + pl.channel * el : nullptr;
  float dD = 0.0f, dbias = 0.0f;
  int turn = 0;

  const int64_t blocks = (r.end - r.begin + kMark - 1) / kMark;
  const int64_t mark0 = first_mark(r, slot);
  for (int64_t m = blocks - 1; m >= 0; --m, turn ^= 1) {
    const int64_t t0 = r.begin + m * kMark;
    const int count = r.end - t0 < kMark ? (int)(r.end - t0) : kMark;
    float x[kMark], raw[kMark], z[kMark], g[kMark], delta[kMark];
#pragma unroll
    for (int j = 0; j < kMark; ++j) {
      const int64_t t = t0 + (j < count ? j : count - 1);
      x[j] = load_one<BF16>(rows.x + t * rows.x_step, own);
      raw[j] = load_one<BF16>(rows.dt + t * rows.dt_step, own);
      g[j] = load_one<BF16>(dy + t * out_step, own);
      z[j] = gated ? load_one<BF16>(rows.z + t * rows.z_step, own) : 0.0f;
    }
    float h[kMark + 1][NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) h[0][n] = start[wave][n][lane];
    if (m > 0) {
      // the first run's marks include the initial state
      const float total = b.mark_totals[(mark0 + m) * a.dim + d];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const float part = b.marks[((mark0 + m) * N + n0 + n) * a.dim + d];
        h[0][n] = r.index == 0 ? part : __builtin_fmaf(exp2_hw(total * A2[n]), h[0][n], part);
      }
    }
    float u[kMark], du[kMark];
#pragma unroll
    for (int j = 0; j < kMark; ++j) {
      u[j] = 0.0f;
      if (j >= count) break;
      const States<NS, BF16> B(rows.B, (t0 + j) * rows.b_step + n0 * el);
      const float v = raw[j] + bias;
      delta[j] = a.softplus ? softplus_f(v) : v;
      const float dx = delta[j] * x[j];
#pragma unroll
      for (int n = 0; n < NS; ++n)
        h[j + 1][n] = __builtin_fmaf(exp2_hw(delta[j] * A2[n]), h[j][n], dx * B[n]);
      du[j] = g[j];
      if (gated) {
        const States<NS, BF16> C(rows.C, (t0 + j) * rows.c_step + n0 * el);
#pragma unroll
        for (int n = 0; n < NS; ++n) u[j] = __builtin_fmaf(C[n], h[j + 1][n], u[j]);
        du[j] = g[j] * z[j] * sigmoid_f(z[j]);
      }
    }
    float inner[kMark], ddelta[kMark];
#pragma unroll
    for (int j = kMark - 1; j >= 0; --j) {
      if (j < count) {
        const States<NS, BF16> B(rows.B, (t0 + j) * rows.b_step + n0 * el);
        const States<NS, BF16> C(rows.C, (t0 + j) * rows.c_step + n0 * el);
        const float dx = mine ? delta[j] * x[j] : 0.0f;
        const float gj = mine ? du[j] : 0.0f;
        LaneSums<NS> sB, sC;
        inner[j] = ddelta[j] = 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float dh = __builtin_fmaf(C[n], du[j], R[n]);
          sC.add(n, gj * h[j + 1][n]);
          sB.add(n, dx * dh);
          inner[j] = __builtin_fmaf(B[n], dh, inner[j]);
          R[n] = dh * exp2_hw(delta[j] * A2[n]);
          const float kept = R[n] * h[j][n];
          ddelta[j] = __builtin_fmaf(kept, A2[n], ddelta[j]);
          dA[n] = __builtin_fmaf(kept, delta[j], dA[n]);
        }
        const float v = lane_total<NS>(sB.sum, sC.sum);
        bc[turn][cw][slice][j][value_of<NS>(lane)] = v;
      }
    }
    if constexpr (SL > 1) {
#pragma unroll
      for (int j = 0; j < kMark; ++j) {
        if (j < count) {
          parts[cw][slice][j][0][lane] = inner[j];
          parts[cw][slice][j][1][lane] = ddelta[j];
          parts[cw][slice][j][2][lane] = u[j];
        }
      }
    }
    __syncthreads();
    // dB and dC of this block of channels
    for (int i = threadIdx.x; i < count * SL * 2 * NS; i += (int)blockDim.x) {
      const int v = i % (2 * NS), s = i / (2 * NS) % SL, j = i / (2 * NS * SL);
      float sum = 0.0f;
      for (int c = 0; c < nchan; ++c) sum += bc[turn][c][s][j][v];
      const int64_t row = ((int64_t)block * a.runs.tokens + t0 + j) * a.ngroups + group;
      b.bc_part[(row * 2 + v / NS) * N + s * NS + v % NS] = sum;
    }
#pragma unroll
    for (int j = 0; j < kMark; ++j) {
      if (j < count && j % SL == slice) {
        float in = inner[j], dd = ddelta[j], uj = u[j];
        if constexpr (SL > 1) {
          in = dd = uj = 0.0f;
#pragma unroll
          for (int s = 0; s < SL; ++s) {
            in += parts[cw][s][j][0][lane];
            dd += parts[cw][s][j][1][lane];
            uj += parts[cw][s][j][2][lane];
          }
        }
        const int64_t t = t0 + j;
        const float v = raw[j] + bias;
        float ddt = __builtin_fmaf(dd, kLn2, in * x[j]);
        if (a.softplus) ddt *= sigmoid_f(v);
        dbias += ddt;
        dD = __builtin_fmaf(du[j], x[j], dD);
        if (mine) {
          store_one<BF16>(dx_out + t * out_step, lane, __builtin_fmaf(in, delta[j], skip * du[j]));
          store_one<BF16>(ddt_out + t * out_step, lane, ddt);
          if (gated) {
            const float sig = sigmoid_f(z[j]);
            const float slope = sig * __builtin_fmaf(z[j], 1.0f - sig, 1.0f);
            store_one<BF16>(dz_out + t * out_step, lane,
                            g[j] * __builtin_fmaf(skip, x[j], uj) * slope);
          }
        }
      }
    }
    if constexpr (SL > 1) __syncthreads();    // (parts are written again)
  }
  // sums over the tokens; of several slices each has some of the tokens
  if constexpr (SL > 1) {
    parts[cw][slice][0][0][lane] = dD;
    parts[cw][slice][0][1][lane] = dbias;
    __syncthreads();
    dD = dbias = 0.0f;
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      dD += parts[cw][s][0][0][lane];
      dbias += parts[cw][s][0][1][lane];
    }
  }
  if (!mine) return;
#pragma unroll
  for (int n = 0; n < NS; ++n) dA_row[(n0 + n) * a.dim] = dA[n];
  if (slice == 0) {
    dA_row[N * a.dim] = dD;
    dA_row[(N + 1) * a.dim] = dbias;
  }
  if (r.index == 0 && b.out.dinit != nullptr)
    store_states<NS>(b.out.dinit + (r.seq * a.dim + d) * N + n0, R);
}

// dB and dC: the sums over the blocks of a group's channels.
template <bool BF16>
__global__ __launch_bounds__(256) void scan_sum_bc_kernel(const BwdArgs b, int n, int parts) {
  const ScanArgs& a = b.f;
  int64_t begin = 0, end = a.runs.tokens;
  if (a.runs.cu != nullptr) {      // rows outside every sequence are left as they are
    begin = seq_bound(a.runs, 0);
    end = seq_bound(a.runs, a.runs.nseq);
  }
  const int64_t row = 2 * n * a.ngroups, all = a.runs.tokens * row;
  const int64_t i = begin * row + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= end * row) return;
  float sum = 0.0f;
  for (int p = 0; p < parts; ++p) sum += b.bc_part[p * all + i];
  const int k = (int)(i % n);
  const int64_t tg = i / (2 * n);
  store_one<BF16>(i / n % 2 ? b.out.dC : b.out.dB, tg * n + k, sum);
}

// dA, dD and ddt_bias: the sums over the slots, in their order.  64 channels of one of
// the n + 2 rows for a workgroup, the slots spread over its four waves.
__global__ __launch_bounds__(256) void scan_sum_slots_kernel(const BwdArgs b, int n) {
  __shared__ float part[4][kWave];
  const ScanArgs& a = b.f;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int k = blockIdx.x % (n + 2);
  const int64_t d = (int64_t)(blockIdx.x / (n + 2)) * kWave + lane;
  float sum = 0.0f;
  if (d < a.dim)
    for (int64_t s = wave; s < b.slots; s += 4) sum += b.dA_part[(s * (n + 2) + k) * a.dim + d];
  part[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || d >= a.dim) return;
  sum = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
  if (k < n)
    b.out.dA[d * n + k] = sum;
  else if (k == n ? b.out.dD != nullptr : b.out.ddt_bias != nullptr)
    (k == n ? b.out.dD : b.out.ddt_bias)[d] = sum;
}

int64_t channel_blocks(const ScanShape& s) {
  return s.ngroups * ((s.dim / s.ngroups + kWave - 1) / kWave);
}

int64_t run_length(const ScanShape& s) {
  const int64_t blocks = channel_blocks(s);
  const int64_t mean = (s.tokens + s.nseq - 1) / s.nseq;
  if (s.nseq * blocks >= 1024) return (4 * mean + kMark - 1) / kMark * kMark;
  int64_t run = (s.tokens * blocks + 2047) / 2048;
  run = (run + kMark - 1) / kMark * kMark;
  return run < 32 ? 32 : run;
}
int64_t most_slots(const ScanShape& s) { return s.tokens / run_length(s) + s.nseq; }
int64_t most_marks(const ScanShape& s) { return s.tokens / kMark + most_slots(s) + 1; }

// Waves of a workgroup of the second walk: N / 16 for each of up to 64 * (4 / slices)
// channels of a group.
struct Wide {
  int slices, channels, blocks;
};
Wide wide_of(const ScanShape& s) {
  Wide w;
  w.slices = s.n <= 16 ? 1 : (int)(s.n / 16);
  const int64_t blocks = (s.dim / s.ngroups + kWave - 1) / kWave;
  const int most = kWaves / w.slices;
  w.channels = (int)(blocks < most ? blocks : most);
  w.blocks = (int)((blocks + w.channels - 1) / w.channels);
  return w;
}

size_t aligned(size_t n) { return (n + 15) & ~(size_t)15; }

struct BwdLayout {
  size_t states, totals, back, marks, mark_totals, dA, bc, all;
};
BwdLayout layout(const ScanShape& s) {
  const size_t f = sizeof(float), slots = (size_t)most_slots(s), marks = (size_t)most_marks(s);
  const size_t D = (size_t)s.dim, N = (size_t)s.n;
  BwdLayout l;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += aligned(n * f);
    return p;
  };
  l.states = take(slots * N * D);
  l.totals = take(slots * D);
  l.back = take(slots * N * D);
  l.marks = take(marks * N * D);
  l.mark_totals = take(marks * D);
  l.dA = take(slots * (N + 2) * D);
  l.bc = take((size_t)wide_of(s).blocks * (size_t)(s.tokens * s.ngroups) * 2 * N);
  l.all = at;
  return l;
}

template <int NS, int SL, bool BF16>
void launch_n(const BwdArgs& b, const Wide& w, int64_t slots, int64_t blocks, hipStream_t st) {
  hipLaunchKernelGGL((scan_local_kernel<NS * SL, BF16>), dim3((unsigned)(slots * blocks)),
                     dim3(kWave), 0, st, b);
  hipLaunchKernelGGL((scan_bwd_kernel<NS, SL, BF16>),
                     dim3((unsigned)(slots * b.f.ngroups * w.blocks)),
                     dim3(kWave * w.channels * w.slices), 0, st, b);
}

}  // namespace

bool scan_bwd_fits(const ScanShape& s) {
  const int64_t rows = 2 * s.n * s.ngroups;
  return most_slots(s) < kScanMaxBlocks / channel_blocks(s) &&
         s.tokens <= (kScanMaxBlocks / 4 - 1) * 256 / rows;
}

size_t scan_bwd_workspace(const ScanShape& s) { return layout(s).all; }

int launch_scan_bwd(const ScanInputs& in, const float* init, const int32_t* cu, const void* dy,
                    const float* dfinal, const ScanGradients& out, void* ws, bool softplus,
                    bool bf16, const ScanShape& s, void* stream) {
  clear_launch_error();
  const BwdLayout l = layout(s);
  char* base = (char*)ws;
  BwdArgs b{};
  ScanArgs& a = b.f;
  a = make_scan_args(in, init, s, softplus);
  a.runs = make_run_grid(cu, s.tokens, s.nseq, run_length(s));
  b.slots = run_slots(a.runs);
  a.states = (float*)(base + l.states);
  a.totals = (float*)(base + l.totals);
  b.back = (float*)(base + l.back);
  b.marks = (float*)(base + l.marks);
  b.mark_totals = (float*)(base + l.mark_totals);
  b.dA_part = (float*)(base + l.dA);
  b.bc_part = (float*)(base + l.bc);
  b.dy = dy;
  b.dfinal = dfinal;
  b.out = out;
  const Wide w = wide_of(s);
  const int64_t blocks = channel_blocks(s);
  hipStream_t st = (hipStream_t)stream;
  switch (s.n) {
#define SSD_SCAN(N, NS, SL)                                        \
  case N:                                                          \
    if (bf16)                                                      \
      launch_n<NS, SL, true>(b, w, b.slots, blocks, st);           \
    else                                                           \
      launch_n<NS, SL, false>(b, w, b.slots, blocks, st);          \
    break
    SSD_SCAN(8, 8, 1);
    SSD_SCAN(16, 16, 1);
    SSD_SCAN(32, 16, 2);
    default:
      SSD_SCAN(64, 16, 4);
#undef SSD_SCAN
  }
  const int64_t values = s.tokens * s.ngroups * 2 * s.n;
  const dim3 grid((unsigned)((values + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL((scan_sum_bc_kernel<true>), grid, dim3(256), 0, st, b, (int)s.n, w.blocks);
  else
    hipLaunchKernelGGL((scan_sum_bc_kernel<false>), grid, dim3(256), 0, st, b, (int)s.n,
                       w.blocks);
  hipLaunchKernelGGL(scan_sum_slots_kernel,
                     dim3((unsigned)((s.dim + kWave - 1) / kWave * (s.n + 2))), dim3(256), 0, st,
                     b, (int)s.n);
  return (int)hipGetLastError();
}

}  // namespace ssd
