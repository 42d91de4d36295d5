// The selective scan over whole (packed) sequences.  Per channel d and state n,
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,   u_t = sum_n C_t h_t + D x_t
#include "ssd_selective_scan.h"

#include "ssd_host.h"

namespace ssd {
namespace {

template <bool BF16, bool OUT>
struct TokenBlock {
  float x[kBlock], dt[kBlock], z[kBlock];
  __device__ __forceinline__ void load(const Rows<BF16>& r, int64_t t0, int64_t end, bool gated) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      const int64_t t = t0 + j < end ? t0 + j : end - 1;
      x[j] = load_one<BF16>(r.x + t * r.x_step, r.lane);
      dt[j] = load_one<BF16>(r.dt + t * r.dt_step, r.lane);
      if (OUT) z[j] = gated ? load_one<BF16>(r.z + t * r.z_step, r.lane) : 0.0f;
    }
  }
};

// One run of one sequence for 64 channels of a group.
//   OUT: outputs, from the state that the runs before it leave
//   else: the state that the run leaves (from zeros, the first run from the initial state)
template <int N, bool BF16, bool OUT>
__global__ __launch_bounds__(kWave) void scan_kernel(const ScanArgs a) {
  const ScanPlace pl(a);
  const Run r = find_run(a.runs, pl.slot);
  if (!r.on) return;
  const bool last = r.index == r.count - 1;
  if (!OUT && last) return;
  const int lane = threadIdx.x;
  const bool mine = lane < pl.lanes;
  const int own = mine ? lane : pl.lanes - 1;
  const int64_t d = pl.channel + own;

  float A2[N], h[N];
  load_states<N>(a.in.A + d * N, A2);
#pragma unroll
  for (int n = 0; n < N; ++n) A2[n] *= kLog2e;
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = 0.0f;
  if (r.index == 0 && a.init != nullptr) {
    if (OUT && !last) {
      load_run<N>(a, r.first + r.count - 1, d, h);
    } else {
      load_states<N>(a.init + (r.seq * a.dim + d) * N, h);
      if (!OUT && mine) store_run<N>(a, r.first + r.count - 1, d, h);
    }
  }
  if constexpr (OUT) fold_runs<N>(a, r.first, pl.slot, d, A2, h);
  const float bias = a.in.dt_bias ? a.in.dt_bias[d] : 0.0f;
  const float skip = OUT && a.in.D ? a.in.D[d] : 0.0f;
  const bool gated = OUT && a.in.z != nullptr;

  const Rows<BF16> rows(a, pl, own, N);
  char* y = OUT ? (char*)a.y + pl.channel * (BF16 ? 2 : 4) : nullptr;
  const int64_t y_step = a.dim * (BF16 ? 2 : 4);
  double total = 0.0;
  TokenBlock<BF16, OUT> next;
  if (r.begin < r.end) next.load(rows, r.begin, r.end, gated);
  for (int64_t t0 = r.begin; t0 < r.end; t0 += kBlock) {
    const TokenBlock<BF16, OUT> cur = next;
    next.load(rows, t0 + kBlock, r.end, gated);
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      if (t0 + j >= r.end) break;
      const States<N, BF16> B(rows.B, (t0 + j) * rows.b_step);
      const float v = cur.dt[j] + bias;
      const float delta = a.softplus ? softplus_f(v) : v;
      const float x = cur.x[j], dx = delta * x;
      if constexpr (OUT) {
        const States<N, BF16> C(rows.C, (t0 + j) * rows.c_step);
        float u[2] = {skip * x, 0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
          h[n] = __builtin_fmaf(exp2_hw(delta * A2[n]), h[n], dx * B[n]);
          u[n & 1] = __builtin_fmaf(C[n], h[n], u[n & 1]);
        }
        float out = u[0] + u[1];
        if (gated) out *= cur.z[j] * sigmoid_f(cur.z[j]);
        if (mine) store_one<BF16>(y + (t0 + j) * y_step, lane, out);
      } else {
        total += delta;
#pragma unroll
        for (int n = 0; n < N; ++n)
          h[n] = __builtin_fmaf(exp2_hw(delta * A2[n]), h[n], dx * B[n]);
      }
    }
  }
  if (!mine) return;
  if constexpr (OUT) {
    if (last && a.fin != nullptr) store_states<N>(a.fin + (r.seq * a.dim + d) * N, h);
  } else {
    store_run<N>(a, pl.slot, d, h);
    a.totals[pl.slot * a.dim + d] = (float)total;
  }
}

// The tokens of a run.  Waves of one run for each channel block of every sequence may
// leave most of the chip idle; runs that start from the states of those before them
// cost a second walk over all but each sequence's last one.
int64_t run_length(const ScanShape& s) {
  const int64_t blocks = s.ngroups * ((s.dim / s.ngroups + kWave - 1) / kWave);
  const int64_t mean = (s.tokens + s.nseq - 1) / s.nseq;
  if (s.nseq * blocks >= 1024) return 4 * mean;
  int64_t run = (s.tokens * blocks + 4095) / 4096;
  run = (run + kBlock - 1) / kBlock * kBlock;
  return run < 32 ? 32 : run;
}

struct ScanPlan {
  RunGrid runs;
  bool split;
  int64_t slots, blocks;   // workgroups for a slot
};

ScanPlan make_plan(const ScanShape& s, const int32_t* cu) {
  ScanPlan p;
  p.runs = make_run_grid(cu, s.tokens, s.nseq, run_length(s));
  p.slots = run_slots(p.runs);
  p.split = cu != nullptr ? s.tokens > p.runs.run : p.runs.per_seq > 1;
  p.blocks = s.ngroups * ((s.dim / s.ngroups + kWave - 1) / kWave);
  return p;
}

// More slots than without cu, so that the workspace's size does not ask for it.
int64_t most_slots(const ScanShape& s) { return s.tokens / run_length(s) + s.nseq; }

template <int N, bool BF16>
int launch_n(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.slots * p.blocks));
  if (p.split)
    hipLaunchKernelGGL((scan_kernel<N, BF16, false>), grid, dim3(kWave), 0, st, a);
  hipLaunchKernelGGL((scan_kernel<N, BF16, true>), grid, dim3(kWave), 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace

bool scan_fits(const ScanShape& s) {
  const int64_t blocks = s.ngroups * ((s.dim / s.ngroups + kWave - 1) / kWave);
  return most_slots(s) < kScanMaxBlocks / blocks;
}

size_t scan_fwd_workspace(const ScanShape& s) {
  if (s.tokens <= run_length(s)) return 16;
  return sizeof(float) * (size_t)(most_slots(s) * s.dim * (s.n + 1));
}

int launch_scan_fwd(const ScanInputs& in, const float* init, const int32_t* cu, void* y,
                    float* fin, void* ws, bool softplus, bool bf16, const ScanShape& s,
                    void* stream) {
  clear_launch_error();
  const ScanPlan p = make_plan(s, cu);
  ScanArgs a = make_scan_args(in, init, s, softplus);
  a.y = y;
  a.fin = fin;
  a.runs = p.runs;
  a.states = (float*)ws;
  a.totals = (float*)ws + p.slots * s.dim * s.n;
  hipStream_t st = (hipStream_t)stream;
  switch (s.n) {
#define SSD_SCAN(N) \
  case N: return bf16 ? launch_n<N, true>(a, p, st) : launch_n<N, false>(a, p, st)
    SSD_SCAN(8);
    SSD_SCAN(16);
    SSD_SCAN(32);
    default:
      SSD_SCAN(64);
#undef SSD_SCAN
  }
}

}  // namespace ssd
