// The selective scan over whole (packed) sequences.  Per channel d and state n,
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,   u_t = sum_n C_t h_t + D x_t
// The decay is another number for each channel, state and token, so the products between tokens
// do not factor into matrix products: what is left is the recurrence, five vector instructions
// for each (token, channel, state), six with outputs (an exponential counts for two).
//
// MI355X design.  A lane owns a channel with all its states, a wave 64 channels of one group:
// sums over states need no exchange, B_t and C_t are the same for the wave and come as scalar
// operands, rows are read and written 64 channels at a time.  What counts then is instructions and
// enough waves (32768 x 5120 with 16 states in bf16: 1.35 GB take 260 us at a copy's rate, a
// walk's instructions 400):
//   - walks have no branch on what a call has (softplus, gate): both values are formed and one
//     picked.  With branches, the compiler moved work across them and spilled (1471 -> 1190 us);
//   - rows are read a block of four tokens ahead, B and C a piece of 32 bytes ahead;
//   - sequences that do not fill the chip are cut into runs (scan_cut, scan_whole).  A first walk
//     leaves the state of every run but the last from zeros; the states at the runs' starts are
//     then h = exp(A sum delta) h + left, joined by a launch of its own or, for few runs, by each
//     run; the second walk has the outputs.  The first walk may take a channel's states in
//     slices, since nothing is summed over them (64 states: scan 439 -> 348 us).
// Time sums are held in 64 bits, since every token rounds them again; all else is fp32.
//
// Measured at one sequence of 32768 tokens of 5120 channels of 16 states in bf16 (means of the
// profiler): first walk 407 us, joining 39, second walk 547 (vector unit busy all the time in both
// walks); it cannot do with a single walk: 80 waves for 1024 SIMDs.  Short calls: 643 tokens of
// 1536 channels 10 + 8 + 10.  64 states take two waves a SIMD, whose 256 registers lack 18 to
// 27 for the outputs (76 bytes of scratch a lane); 32 and fewer fit.
#include "ssd_selective_scan.h"

#include "ssd_host.h"

namespace ssd {
namespace {

// The states at the starts of many runs: a lane owns one state of one channel and goes through a
// sequence's runs, 16 of them on the way at once; a workgroup has 64 channels and four of the N
// states, and every gridDim.y'th sequence.  With `back` it also goes down, through the gradients
// at the runs' starts.
template <int N>
__global__ __launch_bounds__(256) void scan_join_kernel(const ScanArgs a, float* back,
                                                        const float* dfinal) {
  const int lane = threadIdx.x % kWave;
  const int blocks = (int)((a.dim + kWave - 1) / kWave);
  const int n = (int)(blockIdx.x / blocks) * 4 + threadIdx.x / kWave;
  const int64_t d = (int64_t)(blockIdx.x % blocks) * kWave + lane;
  const bool on = d < a.dim;
  const float A2 = on ? in_powers_of_two(a.in.A[d * N + n]) : 0.0f;
  const RunGrid& g = a.runs;
  constexpr int kAhead = 16;
  // 64 sequences at a time: those that have more than one run
  for (int64_t i0 = blockIdx.y; i0 < g.nseq; i0 += (int64_t)gridDim.y * kWave) {
    const int64_t mine = i0 + (int64_t)gridDim.y * lane;
    int first = 0, count = 0;
    if (mine < g.nseq) {
      if (g.cu != nullptr) {
        const int begin = seq_bound(g, g.cu[mine]), end = seq_bound(g, g.cu[mine + 1]);
        first = first_slot(g, begin, (int)mine);
        count = end > begin ? run_count(g, end - begin) : 0;
      } else {
        first = (int)mine * g.per_seq;
        count = g.per_seq;
      }
    }
    uint64_t many = __ballot(count > 1);
    while (many != 0) {
      const int k = __builtin_ctzll(many);
      many &= many - 1;
      const int64_t s0 = __shfl(first, k, kWave), runs = __shfl(count, k, kWave);
      const int64_t seq = i0 + (int64_t)gridDim.y * k;
      if (!on) continue;
      float* state = a.states + (s0 * N + n) * a.dim + d;
      const float* total = a.totals + s0 * a.dim + d;
      const int64_t step = N * a.dim;
      float h = a.init != nullptr ? a.init[(seq * a.dim + d) * N + n] : 0.0f;
      for (int64_t s = 0; s < runs; s += kAhead) {
        float left[kAhead], decay[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int64_t at = s + e < runs ? s + e : runs - 1;
          left[e] = state[at * step];
          decay[e] = exp2_hw(total[at * a.dim] * A2);
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          if (s + e >= runs) break;
          state[(s + e) * step] = h;
          h = s + e == 0 ? left[e] : __builtin_fmaf(decay[e], h, left[e]);
        }
      }
      if (back == nullptr) continue;
      float* grad = back + (s0 * N + n) * a.dim + d;
      float R = dfinal != nullptr ? dfinal[(seq * a.dim + d) * N + n] : 0.0f;
      for (int64_t s = runs - 1; s >= 0; s -= kAhead) {
        float left[kAhead], decay[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int64_t at = s - e > 0 ? s - e : 0;
          left[e] = grad[at * step];
          decay[e] = exp2_hw(total[at * a.dim] * A2);
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          if (s - e < 0) break;
          grad[(s - e) * step] = R;
          R = __builtin_fmaf(decay[e], R, left[e]);
        }
      }
    }
  }
}

// Tokens read at a time; one such block is on the way while another is worked on.
constexpr int kBlock = 4;

// One run of one sequence for 64 channels of a group.
//   OUT: outputs, from the state that the runs before it leave
//   else: the state that the run leaves (from zeros, the first run from the initial state)
// Lanes past the group's end do what its last channel's lane does, and store the same.
// Outputs need all N states of a channel; without, a wave takes NS of them (blockIdx.y).
template <int N, int NS, bool BF16, bool OUT>
__global__ __launch_bounds__(kWave, NS == 64 ? 2 : 1) void scan_kernel(const ScanArgs a) {
  static_assert(!OUT || NS == N, "outputs are sums over the states");
  const ScanPlace pl(a);
  const int n0 = OUT ? 0 : (int)blockIdx.y * NS;
  const int own = (int)threadIdx.x < pl.lanes ? (int)threadIdx.x : pl.lanes - 1;
  const int64_t d = pl.channel + own;
  float A2[NS], h[NS];
  load_states<NS>(a.in.A + d * N + n0, A2);
  const float bias = a.in.dt_bias ? a.in.dt_bias[d] : 0.0f;
  const float skip = OUT && a.in.D ? a.in.D[d] : 0.0f;
  const Run r = find_ordered_run(a.runs, pl.at);
  if (!r.on) return;
  const bool last = r.index == r.count - 1;
  if (!OUT && last) return;
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    A2[n] = in_powers_of_two(A2[n]);
    h[n] = 0.0f;
  }
  if constexpr (OUT) {
    if (a.joined && r.count > 1) {
      load_run<N>(a, r.slot, d, h);
    } else if (r.index > 0) {
      fold_runs<N>(a, r.first, r.slot, d, A2, h, [&](int64_t s, int n) {
        return a.states[(s * N + n) * a.dim + d];
      });
    } else if (a.init != nullptr) {
      if (last)
        load_states<N>(a.init + ((int64_t)r.seq * a.dim + d) * N, h);
      else
        load_run<N>(a, r.first + r.count - 1, d, h);
    }
  } else if (r.index == 0 && a.init != nullptr) {
    load_states<NS>(a.init + ((int64_t)r.seq * a.dim + d) * N + n0, h);
    if (!a.joined) store_run<N>(a.states, a, r.first + r.count - 1, d, n0, h);
  }
  const bool gated = OUT && a.in.z != nullptr;

  Rows<BF16> rows(a, pl, r.begin, own, N, n0);
  const int64_t y_step = a.dim * (BF16 ? 2 : 4);
  char* y = OUT ? (char*)a.y + pl.channel * (BF16 ? 2 : 4) + r.begin * y_step : nullptr;
  const int tokens = (int)(r.end - r.begin);    // (fewer than 2^31)
  typedef StateRows<NS, BF16, OUT> Bc;
  Bc bc(rows.B, rows.C, rows.b_step, rows.c_step, tokens);
  double total = 0.0;
  typedef typename Raw<BF16>::type raw;
  struct Block {
    raw x[kBlock], dt[kBlock], z[kBlock];
  };
  // the next block's rows, `left` of them there (the others read the last one's)
  auto load = [&](Block& b, int left) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      b.x[j] = load_raw<BF16>(rows.x, rows.lane);
      b.dt[j] = load_raw<BF16>(rows.dt, rows.lane);
      if (OUT) b.z[j] = load_raw<BF16>(rows.z, rows.lane);
      if (j + 1 < left || left >= kBlock) {
        rows.x += rows.x_step;
        rows.dt += rows.dt_step;
        rows.z += rows.z_step;
      }
    }
  };
  auto work = [&](const Block& b, int left) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      if (j >= left) break;
      const float v = Raw<BF16>::get(b.dt[j]) + bias;
      const float delta = pick(a.softplus, softplus_f(v), v);
      const float x = Raw<BF16>::get(b.x[j]), dx = delta * x;
      float u[2] = {skip * x, 0.0f};
#pragma unroll
      for (int k = 0; k < Bc::kPieces; ++k) {
        typename Bc::S B, C;
        bc.next(k, B, C);
#pragma unroll
        for (int i = 0; i < Bc::kPiece; ++i) {
          const int n = k * Bc::kPiece + i;
          h[n] = __builtin_fmaf(exp2_hw(delta * A2[n]), h[n], dx * B[i]);
          if (OUT) u[n & 1] = __builtin_fmaf(C[i], h[n], u[n & 1]);
        }
      }
      if constexpr (OUT) {
        const float z = Raw<BF16>::get(b.z[j]), out = u[0] + u[1];
        store_raw<BF16>(y, rows.lane, pick(gated, out * (z * sigmoid_f(z)), out));
        y += y_step;
      } else {
        total += delta;
      }
    }
  };
  Block even, odd;
  if (tokens > 0) load(even, tokens);
  int t = 0;
  for (; t + 3 * kBlock <= tokens; t += 2 * kBlock) {
    load(odd, kBlock);
    work(even, kBlock);
    load(even, kBlock);
    work(odd, kBlock);
  }
  for (; t < tokens; t += kBlock) {
    work(even, tokens - t);
    if (t + kBlock < tokens) load(even, tokens - t - kBlock);
  }
  if constexpr (OUT) {
    if (last && a.fin != nullptr) store_states<N>(a.fin + ((int64_t)r.seq * a.dim + d) * N, h);
  } else {
    store_run<N>(a.states, a, r.slot, d, n0, h);
    a.totals[(int64_t)r.slot * a.dim + d] = (float)total;
  }
}

struct ScanPlan {
  RunGrid runs;
  bool split;
  int64_t slots, blocks;   // workgroups for a slot
};

ScanPlan make_plan(const ScanShape& s, const int32_t* cu) {
  ScanPlan p;
  p.runs = scan_grid(cu, s, false);
  p.slots = run_slots(p.runs);
  p.split = cu != nullptr ? s.tokens > p.runs.whole : p.runs.per_seq > 1;
  p.blocks = channel_blocks(s);
  return p;
}

template <int N>
void join_n(const ScanArgs& a, float* back, const float* dfinal, hipStream_t st) {
  const int64_t blocks = (a.dim + kWave - 1) / kWave * (N / 4);
  const int64_t want = 2048 / blocks;
  const int64_t across = want < 1 ? 1 : (want < a.runs.nseq ? want : a.runs.nseq);
  hipLaunchKernelGGL((scan_join_kernel<N>), dim3((unsigned)blocks, (unsigned)across), dim3(256),
                     0, st, a, back, dfinal);
}

template <int N, bool BF16>
int launch_n(const ScanArgs& a, const ScanPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.slots * p.blocks));
  if (p.split) {
    constexpr int NS = N < 32 ? N : 32;
    hipLaunchKernelGGL((scan_kernel<N, NS, BF16, false>), dim3(grid.x, N / NS), dim3(kWave), 0,
                       st, a);
    if (a.joined) launch_scan_join(a, N, nullptr, nullptr, st);
  }
  hipLaunchKernelGGL((scan_kernel<N, N, BF16, true>), grid, dim3(kWave), 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace

void launch_scan_join(const ScanArgs& a, int64_t n, float* back, const float* dfinal,
                      hipStream_t st) {
  if (n == 8)
    join_n<8>(a, back, dfinal, st);
  else if (n == 16)
    join_n<16>(a, back, dfinal, st);
  else if (n == 32)
    join_n<32>(a, back, dfinal, st);
  else
    join_n<64>(a, back, dfinal, st);
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
  a.joined = joins(p.runs);
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
