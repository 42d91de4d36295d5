// Gradients of the selective scan (ssd_selective_scan.hip).  With e_t = exp(delta_t A), du = dy
// silu(z) and the state's gradient R_t = C_t du_t + e_{t+1} R_{t+1}, every gradient is a sum over
// states, channels or tokens of products of R_t, h_t and h_{t-1} (include/ssd_selective.h).
//
// States are not kept from the forward call (64 bytes for each channel and token of 16 states,
// against 6 of inputs in bf16), and h_{t-1} = (h_t - delta x B) / e_t loses what has decayed.
// So:
//   1. scan_local_kernel goes up every run from zeros and leaves the run's last state, the states
//      at every eighth token (marks), and the gradient that the run's own outputs give the state
//      at its start;
//   2. scan_join_kernel makes the states at the runs' starts and the gradients at their ends from
//      these (few runs: the second walk does it itself);
//   3. scan_bwd_kernel goes down every run, eight tokens at a time: up from the mark with the
//      states in registers, then down through them;
//   4. two kernels add what the second walk leaves of dB and dC (for each block of channels) and
//      of dA, dD and ddt_bias (for each run), in a fixed order: no atomics.
//
// MI355X design.  All of it is bound by vector instructions, so the second walk is laid out for
// few of them: sums over N states of a channel (dx, ddt, dz) want its states in one lane, sums
// over a group's channels (dB, dC) want channels in one lane.  Four states of two channels are the
// middle: a token costs a lane 24 instructions (an exponential counts for two) for each of its 8
// (state, channel) pairs, of which 14 are the formula's: five for h, nine for R, its product with
// the decay and what is summed.  Per token and channel six DPP adds sum over four lanes; dB and dC
// go through LDS, four tokens at a time, where the lanes of a wave add 8 vectors each.  (A channel
// a lane with its sums over lanes by DPP alone: 2634 us for what takes 533 below.)  Nine states of
// 2 x 4 values take 72 of the 256 registers of two waves a SIMD; decays of six of the eight tokens
// wait in LDS, the others are formed again (one exponential costs two instructions). Eight states
// a channel have two lanes a channel, more tokens of their own, and run at one wave a SIMD
// (measured 737 us against 1125 at two, which spill).  Waves of a workgroup share B and C and
// their sums of dB and dC: four of them 622 us and 13 for the sums over blocks, two 606 and 23,
// eight 680 and 8.
//
// Measured at 16384 tokens of 2560 channels of 16 states in bf16 (three sequences; means of the
// profiler): first walk 222 us (vector unit busy 79%), joining 19, second walk 533 (78%: two waves
// a SIMD do not cover LDS reads and barriers; B and C read a token ahead spill, 670), sums 13 + 8.
// 335 MB of marks are written and read; at 5.15 TB/s all bytes of both walks take 350 us.  The
// second walk's 256 registers lack four for 16 and 64 states (20 bytes of scratch a lane), and six
// to 17 where channels are not read in pairs (28 to 72 bytes).
#include "ssd_selective_scan.h"

#include "ssd_host.h"

#include <type_traits>

namespace ssd {
namespace {

constexpr int kWaves = kBwdWaves;
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
  Divide by_wide, by_wide_slot;   // by the second walk's blocks of a group, and of all
};

// The first walk, up the tokens: of each run the state that it leaves, the states inside
// it, and the gradient that its outputs give the state at its start,
//   sum_t (prod_{s<=t} exp(delta_s A)) C_t du_t
// Lanes past the group's end do what its last channel's lane does, and store the same.
// A wave takes NS of a channel's N states (blockIdx.y).
template <int N, int NS, bool BF16>
__global__ __launch_bounds__(kWave) void scan_local_kernel(const BwdArgs b) {
  const ScanArgs& a = b.f;
  const ScanPlace pl(a);
  const int n0 = (int)blockIdx.y * NS;
  const int own = (int)threadIdx.x < pl.lanes ? (int)threadIdx.x : pl.lanes - 1;
  const int64_t d = pl.channel + own;
  float A2[NS], h[NS], decay[NS], back[NS];
  load_states<NS>(a.in.A + d * N + n0, A2);
  const float bias = a.in.dt_bias ? a.in.dt_bias[d] : 0.0f;
  const Run r = find_ordered_run(a.runs, pl.at);
  if (!r.on) return;
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    A2[n] = in_powers_of_two(A2[n]);
    h[n] = 0.0f;
    decay[n] = 1.0f;
    back[n] = 0.0f;
  }
  if (r.index == 0 && a.init != nullptr)
    load_states<NS>(a.init + ((int64_t)r.seq * a.dim + d) * N + n0, h);
  const bool gated = a.in.z != nullptr;
  Rows<BF16> rows(a, pl, r.begin, own, N, n0);
  const int64_t dy_step = a.dim * (BF16 ? 2 : 4);
  const char* dy = (const char*)b.dy + pl.channel * (BF16 ? 2 : 4) + r.begin * dy_step;
  const int64_t mark0 = first_mark(r, r.slot);
  const int tokens = (int)(r.end - r.begin);
  typedef StateRows<NS, BF16, true> Bc;
  Bc bc(rows.B, rows.C, rows.b_step, rows.c_step, tokens);
  double total = 0.0;
  constexpr int kBlock = 4;
  static_assert(kMark == 2 * kBlock, "marks lie between pairs of blocks");
  typedef typename Raw<BF16>::type raw;
  struct Block {
    raw x[kBlock], dt[kBlock], z[kBlock], g[kBlock];
  };
  auto load = [&](Block& k, int left) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      k.x[j] = load_raw<BF16>(rows.x, rows.lane);
      k.dt[j] = load_raw<BF16>(rows.dt, rows.lane);
      k.g[j] = load_raw<BF16>(dy, rows.lane);
      k.z[j] = load_raw<BF16>(rows.z, rows.lane);
      if (j + 1 < left || left >= kBlock) {
        rows.x += rows.x_step;
        rows.dt += rows.dt_step;
        rows.z += rows.z_step;
        dy += dy_step;
      }
    }
  };
  auto mark = [&](int64_t t) {
    const int64_t m = mark0 + t / kMark;
    int64_t step = a.dim;
    asm("" : "+s"(step));      // (its multiples would stay in scalar registers)
    float* p = b.marks + (m * N + n0) * step + d;
#pragma unroll
    for (int n = 0; n < NS; ++n, p += step) *p = h[n];
    b.mark_totals[m * step + d] = (float)total;
  };
  auto work = [&](const Block& k, int left) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      if (j >= left) break;
      const float v = Raw<BF16>::get(k.dt[j]) + bias;
      const float delta = pick(a.softplus, softplus_f(v), v);
      const float dx = delta * Raw<BF16>::get(k.x[j]);
      const float dy = Raw<BF16>::get(k.g[j]), z = Raw<BF16>::get(k.z[j]);
      const float g = pick(gated, dy * (z * sigmoid_f(z)), dy);
      total += delta;
#pragma unroll
      for (int p = 0; p < Bc::kPieces; ++p) {
        typename Bc::S B, C;
        bc.next(p, B, C);
#pragma unroll
        for (int i = 0; i < Bc::kPiece; ++i) {
          const int n = p * Bc::kPiece + i;
          const float e = exp2_hw(delta * A2[n]);
          h[n] = __builtin_fmaf(e, h[n], dx * B[i]);
          decay[n] *= e;
          back[n] = __builtin_fmaf(decay[n], C[i] * g, back[n]);
        }
      }
    }
  };
  Block even, odd;
  if (tokens > 0) load(even, tokens);
  int t = 0;
  for (; t + 3 * kBlock <= tokens; t += 2 * kBlock) {
    if (t > 0) mark(t);
    load(odd, kBlock);
    work(even, kBlock);
    load(even, kBlock);
    work(odd, kBlock);
  }
  for (; t < tokens; t += kBlock) {
    if (t > 0 && t % kMark == 0) mark(t);
    work(even, tokens - t);
    if (t + kBlock < tokens) load(even, tokens - t - kBlock);
  }
  store_run<N>(a.states, a, r.slot, d, n0, h);
  store_run<N>(b.back, a, r.slot, d, n0, back);
  a.totals[(int64_t)r.slot * a.dim + d] = (float)total;
}

// ---- the second walk, down the tokens
// A lane holds four states of two neighbouring channels, the N/4 lanes of a channel pair
// lie side by side: sums over the states are lane exchanges within the group, sums
// over the channels (dB, dC) start within the lane and go on through LDS.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kRowRor8 = 0x128;
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(
      __builtin_amdgcn_mov_dpp(__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

template <int N>
struct Lanes {
  static constexpr int L = N / 4;                        // lanes of a channel pair
  static constexpr int kPairs = kWave / L;               // pairs of a wave
  static constexpr int kChannels = 2 * kPairs;
  static constexpr int kTurns = L < kMark ? L : kMark;   // lanes that share a block's tokens
  static constexpr int kOwn = kMark / kTurns;            // tokens of a lane, kTurns apart

  // The sum over a pair's lanes, in each of them.
  static __device__ __forceinline__ float sum(float v) {
    v += moved<kXor1>(v);
    if (L >= 4) v += moved<kXor2>(v);
    if (L >= 8) v += moved<kHalfMirror>(v);
    if (L >= 16) v += moved<kRowRor8>(v);
    return v;
  }
  // Of several values at once (the call at 16384 x 2560 x 16: one after the other 806 to 808 us
  // in five rounds, this 802 to 804).
  template <int K>
  static __device__ __forceinline__ void sum(float (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += moved<kXor1>(v[k]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (L >= 4) v[k] += moved<kXor2>(v[k]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (L >= 8) v[k] += moved<kHalfMirror>(v[k]);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (L >= 16) v[k] += moved<kRowRor8>(v[k]);
  }
  // The value of the pair's lane `from`.
  template <int FROM>
  static __device__ __forceinline__ float bcast(float v) {
    if constexpr (L == 2) return moved<FROM * 0x55 + 0xA0>(v);          // (f, f, 2+f, 2+f)
    if constexpr (L == 4) return moved<FROM * 0x55>(v);
    return __shfl(v, (threadIdx.x & (kWave - 1) & ~(L - 1)) + FROM, kWave);
  }
};

// One element of two neighbouring channels, as it lies in memory: `at` bytes into a row, and
// `apart` bytes behind it; in one access where every lane has both (`paired`).
template <bool BF16>
struct Pair;
template <>
struct Pair<true> {
  uint32_t w;
  __device__ __forceinline__ void load(rsrc_t row, uint32_t at, uint32_t apart, bool paired) {
    if (paired)
      w = load_b32(row, at);
    else
      w = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row, (int)at, 0, 0) |
          (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row, (int)(at + apart), 0, 0)
              << 16;
  }
  __device__ __forceinline__ float get(int c) const { return c ? bf16_hi(w) : bf16_lo(w); }
  static __device__ __forceinline__ void store(rsrc_t row, uint32_t at, const float (&v)[2],
                                               const bool (&on)[2], bool paired) {
    const uint32_t u = pack_bf16(v[0], v[1]);
    if (paired) {
      if (on[0]) __builtin_amdgcn_raw_buffer_store_b32(u, row, (int)at, 0, 0);
    } else {
      if (on[0]) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)u, row, (int)at, 0, 0);
      if (on[1])
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(u >> 16), row, (int)at + 2, 0, 0);
    }
  }
};
template <>
struct Pair<false> {
  float v[2];
  __device__ __forceinline__ void load(rsrc_t row, uint32_t at, uint32_t apart, bool paired) {
    if (paired) {
      const u32x2 u = load_b64(row, at);
      v[0] = __uint_as_float(u[0]);
      v[1] = __uint_as_float(u[1]);
    } else {
      v[0] = load_f32(row, at);
      v[1] = load_f32(row, at + apart);
    }
  }
  __device__ __forceinline__ float get(int c) const { return v[c]; }
  static __device__ __forceinline__ void store(rsrc_t row, uint32_t at, const float (&v)[2],
                                               const bool (&on)[2], bool paired) {
    const u32x2 u = {__float_as_uint(v[0]), __float_as_uint(v[1])};
    if (paired) {
      if (on[0]) __builtin_amdgcn_raw_buffer_store_b64(u, row, (int)at, 0, 0);
    } else {
      if (on[0]) __builtin_amdgcn_raw_buffer_store_b32(u[0], row, (int)at, 0, 0);
      if (on[1]) __builtin_amdgcn_raw_buffer_store_b32(u[1], row, (int)at + 4, 0, 0);
    }
  }
};

// LDS writes of a wave's lanes before it are seen by their reads behind it (a wave's LDS
// operations keep their order; this keeps the compiler's).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

constexpr int kBatch = 4;      // tokens whose dB and dC are summed over a wave's lanes at once

template <int N, bool BF16, bool PAIRED>
__global__ __launch_bounds__(kWave * kWaves, N == 8 ? 1 : 2) void scan_bwd_kernel(const BwdArgs b) {
  using La = Lanes<N>;
  constexpr int L = La::L, OWN = La::kOwn, TURNS = La::kTurns;
  constexpr int el = BF16 ? 2 : 4;
  __shared__ f32x4 bc_in[2][kMark][2][L];                 // B and C of a block
  __shared__ f32x4 values[kWaves][kBatch][2][kWave];      // dB and dC of each lane
  // Decays that stay besides those that lie in `values`: of two more tokens 795 -> 783 us for
  // 16 states and 1565 -> 1556 for 32; 64 leave no room for them.
  constexpr int kMore = N == 64 ? 0 : 2;
  __shared__ f32x4 more[kWaves][kMore ? kMore : 1][2][kWave];
  __shared__ f32x4 sums[2][kWaves][kMark][2][L];          // and of each wave
  __shared__ f32x4 start[kWaves][2][kWave];               // the state at the run's start

  const ScanArgs& a = b.f;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave, q = lane % L;
  const int place_at = (int)b.by_wide_slot.of(blockIdx.x);
  const uint32_t rest = blockIdx.x - (uint32_t)place_at * b.by_wide_slot.d;
  const int group = (int)b.by_wide.of(rest);
  const int block = (int)(rest - (uint32_t)group * b.by_wide.d);
  // the lane's channels; past the group's end they stand for nothing (zeros), and read the
  // last one's rows (the last two's where they are read in pairs: a group is even then)
  const int at = (block * kWaves + wave) * La::kChannels + lane / L * 2;
  const bool on[2] = {at < a.group_dim, at + 1 < a.group_dim};
  const int64_t base = (int64_t)group * a.group_dim;
  const int64_t d[2] = {base + (on[0] ? at : a.group_dim - (PAIRED ? 2 : 1)),
                        base + (on[1] ? at + 1 : a.group_dim - 1)};

  const Run r = find_ordered_run(a.runs, place_at);
  const int64_t slot = r.slot;
  float* dA_row = b.dA_part + slot * (N + 2) * a.dim;
  if (!r.on || r.begin >= r.end) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!on[c]) continue;
#pragma unroll
      for (int n = 0; n < 4; ++n) dA_row[(4 * q + n) * a.dim + d[c]] = 0.0f;
      if (q == 0) dA_row[N * a.dim + d[c]] = dA_row[(N + 1) * a.dim + d[c]] = 0.0f;
      // an empty sequence passes its final state's gradient on
      if (r.on && b.out.dinit != nullptr) {
        const int64_t i = ((int64_t)r.seq * a.dim + d[c]) * N + 4 * q;
        *(f32x4*)(b.out.dinit + i) =
            b.dfinal ? *(const f32x4*)(b.dfinal + i) : (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
    return;
  }

  float A2[2][4], R[2][4], dA[2][4];
  float bias[2], skip[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const f32x4 A = *(const f32x4*)(a.in.A + d[c] * N + 4 * q);
    f32x4 h = {0.0f, 0.0f, 0.0f, 0.0f}, back = h;
    const int64_t state = ((int64_t)r.seq * a.dim + d[c]) * N + 4 * q;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      A2[c][n] = in_powers_of_two(A[n]);
      dA[c][n] = 0.0f;
    }
    // the state at the run's start, and the gradient of the state at its end
    if (a.joined && r.count > 1) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        h[n] = a.states[(slot * N + 4 * q + n) * a.dim + d[c]];
        back[n] = b.back[(slot * N + 4 * q + n) * a.dim + d[c]];
      }
    } else {
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (r.index == 0) {
        if (a.init != nullptr) load_states<4>(a.init + state, v);
      } else {
        fold_runs<4>(a, r.first, slot, d[c], A2[c], v, [&](int64_t s, int n) {
          return a.states[(s * N + 4 * q + n) * a.dim + d[c]];
        });
      }
      h = (f32x4){v[0], v[1], v[2], v[3]};
      if (b.dfinal != nullptr) back = *(const f32x4*)(b.dfinal + state);
      for (int64_t s = r.first + r.count - 1; s > slot; --s) {
        const float total = a.totals[s * a.dim + d[c]];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          back[n] = __builtin_fmaf(exp2_hw(total * A2[c][n]), back[n],
                                   b.back[(s * N + 4 * q + n) * a.dim + d[c]]);
      }
    }
    start[wave][c][lane] = on[c] ? h : (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < 4; ++n) R[c][n] = on[c] ? back[n] : 0.0f;
    bias[c] = a.in.dt_bias ? a.in.dt_bias[d[c]] : 0.0f;
    skip[c] = a.in.D ? a.in.D[d[c]] : 0.0f;
  }

  constexpr bool paired = PAIRED;
  const bool gated = a.in.z != nullptr;
  const uint32_t place = (uint32_t)(d[0] - base) * el, apart = (uint32_t)(d[1] - d[0]) * el;
  const char* x_row = (const char*)a.in.x + base * el;
  const char* dt_row = (const char*)a.in.dt + base * el;
  // (without a gate rows of x are read in the place of z's, and not used)
  const char* z_row = (const char*)(gated ? a.in.z : a.in.x) + base * el;
  const char* dy_row = (const char*)b.dy + base * el;
  const int64_t x_step = a.x_stride * el, dt_step = a.dt_stride * el;
  const int64_t z_step = (gated ? a.z_stride : a.x_stride) * el;
  const int64_t out_step = a.dim * el;
  const char* B_row = (const char*)a.in.B + (int64_t)group * N * el;
  const char* C_row = (const char*)a.in.C + (int64_t)group * N * el;
  const int64_t b_step = a.b_stride * el, c_step = a.c_stride * el;

  const int blocks = (int)((r.end - r.begin + kMark - 1) / kMark);
  const int64_t mark0 = first_mark(r, slot);
  float dD[2] = {0.0f, 0.0f}, dbias[2] = {0.0f, 0.0f};

  // Where the lane's own tokens of a block of `count` lie behind its first row (those
  // behind the last one read its row).
  struct Place {
    uint32_t x, dt, z, y;
  } own_at[OWN];
  auto put = [&](int count) {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int t = i * TURNS + q % TURNS;
      const uint32_t j = (uint32_t)(t < count ? t : count - 1);
      own_at[i] = {place + j * (uint32_t)x_step, place + j * (uint32_t)dt_step,
                   place + j * (uint32_t)z_step, place + j * (uint32_t)out_step};
    }
  };
  // what a block reads: its tokens' rows, B and C, and the state at its start
  struct Own {
    Pair<BF16> x, raw, z, g;
  } next[OWN];
  constexpr int kBC = (2 * N * kMark + kWave * kWaves - 1) / (kWave * kWaves);
  float bc[kBC];      // values of B and C a thread
  float mark[2][4], mark_total[2];
  const uint32_t mark_at[2] = {(uint32_t)(d[0] - base) * 4, (uint32_t)(d[1] - base) * 4};
  const uint32_t mark_row = (uint32_t)(4 * q) * (uint32_t)a.dim * 4;
  auto load = [&](int m) {
    const int64_t t0 = r.begin + (int64_t)m * kMark;
    const int count = r.end - t0 < kMark ? (int)(r.end - t0) : kMark;
    const rsrc_t xr = row_rsrc(x_row + t0 * x_step), dtr = row_rsrc(dt_row + t0 * dt_step);
    const rsrc_t zr = row_rsrc(z_row + t0 * z_step), yr = row_rsrc(dy_row + t0 * out_step);
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      next[i].x.load(xr, own_at[i].x, apart, paired);
      next[i].raw.load(dtr, own_at[i].dt, apart, paired);
      next[i].z.load(zr, own_at[i].z, apart, paired);
      next[i].g.load(yr, own_at[i].y, apart, paired);
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int v = (int)threadIdx.x + i * kWave * kWaves;
      const int j = v / (2 * N), k = v % N;
      bc[i] = 0.0f;
      if (j < count)
        bc[i] = v % (2 * N) < N ? load_one<BF16>(B_row + (t0 + j) * b_step, k)
                                : load_one<BF16>(C_row + (t0 + j) * c_step, k);
    }
    if (m > 0) {
      const char* p = (const char*)(b.marks + (mark0 + m) * N * a.dim + base);
      const rsrc_t total = row_rsrc(b.mark_totals + (mark0 + m) * a.dim + base);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mark_total[c] = load_f32(total, mark_at[c]);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          mark[c][n] = load_f32(row_rsrc(p + n * (int64_t)a.dim * 4), mark_at[c] + mark_row);
      }
    }
  };
  auto stage = [&](int turn) {
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int v = (int)threadIdx.x + i * kWave * kWaves;
      if (v < 2 * N * kMark) ((float*)bc_in[turn])[v] = bc[i];
    }
  };

  put((int)(r.end - r.begin) - (blocks - 1) * kMark);
  load(blocks - 1);
  stage(0);
  put(kMark);
  __syncthreads();
  int turn = 0;
  for (int m = blocks - 1; m >= 0; --m, turn ^= 1) {
    const int64_t t0 = r.begin + (int64_t)m * kMark;
    const int count = r.end - t0 < kMark ? (int)(r.end - t0) : kMark;
    // the time steps and gradients of the lane's own tokens
    Own own[OWN];
    float delta[OWN][2], dx[OWN][2], du[OWN][2];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      own[i] = next[i];
      // what is past the run's end, or the group's, has neither time nor input nor gradient:
      // nothing branches on it
      const bool there = i * TURNS + q % TURNS < count;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float v = own[i].raw.get(c) + bias[c], z = own[i].z.get(c), dy = own[i].g.get(c);
        delta[i][c] = pick(there, pick(a.softplus, softplus_f(v), v), 0.0f);
        dx[i][c] = pick(there & on[c], delta[i][c] * own[i].x.get(c), 0.0f);
        du[i][c] = pick(there & on[c], pick(gated, dy * (z * sigmoid_f(z)), dy), 0.0f);
      }
    }
    float h[kMark + 1][2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const f32x4 s = start[wave][c][lane];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        h[0][c][n] = s[n];
        // (the first run's marks include the initial state)
        if (m > 0)
          h[0][c][n] = r.index == 0 ? mark[c][n]
                                    : __builtin_fmaf(exp2_hw(mark_total[c] * A2[c][n]), s[n],
                                                     mark[c][n]);
        if (!on[c]) h[0][c][n] = 0.0f;
      }
    }
    // (tokens stay apart: work and reads of many at once would not fit the registers)
    auto fence = [] {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    // The decays of the last tokens wait in LDS, of four where their dB and dC will lie; those
    // of the first are formed again.
    auto up = [&](auto jj) {
      constexpr int j = decltype(jj)::value;
      const f32x4 B = bc_in[turn][j][0][q];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float dl = La::template bcast<j % TURNS>(delta[j / TURNS][c]);
        const float dxj = La::template bcast<j % TURNS>(dx[j / TURNS][c]);
        f32x4 decay;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          decay[n] = exp2_hw(dl * A2[c][n]);
          float v = __builtin_fmaf(decay[n], h[j][c][n], dxj * B[n]);
          asm volatile("" : "+v"(v));      // (formed here, not where it is used)
          h[j + 1][c][n] = v;
        }
        if constexpr (j >= kMark - kBatch)
          values[wave][j % kBatch][c][lane] = decay;
        else if constexpr (j >= kMark - kBatch - kMore)
          more[wave][j - (kMark - kBatch - kMore)][c][lane] = decay;
      }
      fence();
    };
    float inner[OWN][2], ddelta[OWN][2], u[OWN][2];
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) inner[i][c] = ddelta[i][c] = u[i][c] = 0.0f;
    auto down = [&](auto jj) {
      constexpr int j = decltype(jj)::value, i = j / TURNS;
      const f32x4 B = bc_in[turn][j][0][q], C = bc_in[turn][j][1][q];
      f32x4 vB, vC, decay[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if constexpr (j >= kMark - kBatch) {
          decay[c] = values[wave][j % kBatch][c][lane];
        } else if constexpr (j >= kMark - kBatch - kMore) {
          decay[c] = more[wave][j - (kMark - kBatch - kMore)][c][lane];
        } else {
          float dl = La::template bcast<j % TURNS>(delta[i][c]);
          asm volatile("" : "+v"(dl));     // (its products are formed again, not kept)
#pragma unroll
          for (int n = 0; n < 4; ++n) decay[c][n] = exp2_hw(dl * A2[c][n]);
        }
      }
      float in[2] = {0.0f, 0.0f}, dd[2] = {0.0f, 0.0f}, uu[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float dl = La::template bcast<j % TURNS>(delta[i][c]);
        const float dxj = La::template bcast<j % TURNS>(dx[i][c]);
        const float duj = La::template bcast<j % TURNS>(du[i][c]);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float dh = __builtin_fmaf(C[n], duj, R[c][n]);
          vC[n] = c ? __builtin_fmaf(duj, h[j + 1][c][n], vC[n]) : duj * h[j + 1][c][n];
          vB[n] = c ? __builtin_fmaf(dxj, dh, vB[n]) : dxj * dh;
          in[c] = __builtin_fmaf(B[n], dh, in[c]);
          uu[c] = __builtin_fmaf(C[n], h[j + 1][c][n], uu[c]);
          R[c][n] = dh * decay[c][n];
          const float kept = R[c][n] * h[j][c][n];
          dd[c] = __builtin_fmaf(kept, A2[c][n], dd[c]);
          dA[c][n] = __builtin_fmaf(kept, dl, dA[c][n]);
        }
      }
      float whole[6] = {in[0], dd[0], uu[0], in[1], dd[1], uu[1]};
      La::sum(whole);
      const bool own = q % TURNS == j % TURNS;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        inner[i][c] = pick(own, whole[3 * c], inner[i][c]);
        ddelta[i][c] = pick(own, whole[3 * c + 1], ddelta[i][c]);
        u[i][c] = pick(own, whole[3 * c + 2], u[i][c]);
      }
      values[wave][j % kBatch][0][lane] = vB;
      values[wave][j % kBatch][1][lane] = vC;
      fence();
    };
    // the lane's own tokens
    auto finish = [&](int i) {
      const int j = i * TURNS + q;
      if (q >= TURNS || j >= count) return;
      float vx[2], vdt[2], vz[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float x = own[i].x.get(c), v = own[i].raw.get(c) + bias[c];
        const float z = own[i].z.get(c), sig = sigmoid_f(z);
        const float ddt = __builtin_fmaf(ddelta[i][c], kLn2, inner[i][c] * x);
        vdt[c] = pick(a.softplus, ddt * sigmoid_f(v), ddt);
        dbias[c] += vdt[c];
        dD[c] = __builtin_fmaf(du[i][c], x, dD[c]);
        vx[c] = __builtin_fmaf(inner[i][c], delta[i][c], skip[c] * du[i][c]);
        vz[c] = own[i].g.get(c) * __builtin_fmaf(skip[c], x, u[i][c]) *
                (sig * __builtin_fmaf(z, 1.0f - sig, 1.0f));
      }
      const int64_t row = t0 * out_step + base * el;
      Pair<BF16>::store(row_rsrc((char*)b.out.dx + row), own_at[i].y, vx, on, paired);
      Pair<BF16>::store(row_rsrc((char*)b.out.ddt + row), own_at[i].y, vdt, on, paired);
      if (gated)
        Pair<BF16>::store(row_rsrc((char*)b.out.dz + row), own_at[i].y, vz, on, paired);
    };
    // The sums of a batch's dB and dC over the wave's pairs: 8 L of them (token, half, lane
    // of the pair), of kPairs vectors each, are shared by the 64 lanes, eight vectors a lane.
    // `meanwhile` fills the wait for them.
    auto batch = [&](int j0, auto meanwhile) {
      constexpr int kTasks = 2 * kBatch * L;
      constexpr int kParts = kTasks < kWave ? kWave / kTasks : 1;   // lanes of a sum
      constexpr int kRounds = kTasks > kWave ? kTasks / kWave : 1;
      constexpr int kEach = La::kPairs / kParts;
      wave_sync();
#pragma unroll
      for (int round = 0; round < kRounds; ++round) {
        const int part = lane % kParts, task = lane / kParts + round * kWave;
        const int k = task % L, half = task / L % 2, j = task / (2 * L);
        f32x4 v[kEach];
#pragma unroll
        for (int s = 0; s < kEach; ++s)
          // (spread over the banks)
          v[s] = values[wave][j][half][(part * kEach + (s + j) % kEach) * L + k];
        if (round == 0) meanwhile();
        f32x4 sum = v[0];
#pragma unroll
        for (int s = 1; s < kEach; ++s) sum += v[s];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (kParts >= 2) sum[e] += moved<kXor1>(sum[e]);
          if (kParts >= 4) sum[e] += moved<kXor2>(sum[e]);
        }
        if (part == 0) sums[turn][wave][j0 + j][half][k] = sum;
      }
      wave_sync();
    };
    up(std::integral_constant<int, 0>{});
    up(std::integral_constant<int, 1>{});
    up(std::integral_constant<int, 2>{});
    up(std::integral_constant<int, 3>{});
    up(std::integral_constant<int, 4>{});
    up(std::integral_constant<int, 5>{});
    up(std::integral_constant<int, 6>{});
    up(std::integral_constant<int, 7>{});
    down(std::integral_constant<int, 7>{});
    down(std::integral_constant<int, 6>{});
    down(std::integral_constant<int, 5>{});
    down(std::integral_constant<int, 4>{});
    // (tokens are finished, and the next block's rows asked for, where registers are free)
    batch(4, [&] {
#pragma unroll
      for (int i = OWN - 1; i >= 0; --i)
        if (i * TURNS >= kBatch) finish(i);
    });
    if (m > 0) load(m - 1);
    down(std::integral_constant<int, 3>{});
    down(std::integral_constant<int, 2>{});
    down(std::integral_constant<int, 1>{});
    down(std::integral_constant<int, 0>{});
    batch(0, [&] {
#pragma unroll
      for (int i = OWN - 1; i >= 0; --i)
        if (i * TURNS < kBatch) finish(i);
    });
    if (m > 0) stage(turn ^ 1);
    __syncthreads();
    // dB and dC of this block of channels
    for (int i = threadIdx.x; i < count * 2 * L; i += kWave * kWaves) {
      const int k = i % L, half = i / L % 2, j = i / (2 * L);
      f32x4 sum = sums[turn][0][j][half][k];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += sums[turn][w][j][half][k];
      const int64_t row = ((int64_t)block * a.runs.tokens + t0 + j) * a.ngroups + group;
      *(f32x4*)(b.bc_part + (row * 2 + half) * N + 4 * k) = sum;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float sD = La::sum(dD[c]), sb = La::sum(dbias[c]);
    if (!on[c]) continue;
#pragma unroll
    for (int n = 0; n < 4; ++n) dA_row[(4 * q + n) * a.dim + d[c]] = dA[c][n];
    if (q == 0) {
      dA_row[N * a.dim + d[c]] = sD;
      dA_row[(N + 1) * a.dim + d[c]] = sb;
    }
    if (r.index == 0 && b.out.dinit != nullptr)
      *(f32x4*)(b.out.dinit + ((int64_t)r.seq * a.dim + d[c]) * N + 4 * q) =
          (f32x4){R[c][0], R[c][1], R[c][2], R[c][3]};
  }
}

// dB and dC: the sums over the blocks of a group's channels.
template <bool BF16>
__global__ __launch_bounds__(256) void scan_sum_bc_kernel(const BwdArgs b, int n, int parts) {
  const ScanArgs& a = b.f;
  int64_t begin = 0, end = a.runs.tokens;
  if (a.runs.cu != nullptr) {      // rows outside every sequence are left as they are
    begin = seq_bound(a.runs, a.runs.cu[0]);
    end = seq_bound(a.runs, a.runs.cu[a.runs.nseq]);
  }
  const int64_t row = 2 * n * a.ngroups, all = (int64_t)a.runs.tokens * row;
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
#pragma unroll 8
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

template <int N, bool BF16>
void launch_n(const BwdArgs& b, int64_t blocks, int64_t wide, hipStream_t st) {
  constexpr int NS = N < 16 ? N : 16;
  hipLaunchKernelGGL((scan_local_kernel<N, NS, BF16>),
                     dim3((unsigned)(b.slots * blocks), N / NS), dim3(kWave), 0, st, b);
  if (b.f.joined) launch_scan_join(b.f, N, b.back, b.dfinal, st);
  const dim3 grid((unsigned)(b.slots * b.f.ngroups * wide)), threads(kWave * kWaves);
  if (b.f.paired)
    hipLaunchKernelGGL((scan_bwd_kernel<N, BF16, true>), grid, threads, 0, st, b);
  else
    hipLaunchKernelGGL((scan_bwd_kernel<N, BF16, false>), grid, threads, 0, st, b);
}

}  // namespace

int launch_scan_bwd(const ScanInputs& in, const float* init, const int32_t* cu, const void* dy,
                    const float* dfinal, const ScanGradients& out, void* ws, bool softplus,
                    bool bf16, const ScanShape& s, void* stream) {
  clear_launch_error();
  const BwdLayout l = bwd_layout(s);
  char* base = (char*)ws;
  BwdArgs b{};
  ScanArgs& a = b.f;
  a = make_scan_args(in, init, s, softplus);
  a.runs = scan_grid(cu, s, true);
  b.slots = run_slots(a.runs);
  a.joined = joins(a.runs);
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
  const int64_t blocks = channel_blocks(s), wide = wide_blocks(s);
  b.by_wide = Divide(wide);
  b.by_wide_slot = Divide(wide * s.ngroups);
  hipStream_t st = (hipStream_t)stream;
  switch (s.n) {
#define SSD_SCAN(N)                                  \
  case N:                                            \
    bf16 ? launch_n<N, true>(b, blocks, wide, st) : launch_n<N, false>(b, blocks, wide, st); \
    break
    SSD_SCAN(8);
    SSD_SCAN(16);
    SSD_SCAN(32);
    default:
      SSD_SCAN(64);
#undef SSD_SCAN
  }
  const int64_t values = s.tokens * s.ngroups * 2 * s.n;
  const dim3 grid((unsigned)((values + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL((scan_sum_bc_kernel<true>), grid, dim3(256), 0, st, b, (int)s.n, (int)wide);
  else
    hipLaunchKernelGGL((scan_sum_bc_kernel<false>), grid, dim3(256), 0, st, b, (int)s.n,
                       (int)wide);
  hipLaunchKernelGGL(scan_sum_slots_kernel,
                     dim3((unsigned)((s.dim + kWave - 1) / kWave * (s.n + 2))), dim3(256), 0, st,
                     b, (int)s.n);
  return (int)hipGetLastError();
}

}  // namespace ssd
