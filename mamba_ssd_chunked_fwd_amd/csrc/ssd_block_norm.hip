// The norms around a block: the residual add with a scale fused with the
// RMS norm in front of it, and the gated RMS norm behind its mixer, each with
// its gradients.  Per segment (a row, or a group of a row's channels) of n
// values, with r = 1/sqrt(mean(u^2) + eps) and nu = u r:
//   add norm    u = residual + s o x;  residual_out = u;  y = nu o w
//   gated norm  u = x o act(z), y = nu o w        (gate first)
//               u = x,          y = nu o w o act(z)
// and, with e the gradient of nu (dy o w, times act(z) where the gate comes
// last), the gradient of u is r (e - nu mean(e o nu)): the mean of e o nu is
// r mean(e o u), so one pass over the inputs gives both sums (u^2 and e u) and
// nothing is kept from the forward call.
//
// MI355X design.  Each call reads its inputs once and writes its outputs
// once: HBM-bound (gradients: up to 8192 channels, see below).  A team of TS lanes owns a
// segment: NV vectors of eight elements per lane stay in registers between the sums and
// the outputs (where the segment length is no multiple of 8 the vectors start at any
// element, and the last one overlaps the one before).  The sums of a team
// within a wave are lane exchanges; teams of several waves meet once in LDS.
// Teams are tied to a group of channels and walk the rows with the stride of
// the grid, so weights are loaded once per team, and the gradients of weights
// and scales are summed in registers: each workgroup writes one row of
// partial sums, and a second kernel adds those rows in a fixed order.
//
// Measured on MI355X (a device copy moves 5.1 TB/s): add norm of 8191 x 2560 with
// an fp32 stream, forward 44 us (252 MB: 5.7 TB/s), gradients 75 us (377 MB: 5.0) and
// 8 us for the row sums; gated norm of 16384 x 5120 by 64 channels 96 us (5.2);
// its gradients at 8192 x 1536 by rows, fp32 and bf16 mixed, 31 us (176 MB: 5.7) and
// 5 us for the row sums.
// Gradients of segments of more than 8192 channels are not HBM-bound: up to 16 waves of
// two vectors per lane leave 128 registers for eight (add norm) or seven (gated) arrays of
// 16 values, and 110 to 230 bytes per lane of them go through scratch for every row.  4096
// rows of bf16, with the row sums: add norm 8192 channels 96 us (4.2 TB/s of what it
// must move), 12287 398 (1.5), 12288 373 (1.6), 16384 355 (2.3); gated by whole rows 80
// (4.2), 282 (1.8), 263 (1.9) and 252 (2.7).
#include "ssd_block_launch.h"
#include "ssd_device.h"
#include "ssd_host.h"

#include <type_traits>

namespace ssd {
namespace {

constexpr int kNormThreads = 256;
constexpr int kVec = 8;                // elements of a lane's vector
// Waves of a launch: 16 per CU (measured against 8, 12 and 32: with 8 the forward
// calls lose up to 40%, with 32 the gradients' calls 10%).
constexpr int kNormWaves = 4096;

// The eight elements at element offset `i`, as floats, and back (rounded once).
// ENDS: kWhole: the segment length is a multiple of 8, and so is every offset;
// kRagged: it is not, so a vector may start at any element; kShort: a segment may also
// have fewer than eight (zeros stand for the rest).  That form goes to the smallest
// teams alone: its branches for each element cost the widest ones, which have the
// fewest registers to spare, up to 1650 bytes of scratch per lane.
constexpr int kWhole = 0, kRagged = 1, kShort = 2;
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <bool BF16, int ENDS>
__device__ __forceinline__ void load_n(const void* p, int64_t i, int left, float* v) {
  if (ENDS == kShort && left < kVec) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      v[e] = 0.0f;
      if (e < left)
        v[e] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i + e] << 16)
                    : ((const float*)p)[i + e];
    }
  } else if constexpr (BF16) {
    const uint16_t* q = (const uint16_t*)p + i;
    const u32x4 u = ENDS ? (u32x4) * (const u32x4_any*)q : *(const u32x4*)q;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_lo(u[k]);
      v[2 * k + 1] = bf16_hi(u[k]);
    }
  } else {
    const float* q = (const float*)p + i;
    const f32x4 a = ENDS ? (f32x4) * (const f32x4_any*)q : *(const f32x4*)q;
    const f32x4 b = ENDS ? (f32x4) * (const f32x4_any*)(q + 4) : *(const f32x4*)(q + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  }
}
template <bool BF16, int ENDS>
__device__ __forceinline__ void store_n(void* p, int64_t i, int left, const float* v) {
  if (ENDS == kShort && left < kVec) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (e < left) {
        if constexpr (BF16)
          ((uint16_t*)p)[i + e] = (uint16_t)(pack_bf16(v[e], 0.0f) & 0xFFFFu);
        else
          ((float*)p)[i + e] = v[e];
      }
    }
  } else if constexpr (BF16) {
    const u32x4 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7])};
    uint16_t* q = (uint16_t*)p + i;
    if constexpr (ENDS != kWhole)
      *(u32x4_any*)q = u;
    else
      *(u32x4*)q = u;
  } else {
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    float* q = (float*)p + i;
    if constexpr (ENDS != kWhole) {
      *(f32x4_any*)q = a;
      *(f32x4_any*)(q + 4) = b;
    } else {
      *(f32x4*)q = a;
      *(f32x4*)(q + 4) = b;
    }
  }
}

// The lanes of a team: TS of a wave, or (TS = kBlockTeam) the whole workgroup, of
// as many waves as the launch gives it.
constexpr int kBlockTeam = 0;
constexpr int kMaxWaves = 16;
template <int TS>
constexpr int max_threads() { return TS == kBlockTeam ? kMaxWaves * kWave : kNormThreads; }
template <int TS>
__device__ __forceinline__ int team_lanes() { return TS == kBlockTeam ? (int)blockDim.x : TS; }

// Sums of K values over the lanes of a team.  Teams of a workgroup alternate
// between two LDS rows, so one barrier per call is enough: a row is written again
// only after the next call's barrier.
template <int TS, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float (*red)[kMaxWaves][2], int& turn) {
  constexpr int W = TS == kBlockTeam || TS > kWave ? kWave : TS;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], off, kWave);
  }
  if constexpr (TS == kBlockTeam || TS > kWave) {
    const int waves = team_lanes<TS>() / kWave;
    if (threadIdx.x % kWave == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[turn][threadIdx.x / kWave][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = red[turn][0][k];
      for (int i = 1; i < waves; ++i) v[k] += red[turn][i][k];
    }
    turn ^= 1;
  }
}

// Where a team works: its group of channels, its first row and its stride.
struct NormGrid {
  int64_t rows, dim;
  int n;             // channels of a segment
  int groups;        // segments of a row
  int per_block;     // groups of a workgroup's teams (a power of two)
  int shared;        // one set of weights for every group
  float inv_n, eps;
};

template <int TS>
struct Team {
  static constexpr int kTeams = TS == kBlockTeam ? 1 : kNormThreads / (TS ? TS : 1);
  int lane, group, rows_per_block;
  int64_t row, step;
  bool on;
  __device__ __forceinline__ explicit Team(const NormGrid& g) {
    const int team = threadIdx.x / team_lanes<TS>();
    lane = threadIdx.x % team_lanes<TS>();
    group = blockIdx.y * g.per_block + team % g.per_block;
    rows_per_block = kTeams / g.per_block;
    row = (int64_t)blockIdx.x * rows_per_block + team / g.per_block;
    step = (int64_t)gridDim.x * rows_per_block;
    on = group < g.groups;
  }
};

// A lane's vector of a segment of n elements.  In a ragged segment the last vector
// ends with the segment and shares its first `skip` elements with the one before:
// both lanes form and store the same values there, and only one adds them to the
// segment's sums.  (A segment of less than eight elements is one short vector.)
template <int ENDS>
struct Span {
  int c, skip;
  bool on;
  __device__ __forceinline__ Span(int vec, int n) : c(vec * kVec), skip(0), on(vec * kVec < n) {
    if (ENDS != kWhole && n >= kVec && c + kVec > n) {
      skip = c - (n - kVec);
      c = n - kVec;
    }
  }
  __device__ __forceinline__ bool counts(int e) const { return ENDS == kWhole || e >= skip; }
};

template <int NV, int ENDS, int TS>
__device__ __forceinline__ void load_weights(const float* p, const NormGrid& g, const Team<TS>& t,
                                             bool shared, float other, float* w) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
    const int c = sp.c;
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[j * kVec + e] = other;
    if (p != nullptr && t.on && sp.on)
      load_n<false, ENDS>(p, (shared ? 0 : (int64_t)t.group * g.n) + c, g.n - c, w + j * kVec);
  }
}

// One row of partial sums of this workgroup: over its teams of one group, or
// of every group where the weights are shared.
template <int TS, int NV, int ENDS>
__device__ __forceinline__ void store_partial(const float* acc, float* part, const NormGrid& g,
                                              const Team<TS>& t, float* buf) {
  constexpr int kTeams = Team<TS>::kTeams;
  const int team = threadIdx.x / team_lanes<TS>();
  const int span = g.shared ? kTeams : t.rows_per_block;       // teams added up
  const int step = g.shared ? 1 : g.per_block;
  const bool writes = g.shared ? team == 0 : (team < g.per_block && t.on);
  float* row = g.shared ? part + ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * g.n
                        : part + (int64_t)blockIdx.x * g.dim + (int64_t)t.group * g.n;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = acc[j * kVec + e];
    if constexpr (kTeams > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kVec; ++e) buf[e * kNormThreads + threadIdx.x] = v[e];
      __syncthreads();
      if (writes) {
        for (int k = 1; k < span; ++k) {
#pragma unroll
          for (int e = 0; e < kVec; ++e)
            v[e] += buf[e * kNormThreads + threadIdx.x + k * step * TS];
        }
      }
    }
    const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
    const int c = sp.c;
    if (writes && sp.on) store_n<false, ENDS>(row, c, g.n - c, v);
  }
}

// ---------------------------------------------------------------- add norm
template <int TS, int NV, int ENDS, bool XB, bool RB>
__global__ __launch_bounds__(max_threads<TS>()) void add_norm_fwd_kernel(
    const void* x, const void* res, const float* __restrict__ scale,
    const float* __restrict__ weight, void* y, void* res_out, NormGrid g) {
  __shared__ float red[2][kMaxWaves][2];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * kVec], s[NV * kVec];
  load_weights<NV, ENDS, TS>(weight, g, t, false, 1.0f, w);
  load_weights<NV, ENDS, TS>(scale, g, t, false, 1.0f, s);
  for (int64_t row = t.row; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim;
    float h[NV * kVec], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      float xv[kVec] = {}, rv[kVec] = {};
      if (sp.on) {
        load_n<XB, ENDS>(x, base + c, g.n - c, xv);
        if (res) load_n<RB, ENDS>(res, base + c, g.n - c, rv);
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        h[j * kVec + e] = __builtin_fmaf(s[j * kVec + e], xv[e], rv[e]);
        if (sp.counts(e)) sum[0] = __builtin_fmaf(h[j * kVec + e], h[j * kVec + e], sum[0]);
      }
    }
    team_sum<TS, 1>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      if (sp.on) {
        float v[kVec];
        if (res_out) store_n<RB, ENDS>(res_out, base + c, g.n - c, h + j * kVec);
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = h[j * kVec + e] * r * w[j * kVec + e];
        store_n<XB, ENDS>(y, base + c, g.n - c, v);
      }
    }
  }
}

template <int TS, int NV, int ENDS, bool XB, bool RB>
__global__ __launch_bounds__(max_threads<TS>()) void add_norm_bwd_kernel(
    const void* x, const void* res, const float* __restrict__ scale,
    const float* __restrict__ weight, const void* dy, const void* dres_out, void* dx, void* dres,
    float* __restrict__ dscale, float* __restrict__ dweight, NormGrid g) {
  __shared__ float red[2][kMaxWaves][2];
  __shared__ float buf[Team<TS>::kTeams > 1 ? kVec * kNormThreads : 1];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * kVec], s[NV * kVec], dw[NV * kVec] = {}, ds[NV * kVec] = {};
  load_weights<NV, ENDS, TS>(weight, g, t, false, 1.0f, w);
  load_weights<NV, ENDS, TS>(scale, g, t, false, 1.0f, s);
  for (int64_t row = t.row; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim;
    float h[NV * kVec], xs[NV * kVec], dv[NV * kVec], gv[NV * kVec], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      float rv[kVec] = {};
#pragma unroll
      for (int e = 0; e < kVec; ++e) xs[j * kVec + e] = dv[j * kVec + e] = gv[j * kVec + e] = 0.0f;
      if (sp.on) {
        load_n<XB, ENDS>(x, base + c, g.n - c, xs + j * kVec);
        load_n<XB, ENDS>(dy, base + c, g.n - c, dv + j * kVec);
        if (res) load_n<RB, ENDS>(res, base + c, g.n - c, rv);
        if (dres_out) load_n<RB, ENDS>(dres_out, base + c, g.n - c, gv + j * kVec);
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int i = j * kVec + e;
        h[i] = __builtin_fmaf(s[i], xs[i], rv[e]);
        if (sp.counts(e)) {
          sum[0] = __builtin_fmaf(h[i], h[i], sum[0]);
          sum[1] = __builtin_fmaf(w[i] * dv[i], h[i], sum[1]);
        }
      }
    }
    team_sum<TS, 2>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
    const float m = sum[1] * g.inv_n * r;              // mean(w dy n)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      float dxv[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int i = j * kVec + e;
        const float n = h[i] * r;
        gv[i] = __builtin_fmaf(r, __builtin_fmaf(-n, m, w[i] * dv[i]), gv[i]);
        dxv[e] = s[i] * gv[i];
        dw[i] = __builtin_fmaf(dv[i], n, dw[i]);
        ds[i] = __builtin_fmaf(gv[i], xs[i], ds[i]);
      }
      if (sp.on) {
        if (dres) store_n<RB, ENDS>(dres, base + c, g.n - c, gv + j * kVec);
        store_n<XB, ENDS>(dx, base + c, g.n - c, dxv);
      }
    }
  }
  if (dweight) store_partial<TS, NV, ENDS>(dw, dweight, g, t, buf);
  if (dscale) store_partial<TS, NV, ENDS>(ds, dscale, g, t, buf);
}

// -------------------------------------------------------------- gated norm
// act(z) and its derivative.  sigmoid(z) and 1 - sigmoid(z) both come from
// e^{-|z|}, so neither cancels or overflows far out.
__device__ __forceinline__ float gate_act(float z, bool silu, float& d) {
  const float e = exp2_hw(-kLog2e * fabsf(z));
  const float p = __builtin_amdgcn_rcpf(1.0f + e), q = e * p;
  const float sig = z >= 0.0f ? p : q;
  const float ds = p * q;
  d = silu ? __builtin_fmaf(z, ds, sig) : ds;
  return silu ? z * sig : sig;
}

// Waves per SIMD asked for: with five, rows of up to 12288 channels, 12 waves to a row, have
// one workgroup to a CU in place of two (12287 channels of bf16: 96 us in place of 81).
template <int TS, int NV>
constexpr int gate_waves() { return TS == kBlockTeam && NV == 2 ? 6 : 1; }

template <int TS, int NV, int ENDS, bool XB, bool ZB>
__global__ __launch_bounds__(max_threads<TS>(), (gate_waves<TS, NV>())) void gated_norm_fwd_kernel(
    const void* x, const void* z, const float* __restrict__ weight, void* y, bool silu,
    bool first, NormGrid g) {
  __shared__ float red[2][kMaxWaves][2];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * kVec];
  load_weights<NV, ENDS, TS>(weight, g, t, g.shared, 1.0f, w);
  if (!t.on) return;            // whole teams; one of a workgroup is always on
  for (int64_t row = t.row; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim + (int64_t)t.group * g.n;
    float u[NV * kVec], a[NV * kVec], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      float xv[kVec] = {}, zv[kVec] = {}, d;
      if (sp.on) {
        load_n<XB, ENDS>(x, base + c, g.n - c, xv);
        if (z) load_n<ZB, ENDS>(z, base + c, g.n - c, zv);
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int i = j * kVec + e;
        const float act = z ? gate_act(zv[e], silu, d) : 1.0f;
        u[i] = first ? xv[e] * act : xv[e];
        a[i] = first ? 1.0f : act;
        if (sp.counts(e)) sum[0] = __builtin_fmaf(u[i], u[i], sum[0]);
      }
    }
    team_sum<TS, 1>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      if (sp.on) {
        float v[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          v[e] = u[j * kVec + e] * r * w[j * kVec + e] * a[j * kVec + e];
        store_n<ZB, ENDS>(y, base + c, g.n - c, v);
      }
    }
  }
}

template <int TS, int NV, int ENDS, bool XB, bool ZB>
__global__ __launch_bounds__(max_threads<TS>()) void gated_norm_bwd_kernel(
    const void* x, const void* z, const float* __restrict__ weight, const void* dy, void* dx,
    void* dz, float* __restrict__ dweight, bool silu, bool first, NormGrid g) {
  __shared__ float red[2][kMaxWaves][2];
  __shared__ float buf[Team<TS>::kTeams > 1 ? kVec * kNormThreads : 1];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * kVec], dw[NV * kVec] = {};
  load_weights<NV, ENDS, TS>(weight, g, t, g.shared, 1.0f, w);
  for (int64_t row = t.on ? t.row : g.rows; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim + (int64_t)t.group * g.n;
    float xs[NV * kVec], act[NV * kVec], der[NV * kVec], dv[NV * kVec], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      float zv[kVec] = {};
#pragma unroll
      for (int e = 0; e < kVec; ++e) xs[j * kVec + e] = dv[j * kVec + e] = 0.0f;
      if (sp.on) {
        load_n<XB, ENDS>(x, base + c, g.n - c, xs + j * kVec);
        load_n<ZB, ENDS>(dy, base + c, g.n - c, dv + j * kVec);
        if (z) load_n<ZB, ENDS>(z, base + c, g.n - c, zv);
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int i = j * kVec + e;
        der[i] = 0.0f;
        act[i] = z ? gate_act(zv[e], silu, der[i]) : 1.0f;
        const float u = first ? xs[i] * act[i] : xs[i];
        const float en = dv[i] * w[i] * (first ? 1.0f : act[i]);
        if (sp.counts(e)) {
          sum[0] = __builtin_fmaf(u, u, sum[0]);
          sum[1] = __builtin_fmaf(en, u, sum[1]);
        }
      }
    }
    team_sum<TS, 2>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
    const float m = sum[1] * g.inv_n * r;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Span<ENDS> sp(t.lane + team_lanes<TS>() * j, g.n);
      const int c = sp.c;
      float dxv[kVec], dzv[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int i = j * kVec + e;
        const float n = (first ? xs[i] * act[i] : xs[i]) * r;
        const float dn = first ? dv[i] : dv[i] * act[i];
        const float du = r * __builtin_fmaf(-n, m, dn * w[i]);
        dxv[e] = first ? du * act[i] : du;
        dzv[e] = (first ? du * xs[i] : dv[i] * n * w[i]) * der[i];
        dw[i] = __builtin_fmaf(dn, n, dw[i]);
      }
      if (sp.on) {
        store_n<XB, ENDS>(dx, base + c, g.n - c, dxv);
        if (z) store_n<ZB, ENDS>(dz, base + c, g.n - c, dzv);
      }
    }
  }
  if (dweight) store_partial<TS, NV, ENDS>(dw, dweight, g, t, buf);
}

// Adds `parts` rows of `cols` partial sums in a fixed order: 16 slices of the
// rows, each added in turn, then the slices in order.  blockIdx.y: which of two
// sums.
__global__ __launch_bounds__(1024) void sum_rows_kernel(const float* __restrict__ part0,
                                                        float* __restrict__ out0,
                                                        const float* __restrict__ part1,
                                                        float* __restrict__ out1, int parts,
                                                        int cols) {
  const float* part = blockIdx.y ? part1 : part0;
  float* out = blockIdx.y ? out1 : out0;
  __shared__ float buf[16][kWave];
  const int lane = threadIdx.x % kWave, slice = threadIdx.x / kWave;
  const int c = blockIdx.x * kWave + lane;
  float acc = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = slice; p < parts; p += 16) acc += part[(int64_t)p * cols + c];
  }
  buf[slice][lane] = acc;
  __syncthreads();
  if (slice == 0 && c < cols) {
    for (int k = 1; k < 16; ++k) acc += buf[k][lane];
    out[c] = acc;
  }
}

// ---------------------------------------------------------------- launches
struct NormLaunch {
  NormGrid g;
  dim3 grid;
  int threads;
  int parts;      // rows of partial sums
  int cols;
};

// The lanes of a team: enough for one vector each up to a wave, then two vectors
// per lane of a wave, one or two per lane of four waves, and from there on as many
// waves as the segment has vectors for one, then two, per lane.  (Measured for the
// gradients' call: at 5000 channels ten waves of one vector take 50 us where four
// of four took 76; at 2560 five waves of one take 55 us where four of two, of which
// every third lane idles, take 49.)
struct TeamPlan {
  int ts, nv, threads;
};
TeamPlan team_plan(int64_t n) {
  const int64_t u = (n + kVec - 1) / kVec;
  if (u <= 8) return {8, 1, kNormThreads};
  if (u <= 16) return {16, 1, kNormThreads};
  if (u <= 32) return {32, 1, kNormThreads};
  if (u <= 64) return {64, 1, kNormThreads};
  if (u <= 128) return {64, 2, kNormThreads};
  if (u <= 256) return {256, 1, 256};
  if (u <= 512) return {256, 2, 256};
  const int nv = u <= kMaxWaves * kWave ? 1 : 2;
  return {kBlockTeam, nv, (int)((u + nv * kWave - 1) / (nv * kWave)) * kWave};
}

NormLaunch norm_launch(const NormShape& s, float eps) {
  NormLaunch l;
  const TeamPlan plan = team_plan(s.group);
  const int teams = plan.ts == kBlockTeam ? 1 : kNormThreads / plan.ts;
  const int64_t groups = s.dim / s.group;
  int per = 1;
  while (per < teams && per < groups) per *= 2;
  const int64_t gy = (groups + per - 1) / per;
  const int64_t rows_per = teams / per;
  int64_t gx = (s.rows + rows_per - 1) / rows_per;
  const int64_t all = (int64_t)kNormWaves * kWave / plan.threads;
  const int64_t want = (all + gy - 1) / gy;
  if (gx > want) gx = want;
  l.g = NormGrid{s.rows,     s.dim, (int)s.group, (int)groups, per, s.wdim != s.dim,
                 1.0f / (float)s.group, eps};
  l.grid = dim3((unsigned)gx, (unsigned)gy);
  l.threads = plan.threads;
  l.parts = (int)(l.g.shared ? gx * gy : gx);
  l.cols = (int)s.wdim;
  return l;
}

// f(TeamPlan constants, ends) for the plan of a segment of n channels.
template <class F>
void with_plan(int64_t n, F f) {
  const TeamPlan p = team_plan(n);
#define SSD_NORM_PLAN(TS, NV)                                                          \
  if (p.ts == TS && p.nv == NV) {                                                      \
    if (n % kVec)                                                                      \
      return f(std::integral_constant<int, TS>{}, std::integral_constant<int, NV>{},   \
               std::integral_constant<int, TS == 8 ? kShort : kRagged>{});             \
    return f(std::integral_constant<int, TS>{}, std::integral_constant<int, NV>{},     \
             std::integral_constant<int, kWhole>{});                                   \
  }
  SSD_NORM_PLAN(8, 1)
  SSD_NORM_PLAN(16, 1)
  SSD_NORM_PLAN(32, 1)
  SSD_NORM_PLAN(64, 1)
  SSD_NORM_PLAN(64, 2)
  SSD_NORM_PLAN(256, 1)
  SSD_NORM_PLAN(256, 2)
  SSD_NORM_PLAN(kBlockTeam, 1)
  SSD_NORM_PLAN(kBlockTeam, 2)
#undef SSD_NORM_PLAN
}
template <class F>
void with_bool(bool b, F f) {
  if (b) return f(std::true_type{});
  f(std::false_type{});
}

// The sums whose outputs are asked for, in one launch.
int add_rows(const float* p0, float* o0, const float* p1, float* o1, const NormLaunch& l,
             hipStream_t st) {
  if (o0 == nullptr) {
    p0 = p1;
    o0 = o1;
    o1 = nullptr;
  }
  if (o0 == nullptr) return 0;
  const dim3 grid((unsigned)((l.cols + kWave - 1) / kWave), o1 != nullptr ? 2u : 1u);
  hipLaunchKernelGGL(sum_rows_kernel, grid, dim3(1024), 0, st, p0, o0, p1, o1, l.parts, l.cols);
  return (int)hipGetLastError();
}

}  // namespace

size_t norm_bwd_workspace(const NormShape& s, int sums) {
  const NormLaunch l = norm_launch(s, 1.0f);
  const size_t one = ((size_t)l.parts * (size_t)l.cols * sizeof(float) + 15) / 16 * 16;
  return one * (size_t)sums;
}

int launch_add_norm_fwd(const void* x, const void* res, const float* scale, const float* weight,
                        void* y, void* res_out, float eps, bool xbf16, bool rbf16,
                        const NormShape& s, void* stream) {
  clear_launch_error();
  const NormLaunch l = norm_launch(s, eps);
  with_plan(s.group, [&](auto ts, auto nv, auto ends) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(rbf16, [&](auto rb) {
        hipLaunchKernelGGL((add_norm_fwd_kernel<ts(), nv(), ends(), xb(), rb()>), l.grid,
                           dim3((unsigned)l.threads), 0, (hipStream_t)stream, x, res, scale,
                           weight, y, res_out, l.g);
      });
    });
  });
  return (int)hipGetLastError();
}

int launch_add_norm_bwd(const void* x, const void* res, const float* scale, const float* weight,
                        const void* dy, const void* dres_out, void* dx, void* dres,
                        float* dscale, float* dweight, void* ws, float eps, bool xbf16,
                        bool rbf16, const NormShape& s, void* stream) {
  clear_launch_error();
  const NormLaunch l = norm_launch(s, eps);
  float* pw = dweight ? (float*)ws : nullptr;
  float* ps = dscale ? (float*)((char*)ws + norm_bwd_workspace(s, 1)) : nullptr;
  with_plan(s.group, [&](auto ts, auto nv, auto ends) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(rbf16, [&](auto rb) {
        hipLaunchKernelGGL((add_norm_bwd_kernel<ts(), nv(), ends(), xb(), rb()>), l.grid,
                           dim3((unsigned)l.threads), 0, (hipStream_t)stream, x, res, scale,
                           weight, dy, dres_out, dx, dres, ps, pw, l.g);
      });
    });
  });
  const int err = (int)hipGetLastError();
  return err ? err : add_rows(pw, dweight, ps, dscale, l, (hipStream_t)stream);
}

int launch_gated_norm_fwd(const void* x, const void* z, const float* weight, void* y, float eps,
                          bool silu, bool first, bool xbf16, bool zbf16, const NormShape& s,
                          void* stream) {
  clear_launch_error();
  const NormLaunch l = norm_launch(s, eps);
  with_plan(s.group, [&](auto ts, auto nv, auto ends) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(zbf16, [&](auto zb) {
        hipLaunchKernelGGL((gated_norm_fwd_kernel<ts(), nv(), ends(), xb(), zb()>), l.grid,
                           dim3((unsigned)l.threads), 0, (hipStream_t)stream, x, z, weight, y, silu,
                           first, l.g);
      });
    });
  });
  return (int)hipGetLastError();
}

int launch_gated_norm_bwd(const void* x, const void* z, const float* weight, const void* dy,
                          void* dx, void* dz, float* dweight, void* ws, float eps, bool silu,
                          bool first, bool xbf16, bool zbf16, const NormShape& s, void* stream) {
  clear_launch_error();
  const NormLaunch l = norm_launch(s, eps);
  float* pw = dweight ? (float*)ws : nullptr;
  with_plan(s.group, [&](auto ts, auto nv, auto ends) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(zbf16, [&](auto zb) {
        hipLaunchKernelGGL((gated_norm_bwd_kernel<ts(), nv(), ends(), xb(), zb()>), l.grid,
                           dim3((unsigned)l.threads), 0, (hipStream_t)stream, x, z, weight, dy,
                           dx, dz, pw, silu, first, l.g);
      });
    });
  });
  const int err = (int)hipGetLastError();
  return err ? err : add_rows(pw, dweight, nullptr, nullptr, l, (hipStream_t)stream);
}

}  // namespace ssd
