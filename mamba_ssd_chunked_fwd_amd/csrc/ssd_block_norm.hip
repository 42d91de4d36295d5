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
// once: HBM-bound.  A team of TS lanes owns a segment: NV vectors of VE
// elements per lane stay in registers between the sums and the outputs
// (VE = 8, 16-byte loads, where the segment length is a multiple of 8; single
// elements otherwise, whose rows are not 16-byte aligned).  The sums of a team
// within a wave are lane exchanges; teams of four waves meet once in LDS.
// Teams are tied to a group of channels and walk the rows with the stride of
// the grid, so weights are loaded once per team, and the gradients of weights
// and scales are summed in registers: each workgroup writes one row of
// partial sums, and a second kernel adds those rows in a fixed order.
#include "ssd_block_launch.h"
#include "ssd_device.h"
#include "ssd_host.h"

#include <type_traits>

namespace ssd {
namespace {

constexpr int kNormThreads = 256;
// Workgroups of a launch: four per CU (measured against two and eight).
constexpr int kNormBlocks = 1024;

// VE elements at element offset `i`, as floats, and back (rounded once).
template <bool BF16, int VE>
__device__ __forceinline__ void load_n(const void* p, int64_t i, float* v) {
  if constexpr (VE == 1) {
    if constexpr (BF16)
      v[0] = __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
    else
      v[0] = ((const float*)p)[i];
  } else if constexpr (BF16) {
    const u32x4 u = *(const u32x4*)((const uint16_t*)p + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_lo(u[k]);
      v[2 * k + 1] = bf16_hi(u[k]);
    }
  } else {
    const f32x4 a = *(const f32x4*)((const float*)p + i);
    const f32x4 b = *(const f32x4*)((const float*)p + i + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  }
}
template <bool BF16, int VE>
__device__ __forceinline__ void store_n(void* p, int64_t i, const float* v) {
  if constexpr (VE == 1) {
    if constexpr (BF16)
      ((uint16_t*)p)[i] = (uint16_t)(pack_bf16(v[0], 0.0f) & 0xFFFFu);
    else
      ((float*)p)[i] = v[0];
  } else if constexpr (BF16) {
    *(u32x4*)((uint16_t*)p + i) = (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                          pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  } else {
    *(f32x4*)((float*)p + i) = (f32x4){v[0], v[1], v[2], v[3]};
    *(f32x4*)((float*)p + i + 4) = (f32x4){v[4], v[5], v[6], v[7]};
  }
}

// Sums of K values over the TS lanes of a team.  Teams of one workgroup
// (TS = 256) alternate between two LDS rows, so one barrier per call is
// enough: a row is written again only after the next call's barrier.
template <int TS, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float (*red)[4][2], int& turn) {
  constexpr int W = TS < kWave ? TS : kWave;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], off, kWave);
  }
  if constexpr (TS > kWave) {
    const int wave = threadIdx.x / kWave;
    if (threadIdx.x % kWave == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[turn][wave][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      v[k] = (red[turn][0][k] + red[turn][1][k]) + (red[turn][2][k] + red[turn][3][k]);
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
  static constexpr int kTeams = kNormThreads / TS;
  int lane, group, rows_per_block;
  int64_t row, step;
  bool on;
  __device__ __forceinline__ explicit Team(const NormGrid& g) {
    const int team = threadIdx.x / TS;
    lane = threadIdx.x % TS;
    group = blockIdx.y * g.per_block + team % g.per_block;
    rows_per_block = kTeams / g.per_block;
    row = (int64_t)blockIdx.x * rows_per_block + team / g.per_block;
    step = (int64_t)gridDim.x * rows_per_block;
    on = group < g.groups;
  }
};

template <int NV, int VE, int TS>
__device__ __forceinline__ void load_weights(const float* p, const NormGrid& g, const Team<TS>& t,
                                             bool shared, float other, float* w) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t.lane + TS * j) * VE;
#pragma unroll
    for (int e = 0; e < VE; ++e) w[j * VE + e] = other;
    if (p != nullptr && t.on && c < g.n)
      load_n<false, VE>(p, (shared ? 0 : (int64_t)t.group * g.n) + c, w + j * VE);
  }
}

// One row of partial sums of this workgroup: over its teams of one group, or
// of every group where the weights are shared.
template <int TS, int NV, int VE>
__device__ __forceinline__ void store_partial(const float* acc, float* part, const NormGrid& g,
                                              const Team<TS>& t, float* buf) {
  constexpr int kTeams = Team<TS>::kTeams;
  const int team = threadIdx.x / TS;
  const int span = g.shared ? kTeams : t.rows_per_block;       // teams added up
  const int step = g.shared ? 1 : g.per_block;
  const bool writes = g.shared ? team == 0 : (team < g.per_block && t.on);
  float* row = g.shared ? part + ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * g.n
                        : part + (int64_t)blockIdx.x * g.dim + (int64_t)t.group * g.n;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = acc[j * VE + e];
    if constexpr (kTeams > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VE; ++e) buf[e * kNormThreads + threadIdx.x] = v[e];
      __syncthreads();
      if (writes) {
        for (int k = 1; k < span; ++k) {
#pragma unroll
          for (int e = 0; e < VE; ++e) v[e] += buf[e * kNormThreads + threadIdx.x + k * step * TS];
        }
      }
    }
    const int c = (t.lane + TS * j) * VE;
    if (writes && c < g.n) store_n<false, VE>(row, c, v);
  }
}

// ---------------------------------------------------------------- add norm
template <int TS, int NV, int VE, bool XB, bool RB>
__global__ __launch_bounds__(kNormThreads) void add_norm_fwd_kernel(
    const void* x, const void* res, const float* __restrict__ scale,
    const float* __restrict__ weight, void* y, void* res_out, NormGrid g) {
  __shared__ float red[2][4][2];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * VE], s[NV * VE];
  load_weights<NV, VE, TS>(weight, g, t, false, 1.0f, w);
  load_weights<NV, VE, TS>(scale, g, t, false, 1.0f, s);
  for (int64_t row = t.row; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim;
    float h[NV * VE], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      float xv[VE] = {}, rv[VE] = {};
      if (c < g.n) {
        load_n<XB, VE>(x, base + c, xv);
        if (res) load_n<RB, VE>(res, base + c, rv);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        h[j * VE + e] = __builtin_fmaf(s[j * VE + e], xv[e], rv[e]);
        sum[0] = __builtin_fmaf(h[j * VE + e], h[j * VE + e], sum[0]);
      }
    }
    team_sum<TS, 1>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      if (c < g.n) {
        float v[VE];
        if (res_out) store_n<RB, VE>(res_out, base + c, h + j * VE);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[e] = h[j * VE + e] * r * w[j * VE + e];
        store_n<XB, VE>(y, base + c, v);
      }
    }
  }
}

template <int TS, int NV, int VE, bool XB, bool RB>
__global__ __launch_bounds__(kNormThreads) void add_norm_bwd_kernel(
    const void* x, const void* res, const float* __restrict__ scale,
    const float* __restrict__ weight, const void* dy, const void* dres_out, void* dx, void* dres,
    float* __restrict__ dscale, float* __restrict__ dweight, NormGrid g) {
  __shared__ float red[2][4][2];
  __shared__ float buf[Team<TS>::kTeams > 1 ? VE * kNormThreads : 1];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * VE], s[NV * VE], dw[NV * VE] = {}, ds[NV * VE] = {};
  load_weights<NV, VE, TS>(weight, g, t, false, 1.0f, w);
  load_weights<NV, VE, TS>(scale, g, t, false, 1.0f, s);
  for (int64_t row = t.row; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim;
    float h[NV * VE], xs[NV * VE], dv[NV * VE], gv[NV * VE], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      float rv[VE] = {};
#pragma unroll
      for (int e = 0; e < VE; ++e) xs[j * VE + e] = dv[j * VE + e] = gv[j * VE + e] = 0.0f;
      if (c < g.n) {
        load_n<XB, VE>(x, base + c, xs + j * VE);
        load_n<XB, VE>(dy, base + c, dv + j * VE);
        if (res) load_n<RB, VE>(res, base + c, rv);
        if (dres_out) load_n<RB, VE>(dres_out, base + c, gv + j * VE);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = j * VE + e;
        h[i] = __builtin_fmaf(s[i], xs[i], rv[e]);
        sum[0] = __builtin_fmaf(h[i], h[i], sum[0]);
        sum[1] = __builtin_fmaf(w[i] * dv[i], h[i], sum[1]);
      }
    }
    team_sum<TS, 2>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
    const float m = sum[1] * g.inv_n * r;              // mean(w dy n)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      float dxv[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = j * VE + e;
        const float n = h[i] * r;
        gv[i] = __builtin_fmaf(r, __builtin_fmaf(-n, m, w[i] * dv[i]), gv[i]);
        dxv[e] = s[i] * gv[i];
        dw[i] = __builtin_fmaf(dv[i], n, dw[i]);
        ds[i] = __builtin_fmaf(gv[i], xs[i], ds[i]);
      }
      if (c < g.n) {
        if (dres) store_n<RB, VE>(dres, base + c, gv + j * VE);
        store_n<XB, VE>(dx, base + c, dxv);
      }
    }
  }
  if (dweight) store_partial<TS, NV, VE>(dw, dweight, g, t, buf);
  if (dscale) store_partial<TS, NV, VE>(ds, dscale, g, t, buf);
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

template <int TS, int NV, int VE, bool XB, bool ZB>
__global__ __launch_bounds__(kNormThreads) void gated_norm_fwd_kernel(
    const void* x, const void* z, const float* __restrict__ weight, void* y, bool silu,
    bool first, NormGrid g) {
  __shared__ float red[2][4][2];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * VE];
  load_weights<NV, VE, TS>(weight, g, t, g.shared, 1.0f, w);
  if (!t.on) return;            // whole teams; a team of four waves is always on
  for (int64_t row = t.row; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim + (int64_t)t.group * g.n;
    float u[NV * VE], a[NV * VE], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      float xv[VE] = {}, zv[VE] = {}, d;
      if (c < g.n) {
        load_n<XB, VE>(x, base + c, xv);
        if (z) load_n<ZB, VE>(z, base + c, zv);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = j * VE + e;
        const float act = z ? gate_act(zv[e], silu, d) : 1.0f;
        u[i] = first ? xv[e] * act : xv[e];
        a[i] = first ? 1.0f : act;
        sum[0] = __builtin_fmaf(u[i], u[i], sum[0]);
      }
    }
    team_sum<TS, 1>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      if (c < g.n) {
        float v[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) v[e] = u[j * VE + e] * r * w[j * VE + e] * a[j * VE + e];
        store_n<ZB, VE>(y, base + c, v);
      }
    }
  }
}

template <int TS, int NV, int VE, bool XB, bool ZB>
__global__ __launch_bounds__(kNormThreads) void gated_norm_bwd_kernel(
    const void* x, const void* z, const float* __restrict__ weight, const void* dy, void* dx,
    void* dz, float* __restrict__ dweight, bool silu, bool first, NormGrid g) {
  __shared__ float red[2][4][2];
  __shared__ float buf[Team<TS>::kTeams > 1 ? VE * kNormThreads : 1];
  int turn = 0;
  Team<TS> t(g);
  float w[NV * VE], dw[NV * VE] = {};
  load_weights<NV, VE, TS>(weight, g, t, g.shared, 1.0f, w);
  for (int64_t row = t.on ? t.row : g.rows; row < g.rows; row += t.step) {
    const int64_t base = row * g.dim + (int64_t)t.group * g.n;
    float xs[NV * VE], act[NV * VE], der[NV * VE], dv[NV * VE], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      float zv[VE] = {};
#pragma unroll
      for (int e = 0; e < VE; ++e) xs[j * VE + e] = dv[j * VE + e] = 0.0f;
      if (c < g.n) {
        load_n<XB, VE>(x, base + c, xs + j * VE);
        load_n<ZB, VE>(dy, base + c, dv + j * VE);
        if (z) load_n<ZB, VE>(z, base + c, zv);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = j * VE + e;
        der[i] = 0.0f;
        act[i] = z ? gate_act(zv[e], silu, der[i]) : 1.0f;
        const float u = first ? xs[i] * act[i] : xs[i];
        const float en = dv[i] * w[i] * (first ? 1.0f : act[i]);
        sum[0] = __builtin_fmaf(u, u, sum[0]);
        sum[1] = __builtin_fmaf(en, u, sum[1]);
      }
    }
    team_sum<TS, 2>(sum, red, turn);
    const float r = rsqrtf(__builtin_fmaf(sum[0], g.inv_n, g.eps));
    const float m = sum[1] * g.inv_n * r;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t.lane + TS * j) * VE;
      float dxv[VE], dzv[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = j * VE + e;
        const float n = (first ? xs[i] * act[i] : xs[i]) * r;
        const float dn = first ? dv[i] : dv[i] * act[i];
        const float du = r * __builtin_fmaf(-n, m, dn * w[i]);
        dxv[e] = first ? du * act[i] : du;
        dzv[e] = (first ? du * xs[i] : dv[i] * n * w[i]) * der[i];
        dw[i] = __builtin_fmaf(dn, n, dw[i]);
      }
      if (c < g.n) {
        store_n<XB, VE>(dx, base + c, dxv);
        if (z) store_n<ZB, VE>(dz, base + c, dzv);
      }
    }
  }
  if (dweight) store_partial<TS, NV, VE>(dw, dweight, g, t, buf);
}

// Adds `parts` rows of `cols` partial sums in a fixed order: 16 slices of the
// rows, each added in turn, then the slices in order.
__global__ __launch_bounds__(1024) void sum_rows_kernel(const float* __restrict__ part,
                                                        float* __restrict__ out, int parts,
                                                        int cols) {
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
  int parts;      // rows of partial sums
  int cols;
};

// The lanes of a team: enough for one vector each up to a wave, then up to
// four vectors per lane of a wave, then a workgroup.
struct TeamPlan {
  int ts, nv, ve;
};
TeamPlan team_plan(int64_t n) {
  if (n % 8 == 0) {
    const int64_t u = n / 8;
    if (u <= 8) return {8, 1, 8};
    if (u <= 16) return {16, 1, 8};
    if (u <= 32) return {32, 1, 8};
    if (u <= 64) return {64, 1, 8};
    if (u <= 128) return {64, 2, 8};
    if (u <= 256) return {256, 1, 8};
    if (u <= 512) return {256, 2, 8};
    if (u <= 1024) return {256, 4, 8};
    return {256, 8, 8};
  }
  if (n <= 64) return {64, 1, 1};
  if (n <= 256) return {64, 4, 1};
  if (n <= 1024) return {256, 4, 1};
  if (n <= 4096) return {256, 16, 1};
  return {256, 64, 1};
}

NormLaunch norm_launch(const NormShape& s, float eps) {
  NormLaunch l;
  const int teams = kNormThreads / team_plan(s.group).ts;
  const int64_t groups = s.dim / s.group;
  int per = 1;
  while (per < teams && per < groups) per *= 2;
  const int64_t gy = (groups + per - 1) / per;
  const int64_t rows_per = teams / per;
  int64_t gx = (s.rows + rows_per - 1) / rows_per;
  const int64_t want = (kNormBlocks + gy - 1) / gy;
  if (gx > want) gx = want;
  l.g = NormGrid{s.rows,     s.dim, (int)s.group, (int)groups, per, s.wdim != s.dim,
                 1.0f / (float)s.group, eps};
  l.grid = dim3((unsigned)gx, (unsigned)gy);
  l.parts = (int)(l.g.shared ? gx * gy : gx);
  l.cols = (int)s.wdim;
  return l;
}

// f(TeamPlan constants) for the plan of a segment of n channels.
template <class F>
void with_plan(int64_t n, F f) {
  const TeamPlan p = team_plan(n);
  auto is = [&](int ts, int nv, int ve) { return p.ts == ts && p.nv == nv && p.ve == ve; };
#define SSD_NORM_PLAN(TS, NV, VE)                                       \
  if (is(TS, NV, VE)) {                                                 \
    return f(std::integral_constant<int, TS>{}, std::integral_constant<int, NV>{}, \
             std::integral_constant<int, VE>{});                        \
  }
  SSD_NORM_PLAN(8, 1, 8)
  SSD_NORM_PLAN(16, 1, 8)
  SSD_NORM_PLAN(32, 1, 8)
  SSD_NORM_PLAN(64, 1, 8)
  SSD_NORM_PLAN(64, 2, 8)
  SSD_NORM_PLAN(256, 1, 8)
  SSD_NORM_PLAN(256, 2, 8)
  SSD_NORM_PLAN(256, 4, 8)
  SSD_NORM_PLAN(256, 8, 8)
  SSD_NORM_PLAN(64, 1, 1)
  SSD_NORM_PLAN(64, 4, 1)
  SSD_NORM_PLAN(256, 4, 1)
  SSD_NORM_PLAN(256, 16, 1)
  SSD_NORM_PLAN(256, 64, 1)
#undef SSD_NORM_PLAN
}
template <class F>
void with_bool(bool b, F f) {
  if (b) return f(std::true_type{});
  f(std::false_type{});
}

int add_rows(const float* part, float* out, const NormLaunch& l, hipStream_t st) {
  const unsigned blocks = (unsigned)((l.cols + kWave - 1) / kWave);
  hipLaunchKernelGGL(sum_rows_kernel, dim3(blocks), dim3(1024), 0, st, part, out, l.parts,
                     l.cols);
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
  with_plan(s.group, [&](auto ts, auto nv, auto ve) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(rbf16, [&](auto rb) {
        hipLaunchKernelGGL((add_norm_fwd_kernel<ts(), nv(), ve(), xb(), rb()>), l.grid,
                           dim3(kNormThreads), 0, (hipStream_t)stream, x, res, scale, weight, y,
                           res_out, l.g);
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
  with_plan(s.group, [&](auto ts, auto nv, auto ve) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(rbf16, [&](auto rb) {
        hipLaunchKernelGGL((add_norm_bwd_kernel<ts(), nv(), ve(), xb(), rb()>), l.grid,
                           dim3(kNormThreads), 0, (hipStream_t)stream, x, res, scale, weight, dy,
                           dres_out, dx, dres, ps, pw, l.g);
      });
    });
  });
  int err = (int)hipGetLastError();
  if (err == 0 && dweight) err = add_rows(pw, dweight, l, (hipStream_t)stream);
  if (err == 0 && dscale) err = add_rows(ps, dscale, l, (hipStream_t)stream);
  return err;
}

int launch_gated_norm_fwd(const void* x, const void* z, const float* weight, void* y, float eps,
                          bool silu, bool first, bool xbf16, bool zbf16, const NormShape& s,
                          void* stream) {
  clear_launch_error();
  const NormLaunch l = norm_launch(s, eps);
  with_plan(s.group, [&](auto ts, auto nv, auto ve) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(zbf16, [&](auto zb) {
        hipLaunchKernelGGL((gated_norm_fwd_kernel<ts(), nv(), ve(), xb(), zb()>), l.grid,
                           dim3(kNormThreads), 0, (hipStream_t)stream, x, z, weight, y, silu,
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
  with_plan(s.group, [&](auto ts, auto nv, auto ve) {
    with_bool(xbf16, [&](auto xb) {
      with_bool(zbf16, [&](auto zb) {
        hipLaunchKernelGGL((gated_norm_bwd_kernel<ts(), nv(), ve(), xb(), zb()>), l.grid,
                           dim3(kNormThreads), 0, (hipStream_t)stream, x, z, weight, dy, dx, dz,
                           pw, silu, first, l.g);
      });
    });
  });
  int err = (int)hipGetLastError();
  if (err == 0 && dweight) err = add_rows(pw, dweight, l, (hipStream_t)stream);
  return err;
}

}  // namespace ssd
