// The short causal convolution of packed sequences, token-major: over the rows ext = (W-1 rows of
// the initial state, then the sequence's rows of x),
//   pre_t = bias + sum_{k<W} weight_k ext_{t+k},   y_t = pre_t or silu(pre_t)
// its gradients, and its form for single tokens.
//
// MI355X design.  Two or three rows for every token and some 15 operations an element: HBM-bound.
// A lane owns neighbouring channels and goes along a run of tokens with the last W - 1 rows in
// registers, so every row is read once (and W - 1 again at a run's start); the taps stay in
// registers.  Rows of a block of four tokens are on the way while another is worked on.  Runs
// (conv_run) are as long as some 8000 waves allow, the gradients' as some 5600: runs of 64 read 5%
// again, and the gradients' leave as few rows of partial sums of dweight and dbias as that (added
// by a kernel of their own in a fixed order).  The gradients finish a row of dx W - 1 tokens
// later, so their runs go W - 1 tokens past their end and form those tokens' pre-activations
// again.  Sums are fp32, each output rounded once.
//
// Measured at 16384 x 5376 in bf16, 4 taps, calls one behind the other: forward 80 us (353 MB: 4.4
// TB/s), gradients with their sums 128 (529 MB: 4.1), in fp32 153 (705 MB: 4.6) and 234 (1057 MB:
// 4.5); a device copy moves 5.15 TB/s.  (Under the profiler, apart: 78, 132 and 8.)  One token of
// 200 sequences of 5376 channels 6.5 us.
#include "ssd_host.h"
#include "ssd_selective_device.h"
#include "ssd_selective_launch.h"

#include <type_traits>

namespace ssd {
namespace {

struct ConvArgs {
  const void* x;
  const float *weight, *bias;
  const void* init;
  RunGrid runs;
  int64_t dim, x_stride;
  int vectors;               // vectors of a row
  Divide by_blocks;          // by the workgroups of a row
  void *y, *fin;
  // gradients
  const void *dy, *dfinal;
  void *dx, *dinit;
  float* part;               // [slots, W + 1, dim]
  float *dweight, *dbias;
  int64_t slots;
};

// V channels of a row as they lie in memory (V = 1: where rows do not start on whole vectors),
// and as floats.
template <bool BF16, int V>
struct Vec {
  static constexpr int kWords = V == 1 ? 1 : (BF16 ? V / 2 : V);
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (V == 1 && BF16) {
      w[0] = ((const uint16_t*)p)[i];
    } else if constexpr (kWords == 1) {
      w[0] = ((const uint32_t*)p)[BF16 ? i / 2 : i];
    } else if constexpr (kWords == 2) {
      const u32x2 u = *(const u32x2*)((const char*)p + i * (BF16 ? 2 : 4));
      w[0] = u[0];
      w[1] = u[1];
    } else {
      const u32x4 u = *(const u32x4*)((const char*)p + i * (BF16 ? 2 : 4));
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = u[k];
    }
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (BF16)
        v[e] = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
      else
        v[e] = __uint_as_float(w[e]);
    }
  }
};
template <bool BF16, int V>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float (&v)[V]) {
  Vec<BF16, V> u;
  u.load(p, i);
  u.get(v);
}
template <bool BF16, int V>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&v)[V]) {
  if constexpr (V == 1) {
    store_one<BF16>(p, i, v[0]);
  } else if constexpr (BF16 && V == 2) {
    *(uint32_t*)((uint16_t*)p + i) = pack_bf16(v[0], v[1]);
  } else if constexpr (BF16) {
    *(u32x2*)((uint16_t*)p + i) = (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else if constexpr (V == 2) {
    *(f32x2*)((float*)p + i) = (f32x2){v[0], v[1]};
  } else {
    *(f32x4*)((float*)p + i) = (f32x4){v[0], v[1], v[2], v[3]};
  }
}
template <int V>
__device__ __forceinline__ void zero(float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.0f;
}

template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int64_t d, float (&w)[W][V],
                                          float (&bias)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][e] = a.weight[(d + e) * W + k];
    bias[e] = a.bias ? a.bias[d + e] : 0.0f;
  }
}

// ext row i - (W-1) counted from token `t`: a token of the sequence, or a row of the
// initial state before it.
template <int W, bool BF16, int V>
__device__ __forceinline__ void load_row(const ConvArgs& a, const Run& r, int64_t t, int64_t d,
                                         float (&v)[V]) {
  if (t >= r.seq_begin)
    load_vec<BF16, V>(a.x, t * a.x_stride + d, v);
  else if (a.init != nullptr)
    load_vec<BF16, V>(a.init,
                      ((int64_t)r.seq * (W - 1) + (t - r.seq_begin + W - 1)) * a.dim + d, v);
  else
    zero(v);
}

constexpr int kTokens = 4;   // tokens of a block; one is on the way while another is worked on

// One run of one sequence for V channels a thread.
template <int W, bool BF16, int V, bool SILU>
__global__ __launch_bounds__(256) void short_conv_fwd_kernel(const ConvArgs a) {
  const int64_t slot = a.by_blocks.of(blockIdx.x);
  const int vec =
      (int)(blockIdx.x - (uint32_t)slot * a.by_blocks.d) * (int)blockDim.x + threadIdx.x;
  const Run r = find_run(a.runs, (int)slot);
  if (!r.on || vec >= a.vectors) return;
  const int64_t d = (int64_t)vec * V;
  // the next block's rows (those past the end read the last one's)
  auto load = [&](Vec<BF16, V>(&x)[kTokens], int t0) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j)
      x[j].load(a.x, (t0 + j < r.end ? t0 + j : r.end - 1) * a.x_stride + d);
  };
  Vec<BF16, V> even[kTokens], odd[kTokens];
  if (r.begin < r.end) load(even, r.begin);
  float w[W][V], bias[V], ext[W - 1][V], old[W - 1][V];
  load_taps<W, V>(a, d, w, bias);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    load_row<W, BF16, V>(a, r, r.begin - (W - 1) + k, d, ext[k]);
#pragma unroll
    for (int e = 0; e < V; ++e) old[k][e] = ext[k][e];
  }
  auto work = [&](const Vec<BF16, V>(&x)[kTokens], int t0) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      if (t0 + j >= r.end) break;
      float y[V], now[V];
      x[j].get(now);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float v = bias[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v = __builtin_fmaf(w[k][e], ext[k][e], v);
        v = __builtin_fmaf(w[W - 1][e], now[e], v);
        y[e] = SILU ? v * sigmoid_f(v) : v;
#pragma unroll
        for (int k = 0; k < W - 2; ++k) ext[k][e] = ext[k + 1][e];
        ext[W - 2][e] = now[e];
      }
      store_vec<BF16, V>(a.y, (int64_t)(t0 + j) * a.dim + d, y);
    }
  };
  int t0 = r.begin;
  for (; t0 + 2 * kTokens < r.end; t0 += 2 * kTokens) {
    load(odd, t0 + kTokens);
    work(even, t0);
    load(even, t0 + 2 * kTokens);
    work(odd, t0 + kTokens);
  }
  if (t0 + kTokens < r.end) load(odd, t0 + kTokens);
  if (t0 < r.end) work(even, t0);
  if (t0 + kTokens < r.end) work(odd, t0 + kTokens);
  // The final state comes from the first run, which alone has read the initial one
  // (they may be one buffer).
  if (r.index == 0 && a.fin != nullptr) {
    const int64_t len = r.seq_end - r.seq_begin;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[V];
      const int64_t t = r.seq_end - (W - 1) + j;
      if (t >= r.seq_begin) {
        load_vec<BF16, V>(a.x, t * a.x_stride + d, v);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          v[e] = old[j][e];
#pragma unroll
          for (int k = j + 1; k < W - 1; ++k) v[e] = j + len == k ? old[k][e] : v[e];
        }
      }
      store_vec<BF16, V>(a.fin, ((int64_t)r.seq * (W - 1) + j) * a.dim + d, v);
    }
  }
}

// The gradients of one run: dext rows are finished W-1 tokens after their own, so a run
// goes W-1 tokens past its end.
template <int W, bool BF16, int V, bool SILU>
__global__ __launch_bounds__(256) void short_conv_bwd_kernel(const ConvArgs a) {
  const int64_t slot = a.by_blocks.of(blockIdx.x);
  const int vec =
      (int)(blockIdx.x - (uint32_t)slot * a.by_blocks.d) * (int)blockDim.x + threadIdx.x;
  const Run r = find_run(a.runs, (int)slot);
  if (vec >= a.vectors) return;
  const int64_t d = (int64_t)vec * V;
  float dw[W][V], db[V];
  zero(db);
#pragma unroll
  for (int k = 0; k < W; ++k) zero(dw[k]);
  if (r.on) {
    float w[W][V], bias[V], ext[W][V], acc[W][V];
    load_taps<W, V>(a, d, w, bias);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_row<W, BF16, V>(a, r, r.begin - (W - 1) + k, d, ext[k]);
#pragma unroll
    for (int k = 0; k < W; ++k) zero(acc[k]);
    // the gradient of ext row `t` (a token, or a row of the initial state before them)
    auto emit = [&](int64_t t, float (&v)[V]) {
      const int64_t j = t - (r.seq_end - (W - 1));
      const bool token = t >= r.seq_begin;
      if (token ? t < r.begin || t >= r.end : r.index != 0 || a.dinit == nullptr) return;
      if (j >= 0 && a.dfinal != nullptr) {
        float f[V];
        load_vec<BF16, V>(a.dfinal, ((int64_t)r.seq * (W - 1) + j) * a.dim + d, f);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += f[e];
      }
      if (token)
        store_vec<BF16, V>(a.dx, t * a.dim + d, v);
      else
        store_vec<BF16, V>(a.dinit,
                           ((int64_t)r.seq * (W - 1) + (t - r.seq_begin + W - 1)) * a.dim + d,
                           v);
    };
    const int past = r.begin >= r.end ? r.begin
                                      : (r.seq_end - r.end < W - 1 ? r.seq_end : r.end + W - 1);
    struct Rows {
      Vec<BF16, V> x, dy;
    } even[kTokens], odd[kTokens];
    auto load = [&](Rows(&b)[kTokens], int t0) {
#pragma unroll
      for (int j = 0; j < kTokens; ++j) {
        const int64_t t = t0 + j < past ? t0 + j : past - 1;
        b[j].x.load(a.x, t * a.x_stride + d);
        b[j].dy.load(a.dy, t * a.dim + d);
      }
    };
    auto work = [&](const Rows(&b)[kTokens], int t0) {
#pragma unroll
      for (int j = 0; j < kTokens; ++j) {
        const int t = t0 + j;
        if (t >= past) break;
        float g[V];
        b[j].x.get(ext[W - 1]);
        b[j].dy.get(g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (SILU) {
            float v = bias[e];
#pragma unroll
            for (int k = 0; k < W; ++k) v = __builtin_fmaf(w[k][e], ext[k][e], v);
            const float s = sigmoid_f(v);
            g[e] *= s * __builtin_fmaf(v, 1.0f - s, 1.0f);
          }
#pragma unroll
          for (int k = 0; k < W; ++k) acc[k][e] = __builtin_fmaf(w[k][e], g[e], acc[k][e]);
        }
        if (t < r.end) {     // (past it a token counts for the rows before it alone)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            db[e] += g[e];
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][e] = __builtin_fmaf(g[e], ext[k][e], dw[k][e]);
          }
        }
        emit(t - (W - 1), acc[0]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ext[k][e] = ext[k + 1][e];
            acc[k][e] = acc[k + 1][e];
          }
        }
        zero(acc[W - 1]);
      }
    };
    int t0 = r.begin;
    if (t0 < past) load(even, t0);
    for (; t0 + 2 * kTokens < past; t0 += 2 * kTokens) {
      load(odd, t0 + kTokens);
      work(even, t0);
      load(even, t0 + 2 * kTokens);
      work(odd, t0 + kTokens);
    }
    if (t0 + kTokens < past) load(odd, t0 + kTokens);
    if (t0 < past) work(even, t0);
    if (t0 + kTokens < past) work(odd, t0 + kTokens);
    if (past == r.seq_end) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) emit(past - (W - 1) + k, acc[k]);
    }
  }
  float* row = a.part + slot * (W + 1) * a.dim + d;
#pragma unroll
  for (int k = 0; k < W + 1; ++k) {
    if constexpr (V == 1) {
      row[k * a.dim] = k < W ? dw[k < W ? k : 0][0] : db[0];
    } else {
      static_assert(V == 2, "channels of a lane");
      const float* v = k < W ? dw[k < W ? k : 0] : db;
      *(f32x2*)(row + k * a.dim) = (f32x2){v[0], v[1]};
    }
  }
}

// The sums over the slots, in their order: 64 channels of one of the W + 1 rows for a
// workgroup, the slots spread over its waves.
constexpr int kSumWaves = 8;
__global__ __launch_bounds__(kWave * kSumWaves) void short_conv_sum_kernel(const ConvArgs a,
                                                                           int width) {
  __shared__ float part[kSumWaves][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int k = blockIdx.x % (width + 1);
  const int64_t d = (int64_t)(blockIdx.x / (width + 1)) * kWave + lane;
  float sum = 0.0f;
  if (d < a.dim)
#pragma unroll 8
    for (int64_t s = wave; s < a.slots; s += kSumWaves)
      sum += a.part[(s * (width + 1) + k) * a.dim + d];
  part[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || d >= a.dim) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumWaves; ++i) sum += part[i][lane];
  if (k < width) {
    if (a.dweight) a.dweight[d * width + k] = sum;
  } else if (a.dbias) {
    a.dbias[d] = sum;
  }
}

// One token of every sequence: V channels of one sequence a thread.
template <int W, bool BF16, int V, bool SILU>
__global__ __launch_bounds__(256) void short_conv_step_kernel(const ConvArgs a) {
  const int64_t b = a.by_blocks.of(blockIdx.x);
  const int vec = (int)(blockIdx.x - (uint32_t)b * a.by_blocks.d) * (int)blockDim.x + threadIdx.x;
  if (vec >= a.vectors) return;
  const int64_t d = (int64_t)vec * V;
  float w[W][V], bias[V], ext[W][V], y[V];
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    load_vec<BF16, V>(a.fin, (b * (W - 1) + k) * a.dim + d, ext[k]);
  load_vec<BF16, V>(a.x, b * a.x_stride + d, ext[W - 1]);
  load_taps<W, V>(a, d, w, bias);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float v = bias[e];
#pragma unroll
    for (int k = 0; k < W; ++k) v = __builtin_fmaf(w[k][e], ext[k][e], v);
    y[e] = SILU ? v * sigmoid_f(v) : v;
  }
  store_vec<BF16, V>(a.y, b * a.dim + d, y);
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    store_vec<BF16, V>(a.fin, (b * (W - 1) + k) * a.dim + d, ext[k + 1]);
}

// Vectors of V channels where every row of every tensor starts on one.
bool whole_vectors(const ConvShape& s, const void* x, bool bf16, int V) {
  return s.dim % V == 0 && s.x_stride % V == 0 && (uintptr_t)x % (V * (bf16 ? 2 : 4)) == 0;
}

struct ConvGrid {
  int vectors, blocks, threads;
};
ConvGrid conv_grid(const ConvShape& s, int V) {
  ConvGrid g;
  g.vectors = (int)(s.dim / V);
  const int waves = (g.vectors + kWave - 1) / kWave;
  g.threads = kWave * (waves < 4 ? waves : 4);
  g.blocks = (g.vectors + g.threads - 1) / g.threads;
  return g;
}

// Channels of a lane.  Kernels of an earlier form against each other, 16384 x 5376 in bf16:
// forward 8 channels 79 us, 4 72 us (126 registers and 16-byte loads against 60 and 8); gradients
// 8 171, 4 132, 2 123.
constexpr int kFwdVec = 4, kBwdVec = 2;

// f(std::integral_constant W, bool BF16, int V, bool SILU) as types.
template <bool B>
using Flag = std::integral_constant<bool, B>;
template <int I>
using Int = std::integral_constant<int, I>;
template <int V, class F>
void choose(const ConvShape& s, bool bf16, bool vec, bool silu, F f) {
  auto w = [&](auto b, auto v, auto a) {
    if (s.width == 2)
      f(Int<2>{}, b, v, a);
    else if (s.width == 3)
      f(Int<3>{}, b, v, a);
    else
      f(Int<4>{}, b, v, a);
  };
  auto act = [&](auto b, auto v) { silu ? w(b, v, Flag<true>{}) : w(b, v, Flag<false>{}); };
  if (bf16)
    vec ? act(Flag<true>{}, Int<V>{}) : act(Flag<true>{}, Int<1>{});
  else
    vec ? act(Flag<false>{}, Int<V>{}) : act(Flag<false>{}, Int<1>{});
}

ConvArgs conv_args(const void* x, const float* weight, const float* bias, const void* init,
                   const int32_t* cu, const ConvShape& s, bool backward) {
  ConvArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.init = init;
  a.runs = make_run_grid(cu, s.tokens, s.nseq, conv_run(s, backward));
  a.slots = run_slots(a.runs);
  a.dim = s.dim;
  a.x_stride = s.x_stride;
  return a;
}

}  // namespace

int launch_short_conv_fwd(const void* x, const float* weight, const float* bias, const void* init,
                          const int32_t* cu, void* y, void* fin, bool silu, bool bf16,
                          const ConvShape& s, void* stream) {
  clear_launch_error();
  ConvArgs a = conv_args(x, weight, bias, init, cu, s, false);
  a.y = y;
  a.fin = fin;
  const bool vec = whole_vectors(s, x, bf16, kFwdVec);
  choose<kFwdVec>(s, bf16, vec, silu, [&](auto w, auto b, auto v, auto act) {
    const ConvGrid g = conv_grid(s, v.value);
    a.vectors = g.vectors;
    a.by_blocks = Divide(g.blocks);
    hipLaunchKernelGGL(
        (short_conv_fwd_kernel<decltype(w)::value, decltype(b)::value, decltype(v)::value,
                               decltype(act)::value>),
        dim3((unsigned)(a.slots * g.blocks)), dim3(g.threads), 0, (hipStream_t)stream, a);
  });
  return (int)hipGetLastError();
}

int launch_short_conv_bwd(const void* x, const float* weight, const float* bias, const void* init,
                          const int32_t* cu, const void* dy, const void* dfinal, void* dx,
                          float* dweight, float* dbias, void* dinit, void* ws, bool silu,
                          bool bf16, const ConvShape& s, void* stream) {
  clear_launch_error();
  ConvArgs a = conv_args(x, weight, bias, init, cu, s, true);
  a.dy = dy;
  a.dfinal = dfinal;
  a.dx = dx;
  a.dinit = dinit;
  a.part = (float*)ws;
  a.dweight = dweight;
  a.dbias = dbias;
  const bool vec = whole_vectors(s, x, bf16, kBwdVec);
  hipStream_t st = (hipStream_t)stream;
  choose<kBwdVec>(s, bf16, vec, silu, [&](auto w, auto b, auto v, auto act) {
    const ConvGrid g = conv_grid(s, v.value);
    a.vectors = g.vectors;
    a.by_blocks = Divide(g.blocks);
    hipLaunchKernelGGL(
        (short_conv_bwd_kernel<decltype(w)::value, decltype(b)::value, decltype(v)::value,
                               decltype(act)::value>),
        dim3((unsigned)(a.slots * g.blocks)), dim3(g.threads), 0, st, a);
  });
  if (dweight != nullptr || dbias != nullptr)
    hipLaunchKernelGGL(short_conv_sum_kernel,
                       dim3((unsigned)((s.dim + kWave - 1) / kWave * (s.width + 1))),
                       dim3(kWave * kSumWaves), 0, st, a, (int)s.width);
  return (int)hipGetLastError();
}

int launch_short_conv_step(const void* x, const float* weight, const float* bias, void* state,
                           void* y, bool silu, bool bf16, const ConvShape& s, void* stream) {
  clear_launch_error();
  ConvArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.dim = s.dim;
  a.x_stride = s.x_stride;
  a.y = y;
  a.fin = state;
  const bool vec = whole_vectors(s, x, bf16, kFwdVec);
  choose<kFwdVec>(s, bf16, vec, silu, [&](auto w, auto b, auto v, auto act) {
    const ConvGrid g = conv_grid(s, v.value);
    a.vectors = g.vectors;
    a.by_blocks = Divide(g.blocks);
    hipLaunchKernelGGL(
        (short_conv_step_kernel<decltype(w)::value, decltype(b)::value, decltype(v)::value,
                                decltype(act)::value>),
        dim3((unsigned)(s.tokens * g.blocks)), dim3(g.threads), 0, (hipStream_t)stream, a);
  });
  return (int)hipGetLastError();
}

}  // namespace ssd
