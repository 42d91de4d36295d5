// The residual add and RMS norm in front of a block whose projection takes 8 bits:
//   h = residual + s o x,   y = h / sqrt(mean(h^2) + eps) o w,
//   scale = max |y| / top and codes = nearest(y top / max |y|) per group of channels.
//
// MI355X design.  Read once, written once: HBM-bound.  A workgroup owns a row, a lane one or
// two vectors of eight channels, which stay in registers from the read to the codes; groups
// of up to 256 channels lie in up to 32 neighbouring lanes and find their largest value by
// lane exchanges, longer ones meet in LDS.  A code's border may lie anywhere, and a
// value that 32 bits put on its other side comes out a whole step (up to 12%) away, so
// everything between the inputs and the codes is formed in 64 bits, which the
// vector unit does at the rate of 32.  The codes are rounded once: to 32 bits "to odd", then by
// the 8-bit conversion.
//
// Measured at 16384 x 5120, bf16 with an fp32 stream, groups of 128, e4m3: 191 us for 925 MB (4.8
// TB/s; a device copy moves 5.15).  Rows of up to 8192 channels are read a row ahead (two
// vectors a lane do not leave the registers for it, and most of their forms have 12 to 124 bytes of
// scratch: 8192 x 16384 490 us in e4m3, 441 in int8, 3.0 and 3.4 TB/s).  Branches on what a row
// has cost 281 us.
#include "ssd_host.h"
#include "ssd_selective_device.h"
#include "ssd_selective_launch.h"

#include <type_traits>

namespace ssd {
namespace {

constexpr int kVec = 8;
constexpr double kLeast = 1e-30;    // groups below it have codes of 0

struct QuantArgs {
  const void *x, *res;
  const float *scale, *weight;
  void *codes, *res_out;
  float* scales;
  int64_t rows;
  int dim, group;
  double eps, inv_dim;
};

// Eight elements as they lie in memory, and as floats (zeros where fewer are left).
template <bool BF16, bool WHOLE>
struct Eight {
  uint32_t w[BF16 ? 4 : 8];
  __device__ __forceinline__ void load(const void* p, int64_t i, int left) {
    if constexpr (!WHOLE) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if constexpr (BF16) {
          const uint32_t v = e < left ? ((const uint16_t*)p)[i + e] : 0u;
          w[e / 2] = e & 1 ? w[e / 2] | v << 16 : v;
        } else {
          w[e] = e < left ? ((const uint32_t*)p)[i + e] : 0u;
        }
      }
    } else {
      const u32x4* q = (const u32x4*)((const char*)p + i * (BF16 ? 2 : 4));
#pragma unroll
      for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
        const u32x4 u = q[h];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * h + k] = u[k];
      }
    }
  }
  __device__ __forceinline__ void fill(uint32_t v) {
#pragma unroll
    for (int k = 0; k < (BF16 ? 4 : 8); ++k) w[k] = v;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (BF16) return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    return __uint_as_float(w[e]);
  }
};
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store_eight(void* p, int64_t i, int left, const float (&v)[kVec]) {
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (e < left) store_one<BF16>(p, i + e, v[e]);
  } else if constexpr (BF16) {
    *(u32x4*)((uint16_t*)p + i) = (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                          pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  } else {
    *(f32x4*)((float*)p + i) = (f32x4){v[0], v[1], v[2], v[3]};
    *(f32x4*)((float*)p + i + 4) = (f32x4){v[4], v[5], v[6], v[7]};
  }
}

// To 32 bits so that rounding the result again, to fewer bits, rounds v once: cut off, and
// the last bit set if anything was.
__device__ __forceinline__ float to_odd(double v) {
  uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t rest = u & 0x1FFFFFFFu;
  u &= ~(uint64_t)0x1FFFFFFFu;
  if (rest != 0) u |= 0x20000000u;
  return (float)__builtin_bit_cast(double, u);
}

// Eight codes.
template <bool E4M3>
__device__ __forceinline__ u32x2 encode(const double (&v)[kVec]) {
  u32x2 out;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (E4M3) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(to_odd(v[4 * k]), to_odd(v[4 * k + 1]), 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(to_odd(v[4 * k + 2]), to_odd(v[4 * k + 3]), w, true);
      out[k] = (uint32_t)w;
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double q = v[4 * k + e];
        const int c = q == q ? (int)__builtin_rint(q) : 0;
        w |= (uint32_t)(c & 0xFF) << (8 * e);
      }
      out[k] = w;
    }
  }
  return out;
}

constexpr int kMaxWaves = 16;

// GROUPED: groups of 16 to 256 channels; otherwise the row is one.
template <int NV, bool XBF16, bool RBF16, bool E4M3, bool GROUPED, bool WHOLE>
__global__ __launch_bounds__(kMaxWaves* kWave) void add_norm_quant_kernel(const QuantArgs a) {
  __shared__ double red[2][2][kMaxWaves];
  int turn = 0;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int waves = (int)blockDim.x / kWave;
  const double top = E4M3 ? 448.0 : 127.0;

  // a lane's channels: their scale, weight and the next row's values.  What is not there, and
  // lanes past the row's end, have ones and zeros, so nothing below asks for them.
  Eight<false, WHOLE> s[NV], w[NV];
  Eight<XBF16, WHOLE> x[NV];
  Eight<RBF16, WHOLE> r[NV];
  const auto channel = [&](int j) { return ((int)threadIdx.x + j * (int)blockDim.x) * kVec; };
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      if (c >= a.dim) continue;
      x[j].load(a.x, row * a.dim + c, a.dim - c);
      if (a.res) r[j].load(a.res, row * a.dim + c, a.dim - c);
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    x[j].fill(0);
    r[j].fill(0);
    s[j].fill(__float_as_uint(1.0f));
    w[j].fill(__float_as_uint(1.0f));
  }
  // Rows of one vector a lane are read a row ahead, and scales and weights once; two vectors
  // do not leave the registers for it.
  constexpr bool kAhead = NV == 1;
  const auto load_params = [&] {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      if (c >= a.dim) continue;
      if (a.scale) s[j].load(a.scale, c, a.dim - c);
      if (a.weight) w[j].load(a.weight, c, a.dim - c);
    }
  };
  if (kAhead) {
    load(blockIdx.x);
    load_params();
  }
  const int64_t groups = a.dim / a.group;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    // h, the sum of its squares, then h o w (whose largest value is the group's: the row's
    // factor is not needed for the codes)
    double h[NV][kVec], most[NV], sum = 0.0;
    if (!kAhead) {
      load(row);
      asm volatile("" ::: "memory");     // (scales and weights are not kept from row to row)
      load_params();
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      float rounded[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const double v = __builtin_fma((double)s[j].get(e), (double)x[j].get(e),
                                       (double)r[j].get(e));
        sum = __builtin_fma(v, v, sum);
        rounded[e] = (float)v;
        h[j][e] = v;
      }
      if (a.res_out && c < a.dim)
        store_eight<RBF16, WHOLE>(a.res_out, row * a.dim + c, a.dim - c, rounded);
    }
    if (kAhead && row + gridDim.x < a.rows) load(row + gridDim.x);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // (a value that is not finite makes bad a NaN, and the largest value with it)
      double bad = 0.0;
      most[j] = 0.0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        h[j][e] *= (double)w[j].get(e);
        most[j] = __builtin_fmax(most[j], __builtin_fabs(h[j][e]));
        bad = __builtin_fma(h[j][e], 0.0, bad);
      }
      most[j] = bad == 0.0 ? most[j] : bad;
    }
    // of two values, the larger, or one that is a NaN
    const auto larger = [](double p, double q) { return p > q || p != p ? p : q; };
    if constexpr (GROUPED) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        for (int off = 1; off < a.group / kVec; off <<= 1)
          most[j] = larger(most[j], __shfl_xor(most[j], off, kWave));
      }
    } else {
#pragma unroll
      for (int j = 1; j < NV; ++j) most[0] = larger(most[0], most[j]);
#pragma unroll
      for (int off = kWave / 2; off > 0; off >>= 1)
        most[0] = larger(most[0], __shfl_xor(most[0], off, kWave));
    }
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
    if (waves > 1) {
      if (lane == 0) {
        red[turn][0][wave] = sum;
        red[turn][1][wave] = most[0];
      }
      __syncthreads();
      sum = 0.0;
      for (int k = 0; k < waves; ++k) {
        sum += red[turn][0][k];
        if (!GROUPED) most[0] = larger(most[0], red[turn][1][k]);
      }
      turn ^= 1;      // (written again behind the next row's barrier)
    }
    const double rstd = 1.0 / __builtin_sqrt(__builtin_fma(sum, a.inv_dim, a.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      if (c >= a.dim) continue;
      const double m = GROUPED ? most[j] : most[0], y = m * rstd;
      // h top / m with the product's error taken back, so that a value on a border lies on it
      // (2 us of the 191)
      const bool some = y >= kLeast;
      const double inv = some ? 1.0 / m : 0.0, by = some ? m : 0.0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const double v = h[j][e] * top, q = v * inv;
        h[j][e] = __builtin_fma(__builtin_fma(-q, by, v), inv, q);
      }
      const u32x2 codes = encode<E4M3>(h[j]);
      uint8_t* out = (uint8_t*)a.codes + row * a.dim + c;
      if constexpr (WHOLE) {
        *(u32x2*)out = codes;
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (c + e < a.dim) out[e] = (uint8_t)(codes[e / 4] >> (8 * (e % 4)));
      }
      if (GROUPED ? c % a.group == 0 : c == 0)
        a.scales[row * groups + (GROUPED ? c / a.group : 0)] = (float)(y / top);
    }
  }
}

template <int NV, bool XBF16, bool RBF16, bool E4M3>
void launch_t(const QuantArgs& a, bool grouped, bool whole, int blocks, int threads,
              hipStream_t st) {
#define SSD_QUANT(G, W)                                                                       \
  hipLaunchKernelGGL((add_norm_quant_kernel<NV, XBF16, RBF16, E4M3, G, W>), dim3(blocks),     \
                     dim3(threads), 0, st, a)
  if (grouped)
    SSD_QUANT(true, true);
  else if (whole)
    SSD_QUANT(false, true);
  else
    SSD_QUANT(false, false);
#undef SSD_QUANT
}

}  // namespace

int launch_add_norm_quant(const void* x, const void* res, const float* scale, const float* weight,
                          void* codes, float* scales, void* res_out, int64_t rows, int64_t dim,
                          int64_t group, float eps, bool e4m3, bool xbf16, bool rbf16,
                          void* stream) {
  clear_launch_error();
  const QuantArgs a{x, res, scale, weight, codes, res_out, scales, rows, (int)dim, (int)group,
                    (double)eps, 1.0 / (double)dim};
  const int vectors = (int)((dim + kVec - 1) / kVec);
  const int nv = vectors > kMaxWaves * kWave ? 2 : 1;
  const int waves = (vectors + nv * kWave - 1) / (nv * kWave);
  // as many whole workgroups (of 1 to 16 waves) for each of the 256 CUs as its registers hold:
  // 20 waves
  const int64_t most = 256 * (20 / waves);
  const int blocks = (int)(rows < most ? rows : most);
  const bool grouped = group == 16 || group == 32 || group == 64 || group == 128 || group == 256;
  const bool whole = dim % kVec == 0;
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto n, auto xb, auto rb, auto q) {
    launch_t<decltype(n)::value, decltype(xb)::value, decltype(rb)::value, decltype(q)::value>(
        a, grouped, whole, blocks, waves * kWave, st);
  };
  auto code = [&](auto n, auto xb, auto rb) {
    e4m3 ? go(n, xb, rb, std::true_type{}) : go(n, xb, rb, std::false_type{});
  };
  auto res_type = [&](auto n, auto xb) {
    rbf16 ? code(n, xb, std::true_type{}) : code(n, xb, std::false_type{});
  };
  auto x_type = [&](auto n) {
    xbf16 ? res_type(n, std::true_type{}) : res_type(n, std::false_type{});
  };
  if (nv == 1)
    x_type(std::integral_constant<int, 1>{});
  else
    x_type(std::integral_constant<int, 2>{});
  return (int)hipGetLastError();
}

}  // namespace ssd
