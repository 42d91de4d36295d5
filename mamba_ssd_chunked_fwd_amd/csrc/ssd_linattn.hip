// Linear attention with a decay for each head over whole (packed) sequences,
// and its gradients.  Per (sequence, head), with lam = exp(log_decay_h):
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t
// and for the gradients, with R_t that of S_t,
//   R_t = scale q_t do_t^T + lam R_{t+1}      (dfinal past the last token)
//   dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,  dinit = lam R_1
//
// All four are one walk over the tokens, with an operand triple (X, Y, Z):
//   M = lam M + cz Y_t Z_t^T (before the output);  out_t = cx X_t^T M
//             walk    X   Y   Z    M        cx     cz
//   o         up      q   k   v    S        scale  1
//   dq        up      do  v   k    S^T      scale  1
//   dk        down    v   do  q    R^T      1      scale
//   dv        down    k   q   do   R        1      scale
// A walk up starts from the initial state and decays M before each token; one
// down starts from dfinal and decays M after each, so what it holds at the end
// is lam R_1.
#include "ssd_block_launch.h"
#include "ssd_device.h"
#include "ssd_host.h"

#include <type_traits>

namespace ssd {
namespace {

// One walk.  The row strides are in elements; head h of an operand starts at
// (h / share) * size.
struct Walk {
  const void *x, *y, *z;
  void* out;            // rows of the element type, or fp32 partial rows per head
  const float* start;   // [nseq, H, K, V] or null
  float* end;           // [nseq, H, K, V] or null
  int xshare, yshare, zshare, oshare;   // heads that share one of the operand's
  float cx, cz;
  bool down;
  bool turned;          // M is V x K: the transpose of the states in memory
  bool f32out;
};

struct Walks {
  Walk w[3];
};

struct Seqs {
  const int32_t* cu;
  int64_t tokens, len;
  int nseq;
  __device__ __forceinline__ int64_t at(int i) const {
    if (cu == nullptr) return i * len;
    const int64_t v = cu[i];
    return v < 0 ? 0 : v > tokens ? tokens : v;
  }
};

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  else
    return ((const float*)p)[i];
}

// One workgroup for each (sequence, head, walk); thread c owns column c of M.
template <int YD, int ZD, bool BF16>
__device__ void walk_tokens(const Walk& w, const Seqs& sq, const float* log_decay, int i, int h,
                            int H, float* xy) {
  const int c = threadIdx.x;
  const int64_t t0 = sq.at(i);
  const int64_t len = sq.at(i + 1) - t0;
  // -inf: no memory; the clamp keeps 0 * log_decay from being NaN
  const float lam = expf(fmaxf(log_decay[h], -1e30f));
  const int64_t sbase = ((int64_t)i * H + h) * YD * ZD;
  float m[YD];
#pragma unroll
  for (int r = 0; r < YD; ++r)
    m[r] = w.start ? w.start[sbase + (w.turned ? (int64_t)c * YD + r : (int64_t)r * ZD + c)] : 0.0f;
  const int64_t xs = (int64_t)(H / w.xshare) * YD, ys = (int64_t)(H / w.yshare) * YD;
  const int64_t zs = (int64_t)(H / w.zshare) * ZD, os = (int64_t)(H / w.oshare) * ZD;
  for (int64_t n = 0; n < len; ++n) {
    const int64_t t = t0 + (w.down ? len - 1 - n : n);
    __syncthreads();
    for (int r = c; r < YD; r += ZD) {
      xy[r] = load1<BF16>(w.x, t * xs + (int64_t)(h / w.xshare) * YD + r);
      xy[YD + r] = load1<BF16>(w.y, t * ys + (int64_t)(h / w.yshare) * YD + r);
    }
    __syncthreads();
    const float zv = w.cz * load1<BF16>(w.z, t * zs + (int64_t)(h / w.zshare) * ZD + c);
    float acc = 0.0f;
#pragma unroll
    for (int r = 0; r < YD; ++r) {
      m[r] = __builtin_fmaf(xy[YD + r], zv, w.down ? m[r] : lam * m[r]);
      acc = __builtin_fmaf(xy[r], m[r], acc);
      if (w.down) m[r] *= lam;
    }
    acc *= w.cx;
    const int64_t oi = t * os + (int64_t)(h / w.oshare) * ZD + c;
    if (!BF16 || w.f32out)
      ((float*)w.out)[oi] = acc;
    else
      ((uint16_t*)w.out)[oi] = (uint16_t)(pack_bf16(acc, 0.0f) & 0xFFFFu);
  }
  if (w.end) {
#pragma unroll
    for (int r = 0; r < YD; ++r) w.end[sbase + (int64_t)r * ZD + c] = m[r];
  }
}

template <int YD, int ZD, bool BF16>
__global__ __launch_bounds__(ZD) void walk_kernel(Walk w, Seqs sq,
                                                  const float* __restrict__ log_decay, int H) {
  __shared__ float xy[2 * YD];
  walk_tokens<YD, ZD, BF16>(w, sq, log_decay, blockIdx.x / H, blockIdx.x % H, H, xy);
}

// Sums the partial rows of the heads of each group, in their order.
template <bool BF16>
__global__ __launch_bounds__(256) void sum_heads_kernel(const float* __restrict__ part,
                                                        void* __restrict__ out, Seqs sq, int G,
                                                        int share, int D) {
  const int64_t t0 = sq.at(0), t1 = sq.at(sq.nseq);
  const int64_t row = (int64_t)G * D / 4;
  const int64_t end = t1 * row, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t u = t0 * row + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < end; u += step) {
    const int64_t e = u * 4, tg = e / D;
    const int d = (int)(e % D);
    const float* p = part + tg * share * D + d;
    f32x4 acc = *(const f32x4*)p;
    for (int k = 1; k < share; ++k) acc += *(const f32x4*)(p + (int64_t)k * D);
    if constexpr (BF16)
      *(u32x2*)((uint16_t*)out + e) =
          (u32x2){pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3])};
    else
      *(f32x4*)((float*)out + e) = acc;
  }
}

template <int YD, int ZD>
int launch_walk(const Walk& w, const Seqs& sq, const float* ld, bool bf16, const LinattnShape& s,
                hipStream_t st) {
  const dim3 grid((unsigned)(s.nseq * s.nheads)), block(ZD);
  if (bf16)
    hipLaunchKernelGGL((walk_kernel<YD, ZD, true>), grid, block, 0, st, w, sq, ld, (int)s.nheads);
  else
    hipLaunchKernelGGL((walk_kernel<YD, ZD, false>), grid, block, 0, st, w, sq, ld,
                       (int)s.nheads);
  return (int)hipGetLastError();
}

int walk_dims(const Walk& w, const Seqs& sq, const float* ld, bool bf16, const LinattnShape& s,
              int yd, int zd, hipStream_t st) {
  if (yd == 64)
    return zd == 64 ? launch_walk<64, 64>(w, sq, ld, bf16, s, st)
                    : launch_walk<64, 128>(w, sq, ld, bf16, s, st);
  return zd == 64 ? launch_walk<128, 64>(w, sq, ld, bf16, s, st)
                  : launch_walk<128, 128>(w, sq, ld, bf16, s, st);
}

int sum_heads(const float* part, void* out, const Seqs& sq, bool bf16, const LinattnShape& s,
              hipStream_t st) {
  const int64_t units = s.tokens * s.ngroups * s.dk / 4;
  const unsigned blocks = (unsigned)(units < 256 * 2048 ? (units + 255) / 256 : 2048);
  const int share = (int)(s.nheads / s.ngroups);
  if (bf16)
    hipLaunchKernelGGL((sum_heads_kernel<true>), dim3(blocks), dim3(256), 0, st, part, out, sq,
                       (int)s.ngroups, share, (int)s.dk);
  else
    hipLaunchKernelGGL((sum_heads_kernel<false>), dim3(blocks), dim3(256), 0, st, part, out, sq,
                       (int)s.ngroups, share, (int)s.dk);
  return (int)hipGetLastError();
}

Seqs seqs_of(const int32_t* cu, const LinattnShape& s) {
  return Seqs{cu, s.tokens, s.tokens / s.nseq, (int)s.nseq};
}

}  // namespace

size_t linattn_workspace(const LinattnShape& s, bool bf16, bool backward) {
  (void)bf16;
  size_t n = 16;
  if (backward && s.grouped()) n += 2 * sizeof(float) * (size_t)s.tokens * s.nheads * s.dk;
  return n;
}

int launch_linattn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                       const float* init, const int32_t* cu, void* o, float* fin, void* ws,
                       float scale, bool bf16, const LinattnShape& s, void* stream) {
  (void)ws;
  clear_launch_error();
  const int share = (int)(s.nheads / s.ngroups);
  const Walk w{q, k, v, o, init, fin, share, share, 1, 1, scale, 1.0f, false, false, false};
  return walk_dims(w, seqs_of(cu, s), log_decay, bf16, s, (int)s.dk, (int)s.dv,
                   (hipStream_t)stream);
}

int launch_linattn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                       const float* init, const int32_t* cu, const void* dout,
                       const float* dfinal, void* dq, void* dk, void* dv, float* dinit,
                       void* ws, float scale, bool bf16, const LinattnShape& s, void* stream) {
  clear_launch_error();
  hipStream_t st = (hipStream_t)stream;
  const int share = (int)(s.nheads / s.ngroups), K = (int)s.dk, V = (int)s.dv;
  const bool parts = s.grouped();
  float* pq = (float*)ws;
  float* pk = pq + (size_t)s.tokens * s.nheads * s.dk;
  const Seqs sq = seqs_of(cu, s);
  const Walk wq{dout, v, k,     parts ? (void*)pq : dq, init,  nullptr, 1,
                1,    share, 1, scale,                  1.0f,  false,   true, parts};
  const Walk wk{v, dout,  q, parts ? (void*)pk : dk, dfinal, nullptr, 1,
                1, share, 1, 1.0f,                   scale,  true,    true, parts};
  const Walk wv{k, q, dout, dv, dfinal, dinit, share, share, 1, 1, 1.0f, scale, true, false, false};
  // dv last: dinit may be the buffer of dfinal
  int err = walk_dims(wq, sq, log_decay, bf16, s, V, K, st);
  if (err == 0) err = walk_dims(wk, sq, log_decay, bf16, s, V, K, st);
  if (err == 0) err = walk_dims(wv, sq, log_decay, bf16, s, K, V, st);
  if (err == 0 && parts) err = sum_heads(pq, dq, sq, bf16, s, st);
  if (err == 0 && parts) err = sum_heads(pk, dk, sq, bf16, s, st);
  return err;
}

}  // namespace ssd
