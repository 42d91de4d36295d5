// Linear attention with a decay for each head over whole (packed) sequences,
// and its gradients.  Per (sequence, head), with lam = exp(log_decay_h):
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t
// and for the gradients, with R_t that of S_t,
//   R_t = scale q_t do_t^T + lam R_{t+1}      (dfinal past the last token)
//   dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,  dinit = lam R_1
//
// All four are one walk over the tokens, with an operand triple (X, Y, Z):
//   M = lam M + cz Y_t Z_t^T;  out_t = cx X_t^T M
//             walk    X   Y   Z    M        cx     cz
//   o         up      q   k   v    S        scale  1
//   dq        up      do  v   k    S^T      scale  1
//   dk        down    v   do  q    R^T      1      scale
//   dv        down    k   q   do   R        1      scale
// A walk up starts from the initial state and decays M before each token; one
// down starts from dfinal and decays M after each, so what it holds at the end
// is lam R_1.  In chunks of C tokens, i and j counted in the walk's order, n
// tokens in the chunk, a = 1 up and 0 down:
//   out_i = cx lam^{i+a} X_i^T M + sum_{j<=i} cx cz lam^{i-j} (X_i . Y_j) Z_j
//   M     = lam^n M + sum_j cz lam^{n-a-j} Y_j Z_j^T
//
// MI355X design.  One workgroup of four waves walks one run of chunks of a
// (sequence, head) with M in its accumulators (a wave owns ZD/4 columns, all
// rows), so per token the inputs are read and the output is written once and no
// chunk's state touches memory.  Every product takes an operand as it sits
// in registers:
//   - M as left by the matrix instructions (a lane holds one column and four
//     consecutive rows of each block) is the operand of X^T M whose k slots
//     run over those rows; X is read from LDS in the same slot order;
//   - the scores are formed transposed (Y X^T: a lane holds one token i and four
//     consecutive j), so decayed, masked by a select and rounded they are the
//     operand of the sum over j as they sit; Z comes from the LDS transpose read;
//   - the output comes out transposed too, one token and 8 (fp32: 4)
//     consecutive columns per lane: 16-byte stores.
// bf16 tensors: 16x16x32 bf16 products, chunks of 64.  M and the scores are
// rounded to bf16 as operands (each adds as much error to `out` as its own
// rounding does); in M's update the decayed Z is split into two bf16 terms, so
// that the fp32 state keeps 16 bits of each product.  fp32 tensors: 16x16x4 fp32
// products, chunks of 32 (the scores' share grows with the chunk, and these
// calls are bound by the matrix pipe).
//
// The chains of a call are few (sequences x heads) and long, so each is cut
// into runs of `run` tokens, walked at once by (about) two workgroups per CU:
//   1. run_states: what every run but the last adds to M from zero;
//   2. run_starts: M at the start of every run, in place (lam^run from run to
//      run, an element per thread);
//   3. walks: the runs.
// A call whose chains are all no longer than a run goes straight to 3.  The
// powers of lam that are multiplied up along a chain are taken in 64 bits and
// kept as two fp32 terms: the rounding of one factor would otherwise grow with
// the number of chunks.
#include "ssd_block_launch.h"
#include "ssd_device.h"
#include "ssd_host.h"

#include <type_traits>

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr uint32_t kPastRange = 0x7FFF0000u;

// One walk.  Head h of an operand is its head h / share.
struct Walk {
  const void *x, *y, *z;
  void* out;            // rows of the element type, or fp32 partial rows per head
  const float* start;   // [nseq, H, K, V] or null
  float* end;           // [nseq, H, K, V] or null
  float* slots;         // states at the runs' starts, in accumulator order
  int xshare, yshare, zshare, oshare;
  float cx, cz;
  bool down;
  bool turned;          // M is V x K: the transpose of the states in memory
  bool f32out;
};

struct Walks {
  Walk w[3];
};

// The sequences and how they are cut.  Sequence i's runs are the grid's
// items at(i) / run + i, ...: the items of one sequence end before the next
// one's begin, because ceil(n / run) <= floor(b / run) - floor(a / run) + 1.
// Its state slots begin at floor(2 at(i) / run), which leaves room for all
// its runs wherever there is more than one.
struct Seqs {
  const int32_t* cu;
  int64_t tokens, len;
  int nseq, run;
  __device__ __forceinline__ int64_t at(int i) const {
    if (cu == nullptr) return i * len;
    const int64_t v = cu[i];
    return v < 0 ? 0 : v > tokens ? tokens : v;
  }
};

// A workgroup's run: sequence, its first token and length, the run's number
// and how many there are; seq < 0: none.
struct Run {
  int seq, r, nruns;
  int64_t t0, len;
  int64_t slot;
};

__device__ __forceinline__ Run find_run(const Seqs& s, int item) {
  int before = 0;                        // sequences that begin at or before the item
  for (int i0 = 0; i0 < s.nseq; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    const int n = __syncthreads_count(i < s.nseq && s.at(i) / s.run + i <= item);
    before += n;
    if (n < kThreads) break;
  }
  Run out{before - 1, 0, 0, 0, 0, 0};
  if (out.seq < 0) return out;
  out.t0 = s.at(out.seq);
  const int64_t end = s.at(out.seq + 1);
  out.len = end > out.t0 ? end - out.t0 : 0;
  out.nruns = out.len > s.run ? (int)((out.len + s.run - 1) / s.run) : 1;
  const int64_t r = item - (out.t0 / s.run + out.seq);
  out.r = (int)r;
  out.slot = 2 * out.t0 / s.run + r;
  if (r < 0 || r >= out.nruns) out.seq = -1;
  return out;
}

// Consecutive logical items on one XCD (blocks are dealt round-robin).
__device__ __forceinline__ int xcd_map(int bid, int total) {
  if (total % 8) return bid;
  return (bid % 8) * (total / 8) + bid / 8;
}

// log2 of lam.  The clamp keeps a head without memory (log_decay -inf) from
// giving 0 * inf: 2^(-1e30) is 0 and 2^0 is 1.
__device__ __forceinline__ float log2_decay(const float* ld, int h) {
  return fmaxf(ld[h], -1e30f) * kLog2e;
}
// lam^n as two fp32 terms.
struct Power {
  float hi, lo;
};
__device__ __forceinline__ Power power(const float* ld, int h, int n) {
  const double d = exp((double)fmaxf(ld[h], -1e30f) * (double)n);
  const float hi = (float)d;
  return Power{hi, (float)(d - (double)hi)};
}
__device__ __forceinline__ float times(Power p, float v) {
  return __builtin_fmaf(p.hi, v, p.lo * v);
}

template <int YD, int ZD, bool BF16>
struct Shape2 {
  static constexpr int ES = BF16 ? 2 : 4;
  static constexpr int C = BF16 ? 64 : 32;           // tokens per chunk
  static constexpr int NB = C / 16;                  // token blocks
  static constexpr int NY = YD / 16;                 // row blocks of M
  static constexpr int NZ = ZD / (16 * kWaves);      // column blocks of a wave
  // LDS row strides, in elements: with these the 16 rows of an operand read and
  // the 4 rows of a transpose read fall on different banks.
  static constexpr int YS = BF16 ? (YD == 128 ? 152 : 72) : YD + 4;
  static constexpr int ZS = BF16 ? (ZD == 128 ? 152 : 72) : ZD + 4;
  static constexpr int XBYTES = C * YS * ES;
  static constexpr int ZBYTES = C * ZS * ES;
  static constexpr int YU = C * YD * ES / 16 / kThreads;   // 16-byte units per thread
  static constexpr int ZU = C * ZD * ES / 16 / kThreads;
  // Column of M that row (or lane) rho of a wave's column block nz stands for.
  static __device__ __forceinline__ int zcol(int wave, int nz, int rho) {
    if constexpr (BF16) return 16 * NZ * wave + 4 * NZ * (rho >> 2) + 4 * nz + (rho & 3);
    return 16 * NZ * wave + 16 * nz + rho;
  }
};

// A tile of `n` token rows in the walk's order: its descriptor and each
// thread's units.
template <int D, int C, int ES, int U>
struct Tile {
  u32x4 v[U];
  __device__ __forceinline__ void issue(const void* base, int64_t heads, int head, int64_t lowest,
                                        int n, bool down) {
    const uint32_t row = (uint32_t)(heads * D * ES);
    const rsrc_t r = make_rsrc((const char*)base + (lowest * heads + head) * (D * ES),
                               (uint32_t)(n - 1) * row + D * ES);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = (int)threadIdx.x + kThreads * j;
      const int i = u / (D * ES / 16), c = u % (D * ES / 16);
      const uint32_t off = (uint32_t)(down ? n - 1 - i : i) * row + c * 16;
      v[j] = load_b128(r, i < n ? off : kPastRange);
    }
  }
  __device__ __forceinline__ void commit(char* lds, int stride) const {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = (int)threadIdx.x + kThreads * j;
      const int i = u / (D * ES / 16), c = u % (D * ES / 16);
      *(u32x4*)(lds + i * stride * ES + c * 16) = v[j];
    }
  }
};

// One run of one walk; with OUT the outputs too, else only M from zero.
template <int YD, int ZD, bool BF16, bool OUT>
__device__ __forceinline__ void walk_run(const Walk& w, const Seqs& sq, const Run& run,
                                         const float* log_decay, int h, int H, char* lds) {
  using S = Shape2<YD, ZD, BF16>;
  constexpr int C = S::C, NB = S::NB, NY = S::NY, NZ = S::NZ, YS = S::YS, ZS = S::ZS;
  constexpr int ES = S::ES;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
  const int lr = lane & 15, lq = lane >> 4;
  char* xs = lds;
  char* ys = lds + (OUT ? S::XBYTES : 0);
  char* zs = ys + S::XBYTES;

  const float l2 = log2_decay(log_decay, h);
  const int a = w.down ? 0 : 1;
  const int64_t p0 = (int64_t)run.r * sq.run;
  const int len = (int)(run.len - p0 < sq.run ? run.len - p0 : sq.run);

  // M[y][z]: block (yb, nz) holds rows 16 yb + 4 lq + r, column zcol(nz, lr).
  f32x4 m[NY][NZ];
  const int64_t sbase = ((int64_t)run.seq * H + h) * YD * ZD;
  const bool from_slot = OUT && run.nruns > 1;
#pragma unroll
  for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
    for (int nz = 0; nz < NZ; ++nz) {
      m[yb][nz] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
      if (from_slot) {
        m[yb][nz] = *(const f32x4*)(w.slots + (run.slot * H + h) * YD * ZD +
                                    ((yb * NZ + nz) * kThreads + tid) * 4);
      } else if (OUT && w.start != nullptr) {
        const int y = 16 * yb + 4 * lq, z = S::zcol(wave, nz, lr);
        if (w.turned) {
          m[yb][nz] = *(const f32x4*)(w.start + sbase + z * YD + y);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) m[yb][nz][r] = w.start[sbase + (y + r) * ZD + z];
        }
      }
    }
  }

  // Decays: of the scores by block distance, of X^T M by token, of Z by token.
  float dec[NB][4], ex[NB], wz[NB][4];
  const float cs = w.cx * w.cz;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 16 * b + lr - 4 * lq - r;
      dec[b][r] = d >= 0 ? cs * exp2_hw(l2 * (float)d) : 0.0f;
      wz[b][r] = w.cz * exp2_hw(l2 * (float)(C - a - (16 * b + 4 * lq + r)));
    }
    ex[b] = w.cx * exp2_hw(l2 * (float)(16 * b + lr + a));
  }
  Power lam_n = power(log_decay, h, C);

  Tile<YD, C, ES, S::YU> tx, ty;
  Tile<ZD, C, ES, S::ZU> tz;
  auto issue = [&](int p) {
    const int n = len - p < C ? len - p : C;
    const int64_t lowest =
        w.down ? run.t0 + run.len - p0 - p - n : run.t0 + p0 + p;
    if constexpr (OUT) tx.issue(w.x, H / w.xshare, h / w.xshare, lowest, n, w.down);
    ty.issue(w.y, H / w.yshare, h / w.yshare, lowest, n, w.down);
    tz.issue(w.z, H / w.zshare, h / w.zshare, lowest, n, w.down);
  };
  if (len > 0) issue(0);
  for (int p = 0; p < len; p += C) {
    const int n = len - p < C ? len - p : C;
    __syncthreads();
    if constexpr (OUT) tx.commit(xs, YS);
    ty.commit(ys, YS);
    tz.commit(zs, ZS);
    __syncthreads();
    if (p + C < len) issue(p + C);
    if (n < C) {
      lam_n = power(log_decay, h, n);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * b + 4 * lq + r;
          wz[b][r] = j < n ? w.cz * exp2_hw(l2 * (float)(n - a - j)) : 0.0f;
        }
      }
    }

    // The output rows' descriptor.
    const int64_t lowest = w.down ? run.t0 + run.len - p0 - p - n : run.t0 + p0 + p;
    const int64_t oheads = H / w.oshare;
    const bool f32o = !BF16 || w.f32out;
    const int oes = f32o ? 4 : 2;
    const uint32_t orow = (uint32_t)(oheads * ZD * oes);
    const rsrc_t orr = make_rsrc((char*)w.out + (lowest * oheads + h / w.oshare) * (ZD * oes),
                                 (uint32_t)(n - 1) * orow + ZD * oes);
    auto store_out = [&](int tb, const f32x4 (&o)[NZ]) {
      const int i = 16 * tb + lr;
      const uint32_t at = i < n ? (uint32_t)(w.down ? n - 1 - i : i) * orow : kPastRange;
#pragma unroll
      for (int nz = 0; nz < NZ; ++nz) {
        const uint32_t off = at + S::zcol(wave, nz, 4 * lq) * oes;
        if (f32o) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[nz]), orr, (int)off,
                                                 0, 0);
        } else if constexpr (NZ == 2) {
          if (nz == 0)
            __builtin_amdgcn_raw_buffer_store_b128(
                (u32x4){pack_bf16(o[0][0], o[0][1]), pack_bf16(o[0][2], o[0][3]),
                        pack_bf16(o[1][0], o[1][1]), pack_bf16(o[1][2], o[1][3])},
                orr, (int)off, 0, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b64(
              (u32x2){pack_bf16(o[0][0], o[0][1]), pack_bf16(o[0][2], o[0][3])}, orr, (int)off, 0,
              0);
        }
      }
    };

    if constexpr (BF16) {
      const uint16_t* xl = (const uint16_t*)xs;
      const uint16_t* yl = (const uint16_t*)ys;
      const uint16_t* zl = (const uint16_t*)zs;
      // Z with tokens along the k slots: 32 kk + 4 lq + 0..3 and + 16
      u32x4 zf[NB / 2][NZ];
#pragma unroll
      for (int kk = 0; kk < NB / 2; ++kk) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
          const uint16_t* zp = zl + (32 * kk + 4 * lq + (lr >> 2)) * ZS +
                               S::zcol(wave, nz, 4 * (lr & 3));
          const u32x2 z0 = lds_read_tr16(zp), z1 = lds_read_tr16(zp + 16 * ZS);
          zf[kk][nz] = (u32x4){z0[0], z0[1], z1[0], z1[1]};
        }
      }
      auto row_frag = [&](const uint16_t* base, int i, int kk) {
        const uint16_t* q = base + i * YS + 32 * kk + 4 * lq;
        const u32x2 q0 = *(const u32x2*)q, q1 = *(const u32x2*)(q + 16);
        return (u32x4){q0[0], q0[1], q1[0], q1[1]};
      };
      if constexpr (OUT) {
        u32x4 mb[NY / 2][NZ];
#pragma unroll
        for (int kk = 0; kk < NY / 2; ++kk) {
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) {
            const f32x4 m0 = m[2 * kk][nz], m1 = m[2 * kk + 1][nz];
            mb[kk][nz] = (u32x4){pack_bf16(m0[0], m0[1]), pack_bf16(m0[2], m0[3]),
                                 pack_bf16(m1[0], m1[1]), pack_bf16(m1[2], m1[3])};
          }
        }
#pragma unroll
        for (int tb = 0; tb < NB; ++tb) {
          u32x4 xf[NY / 2];
          f32x4 o[NZ] = {};
#pragma unroll
          for (int kk = 0; kk < NY / 2; ++kk) {
            xf[kk] = row_frag(xl, 16 * tb + lr, kk);
#pragma unroll
            for (int nz = 0; nz < NZ; ++nz) o[nz] = mfma_bf16(mb[kk][nz], xf[kk], o[nz]);
          }
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) o[nz] *= ex[tb];
#pragma unroll
          for (int sp = 0; sp <= tb / 2; ++sp) {
            f32x4 d[2] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int sb = 2 * sp + e;
              if (sb <= tb) {
#pragma unroll
                for (int kk = 0; kk < NY / 2; ++kk)
                  d[e] = mfma_bf16(row_frag(yl, 16 * sb + lr, kk), xf[kk], d[e]);
                // where j > i the score is selected away, never multiplied by 0
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  d[e][r] = (sb < tb || lr >= 4 * lq + r) ? d[e][r] * dec[tb - sb][r] : 0.0f;
              }
            }
            const u32x4 pf = {pack_bf16(d[0][0], d[0][1]), pack_bf16(d[0][2], d[0][3]),
                              pack_bf16(d[1][0], d[1][1]), pack_bf16(d[1][2], d[1][3])};
#pragma unroll
            for (int nz = 0; nz < NZ; ++nz) o[nz] = mfma_bf16(zf[sp][nz], pf, o[nz]);
          }
          store_out(tb, o);
        }
      }
      // M = lam^n M + Y^T (wz o Z), the decayed Z as two bf16 terms
      u32x4 zh[NB / 2][NZ], zlo[NB / 2][NZ];
#pragma unroll
      for (int kk = 0; kk < NB / 2; ++kk) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t u = zf[kk][nz][e];
            const float* f = wz[2 * kk + e / 2] + 2 * (e % 2);
            split_bf16(bf16_lo(u) * f[0], bf16_hi(u) * f[1], hi[e], lo[e]);
          }
          zh[kk][nz] = make_u32x4(hi);
          zlo[kk][nz] = make_u32x4(lo);
        }
      }
#pragma unroll
      for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
          for (int r = 0; r < 4; ++r) m[yb][nz][r] = times(lam_n, m[yb][nz][r]);
        }
#pragma unroll
        for (int kk = 0; kk < NB / 2; ++kk) {
          const uint16_t* yp = yl + (32 * kk + 4 * lq + (lr >> 2)) * YS + 16 * yb + 4 * (lr & 3);
          const u32x2 y0 = lds_read_tr16(yp), y1 = lds_read_tr16(yp + 16 * YS);
          const u32x4 yf = {y0[0], y0[1], y1[0], y1[1]};
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) {
            m[yb][nz] = mfma_bf16(yf, zh[kk][nz], m[yb][nz]);
            m[yb][nz] = mfma_bf16(yf, zlo[kk][nz], m[yb][nz]);
          }
        }
      }
    } else {
      const float* xl = (const float*)xs;
      const float* yl = (const float*)ys;
      const float* zl = (const float*)zs;
      f32x4 zf[NB][NZ];
#pragma unroll
      for (int sb = 0; sb < NB; ++sb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            zf[sb][nz][r] = zl[(16 * sb + 4 * lq + r) * ZS + S::zcol(wave, nz, lr)];
        }
      }
      if constexpr (OUT) {
#pragma unroll
        for (int tb = 0; tb < NB; ++tb) {
          f32x4 xf[NY], o[NZ] = {};
#pragma unroll
          for (int yb = 0; yb < NY; ++yb) {
            xf[yb] = *(const f32x4*)(xl + (16 * tb + lr) * YS + 16 * yb + 4 * lq);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
              for (int nz = 0; nz < NZ; ++nz) o[nz] = mfma_f32(m[yb][nz][r], xf[yb][r], o[nz]);
            }
          }
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) o[nz] *= ex[tb];
#pragma unroll
          for (int sb = 0; sb <= tb; ++sb) {
            f32x4 d = {};
#pragma unroll
            for (int yb = 0; yb < NY; ++yb) {
              const f32x4 yf = *(const f32x4*)(yl + (16 * sb + lr) * YS + 16 * yb + 4 * lq);
#pragma unroll
              for (int r = 0; r < 4; ++r) d = mfma_f32(yf[r], xf[yb][r], d);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              d[r] = (sb < tb || lr >= 4 * lq + r) ? d[r] * dec[tb - sb][r] : 0.0f;
#pragma unroll
              for (int nz = 0; nz < NZ; ++nz) o[nz] = mfma_f32(zf[sb][nz][r], d[r], o[nz]);
            }
          }
          store_out(tb, o);
        }
      }
#pragma unroll
      for (int sb = 0; sb < NB; ++sb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
          for (int r = 0; r < 4; ++r) zf[sb][nz][r] *= wz[sb][r];
        }
      }
#pragma unroll
      for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
          for (int r = 0; r < 4; ++r) m[yb][nz][r] = times(lam_n, m[yb][nz][r]);
        }
#pragma unroll
        for (int sb = 0; sb < NB; ++sb) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float yv = yl[(16 * sb + 4 * lq + r) * YS + 16 * yb + lr];
#pragma unroll
            for (int nz = 0; nz < NZ; ++nz) m[yb][nz] = mfma_f32(yv, zf[sb][nz][r], m[yb][nz]);
          }
        }
      }
    }
  }

  if constexpr (OUT) {
    if (w.end != nullptr && run.r == run.nruns - 1) {
#pragma unroll
      for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            w.end[sbase + (16 * yb + 4 * lq + r) * ZD + S::zcol(wave, nz, lr)] = m[yb][nz][r];
        }
      }
    }
  } else {
    float* slot = w.slots + ((run.slot + 1) * H + h) * YD * ZD;
#pragma unroll
    for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
      for (int nz = 0; nz < NZ; ++nz)
        *(f32x4*)(slot + ((yb * NZ + nz) * kThreads + tid) * 4) = m[yb][nz];
    }
  }
}

// Workgroup (item, head, walk), the walk fastest, then the head: what shares
// operands runs on one XCD at about the same time.
template <int K, int V, bool BF16, int NW, bool OUT>
__global__ __launch_bounds__(kThreads) void walk_kernel(Walks ws, Seqs sq,
                                                        const float* __restrict__ log_decay,
                                                        int H) {
  using SA = Shape2<K, V, BF16>;
  using SB = Shape2<V, K, BF16>;
  constexpr int XA = (OUT ? 2 : 1) * SA::XBYTES + SA::ZBYTES;
  constexpr int XB = (OUT ? 2 : 1) * SB::XBYTES + SB::ZBYTES;
  __shared__ __attribute__((aligned(16))) char lds[NW == 1 || XA > XB ? XA : XB];
  const int id = xcd_map(blockIdx.x, gridDim.x);
  const Walk& w = ws.w[NW == 1 ? 0 : id % NW];
  const int h = id / NW % H, item = id / NW / H;
  const Run run = find_run(sq, item);
  if (run.seq < 0 || (!OUT && run.r + 1 >= run.nruns)) return;
  if constexpr (NW == 1 || K == V) {
    walk_run<K, V, BF16, OUT>(w, sq, run, log_decay, h, H, lds);
  } else {
    if (w.turned)
      walk_run<V, K, BF16, OUT>(w, sq, run, log_decay, h, H, lds);
    else
      walk_run<K, V, BF16, OUT>(w, sq, run, log_decay, h, H, lds);
  }
}

// M at the start of each run of the sequences that have more than one:
// slot 0 = start, slot r = lam^run slot r-1 + slot r.  One thread per four
// elements; blockIdx.x = (walk, head, part of the state), blockIdx.y strides over
// the sequences.
template <int K, int V, bool BF16>
__global__ __launch_bounds__(kThreads) void run_starts_kernel(Walks ws, Seqs sq,
                                                              const float* __restrict__ log_decay,
                                                              int H) {
  constexpr int PARTS = K * V / 4 / kThreads;
  const int part = blockIdx.x % PARTS, h = blockIdx.x / PARTS % H;
  const Walk& w = ws.w[blockIdx.x / PARTS / H];
  const int tid = threadIdx.x, wave = tid / kWave, lr = tid & 15, lq = (tid % kWave) >> 4;
  const Power lam = power(log_decay, h, sq.run);
  for (int i = blockIdx.y; i < sq.nseq; i += gridDim.y) {
    const int64_t t0 = sq.at(i), len = sq.at(i + 1) - t0;
    if (len <= sq.run) continue;
    const int nruns = (int)((len + sq.run - 1) / sq.run);
    float* slot = w.slots + (2 * t0 / sq.run * H + h) * K * V + (part * kThreads + tid) * 4;
    const int64_t step = (int64_t)H * K * V;
    f32x4 m = {0.0f, 0.0f, 0.0f, 0.0f};
    if (w.start != nullptr) {
      const float* start = w.start + ((int64_t)i * H + h) * K * V;
      // `part` is yb NZ + nz of the walk's own shape
      if (w.turned) {
        using S = Shape2<V, K, BF16>;
        const int y = 16 * (part / S::NZ) + 4 * lq, z = S::zcol(wave, part % S::NZ, lr);
        m = *(const f32x4*)(start + z * V + y);
      } else {
        using S = Shape2<K, V, BF16>;
        const int y = 16 * (part / S::NZ) + 4 * lq, z = S::zcol(wave, part % S::NZ, lr);
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r] = start[(y + r) * V + z];
      }
    }
    *(f32x4*)slot = m;
#pragma unroll 4
    for (int r = 1; r < nruns; ++r) {
      const f32x4 add = *(const f32x4*)(slot + r * step);
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = times(lam, m[e]) + add[e];
      *(f32x4*)(slot + r * step) = m;
    }
  }
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

// Tokens of a run: two workgroups per CU over all walks, whole chunks, and
// at least four chunks (the states at a run's ends cost about as much traffic
// as four chunks' tokens).
constexpr int64_t kWantRuns = 512;
constexpr int64_t kMinChunks = 4;

int run_tokens(const LinattnShape& s, bool bf16, int walks) {
  const int64_t C = bf16 ? 64 : 32;
  const int64_t all = s.tokens * s.nheads * walks;
  int64_t chunks = (all + kWantRuns * C - 1) / (kWantRuns * C);
  if (chunks < kMinChunks) chunks = kMinChunks;
  const int64_t most = (s.tokens + C - 1) / C;
  return (int)((chunks < most ? chunks : most) * C);
}

int64_t slots_of(const LinattnShape& s, int run) {
  return s.tokens <= run ? 0 : 2 * s.tokens / run + 2;
}

template <int K, int V, bool BF16, int NW>
int launch_walks(const Walks& w, const Seqs& sq, const float* ld, const LinattnShape& s,
                 hipStream_t st) {
  const int H = (int)s.nheads;
  const int64_t items = s.tokens / sq.run + s.nseq;
  const dim3 grid((unsigned)(items * H * NW)), block(kThreads);
  // no sequence of these is longer than a run
  const bool whole = (sq.cu == nullptr ? sq.len : s.tokens) <= sq.run;
  if (!whole) {
    hipLaunchKernelGGL((walk_kernel<K, V, BF16, NW, false>), grid, block, 0, st, w, sq, ld, H);
    const unsigned parts = (unsigned)(K * V / 4 / kThreads * H * NW);
    hipLaunchKernelGGL((run_starts_kernel<K, V, BF16>),
                       dim3(parts, (unsigned)(s.nseq < 8 ? s.nseq : 8)), block, 0, st, w, sq, ld,
                       H);
  }
  hipLaunchKernelGGL((walk_kernel<K, V, BF16, NW, true>), grid, block, 0, st, w, sq, ld, H);
  return (int)hipGetLastError();
}

template <int NW>
int walks_of(const Walks& w, const Seqs& sq, const float* ld, bool bf16, const LinattnShape& s,
             hipStream_t st) {
  auto go = [&](auto k, auto v) {
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    return bf16 ? launch_walks<K, V, true, NW>(w, sq, ld, s, st)
                : launch_walks<K, V, false, NW>(w, sq, ld, s, st);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  if (s.dk == 64) return s.dv == 64 ? go(I64{}, I64{}) : go(I64{}, I128{});
  return s.dv == 64 ? go(I128{}, I64{}) : go(I128{}, I128{});
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

Seqs seqs_of(const int32_t* cu, const LinattnShape& s, int run) {
  return Seqs{cu, s.tokens, s.tokens / s.nseq, (int)s.nseq, run};
}

size_t slot_floats(const LinattnShape& s, int run) {
  return (size_t)slots_of(s, run) * s.nheads * s.dk * s.dv;
}

}  // namespace

size_t linattn_workspace(const LinattnShape& s, bool bf16, bool backward) {
  const int walks = backward ? 3 : 1;
  size_t n = slot_floats(s, run_tokens(s, bf16, walks)) * walks;
  if (backward && s.grouped()) n += 2 * (size_t)s.tokens * s.nheads * s.dk;
  return 16 + sizeof(float) * n;
}

int launch_linattn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                       const float* init, const int32_t* cu, void* o, float* fin, void* ws,
                       float scale, bool bf16, const LinattnShape& s, void* stream) {
  clear_launch_error();
  const int share = (int)(s.nheads / s.ngroups);
  Walks w{};
  w.w[0] = Walk{q, k, v, o, init, fin, (float*)ws, share, share, 1, 1, scale, 1.0f, false, false,
                false};
  return walks_of<1>(w, seqs_of(cu, s, run_tokens(s, bf16, 1)), log_decay, bf16, s,
                     (hipStream_t)stream);
}

int launch_linattn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                       const float* init, const int32_t* cu, const void* dout,
                       const float* dfinal, void* dq, void* dk, void* dv, float* dinit,
                       void* ws, float scale, bool bf16, const LinattnShape& s, void* stream) {
  clear_launch_error();
  hipStream_t st = (hipStream_t)stream;
  const int share = (int)(s.nheads / s.ngroups);
  const bool parts = s.grouped();
  const int run = run_tokens(s, bf16, 3);
  const size_t one = slot_floats(s, run);
  float* slots = (float*)ws;
  float* pq = slots + 3 * one;
  float* pk = pq + (size_t)s.tokens * s.nheads * s.dk;
  const Seqs sq = seqs_of(cu, s, run);
  Walks w{};
  w.w[0] = Walk{dout, v,     k, parts ? (void*)pq : dq, init, nullptr, slots,
                1,    1, share, parts ? 1 : share,      scale, 1.0f,   false, true, parts};
  w.w[1] = Walk{v, dout,  q, parts ? (void*)pk : dk, dfinal, nullptr, slots + one,
                1, 1, share, parts ? 1 : share,      1.0f,   scale,   true, true, parts};
  w.w[2] = Walk{k,     q,     dout, dv, dfinal, dinit, slots + 2 * one,
                share, share, 1,    1,  1.0f,   scale, true, false, false};
  int err = walks_of<3>(w, sq, log_decay, bf16, s, st);
  if (err == 0 && parts) err = sum_heads(pq, dq, sq, bf16, s, st);
  if (err == 0 && parts) err = sum_heads(pk, dk, sq, bf16, s, st);
  return err;
}

}  // namespace ssd
