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
//     consecutive j), the blocks on and below the diagonal shared out among the
//     waves; decayed and masked by a select they go through LDS, in slot order
//     again, to every wave; Z comes from the LDS transpose read;
//   - the output comes out transposed too, one token and 8 (fp32, or 64 columns: 4)
//     consecutive columns per lane: 16- or 8-byte stores.
// bf16 tensors: 16x16x32 bf16 products, chunks of 64.  Every operand that is not a
// tensor itself is split into two bf16 terms, which leave 2^-16 of it at most: the
// scores, M in X^T M (one term would leave 2^-8 |X|^T |M|, which is not small beside
// an output whose products cancel: keys of one mean and queries that sum to zero gave
// outputs off by a tenth) and the decayed Z in M's update (three where M goes on to
// an fp32 state in memory: the product is then as exact as an fp32 one).  fp32 tensors:
// 16x16x4 fp32 products, chunks of 32 (the scores' share grows with the chunk, and these
// calls are bound by the matrix pipe).
//
// The chains of a call are few (sequences x heads) and long, so each is cut
// into runs of equal numbers of chunks, walked at once by the two or three
// workgroups a CU holds:
//   1. run_states: M at the end of the first run, and what every later run but
//      the last adds to M from zero, into a slot each;
//   2. run_starts, for sequences of more than kFold runs: M at the start of every
//      run, in place (lam^run from run to run, an element per thread);
//   3. walks: the runs.  In a sequence of few runs each walk goes through the
//      slots before its own itself.
// A call whose chains are all no longer than a run goes straight to 3.  The
// powers of lam that are multiplied up along a chain are taken in 64 bits and
// kept as two fp32 terms, or corrected from chunk to chunk: the rounding of one
// factor would otherwise grow with the number of chunks.
//
// Measured on MI355X (bf16; a device copy moves 5.1 TB/s; kernels under the profiler).
// 8 x 2048 tokens, 16 heads of 128 x 128: run_states 40 us, walks 92 us (300 MB: 3.3
// TB/s).  Gradients of 16384 tokens, 32 heads of 128 x 128: run_states 153 us, the three
// walks 435 us (1.5 GB: 3.4 TB/s; matrix pipe 26% busy, vector unit 35%, LDS 27%).
// 65536 tokens, 32 heads of 128 x 64 on one group: run_states 141 us, walks 328 us; there q
// and k come from the caches, and the LDS (49% busy), the vector unit (44%) and
// the matrix pipe (27%) bound it together.
#include "ssd_block_launch.h"
#include "ssd_device.h"
#include "ssd_host.h"

#include <climits>
#include <type_traits>

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
// A walk goes through the slots before its own itself in sequences of up to this
// many runs: up to kFold - 1 slots are then read by each run, where run_starts reads
// and writes each once and costs a launch.  8 sequences of 2048 tokens, 16 heads of 128 x
// 128, which are 4 runs each: 110 us against 118 with run_starts for all.  Where the host
// does not know the lengths (cu_seqlens) the launch is made whenever the tokens would
// be enough for more runs in one sequence, and passes the shorter ones by, some 5 us: 115
// us there, against 120.
constexpr int kFold = 4;
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kPastRange = 0x7FFF0000u;

// One walk.  Head h of an operand is its head h / share.
struct Walk {
  const void *x, *y, *z;
  void* out;            // rows of the element type, or fp32 partial rows per head
  const float* start;   // [nseq, H, K, V] or null
  float* end;           // [nseq, H, K, V] or null
  float* slots;         // states at the runs' starts, in accumulator order
  float* slots_t;       // the slots of the walk with the transposed M, or null
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
  int nseq, run, chunk;
  __device__ __forceinline__ int64_t at(int i) const {
    if (cu == nullptr) return i * len;
    const int64_t v = cu[i];
    return v < 0 ? 0 : v > tokens ? tokens : v;
  }
};

// Tokens of each run of a sequence of `len`: at most s.run, whole chunks, the
// same for all runs but the last.
__device__ __forceinline__ int run_length(const Seqs& s, int64_t len) {
  const int64_t chunks = (len + s.chunk - 1) / s.chunk;
  const int64_t n = (len + s.run - 1) / s.run;
  return n > 1 ? (int)((chunks + n - 1) / n) * s.chunk : s.run;
}

// A workgroup's run: sequence, its first token and length, the run's number,
// how many there are and how many tokens each has; seq < 0: none.
struct Run {
  int seq, r, nruns, each;
  int64_t t0, len;
  int64_t slot;           // of the sequence's first run
};

// Sequences that begin at or before the item: a search in which every thread tests
// the last of its share of those in question (one round up to 256 sequences, two up
// to 65536).
__device__ __forceinline__ Run find_run(const Seqs& s, int item) {
  int before = 0, left = s.nseq;
  while (left > 0) {
    const int share = (left + kThreads - 1) / kThreads, end = before + left;
    const int i = before + ((int)threadIdx.x + 1) * share - 1;
    before += share * __syncthreads_count(i < end && s.at(i) / s.run + i <= item);
    left = share - 1 < end - before ? share - 1 : end - before;
  }
  Run out{before - 1, 0, 0, 0, 0, 0, 0};
  if (out.seq < 0) return out;
  out.t0 = s.at(out.seq);
  const int64_t end = s.at(out.seq + 1);
  out.len = end > out.t0 ? end - out.t0 : 0;
  out.each = run_length(s, out.len);
  out.nruns = out.len > out.each ? (int)((out.len + out.each - 1) / out.each) : 1;
  const int64_t r = item - (out.t0 / s.run + out.seq);
  out.r = (int)r;
  out.slot = 2 * out.t0 / s.run;
  if (r < 0 || r >= out.nruns) out.seq = -1;
  return out;
}

// log_decay of a head, and log2 of lam.  The clamp keeps a head without memory
// (-inf) from giving 0 * inf: e^(-1e30) is 0 and e^0 is 1.  NaN stays NaN.
__device__ __forceinline__ float decay_of(const float* ld, int h) {
  return ld[h] < -1e30f ? -1e30f : ld[h];
}
__device__ __forceinline__ float log2_decay(const float* ld, int h) {
  return decay_of(ld, h) * kLog2e;
}
// lam^n as two fp32 terms.
struct Power {
  float hi, lo;
};
__device__ __forceinline__ Power power(const float* ld, int h, int n) {
  const double d = exp((double)decay_of(ld, h) * (double)n);
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
  static constexpr int YS = BF16 ? YD + 16 : YD + 4;
  static constexpr int ZS = BF16 ? (ZD == 128 ? 144 : 72) : ZD + 4;
  static constexpr int PS = BF16 ? C + 8 : C + 4;
  static constexpr int XBYTES = C * YS * ES;
  static constexpr int ZBYTES = C * ZS * ES;
  static constexpr int PBYTES = (BF16 ? 2 : 1) * C * PS * ES;   // the scores, bf16 as two terms
  // A 128 x 128 M leaves registers for two workgroups of a CU only, whose LDS has
  // room for the scores beside X (a barrier less per chunk) and whose registers
  // have some left for the decays: 1 to 2% of such a walk.  The others have room for three
  // (resident() says which take them) by letting the scores take X's place and the
  // decays wait in LDS.
  static constexpr bool ROOMY = YD == 128 && ZD == 128;
  static constexpr int DBYTES = 3 * kWave * 16;                 // decays, four per lane
  static constexpr int WBYTES = C * 4;                          // the weights of Z
  static constexpr int XPBYTES =
      ROOMY ? XBYTES + PBYTES : XBYTES > PBYTES ? XBYTES : PBYTES;   // X and the scores
  static constexpr int BADBYTES = 16 + ZD * 4;                  // values that are not finite
  static constexpr int BYTES =
      WBYTES + XBYTES + ZBYTES + XPBYTES + (ROOMY ? 0 : DBYTES) + BADBYTES;
  static constexpr int STATE_BYTES = XBYTES + ZBYTES + WBYTES;
  static constexpr int YU = C * YD * ES / 16 / kThreads;   // 16-byte units per thread
  static constexpr int ZU = C * ZD * ES / 16 / kThreads;
  // Column of M that row (or lane) rho of a wave's column block nz stands for.
  static __device__ __forceinline__ int zcol(int wave, int nz, int rho) {
    if constexpr (BF16) return 16 * NZ * wave + 4 * NZ * (rho >> 2) + 4 * nz + (rho & 3);
    return 16 * NZ * wave + 16 * nz + rho;
  }
  // Place of M[y][z] in a slot: blocks (yb, nz) of a value per thread and row.
  static __device__ __forceinline__ int order(int y, int z) {
    const int wave = z / (16 * NZ), in = z % (16 * NZ);
    const int nz = BF16 ? in % (4 * NZ) / 4 : in / 16;
    const int rho = BF16 ? in / (4 * NZ) * 4 + in % 4 : in % 16;
    const int thread = wave * kWave + (y % 16) / 4 * 16 + rho;
    return ((y / 16 * NZ + nz) * kThreads + thread) * 4 + y % 4;
  }
};

// Place of column c of a bf16 row that is read along the k slots of a product:
// within 32 columns, the slots of one lane group (columns 4 g + 0..3 and 16 on)
// side by side, so that a lane reads its eight with one 16-byte load (two 8-byte
// loads of a row take twice the LDS cycles, 16 against 8 of a wave). Four
// columns stay together.
__device__ __forceinline__ int slot_of(int c) {
  return (c & ~31) + 8 * ((c >> 2) & 3) + 4 * ((c >> 4) & 1) + (c & 3);
}

// A tile of `n` token rows in the walk's order: its descriptor and each
// thread's units.
template <int D, int C, int ES, int U>
struct Tile {
  u32x4 v[U];
  __device__ __forceinline__ void issue(const void* base, int64_t heads, int head, int64_t lowest,
                                        int n, bool down, int tid) {
    const uint32_t row = (uint32_t)(heads * D * ES);
    const rsrc_t r = make_rsrc((const char*)base + (lowest * heads + head) * (D * ES),
                               (uint32_t)(n - 1) * row + D * ES);
    constexpr int PER = D * ES / 16, STEP = kThreads / PER;    // units of a row, rows at a time
    const int i = tid / PER, c = tid % PER;
    // (one form for whole and ragged tiles: a branch here keeps the loads from being
    // spread over the products around them, and costs 10% of a 128 x 128 walk)
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int ij = i + j * STEP;
      const uint32_t off = (uint32_t)(down ? n - 1 - ij : ij) * row + c * 16;
      v[j] = load_b128(r, ij < n ? off : kPastRange);
    }
  }
  template <bool SLOTS>
  __device__ __forceinline__ void commit(char* lds, int stride, int tid) const {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      constexpr int PER = D * ES / 16, STEP = kThreads / PER;
      const int c = tid % PER;
      char* row = lds + (tid / PER + j * STEP) * stride * ES;
      if constexpr (SLOTS) {
        *(u32x2*)(row + slot_of(8 * c) * 2) = (u32x2){v[j][0], v[j][1]};
        *(u32x2*)(row + slot_of(8 * c + 4) * 2) = (u32x2){v[j][2], v[j][3]};
      } else {
        *(u32x4*)(row + c * 16) = v[j];
      }
    }
  }
};

// The output rows of a chunk: block (tb, nz) holds token 16 tb + lr of the
// chunk and four columns of the wave's block nz.
template <int YD, int ZD, bool BF16, int NB, int NZ>
__device__ __forceinline__ void store_rows(const Walk& w, const f32x4 (&o)[NB][NZ],
                                           int64_t lowest, int n, int h, int H, int wave,
                                           int lr, int lq) {
  using S = Shape2<YD, ZD, BF16>;
  const int64_t oheads = H / w.oshare;
  const bool f32o = !BF16 || w.f32out;
  const int oes = f32o ? 4 : 2;
  const uint32_t orow = (uint32_t)(oheads * ZD * oes);
  const rsrc_t orr = make_rsrc((char*)w.out + (lowest * oheads + h / w.oshare) * (ZD * oes),
                               (uint32_t)(n - 1) * orow + ZD * oes);
#pragma unroll
  for (int tb = 0; tb < NB; ++tb) {
    const int i = 16 * tb + lr;
    const uint32_t at = i < n ? (uint32_t)(w.down ? n - 1 - i : i) * orow : kPastRange;
    if (f32o) {
#pragma unroll
      for (int nz = 0; nz < NZ; ++nz)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[tb][nz]), orr,
                                               (int)(at + S::zcol(wave, nz, 4 * lq) * 4), 0, 0);
    } else {
      const int off = (int)(at + S::zcol(wave, 0, 4 * lq) * 2);
      const u32x2 a = {pack_bf16(o[tb][0][0], o[tb][0][1]), pack_bf16(o[tb][0][2], o[tb][0][3])};
      if constexpr (NZ == 2) {
        const u32x2 b = {pack_bf16(o[tb][1][0], o[tb][1][1]),
                         pack_bf16(o[tb][1][2], o[tb][1][3])};
        __builtin_amdgcn_raw_buffer_store_b128((u32x4){a[0], a[1], b[0], b[1]}, orr, off, 0, 0);
      } else {
        __builtin_amdgcn_raw_buffer_store_b64(a, orr, off, 0, 0);
      }
    }
  }
}

// Values of Z that are not finite.  In the scores' product a value stands beside
// scores of 0 for the tokens before it, and 0 times it would reach them.  So a
// thread that brings one takes it out of the tile and notes its token for its
// column; the outputs of the column are NaN from that token on, and so is M's column at
// the end.  (Looking for them costs 1 to 2% of a walk; done on the operand as a wave
// reads it, whose registers it lengthens, up to 10%.)
template <bool BF16, int U>
__device__ __forceinline__ bool holds_bad(const u32x4 (&v)[U]) {
  if constexpr (BF16) {
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < 4 * U; ++i)
      top = __builtin_elementwise_max(top,
                                      __builtin_bit_cast(u16x2, v[i / 4][i % 4] & 0x7FFF7FFFu));
    return top[0] >= 0x7F80 || top[1] >= 0x7F80;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4 * U; ++i) top = max(top, v[i / 4][i % 4] & 0x7FFFFFFFu);
  return top >= 0x7F800000u;
}
// The thread's own values of the tile, whose first token is the walk's p-th.
template <int ZD, int ZS, int U, typename T>
__device__ __forceinline__ void take_out_bad(T* zs, int* first, int* bad, int p, int tid) {
  constexpr int PER = ZD * sizeof(T) / 16, STEP = kThreads / PER, E = 16 / sizeof(T);
  constexpr T INF = (T)(sizeof(T) == 2 ? 0x7F80u : 0x7F800000u);
#pragma nounroll
  for (int u = 0; u < U * E; ++u) {
    const int i = tid / PER + u / E * STEP, c = tid % PER * E + u % E;
    if ((zs[i * ZS + c] & INF) == INF) {
      zs[i * ZS + c] = 0;
      atomicMin(first + c, p + i);
      *bad = 1;
    }
  }
}
template <int YD, int ZD, bool BF16>
__device__ __forceinline__ void store_bad(const Walk& w, const int* first, int p, int64_t lowest,
                                          int n, int h, int H, int wave, int lr, int lq) {
  using S = Shape2<YD, ZD, BF16>;
  const int64_t oheads = H / w.oshare;
#pragma nounroll
  for (int c = 0; c < 4 * S::NZ; ++c) {
    const int col = S::zcol(wave, c / 4, 4 * lq + c % 4);
#pragma nounroll
    for (int i = lr; i < n; i += 16) {
      if (p + i < first[col]) continue;
      const int64_t at =
          ((lowest + (w.down ? n - 1 - i : i)) * oheads + h / w.oshare) * ZD + col;
      if (!BF16 || w.f32out)
        ((uint32_t*)w.out)[at] = 0x7FC00000u;
      else
        ((uint16_t*)w.out)[at] = 0x7FC0;
    }
  }
}

// lam^C from chunk to chunk: the factor that brings the product of all factors
// so far nearest to the exact power, so the roundings do not add up.
struct Factor {
  Power p;
  float off;              // relative error of the product
  __device__ __forceinline__ float next() {
    const float t = __builtin_fmaf(-p.hi, off, p.lo);
    const float f = p.hi + t;
    // (a power this small leaves nothing of the chunk before; the reciprocal of a
    // denormal one would be infinite)
    off = p.hi < 1e-30f ? 0.0f : ((f - p.hi) - t) * __builtin_amdgcn_rcpf(p.hi);
    return f;
  }
};

// Four fp32 values as bf16, and what the rounding left, as bf16 again.
__device__ __forceinline__ void split4(const f32x4& v, u32x2& hi, u32x2& lo) {
  uint32_t h0, h1, l0, l1;
  split_bf16(v[0], v[1], h0, l0);
  split_bf16(v[2], v[3], h1, l1);
  hi = (u32x2){h0, h1};
  lo = (u32x2){l0, l1};
}
__device__ __forceinline__ u32x4 join(u32x2 a, u32x2 b) { return (u32x4){a[0], a[1], b[0], b[1]}; }

// One run of one walk; with OUT the outputs too, else only M from zero.
template <int YD, int ZD, bool BF16, bool OUT>
__device__ __forceinline__ void walk_run(const Walk& w, const Seqs& sq, const Run& run,
                                         const float* log_decay, int h, int H, char* lds) {
  using S = Shape2<YD, ZD, BF16>;
  constexpr int C = S::C, NB = S::NB, NY = S::NY, NZ = S::NZ, YS = S::YS, ZS = S::ZS, PS = S::PS;
  constexpr int ES = S::ES;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lr = lane & 15, lq = lane >> 4;
  float* wtab = (float*)lds;
  char* ys = lds + S::WBYTES;
  char* zs = ys + S::XBYTES;
  char* xs = zs + S::ZBYTES;
  char* ps = S::ROOMY ? xs + S::XBYTES : xs;
  f32x4* dtab = (f32x4*)(xs + S::XPBYTES);
  int* bad = (int*)(lds + S::BYTES - S::BADBYTES);   // whether there was one
  int* first = bad + 4;                              // its token, per column

  // Whether M goes on to a state in memory, where fp32 is asked for, or only
  // into outputs of the tensors' type.
  const bool exact = w.end != nullptr && run.r == run.nruns - 1;
  const float l2 = log2_decay(log_decay, h);
  const int a = w.down ? 0 : 1;
  const int64_t p0 = (int64_t)run.r * run.each;
  const int len = (int)(run.len - p0 < run.each ? run.len - p0 : run.each);

  // M[y][z]: block (yb, nz) holds rows 16 yb + 4 lq + r, column zcol(nz, lr).
  f32x4 m[NY][NZ];
  const int64_t sbase = ((int64_t)run.seq * H + h) * YD * ZD;
  const int64_t step = (int64_t)H * YD * ZD;               // from slot to slot
  float* slot = w.slots + run.slot * step + (int64_t)h * YD * ZD + tid * 4;
  // States taken on in place: the first run's start is kept in slot 0, because
  // the last run may write its end before the first has read it.
  const bool kept = w.start != nullptr && w.start == w.end && run.nruns > 1;
  if (OUT && run.nruns > 1 && (run.r > 0 || kept)) {
    const bool folded = run.nruns <= kFold;
    const int from = run.r == 0 ? 0 : folded ? 1 : run.r;
#pragma unroll
    for (int i = 0; i < NY * NZ; ++i)
      m[i / NZ][i % NZ] = *(const f32x4*)(slot + from * step + i * kThreads * 4);
    if (folded && run.r > 1) {
      const Power lam = power(log_decay, h, run.each);
      for (int r = 2; r <= run.r; ++r) {
#pragma unroll
        for (int i = 0; i < NY * NZ; ++i) {
          const f32x4 add = *(const f32x4*)(slot + r * step + i * kThreads * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m[i / NZ][i % NZ][e] = times(lam, m[i / NZ][i % NZ][e]) + add[e];
        }
      }
    }
  } else if (run.r == 0 && w.start != nullptr && w.turned) {
#pragma unroll
    for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
      for (int nz = 0; nz < NZ; ++nz)
        m[yb][nz] = *(const f32x4*)(w.start + sbase + S::zcol(wave, nz, lr) * YD + 16 * yb +
                                    4 * lq);
    }
  } else if (run.r == 0 && w.start != nullptr) {
#pragma unroll
    for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
      for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          m[yb][nz][r] =
              w.start[sbase + (16 * yb + 4 * lq + r) * ZD + S::zcol(wave, nz, lr)];
      }
    }
  } else {
#pragma unroll
    for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
      for (int nz = 0; nz < NZ; ++nz) m[yb][nz] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }
  }
  if constexpr (!OUT) {
    if (run.r == 0 && kept) {
#pragma unroll
      for (int i = 0; i < NY * NZ; ++i) *(f32x4*)(slot + i * kThreads * 4) = m[i / NZ][i % NZ];
    }
  }

  // Per lane: the decays of its four scores in a diagonal block, in the block below
  // it, and those of X^T M for its token of each block.
  f32x4 d0 = {}, d1 = {}, dx = {};
  if (OUT && (S::ROOMY || wave == 0)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = lr - 4 * lq - r;
      d0[r] = d >= 0 ? w.cx * w.cz * exp2_hw(l2 * (float)d) : 0.0f;
      d1[r] = w.cx * w.cz * exp2_hw(l2 * (float)(16 + d));
      if (r < NB) dx[r] = w.cx * exp2_hw(l2 * (float)(16 * r + lr + a));
    }
    if constexpr (!S::ROOMY) {
      dtab[lane] = d0;
      dtab[kWave + lane] = d1;
      dtab[2 * kWave + lane] = dx;
    }
  }
  Factor lam{power(log_decay, h, C), 0.0f};
  if (OUT && tid < ZD) {
    *bad = 0;
    first[tid] = INT_MAX;
  }

  Tile<YD, C, ES, S::YU> tx, ty;
  Tile<ZD, C, ES, S::ZU> tz;
  auto lowest_of = [&](int p, int n) {
    return w.down ? run.t0 + run.len - p0 - p - n : run.t0 + p0 + p;
  };
  auto issue = [&](int p, int tid) {
    const int n = len - p < C ? len - p : C;
    const int64_t lowest = lowest_of(p, n);
    if constexpr (OUT) tx.issue(w.x, H / w.xshare, h / w.xshare, lowest, n, w.down, tid);
    ty.issue(w.y, H / w.yshare, h / w.yshare, lowest, n, w.down, tid);
    tz.issue(w.z, H / w.zshare, h / w.zshare, lowest, n, w.down, tid);
  };
  if (len > 0) issue(0, tid);
  for (int p = 0; p < len; p += C) {
    const int n = len - p < C ? len - p : C;
    // The thread's addresses are formed anew for every chunk: kept across chunks
    // they would take some 50 registers and be spilled.
    int fresh = tid;
    asm volatile("" : "+v"(fresh));
    const int lr = fresh & 15, lq = fresh >> 4 & 3;
    __syncthreads();
    if constexpr (OUT) tx.template commit<BF16>(xs, YS, fresh);
    ty.template commit<BF16>(ys, YS, fresh);
    tz.template commit<false>(zs, ZS, fresh);
    if (OUT && __builtin_expect(holds_bad<BF16>(tz.v), 0)) {
      using T = std::conditional_t<BF16, uint16_t, uint32_t>;
      take_out_bad<ZD, ZS, S::ZU, T>((T*)zs, first, bad, p, fresh);
    }
    if (tid < C) wtab[tid] = tid < n ? w.cz * exp2_hw(l2 * (float)(n - a - tid)) : 0.0f;
    __syncthreads();
    const bool any_bad = OUT && __builtin_amdgcn_readfirstlane(*bad) != 0;
    if constexpr (!BF16) {
      if (p + C < len) issue(p + C, fresh);
    }

    // Scores of tokens j = 4 lq + 0..3 of a block for token i = lr of the block
    // `apart` blocks on.  Where j > i the score is selected away, never multiplied
    // by 0.
    auto decayed = [&](f32x4& d, int apart) {
      const f32x4 dec = S::ROOMY ? (apart > 0 ? d1 : d0)
                                 : dtab[(apart > 0 ? kWave : 0) + (fresh & (kWave - 1))];
      const float far = exp2_hw(l2 * (float)(16 * (apart > 1 ? apart - 1 : 0)));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = d[r] * (dec[r] * far);
        d[r] = apart > 0 || lr >= 4 * lq + r ? v : 0.0f;
      }
    };
    if constexpr (BF16) {
      const uint16_t* xl = (const uint16_t*)xs;
      const uint16_t* yl = (const uint16_t*)ys;
      const uint16_t* zl = (const uint16_t*)zs;
      uint16_t* ph = (uint16_t*)ps;
      uint16_t* pl = ph + C * PS;
      // eight k slots of row i: columns 32 kk + 4 lq + 0..3 and 16 on
      auto row_frag = [&](const uint16_t* base, int stride, int i, int kk) {
        return *(const u32x4*)(base + i * stride + 32 * kk + 8 * lq);
      };
      f32x4 o[NB][NZ] = {};
      if constexpr (OUT) {
        // (1) the ten score blocks on and below the diagonal, transposed (Y X^T),
        // two or three per wave; where they take X's place they wait until it is read
        u32x2 sh[3], sl[3];
        auto score = [&](int id, u32x2& hi, u32x2& lo) {
          const int tb = id > 5 ? 3 : id > 2 ? 2 : id > 0 ? 1 : 0, sb = id - tb * (tb + 1) / 2;
          f32x4 d = {};
#pragma unroll
          for (int kk = 0; kk < NY / 2; ++kk)
            d = mfma_bf16(row_frag(yl, YS, 16 * sb + lr, kk), row_frag(xl, YS, 16 * tb + lr, kk),
                          d);
          decayed(d, tb - sb);
          split4(d, hi, lo);
        };
        score(wave, sh[0], sl[0]);
        score(wave + 4, sh[1], sl[1]);
        if (wave < 2) score(wave + 8, sh[2], sl[2]);
        auto write_scores = [&] {
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const int id = wave + 4 * e;
            if (id > 9) break;
            const int tb = id > 5 ? 3 : id > 2 ? 2 : id > 0 ? 1 : 0, sb = id - tb * (tb + 1) / 2;
            const int at = (16 * tb + lr) * PS + slot_of(16 * sb) + 8 * lq;
            *(u32x2*)(ph + at) = sh[e];
            *(u32x2*)(pl + at) = sl[e];
            if (sb == tb && tb % 2 == 0) {   // the block above the diagonal is read too
              *(u32x2*)(ph + at + 4) = (u32x2){0, 0};
              *(u32x2*)(pl + at + 4) = (u32x2){0, 0};
            }
          }
        };
        if constexpr (S::ROOMY) write_scores();
        // (2) X^T M, transposed, for all tokens; M as two bf16 terms
#pragma unroll
        for (int kk = 0; kk < NY / 2; ++kk) {
          u32x4 xf[NB];
#pragma unroll
          for (int tb = 0; tb < NB; ++tb) xf[tb] = row_frag(xl, YS, 16 * tb + lr, kk);
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) {
            u32x2 h0, l0, h1, l1;
            split4(m[2 * kk][nz], h0, l0);
            split4(m[2 * kk + 1][nz], h1, l1);
            const u32x4 mt[2] = {join(h0, h1), join(l0, l1)};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int tb = 0; tb < NB; ++tb) o[tb][nz] = mfma_bf16(mt[e], xf[tb], o[tb][nz]);
            }
          }
          // (one slice of M at a time: its terms formed ahead would be spilled by the
          // gradients of 64 x 128 and 128 x 64 states, 2 to 7% of them)
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int tb = 0; tb < NB; ++tb) {
          const float ex = S::ROOMY ? dx[tb] : dtab[2 * kWave + (fresh & (kWave - 1))][tb];
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) o[tb][nz] *= ex;
        }
        if constexpr (!S::ROOMY) {
          __syncthreads();
          write_scores();
        }
        __syncthreads();
      }
      // Z with tokens along the k slots: 32 kk + 4 lq + 0..3 and 16 on
      auto z_frag = [&](int kk, int nz) {
        const uint16_t* zp = zl + (32 * kk + 4 * lq + (lr >> 2)) * ZS +
                             S::zcol(wave, nz, 4 * (lr & 3));
        return join(lds_read_tr16(zp), lds_read_tr16(zp + 16 * ZS));
      };
      // (3) the scores' part of the output
      if constexpr (OUT) {
#pragma unroll
        for (int kk = 0; kk < NB / 2; ++kk) {
          u32x4 zf[NZ];
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) zf[nz] = z_frag(kk, nz);
#pragma unroll
          for (int term = 0; term < 2; ++term) {
#pragma unroll
            for (int tb = 2 * kk; tb < NB; ++tb) {
              const u32x4 pf = row_frag(term ? pl : ph, PS, 16 * tb + lr, kk);
#pragma unroll
              for (int nz = 0; nz < NZ; ++nz) o[tb][nz] = mfma_bf16(zf[nz], pf, o[tb][nz]);
            }
          }
        }
        store_rows<YD, ZD, BF16>(w, o, lowest_of(p, n), n, h, H, wave, lr, lq);
        if (__builtin_expect(any_bad, 0))
          store_bad<YD, ZD, BF16>(w, first, p, lowest_of(p, n), n, h, H, wave, lr, lq);
        __builtin_amdgcn_sched_barrier(0);   // o's registers are free from here on
      }
      if (p + C < len) issue(p + C, fresh);
      // (4) M = lam^n M + Y^T (wz o Z), the decayed Z as two bf16 terms, and a third
      // where `exact`
      const float f = n == C ? lam.next() : exp2_hw(l2 * (float)n);
#pragma unroll
      for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) m[yb][nz] *= f;
      }
      auto update = [&](auto first, auto last) {
        constexpr int T0 = decltype(first)::value, T1 = decltype(last)::value;
#pragma unroll
        for (int kk = 0; kk < NB / 2; ++kk) {
          u32x4 zt[3][NZ];
          const f32x4 w0 = *(const f32x4*)(wtab + 32 * kk + 4 * lq);
          const f32x4 w1 = *(const f32x4*)(wtab + 32 * kk + 16 + 4 * lq);
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) {
            const u32x4 zf = z_frag(kk, nz);
            uint32_t t[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v0 = bf16_lo(zf[e]) * (e < 2 ? w0[2 * e] : w1[2 * e - 4]);
              const float v1 = bf16_hi(zf[e]) * (e < 2 ? w0[2 * e + 1] : w1[2 * e - 3]);
              split3_bf16(v0, v1, t[0][e], t[1][e], t[2][e]);
            }
#pragma unroll
            for (int e = 0; e < 3; ++e) zt[e][nz] = make_u32x4(t[e]);
          }
          constexpr int YG = 4;                // row blocks at a time: independent products
#pragma unroll
          for (int y0 = 0; y0 < NY; y0 += YG) {
            u32x4 yf[YG];
#pragma unroll
            for (int y = 0; y < YG; ++y) {
              const uint16_t* yp = yl + (32 * kk + 4 * lq + (lr >> 2)) * YS + 8 * (lr & 3) +
                                   slot_of(16 * (y0 + y));
              yf[y] = join(lds_read_tr16(yp), lds_read_tr16(yp + 16 * YS));
            }
#pragma unroll
            for (int e = T0; e <= T1; ++e) {
#pragma unroll
              for (int y = 0; y < YG; ++y) {
#pragma unroll
                for (int nz = 0; nz < NZ; ++nz)
                  m[y0 + y][nz] = mfma_bf16(yf[y], zt[e][nz], m[y0 + y][nz]);
              }
            }
          }
        }
      };
      using Term0 = std::integral_constant<int, 0>;
      using Term1 = std::integral_constant<int, 1>;
      using Term2 = std::integral_constant<int, 2>;
      if constexpr (OUT) {
        update(Term0{}, Term1{});
        if (exact) update(Term2{}, Term2{});
      } else {
        update(Term0{}, Term2{});
      }
    } else {
      const float* xl = (const float*)xs;
      const float* yl = (const float*)ys;
      const float* zl = (const float*)zs;
      float* pl = (float*)ps;
      f32x4 o[NB][NZ] = {};
      if constexpr (OUT) {
        // (1) the three score blocks of a chunk, one per wave
        const int tb3 = (wave + 1) / 2, sb3 = wave / 2;
        f32x4 d = {};
        if (wave < 3) {
          const int tb = tb3, sb = sb3;
#pragma unroll
          for (int yb = 0; yb < NY; ++yb) {
            const f32x4 xf = *(const f32x4*)(xl + (16 * tb + lr) * YS + 16 * yb + 4 * lq);
            const f32x4 yf = *(const f32x4*)(yl + (16 * sb + lr) * YS + 16 * yb + 4 * lq);
#pragma unroll
            for (int r = 0; r < 4; ++r) d = mfma_f32(yf[r], xf[r], d);
          }
          decayed(d, tb - sb);
        }
        // (2) X^T M
#pragma unroll
        for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
          for (int tb = 0; tb < NB; ++tb) {
            const f32x4 xf = *(const f32x4*)(xl + (16 * tb + lr) * YS + 16 * yb + 4 * lq);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
              for (int nz = 0; nz < NZ; ++nz) o[tb][nz] = mfma_f32(m[yb][nz][r], xf[r], o[tb][nz]);
            }
          }
        }
#pragma unroll
        for (int tb = 0; tb < NB; ++tb) {
          const float ex = S::ROOMY ? dx[tb] : dtab[2 * kWave + (fresh & (kWave - 1))][tb];
#pragma unroll
          for (int nz = 0; nz < NZ; ++nz) o[tb][nz] *= ex;
        }
        if constexpr (!S::ROOMY) __syncthreads();
        if (wave < 3) *(f32x4*)(pl + (16 * tb3 + lr) * PS + 16 * sb3 + 4 * lq) = d;
        __syncthreads();
      }
      // (3)
      f32x4 zf[NB][NZ];
#pragma unroll
      for (int sb = 0; sb < NB; ++sb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            zf[sb][nz][r] = zl[(16 * sb + 4 * lq + r) * ZS + S::zcol(wave, nz, lr)];
        }
        if constexpr (OUT) {
#pragma unroll
          for (int tb = sb; tb < NB; ++tb) {
            const f32x4 pf = *(const f32x4*)(pl + (16 * tb + lr) * PS + 16 * sb + 4 * lq);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
              for (int nz = 0; nz < NZ; ++nz) o[tb][nz] = mfma_f32(zf[sb][nz][r], pf[r], o[tb][nz]);
            }
          }
        }
        const f32x4 wv = *(const f32x4*)(wtab + 16 * sb + 4 * lq);
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) zf[sb][nz] *= wv;
      }
      const float f = n == C ? lam.next() : exp2_hw(l2 * (float)n);
#pragma unroll
      for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) m[yb][nz] *= f;
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
      if constexpr (OUT) {
        store_rows<YD, ZD, BF16>(w, o, lowest_of(p, n), n, h, H, wave, lr, lq);
        if (__builtin_expect(any_bad, 0))
          store_bad<YD, ZD, BF16>(w, first, p, lowest_of(p, n), n, h, H, wave, lr, lq);
      }
    }
  }

  if constexpr (OUT) {
    if (w.end != nullptr && run.r == run.nruns - 1) {
      if (len > 0 && *bad != 0) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
          if (first[S::zcol(wave, nz, lr)] == INT_MAX) continue;
#pragma unroll
          for (int yb = 0; yb < NY; ++yb) m[yb][nz] += __builtin_nanf("");
        }
      }
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
    slot += (run.r + 1) * step;
#pragma unroll
    for (int i = 0; i < NY * NZ; ++i) *(f32x4*)(slot + i * kThreads * 4) = m[i / NZ][i % NZ];
    if (w.slots_t != nullptr) {
      float* st = w.slots_t + (run.slot + run.r + 1) * step + (int64_t)h * YD * ZD;
      using T = Shape2<ZD, YD, BF16>;
#pragma unroll
      for (int yb = 0; yb < NY; ++yb) {
#pragma unroll
        for (int nz = 0; nz < NZ; ++nz) {
          const int z = S::zcol(wave, nz, lr);
#pragma unroll
          for (int r = 0; r < 4; ++r) st[T::order(z, 16 * yb + 4 * lq + r)] = m[yb][nz][r];
        }
      }
    }
  }
}

// Workgroups of a CU: what the registers leave room for (a workgroup has one wave on
// each SIMD), and the LDS.  Two for a 128 x 128 M, and for outputs of bf16 tensors by a
// 64 x 128 one, whose two column blocks for each wave spill with three (two against three,
// 8 x 2048 tokens, 16 heads: 84 and 110 us; 9000, 5461 and 1923 tokens: 89 and 114).  The
// gradients of 64 x 128 and 128 x 64 states have such a walk too and spill some 25
// registers with three, but keep them: with two the runs, which are whole chunks, can fill
// the CUs less evenly (24 heads on 8 groups, 4 x 2048 tokens: 284 and 300 us; seven
// documents of 41 to 5000 tokens: 424 and 347).  fp32 tensors and an M of 64 columns do
// not spill with three (128 x 64, 65536 tokens, 32 heads: 484 and 439 us).
template <int K, int V, bool BF16, int NW>
constexpr int resident() { return V == 128 && (K == 128 || (BF16 && NW == 1)) ? 2 : 3; }

// Workgroup (item, walk, head), the head fastest.  Blocks are dealt to the 8 XCDs
// in turn, so with H a multiple of 8 every XCD gets the walks of H/8 consecutive
// heads, which share operands.  Items without a run (up to nseq of them) come
// last: in between they would leave CUs with one workgroup and others with three.
template <int K, int V, bool BF16, int NW, bool OUT>
__global__ __launch_bounds__(kThreads, (resident<K, V, BF16, NW>())) void walk_kernel(
    Walks ws, Seqs sq, const float* __restrict__ log_decay, int H) {
  using SA = Shape2<K, V, BF16>;
  using SB = Shape2<V, K, BF16>;
  constexpr int XA = OUT ? SA::BYTES : SA::STATE_BYTES;
  constexpr int XB = OUT ? SB::BYTES : SB::STATE_BYTES;
  __shared__ __attribute__((aligned(16))) char lds[NW == 1 || XA > XB ? XA : XB];
  const int b = (int)(blockIdx.x % H), id = (int)(blockIdx.x / H);
  const int h = H % 8 ? b : b % 8 * (H / 8) + b / 8;
  const Walk& w = ws.w[id % NW];
  const int item = id / NW;
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

// M at the start of each run of the sequences of more than kFold runs: slot r =
// lam^run slot r-1 + slot r, from slot 1 on.  One thread per four elements;
// blockIdx.x = (walk, head, part of the state), blockIdx.y strides over the
// sequences.
__global__ __launch_bounds__(kThreads) void run_starts_kernel(Walks ws, Seqs sq,
                                                              const float* __restrict__ log_decay,
                                                              int H, int state) {
  const int parts = state / 4 / kThreads;
  const int part = blockIdx.x % parts, h = blockIdx.x / parts % H;
  float* slots = ws.w[blockIdx.x / parts / H].slots;
  const int64_t step = (int64_t)H * state;
  for (int i = blockIdx.y; i < sq.nseq; i += gridDim.y) {
    const int64_t t0 = sq.at(i), len = sq.at(i + 1) - t0;
    if (len <= sq.run) continue;
    const int each = run_length(sq, len);
    const int nruns = (int)((len + each - 1) / each);
    if (nruns <= kFold) continue;
    const Power lam = power(log_decay, h, each);
    float* slot = slots + 2 * t0 / sq.run * step + (int64_t)h * state +
                  (part * kThreads + (int)threadIdx.x) * 4;
    f32x4 m = *(const f32x4*)(slot + step);
#pragma unroll 8
    for (int r = 2; r < nruns; ++r) {
      const f32x4 add = *(const f32x4*)(slot + r * step);
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = times(lam, m[e]) + add[e];
      *(f32x4*)(slot + r * step) = m;
    }
  }
}

// Sums the partial rows of the heads of each group, in their order; blockIdx.y:
// which of two gradients.
template <bool BF16>
__global__ __launch_bounds__(256) void sum_heads_kernel(const float* __restrict__ part0,
                                                        void* __restrict__ out0,
                                                        const float* __restrict__ part1,
                                                        void* __restrict__ out1, Seqs sq, int G,
                                                        int share, int D) {
  const float* part = blockIdx.y ? part1 : part0;
  void* out = blockIdx.y ? out1 : out0;
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

// Tokens of a run: whole chunks, as few as keep the runs of all walks within the
// workgroups the 256 CUs hold at once (a few more would wait for a second round),
// with two thirds of a run allowed for the end of each sequence; at least two
// chunks (a shorter run costs more in states and in the launch that forms them
// than it saves).
constexpr int64_t kCus = 256;
constexpr int64_t kMinChunks = 2;

int run_tokens(const LinattnShape& s, bool bf16, int walks) {
  const int64_t C = bf16 ? 64 : 32;
  const bool two = s.dv == 128 && (s.dk == 128 || (bf16 && walks == 1));
  const int64_t wgs = kCus * (two ? resident<128, 128, true, 1>() : resident<64, 64, true, 1>());
  const int64_t each = 3 * wgs / (s.nheads * walks);           // thirds of runs for a head
  const int64_t ends = 2 * s.nseq < each / 2 ? 2 * s.nseq : each / 2;
  int64_t chunks = each > ends ? (3 * s.tokens + (each - ends) * C - 1) / ((each - ends) * C)
                               : (s.tokens + C - 1) / C;
  if (chunks < kMinChunks) chunks = kMinChunks;
  const int64_t most = (s.tokens + C - 1) / C;
  return (int)((chunks < most ? chunks : most) * C);
}

int64_t slots_of(const LinattnShape& s, int run) {
  return s.tokens <= run ? 0 : 2 * s.tokens / run + 2;
}

// `states`: the walks whose runs' states are formed (their slots_t serve the
// others).
template <int K, int V, bool BF16, int NW, int NS>
int launch_walks(const Walks& w, const Walks& states, const Seqs& sq, const float* ld,
                 const LinattnShape& s, hipStream_t st) {
  const int H = (int)s.nheads;
  const int64_t items = s.tokens / sq.run + s.nseq;
  const dim3 block(kThreads);
  const int64_t longest = sq.cu == nullptr ? sq.len : s.tokens;   // that a sequence may be
  if (longest > sq.run) {
    hipLaunchKernelGGL((walk_kernel<K, V, BF16, NS, false>), dim3((unsigned)(items * H * NS)),
                       block, 0, st, states, sq, ld, H);
    if (longest > (int64_t)kFold * sq.run) {
      const unsigned parts = (unsigned)(K * V / 4 / kThreads * H * NW);
      // (workgroups pass sequences of few runs by; of many, most must be)
      const int64_t most = s.nseq < 512 ? 8 : s.nseq < 65536 ? s.nseq / 64 : 1024;
      hipLaunchKernelGGL(run_starts_kernel, dim3(parts, (unsigned)(s.nseq < most ? s.nseq : most)),
                         block, 0, st, w, sq, ld, H, K * V);
    }
  }
  hipLaunchKernelGGL((walk_kernel<K, V, BF16, NW, true>), dim3((unsigned)(items * H * NW)), block,
                     0, st, w, sq, ld, H);
  return (int)hipGetLastError();
}

template <int NW, int NS>
int walks_of(const Walks& w, const Walks& states, const Seqs& sq, const float* ld, bool bf16,
             const LinattnShape& s, hipStream_t st) {
  auto go = [&](auto k, auto v) {
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    return bf16 ? launch_walks<K, V, true, NW, NS>(w, states, sq, ld, s, st)
                : launch_walks<K, V, false, NW, NS>(w, states, sq, ld, s, st);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  if (s.dk == 64) return s.dv == 64 ? go(I64{}, I64{}) : go(I64{}, I128{});
  return s.dv == 64 ? go(I128{}, I64{}) : go(I128{}, I128{});
}

int sum_heads(const float* pq, void* dq, const float* pk, void* dk, const Seqs& sq, bool bf16,
              const LinattnShape& s, hipStream_t st) {
  const int64_t units = s.tokens * s.ngroups * s.dk / 4;
  const unsigned blocks = (unsigned)(units < 256 * 2048 ? (units + 255) / 256 : 2048);
  const int share = (int)(s.nheads / s.ngroups);
  if (bf16)
    hipLaunchKernelGGL((sum_heads_kernel<true>), dim3(blocks, 2), dim3(256), 0, st, pq, dq, pk,
                       dk, sq, (int)s.ngroups, share, (int)s.dk);
  else
    hipLaunchKernelGGL((sum_heads_kernel<false>), dim3(blocks, 2), dim3(256), 0, st, pq, dq, pk,
                       dk, sq, (int)s.ngroups, share, (int)s.dk);
  return (int)hipGetLastError();
}

Seqs seqs_of(const int32_t* cu, const LinattnShape& s, int run, bool bf16) {
  return Seqs{cu, s.tokens, s.tokens / s.nseq, (int)s.nseq, run, bf16 ? 64 : 32};
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
  w.w[0] = Walk{q,     k,     v, o, init,  fin,  (float*)ws, nullptr,
                share, share, 1, 1, scale, 1.0f, false,      false, false};
  return walks_of<1, 1>(w, w, seqs_of(cu, s, run_tokens(s, bf16, 1), bf16), log_decay, bf16, s,
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
  const Seqs sq = seqs_of(cu, s, run, bf16);
  Walks w{}, states{};
  w.w[0] = Walk{dout, v,     k, parts ? (void*)pq : dq, init,  nullptr, slots, nullptr, 1,
                1,    share, parts ? 1 : share,         scale, 1.0f,    false, true,    parts};
  w.w[1] = Walk{v, dout,  q, parts ? (void*)pk : dk, dfinal, nullptr, slots + one, nullptr, 1,
                1, share, parts ? 1 : share,         1.0f,   scale,   true,        true,    parts};
  w.w[2] = Walk{k,     q, dout, dv,   dfinal, dinit, slots + 2 * one, nullptr, share,
                share, 1, 1,    1.0f, scale,  true,  false,           false};
  // dk walks with the transpose of dv's M, whose runs' states serve both
  states.w[0] = w.w[0];
  states.w[1] = w.w[2];
  states.w[1].slots_t = w.w[1].slots;
  const int err = walks_of<3, 2>(w, states, sq, log_decay, bf16, s, st);
  return err || !parts ? err : sum_heads(pq, dq, pk, dk, sq, bf16, s, st);
}

}  // namespace ssd
