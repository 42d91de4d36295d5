/*
 * ssd_selective.h -- C ABI of libssd, third part: the operators of a block
 * with a selective state space, whose decay is formed from the input for each
 * channel, state and token:
 *   - the short causal convolution in front of it, over whole (packed)
 *     sequences, its gradients, and its form for single tokens;
 *   - the selective scan over whole (packed) sequences, its gradients, and its
 *     recurrent form for single tokens;
 *   - the residual add and norm in front of a block whose projection takes 8
 *     bits (ssd_add_norm_fwd's formula, the output as codes with scales).
 *
 * The conventions are those of ssd_block.h: device pointers, row-major; the
 * caller owns every buffer, workspaces included; stream-ordered, asynchronous
 * calls that allocate nothing, keep no state and may run at once on different
 * streams (with a workspace each); every argument is checked on the host
 * before any HIP call.  Pointers are 16-byte aligned and arrays contiguous,
 * but where an entry names a row stride: such an input may be columns of a
 * wider array (the halves of one projection), starts on a multiple of its element
 * size (B and C: of 4 bytes), and its rows are `stride` elements apart (0: contiguous; up
 * to 2^26).
 * No output may overlap an input or another output unless an entry says so.
 *
 * Sequences are packed as in ssd_linattn_fwd: cu_seqlens, if not NULL, is a
 * DEVICE array of nseq + 1 int32, not descending: sequence i holds tokens
 * cu_seqlens[i] .. cu_seqlens[i+1]-1 and may be empty.  Rows outside every
 * sequence are not read and left as they are (gradients too).  NULL: nseq sequences of
 * tokens / nseq tokens each.  Entries outside [0, tokens] are taken as the
 * nearer end; where entries descend a call still reads and writes nothing out
 * of range, but its results are undefined.
 */
#ifndef SSD_SELECTIVE_H_
#define SSD_SELECTIVE_H_

#include "ssd_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The short causal convolution.  Per sequence and channel d, over the rows
 * ext = (the W-1 rows of init_state, then the sequence's rows of x):
 *     pre_t = bias_d + sum_{k<W} weight[d,k] ext_{t+k}
 *     y_t = pre_t, or silu(pre_t)                 (t = 0, 1, ...)
 *     final_state = the last W-1 rows of ext
 * x [tokens, dim] (row stride x_stride), y [tokens, dim], states
 * [nseq, W-1, dim] in `dtype`; weight [dim, W], bias [dim] fp32.  bias NULL:
 * zeros; init_state NULL: zeros; final_state NULL: not stored.  final_state may
 * be the same buffer as init_state.  Sums are fp32, rounded once.
 *
 * For x channel-first, without states, packing or gate, this is ssd_causal_conv1d.
 * Supported: W in {2, 3, 4}, dim up to 2^20, nseq below 2^22.
 */
typedef enum { SSD_CONV_NONE = 0, SSD_CONV_SILU = 1 } ssd_conv_act;

typedef struct {
    int64_t tokens;    /* rows of x and y                            */
    int64_t nseq;      /* sequences                                  */
    int64_t dim;       /* channels                                   */
    int64_t width;     /* W, taps                                    */
    int64_t x_stride;  /* elements between rows of x (0: dim)        */
} ssd_short_conv_dims;

ssd_status ssd_short_conv_fwd(const void *x, const float *weight, const float *bias,
                              const void *init_state, const int32_t *cu_seqlens, void *y,
                              void *final_state, ssd_conv_act act, ssd_dtype dtype,
                              const ssd_short_conv_dims *dims, void *stream);

/*
 * Its gradients, from the inputs of the forward call: with g_t = dy_t times the
 * derivative of the activation at pre_t,
 *     dext_{t+k} = sum_k weight[d,k] g_t   (+ dfinal in its last W-1 rows)
 *     dweight[d,k] = sum_t g_t ext_{t+k}        dbias_d = sum_t g_t
 * dy, dx [tokens, dim], dfinal, dinit [nseq, W-1, dim] in dtype; dweight [dim, W],
 * dbias [dim] fp32.  dfinal NULL: zeros; dinit, dweight, dbias NULL: not formed.
 * dinit must not overlap dfinal.  The sums over tokens are taken in a fixed order.
 */
size_t ssd_short_conv_bwd_workspace_bytes(const ssd_short_conv_dims *dims);
ssd_status ssd_short_conv_bwd(const void *x, const float *weight, const float *bias,
                              const void *init_state, const int32_t *cu_seqlens,
                              const void *dy, const void *dfinal, void *dx, float *dweight,
                              float *dbias, void *dinit, void *workspace,
                              size_t workspace_bytes, ssd_conv_act act, ssd_dtype dtype,
                              const ssd_short_conv_dims *dims, void *stream);

/*
 * One token for every sequence of a batch: x [batch, dim] (row stride
 * x_stride), y [batch, dim], state [batch, W-1, dim] (read, and written with x
 * behind its last rows).  dims->tokens is the batch; dims->nseq is not read.
 */
ssd_status ssd_short_conv_step(const void *x, const float *weight, const float *bias,
                               void *state, void *y, ssd_conv_act act, ssd_dtype dtype,
                               const ssd_short_conv_dims *dims, void *stream);

/*
 * The selective scan.  Per sequence and channel d, with group g = d / (dim/ngroups):
 *     delta_t = softplus(dt_t + dt_bias_d)     (without softplus: dt_t + dt_bias_d)
 *     h_t[n] = exp(delta_t A[d,n]) h_{t-1}[n] + delta_t x_t B_t[g,n]
 *     u_t = sum_n C_t[g,n] h_t[n] + D_d x_t
 *     y_t = u_t silu(z_t)
 * x, dt, z [tokens, dim] (row strides of their own), y [tokens, dim], B, C
 * [tokens, ngroups, N] (row strides of their own) in `dtype`; A [dim, N], D, dt_bias
 * [dim], init_state and final_state [nseq, dim, N] fp32.  D, dt_bias, init_state NULL:
 * zeros; z NULL: no gate; final_state NULL: not stored.  final_state may be the same
 * buffer as init_state.  A is finite.  All arithmetic is fp32, y rounded once.
 *
 * Decays are meant to be at most 1 (delta A <= 0).  Larger ones give what the recurrence gives
 * while the product of any stretch of a sequence's decays stays below 2^127; where one passes
 * it, results (and gradients) may be NaN even if every state stays finite, as one of 0 does: the
 * products of whole runs of tokens are formed by themselves.
 *
 * Supported: N in {8, 16, 32, 64}, dim up to 2^20, nseq below 2^22 and, with the blocks of
 * 64 channels that the groups have, nseq * blocks below some 2^26 (a launch has fewer than
 * 2^32 threads); anything else valid returns SSD_ERR_UNSUPPORTED.
 */
typedef struct {
    int64_t tokens;    /* rows of x, dt, z, B, C and y               */
    int64_t nseq;      /* sequences                                  */
    int64_t dim;       /* channels                                   */
    int64_t dstate;    /* N, states of a channel                     */
    int64_t ngroups;   /* groups of B and C; dim % ngroups == 0      */
    int64_t x_stride, dt_stride, z_stride;   /* elements between rows (0: dim)        */
    int64_t b_stride, c_stride;              /* the same of B and C (0: ngroups * N)  */
} ssd_selective_scan_dims;

/* Bytes of device workspace the two calls below need; 0 when dims is NULL or
 * invalid (a valid shape that needs none also reports at least 16). */
size_t ssd_selective_scan_fwd_workspace_bytes(const ssd_selective_scan_dims *dims,
                                              ssd_dtype dtype);
size_t ssd_selective_scan_bwd_workspace_bytes(const ssd_selective_scan_dims *dims,
                                              ssd_dtype dtype);

ssd_status ssd_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *B,
                                  const void *C, const float *D, const void *z,
                                  const float *dt_bias, const float *init_state,
                                  const int32_t *cu_seqlens, void *y, float *final_state,
                                  void *workspace, size_t workspace_bytes, int softplus,
                                  ssd_dtype dtype, const ssd_selective_scan_dims *dims,
                                  void *stream);

/*
 * Its gradients, from the inputs of the forward call: with du = dy silu(z) and
 * R_t the gradient of h_t, R_t = C_t du_t + exp(delta_{t+1} A) R_{t+1} (dfinal in the place
 * of the second term at the last token), and K_t = R_t exp(delta_t A) h_{t-1},
 *     dB_t[g] = sum_d R_t delta_t x_t        dC_t[g] = sum_d du_t h_t
 *     dx_t = delta_t sum_n R_t B_t + D du_t  ddelta_t = x_t sum_n R_t B_t + sum_n K_t A
 *     dA = sum_t K_t delta_t                 dD = sum_t du_t x_t
 *     dz_t = dy_t u_t silu'(z_t)             ddt_t = ddelta_t softplus'(dt_t + dt_bias)
 *     ddt_bias = sum_t ddt_t                 dinit = exp(delta_1 A) R_1
 * (d over the group's channels; t over the tokens of every sequence).  dy [tokens, dim];
 * dx, ddt, dz [tokens, dim], dB, dC [tokens, ngroups, N] in dtype, contiguous; dA [dim, N],
 * dD, ddt_bias [dim], dfinal, dinit [nseq, dim, N] fp32.  dz is given exactly when z
 * is; dfinal NULL: zeros; dD, ddt_bias, dinit NULL: not formed.  dinit must not overlap
 * dfinal.  Sums over channels and tokens are taken in a fixed order.
 */
ssd_status ssd_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *B,
                                  const void *C, const float *D, const void *z,
                                  const float *dt_bias, const float *init_state,
                                  const int32_t *cu_seqlens, const void *dy,
                                  const float *dfinal, void *dx, void *ddt, float *dA, void *dB,
                                  void *dC, float *dD, void *dz, float *ddt_bias, float *dinit,
                                  void *workspace, size_t workspace_bytes, int softplus,
                                  ssd_dtype dtype, const ssd_selective_scan_dims *dims,
                                  void *stream);

/*
 * One token for every sequence of a batch, the state [batch, dim, N] updated in
 * place.  x, dt, z, y [batch, dim], B, C [batch, ngroups, N].  dims->tokens is the batch;
 * dims->nseq is not read.
 */
ssd_status ssd_selective_scan_step(const void *x, const void *dt, const float *A, const void *B,
                                   const void *C, const float *D, const void *z,
                                   const float *dt_bias, float *state, void *y, int softplus,
                                   ssd_dtype dtype, const ssd_selective_scan_dims *dims,
                                   void *stream);

/*
 * ssd_add_norm_fwd with its output in 8 bits.  Per row:
 *     h = residual + res_scale o x;  y = h / sqrt(mean(h^2) + eps) o weight
 * and per group of `group` channels (a divisor of dim), with top = 448 (e4m3) or 127 (int8):
 *     scales = max |y| / top        codes = the 8-bit value nearest to y top / max |y|
 * (ties to even), so that codes o scales stands for y.  codes [rows, dim] bytes;
 * scales [rows, dim/group] fp32; the rest as in ssd_add_norm_fwd.  All arithmetic is
 * in 64 bits, so a code is the nearest one but where the value lies within some 1e-15 of a
 * border (on one, where the 64-bit products are exact, it is the even one).  A group of
 * zeros (or of values below 1e-30) has codes of 0.  A row that holds a value that is not
 * finite has scales of NaN where its group does, as ssd_add_norm_fwd's y would.
 * residual_out may be the same buffer as residual.
 * Supported: dim up to 16384; group = dim, or 16, 32, 64, 128 or 256.
 */
typedef enum { SSD_CODE_E4M3 = 0, SSD_CODE_INT8 = 1 } ssd_code;

ssd_status ssd_add_norm_quant_fwd(const void *x, const void *residual, const float *res_scale,
                                  const float *weight, void *codes, float *scales,
                                  void *residual_out, int64_t rows, int64_t dim, int64_t group,
                                  float eps, ssd_code code, ssd_dtype x_dtype,
                                  ssd_dtype res_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_SELECTIVE_H_ */
