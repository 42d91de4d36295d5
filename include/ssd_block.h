/*
 * ssd_block.h -- C ABI of libssd, second part: the operators of a recurrent
 * language-model block besides the SSD itself (include/ssd.h):
 *   - linear attention with a decay for each head over whole (packed)
 *     sequences, its gradients, and its recurrent form for single tokens;
 *   - the residual add with a scale fused with the norm in front of a block,
 *     and its gradients;
 *   - the gated norm behind a block's mixer, and its gradients.
 *
 * The conventions are those of ssd.h: device pointers to contiguous
 * row-major arrays, each 16-byte aligned; the caller owns every buffer,
 * workspaces included; stream-ordered, asynchronous calls that allocate
 * nothing, keep no state and may run at once on different streams (with a
 * workspace each); every argument is checked on the host before any HIP
 * call.  Element types: tensors are fp32 or bf16 as each entry says; states,
 * decays, norm weights and residual scales, and their gradients, are fp32.
 * No output may overlap an input or another output unless an entry says so.
 */
#ifndef SSD_BLOCK_H_
#define SSD_BLOCK_H_

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay for each head.  Per sequence and head h, with
 * group g = h / (nheads/ngroups), lam = exp(log_decay[h]):
 *     S_t = lam S_{t-1} + k_t v_t^T          (state, dk x dv; S_0 = init)
 *     o_t = scale q_t^T S_t
 * q, k [tokens, G, K] (shared by the heads of a group, as B and C are in the
 * SSD), v, o [tokens, H, V] in `dtype`; log_decay [H] fp32, <= 0 (0: no
 * decay; -inf: no memory).
 *
 * Sequences lie one behind the other.  cu_seqlens, if not NULL, is a DEVICE
 * array of nseq + 1 int32, not descending: sequence i holds tokens
 * cu_seqlens[i] .. cu_seqlens[i+1]-1 and may be empty.  Rows outside
 * every sequence are not read and left as they are.  NULL: nseq sequences of
 * tokens / nseq tokens each.  Entries outside [0, tokens] are taken as the
 * nearer end; where entries descend a call still reads and writes nothing out
 * of range, but its results are undefined.
 *
 * For sequences of equal length with V = 64 these are ssd_forward's results for
 * x = v, B = k, C = scale q, dt = 1, A = log_decay and D = 0 (there with every chunk's
 * state in memory), and the single token's call ssd_decode_step's with the state
 * transposed.  Here are packed sequences, values of 128, K and V in any pairing,
 * gradients, and outputs without the states.
 *
 * Supported: K and V in {64, 128}, up to 32768 heads, tokens * nheads below 2^27,
 * nseq * nheads below 2^22 (of the recurrent form: tokens * nheads below 2^24);
 * anything else valid returns SSD_ERR_UNSUPPORTED.
 */
typedef struct {
    int64_t tokens;     /* T, rows of q, k, v and o               */
    int64_t nseq;       /* sequences                              */
    int64_t nheads;     /* H, heads of v, o and the states         */
    int64_t ngroups;    /* G, heads of q and k; H % G == 0         */
    int64_t dk;         /* K, size of q_t and k_t (rows of S)       */
    int64_t dv;         /* V, size of v_t and o_t (columns of S)    */
} ssd_linattn_dims;

/* Bytes of device workspace the two calls below need; 0 when dims is NULL or
 * invalid (a valid shape that needs none also reports at least 16). */
size_t ssd_linattn_fwd_workspace_bytes(const ssd_linattn_dims *dims, ssd_dtype dtype);
size_t ssd_linattn_bwd_workspace_bytes(const ssd_linattn_dims *dims, ssd_dtype dtype);

/*
 * Whole sequences.  init_state [nseq, H, K, V] fp32 or NULL (zeros);
 * final_state [nseq, H, K, V] fp32 (written; an empty sequence's is its
 * initial state) or NULL.  They may be the same buffer (sequences continued
 * in place).  Sums and states are fp32; for bf16 tensors the
 * states, scores and decayed values enter products as two bf16 terms, which leave at
 * most 2^-16 of each.  A value of v that is not
 * finite leaves its column of o, from its token on, and of the final state NaN or
 * infinite, and the tokens before it as they would be without (and so for k, q and
 * dout in the gradients' walks).
 */
ssd_status ssd_linattn_fwd(const void *q, const void *k, const void *v,
                           const float *log_decay, const float *init_state,
                           const int32_t *cu_seqlens, void *o, float *final_state,
                           void *workspace, size_t workspace_bytes, float scale,
                           ssd_dtype dtype, const ssd_linattn_dims *dims, void *stream);

/*
 * Gradients of the call above: dout [tokens, H, V] in dtype; dfinal
 * [nseq, H, K, V] fp32 or NULL (final_state not used).  With R_t the gradient of
 * S_t, R_t = scale q_t dout_t^T + lam R_{t+1} (dfinal in the place of lam
 * R_{t+1} at the last token):
 *     dq_t = scale sum_h S_t dout_t     dk_t = sum_h R_t v_t   (h over the group)
 *     dv_t = R_t^T k_t                  dinit = lam R_1
 * dq, dk [tokens, G, K], dv [tokens, H, V] in dtype (written); dinit
 * [nseq, H, K, V] fp32 (written) or NULL, and must not overlap dfinal
 * (SSD_ERR_INVALID_ARGUMENT).  log_decay is a constant of the model: it has no
 * gradient here.
 */
ssd_status ssd_linattn_bwd(const void *q, const void *k, const void *v,
                           const float *log_decay, const float *init_state,
                           const int32_t *cu_seqlens, const void *dout,
                           const float *dfinal, void *dq, void *dk, void *dv,
                           float *dinit, void *workspace, size_t workspace_bytes,
                           float scale, ssd_dtype dtype, const ssd_linattn_dims *dims,
                           void *stream);

/*
 * One token for every sequence of a batch, in place: S = lam S + k v^T,
 * o = scale q^T S.  q, k [batch, G, K], v, o [batch, H, V] in dtype; state
 * [batch, H, K, V] fp32 (read and written).  dims->tokens is the batch;
 * dims->nseq is not read.
 */
ssd_status ssd_linattn_step(const void *q, const void *k, const void *v,
                            const float *log_decay, float *state, void *o, float scale,
                            ssd_dtype dtype, const ssd_linattn_dims *dims, void *stream);

/*
 * The norm in front of a block, with the residual add before it.  Per row of
 * `dim` channels:
 *     h = residual + res_scale o x
 *     y = h / sqrt(mean(h^2) + eps) o weight
 * x, y [rows, dim] in x_dtype; residual, residual_out [rows, dim] in
 * res_dtype; res_scale, weight [dim] fp32.  residual NULL: zeros (the first
 * block); res_scale or weight NULL: ones; residual_out NULL: h is not stored.
 * y is formed from h before h is rounded to res_dtype.  residual_out may be
 * the same buffer as residual, and y the same as x.  eps > 0.  The squares are summed
 * in fp32: rows of values beyond some 1e17 overflow to y = 0 (here and below).
 * Supported: dim up to 16384.
 */
ssd_status ssd_add_norm_fwd(const void *x, const void *residual, const float *res_scale,
                            const float *weight, void *y, void *residual_out, int64_t rows,
                            int64_t dim, float eps, ssd_dtype x_dtype, ssd_dtype res_dtype,
                            void *stream);

/*
 * Its gradients, from the inputs of the forward call: with r = 1/sqrt(mean(h^2)
 * + eps) and n = h r,
 *     g = dresidual_out + r (weight o dy - n mean(weight o dy o n))
 *     dresidual = g    dx = res_scale o g
 *     dres_scale = sum_rows g o x    dweight = sum_rows dy o n
 * dy [rows, dim] in x_dtype; dresidual_out [rows, dim] in res_dtype or NULL
 * (zeros); dx in x_dtype; dresidual in res_dtype or NULL; dres_scale and
 * dweight [dim] fp32 or NULL.  dresidual may be the same buffer as
 * dresidual_out, and dx the same as dy.  dres_scale needs res_scale.  The row
 * sums are taken in a fixed order.
 */
size_t ssd_add_norm_bwd_workspace_bytes(int64_t rows, int64_t dim);
ssd_status ssd_add_norm_bwd(const void *x, const void *residual, const float *res_scale,
                            const float *weight, const void *dy, const void *dresidual_out,
                            void *dx, void *dresidual, float *dres_scale, float *dweight,
                            void *workspace, size_t workspace_bytes, int64_t rows, int64_t dim,
                            float eps, ssd_dtype x_dtype, ssd_dtype res_dtype, void *stream);

/*
 * The gated norm behind a mixer, over groups of `group` channels (a divisor
 * of dim; group = dim: the whole row):
 *     gate_first:      u = x o act(z);  y = u / sqrt(mean(u^2) + eps) o weight
 *     otherwise:       y = x / sqrt(mean(x^2) + eps) o weight o act(z)
 * with the mean over each group.  act: SSD_GATE_SILU z sigmoid(z), or
 * SSD_GATE_SIGMOID.  x [rows, dim] in x_dtype; z, y [rows, dim] in
 * z_dtype; z NULL: no gate.  weight [weight_dim] fp32 or NULL, weight_dim
 * being dim, or group (one set of weights for every group).  y may be the
 * same buffer as z, or as x where the types are equal.  eps > 0.
 * Supported: group up to 16384, dim up to 2^27 and to 65535 groups.
 */
typedef enum { SSD_GATE_SILU = 0, SSD_GATE_SIGMOID = 1 } ssd_gate;

typedef struct {
    int64_t rows;
    int64_t dim;
    int64_t group;       /* channels normed together               */
    int64_t weight_dim;  /* dim or group                            */
} ssd_gated_norm_dims;

ssd_status ssd_gated_norm_fwd(const void *x, const void *z, const float *weight, void *y,
                              float eps, ssd_gate gate, int gate_first, ssd_dtype x_dtype,
                              ssd_dtype z_dtype, const ssd_gated_norm_dims *dims,
                              void *stream);

/*
 * Its gradients, from the inputs of the forward call: dy [rows, dim] in
 * z_dtype; dx in x_dtype; dz in z_dtype (NULL exactly when z is); dweight
 * [weight_dim] fp32 or NULL.  dz may be the same buffer as dy.  The row sums
 * are taken in a fixed order.
 */
size_t ssd_gated_norm_bwd_workspace_bytes(const ssd_gated_norm_dims *dims);
ssd_status ssd_gated_norm_bwd(const void *x, const void *z, const float *weight,
                              const void *dy, void *dx, void *dz, float *dweight,
                              void *workspace, size_t workspace_bytes, float eps,
                              ssd_gate gate, int gate_first, ssd_dtype x_dtype,
                              ssd_dtype z_dtype, const ssd_gated_norm_dims *dims,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_BLOCK_H_ */
