// ssd_block_api.cpp -- the C ABI of the block operators (declared in
// include/ssd_block.h).  As in ssd_api.cpp, every entry point validates its
// arguments on the host before any HIP call, then enqueues its kernels on the
// caller's stream: no allocation, no host synchronisation, no state.
#include <climits>
#include <cstddef>
#include <cstdint>

#include "ssd_block.h"
#include "ssd_block_launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
bool ok_opt(const void* p) { return p == nullptr || aligned16(p); }
bool ok_dtype(ssd_dtype t) { return t == SSD_F32 || t == SSD_BF16; }
ssd_status from_hip(int err) { return err == 0 ? SSD_OK : SSD_ERR_HIP; }

// Rows of one tensor are addressed with 64-bit offsets; what is bounded is
// each dimension and the number of workgroups of a launch: of 256 threads below
// 2^24, because a launch has at most 2^32 - 1 threads along an axis.
constexpr int64_t kMaxBlocks = (1 << 24) - 1;
constexpr int64_t kMaxTokenHeads = (1 << 27) - 1;

ssd_status check_linattn(const ssd_linattn_dims* d, bool step, ssd::LinattnShape* out) {
  if (d == nullptr) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t nseq = step ? 1 : d->nseq;
  const int64_t v[6] = {d->tokens, nseq, d->nheads, d->ngroups, d->dk, d->dv};
  for (int64_t e : v)
    if (e < 1 || e > INT32_MAX) return SSD_ERR_INVALID_ARGUMENT;
  if (d->nheads % d->ngroups != 0) return SSD_ERR_INVALID_ARGUMENT;
  // lengths in tokens, rounded up to chunks, and runs' numbers are 32-bit
  if (d->tokens > kMaxTokenHeads / d->nheads) return SSD_ERR_UNSUPPORTED;
  // a single token's call has one workgroup per head of a sequence where there are
  // many; the others up to three, and below 2^20 more for the runs
  if ((step ? d->tokens : 4 * nseq) > kMaxBlocks / d->nheads) return SSD_ERR_UNSUPPORTED;
  if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128)) return SSD_ERR_UNSUPPORTED;
  // one row of a tensor, and the 64 rows of a tile, stay below 2 GiB
  if (d->nheads > (1 << 15)) return SSD_ERR_UNSUPPORTED;
  *out = ssd::LinattnShape{d->tokens, nseq, d->nheads, d->ngroups, d->dk, d->dv};
  return SSD_OK;
}

// Sequences of equal length need tokens to divide by their number.
bool ok_lengths(const int32_t* cu, const ssd::LinattnShape& s) {
  return cu != nullptr ? (reinterpret_cast<uintptr_t>(cu) & 3u) == 0 : s.tokens % s.nseq == 0;
}

// Whether two byte ranges of length n (either may be null) share any byte.
bool overlap(const void* a, const void* b, size_t n) {
  if (a == nullptr || b == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + n && y < x + n;
}

size_t state_bytes(const ssd::LinattnShape& s) {
  return sizeof(float) * (size_t)(s.nseq * s.nheads) * (size_t)(s.dk * s.dv);
}

bool ok_workspace(const void* ws, size_t have, size_t need) {
  return ok_ptr(ws) && have >= need;
}

ssd_status check_norm(int64_t rows, int64_t dim, int64_t group, int64_t wdim, float eps,
                      ssd::NormShape* out) {
  if (rows < 1 || dim < 1 || group < 1 || rows > INT32_MAX || dim > INT32_MAX)
    return SSD_ERR_INVALID_ARGUMENT;
  if (group > dim || dim % group != 0 || (wdim != dim && wdim != group))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!(eps > 0.0f)) return SSD_ERR_INVALID_ARGUMENT;
  // (dim: the row sums take 1024 threads for 64 channels)
  if (group > ssd::kNormMaxGroup || dim > (1 << 27)) return SSD_ERR_UNSUPPORTED;
  // a row's groups are spread over the second grid axis, 65535 at most, of
  // at least one group each
  if (dim / group > 65535) return SSD_ERR_UNSUPPORTED;
  *out = ssd::NormShape{rows, dim, group, wdim};
  return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_linattn_fwd_workspace_bytes(const ssd_linattn_dims* dims, ssd_dtype dtype) {
  ssd::LinattnShape s;
  if (!ok_dtype(dtype) || check_linattn(dims, false, &s) != SSD_OK) return 0;
  return ssd::linattn_workspace(s, dtype == SSD_BF16, false);
}

size_t ssd_linattn_bwd_workspace_bytes(const ssd_linattn_dims* dims, ssd_dtype dtype) {
  ssd::LinattnShape s;
  if (!ok_dtype(dtype) || check_linattn(dims, false, &s) != SSD_OK) return 0;
  return ssd::linattn_workspace(s, dtype == SSD_BF16, true);
}

ssd_status ssd_linattn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                           const float* init_state, const int32_t* cu_seqlens, void* o,
                           float* final_state, void* workspace, size_t workspace_bytes,
                           float scale, ssd_dtype dtype, const ssd_linattn_dims* dims,
                           void* stream) {
  ssd::LinattnShape s;
  const ssd_status st = check_linattn(dims, false, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(dtype) || !ok_lengths(cu_seqlens, s)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(log_decay) || !ok_opt(init_state) ||
      !ok_ptr(o) || !ok_opt(final_state))
    return SSD_ERR_INVALID_ARGUMENT;
  // the whole buffer in place, or apart from it
  if (init_state != final_state && overlap(init_state, final_state, state_bytes(s)))
    return SSD_ERR_INVALID_ARGUMENT;
  const bool bf16 = dtype == SSD_BF16;
  if (!ok_workspace(workspace, workspace_bytes, ssd::linattn_workspace(s, bf16, false)))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_linattn_fwd(q, k, v, log_decay, init_state, cu_seqlens, o,
                                          final_state, workspace, scale, bf16, s, stream));
}

ssd_status ssd_linattn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                           const float* init_state, const int32_t* cu_seqlens, const void* dout,
                           const float* dfinal, void* dq, void* dk, void* dv, float* dinit,
                           void* workspace, size_t workspace_bytes, float scale, ssd_dtype dtype,
                           const ssd_linattn_dims* dims, void* stream) {
  ssd::LinattnShape s;
  const ssd_status st = check_linattn(dims, false, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(dtype) || !ok_lengths(cu_seqlens, s)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(log_decay) || !ok_opt(init_state) ||
      !ok_ptr(dout) || !ok_opt(dfinal) || !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dv) ||
      !ok_opt(dinit))
    return SSD_ERR_INVALID_ARGUMENT;
  // dk is walked from dfinal while dv's walk writes dinit
  if (overlap(dfinal, dinit, state_bytes(s))) return SSD_ERR_INVALID_ARGUMENT;
  const bool bf16 = dtype == SSD_BF16;
  if (!ok_workspace(workspace, workspace_bytes, ssd::linattn_workspace(s, bf16, true)))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_linattn_bwd(q, k, v, log_decay, init_state, cu_seqlens, dout,
                                          dfinal, dq, dk, dv, dinit, workspace, scale, bf16, s,
                                          stream));
}

ssd_status ssd_linattn_step(const void* q, const void* k, const void* v, const float* log_decay,
                            float* state, void* o, float scale, ssd_dtype dtype,
                            const ssd_linattn_dims* dims, void* stream) {
  ssd::LinattnShape s;
  const ssd_status st = check_linattn(dims, true, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(dtype)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(log_decay) || !ok_ptr(state) ||
      !ok_ptr(o))
    return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_linattn_step(q, k, v, log_decay, state, o, scale,
                                           dtype == SSD_BF16, s, stream));
}

ssd_status ssd_add_norm_fwd(const void* x, const void* residual, const float* res_scale,
                            const float* weight, void* y, void* residual_out, int64_t rows,
                            int64_t dim, float eps, ssd_dtype x_dtype, ssd_dtype res_dtype,
                            void* stream) {
  ssd::NormShape s;
  const ssd_status st = check_norm(rows, dim, dim, dim, eps, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(x_dtype) || !ok_dtype(res_dtype)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(x) || !ok_opt(residual) || !ok_opt(res_scale) || !ok_opt(weight) || !ok_ptr(y) ||
      !ok_opt(residual_out))
    return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_add_norm_fwd(x, residual, res_scale, weight, y, residual_out, eps,
                                           x_dtype == SSD_BF16, res_dtype == SSD_BF16, s,
                                           stream));
}

size_t ssd_add_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  ssd::NormShape s;
  if (check_norm(rows, dim, dim, dim, 1.0f, &s) != SSD_OK) return 0;
  return ssd::norm_bwd_workspace(s, 2);
}

ssd_status ssd_add_norm_bwd(const void* x, const void* residual, const float* res_scale,
                            const float* weight, const void* dy, const void* dresidual_out,
                            void* dx, void* dresidual, float* dres_scale, float* dweight,
                            void* workspace, size_t workspace_bytes, int64_t rows, int64_t dim,
                            float eps, ssd_dtype x_dtype, ssd_dtype res_dtype, void* stream) {
  ssd::NormShape s;
  const ssd_status st = check_norm(rows, dim, dim, dim, eps, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(x_dtype) || !ok_dtype(res_dtype)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(x) || !ok_opt(residual) || !ok_opt(res_scale) || !ok_opt(weight) || !ok_ptr(dy) ||
      !ok_opt(dresidual_out) || !ok_ptr(dx) || !ok_opt(dresidual) || !ok_opt(dres_scale) ||
      !ok_opt(dweight))
    return SSD_ERR_INVALID_ARGUMENT;
  if (dres_scale != nullptr && res_scale == nullptr) return SSD_ERR_INVALID_ARGUMENT;
  if (dresidual != nullptr && residual == nullptr) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_workspace(workspace, workspace_bytes, ssd::norm_bwd_workspace(s, 2)))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_add_norm_bwd(x, residual, res_scale, weight, dy, dresidual_out, dx,
                                           dresidual, dres_scale, dweight, workspace, eps,
                                           x_dtype == SSD_BF16, res_dtype == SSD_BF16, s,
                                           stream));
}

ssd_status ssd_gated_norm_fwd(const void* x, const void* z, const float* weight, void* y,
                              float eps, ssd_gate gate, int gate_first, ssd_dtype x_dtype,
                              ssd_dtype z_dtype, const ssd_gated_norm_dims* dims,
                              void* stream) {
  if (dims == nullptr) return SSD_ERR_INVALID_ARGUMENT;
  ssd::NormShape s;
  const ssd_status st = check_norm(dims->rows, dims->dim, dims->group, dims->weight_dim, eps, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(x_dtype) || !ok_dtype(z_dtype)) return SSD_ERR_INVALID_ARGUMENT;
  if (gate != SSD_GATE_SILU && gate != SSD_GATE_SIGMOID) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(x) || !ok_opt(z) || !ok_opt(weight) || !ok_ptr(y)) return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_gated_norm_fwd(x, z, weight, y, eps, gate == SSD_GATE_SILU,
                                             gate_first != 0, x_dtype == SSD_BF16,
                                             z_dtype == SSD_BF16, s, stream));
}

size_t ssd_gated_norm_bwd_workspace_bytes(const ssd_gated_norm_dims* dims) {
  ssd::NormShape s;
  if (dims == nullptr ||
      check_norm(dims->rows, dims->dim, dims->group, dims->weight_dim, 1.0f, &s) != SSD_OK)
    return 0;
  return ssd::norm_bwd_workspace(s, 1);
}

ssd_status ssd_gated_norm_bwd(const void* x, const void* z, const float* weight, const void* dy,
                              void* dx, void* dz, float* dweight, void* workspace,
                              size_t workspace_bytes, float eps, ssd_gate gate, int gate_first,
                              ssd_dtype x_dtype, ssd_dtype z_dtype,
                              const ssd_gated_norm_dims* dims, void* stream) {
  if (dims == nullptr) return SSD_ERR_INVALID_ARGUMENT;
  ssd::NormShape s;
  const ssd_status st = check_norm(dims->rows, dims->dim, dims->group, dims->weight_dim, eps, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(x_dtype) || !ok_dtype(z_dtype)) return SSD_ERR_INVALID_ARGUMENT;
  if (gate != SSD_GATE_SILU && gate != SSD_GATE_SIGMOID) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_ptr(x) || !ok_opt(z) || !ok_opt(weight) || !ok_ptr(dy) || !ok_ptr(dx) || !ok_opt(dz) ||
      !ok_opt(dweight))
    return SSD_ERR_INVALID_ARGUMENT;
  if ((z == nullptr) != (dz == nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_workspace(workspace, workspace_bytes, ssd::norm_bwd_workspace(s, 1)))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_gated_norm_bwd(x, z, weight, dy, dx, dz, dweight, workspace, eps,
                                             gate == SSD_GATE_SILU, gate_first != 0,
                                             x_dtype == SSD_BF16, z_dtype == SSD_BF16, s,
                                             stream));
}

}  // extern "C"
