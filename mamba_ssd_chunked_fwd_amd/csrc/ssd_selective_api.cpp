// ssd_selective_api.cpp -- the C ABI of the operators around a selective state
// space (declared in include/ssd_selective.h).  As in ssd_api.cpp, every entry point
// validates its arguments on the host before any HIP call, then enqueues its
// kernels on the caller's stream: no allocation, no host synchronisation, no state.
#include <climits>
#include <cstddef>
#include <cstdint>

#include "ssd_selective.h"
#include "ssd_selective_launch.h"
#include "ssd_selective_plan.h"

namespace {

bool on_bytes(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && on_bytes(p, 16); }
bool ok_opt(const void* p) { return p == nullptr || on_bytes(p, 16); }
// the first row of an input with a row stride
bool ok_rows(const void* p, uintptr_t n) { return p != nullptr && on_bytes(p, n); }
bool ok_dtype(ssd_dtype t) { return t == SSD_F32 || t == SSD_BF16; }
ssd_status from_hip(int err) { return err == 0 ? SSD_OK : SSD_ERR_HIP; }

constexpr int64_t kMaxDim = 1 << 20;
constexpr int64_t kMaxSequences = (1 << 22) - 1;

// A row stride, 0 standing for contiguous rows; -1 if it is none.  (Eight rows of fp32
// lie within 2^31 bytes.)
constexpr int64_t kMaxStride = 1 << 26;
int64_t stride_of(int64_t stride, int64_t row) {
  if (stride == 0) return row;
  return stride < row || stride > kMaxStride ? -1 : stride;
}

// Whether two byte ranges of length n (either may be null) share any byte.
bool overlap(const void* a, const void* b, size_t n) {
  if (a == nullptr || b == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + n && y < x + n;
}

// Sequences of equal length need tokens to divide by their number.
bool ok_lengths(const int32_t* cu, int64_t tokens, int64_t nseq) {
  return cu != nullptr ? on_bytes(cu, 4) : tokens % nseq == 0;
}

bool ok_workspace(const void* ws, size_t have, size_t need) {
  return ok_ptr(ws) && have >= need;
}

enum class Form { kForward, kBackward, kStep };

ssd_status check_conv(const ssd_short_conv_dims* d, Form form, ssd::ConvShape* out) {
  if (d == nullptr) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t nseq = form == Form::kStep ? 1 : d->nseq;
  const int64_t v[4] = {d->tokens, nseq, d->dim, d->width};
  for (int64_t e : v)
    if (e < 1 || e > INT32_MAX) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t stride = stride_of(d->x_stride, d->dim);
  if (stride < 0) return SSD_ERR_INVALID_ARGUMENT;
  if (d->width < 2 || d->width > 4 || d->dim > kMaxDim || nseq > kMaxSequences)
    return SSD_ERR_UNSUPPORTED;
  const ssd::ConvShape s{d->tokens, nseq, d->dim, d->width, stride};
  if (!ssd::conv_grid_fits(s, form == Form::kBackward, form == Form::kStep))
    return SSD_ERR_UNSUPPORTED;
  *out = s;
  return SSD_OK;
}

bool ok_conv_act(ssd_conv_act a) { return a == SSD_CONV_NONE || a == SSD_CONV_SILU; }
uintptr_t size_of(ssd_dtype t) { return t == SSD_BF16 ? 2 : 4; }
size_t conv_state_bytes(const ssd::ConvShape& s, ssd_dtype t) {
  return (size_t)(s.nseq * (s.width - 1)) * (size_t)s.dim * size_of(t);
}

ssd_status check_scan(const ssd_selective_scan_dims* d, Form form, ssd_dtype dtype,
                      ssd::ScanShape* out) {
  if (d == nullptr || !ok_dtype(dtype)) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t nseq = form == Form::kStep ? 1 : d->nseq;
  const int64_t v[5] = {d->tokens, nseq, d->dim, d->dstate, d->ngroups};
  for (int64_t e : v)
    if (e < 1 || e > INT32_MAX) return SSD_ERR_INVALID_ARGUMENT;
  if (d->dim % d->ngroups != 0) return SSD_ERR_INVALID_ARGUMENT;
  if (d->dstate != 8 && d->dstate != 16 && d->dstate != 32 && d->dstate != 64)
    return SSD_ERR_UNSUPPORTED;
  if (d->dim > kMaxDim || nseq > kMaxSequences) return SSD_ERR_UNSUPPORTED;
  const int64_t bc = d->ngroups * d->dstate;
  ssd::ScanShape s{d->tokens, nseq, d->dim, d->dstate, d->ngroups,
                   stride_of(d->x_stride, d->dim), stride_of(d->dt_stride, d->dim),
                   stride_of(d->z_stride, d->dim), stride_of(d->b_stride, bc),
                   stride_of(d->c_stride, bc)};
  if (s.x_stride < 0 || s.dt_stride < 0 || s.z_stride < 0 || s.b_stride < 0 || s.c_stride < 0)
    return SSD_ERR_INVALID_ARGUMENT;
  // rows of B and C are read in 4-byte words
  if (dtype == SSD_BF16 && (s.b_stride % 2 != 0 || s.c_stride % 2 != 0))
    return SSD_ERR_INVALID_ARGUMENT;
  if (form == Form::kStep ? !ssd::scan_step_grid_fits(s)
                          : !ssd::scan_grid_fits(s, form == Form::kBackward))
    return SSD_ERR_UNSUPPORTED;
  *out = s;
  return SSD_OK;
}

bool ok_scan_inputs(const ssd::ScanInputs& in, ssd_dtype t) {
  const uintptr_t n = size_of(t);
  return ok_rows(in.x, n) && ok_rows(in.dt, n) && ok_ptr(in.A) && ok_rows(in.B, 4) &&
         ok_rows(in.C, 4) && ok_opt(in.D) && (in.z == nullptr || on_bytes(in.z, n)) &&
         ok_opt(in.dt_bias);
}
size_t scan_state_bytes(const ssd::ScanShape& s) {
  return sizeof(float) * (size_t)(s.nseq * s.dim) * (size_t)s.n;
}

}  // namespace

extern "C" {

ssd_status ssd_short_conv_fwd(const void* x, const float* weight, const float* bias,
                              const void* init_state, const int32_t* cu_seqlens, void* y,
                              void* final_state, ssd_conv_act act, ssd_dtype dtype,
                              const ssd_short_conv_dims* dims, void* stream) {
  ssd::ConvShape s;
  const ssd_status st = check_conv(dims, Form::kForward, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(dtype) || !ok_conv_act(act) || !ok_lengths(cu_seqlens, s.tokens, s.nseq))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_rows(x, size_of(dtype)) || !ok_ptr(weight) || !ok_opt(bias) || !ok_opt(init_state) ||
      !ok_ptr(y) || !ok_opt(final_state))
    return SSD_ERR_INVALID_ARGUMENT;
  // the whole buffer in place, or apart from it
  if (init_state != final_state &&
      overlap(init_state, final_state, conv_state_bytes(s, dtype)))
    return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_short_conv_fwd(x, weight, bias, init_state, cu_seqlens, y,
                                             final_state, act == SSD_CONV_SILU,
                                             dtype == SSD_BF16, s, stream));
}

size_t ssd_short_conv_bwd_workspace_bytes(const ssd_short_conv_dims* dims) {
  ssd::ConvShape s;
  if (check_conv(dims, Form::kBackward, &s) != SSD_OK) return 0;
  return ssd::conv_bwd_bytes(s);
}

ssd_status ssd_short_conv_bwd(const void* x, const float* weight, const float* bias,
                              const void* init_state, const int32_t* cu_seqlens,
                              const void* dy, const void* dfinal, void* dx, float* dweight,
                              float* dbias, void* dinit, void* workspace,
                              size_t workspace_bytes, ssd_conv_act act, ssd_dtype dtype,
                              const ssd_short_conv_dims* dims, void* stream) {
  ssd::ConvShape s;
  const ssd_status st = check_conv(dims, Form::kBackward, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(dtype) || !ok_conv_act(act) || !ok_lengths(cu_seqlens, s.tokens, s.nseq))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_rows(x, size_of(dtype)) || !ok_ptr(weight) || !ok_opt(bias) || !ok_opt(init_state) ||
      !ok_ptr(dy) || !ok_opt(dfinal) || !ok_ptr(dx) || !ok_opt(dweight) || !ok_opt(dbias) ||
      !ok_opt(dinit))
    return SSD_ERR_INVALID_ARGUMENT;
  if (overlap(dfinal, dinit, conv_state_bytes(s, dtype))) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_workspace(workspace, workspace_bytes, ssd::conv_bwd_bytes(s)))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_short_conv_bwd(x, weight, bias, init_state, cu_seqlens, dy, dfinal,
                                             dx, dweight, dbias, dinit, workspace,
                                             act == SSD_CONV_SILU, dtype == SSD_BF16, s, stream));
}

ssd_status ssd_short_conv_step(const void* x, const float* weight, const float* bias,
                               void* state, void* y, ssd_conv_act act, ssd_dtype dtype,
                               const ssd_short_conv_dims* dims, void* stream) {
  ssd::ConvShape s;
  const ssd_status st = check_conv(dims, Form::kStep, &s);
  if (st != SSD_OK) return st;
  if (!ok_dtype(dtype) || !ok_conv_act(act)) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_rows(x, size_of(dtype)) || !ok_ptr(weight) || !ok_opt(bias) || !ok_ptr(state) ||
      !ok_ptr(y))
    return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_short_conv_step(x, weight, bias, state, y, act == SSD_CONV_SILU,
                                              dtype == SSD_BF16, s, stream));
}

size_t ssd_selective_scan_fwd_workspace_bytes(const ssd_selective_scan_dims* dims,
                                              ssd_dtype dtype) {
  ssd::ScanShape s;
  if (check_scan(dims, Form::kForward, dtype, &s) != SSD_OK) return 0;
  return ssd::scan_fwd_bytes(s);
}

size_t ssd_selective_scan_bwd_workspace_bytes(const ssd_selective_scan_dims* dims,
                                              ssd_dtype dtype) {
  ssd::ScanShape s;
  if (check_scan(dims, Form::kBackward, dtype, &s) != SSD_OK) return 0;
  return ssd::bwd_layout(s).all;
}

ssd_status ssd_selective_scan_fwd(const void* x, const void* dt, const float* A, const void* B,
                                  const void* C, const float* D, const void* z,
                                  const float* dt_bias, const float* init_state,
                                  const int32_t* cu_seqlens, void* y, float* final_state,
                                  void* workspace, size_t workspace_bytes, int softplus,
                                  ssd_dtype dtype, const ssd_selective_scan_dims* dims,
                                  void* stream) {
  ssd::ScanShape s;
  const ssd_status st = check_scan(dims, Form::kForward, dtype, &s);
  if (st != SSD_OK) return st;
  const ssd::ScanInputs in{x, dt, A, B, C, D, z, dt_bias};
  if (!ok_lengths(cu_seqlens, s.tokens, s.nseq) || !ok_scan_inputs(in, dtype) ||
      !ok_opt(init_state) || !ok_ptr(y) || !ok_opt(final_state))
    return SSD_ERR_INVALID_ARGUMENT;
  if (init_state != final_state && overlap(init_state, final_state, scan_state_bytes(s)))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_workspace(workspace, workspace_bytes, ssd::scan_fwd_bytes(s)))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_scan_fwd(in, init_state, cu_seqlens, y, final_state, workspace,
                                       softplus != 0, dtype == SSD_BF16, s, stream));
}

ssd_status ssd_selective_scan_bwd(const void* x, const void* dt, const float* A, const void* B,
                                  const void* C, const float* D, const void* z,
                                  const float* dt_bias, const float* init_state,
                                  const int32_t* cu_seqlens, const void* dy,
                                  const float* dfinal, void* dx, void* ddt, float* dA, void* dB,
                                  void* dC, float* dD, void* dz, float* ddt_bias, float* dinit,
                                  void* workspace, size_t workspace_bytes, int softplus,
                                  ssd_dtype dtype, const ssd_selective_scan_dims* dims,
                                  void* stream) {
  ssd::ScanShape s;
  const ssd_status st = check_scan(dims, Form::kBackward, dtype, &s);
  if (st != SSD_OK) return st;
  const ssd::ScanInputs in{x, dt, A, B, C, D, z, dt_bias};
  const ssd::ScanGradients out{dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit};
  if (!ok_lengths(cu_seqlens, s.tokens, s.nseq) || !ok_scan_inputs(in, dtype) ||
      !ok_opt(init_state) || !ok_ptr(dy) || !ok_opt(dfinal) || !ok_ptr(dx) || !ok_ptr(ddt) ||
      !ok_ptr(dA) || !ok_ptr(dB) || !ok_ptr(dC) || !ok_opt(dD) || !ok_opt(dz) ||
      !ok_opt(ddt_bias) || !ok_opt(dinit) || (z == nullptr) != (dz == nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  if (overlap(dfinal, dinit, scan_state_bytes(s))) return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_workspace(workspace, workspace_bytes, ssd::bwd_layout(s).all))
    return SSD_ERR_WORKSPACE;
  return from_hip(ssd::launch_scan_bwd(in, init_state, cu_seqlens, dy, dfinal, out, workspace,
                                       softplus != 0, dtype == SSD_BF16, s, stream));
}

ssd_status ssd_selective_scan_step(const void* x, const void* dt, const float* A, const void* B,
                                   const void* C, const float* D, const void* z,
                                   const float* dt_bias, float* state, void* y, int softplus,
                                   ssd_dtype dtype, const ssd_selective_scan_dims* dims,
                                   void* stream) {
  ssd::ScanShape s;
  const ssd_status st = check_scan(dims, Form::kStep, dtype, &s);
  if (st != SSD_OK) return st;
  const ssd::ScanInputs in{x, dt, A, B, C, D, z, dt_bias};
  if (!ok_scan_inputs(in, dtype) || !ok_ptr(state) || !ok_ptr(y))
    return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_scan_step(in, state, y, softplus != 0, dtype == SSD_BF16, s,
                                        stream));
}

ssd_status ssd_add_norm_quant_fwd(const void* x, const void* residual, const float* res_scale,
                                  const float* weight, void* codes, float* scales,
                                  void* residual_out, int64_t rows, int64_t dim, int64_t group,
                                  float eps, ssd_code code, ssd_dtype x_dtype,
                                  ssd_dtype res_dtype, void* stream) {
  if (rows < 1 || dim < 1 || group < 1 || rows > INT32_MAX || dim > INT32_MAX || group > dim ||
      dim % group != 0 || !(eps > 0.0f))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!ok_dtype(x_dtype) || !ok_dtype(res_dtype) ||
      (code != SSD_CODE_E4M3 && code != SSD_CODE_INT8))
    return SSD_ERR_INVALID_ARGUMENT;
  if (dim > ssd::kQuantMaxDim) return SSD_ERR_UNSUPPORTED;
  if (group != dim && group != 16 && group != 32 && group != 64 && group != 128 && group != 256)
    return SSD_ERR_UNSUPPORTED;
  if (!ok_ptr(x) || !ok_opt(residual) || !ok_opt(res_scale) || !ok_opt(weight) ||
      !ok_ptr(codes) || !ok_ptr(scales) || !ok_opt(residual_out))
    return SSD_ERR_INVALID_ARGUMENT;
  return from_hip(ssd::launch_add_norm_quant(x, residual, res_scale, weight, codes, scales,
                                             residual_out, rows, dim, group, eps,
                                             code == SSD_CODE_E4M3, x_dtype == SSD_BF16,
                                             res_dtype == SSD_BF16, stream));
}

}  // extern "C"
