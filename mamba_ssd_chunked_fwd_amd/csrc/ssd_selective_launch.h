// ssd_selective_launch.h -- host-side launchers of the operators around a
// selective state space (internal to libssd; declared to users in
// include/ssd_selective.h).  Arguments arrive already validated by the C ABI
// layer; each launcher returns the hipError_t of its launches as an int (0 =
// success).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd_selective.h"

namespace ssd {

struct ConvShape {
  int64_t tokens, nseq, dim, width, x_stride;
};

int launch_short_conv_fwd(const void* x, const float* weight, const float* bias, const void* init,
                          const int32_t* cu, void* y, void* fin, bool silu, bool bf16,
                          const ConvShape& s, void* stream);
int launch_short_conv_bwd(const void* x, const float* weight, const float* bias, const void* init,
                          const int32_t* cu, const void* dy, const void* dfinal, void* dx,
                          float* dweight, float* dbias, void* dinit, void* ws, bool silu,
                          bool bf16, const ConvShape& s, void* stream);
int launch_short_conv_step(const void* x, const float* weight, const float* bias, void* state,
                           void* y, bool silu, bool bf16, const ConvShape& s, void* stream);

struct ScanShape {
  int64_t tokens, nseq, dim, n, ngroups;
  int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;
};
struct ScanInputs {
  const void *x, *dt;
  const float* A;
  const void *B, *C;
  const float* D;
  const void* z;
  const float* dt_bias;
};
struct ScanGradients {
  void *dx, *ddt;
  float* dA;
  void *dB, *dC;
  float* dD;
  void* dz;
  float *ddt_bias, *dinit;
};
int launch_scan_fwd(const ScanInputs& in, const float* init, const int32_t* cu, void* y,
                    float* fin, void* ws, bool softplus, bool bf16, const ScanShape& s,
                    void* stream);
int launch_scan_bwd(const ScanInputs& in, const float* init, const int32_t* cu, const void* dy,
                    const float* dfinal, const ScanGradients& out, void* ws, bool softplus,
                    bool bf16, const ScanShape& s, void* stream);
int launch_scan_step(const ScanInputs& in, float* state, void* y, bool softplus, bool bf16,
                     const ScanShape& s, void* stream);

constexpr int64_t kQuantMaxDim = 16384;
int launch_add_norm_quant(const void* x, const void* res, const float* scale, const float* weight,
                          void* codes, float* scales, void* res_out, int64_t rows, int64_t dim,
                          int64_t group, float eps, bool e4m3, bool xbf16, bool rbf16,
                          void* stream);

}  // namespace ssd
