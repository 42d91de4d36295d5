// ssd_block_launch.h -- host-side launchers of the block operators (internal
// to libssd; declared to users in include/ssd_block.h).  Arguments arrive
// already validated by the C ABI layer; each launcher returns the hipError_t
// of its launches as an int (0 = success).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd_block.h"

namespace ssd {

struct LinattnShape {
  int64_t tokens, nseq, nheads, ngroups, dk, dv;
  bool grouped() const { return ngroups != nheads; }
};

int launch_linattn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                       const float* init, const int32_t* cu, void* o, float* fin, void* ws,
                       float scale, bool bf16, const LinattnShape& s, void* stream);
int launch_linattn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                       const float* init, const int32_t* cu, const void* dout,
                       const float* dfinal, void* dq, void* dk, void* dv, float* dinit,
                       void* ws, float scale, bool bf16, const LinattnShape& s, void* stream);
// Bytes of workspace the launchers above use.
size_t linattn_workspace(const LinattnShape& s, bool bf16, bool backward);

int launch_linattn_step(const void* q, const void* k, const void* v, const float* log_decay,
                        float* state, void* o, float scale, bool bf16, const LinattnShape& s,
                        void* stream);

// Rows of `dim` channels, normed by groups of `group`; weights of `wdim`.
struct NormShape {
  int64_t rows, dim, group, wdim;
};
constexpr int64_t kNormMaxGroup = 16384;

int launch_add_norm_fwd(const void* x, const void* res, const float* scale, const float* weight,
                        void* y, void* res_out, float eps, bool xbf16, bool rbf16,
                        const NormShape& s, void* stream);
int launch_add_norm_bwd(const void* x, const void* res, const float* scale, const float* weight,
                        const void* dy, const void* dres_out, void* dx, void* dres,
                        float* dscale, float* dweight, void* ws, float eps, bool xbf16,
                        bool rbf16, const NormShape& s, void* stream);
int launch_gated_norm_fwd(const void* x, const void* z, const float* weight, void* y, float eps,
                          bool silu, bool first, bool xbf16, bool zbf16, const NormShape& s,
                          void* stream);
int launch_gated_norm_bwd(const void* x, const void* z, const float* weight, const void* dy,
                          void* dx, void* dz, float* dweight, void* ws, float eps, bool silu,
                          bool first, bool xbf16, bool zbf16, const NormShape& s, void* stream);
// Bytes of the partial row sums of one (add norm: of two) gradients.
size_t norm_bwd_workspace(const NormShape& s, int sums);

}  // namespace ssd
