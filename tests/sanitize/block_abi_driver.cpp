// Host-only driver of the block operators' C ABI (ssd_block_api.cpp linked against the
// stand-in launchers below), built with AddressSanitizer and
// UndefinedBehaviorSanitizer.  It exercises every entry point's checks, with sizes
// whose products pass 64 bits among them, and for valid calls what reaches the
// launchers.  Exits non-zero on the first mismatch; the sanitizers abort on the first
// memory or undefined-behaviour error.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "ssd_block.h"
#include "ssd_block_launch.h"

namespace {

struct Call {
  const char* name = "";
  ssd::LinattnShape la{};
  ssd::NormShape norm{};
  const void* p[4] = {};
  bool flag[4] = {};
  float f = 0;
} last;
int ncalls = 0, fail_with = 0, failures = 0;

int record(const char* name, const void* a, const void* b, const void* c, const void* d, float f,
           bool f0 = false, bool f1 = false, bool f2 = false, bool f3 = false) {
  last = Call{};
  last.name = name;
  const void* p[4] = {a, b, c, d};
  const bool flag[4] = {f0, f1, f2, f3};
  std::memcpy(last.p, p, sizeof p);
  std::memcpy(last.flag, flag, sizeof flag);
  last.f = f;
  ++ncalls;
  return fail_with;
}

}  // namespace

namespace ssd {
int launch_linattn_fwd(const void* q, const void*, const void*, const float*, const float* init,
                       const int32_t* cu, void* o, float*, void*, float scale, bool bf16,
                       const LinattnShape& s, void*) {
  const int r = record("linattn_fwd", q, init, cu, o, scale, bf16);
  last.la = s;
  return r;
}
int launch_linattn_bwd(const void*, const void*, const void*, const float*, const float*,
                       const int32_t* cu, const void* dout, const float* dfinal, void*, void*,
                       void*, float* dinit, void*, float scale, bool bf16, const LinattnShape& s,
                       void*) {
  const int r = record("linattn_bwd", cu, dout, dfinal, dinit, scale, bf16);
  last.la = s;
  return r;
}
size_t linattn_workspace(const LinattnShape&, bool bf16, bool backward) {
  return 1024 * (1 + bf16 + 2 * backward);
}
int launch_linattn_step(const void* q, const void*, const void* v, const float*, float* state,
                        void* o, float scale, bool bf16, const LinattnShape& s, void*) {
  const int r = record("linattn_step", q, v, state, o, scale, bf16);
  last.la = s;
  return r;
}
int launch_add_norm_fwd(const void* x, const void* res, const float*, const float*, void* y,
                        void* res_out, float eps, bool xb, bool rb, const NormShape& s, void*) {
  const int r = record("add_norm_fwd", x, res, y, res_out, eps, xb, rb);
  last.norm = s;
  return r;
}
int launch_add_norm_bwd(const void*, const void*, const float*, const float*, const void*,
                        const void*, void* dx, void* dres, float* dscale, float* dweight, void*,
                        float eps, bool xb, bool rb, const NormShape& s, void*) {
  const int r = record("add_norm_bwd", dx, dres, dscale, dweight, eps, xb, rb);
  last.norm = s;
  return r;
}
int launch_gated_norm_fwd(const void* x, const void* z, const float* w, void* y, float eps,
                          bool silu, bool first, bool xb, bool zb, const NormShape& s, void*) {
  const int r = record("gated_norm_fwd", x, z, w, y, eps, silu, first, xb, zb);
  last.norm = s;
  return r;
}
int launch_gated_norm_bwd(const void*, const void* z, const float*, const void*, void* dx,
                          void* dz, float* dweight, void*, float eps, bool silu, bool first,
                          bool xb, bool zb, const NormShape& s, void*) {
  const int r = record("gated_norm_bwd", z, dx, dz, dweight, eps, silu, first, xb, zb);
  last.norm = s;
  return r;
}
size_t norm_bwd_workspace(const NormShape&, int sums) { return 512 * (size_t)sums; }
}  // namespace ssd

namespace {

#define CHECK(cond)                                                                 \
  do {                                                                              \
    if (!(cond)) {                                                                  \
      std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                                   \
    }                                                                               \
  } while (0)
#define REACHED(n) (ncalls == 1 && std::strcmp(last.name, n) == 0)

constexpr ssd_status INV = SSD_ERR_INVALID_ARGUMENT, UNS = SSD_ERR_UNSUPPORTED,
                     WS = SSD_ERR_WORKSPACE;

// Real, 16-byte aligned allocations that the stand-ins never dereference.
alignas(16) unsigned char arena[1 << 16];
float* P(int k) { return (float*)(arena + 1024 * k); }
float* MIS(int k) { return (float*)(arena + 1024 * k + 4); }

void reset() {
  ncalls = 0;
  fail_with = 0;
}

ssd_linattn_dims ldims(int64_t T = 512, int64_t n = 2, int64_t H = 4, int64_t G = 2,
                       int64_t K = 128, int64_t V = 64) {
  return ssd_linattn_dims{T, n, H, G, K, V};
}

struct Fwd {
  const void *q = P(1), *k = P(2), *v = P(3);
  const float *ld = P(4), *init = nullptr;
  const int32_t* cu = nullptr;
  void* o = P(5);
  float* fin = nullptr;
  void* ws = P(20);
  size_t n = 1 << 20;
  ssd_dtype dt = SSD_BF16;
  ssd_status operator()(const ssd_linattn_dims* d) const {
    return ssd_linattn_fwd(q, k, v, ld, init, cu, o, fin, ws, n, 0.5f, dt, d, nullptr);
  }
};
struct Bwd {
  const void *q = P(1), *k = P(2), *v = P(3), *dout = P(6);
  const float *ld = P(4), *init = nullptr, *dfinal = nullptr;
  const int32_t* cu = nullptr;
  void *dq = P(7), *dk = P(8), *dv = P(9);
  float* dinit = nullptr;
  void* ws = P(20);
  size_t n = 1 << 20;
  ssd_dtype dt = SSD_BF16;
  ssd_status operator()(const ssd_linattn_dims* d) const {
    return ssd_linattn_bwd(q, k, v, ld, init, cu, dout, dfinal, dq, dk, dv, dinit, ws, n, 0.5f,
                           dt, d, nullptr);
  }
};
struct Step {
  const void *q = P(1), *k = P(2), *v = P(3);
  const float* ld = P(4);
  float* state = P(5);
  void* o = P(6);
  ssd_dtype dt = SSD_BF16;
  ssd_status operator()(const ssd_linattn_dims* d) const {
    return ssd_linattn_step(q, k, v, ld, state, o, 0.5f, dt, d, nullptr);
  }
};

void test_linattn_dims() {
  struct Case {
    ssd_linattn_dims d;
    ssd_status want;
  } cases[] = {
      {ldims(0), INV},
      {ldims(INT64_MAX), INV},
      {ldims(INT64_MIN), INV},
      {ldims(512, 2, 0), INV},
      {ldims(512, 2, 4, 3), INV},
      {ldims(512, 2, 4, 0), INV},
      {ldims(512, 2, 4, 2, 96), UNS},
      {ldims(512, 2, 4, 2, 128, 256), UNS},
      {ldims(512, 2, 4, 2, INT64_MIN), INV},
      {ldims(1 << 30), UNS},
      // products that would pass 32 and 64 bits
      {ldims(INT32_MAX, 1, INT32_MAX, 1), UNS},
      {ldims(1, 1, INT32_MAX, 1, INT32_MAX, INT32_MAX), UNS},
      {ldims(1, 1, 1 << 16, 1), UNS},
  };
  for (const Case& c : cases) {
    reset();
    CHECK(Fwd()(&c.d) == c.want);
    CHECK(Bwd()(&c.d) == c.want);
    CHECK(Step()(&c.d) == c.want);
    CHECK(ssd_linattn_fwd_workspace_bytes(&c.d, SSD_F32) == 0);
    CHECK(ssd_linattn_bwd_workspace_bytes(&c.d, SSD_BF16) == 0);
    CHECK(ncalls == 0);
  }
  // the number of sequences: read by all but the single token's call
  for (int64_t n : {(int64_t)0, INT64_MIN, INT64_MAX}) {
    const ssd_linattn_dims d = ldims(512, n);
    reset();
    CHECK(Fwd()(&d) == INV && Bwd()(&d) == INV);
    CHECK(Step()(&d) == SSD_OK && REACHED("linattn_step"));
  }
  const ssd_linattn_dims many = ldims(512, INT32_MAX), odd = ldims(512, 3);
  reset();
  Fwd packed;
  packed.cu = (const int32_t*)P(10);
  CHECK(packed(&many) == UNS && Fwd()(&odd) == INV && Bwd()(&odd) == INV && ncalls == 0);
  CHECK(packed(&odd) == SSD_OK && REACHED("linattn_fwd"));
  CHECK(Fwd()(nullptr) == INV && Bwd()(nullptr) == INV && Step()(nullptr) == INV);
  CHECK(ssd_linattn_fwd_workspace_bytes(nullptr, SSD_F32) == 0);
}

void test_linattn_arguments() {
  const ssd_linattn_dims d = ldims();
  reset();
#define BAD(T, field, value)                 \
  do {                                       \
    T c;                                     \
    c.field = value;                         \
    CHECK(c(&d) == INV);                     \
  } while (0)
#define BAD_PTR(T, field)                    \
  BAD(T, field, nullptr);                    \
  BAD(T, field, MIS(11))
  BAD_PTR(Fwd, q); BAD_PTR(Fwd, k); BAD_PTR(Fwd, v); BAD_PTR(Fwd, ld); BAD_PTR(Fwd, o);
  BAD(Fwd, init, MIS(11)); BAD(Fwd, fin, MIS(11)); BAD(Fwd, cu, (const int32_t*)(arena + 2));
  BAD_PTR(Bwd, q); BAD_PTR(Bwd, k); BAD_PTR(Bwd, v); BAD_PTR(Bwd, ld); BAD_PTR(Bwd, dout);
  BAD_PTR(Bwd, dq); BAD_PTR(Bwd, dk); BAD_PTR(Bwd, dv); BAD(Bwd, init, MIS(11));
  BAD(Bwd, dfinal, MIS(11)); BAD(Bwd, dinit, MIS(11)); BAD(Bwd, cu, (const int32_t*)(arena + 2));
  BAD_PTR(Step, q); BAD_PTR(Step, k); BAD_PTR(Step, v); BAD_PTR(Step, ld);
  BAD_PTR(Step, state); BAD_PTR(Step, o);
  CHECK(ncalls == 0);
  // workspaces, in both types
  for (ssd_dtype dt : {SSD_F32, SSD_BF16}) {
    Fwd f;
    Bwd b;
    f.dt = b.dt = dt;
    f.n = ssd_linattn_fwd_workspace_bytes(&d, dt);
    b.n = ssd_linattn_bwd_workspace_bytes(&d, dt);
    CHECK(f.n == 1024u * (1 + dt) && b.n == 1024u * (3 + dt));
    reset();
    CHECK(f(&d) == SSD_OK && REACHED("linattn_fwd") && last.flag[0] == (dt == SSD_BF16));
    reset();
    CHECK(b(&d) == SSD_OK && REACHED("linattn_bwd") && last.f == 0.5f);
    --f.n;
    --b.n;
    reset();
    CHECK(f(&d) == WS && b(&d) == WS);
    ++f.n;
    ++b.n;
    f.ws = b.ws = MIS(20);
    CHECK(f(&d) == WS && b(&d) == WS);
    f.ws = b.ws = nullptr;
    CHECK(f(&d) == WS && b(&d) == WS && ncalls == 0);
  }
  // states: 2 * 4 * 128 * 64 floats; continued in place, or apart
  const size_t n = 4u * 2 * 4 * 128 * 64;
  unsigned char* big = (unsigned char*)std::aligned_alloc(16, 3 * n);
  for (int64_t off : {(int64_t)16, (int64_t)n - 16, -(int64_t)n + 16}) {
    Fwd f;
    f.init = (const float*)(big + n);
    f.fin = (float*)(big + n + off);
    CHECK(f(&d) == INV);
  }
  reset();
  Fwd f;
  f.init = (const float*)(big + n);
  f.fin = (float*)(big + n);
  CHECK(f(&d) == SSD_OK && REACHED("linattn_fwd") && last.p[1] == big + n);
  for (int64_t off : {(int64_t)n, -(int64_t)n}) {
    f.fin = (float*)(big + n + off);
    CHECK(f(&d) == SSD_OK);
  }
  for (int64_t off : {(int64_t)0, (int64_t)16, (int64_t)n - 16, -(int64_t)n + 16}) {
    Bwd b;
    b.dfinal = (const float*)(big + n);
    b.dinit = (float*)(big + n + off);
    reset();
    CHECK(b(&d) == INV && ncalls == 0);
  }
  Bwd b;
  b.dfinal = (const float*)(big + n);
  b.dinit = (float*)(big + 2 * n);
  CHECK(b(&d) == SSD_OK && REACHED("linattn_bwd") && last.p[3] == big + 2 * n);
  std::free(big);
  // what reaches the launchers, and a launch that fails
  reset();
  CHECK(Step()(&d) == SSD_OK && REACHED("linattn_step"));
  CHECK(last.la.tokens == 512 && last.la.nseq == 1 && last.la.dk == 128 && last.la.dv == 64);
  CHECK(last.la.grouped() && last.p[2] == P(5) && last.p[3] == P(6));
  fail_with = 98;
  CHECK(Fwd()(&d) == SSD_ERR_HIP && Bwd()(&d) == SSD_ERR_HIP && Step()(&d) == SSD_ERR_HIP);
  reset();
}

ssd_status add_fwd(int64_t rows, int64_t dim, float eps = 1e-5f, const void* x = P(1),
                   const void* res = P(2), const float* s = P(3), const float* w = P(4),
                   void* y = P(5), void* ro = P(6)) {
  return ssd_add_norm_fwd(x, res, s, w, y, ro, rows, dim, eps, SSD_BF16, SSD_F32, nullptr);
}
ssd_status add_bwd(int64_t rows, int64_t dim, float eps = 1e-5f, const void* res = P(2),
                   const float* s = P(3), float* ds = P(9), void* dres = P(8), void* ws = P(20),
                   size_t n = 1 << 20) {
  return ssd_add_norm_bwd(P(1), res, s, P(4), P(5), P(6), P(7), dres, ds, P(10), ws, n, rows, dim,
                          eps, SSD_F32, SSD_BF16, nullptr);
}

void test_add_norm() {
  reset();
  for (int64_t rows : {(int64_t)0, INT64_MIN, (int64_t)INT32_MAX + 1, INT64_MAX})
    CHECK(add_fwd(rows, 64) == INV && add_bwd(rows, 64) == INV &&
          ssd_add_norm_bwd_workspace_bytes(rows, 64) == 0);
  for (int64_t dim : {(int64_t)0, INT64_MIN, INT64_MAX})
    CHECK(add_fwd(4, dim) == INV && add_bwd(4, dim) == INV &&
          ssd_add_norm_bwd_workspace_bytes(4, dim) == 0);
  for (int64_t dim : {(int64_t)16385, (int64_t)INT32_MAX})
    CHECK(add_fwd(4, dim) == UNS && add_bwd(4, dim) == UNS);
  for (float eps : {0.0f, -1.0f, NAN, -INFINITY})
    CHECK(add_fwd(4, 64, eps) == INV && add_bwd(4, 64, eps) == INV);
  CHECK(add_fwd(4, 64, 1e-5f, nullptr) == INV && add_fwd(4, 64, 1e-5f, MIS(1)) == INV);
  CHECK(add_fwd(4, 64, 1e-5f, P(1), MIS(2)) == INV);
  CHECK(add_fwd(4, 64, 1e-5f, P(1), P(2), MIS(3)) == INV);
  CHECK(add_fwd(4, 64, 1e-5f, P(1), P(2), P(3), MIS(4)) == INV);
  CHECK(add_fwd(4, 64, 1e-5f, P(1), P(2), P(3), P(4), nullptr) == INV);
  CHECK(add_fwd(4, 64, 1e-5f, P(1), P(2), P(3), P(4), P(5), MIS(6)) == INV);
  CHECK(add_bwd(4, 64, 1e-5f, P(2), nullptr) == INV);          // the gradient of no scale
  CHECK(add_bwd(4, 64, 1e-5f, nullptr) == INV);                // and of no residual
  const size_t need = ssd_add_norm_bwd_workspace_bytes(4, 64);
  CHECK(need == 1024);
  CHECK(add_bwd(4, 64, 1e-5f, P(2), P(3), P(9), P(8), P(20), need - 1) == WS);
  CHECK(add_bwd(4, 64, 1e-5f, P(2), P(3), P(9), P(8), nullptr, need) == WS);
  CHECK(ncalls == 0);
  CHECK(add_fwd(INT32_MAX, 16384, 1e-5f, P(1), nullptr, nullptr, nullptr, P(1), nullptr) ==
        SSD_OK);
  CHECK(REACHED("add_norm_fwd") && last.flag[0] && !last.flag[1] && last.p[1] == nullptr);
  CHECK(last.norm.rows == INT32_MAX && last.norm.dim == 16384 && last.norm.group == 16384);
  reset();
  CHECK(add_bwd(4, 64, 1e-5f, P(2), P(3), P(9), P(8), P(20), need) == SSD_OK);
  CHECK(REACHED("add_norm_bwd") && !last.flag[0] && last.flag[1] && last.p[2] == P(9));
  fail_with = 1;
  CHECK(add_fwd(4, 64) == SSD_ERR_HIP && add_bwd(4, 64) == SSD_ERR_HIP);
  reset();
}

void test_gated_norm() {
  using D = ssd_gated_norm_dims;
  auto fwd = [](const D* d, const void* x = P(1), const void* z = P(2), const float* w = P(3),
                void* y = P(4), float eps = 1e-5f) {
    return ssd_gated_norm_fwd(x, z, w, y, eps, SSD_GATE_SIGMOID, 7, SSD_F32, SSD_BF16, d,
                              nullptr);
  };
  auto bwd = [](const D* d, const void* z = P(2), void* dz = P(6), float* dw = P(7),
                void* ws = P(20), size_t n = 1 << 20) {
    return ssd_gated_norm_bwd(P(1), z, P(3), P(4), P(5), dz, dw, ws, n, 1e-5f, SSD_GATE_SILU, 0,
                              SSD_BF16, SSD_F32, d, nullptr);
  };
  struct Case {
    D d;
    ssd_status want;
  } cases[] = {
      {{0, 128, 64, 64}, INV},
      {{4, 0, 64, 64}, INV},
      {{4, 128, 0, 64}, INV},
      {{4, 128, -64, -64}, INV},
      {{4, 128, 48, 48}, INV},
      {{4, 128, 256, 256}, INV},
      {{4, 128, 64, 32}, INV},
      {{INT64_MAX, INT64_MAX, INT64_MAX, INT64_MAX}, INV},
      {{INT64_MIN, 128, 64, 64}, INV},
      {{4, INT32_MAX, INT32_MAX, INT32_MAX}, UNS},
      {{4, 20000, 20000, 20000}, UNS},
      {{4, 1 << 28, 1 << 14, 1 << 14}, UNS},
      {{4, 1 << 20, 8, 8}, UNS},
  };
  reset();
  for (const Case& c : cases) {
    CHECK(fwd(&c.d) == c.want && bwd(&c.d) == c.want);
    CHECK(ssd_gated_norm_bwd_workspace_bytes(&c.d) == 0);
  }
  const D d{4, 128, 64, 64};
  CHECK(fwd(nullptr) == INV && bwd(nullptr) == INV);
  CHECK(ssd_gated_norm_bwd_workspace_bytes(nullptr) == 0);
  CHECK(fwd(&d, nullptr) == INV && fwd(&d, MIS(1)) == INV && fwd(&d, P(1), MIS(2)) == INV);
  CHECK(fwd(&d, P(1), P(2), MIS(3)) == INV && fwd(&d, P(1), P(2), P(3), nullptr) == INV);
  CHECK(fwd(&d, P(1), P(2), P(3), P(4), 0.0f) == INV);
  CHECK(bwd(&d, nullptr) == INV && bwd(&d, P(2), nullptr) == INV);
  CHECK(bwd(&d, P(2), P(6), MIS(7)) == INV);
  CHECK(bwd(&d, P(2), P(6), P(7), P(20), 511) == WS && bwd(&d, P(2), P(6), P(7), MIS(20)) == WS);
  CHECK(ncalls == 0);
  CHECK(fwd(&d, P(1), nullptr, nullptr, P(1)) == SSD_OK && REACHED("gated_norm_fwd"));
  CHECK(!last.flag[0] && last.flag[1] && !last.flag[2] && last.flag[3]);
  CHECK(last.norm.group == 64 && last.norm.wdim == 64 && last.norm.dim == 128);
  reset();
  CHECK(bwd(&d, nullptr, nullptr, nullptr, P(20), 512) == SSD_OK && REACHED("gated_norm_bwd"));
  CHECK(last.flag[0] && !last.flag[1] && last.flag[2] && !last.flag[3] && last.p[1] == P(5));
  fail_with = 1;
  CHECK(fwd(&d) == SSD_ERR_HIP && bwd(&d) == SSD_ERR_HIP);
  reset();
}

}  // namespace

int main() {
  test_linattn_dims();
  test_linattn_arguments();
  test_add_norm();
  test_gated_norm();
  if (failures) {
    std::fprintf(stderr, "block_abi_driver: %d check(s) failed\n", failures);
    return 1;
  }
  std::printf("block_abi_driver: all checks passed\n");
  return 0;
}
