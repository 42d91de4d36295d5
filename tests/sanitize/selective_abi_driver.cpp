// Host-only driver of the C ABI of the operators around a selective state space
// (ssd_selective_api.cpp linked against the stand-in launchers below) and of the plan by
// which they cut packed sequences (ssd_selective_plan.h), built with AddressSanitizer and
// UndefinedBehaviorSanitizer.  Exits non-zero on the first mismatch; the sanitizers abort
// on the first memory or undefined-behaviour error.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "ssd_selective.h"
#include "ssd_selective_launch.h"
#include "ssd_selective_plan.h"

namespace {

struct Call {
  const char* name = "";
  ssd::ConvShape conv{};
  ssd::ScanShape scan{};
  ssd::ScanInputs in{};
  ssd::ScanGradients out{};
  const void* p[4] = {};
  bool flag[4] = {};
  int64_t n[3] = {};
} last;
int ncalls = 0, fail_with = 0, failures = 0;

Call& record(const char* name, const void* a, const void* b, const void* c, const void* d,
             bool f0, bool f1) {
  last = Call{};
  last.name = name;
  const void* p[4] = {a, b, c, d};
  std::memcpy(last.p, p, sizeof p);
  last.flag[0] = f0;
  last.flag[1] = f1;
  ++ncalls;
  return last;
}

}  // namespace

namespace ssd {
int launch_short_conv_fwd(const void*, const float*, const float* bias, const void* init,
                          const int32_t* cu, void*, void* fin, bool silu, bool bf16,
                          const ConvShape& s, void*) {
  record("conv_fwd", bias, init, cu, fin, silu, bf16).conv = s;
  return fail_with;
}
int launch_short_conv_bwd(const void*, const float*, const float*, const void*, const int32_t*,
                          const void*, const void* dfinal, void*, float* dweight, float*,
                          void* dinit, void* ws, bool silu, bool bf16, const ConvShape& s,
                          void*) {
  record("conv_bwd", dfinal, dweight, dinit, ws, silu, bf16).conv = s;
  return fail_with;
}
int launch_short_conv_step(const void* x, const float*, const float* bias, void* state, void* y,
                           bool silu, bool bf16, const ConvShape& s, void*) {
  record("conv_step", x, bias, state, y, silu, bf16).conv = s;
  return fail_with;
}
int launch_scan_fwd(const ScanInputs& in, const float* init, const int32_t* cu, void* y,
                    float* fin, void*, bool softplus, bool bf16, const ScanShape& s, void*) {
  Call& c = record("scan_fwd", init, cu, y, fin, softplus, bf16);
  c.scan = s;
  c.in = in;
  return fail_with;
}
int launch_scan_bwd(const ScanInputs& in, const float* init, const int32_t*, const void* dy,
                    const float* dfinal, const ScanGradients& out, void* ws, bool softplus,
                    bool bf16, const ScanShape& s, void*) {
  Call& c = record("scan_bwd", init, dy, dfinal, ws, softplus, bf16);
  c.scan = s;
  c.in = in;
  c.out = out;
  return fail_with;
}
int launch_scan_step(const ScanInputs& in, float* state, void* y, bool softplus, bool bf16,
                     const ScanShape& s, void*) {
  Call& c = record("scan_step", state, y, nullptr, nullptr, softplus, bf16);
  c.scan = s;
  c.in = in;
  return fail_with;
}
int launch_add_norm_quant(const void*, const void* res, const float*, const float*, void* codes,
                          float* scales, void* res_out, int64_t rows, int64_t dim, int64_t group,
                          float, bool e4m3, bool xbf16, bool rbf16, void*) {
  Call& c = record("quant", res, codes, scales, res_out, e4m3, xbf16);
  c.flag[2] = rbf16;
  c.n[0] = rows;
  c.n[1] = dim;
  c.n[2] = group;
  return fail_with;
}
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

void* at(uintptr_t p) { return reinterpret_cast<void*>(p); }
float* fat(uintptr_t p) { return reinterpret_cast<float*>(p); }
int32_t* iat(uintptr_t p) { return reinterpret_cast<int32_t*>(p); }
constexpr uintptr_t X = 0x7f0000000000, Y = 0x7f1000000000, W = 0x7f2000000000,
                    S0 = 0x7f3000000000, S1 = 0x7f4000000000;

ssd_status conv(const ssd_short_conv_dims& d, int form, uintptr_t init = 0, uintptr_t fin = 0,
                uintptr_t x = X, size_t ws = ~(size_t)0, int act = 1, int dtype = SSD_BF16,
                uintptr_t cu = 0) {
  ncalls = 0;
  const auto a = (ssd_conv_act)act;
  const auto t = (ssd_dtype)dtype;
  if (form == 0)
    return ssd_short_conv_fwd(at(x), fat(W), nullptr, at(init), iat(cu), at(Y), at(fin), a, t, &d,
                              nullptr);
  if (form == 1)
    return ssd_short_conv_bwd(at(x), fat(W), nullptr, nullptr, iat(cu), at(Y), at(init), at(Y),
                              nullptr, nullptr, at(fin), at(S0), ws, a, t, &d, nullptr);
  return ssd_short_conv_step(at(x), fat(W), nullptr, at(init ? init : S0), at(Y), a, t, &d,
                             nullptr);
}

void conv_checks() {
  const ssd_short_conv_dims ok{64, 2, 96, 4, 0};
  CHECK(conv(ok, 0) == SSD_OK && REACHED("conv_fwd") && last.conv.x_stride == 96 &&
        last.conv.nseq == 2 && last.flag[0] && last.flag[1]);
  CHECK(conv(ok, 1) == SSD_OK && REACHED("conv_bwd"));
  CHECK(conv(ok, 2) == SSD_OK && REACHED("conv_step") && last.conv.nseq == 1);
  CHECK(ssd_short_conv_bwd_workspace_bytes(&ok) ==
        ssd::conv_bwd_bytes(ssd::ConvShape{64, 2, 96, 4, 96}));
  const int64_t big[] = {0, -1, INT64_MIN, INT64_MAX, (int64_t)1 << 31, (int64_t)1 << 62};
  for (int64_t v : big)
    for (int field = 0; field < 5; ++field) {
      ssd_short_conv_dims d = ok;
      int64_t* f[] = {&d.tokens, &d.nseq, &d.dim, &d.width, &d.x_stride};
      *f[field] = v;
      for (int form = 0; form < 3; ++form) {
        if ((field == 4 && v == 0) || (field == 1 && form == 2)) continue;
        CHECK(conv(d, form) != SSD_OK && ncalls == 0);
      }
      if (!(field == 4 && v == 0)) CHECK(ssd_short_conv_bwd_workspace_bytes(&d) == 0);
    }
  CHECK(ssd_short_conv_fwd(at(X), fat(W), nullptr, nullptr, nullptr, at(Y), nullptr,
                           SSD_CONV_SILU, SSD_BF16, nullptr, nullptr) == INV);
  const size_t state = 2 * 3 * 96 * 2;
  CHECK(conv(ok, 0, S0, S0) == SSD_OK);
  CHECK(conv(ok, 0, S0, S0 + state) == SSD_OK);
  CHECK(conv(ok, 0, S0, S0 + state - 16) == INV);
  CHECK(conv(ok, 0, S0 + state - 16, S0) == INV);
  CHECK(conv(ok, 1, S1, S1) == INV);
  CHECK(conv(ok, 1, S1, S1 + state) == SSD_OK);
  CHECK(conv(ok, 0, 0, 0, X + 2) == SSD_OK);
  CHECK(conv(ok, 0, 0, 0, X + 1) == INV);
  CHECK(conv(ok, 0, 0, 0, X + 2, 0, 1, SSD_F32) == INV);
  CHECK(conv(ok, 0, 0, 0, X, 0, 2) == INV);
  CHECK(conv(ok, 0, 0, 0, X, 0, 1, 7) == INV);
  CHECK(conv(ok, 0, 0, 0, X, 0, 1, SSD_BF16, 0x1002) == INV);
  const size_t need = ssd_short_conv_bwd_workspace_bytes(&ok);
  CHECK(conv(ok, 1, 0, 0, X, need) == SSD_OK && conv(ok, 1, 0, 0, X, need - 1) == WS);
  ssd_short_conv_dims d = ok;
  d.tokens = 65;                                  // not two equal lengths
  CHECK(conv(d, 0) == INV && conv(d, 0, 0, 0, X, 0, 1, SSD_BF16, 0x1004) == SSD_OK);
  fail_with = 1;
  CHECK(conv(ok, 0) == SSD_ERR_HIP && conv(ok, 1) == SSD_ERR_HIP && conv(ok, 2) == SSD_ERR_HIP);
  fail_with = 0;
}

struct ScanPtrs {
  uintptr_t x = X, dt = X, A = X, B = X, C = X, D = 0, z = 0, bias = 0, init = 0, cu = 0, y = Y,
            fin = 0, dz = 0;
  size_t ws = ~(size_t)0;
  int dtype = SSD_BF16;
};

ssd_status scan(const ssd_selective_scan_dims& d, int form, const ScanPtrs& p = {}) {
  ncalls = 0;
  const auto t = (ssd_dtype)p.dtype;
  if (form == 0)
    return ssd_selective_scan_fwd(at(p.x), at(p.dt), fat(p.A), at(p.B), at(p.C), fat(p.D),
                                  at(p.z), fat(p.bias), fat(p.init), iat(p.cu), at(p.y),
                                  fat(p.fin), at(W), p.ws, 1, t, &d, nullptr);
  if (form == 1)
    return ssd_selective_scan_bwd(at(p.x), at(p.dt), fat(p.A), at(p.B), at(p.C), fat(p.D),
                                  at(p.z), fat(p.bias), nullptr, iat(p.cu), at(p.y), fat(p.init),
                                  at(Y), at(Y), fat(Y), at(Y), at(Y), nullptr,
                                  at(p.dz ? p.dz : p.z), nullptr, fat(p.fin), at(W), p.ws, 1, t,
                                  &d, nullptr);
  return ssd_selective_scan_step(at(p.x), at(p.dt), fat(p.A), at(p.B), at(p.C), fat(p.D), at(p.z),
                                 fat(p.bias), fat(p.init ? p.init : S0), at(p.y), 1, t, &d,
                                 nullptr);
}

void scan_checks() {
  const char* names[] = {"scan_fwd", "scan_bwd", "scan_step"};
  const ssd_selective_scan_dims ok{96, 3, 80, 16, 2, 0, 0, 0, 0, 0};
  for (int form = 0; form < 3; ++form) {
    CHECK(scan(ok, form) == SSD_OK && REACHED(names[form]) && last.scan.b_stride == 32 &&
          last.scan.x_stride == 80 && last.scan.nseq == (form == 2 ? 1 : 3));
    const int64_t big[] = {0, -1, INT64_MIN, INT64_MAX, (int64_t)1 << 31, (int64_t)1 << 62};
    for (int64_t v : big)
      for (int field = 0; field < 10; ++field) {
        ssd_selective_scan_dims d = ok;
        int64_t* f[] = {&d.tokens, &d.nseq, &d.dim, &d.dstate, &d.ngroups,
                        &d.x_stride, &d.dt_stride, &d.z_stride, &d.b_stride, &d.c_stride};
        *f[field] = v;
        if ((field > 4 && v == 0) || (field == 1 && form == 2)) continue;
        CHECK(scan(d, form) != SSD_OK && ncalls == 0);
        if (form == 0) CHECK(ssd_selective_scan_fwd_workspace_bytes(&d, SSD_BF16) == 0);
        if (form == 1) CHECK(ssd_selective_scan_bwd_workspace_bytes(&d, SSD_BF16) == 0);
      }
    ssd_selective_scan_dims d = ok;
    d.b_stride = 33;
    CHECK(scan(d, form) == INV);
    ScanPtrs f32;
    f32.dtype = SSD_F32;
    CHECK(scan(d, form, f32) == SSD_OK);
    d = ok;
    d.dstate = 24;
    CHECK(scan(d, form) == UNS);
    d = ok;
    d.ngroups = 3;
    CHECK(scan(d, form) == INV);
    d = ok;
    d.tokens = 1 << 21, d.nseq = 1 << 21, d.dim = 1 << 20, d.ngroups = 1;
    CHECK(scan(d, form) == UNS);
    uintptr_t ScanPtrs::*needed[] = {&ScanPtrs::x, &ScanPtrs::dt, &ScanPtrs::A, &ScanPtrs::B,
                                     &ScanPtrs::C, &ScanPtrs::y};
    for (auto m : needed) {
      ScanPtrs p;
      p.*m = 0;
      CHECK(scan(ok, form, p) == INV && ncalls == 0);
      p.*m = X + 1;
      CHECK(scan(ok, form, p) == INV && ncalls == 0);
    }
    ScanPtrs p;
    p.D = X + 4;
    CHECK(scan(ok, form, p) == INV);
    p = ScanPtrs{};
    p.z = X + 2;
    p.dz = X;
    CHECK(scan(ok, form, p) == SSD_OK && last.in.z == at(X + 2));
    fail_with = 1;
    CHECK(scan(ok, form) == SSD_ERR_HIP);
    fail_with = 0;
  }
  ScanPtrs p;
  p.dz = X;                                          // dz without z
  CHECK(scan(ok, 1, p) == INV);
  const size_t state = 4 * 3 * 80 * 16;
  p = ScanPtrs{};
  p.init = S0;
  p.fin = S0;
  CHECK(scan(ok, 0, p) == SSD_OK && scan(ok, 1, p) == INV);
  p.fin = S0 + state;
  CHECK(scan(ok, 0, p) == SSD_OK && scan(ok, 1, p) == SSD_OK);
  p.fin = S0 + state - 16;
  CHECK(scan(ok, 0, p) == INV && scan(ok, 1, p) == INV);
  ssd_selective_scan_dims d = ok;
  d.tokens = 97;
  CHECK(scan(d, 0) == INV && scan(d, 1) == INV);
  for (int form = 0; form < 2; ++form) {
    ScanPtrs w;
    w.ws = form == 0 ? ssd_selective_scan_fwd_workspace_bytes(&ok, SSD_BF16)
                     : ssd_selective_scan_bwd_workspace_bytes(&ok, SSD_BF16);
    CHECK(w.ws > 0 && scan(ok, form, w) == SSD_OK);
    --w.ws;
    CHECK(scan(ok, form, w) == WS);
  }
}

ssd_status quant(int64_t rows, int64_t dim, int64_t group, float eps = 1e-5f, int code = 0,
                 uintptr_t x = X, uintptr_t codes = Y) {
  ncalls = 0;
  return ssd_add_norm_quant_fwd(at(x), nullptr, nullptr, nullptr, at(codes), fat(W), nullptr, rows,
                                dim, group, eps, (ssd_code)code, SSD_BF16, SSD_F32, nullptr);
}

void quant_checks() {
  CHECK(quant(3, 512, 128) == SSD_OK && REACHED("quant") && last.n[0] == 3 && last.n[1] == 512 &&
        last.n[2] == 128 && last.flag[1] && !last.flag[2]);
  CHECK(quant(3, 515, 515) == SSD_OK);
  CHECK(quant(3, 512, 96) == INV && quant(3, 96, 48) == UNS && quant(3, 16385, 16385) == UNS);
  const int64_t bad[] = {0, -1, INT64_MIN, INT64_MAX, (int64_t)1 << 31};
  for (int64_t v : bad)
    CHECK(quant(v, 512, 128) != SSD_OK && quant(3, v, 128) != SSD_OK && quant(3, 512, v) != SSD_OK);
  const float nan = std::nanf("");
  CHECK(quant(3, 512, 128, 0.0f) == INV && quant(3, 512, 128, nan) == INV);
  CHECK(quant(3, 512, 128, 1e-5f, 2) == INV && quant(3, 512, 128, 1e-5f, 0, X + 2) == INV &&
        quant(3, 512, 128, 1e-5f, 0, X, 0) == INV);
  fail_with = 1;
  CHECK(quant(3, 512, 128) == SSD_ERR_HIP);
  fail_with = 0;
}

// ---- the plan
ssd::Run run_of(const ssd::RunGrid& g, int slot) {
  if (g.cu == nullptr) return ssd::equal_run(g, slot);
  int seq = 0;
  for (int i = 1; i < g.nseq; ++i)
    if (ssd::first_slot(g, ssd::seq_bound(g, g.cu[i]), i) <= slot) seq = i;
  return ssd::packed_run(g, slot, seq, ssd::seq_bound(g, g.cu[seq]),
                         ssd::seq_bound(g, g.cu[seq + 1]));
}

// Every token lies in one run of its own sequence, and every sequence has its runs in a row.
void check_runs(const ssd::RunGrid& g, int64_t slots, const std::vector<int32_t>& cu) {
  std::vector<int> seen(g.tokens, 0), runs(g.nseq, 0);
  for (int slot = 0; slot < slots; ++slot) {
    const ssd::Run r = run_of(g, slot);
    if (!r.on) continue;
    CHECK(r.seq >= 0 && r.seq < g.nseq);
    CHECK(r.seq_begin == cu[r.seq] && r.seq_end == cu[r.seq + 1]);
    CHECK(r.first + r.index == slot && r.first >= 0 && r.first + r.count <= slots);
    CHECK(r.begin >= r.seq_begin && r.begin <= r.end && r.end <= r.seq_end &&
          r.end - r.begin <= g.run);
    ++runs[r.seq];
    for (int t = r.begin; t < r.end; ++t) ++seen[t];
    CHECK(r.count == runs[r.seq] || r.index + 1 < r.count);
  }
  for (int t = 0; t < g.tokens; ++t) CHECK(seen[t] == (t >= cu.front() && t < cu.back()));
  for (int i = 0; i < g.nseq; ++i) {
    const int len = cu[i + 1] - cu[i];
    CHECK(runs[i] == (len > 0 ? (len + g.run - 1) / g.run : 1));
  }
}

void plan_checks() {
  std::mt19937 rng(11);
  auto below = [&](int n) { return (int)(rng() % (unsigned)n); };
  for (int64_t d : {1, 2, 3, 7, 8, 24, 28, 64, 1000, 65537, INT32_MAX - 7, INT32_MAX}) {
    const ssd::Divide by(d);
    for (uint32_t n : {0u, 1u, (uint32_t)d - 1, (uint32_t)d, (uint32_t)INT32_MAX})
      CHECK(by.of(n) == n / (uint32_t)d);
    for (int i = 0; i < 1000; ++i) {
      const uint32_t n = rng() >> 1;
      CHECK(by.of(n) == n / (uint32_t)d);
    }
  }
  for (int i = 0; i < 200; ++i) {
    const int nseq = 1 + below(i % 2 ? 5 : 90), tokens = 1 + below(3000);
    std::vector<int32_t> cu(nseq + 1);
    for (auto& v : cu) v = below(tokens + 1);
    std::sort(cu.begin(), cu.end());
    if (i % 3) cu.front() = 0, cu.back() = tokens;
    const ssd::ScanShape s{tokens, nseq, 64 * (1 + below(40)), 16, 1, 0, 0, 0, 0, 0};
    for (int which = 0; which < 4; ++which) {
      const bool back = which % 2;
      const ssd::ConvShape c{tokens, nseq, s.dim, 4, s.dim};
      const int64_t run = which < 2 ? ssd::scan_run(s, back) : ssd::conv_run(c, back);
      const int64_t slots = which < 2 ? ssd::scan_slots(s, back) : ssd::conv_slots(c, back);
      const auto g = ssd::make_run_grid(cu.data(), tokens, nseq, run);
      CHECK(ssd::run_slots(g) == slots);
      check_runs(g, slots, cu);
      if (which == 1) {
        // marks: each run's ceil(len / kMark) from its first on, in order and inside their number
        CHECK(run % ssd::kMark == 0);
        int64_t before = 0;
        for (int slot = 0; slot < slots; ++slot) {
          const ssd::Run r = run_of(g, slot);
          if (!r.on) continue;
          const int64_t first = ssd::first_mark(r, slot);
          CHECK(first >= before);
          before = first + (r.end - r.begin + ssd::kMark - 1) / ssd::kMark;
          CHECK(before <= ssd::scan_marks(s));
        }
      }
      // and with equal lengths: fewer slots, never more than those that workspaces hold
      std::vector<int32_t> even(nseq + 1);
      const int len = 1 + below(300);
      for (int j = 0; j <= nseq; ++j) even[j] = j * len;
      const auto e = ssd::make_run_grid(nullptr, (int64_t)nseq * len, nseq, run);
      CHECK(ssd::run_slots(e) <= e.tokens / e.run + e.nseq);
      check_runs(e, ssd::run_slots(e), even);
      // bounds that descend or lie outside give runs inside the tokens and the slots all the same
      std::vector<int32_t> wild(nseq + 1);
      for (auto& v : wild) v = (int32_t)(rng() >> 1) % (3 * tokens) - tokens;
      wild[below(nseq + 1)] = i % 2 ? INT32_MIN : INT32_MAX;
      auto w = g;
      w.cu = wild.data();
      for (int slot = 0; slot < slots; ++slot)
        for (int seq = 0; seq < nseq; ++seq) {
          const ssd::Run r = ssd::packed_run(w, slot, seq, ssd::seq_bound(w, wild[seq]),
                                             ssd::seq_bound(w, wild[seq + 1]));
          if (!r.on) continue;
          CHECK(r.begin >= 0 && r.begin <= r.end && r.end <= tokens && r.end - r.begin <= w.run);
          CHECK(r.first >= 0 && r.first + r.count <= slots);
          if (which == 1)
            CHECK(ssd::first_mark(r, slot) + (r.end - r.begin + 7) / 8 <= ssd::scan_marks(s));
        }
    }
  }
  // runs of a whole sequence where the sequences alone fill the chip
  const ssd::ScanShape many{64 * 1024, 64, 5120, 16, 1, 0, 0, 0, 0, 0};
  CHECK(ssd::scan_run(many, false) == 4096 && ssd::scan_run(many, true) == 4096);
  // the largest shapes that are taken have workspaces of no more than 2^63 bytes
  for (int64_t tokens : {(int64_t)1, (int64_t)1 << 24, (int64_t)INT32_MAX})
    for (int64_t dim : {(int64_t)1, (int64_t)4096, (int64_t)1 << 20}) {
      const ssd::ScanShape s{tokens, 1, dim, 64, 1, 0, 0, 0, 0, 0};
      if (ssd::scan_grid_fits(s, true)) CHECK(ssd::bwd_layout(s).all < (size_t)1 << 62);
      if (ssd::scan_grid_fits(s, false)) CHECK(ssd::scan_fwd_bytes(s) < (size_t)1 << 62);
    }
}

}  // namespace

int main() {
  conv_checks();
  scan_checks();
  quant_checks();
  plan_checks();
  if (failures != 0) return 1;
  std::printf("all checks passed\n");
  return 0;
}
