// Host-side exercise of the node layers' C ABI for an AddressSanitizer / UBSan
// build of their argument checks, layouts and workspace sizes.  It touches no
// device memory: every call below must be answered or rejected on the host
// before any launch.  Exit status 0 when every check holds.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <string>
#include <vector>

#include "tpconv_layers.h"

static int failures = 0;
#define CHECK(cond)                                                    \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "check failed (line %d): %s\n", __LINE__, #cond); \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

static void* fake(uintptr_t a) { return reinterpret_cast<void*>(a); }

static void norms() {
  std::string sixteen = "3x0e", many = "3x0e";
  for (int i = 1; i < 16; ++i) sixteen += "+2x1o";
  for (int i = 1; i < 17; ++i) many += "+2x1o";
  const char* good[] = {"1x0e", "1024x0e", "64x0e+64x1o+64x2e+64x3o", "5x0o+7x0e+3x1e+8193x0e", sixteen.c_str()};
  for (const char* irreps : good)
    for (int t = 0; t < 4; ++t) {
      tpconv_norm_desc d{irreps, 1e-5f, t & 1, t >> 1};
      tpconv_norm n = nullptr;
      CHECK(tpconv_norm_create(&n, &d) == TPCONV_SUCCESS && n);
      int64_t F = 0, w = 0, b = 0;
      int32_t irs = 0;
      CHECK(tpconv_norm_info(n, &F, &irs, &w, &b) == TPCONV_SUCCESS && F > 0 && irs > 0 && w >= b);
      CHECK(tpconv_norm_info(n, nullptr, nullptr, nullptr, nullptr) == TPCONV_SUCCESS);
      size_t last = 0;
      for (int64_t N : {0ll, 1ll, 63ll, 4096ll, 2147483646ll}) {
        size_t s = 0;
        CHECK(tpconv_norm_workspace_size(n, N, &s) == TPCONV_SUCCESS && s >= last);
        last = s;
      }
      CHECK(tpconv_norm_workspace_size(n, -1, &last) != TPCONV_SUCCESS);
      CHECK(tpconv_norm_forward(n, 4, nullptr, nullptr, nullptr, fake(64), nullptr, nullptr) != TPCONV_SUCCESS);
      CHECK(tpconv_norm_backward(n, 4, fake(64), nullptr, (float*)fake(64), nullptr, nullptr, (float*)fake(64), nullptr,
                                 fake(72), size_t(1) << 40, nullptr) == TPCONV_ERROR_WORKSPACE);
      CHECK(tpconv_norm_destroy(n) == TPCONV_SUCCESS);
    }
  const char* bad[] = {nullptr, "", "x0e", "8x4e", "8x0e+", "-3x0e", "8x0f", "99999999999999999999x0e", many.c_str()};
  for (const char* irreps : bad) {
    tpconv_norm_desc d{irreps, 1e-5f, 0, 0};
    tpconv_norm n = nullptr;
    CHECK(tpconv_norm_create(&n, &d) != TPCONV_SUCCESS && !n);
  }
  CHECK(tpconv_norm_create(nullptr, nullptr) != TPCONV_SUCCESS);
  CHECK(tpconv_norm_destroy(nullptr) == TPCONV_SUCCESS);
}

static void linears() {
  struct { const char *in, *out; } good[] = {{"1x0e", "1x0e"}, {"64x0e+32x1o", "16x1o+8x0e+4x0e"}, {"8x0e", "8x1o"},
                                             {"1000000x0e", "1x0e"}};
  for (auto& g : good)
    for (int groups : {1, 3, 64, 65, 4096}) {
      tpconv_linear_desc d{};
      d.irreps_in = g.in;
      d.irreps_out = g.out;
      d.num_groups = groups;
      tpconv_linear l = nullptr;
      CHECK(tpconv_linear_create(&l, &d) == TPCONV_SUCCESS && l);
      int64_t fi = 0, fo = 0, wn = 0;
      int32_t nb = 0, count = 0;
      CHECK(tpconv_linear_info(l, &fi, &fo, &wn, &nb) == TPCONV_SUCCESS && fi > 0 && fo > 0);
      int64_t sum = 0;
      for (int32_t i = 0; i < nb; ++i) {
        int32_t ir[2], shape[2];
        int64_t off = -1;
        CHECK(tpconv_linear_block(l, i, ir, shape, &off) == TPCONV_SUCCESS && off == sum);
        sum += (int64_t)shape[0] * shape[1];
      }
      CHECK(sum == wn);
      CHECK(tpconv_linear_block(l, nb, nullptr, nullptr, nullptr) != TPCONV_SUCCESS);
      CHECK(tpconv_linear_block(l, -1, nullptr, nullptr, nullptr) != TPCONV_SUCCESS);
      CHECK(tpconv_linear_weight_blocks(l, nullptr, 0, &count) == TPCONV_SUCCESS && count == nb);
      std::vector<tpconv_matrix_block> blocks(count);
      if (count > 0) {
        CHECK(tpconv_linear_weight_blocks(l, blocks.data(), count - 1, &count) != TPCONV_SUCCESS);
        CHECK(tpconv_linear_weight_blocks(l, blocks.data(), (int32_t)blocks.size(), &count) == TPCONV_SUCCESS);
      }
      size_t s = 0;
      for (int64_t N : {0ll, 1ll, 1000ll, 1000000ll}) {
        CHECK(tpconv_linear_groups_workspace_size(l, N, &s) == TPCONV_SUCCESS && s > 0);
        CHECK(tpconv_linear_workspace_size(l, TPCONV_OP_FORWARD, N, &s) == TPCONV_SUCCESS);
        CHECK(tpconv_linear_workspace_size(l, TPCONV_OP_BACKWARD, N, &s) == TPCONV_SUCCESS);
      }
      CHECK(tpconv_linear_workspace_size(l, 99, 4, &s) != TPCONV_SUCCESS);
      CHECK(tpconv_linear_groups(l, 4, (int32_t*)fake(64), (int32_t*)fake(64), (int32_t*)fake(64), 1, fake(68),
                                 size_t(1) << 40, nullptr) == TPCONV_ERROR_WORKSPACE);
      CHECK(tpconv_linear_forward(l, -1, nullptr, nullptr, fake(64), fake(64), fake(64), nullptr, 0, nullptr) !=
            TPCONV_SUCCESS);
      CHECK(tpconv_linear_destroy(l) == TPCONV_SUCCESS);
    }
  std::string in = "1x0e";
  for (int i = 1; i < 9; ++i) in += "+1x0e";
  for (const char* side : {"", "x", "3x5e", in.c_str()}) {
    tpconv_linear_desc d{};
    d.irreps_in = d.irreps_out = side;
    d.num_groups = 1;
    tpconv_linear l = nullptr;
    CHECK(tpconv_linear_create(&l, &d) != TPCONV_SUCCESS && !l);
  }
}

static void muons() {
  const float coef[] = {3.4445f, -4.775f, 2.0315f, 3.4445f, -4.775f, 2.0315f, 3.4445f, -4.775f, 2.0315f};
  const int32_t shapes[][2] = {{1, 1}, {32, 32}, {33, 32}, {32, 513}, {128, 129}, {1000, 40}, {1024, 2048}, {32768, 32768}};
  for (auto& sh : shapes)
    for (int64_t count : {0ll, 1ll, 7ll}) {
      std::vector<tpconv_matrix_block> b;
      for (int i = 0; i < 64; ++i) b.push_back({sh[0], sh[1], count, 0, (int64_t)sh[0] * sh[1] + i});
      tpconv_muon_desc d{64, b.data(), 3, coef, 1e-7f};
      tpconv_muon m = nullptr;
      CHECK(tpconv_muon_create(&m, &d) == TPCONV_SUCCESS && m);
      size_t s = 0;
      CHECK(tpconv_muon_workspace_size(m, &s) == TPCONV_SUCCESS);
      if (s > 0) {
        CHECK(tpconv_muon_orthogonalize(m, (float*)fake(64), (float*)fake(64), fake(72), s, nullptr) ==
              TPCONV_ERROR_WORKSPACE);
        CHECK(tpconv_muon_orthogonalize(m, (float*)fake(64), (float*)fake(64), fake(64), s - 1, nullptr) ==
              TPCONV_ERROR_WORKSPACE);
      }
      CHECK(tpconv_muon_step(m, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) !=
            TPCONV_SUCCESS);
      CHECK(tpconv_muon_destroy(m) == TPCONV_SUCCESS);
    }
  tpconv_matrix_block one{4, 4, 1, 0, 16};
  const float wild[][3] = {{NAN, 0.f, 0.f}, {INFINITY, 0.f, 0.f}, {3e38f, 3e38f, 3e38f}};
  for (auto& w : wild) {
    tpconv_muon_desc d{1, &one, 1, w, 1e-7f};
    tpconv_muon m = nullptr;
    CHECK(tpconv_muon_create(&m, &d) != TPCONV_SUCCESS && !m);
  }
  const tpconv_matrix_block wrong[] = {{0, 4, 1, 0, 16}, {4, 4, -1, 0, 16}, {4, 4, 1, -1, 16}, {4, 4, 1, 0, 15},
                                       {INT32_MAX, INT32_MAX, 1, 0, INT64_MAX}};
  for (const auto& w : wrong) {
    tpconv_muon_desc d{1, &w, 3, coef, 1e-7f};
    tpconv_muon m = nullptr;
    CHECK(tpconv_muon_create(&m, &d) == TPCONV_ERROR_INVALID_VALUE && !m);
  }
  CHECK(tpconv_muon_destroy(nullptr) == TPCONV_SUCCESS);
}

static void plans() {
  struct { const char *in, *out; } sides[] = {{"8x0e+8x1o", "8x0e+8x1o"}, {"8x0e+4x1o", "16x0e+2x1o"}};
  for (auto& g : sides) {
    tpconv_desc d{};
    d.irreps_in = g.in;
    d.irreps_out = g.out;
    d.sh_lmax = 1;
    d.num_basis = 8;
    d.cutoff = 5.f;
    d.envelope_p = 6;
    tpconv_plan p = nullptr;
    CHECK(tpconv_plan_create(&p, &d) == TPCONV_SUCCESS);
    int32_t count = 0;
    CHECK(tpconv_plan_weight_blocks(p, nullptr, 0, &count) == TPCONV_SUCCESS && count > 0);
    std::vector<tpconv_matrix_block> b(count);
    CHECK(tpconv_plan_weight_blocks(p, b.data(), count, &count) == TPCONV_SUCCESS);
    int64_t wn = 0, sum = 0;
    CHECK(tpconv_plan_info(p, nullptr, &wn, nullptr, nullptr, nullptr, nullptr) == TPCONV_SUCCESS);
    for (const auto& m : b) sum += m.count * m.rows * m.cols;
    CHECK(sum == wn);
    CHECK(tpconv_plan_destroy(p) == TPCONV_SUCCESS);
  }
}

int main() {
  norms();
  linears();
  muons();
  plans();
  if (failures) return 1;
  std::puts("host sanitizer checks passed");
  return 0;
}
