// Host-side exercise of the C ABI of include/tpconv_attention.h for an
// AddressSanitizer / UBSan build of its argument checks, layouts and workspace
// sizes.  It touches no device memory: every call below must be answered or
// rejected on the host before any launch.  Exit status 0 when every check holds.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "tpconv_attention.h"

static int failures = 0;
#define CHECK(cond)                                                    \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "check failed (line %d): %s\n", __LINE__, #cond); \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

template <typename T = float>
static T* fake(uintptr_t a = 64) {
  return reinterpret_cast<T*>(a);
}
static const size_t kBig = size_t(1) << 60;

static void attentions() {
  std::string sixteen = "4x0e", many = "4x0e";
  for (int i = 1; i < 16; ++i) sixteen += "+4x1o";
  for (int i = 1; i < 17; ++i) many += "+4x1o";
  const char* good[] = {"4x0e", "256x0e", "8x0e+4x1o", "16x0e+16x1o+16x2e+16x3o", sixteen.c_str()};
  for (const char* qk : good)
    for (const char* v : good)
      for (int heads : {1, 2, 4})
        for (int t = 0; t < 4; ++t) {
          tpconv_attention_desc d{qk, v, heads, 0.5f, t == 3 ? 30.f : 0.f, t & 1, t >> 1};
          tpconv_attention a = nullptr;
          CHECK(tpconv_attention_create(&a, &d) == TPCONV_SUCCESS && a);
          int64_t fq = 0, fv = 0, saved = 0;
          int32_t dq = 0, dv = 0;
          CHECK(tpconv_attention_info(a, &fq, &fv, &dq, &dv) == TPCONV_SUCCESS && fq == (int64_t)dq * heads &&
                fv == (int64_t)dv * heads);
          CHECK(tpconv_attention_info(a, nullptr, nullptr, nullptr, nullptr) == TPCONV_SUCCESS);
          CHECK(tpconv_attention_saved_size(a, 1000, &saved) == TPCONV_SUCCESS &&
                saved == 2000 * heads + (t >> 1 ? 1000 * fv : 0));
          CHECK(tpconv_attention_saved_size(a, -1, &saved) != TPCONV_SUCCESS);
          for (int64_t n : {0ll, 1ll, 31ll, 4096ll, 100000ll})
            for (int64_t g : {0ll, 1ll, 77ll, 4096ll})
              for (int form = 0; form < 3; ++form)
                for (int op : {(int)TPCONV_OP_FORWARD, (int)TPCONV_OP_BACKWARD}) {
                  tpconv_attention_batch b{g, n, fake<int32_t>(), form == 1 ? nullptr : fake(), 0, nullptr, nullptr};
                  if (form == 2) {
                    b.num_keys = 3 * n;
                    b.key_offsets = fake<int32_t>();
                    b.key_pos = fake();
                  }
                  size_t bytes = 1;
                  CHECK(tpconv_attention_workspace_size(a, op, &b, &bytes) == TPCONV_SUCCESS && bytes % 16 == 0);
                }
          tpconv_attention_batch b{1, 3, nullptr, fake(), 0, nullptr, nullptr};
          tpconv_attention_inputs in{fake<void>(), fake<void>(), fake<void>(), 0, 0, 0, fake()};
          tpconv_attention_grads g{};
          CHECK(tpconv_attention_forward(a, &b, &in, nullptr, nullptr, nullptr, 0, nullptr) != TPCONV_SUCCESS);
          CHECK(tpconv_attention_backward(a, &b, &in, fake(), fake(), fake(), &g, fake<void>(), kBig, nullptr) !=
                TPCONV_SUCCESS);
          g.grad_q = fake();
          CHECK(tpconv_attention_backward(a, &b, &in, fake(), fake(), fake(), &g, fake<void>(72), kBig, nullptr) ==
                TPCONV_ERROR_WORKSPACE);
          g.q_stride = fq - 1;
          CHECK(tpconv_attention_backward(a, &b, &in, fake(), fake(), fake(), &g, fake<void>(), kBig, nullptr) !=
                TPCONV_SUCCESS);
          b.num_graphs = 0;  // without offsets
          CHECK(tpconv_attention_forward(a, &b, &in, fake<void>(), nullptr, fake<void>(), kBig, nullptr) != TPCONV_SUCCESS);
          b.offsets = fake<int32_t>();  // no graphs: nothing to do
          CHECK(tpconv_attention_forward(a, &b, &in, fake<void>(), nullptr, nullptr, 0, nullptr) == TPCONV_SUCCESS);
          b.num_graphs = b.num_queries = 2147483646ll;
          size_t bytes = 0;
          CHECK(tpconv_attention_workspace_size(a, TPCONV_OP_BACKWARD, &b, &bytes) == TPCONV_ERROR_UNSUPPORTED);
          CHECK(tpconv_attention_destroy(a) == TPCONV_SUCCESS);
        }
  const char* bad[] = {nullptr, "", "x0e", "8x4e", "8x0e+", "-3x0e", "6x0e", "99999999999999999999x0e",
                       "2147483644x0e", "1028x0e", many.c_str()};
  for (const char* irreps : bad)
    for (int side = 0; side < 2; ++side) {
      tpconv_attention_desc d{side ? irreps : "8x0e", side ? "8x0e" : irreps, 4, 1.f, 0.f, 0, 0};
      tpconv_attention a = nullptr;
      CHECK(tpconv_attention_create(&a, &d) != TPCONV_SUCCESS && !a);
    }
  CHECK(tpconv_attention_create(nullptr, nullptr) != TPCONV_SUCCESS);
  CHECK(tpconv_attention_destroy(nullptr) == TPCONV_SUCCESS);
  CHECK(tpconv_attention_info(nullptr, nullptr, nullptr, nullptr, nullptr) != TPCONV_SUCCESS);
}

static void embeds() {
  for (int32_t rows : {1, 255, 256, 70000, 1 << 24})
    for (int32_t f : {1, 3, 64, 65, 128, 1000, 65536}) {
      tpconv_embed_desc d{rows, f, 2.f, 0, 1};
      tpconv_embed e = nullptr;
      CHECK(tpconv_embed_create(&e, &d) == TPCONV_SUCCESS && e);
      size_t last = 0;
      for (int64_t n : {0ll, 1ll, 128ll, 129ll, 4096ll, 4097ll, 65536ll, 65537ll, 2147483646ll}) {
        size_t s = 0;
        CHECK(tpconv_embed_workspace_size(e, n, &s) == TPCONV_SUCCESS && (n <= 128) == (s == 0));
        CHECK(s == 0 || s >= (size_t)n * 8);
        last = s;
      }
      CHECK(tpconv_embed_workspace_size(e, -1, &last) != TPCONV_SUCCESS);
      CHECK(tpconv_embed_forward(e, 5, nullptr, fake(), fake(), nullptr) != TPCONV_SUCCESS);
      CHECK(tpconv_embed_backward(e, 200, fake<int32_t>(), fake(), fake(), fake<void>(), 10, nullptr) ==
            TPCONV_ERROR_WORKSPACE);
      CHECK(tpconv_embed_destroy(e) == TPCONV_SUCCESS);
    }
  for (tpconv_embed_desc d : {tpconv_embed_desc{0, 4, 1.f, 0, 0}, {4, 0, 1.f, 0, 0}, {4, 4, NAN, 0, 0}, {4, 4, 1.f, 2, 0}}) {
    tpconv_embed e = nullptr;
    CHECK(tpconv_embed_create(&e, &d) != TPCONV_SUCCESS && !e);
  }
  CHECK(tpconv_embed_destroy(nullptr) == TPCONV_SUCCESS);
}

static void dropouts() {
  for (const char* irreps : {"1x0e", "9x0e+5x1o+8x2e+7x3o", "4096x0e"})
    for (float p : {0.f, 0.1f, 0.999999f, 1.f}) {
      tpconv_dropout_desc d{irreps, p, 1, 0};
      tpconv_dropout h = nullptr;
      CHECK(tpconv_dropout_create(&h, &d) == TPCONV_SUCCESS && h);
      int64_t F = 0;
      float used = -1.f;
      CHECK(tpconv_dropout_info(h, &F, &used) == TPCONV_SUCCESS && F > 0 && std::fabs(used - p) <= 1.f / 131072);
      CHECK(tpconv_dropout_info(h, nullptr, nullptr) == TPCONV_SUCCESS);
      CHECK(tpconv_dropout_forward(h, 3, fake<void>(), fake<int64_t>(), nullptr, fake<void>(), nullptr) != TPCONV_SUCCESS);
      CHECK(tpconv_dropout_backward(h, 3, fake(), nullptr, fake(), nullptr) != TPCONV_SUCCESS);
      CHECK(tpconv_dropout_destroy(h) == TPCONV_SUCCESS);
    }
  for (float p : {-0.1f, 1.5f, NAN, INFINITY}) {
    tpconv_dropout_desc d{"8x0e", p, 0, 0};
    tpconv_dropout h = nullptr;
    CHECK(tpconv_dropout_create(&h, &d) != TPCONV_SUCCESS && !h);
  }
  CHECK(tpconv_dropout_destroy(nullptr) == TPCONV_SUCCESS);
}

int main() {
  attentions();
  embeds();
  dropouts();
  if (failures) return 1;
  std::puts("host sanitizer checks passed");
  return 0;
}
