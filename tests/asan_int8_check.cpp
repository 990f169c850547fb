// Host-side driver for the AddressSanitizer pass over the argument checks of the
// int8 and expert calls (built and run by test_host_asan_int8.py; no GPU needed).
// Every call below is answered on the host before anything is launched.  Exits 0
// when every status is the expected one.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "qgemm.h"

namespace {

int failures = 0;

void expect(const char* what, long long got, long long want) {
  if (got != want) {
    std::printf("FAIL %s: got %lld, want %lld\n", what, got, want);
    ++failures;
  }
}

// addresses that are never read
template <class T>
T* at(uintptr_t v) {
  return reinterpret_cast<T*>(v);
}

constexpr int64_t kBig = (int64_t)1 << 31, kHuge = INT64_MAX;

struct Quantize {
  int type = QGEMM_F16;
  void* x = at<void>(0x100000);
  int8_t* codes = at<int8_t>(0x200000);
  float* scale = at<float>(0x300000);
  int64_t rows = 4, K = 64, stride = 64;
  int call() const { return qgemm_quantize_int8(type, x, codes, scale, rows, K, stride, nullptr); }
};

struct Prepack {
  int8_t* w = at<int8_t>(0x100000);
  void* packed = at<void>(0x400000);
  int64_t experts = 3, K = 64, N = 32;
  int gated = 0;
  int call() const { return qgemm_prepack_w8a8(w, packed, experts, K, N, gated, nullptr); }
};

struct Product {
  int type = QGEMM_BF16;
  int8_t* a = at<int8_t>(0x100000);
  float *a_scale = at<float>(0x200000), *w_scale = at<float>(0x300000);
  void *packed = at<void>(0x400000), *out = at<void>(0x500000);
  int32_t *offsets = at<int32_t>(0x600000), *rows = at<int32_t>(0x700000);
  int64_t a_rows = 4, M = 9, N = 32, K = 64, experts = 3;
  int gated = 1;
  int call() const {
    return qgemm_w8a8_experts(type, a, a_scale, packed, w_scale, offsets, rows, out, a_rows, M, N, K, experts,
                              gated, nullptr);
  }
};

struct Plan {
  int bytes = 8;
  void* ids = at<void>(0x100000);
  int32_t *offsets = at<int32_t>(0x200000), *rows = at<int32_t>(0x300000), *places = at<int32_t>(0x400000);
  void* workspace = at<void>(0x500000);
  int64_t tokens = 5, top = 2, experts = 6;
  int call() const {
    return qgemm_expert_plan(bytes, ids, offsets, rows, places, workspace, tokens, top, experts, nullptr);
  }
};

struct Combine {
  int type = QGEMM_F16;
  void *y = at<void>(0x100000), *out = at<void>(0x400000);
  int32_t* places = at<int32_t>(0x200000);
  float* gates = at<float>(0x300000);
  int64_t rows = 9, tokens = 5, top = 2, N = 24;
  int call() const { return qgemm_expert_combine(type, y, places, gates, out, rows, tokens, top, N, nullptr); }
};

template <class Call, class Change>
void refused(const char* what, int want, Change change) {
  Call c;
  change(c);
  expect(what, c.call(), want);
}

// Each size in turn at the ends of its type: refused, without overflow.
template <class Call>
void sizes(const char* what, int64_t Call::*field) {
  for (int64_t v : {(int64_t)-1, INT64_MIN, kHuge, kHuge - 15, kBig, kBig * kBig / 2}) {
    Call c;
    c.*field = v;
    expect(what, c.call(), QGEMM_ERR_SHAPE);
  }
}

}  // namespace

int main() {
  sizes<Quantize>("quantize rows", &Quantize::rows);
  sizes<Quantize>("quantize K", &Quantize::K);
  for (int64_t v : {(int64_t)-1, INT64_MIN, kHuge, (int64_t)1 << 40}) {   // 2^31 is a stride like others
    Quantize q;
    q.stride = v;
    expect("quantize stride", q.call(), QGEMM_ERR_SHAPE);
  }
  sizes<Prepack>("prepack experts", &Prepack::experts);
  sizes<Prepack>("prepack K", &Prepack::K);
  sizes<Prepack>("prepack N", &Prepack::N);
  sizes<Product>("product a_rows", &Product::a_rows);
  sizes<Product>("product M", &Product::M);
  sizes<Product>("product N", &Product::N);
  sizes<Product>("product K", &Product::K);
  sizes<Product>("product experts", &Product::experts);
  sizes<Plan>("plan tokens", &Plan::tokens);
  sizes<Plan>("plan top", &Plan::top);
  sizes<Plan>("plan experts", &Plan::experts);
  sizes<Combine>("combine rows", &Combine::rows);
  sizes<Combine>("combine tokens", &Combine::tokens);
  sizes<Combine>("combine top", &Combine::top);
  sizes<Combine>("combine N", &Combine::N);
  refused<Quantize>("quantize rows and stride", QGEMM_ERR_SHAPE, [](Quantize& q) {
    q.rows = kBig - 1;
    q.stride = ((int64_t)1 << 40) - 8;
  });
  refused<Quantize>("quantize overlap", QGEMM_ERR_OVERLAP, [](Quantize& q) { q.codes = at<int8_t>(0x1000f0); });
  refused<Quantize>("quantize at the end of memory", QGEMM_ERR_OVERLAP, [](Quantize& q) {
    q.x = at<void>(UINTPTR_MAX - 15);   // wraps round
    q.codes = at<int8_t>(0x10);
  });
  refused<Product>("product overlap", QGEMM_ERR_OVERLAP, [](Product& p) { p.out = p.rows; });
  refused<Plan>("plan overlap", QGEMM_ERR_OVERLAP, [](Plan& p) { p.rows = p.places; });
  refused<Combine>("combine overlap", QGEMM_ERR_OVERLAP, [](Combine& c) { c.out = c.y; });
  refused<Plan>("plan pairs", QGEMM_ERR_SHAPE, [](Plan& p) { p.tokens = p.top = kBig - 1; });
  expect("plan workspace", qgemm_expert_plan_workspace_bytes(kHuge, 4), QGEMM_ERR_SHAPE);
  expect("prepack bytes", qgemm_prepack_w8a8_bytes(1024, 131056, 16000, 0),
         (int64_t)1024 * 131072 * 16000);
  int64_t r, c, k;
  for (int64_t v : {(int64_t)-1, INT64_MIN, kHuge, kBig})
    for (int i = 0; i < 4; ++i)
      expect("tile", qgemm_w8a8_tile(i == 0 ? v : 4, i == 1 ? v : 32, i == 2 ? v : 64, i == 3 ? v : 2, 0, &r, &c, &k),
             QGEMM_ERR_SHAPE);
  expect("tile of nothing", qgemm_w8a8_tile(0, 0, 0, 0, 0, &r, &c, &k), QGEMM_OK);
  std::printf("%s (%d failures)\n", failures ? "FAILED" : "ok", failures);
  return failures ? 1 : 0;
}
