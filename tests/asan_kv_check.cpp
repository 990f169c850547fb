// Host-side driver for the AddressSanitizer pass over the key-value cache
// calls' argument checks (built and run by test_host_asan_kv.py; no GPU needed).
// Every call below is answered on the host before anything is launched.  Exits
// 0 when every status is the expected one.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

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

struct Plan {
  int32_t* table = at<int32_t>(0x100000);
  const int32_t *cached = at<int32_t>(0x200000), *added = at<int32_t>(0x210000),
                *free_pages = at<int32_t>(0x220000);
  int32_t *lens = at<int32_t>(0x300000), *cu_tokens = at<int32_t>(0x310000),
          *cu_pages = at<int32_t>(0x320000);
  int64_t* slots = at<int64_t>(0x330000);
  int64_t batch = 4, width = 8, stride = 8, num_free = 9, page_size = 16, tokens = 4;
  int call() const {
    return qgemm_kv_plan(table, cached, added, free_pages, lens, cu_tokens, cu_pages, slots, batch, width,
                         stride, num_free, page_size, tokens, nullptr);
  }
};

struct Append {
  int type = QGEMM_F16, cache_type = QGEMM_F16;
  void *k = at<void>(0x100000), *v = at<void>(0x110000);
  int64_t* slots = at<int64_t>(0x120000);
  void *k_cache = at<void>(0x200000), *v_cache = at<void>(0x300000);
  float *k_scale = nullptr, *v_scale = nullptr;
  int64_t tokens = 4, heads = 2, dim = 64, kt = 128, kh = 64, vt = 128, vh = 64, pages = 5, page_size = 16,
          page = 2048, head = 1024, token = 64;
  int call() const {
    return qgemm_kv_append(type, cache_type, k, v, slots, k_cache, v_cache, k_scale, v_scale, tokens, heads,
                           dim, kt, kh, vt, vh, pages, page_size, page, head, token, nullptr);
  }
};

struct Attend {
  int type = QGEMM_BF16, cache_type = QGEMM_BF16;
  void *q = at<void>(0x100000), *k_cache = at<void>(0x200000), *v_cache = at<void>(0x300000);
  int32_t *table = at<int32_t>(0x400000), *lens = at<int32_t>(0x410000);
  float *k_scale = nullptr, *v_scale = nullptr;
  void *out = at<void>(0x420000), *workspace = at<void>(0x500000);
  int64_t batch = 3, heads = 8, kv_heads = 2, dim = 64, qb = 512, qh = 64, pages = 5, page_size = 16,
          page = 2048, head = 1024, token = 64, width = 8, stride = 8, max_len = 128, window = 0;
  int call() const {
    return qgemm_paged_attention(type, cache_type, q, k_cache, v_cache, table, lens, k_scale, v_scale, out,
                                 workspace, batch, heads, kv_heads, dim, qb, qh, pages, page_size, page, head,
                                 token, width, stride, max_len, window, 0.125f, nullptr);
  }
};

template <class Call, class Change>
void refused(const char* what, int want, Change change) {
  Call c;
  change(c);
  expect(what, c.call(), want);
}

}  // namespace

int main() {
  setenv("QGEMM_ARCH_OVERRIDE", "gfx950", 1);

  refused<Plan>("plan batch", QGEMM_ERR_SHAPE, [](Plan& p) { p.batch = -1; });
  refused<Plan>("plan batch limit", QGEMM_ERR_SHAPE, [](Plan& p) { p.batch = kBig; });
  refused<Plan>("plan width", QGEMM_ERR_SHAPE, [](Plan& p) { p.width = kHuge; });
  refused<Plan>("plan stride", QGEMM_ERR_SHAPE, [](Plan& p) { p.stride = 7; });
  refused<Plan>("plan stride limit", QGEMM_ERR_SHAPE, [](Plan& p) { p.stride = kHuge; });
  refused<Plan>("plan table of 2^70", QGEMM_ERR_SHAPE, [](Plan& p) {
    p.batch = kBig - 1;
    p.stride = ((int64_t)1 << 40) - 1;
  });
  refused<Plan>("plan free", QGEMM_ERR_SHAPE, [](Plan& p) { p.num_free = -1; });
  refused<Plan>("plan page size", QGEMM_ERR_SHAPE, [](Plan& p) { p.page_size = 0; });
  refused<Plan>("plan tokens", QGEMM_ERR_SHAPE, [](Plan& p) { p.tokens = kHuge; });
  refused<Plan>("plan null", QGEMM_ERR_NULL, [](Plan& p) { p.cu_pages = nullptr; });
  refused<Plan>("plan slots null", QGEMM_ERR_NULL, [](Plan& p) { p.slots = nullptr; });
  refused<Plan>("plan align", QGEMM_ERR_ALIGN, [](Plan& p) { p.slots = at<int64_t>(0x330004); });
  refused<Plan>("plan overlap", QGEMM_ERR_OVERLAP, [](Plan& p) { p.lens = p.table + 31; });
  refused<Plan>("plan overlap of the largest", QGEMM_ERR_OVERLAP, [](Plan& p) {
    p.batch = kBig - 1;
    p.stride = (int64_t)1 << 29;
  });
  refused<Plan>("plan overlap at the end of memory", QGEMM_ERR_OVERLAP, [](Plan& p) {
    p.cu_tokens = at<int32_t>(UINTPTR_MAX - 19);
    p.cu_pages = p.cu_tokens;
  });

  refused<Append>("append type", QGEMM_ERR_FORMAT, [](Append& a) { a.type = 7; });
  refused<Append>("append pool type", QGEMM_ERR_FORMAT, [](Append& a) { a.cache_type = QGEMM_BF16; });
  refused<Append>("append scales", QGEMM_ERR_NULL, [](Append& a) { a.cache_type = QGEMM_E4M3; });
  refused<Append>("append dim", QGEMM_ERR_SHAPE, [](Append& a) { a.dim = kHuge; });
  refused<Append>("append heads", QGEMM_ERR_SHAPE, [](Append& a) { a.heads = kHuge; });
  refused<Append>("append pages", QGEMM_ERR_SHAPE, [](Append& a) { a.pages = kBig - 1; });
  refused<Append>("append page size", QGEMM_ERR_SHAPE, [](Append& a) { a.page_size = kBig - 1; });
  refused<Append>("append page stride", QGEMM_ERR_SHAPE, [](Append& a) { a.page = kHuge; });
  refused<Append>("append head stride", QGEMM_ERR_SHAPE, [](Append& a) { a.head = kBig * 64 - 64; a.heads = 3; });
  refused<Append>("append token stride", QGEMM_ERR_SHAPE, [](Append& a) { a.token = 65; });
  refused<Append>("append tokens", QGEMM_ERR_SHAPE, [](Append& a) { a.tokens = kBig - 1; });
  refused<Append>("append view", QGEMM_ERR_SHAPE, [](Append& a) { a.kt = (int64_t)1 << 40; });
  refused<Append>("append align", QGEMM_ERR_ALIGN, [](Append& a) { a.v = at<void>(0x110008); });
  refused<Append>("append nothing", QGEMM_OK, [](Append& a) { a.tokens = 0; });
  refused<Append>("append no pool", QGEMM_OK, [](Append& a) { a.pages = 0; });

  refused<Attend>("attention heads", QGEMM_ERR_SHAPE, [](Attend& a) { a.heads = 9; });
  refused<Attend>("attention kv heads", QGEMM_ERR_SHAPE, [](Attend& a) { a.kv_heads = 0; });
  refused<Attend>("attention batch", QGEMM_ERR_SHAPE, [](Attend& a) { a.batch = kBig - 1; a.heads = kBig - 2; });
  refused<Attend>("attention length", QGEMM_ERR_SHAPE, [](Attend& a) { a.max_len = kHuge; });
  refused<Attend>("attention tiles", QGEMM_ERR_SHAPE, [](Attend& a) { a.batch = 1 << 19; a.max_len = kBig / 2 - 1; });
  refused<Attend>("attention window", QGEMM_ERR_SHAPE, [](Attend& a) { a.window = -1; });
  refused<Attend>("attention width", QGEMM_ERR_SHAPE, [](Attend& a) { a.width = kHuge; });
  refused<Attend>("attention stride", QGEMM_ERR_SHAPE, [](Attend& a) { a.stride = 7; });
  refused<Attend>("attention q", QGEMM_ERR_SHAPE, [](Attend& a) { a.qh = -8; });
  refused<Attend>("attention pool", QGEMM_ERR_SHAPE, [](Attend& a) { a.page = kBig * 64 - 64; });
  refused<Attend>("attention workspace", QGEMM_ERR_NULL, [](Attend& a) { a.max_len = 100000; a.workspace = nullptr; });
  refused<Attend>("attention lens", QGEMM_ERR_ALIGN, [](Attend& a) { a.lens = at<int32_t>(0x410002); });
  refused<Attend>("attention nothing", QGEMM_OK, [](Attend& a) { a.batch = 0; });

  expect("workspace", qgemm_paged_attention_workspace_bytes(3, 8, 2, 64, 128, 0), 0);
  expect("workspace shared", qgemm_paged_attention_workspace_bytes(1, 1, 1, 256, kBig / 2 - 1, 0) > 0, 1);
  expect("workspace window", qgemm_paged_attention_workspace_bytes(1, 1, 1, 256, kBig / 2 - 1, 16), 0);
  expect("workspace none", qgemm_paged_attention_workspace_bytes(0, 8, 2, 64, 128, 0), 0);
  expect("workspace batch", qgemm_paged_attention_workspace_bytes(kBig - 1, kBig - 1, 1, 64, 128, 0),
         QGEMM_ERR_SHAPE);
  expect("workspace dim", qgemm_paged_attention_workspace_bytes(3, 8, 2, 40, 128, 0), QGEMM_ERR_SHAPE);

  std::printf("%s (%d failures)\n", failures ? "FAILED" : "ok", failures);
  return failures != 0;
}
