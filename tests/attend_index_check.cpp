// Host check of the paged attention's index arithmetic (attend.h): quotients by the page size,
// key lists against their definition, table and page accesses of bad tables against the buffers'
// bounds, and the split of steps over workgroups.  Prints "ok" or the first difference.
#include <stdio.h>
#include <stdlib.h>

#include <set>
#include <vector>

#include "../tenant_serving_bitdelta_amd/csrc/attend.h"

using namespace bd;

#define CHECK(c, ...)                 \
  do {                                \
    if (!(c)) {                       \
      printf("line %d: ", __LINE__);  \
      printf(__VA_ARGS__);            \
      printf("\n");                   \
      return 1;                       \
    }                                 \
  } while (0)

static uint64_t rng_state = 12345;
static uint32_t rnd() {
  rng_state = rng_state * 6364136223846793005ull + 1442695040888963407ull;
  return (uint32_t)(rng_state >> 33);
}

static int check_div() {
  std::vector<uint32_t> ds;
  for (uint32_t d = 1; d <= 300; ++d) ds.push_back(d);
  for (int i = 0; i < 200; ++i) ds.push_back(1 + rnd() % 0x7fffffffu);
  ds.push_back(0x7fffffffu);
  ds.push_back(1u << 30);
  for (uint32_t d : ds) {
    const PageDiv p = make_page_div(d);
    auto one = [&](uint32_t n) { return page_quotient((int)n, p) == (int)(n / d); };
    for (uint32_t n = 0; n < 2000; ++n) CHECK(one(n), "%u / %u", n, d);
    for (int i = 0; i < 2000; ++i) {
      const uint32_t n = rnd() & 0x7fffffffu;
      CHECK(one(n), "%u / %u", n, d);
      const uint32_t e = n / d * d;
      CHECK(one(e) && (e == 0 || one(e - 1)), "around %u / %u", e, d);
    }
    CHECK(one(0x7fffffffu), "2^31 - 1 / %u", d);
  }
  return 0;
}

static int check_window() {
  for (int it = 0; it < 4000; ++it) {
    const int len = rnd() % 60, nq = 1 + rnd() % 9, window = 1 + rnd() % 70, sinks = rnd() % 12;
    const int p0 = len - nq;
    const KeyList l = window_keys(nullptr, 0, len, p0, window, sinks);
    CHECK(l.n >= 0 && l.na >= 0 && l.na <= l.n, "list sizes");
    std::set<int> got;
    for (int vp = 0; vp < l.n; ++vp) {
      const int kp = key_position(l, vp);
      CHECK(kp >= 0 && kp < len, "key %d of %d", kp, len);
      CHECK(got.insert(kp).second, "key %d twice", kp);
    }
    for (int p = p0; p < len; ++p)
      for (int j = 0; j <= p; ++j)
        if (p - j < window || j < sinks)
          CHECK(got.count(j), "key %d of token %d missing (len %d window %d sinks %d)", j, p, len,
                window, sinks);
  }
  return 0;
}

static int check_bad_tables() {
  // every access a lookup makes stays inside the table row and the cache
  for (int it = 0; it < 3000; ++it) {
    const int page = 1 + rnd() % 40, width = rnd() % 7, pwidth = rnd() % 5, pages = 1 + rnd() % 9;
    std::vector<int> t(width), pt(pwidth);
    const int bad[] = {-1, -2147483647 - 1, 2147483647, pages, pages + 1};
    for (int& x : t) x = rnd() % 3 ? (int)(rnd() % pages) : bad[rnd() % 5];
    for (int& x : pt) x = rnd() % 3 ? (int)(rnd() % pages) : bad[rnd() % 5];
    const int len = rnd() % (width * page + 1), plen = rnd() % (pwidth * page + 1);
    KeyList l{pt.data(), t.data(), pwidth, width, plen, 0, plen + len};
    if (rnd() % 2) {
      l = window_keys(t.data(), width, len, len - 1 - (int)(rnd() % 5), 1 + rnd() % 50, rnd() % 9);
    }
    const PageDiv d = make_page_div(page);
    for (int vp = 0; vp < l.n + 400; ++vp) {
      const int kp = key_position(l, vp);
      const int q = page_quotient(kp < 0 ? 0 : kp, d);
      const int at = key_table_index(l, vp, q);
      if (vp >= l.n) CHECK(at < 0, "past the end");
      if (at < 0) continue;
      const bool first = vp < l.na;
      CHECK(at < (first ? l.wa : l.wb), "table entry %d", at);
      const int raw = (first ? l.ta : l.tb)[at];
      const int id = page_id_checked(raw, pages);
      CHECK((id >= 0) == (raw >= 0 && raw < pages), "page %d", raw);
      const int slot = kp - q * page;
      CHECK(slot >= 0 && slot < page, "slot %d", slot);
    }
  }
  // offsets past 32 bits
  CHECK(page_row_bytes(70000, 15, 65536, 16) == 70000ll * 65536 * 16 + 15 * 256, "64-bit offset");
  CHECK(page_row_bytes(3, 5, 0xFFFFFFFFu, 1) == 3ll * 0xFFFFFFFFll * 16 + 80, "widest stride");
  return 0;
}

static int check_split() {
  for (int it = 0; it < 3000; ++it) {
    const int64_t total = 1 + (it % 5 == 0 ? (int64_t)rnd() * 7 : rnd() % 5000);
    const int workers = split_workers(total, 1 + rnd() % 900);
    for (int w = 0; w < workers; ++w)
      CHECK(split_begin(w, total, workers) < split_begin(w + 1, total, workers), "an idle worker");
    CHECK(split_begin(0, total, workers) == 0 && split_begin(workers, total, workers) == total, "ends");
    for (int i = 0; i < 200; ++i) {
      const int64_t x = (int64_t)(((uint64_t)rnd() << 20 ^ rnd()) % (uint64_t)total);
      const int w = split_owner(x, total, workers);
      CHECK(w >= 0 && w < workers && split_begin(w, total, workers) <= x &&
                x < split_begin(w + 1, total, workers),
            "owner of %lld of %lld", (long long)x, (long long)total);
    }
  }
  return 0;
}

int main() {
  if (check_div() || check_window() || check_bad_tables() || check_split()) return 1;
  printf("ok\n");
  return 0;
}
