// Host check of a chunk's query rows (attend.h): which are computed, and at which positions, against
// their definition row by row; offsets of any value stay inside the tokens.  Prints "ok" or the first
// difference.
#include <limits.h>
#include <stdio.h>

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

static int check_small() {
  for (int tokens = 1; tokens < 9; ++tokens)
    for (int q0 = -4; q0 < 12; ++q0)
      for (int q1 = -4; q1 < 14; ++q1)
        for (int most = 1; most < 12; ++most)
          for (int len = 0; len < 12; len += 3) {
            const ChunkRows c = chunk_rows(q0, q1, len, most, tokens);
            int n = 0;
            for (int row = q0; row < q1; ++row) {
              if (row < 0 || row >= tokens || row >= q0 + most) continue;
              CHECK(row == c.first + n, "rows %d .. %d: row %d", q0, q1, row);
              CHECK(c.p0 + n == len - (q1 - row), "rows %d .. %d: position of row %d", q0, q1, row);
              ++n;
            }
            CHECK(n == c.count, "rows %d .. %d of %d, at most %d: %d", q0, q1, tokens, most, c.count);
            // the list of the unit's keys ends with its last token
            const KeyList l = window_keys(nullptr, 0, c.p0 + c.count < 0 ? 0 : c.p0 + c.count, c.p0, 5, 2);
            for (int vp = 0; vp < l.n; ++vp)
              CHECK(key_position(l, vp) >= 0 && key_position(l, vp) < c.p0 + c.count, "a key past the end");
          }
  return 0;
}

static int check_any_offsets() {
  const int at[] = {INT_MIN, INT_MIN + 1, -(1 << 30), -7, -1, 0, 1, 5, 100, 1 << 30, INT_MAX - 1, INT_MAX};
  for (int q0 : at)
    for (int q1 : at)
      for (int len : {0, 1, 50, 1 << 30})
        for (int most : {1, 64, INT_MAX})
          for (int tokens : {1, 100, 1 << 30}) {
            const ChunkRows c = chunk_rows(q0, q1, len, most, tokens);
            CHECK(c.count >= 0 && c.count <= most, "count");
            CHECK(c.count == 0 || (c.first >= 0 && c.count <= tokens - c.first), "rows outside");
            CHECK(c.p0 >= -(1 << 30) && c.p0 <= len, "position %d", c.p0);
            CHECK((int64_t)c.p0 + c.count <= len, "a token past the last key");
          }
  return 0;
}

int main() {
  if (check_small() || check_any_offsets()) return 1;
  printf("ok\n");
  return 0;
}
