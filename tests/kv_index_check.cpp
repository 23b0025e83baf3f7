// Walks the addresses the cache kernels form, on the host: every row a tile, a
// slot or a bad page-table entry leads to lies inside the cache's arrays.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "kv_common.h"

using namespace awq;

static int fails = 0;
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); ++fails; } } while (0)

int main() {
  const int32_t lowest = -2147483647 - 1, highest = 2147483647;
  for (int ps : {4, 5, 6, 10})
    for (int heads : {1, 3, 8})
      for (int64_t pages : {int64_t(1), int64_t(2), int64_t(7), (int64_t(1) << (31 - ps)) - 1}) {
        const KvShape s{pages, heads, ps};
        const int64_t P = int64_t(1) << ps, rows = pages * heads * P;
        for (int32_t e : {lowest, -1, 0, (int32_t)(pages - 1), (int32_t)pages, highest}) {
          const int page = kv_page(s, e);
          CHECK(page == -1 || (page == e && page >= 0 && page < pages));
          CHECK((e >= 0 && e < pages) == (page >= 0));
          for (int64_t t : {int64_t(0), int64_t(16), P - 16, P, 5 * P + 16 * (P / 32)})
            for (int h : {0, heads - 1}) {
              const int64_t r = kv_tile_row(s, page, t, h);
              CHECK(r >= 0 && r % 16 == 0 && r + 15 < rows);
              if (page >= 0)
                for (int i = 0; i < 16; ++i) CHECK(kv_row(s, page * P + (t + i) % P, h) == r + i);
            }
        }
        for (int64_t slot : {int64_t(lowest), int64_t(-1), int64_t(0), P - 1, P, pages * P - 1, pages * P, int64_t(highest)}) {
          CHECK(kv_slot_ok(s, slot) == (slot >= 0 && slot < pages * P));
          if (kv_slot_ok(s, slot))
            for (int h : {0, heads - 1}) {
              const int64_t r = kv_row(s, slot, h);
              CHECK(r >= 0 && r < rows);
              CHECK(r == ((slot / P) * heads + h) * P + slot % P);
            }
        }
        for (int32_t n : {lowest, -1, 0, 1, 17, highest})
          for (int64_t width : {int64_t(1), int64_t(3)})
            for (int64_t most : {int64_t(1), int64_t(40), int64_t(1) << 25}) {
              const int64_t len = kv_length(s, n, width, most);
              CHECK(len >= 0 && len <= width * P && len <= most && (n < 0 ? len == 0 : len <= n));
              CHECK(len == 0 || (len - 1) / 16 * 16 / P < width);
            }
      }
  std::printf(fails ? "FAILED\n" : "ok\n");
  return fails != 0;
}
