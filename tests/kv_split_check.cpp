// Cuts batches into attention's pieces on the host, as the kernels do: the pieces are every
// token once, all their numbers lie inside the workspace, and only an empty sequence has
// an empty piece.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "kv_common.h"

using namespace awq;

static int fails = 0;
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); ++fails; } } while (0)

static void walk(const std::vector<int>& len, int bound, int heads, int most) {
  const int B = (int)len.size();
  int64_t units = 0;
  for (int n : len) units += kv_units(n);
  const int shift = kv_piece_shift(units, heads, most);
  CHECK(shift >= 0 && shift < 19);
  int64_t number = 0;
  for (int n : len) {
    const int u = kv_units(n), pieces = kv_pieces(u, shift), span = (u + pieces - 1) / pieces * kKvUnit;
    int next = 0;
    for (int c = 0; c < pieces; ++c, ++number) {
      const int t0 = c * span, count = n - t0 < span ? n - t0 : span;
      CHECK(t0 == next && (count > 0 || n <= 0));
      next = t0 + (count > 0 ? count : 0);
    }
    CHECK(next == (n > 0 ? n : 0));
  }
  CHECK(number <= kv_most_pieces(B, bound, heads, most));
}

int main() {
  std::srand(1);
  for (int heads : {1, 8, 33, 600, 2000})
    for (int most : {256, 1024, 1536})
      for (int bound : {513, 2000, 100000, 1 << 25})
        for (int turn = 0; turn < 30; ++turn) {
          std::vector<int> len(1 + std::rand() % (turn < 3 ? 256 : 40));
          const int top = turn % 3 == 0 ? bound : (turn % 3 == 1 ? 1 + bound / 64 : 300);
          for (int& n : len) n = std::rand() % 5 ? (int)((std::rand() % 1000003 * 1LL * top) / 1000003) : 0;
          if (turn % 7 == 0) len[0] = bound;
          if ((int64_t)len.size() * top > 40000000) len.resize(2);
          walk(len, bound, heads, most);
        }
  std::printf(fails ? "FAILED\n" : "ok\n");
  return fails != 0;
}
