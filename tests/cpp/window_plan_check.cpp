// Checks the closed forms of chunk_plan.h's windowed requests against loops over keys. Exits 0
// if they hold.
#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "chunk_plan.h"

using namespace pda;

static void require(bool ok, const char* what, const WindowReq& r) {
  if (ok) return;
  std::printf("%s: n %d L %d lt %d window %d sink tiles %d\n", what, r.n, r.L, r.lt, r.window,
              r.sink_tiles);
  std::exit(1);
}

int main() {
  unsigned seed = 7;
  auto rnd = [&](int m) { return static_cast<int>((seed = seed * 1664525u + 1013904223u) >> 8) % m; };
  for (int it = 0; it < 30000; ++it) {
    WindowReq r;
    r.lt = 3 + rnd(6);
    r.n = it < 8000 ? 1 + rnd(600) : 1 + rnd(9000);
    r.L = r.n + (rnd(3) ? rnd(it % 2 ? 300 : 20000) : 0);
    const int kinds[] = {1, 1 + rnd(16), 1 + rnd(300), 1 + rnd(5000), 1 + rnd(1 << 30)};
    r.window = kinds[rnd(5)];
    const int sinks[] = {0, 1, 1 + rnd(4), 1 + rnd(200), 1 << 23};
    r.sink_tiles = sinks[rnd(5)];
    const int tok = 1 << r.lt;
    long long sum = 0;
    for (int i = 0; i < r.items(); ++i) {
      require(r.units_before(i) == sum, "units_before", r);
      const int first = r.L - r.n + i * tok, last = r.L - r.n + std::min((i + 1) * tok, r.n) - 1;
      const int lowest = std::max(0, first - r.window + 1);
      require(r.lowest(i) == lowest, "lowest", r);
      // a tile is the item's if it holds first tokens or reaches the first token's window
      int tiles = 0, before = 0;
      for (int j = 0; j <= last / 128; ++j) {
        const bool in = j < r.sink_tiles || j >= lowest / 128;
        const int real = tiles + (tiles >= r.sink_tiles ? r.skipped(i) : 0);
        if (in) require(real == j, "key tile", r);
        tiles += in;
        before += !in;
      }
      require(r.skipped(i) == before && r.tiles(i) == tiles, "tiles", r);
      require(r.item_of(static_cast<int>(sum)) == i &&
                  r.item_of(static_cast<int>(sum) + tiles + kItemUnits - 1) == i,
              "item_of", r);
      sum += tiles + kItemUnits;
    }
    require(r.units() == sum, "units", r);
  }
  // long histories, where intermediate sums pass 32 bits
  for (int k = 0; k < 200; ++k) {
    WindowReq r;
    r.lt = 3 + rnd(6);
    r.n = 1 + rnd(4000);
    r.L = (1 << 24) + rnd((1 << 30) - (1 << 24) - 5000);
    r.window = rnd(2) ? 1 + rnd(20000) : 1 + rnd(1 << 24);
    r.sink_tiles = rnd(3) ? rnd(4) : 1 << 23;
    long long sum = 0;
    for (int i = 0; i < r.items() && sum < (1ll << 30); ++i) {
      require(r.units_before(i) == sum, "long", r);
      sum += r.tiles(i) + kItemUnits;
    }
  }
  std::puts("ok");
  return 0;
}
