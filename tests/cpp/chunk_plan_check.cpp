// Checks chunk_plan.h's closed forms against loops, and that the workers' snapped ranges cover
// every key tile of every item once, in pieces no shorter than asked for. Exits 0 if they do.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "chunk_plan.h"

using namespace pda;

static void require(bool ok, const char* what, int n, int L, int lt) {
  if (ok) return;
  std::printf("%s: n %d L %d lt %d\n", what, n, L, lt);
  std::exit(1);
}

int main() {
  unsigned seed = 1;
  auto rnd = [&](int m) { return static_cast<int>((seed = seed * 1664525u + 1013904223u) >> 8) % m; };
  for (int it = 0; it < 20000; ++it) {
    ChunkReq r;
    r.lt = 3 + rnd(6);
    r.n = it < 4000 ? 1 + rnd(600) : 1 + rnd(9000);
    r.L = r.n + (rnd(3) ? rnd(it % 2 ? 300 : 20000) : 0);
    long long sum = 0;
    const int tok = 1 << r.lt;
    require(r.items() == (r.n + tok - 1) / tok, "items", r.n, r.L, r.lt);
    for (int i = 0; i < r.items(); ++i) {
      require(r.units_before(i) == sum, "units_before", r.n, r.L, r.lt);
      const int last = (i + 1) * tok < r.n ? (i + 1) * tok : r.n;
      const int tiles = (r.L - r.n + last + 127) / 128;
      require(r.tiles(i) == tiles, "tiles", r.n, r.L, r.lt);
      require(r.item_of(sum) == i && r.item_of(sum + tiles) == i, "item_of", r.n, r.L, r.lt);
      sum += tiles + kItemUnits;
    }
    require(r.units() == sum, "units", r.n, r.L, r.lt);
  }
  // intermediate sums past 32 bits cancel: long histories, few rows of small items
  for (int k = 0; k < 40; ++k) {
    ChunkReq r;
    r.lt = 3 + rnd(6);
    r.n = 1 + rnd(4000);
    r.L = (1 << 24) + rnd(1 << 28);
    long long sum = 0;
    for (int i = 0; i < r.items() && sum < (1ll << 30); ++i) {
      require(r.units_before(i) == sum, "long", r.n, r.L, r.lt);
      sum += r.tiles(i) + kItemUnits;
    }
  }
  for (int it = 0; it < 300; ++it) {
    std::vector<ChunkReq> reqs;
    const int B = 1 + rnd(9), H_kv = 1 + rnd(4), lt = 3 + rnd(6), least = 1 + rnd(6);
    std::vector<long long> start;
    std::vector<int> tiles;
    long long W = 0;
    for (int b = 0; b < B; ++b) {
      ChunkReq r;
      r.lt = lt;
      r.n = rnd(4) ? 1 + rnd(900) : 1;
      r.L = r.n + rnd(6000);
      for (int k = 0; k < H_kv; ++k)
        for (int i = 0; i < r.items(); ++i) {
          start.push_back(W);
          tiles.push_back(r.tiles(i));
          W += r.tiles(i) + kItemUnits;
        }
    }
    const int workers = chunk_workers(W, 1 + rnd(152), 1 + rnd(8));
    std::vector<std::vector<int>> seen;
    for (int t : tiles) seen.push_back(std::vector<int>(t, 0));
    auto snapped = [&](int c) -> long long {
      const int u = chunk_cut(static_cast<int>(W), workers, c);
      if (u >= W) return W;
      size_t i = 0;
      while (i + 1 < start.size() && start[i + 1] <= u) ++i;
      return chunk_snap(u, static_cast<int>(start[i]), tiles[i], least);
    };
    require(snapped(0) == 0 && snapped(workers) == W, "ends", B, H_kv, lt);
    for (int c = 0; c < workers; ++c) {
      const long long s0 = snapped(c), s1 = snapped(c + 1);
      require(s0 <= s1, "order", B, H_kv, lt);
      int inside = 0;
      for (size_t i = 0; i < start.size(); ++i) {
        const long long end = start[i] + tiles[i] + kItemUnits;
        const long long a = s0 > start[i] ? s0 : start[i], b = s1 < end ? s1 : end;
        if (a >= b) continue;
        const int ja = a == start[i] ? 0 : static_cast<int>(a - start[i] - kItemUnits);
        const int jb = b == end ? tiles[i] : static_cast<int>(b - start[i] - kItemUnits);
        require(jb > ja, "empty piece", B, H_kv, lt);
        if (jb - ja < tiles[i]) require(jb - ja >= least || workers > W / least, "short piece", jb - ja, least, lt);
        inside += ja > 0;
        for (int j = ja; j < jb; ++j) seen[i][j]++;
      }
      require(inside <= 1, "pieces that start inside", B, H_kv, lt);
    }
    for (auto& s : seen)
      for (int x : s) require(x == 1, "tile covered once", B, H_kv, lt);
  }
  std::puts("ok");
  return 0;
}
