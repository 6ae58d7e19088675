// chunk_plan.h -- how chunk attention cuts a ragged batch into work: items, units, pieces.
// Host and device code both use it (a host test checks its arithmetic against loops).
//
// A request's query rows, G heads of a kv-head times its n new tokens, are cut into items of
// 2^lt tokens (256 rows on the tensor cores). An item attends to keys [0, p + 1), p the
// position of its last token, in tiles of 128 keys, and counts as tiles + 4 units: its own
// start and end, with the masked tiles, cost about four tiles (weighed as one, the busiest
// block of a batch of short prompts had a quarter more to do than the mean one). Units are
// numbered request after request, kv-head after kv-head, item after item, and each of the
// launch's workers takes an equal, contiguous range of them, so the split is even whatever the
// lengths; an item cut by a range's end is merged afterwards.
#pragma once

#if defined(__CUDACC__)
#define PDA_CHUNK_HD __host__ __device__ __forceinline__
#else
#define PDA_CHUNK_HD inline
#endif

namespace pda {

constexpr int kChunkKeys = 128;    // keys of a tile
constexpr int kItemUnits = 4;      // units of an item besides its tiles

// Units fit 31 bits: the host refuses sizes whose bound on them does not. What only passes
// through larger values on the way is unsigned, where wrapping cancels.
struct ChunkReq {
  int n, L;     // new tokens, and all of them; n <= L
  int lt;       // log2 of an item's tokens
  PDA_CHUNK_HD int items() const {
    return static_cast<int>((static_cast<unsigned>(n) + (1u << lt) - 1) >> lt);
  }
  // key tiles of item i
  PDA_CHUNK_HD int tiles(int i) const {
    const unsigned end = (static_cast<unsigned>(i) + 1) << lt;
    const int last = L - n + static_cast<int>(end < static_cast<unsigned>(n) ? end : n) - 1;
    return (last >> 7) + 1;
  }
  // x (x - 1) / 2
  static PDA_CHUNK_HD unsigned pairs(unsigned x) {
    return (x & 1) != 0 ? x * ((x - 1) >> 1) : (x >> 1) * (x - 1);
  }
  // sum of floor(y / 2^s) over 0 <= y < x
  static PDA_CHUNK_HD unsigned floor_sum(unsigned x, int s) {
    const unsigned q = x >> s;
    return (pairs(q) << s) + q * (x - (q << s));
  }
  // units of items [0, i), i < items(): all of them full. With a = L - n, item j's last
  // position is a + (j + 1) 2^lt - 1, so its tiles are a floor of an arithmetic progression.
  PDA_CHUNK_HD int units_before(int i) const {
    const int a1 = L - n - 1;  // may be -1: the shifts below round down
    const unsigned m = i;
    if (lt >= 7)
      return static_cast<int>(m * ((a1 >> 7) + 1 + kItemUnits) + (pairs(m + 1) << (lt - 7)));
    const int s = 7 - lt;
    const unsigned x0 = (a1 >> lt) + 1;
    return static_cast<int>((1 + kItemUnits) * m + floor_sum(x0 + m, s) - floor_sum(x0, s));
  }
  // units of one kv-head
  PDA_CHUNK_HD int units() const {
    if (n == 0) return 0;
    const int last = items() - 1;
    return units_before(last) + tiles(last) + kItemUnits;
  }
  // the item that holds unit w of a kv-head
  PDA_CHUNK_HD int item_of(int w) const {
    int lo = 0, hi = items() - 1;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (units_before(mid) <= w)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

// The same with a sliding window: an item attends to the first tokens' tiles and to those from its
// first token's window on, tiles between are left out, so its tile j is key tile j, or
// j + skipped(i) behind the first tokens'.
struct WindowReq : ChunkReq {
  int window;      // keys a token sees up to itself, >= 1
  int sink_tiles;  // key tiles that hold first tokens
  // first key of the window of item i's first token
  PDA_CHUNK_HD int lowest(int i) const {
    const int a = L - n + static_cast<int>(static_cast<unsigned>(i) << lt) - window + 1;
    return a > 0 ? a : 0;
  }
  PDA_CHUNK_HD int skipped(int i) const {
    const int s = (lowest(i) >> 7) - sink_tiles;
    return s > 0 ? s : 0;
  }
  PDA_CHUNK_HD int tiles(int i) const { return ChunkReq::tiles(i) - skipped(i); }
  // skipped tiles of items [0, i): of those from the first item on whose window starts behind the
  // first tokens' tiles, floors of an arithmetic progression again
  PDA_CHUNK_HD unsigned skipped_before(int i) const {
    const int a = L - n - window + 1;
    const int from = (sink_tiles + 1) << 7;  // the window's start where the first tile is skipped
    const unsigned up = from > a ? static_cast<unsigned>(from) - static_cast<unsigned>(a) : 0u;
    const unsigned j0 = (up >> lt) + ((up & ((1u << lt) - 1)) != 0);
    const unsigned m = i;
    if (j0 >= m) return 0;
    unsigned sum;
    if (lt >= 7) {
      sum = (m - j0) * static_cast<unsigned>(a >> 7) + ((pairs(m) - pairs(j0)) << (lt - 7));
    } else {
      const unsigned x0 = static_cast<unsigned>(a >> lt);
      sum = floor_sum(x0 + m, 7 - lt) - floor_sum(x0 + j0, 7 - lt);
    }
    return sum - (m - j0) * static_cast<unsigned>(sink_tiles);
  }
  PDA_CHUNK_HD int units_before(int i) const {
    return static_cast<int>(static_cast<unsigned>(ChunkReq::units_before(i)) - skipped_before(i));
  }
  PDA_CHUNK_HD int units() const {
    if (n == 0) return 0;
    const int last = items() - 1;
    return units_before(last) + tiles(last) + kItemUnits;
  }
  PDA_CHUNK_HD int item_of(int w) const {
    int lo = 0, hi = items() - 1;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (units_before(mid) <= w)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

// Where a cut at unit u of an item that starts at unit `start` really falls: before key tile
// u - start - kItemUnits, or at the item's start or end where that leaves a piece of fewer than
// `least` tiles.
PDA_CHUNK_HD int chunk_snap(int u, int start, int tiles, int least) {
  const int j = u - start - kItemUnits;
  if (j < least) return start;
  if (tiles - j < least) return start + tiles + kItemUnits;
  return u;
}

// First unit of worker c's range, before snapping.
PDA_CHUNK_HD int chunk_cut(int units, int workers, int c) {
  const unsigned w = workers, q = static_cast<unsigned>(units) / w, r = units - q * w;
  return static_cast<int>(c * q + c * r / w);
}

// Workers a launch of `units` units uses: no more than leave each `least` of them.
PDA_CHUNK_HD int chunk_workers(long long units, int workers, int least) {
  const long long most = units >> 30 != 0 ? workers
                                          : (static_cast<unsigned>(units) + least - 1) /
                                                static_cast<unsigned>(least);
  return most < 1 ? 1 : most < workers ? static_cast<int>(most) : workers;
}

}  // namespace pda
