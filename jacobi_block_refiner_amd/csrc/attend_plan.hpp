// How a call of the block attention is cut into items, and how many partial results it can leave.
// Plain integer functions, so they compile for the host alone too.
#pragma once

#include "xpress.h"

#include <algorithm>
#include <cstdint>

namespace xpress {

constexpr int kSlim = 2, kNarrow = 4, kWide = 8;  // waves (of 32 query rows) of an item
constexpr int kIds = 1024;  // table entries an item keeps in LDS: bounds its range of keys

struct AttendPlan {
  bool wide;  // the shared part goes to a launch of wide items
  int tiles_sh, s_sh, chunk_sh, tiles_own, s_own;
  int slots() const { return s_sh + s_own; }
};

constexpr int kTile = 64;  // the shared part is a multiple of it
constexpr int narrow_step(int D) { return D == 64 ? 64 : 32; }  // keys of a tile
constexpr int kWideStep = 64;
constexpr int kCUs = 256;
// Query rows a head from which the shared part goes to wide items, D 128 alone. Narrow against wide,
// us a call: 512 rows, 8192 keys 39 and 54; 1024 rows, 4096 keys 39 and 50; 1536 rows, 4096 keys 58
// and 53; 2048 rows, 4096 keys 62 and 59; 2048 rows, 16384 keys 197 and 160; 4096 rows, 2048 keys 65
// and 59; 20480 rows, 16384 keys 1579 and 1495. At D 64 (4096 and 16384 rows, 8192 keys) 62 and 80,
// 199 and 244: its tiles have half the products for the same weights; at D 256 (2048 and 8192 rows)
// 177 and 205, 510 and 638: one wave's sums alone take 256 registers.
constexpr int kWideRows = 1536;
constexpr int kWideItems = 2048;  // wide items at most, unless one split a tile makes more
// Narrow items wanted where the rows alone give fewer: kItems without a shared part; with one, of the
// shared part half of it at D 64 (three workgroups a CU) and a quarter else (two, one): more slots
// cost their join (16 requests of 16 tokens x 4 heads, 4096 shared and 512 own keys, D 128: 47 us
// with 512 items of the shared part, 42 with 256; 32 requests of 16 tokens x 32 heads at D 64, 8192
// shared: 66 with 512, 82 with 256), and of the requests' own half of it, but a quarter at D 256 (32
// requests decoding, D 128: 33 us with 512, 38 with 256; 32 requests at D 256: 159 and 156).
constexpr int kItems = 1024;
constexpr int kLeast = 128;  // keys of a split of one request's own at least,
constexpr int kLeastShared = 256;  // and of the shared part (more splits cost the join: 41 -> 36 us)
constexpr int kFewRows = 2048;  // rows of out up to which the join takes four groups of slots
constexpr int kSplits = 64;  // splits of one row's keys at most (more where ids do not fit in LDS)

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Keys of one item at most: its table entries have to fit in LDS.
inline int64_t most_keys(const xpress_cache& c) { return (int64_t)(kIds - 2) * c.page / 64 * 64; }

inline AttendPlan plan_of(const xpress_cache& c, int N, int B, int Hq, int shared) {
  const int G = Hq / c.Hkv;
  const int64_t cap = (int64_t)c.table_ld * c.page, most = most_keys(c), own = cap - shared;
  const int64_t rows = (int64_t)N * B * G;
  AttendPlan p{};
  p.wide = shared > 0 && c.D == 128 && rows >= kWideRows;
  p.tiles_own = (int)ceil_div((int64_t)B * G, kNarrow * 32);
  const int want = p.wide ? kCUs
                   : shared == 0 ? kItems
                   : c.D == 256  ? kItems / 4
                                 : kItems / 2;
  int64_t s = ceil_div(want, (int64_t)N * c.Hkv * p.tiles_own);
  s = std::max<int64_t>(1, std::min({s, ceil_div(own, p.wide ? 4 * kLeast : kLeast), (int64_t)kSplits}));
  // (a request that does not see the whole shared part has less than shared + B keys, all its own)
  p.s_own = (int)std::max(s, ceil_div(std::max(own, std::min<int64_t>(cap, (int64_t)shared + B)), most));
  if (shared > 0) {
    const int KT = p.wide ? kWideStep : narrow_step(c.D);
    p.tiles_sh = (int)ceil_div(rows, (p.wide ? kWide : kNarrow) * 32);
    const int64_t tiles = (int64_t)c.Hkv * p.tiles_sh;
    if (p.wide) {
      // One workgroup a CU: rounds of the card times the keys of an item, with what an item's start
      // and end and one more slot to join cost in tiles.
      int64_t best = 0;
      s = 1;
      for (int64_t x = 1; x <= std::min<int64_t>(kSplits, ceil_div(shared, 4 * KT)); ++x) {
        if (x > 1 && tiles * x > kWideItems) break;
        const int64_t cost = ceil_div(tiles * x, kCUs) * (ceil_div(shared, x * KT) + 4) +
                             x * rows * c.Hkv / (kCUs * 32);
        if (best == 0 || cost < best) {
          best = cost;
          s = x;
        }
      }
    } else {
      s = ceil_div(c.D == 64 ? kItems / 2 : kItems / 4, tiles);
      s = std::max<int64_t>(1, std::min({s, ceil_div(shared, kLeastShared), (int64_t)kSplits}));
    }
    s = std::max(s, ceil_div(shared, most));
    p.chunk_sh = (int)(ceil_div(ceil_div(shared, s), KT) * KT);
    p.s_sh = (int)ceil_div(shared, p.chunk_sh);
  }
  return p;
}

// Largest number of (row of the batch, slot) pairs of any N <= n and any shared: with A items
// wanted for n requests, n * ceil(A / n) <= A + n; every bound grows with n.
inline int64_t most_row_slots(const xpress_cache& c, int n, int B, int Hq) {
  const int G = Hq / c.Hkv;
  const int64_t cap = (int64_t)c.table_ld * c.page, ids = ceil_div(cap, most_keys(c));
  const int64_t tiles = ceil_div((int64_t)B * G, kNarrow * 32);
  const int64_t fits = std::min<int64_t>(kSplits, ceil_div(cap, kLeast));
  const int64_t own = std::min(ceil_div(kItems, c.Hkv * tiles) + n, n * fits);
  // (a narrow call splits as far as kItems / 2 items, a wide one as far as kWideItems)
  const int64_t sh = std::min(
      ceil_div((int64_t)kWideItems * kWide * 32, (int64_t)c.Hkv * B * G) + n, n * fits);
  return std::max<int64_t>(own, n * ids) + std::max<int64_t>(sh, n * ids);
}

}  // namespace xpress
