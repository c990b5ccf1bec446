// How a call of the block attention is cut into items, and how many partial results it can leave.
// Plain integer functions, so they compile for the host alone too.
#pragma once

#include "cache_index.hpp"
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
// Keys of a tile. From 4 bits two stages of 64 keys fit where 16 bits take four of 32, and a tile's codes
// are asked for a tile ahead: us a call with 64 and 32, D 128: 128 requests decoding behind 16,384 tokens 65
// and 73, 32 behind 32,768 41 and 45; D 256: 32 blocks of 16 behind 8192 266 and 328, 64 of up to 2000
// tokens 217 and 248. (A slim item of 64 has no registers for it.)
constexpr int kSlimStep = 32;
constexpr int narrow_step(int D, bool mx4) { return D == 64 || mx4 ? 64 : 32; }
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
    const int KT = p.wide ? kWideStep : narrow_step(c.D, c.dtype > 15u);
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

// The register path over 4 bits (few_kernel).
constexpr int kFewTile = 32;   // keys of a step of a wave
constexpr int kFewRequests = 4096;  // more are not cut: a part a pair
constexpr int kFewRows4 = 64;  // query rows of a request and head at most

// Workgroups on a CU, by the registers.
constexpr int few_per_cu(int D) { return D == 64 ? 3 : 2; }
// Row tiles of a wave, waves of a part, and parts of the sequence. At D 256 two row tiles would have a
// SIMD to themselves and no registers left.
constexpr int few_row_tiles(int D, int R) { return R <= 16 || D == 256 ? 1 : 2; }
constexpr int few_waves(int D, int R) {
  const int n = (R - 1) / (16 * few_row_tiles(D, R));
  return n == 0 ? 1 : n == 1 ? 2 : 4;
}
constexpr int few_parts(int D, int R) { return kCUs * few_per_cu(D) * 4 / few_waves(D, R); }

// Whether it takes the own keys of N requests with R query rows a head. Up to 32 rows: always, and up to 64
// from so many keys of all heads on (by what the tables hold), where the items' meetings cost more than
// reading codes in several waves. 16 tokens of 4 heads a head, 8 heads, tables of up to so many own
// tokens, us a call, few_kernel and items:
//   D 64: 64 x 4000 57 and 67, 64 x 2000 41 and 43, 8 x 16,000 37 and 41; 64 x 1000 34 and 31, 32 x 2000
//   33 and 32, 4 x 16,000 31 and 28, 1 x 16,000 25 and 19.
//   D 128: 64 x 4000 93 and 120, 64 x 1000 48 and 50, 8 x 4000 31 and 34, 2 x 16,000 32 and 38; 64 x 300
//   36 and 35, 16 x 1000 28 and 27, 4 x 4000 28 and 28, 1 x 16,000 27 and 25. Not taken where it wins: 8 x
//   2000 27 and 29; taken where it loses: 32 x 1000 37 and 36.
//   D 256: 64 x 4000 182 and 275, 64 x 300 58 and 64, 8 x 2000 37 and 47, 1 x 16,000 38 and 43; 16 x 300 31
//   and 27, 8 x 1000 34 and 30, 2 x 4000 31 and 30, 1 x 4000 29 and 24. Not taken where it wins: 4 x 1000 26
//   and 29, 1 x 300 15 and 19.
// (More rows, 80 and 128: 64 x 4000 at D 128 137 and 123, 154 and 135; at D 64 87 and 77, 95 and 83.)
constexpr int64_t few_keys(int D) { return D == 64 ? 3 << 18 : D == 128 ? 7 << 15 : 7 << 14; }
inline bool few_rows(const xpress_cache& c, int N, int R, int shared) {
  const int64_t keys = (int64_t)N * c.Hkv * ((int64_t)c.table_ld * c.page - shared);
  return R <= 32 || (R <= kFewRows4 && keys >= few_keys(c.D));
}

// A (request, head) pair whose keys lie in several parts of the sequence of all: it begins in this one.
struct Cut {
  int pair, slots;  // (0: it is whole, or none begins here)
  int part, slot;   // where it begins, its slot there; then slots 2 (part + 1), 2 (part + 2), ..
};
// A record as the join uses it: inside the pairs and the 2 * parts slots, whatever it holds. (Where
// another stream changes lengths during a call, a pair may begin in no part, and its record is an old one.)
XP_HD Cut cut_inside(Cut c, int pairs, int parts) {
  auto within = [](int x, int lo, int hi) { return x < lo ? lo : (x < hi ? x : hi); };
  c.pair = within(c.pair, 0, pairs - 1);
  c.part = within(c.part, 0, parts - 1);
  c.slot = 2 * c.part + (c.slot & 1);
  c.slots = within(c.slots, 0, parts - c.part);
  return c;
}

// A wave holds the page ids of 64 tiles, from `from` on, and finds each tile's addresses while it works
// on the one before. At tile t of those up to t1: whether the next tile's ids have to be read first, and
// up to where it can then go on (past t, always).
inline constexpr int kFewIds = 64;
XP_HD bool few_ids_wanted(int t, int from, int t1) { return t + 1 < t1 && t + 1 - from >= kFewIds; }
XP_HD int few_run_end(int t, int from, int t1) {
  const int known = from + kFewIds - 1;  // the last tile whose ids are held
  return t + 1 < t1 && known < t1 ? known : t1;
}

}  // namespace xpress
