// Attention of drafted blocks over a paged cache of 4 bits (gfx950).
//
// Query rows of the shared part, and of requests with many of them a head, go to the items of
// attend_kernel.hpp. The requests' own keys with up to 32 rows a head (decoding, short blocks; up to 64
// over long contexts) are HBM's: 2 * 17 D / 32 bytes a key for few operations. few_kernel reads them
// straight into the matrix core's registers, a wave 16 or 32 rows; one, two or four waves of a workgroup
// take a request's rows and read the same keys, from HBM once.
//
// All (request, head) pairs' tiles of 32 keys form one sequence, which is cut into as many equal parts
// as there are waves (or such groups of them) on the card, whatever the lengths: a wave finds its part
// from the lengths themselves. A pair that lies in one part is finished there; where it is cut, each part
// leaves (sums, unit of the weights, their sum) in a slot, and join_kernel joins them. Beside a shared
// part all pairs leave theirs, and are joined with its items'. (One wave a pair that read the shared
// slots too took 120 of 133 us at 32 requests behind 4096 tokens.)
#include "attend_kernel.hpp"

namespace xpress {

namespace {

struct Few {
  Args a;
  int parts;  // of the sequence, where it is cut; else 0
  int least;  // tiles of a part at least
  int waves;  // of a part, with 16 RT rows each: 1, 2 or 4
  bool by_pair;  // cut[] is of the pairs; else of the parts: of the pair that begins there and goes on
  float* po;   // [2 * parts, R, D]
  float2* pml; // [2 * parts, R]
  Cut* cut;
};

typedef float f32x4v __attribute__((ext_vector_type(4)));

template <bool F16>
__device__ __forceinline__ f32x4v mfma16(const s16x8& a, const s16x8& b, const f32x4v& c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// N words from an address that is aligned to all of them.
template <int N> __device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
}

// A wave's 16 RT query rows against tiles of 32 keys, all in registers. Scores are formed transposed,
// S^T = K Q^T (16 keys x 16 queries): a lane holds four keys' of one query, and as weights they are the
// right operand of O^T = V^T P^T as they stand. The lane's bytes of K are eight channels of each of the
// product's steps, and K's and V's conversion to 16 bits takes one instruction a pair (V one more, to
// put two tokens of a channel beside each other). 32 keys of 16 queries at D 128 take about 250 vector
// instructions, 1000 cycles; at 5 TB/s a SIMD has 2000.
template <bool F16, int D, int RT> struct FewCore {
  static constexpr int NG = D / 32;
  static constexpr float kLift = F16 ? 7.f : -37.f;  // as in Core
  static constexpr float kHuge = 0x1p20f;

  int lane, i, q;
  uint32_t k_at, ks_at, v_at, vs_at;  // the lane's bytes in a tile of 16 tokens
  uint32_t ks_bit;                    // of its scale in the four bytes at ks_at
  float c;
  // A tile of 32 keys as a lane holds it, 16 tokens and 16. With lane = 16 q + i: of K, token i, the
  // q-th quarter of the channels (of 256 channels two eighths); of V, the pairs of channels i of all
  // groups, tokens 4q..4q+3.
  uint32_t kc[2][NG], ks[2][D == 256 ? 2 : 1], vc[2][NG], vs[2][NG];
  s16x8 qf[RT][NG];
  f32x4v s[RT][2];
  s16x8 pf[RT];
  f32x4v o[RT][NG][2];  // channels 32g + 8q + 2r (and + 1) of query i
  float m[RT], l[RT], shift[RT];
  uint64_t huge[RT];

  __device__ __forceinline__ void begin(float scale) {
    lane = threadIdx.x & 63;
    i = lane & 15;
    q = lane >> 4;
    c = scale;
    k_at = i * (D / 2) + q * (D == 256 ? 16 : D / 8);
    const uint32_t at = mx4_k_scale(D, i, D == 64 ? q / 2 : q);
    ks_at = at & ~3u;
    ks_bit = at % 4 * 8;
    v_at = lane * (D / 8);
    vs_at = mx4_v_scale(D, 4 * q, 0);
  }
  // Channel of the lane's eight of step s of the product.
  __device__ __forceinline__ int channel(int s) const {
    return D == 64 ? 16 * q + 8 * s : s / 4 * 128 + 32 * q + 8 * (s % 4);
  }
  __device__ __forceinline__ void take(int rt, const uint16_t* row) {
#pragma unroll
    for (int s = 0; s < NG; ++s) qf[rt][s] = *reinterpret_cast<const s16x8*>(row + channel(s));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int g = 0; g < NG; ++g) o[rt][g][0] = o[rt][g][1] = f32x4v{};
      m[rt] = -1e30f;
      l[rt] = 0.f;
      huge[rt] = ~0ull;
    }
  }

  // The lane's bytes of tiles of K and of V. (A scalar base and a 32-bit offset of the lane, as long as
  // the compiler does not widen the offset ahead of the loop.)
  static __device__ __forceinline__ uint32_t here(uint32_t offset) {
    asm volatile("" : "+v"(offset));
    return offset;
  }
  __device__ __forceinline__ void load_k(const uint8_t* const (&k)[2]) {
    const uint32_t k_at = here(this->k_at), ks_at = here(this->ks_at);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if constexpr (D == 256) {
        const uint4 a = *reinterpret_cast<const uint4*>(k[x] + k_at);
        const uint4 b = *reinterpret_cast<const uint4*>(k[x] + (k_at + 64));
        kc[x][0] = a.x, kc[x][1] = a.y, kc[x][2] = a.z, kc[x][3] = a.w;
        kc[x][4] = b.x, kc[x][5] = b.y, kc[x][6] = b.z, kc[x][7] = b.w;
        ks[x][1] = *reinterpret_cast<const uint32_t*>(k[x] + (ks_at + 4));
      } else {
        load_words<NG>(k[x] + k_at, kc[x]);
      }
      ks[x][0] = *reinterpret_cast<const uint32_t*>(k[x] + ks_at);
    }
  }
  __device__ __forceinline__ void load_v(const uint8_t* const (&v)[2]) {
    const uint32_t v_at = here(this->v_at), vs_at = here(this->vs_at);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      load_words<NG>(v[x] + v_at, vc[x]);
      load_words<NG>(v[x] + vs_at, vs[x]);
    }
  }

  __device__ __forceinline__ s16x8 k_frag(int x, int s) const {
    const float scale = mx4_scale<0>(ks[x][D == 256 ? s / 4 : 0] >> ks_bit);
    const uint32_t w = kc[x][s];
    return __builtin_bit_cast(s16x8, make_uint4(mx4_pair<F16, 0>(w, scale), mx4_pair<F16, 1>(w, scale),
                                                mx4_pair<F16, 2>(w, scale), mx4_pair<F16, 3>(w, scale)));
  }

  // Scores of the tile; weights, where query i of row tile rt sees the keys below vis (a lane's are
  // 4q.. and 16 + 4q..); their products with its values, `end` keys of which are the row's. Each takes
  // the tile's bytes out of its registers, and the next tile's loads go there behind it.
  __device__ __forceinline__ void scores() {
#pragma unroll
    for (int d = 0; d < NG; ++d) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const s16x8 k = k_frag(x, d);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          s[rt][x] = mfma16<F16>(k, qf[rt][d], d == 0 ? f32x4v{} : s[rt][x]);
      }
    }
  }
  __device__ __forceinline__ void weights(const int (&vis)[RT], bool masked) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (masked) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[rt][x][r] = 16 * x + 4 * q + r < vis[rt] ? s[rt][x][r] : -INFINITY;
      }
      rise(rt);
      float sum[2] = {l[rt], 0.f};
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = __builtin_amdgcn_exp2f(fmaf(s[rt][j / 2][j % 2 * 2], c, shift[rt]));
        const float b = __builtin_amdgcn_exp2f(fmaf(s[rt][j / 2][j % 2 * 2 + 1], c, shift[rt]));
        sum[j % 2] += a + b;
        w[j] = pack2<F16>(a, b);
      }
      l[rt] = sum[0] + sum[1];
      pf[rt] = __builtin_bit_cast(s16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
  __device__ __forceinline__ void values(int end, bool masked) {
    if (masked) {
      // keys past the end: a scale of 1, as what lies there could stand for infinity
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = min(max(end - 16 * x - 4 * q, 0), 4);
        const uint32_t keep = n == 4 ? ~0u : (1u << 8 * n) - 1;
#pragma unroll
        for (int g = 0; g < NG; ++g) vs[x][g] = (vs[x][g] & keep) | (0x7f7f7f7fu & ~keep);
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      __builtin_amdgcn_sched_barrier(0);
      uint32_t even[4], odd[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t w = vc[x][g], e = vs[x][g];
        const uint32_t a = mx4_pair<F16, 0>(w, mx4_scale<0>(e)), b = mx4_pair<F16, 1>(w, mx4_scale<1>(e));
        const uint32_t d = mx4_pair<F16, 2>(w, mx4_scale<2>(e)), f = mx4_pair<F16, 3>(w, mx4_scale<3>(e));
        even[2 * x] = low_halves(a, b), even[2 * x + 1] = low_halves(d, f);
        odd[2 * x] = high_halves(a, b), odd[2 * x + 1] = high_halves(d, f);
      }
      const s16x8 ve = __builtin_bit_cast(s16x8, make_uint4(even[0], even[1], even[2], even[3]));
      const s16x8 vo = __builtin_bit_cast(s16x8, make_uint4(odd[0], odd[1], odd[2], odd[3]));
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        o[rt][g][0] = mfma16<F16>(ve, pf[rt], o[rt][g][0]);
        o[rt][g][1] = mfma16<F16>(vo, pf[rt], o[rt][g][1]);
      }
    }
  }

  // log2 of the weights' unit.
  __device__ __forceinline__ float unit(int rt) const { return fmaf(m[rt], c, -kLift); }

  // As Core::rise: the sums are rescaled only where some row's maximum grew by more than 2^8 in weight.
  // The four lanes of a query have one maximum; they exchange theirs only then.
  __device__ __forceinline__ void rise(int rt) {
    float top = s[rt][0][0];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, s[rt][x][r]);
    if ((__ballot((top - m[rt]) * c > 8.f) | huge[rt]) != 0) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      raise(rt, fmaxf(m[rt], top));
      shift[rt] = -unit(rt);
      huge[rt] = __ballot(fabsf(shift[rt]) > kHuge);
      if (huge[rt] != 0) {
        s[rt][0] -= m[rt];
        s[rt][1] -= m[rt];
        shift[rt] = kLift;
      }
    }
  }
  __device__ __forceinline__ void raise(int rt, float to) {
    const float alpha = __builtin_amdgcn_exp2f((m[rt] - to) * c);
    l[rt] *= alpha;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      o[rt][g][0] *= alpha;
      o[rt][g][1] *= alpha;
    }
    m[rt] = to;
  }
};

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t scalar(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x);
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 | lo);
}

// Tiles of a request's own keys (one at least: it writes what the request has without them).
__device__ __forceinline__ int own_tiles(const Args& A, int len) {
  return max((len - own_begin(len, A.B, A.shared) + kFewTile - 1) / kFewTile, 1);
}

template <bool F16, int D, int RT>
__device__ __forceinline__ void few_part(const Few& F, int block) {
  constexpr int NG = D / 32;
  const Args& A = F.a;
  const int wave = scalar((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int R = A.B * A.G;
  // this wave's rows, and its part of the sequence: tiles [at, end) of all, beginning in a request with
  // `before` tiles a head in front of it
  const int per_block = 4 / F.waves, part = block * per_block + wave / F.waves;
  const int row0 = wave % F.waves * 16 * RT;
  int64_t at, end, before = 0, each = 0;
  int request, row, len;
  if (F.parts) {
    __shared__ int64_t s_scan[4], s_before[4];
    __shared__ int s_request[4], s_row[4], s_len[4];
    // each thread a run of requests
    const int per = (A.N + 255) / 256, r0 = threadIdx.x * per;
    int64_t mine = 0;
    for (int r = r0; r < min(r0 + per, A.N); ++r) mine += own_tiles(A, list_len(A, r));
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    if (lane == 63) s_scan[wave] = x;
    __syncthreads();
    int64_t all = 0;
    x -= mine;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      x += w < wave ? s_scan[w] : 0;
      all += s_scan[w];
    }
    all = scalar(all) * A.Hkv;
    each = all < (int64_t)1 << 31 ? (uint32_t)all / (uint32_t)F.parts : all / F.parts;
    each = max(each + (each * F.parts < all), (int64_t)F.least);
    for (int w = 0; w < per_block; ++w) {  // the thread of the request in which the part begins
      const int64_t from = (block * per_block + w) * each;
      if (from < x * A.Hkv || from >= (x + mine) * A.Hkv) continue;
      int r = r0;
      int64_t y = x;
      for (;; ++r) {
        const int n = own_tiles(A, list_len(A, r));
        if (from < (y + n) * A.Hkv || r + 1 >= min(r0 + per, A.N)) break;
        y += n;
      }
      s_request[w] = r;
      s_before[w] = y;
      s_row[w] = list_row(A, r);
      s_len[w] = list_len(A, r);
    }
    __syncthreads();
    at = part * each;
    end = min(at + each, all);
    if (at >= all) {
      if (lane == 0 && row0 == 0 && !F.by_pair) F.cut[part].slots = 0;
      return;
    }
    if (row0 >= R) return;
    request = scalar(s_request[wave / F.waves]);
    before = scalar(s_before[wave / F.waves]);
    row = scalar(s_row[wave / F.waves]);
    len = scalar(s_len[wave / F.waves]);
  } else {
    if (part >= (int64_t)A.N * A.Hkv || row0 >= R) return;
    request = part / A.Hkv;
    row = scalar(list_row(A, request));
    len = row < 0 ? 0 : clamp_len(scalar(A.len[row]), A.ld, A.shift);
    at = part % A.Hkv;  // (of the request's pairs)
    end = at + 1;
  }

  const int64_t head_bytes = mx4_tiles_bytes(D, A.shift), page_bytes = A.Hkv * head_bytes;
  const int page_mask = (1 << A.shift) - 1;
  Cut cut{0, 0, 0, 0};
  int slot = 2 * part;  // of the first pair here; then of the last
  FewCore<F16, D, RT> w;
  w.begin(A.c);

  // The tiles of one pair in this part. While it is worked on, the next one's page ids are on their
  // way, and behind its last scores the next one's first tile.
  struct Segment {
    int request, hk, len, first, tiles, t0, t1;
    const int32_t* table;
    int id0, id1;  // page ids of its tiles from `ids_from` on (of their two halves), a lane each
    int ids_from;
  };
  // First key of the row's last tile of 16.
  auto last_tile = [&](const Segment& g) { return max(g.len - 1, 0) & ~15; };
  auto ask_ids = [&](Segment& g, int from) {
    g.ids_from = from;
    const int pos = g.first + min(from + lane, g.t1 - 1) * kFewTile, last = last_tile(g);
    g.id0 = g.table[min(pos, last) >> A.shift];
    g.id1 = g.table[min(pos + 16, last) >> A.shift];
  };
  int len_ahead = 0;  // of the request behind the last one opened, as it was read
  auto read_len = [&](int r) {
    const int row = r < A.N ? list_row(A, r) : -1;
    return row < 0 ? 0 : A.len[row];
  };
  auto set_request = [&](Segment& g, int r, int row, int len) {
    g.request = r;
    g.len = len;
    g.first = own_begin(len, A.B, A.shared);
    g.tiles = own_tiles(A, len);
    g.table = A.table + (int64_t)max(row, 0) * A.ld;
    len_ahead = read_len(r + 1);
  };
  // The part's tiles of the request's head hk from t0 on.
  auto open = [&](Segment& g, int hk, int t0) {
    g.hk = hk;
    g.t0 = t0;
    g.t1 = F.parts ? (int)min((int64_t)g.tiles, t0 + (end - at)) : g.tiles;
    ask_ids(g, t0);
  };
  const uint8_t *k_next[2], *v_next[2];
  auto turn = [&](const Segment& g, int t) {
    const int pos = g.first + t * kFewTile, last = last_tile(g), nth = t - g.ids_from;
    const int p0 = min(pos, last), p1 = min(pos + 16, last);
    const int i0 = clamp_page(__builtin_amdgcn_readlane(g.id0, nth), A.n_pages);
    const int i1 = clamp_page(__builtin_amdgcn_readlane(g.id1, nth), A.n_pages);
    const int64_t a = i0 * page_bytes + g.hk * head_bytes + ((p0 & page_mask) >> 4) * mx4_tile_bytes(D);
    const int64_t b = i1 * page_bytes + g.hk * head_bytes + ((p1 & page_mask) >> 4) * mx4_tile_bytes(D);
    k_next[0] = static_cast<const uint8_t*>(A.k) + a, k_next[1] = static_cast<const uint8_t*>(A.k) + b;
    v_next[0] = static_cast<const uint8_t*>(A.v) + a, v_next[1] = static_cast<const uint8_t*>(A.v) + b;
  };
  auto take = [&](const Segment& g) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rl = min(row0 + rt * 16 + w.i, R - 1);
      w.take(rt, A.q + ((int64_t)g.request * A.B + rl / A.G) * A.q_ld +
                     (int64_t)(g.hk * A.G + rl % A.G) * D);
    }
  };

  Segment g;
  set_request(g, request, row, len);
  {
    // tiles of the request in front (below 2^31, as a table holds 2^28 tokens; where another stream
    // changes lengths meanwhile, results are unspecified, but inside the cache)
    const uint32_t in = F.parts ? (uint32_t)(at - before * A.Hkv) : (uint32_t)at * g.tiles;
    open(g, min((int)(in / g.tiles), A.Hkv - 1), (int)(in % g.tiles));
  }
  take(g);
  turn(g, g.t0);
  w.load_k(k_next);
  w.load_v(v_next);
  while (true) {
    const int64_t g0 = before * A.Hkv + (int64_t)g.hk * g.tiles;  // the pair's first tile of all
    const int all_see = in_sight(g.len, A.B, 0);
    at += g.t1 - g.t0;
    const bool other = g.hk + 1 == A.Hkv;
    const bool more = F.parts && at < end && !(other && g.request + 1 >= A.N);
    Segment next = g;
    if (more) {
      if (other) {
        const int row = scalar(list_row(A, g.request + 1));
        const int len = scalar(len_ahead);
        set_request(next, g.request + 1, row, row < 0 ? 0 : clamp_len(len, A.ld, A.shift));
      }
      open(next, other ? 0 : g.hk + 1, 0);
    }
    int vis[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) vis[rt] = in_sight(g.len, A.B, min(row0 + rt * 16 + w.i, R - 1) / A.G);
    w.clear();
    for (int t = g.t0; t < g.t1;) {
      if (few_ids_wanted(t, g.ids_from, g.t1)) ask_ids(g, t + 1);
      // the page ids are in: a load that may be under way where the loop begins makes the compiler wait
      // for all loads in every round of it
      asm volatile("" : "+v"(g.id0), "+v"(g.id1));
      const int to = few_run_end(t, g.ids_from, g.t1);
#pragma unroll 1
      for (; t < to; ++t) {
        const int at_key = g.first + t * kFewTile;
        const bool masked = at_key + kFewTile > all_see;
        int see[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) see[rt] = vis[rt] - at_key;
        w.scores();
        __builtin_amdgcn_sched_barrier(0);
        if (t + 1 < g.t1)
          turn(g, t + 1);
        else if (more)
          turn(next, 0);
        w.load_k(k_next);
        __builtin_amdgcn_sched_barrier(0);
        w.weights(see, masked);
        w.values(g.len - at_key, masked);
        __builtin_amdgcn_sched_barrier(0);
        w.load_v(v_next);
      }
    }
    if (RT == 1 && more) take(next);  // (two row tiles' queries have no registers beside the sums)

    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float l = w.l[rt];
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      const int rl = row0 + rt * 16 + w.i;
      if (rl >= R) continue;
      float o[NG][8];
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int x = 0; x < 8; ++x) o[c][x] = l == 0.f ? 0.f : w.o[rt][c][x % 2][x / 2];
      const int64_t token = (int64_t)g.request * A.B + rl / A.G;
      const int hq = g.hk * A.G + rl % A.G;
      const int64_t out_row = token * A.Hq + hq;
      if (!whole || A.slots_sh) {
        const int64_t to = whole ? A.slots_sh * (int64_t)A.N * A.B * A.Hq + out_row
                                 : (int64_t)slot * R + rl;
        float* po = (whole ? A.po : F.po) + to * D + 8 * w.q;
#pragma unroll
        for (int c = 0; c < NG; ++c) {
          *reinterpret_cast<float4*>(po + 32 * c) = make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
          *reinterpret_cast<float4*>(po + 32 * c + 4) = make_float4(o[c][4], o[c][5], o[c][6], o[c][7]);
        }
        if (w.q == 0) (whole ? A.pml : F.pml)[to] = make_float2(w.unit(rt), l);
        continue;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t* out = A.out + token * A.out_ld + (int64_t)hq * D + 8 * w.q;
#pragma unroll
      for (int c = 0; c < NG; ++c)
        *reinterpret_cast<uint4*>(out + 32 * c) = make_uint4(
            pack2<F16>(o[c][0] * inv, o[c][1] * inv), pack2<F16>(o[c][2] * inv, o[c][3] * inv),
            pack2<F16>(o[c][4] * inv, o[c][5] * inv), pack2<F16>(o[c][6] * inv, o[c][7] * inv));
      if (A.lse && w.q == 0)
        A.lse[out_row] = l == 0.f ? -INFINITY : (w.unit(rt) + log2f(l)) * 0.69314718056f;
    }
    if (F.parts && g.t0 == 0) {  // the pair begins here
      const int pair = g.request * A.Hkv + g.hk;
      const Cut c{pair, whole ? 0 : (int)((g0 + g.tiles - 1) / each - part) + 1, part, slot};
      if (F.by_pair) {
        if (lane == 0 && row0 == 0) F.cut[pair] = c;
      } else if (!whole) {
        cut = c;
      }
    }
    if (!more) break;
    if (RT != 1) take(next);
    slot = 2 * part + 1;
    if (next.request != g.request) before += g.tiles;
    g = next;
  }
  if (F.parts && !F.by_pair && lane == 0 && row0 == 0) F.cut[part] = cut;
}

// 64 requests decoding up to 32,768 tokens each (8 heads of 128, 5 queries each, 1.14 GB): 220 us, 5.2
// TB/s (a copy reaches 4.7 to 5.2, reads alone 5.9). One of 1000 tokens: 8.8 us, of them 2.3 for the lengths
// and 1.5 for the first tile of keys, and 4.1 of join_kernel.
template <bool F16, int D, int RT>
__global__ __launch_bounds__(256, few_per_cu(D)) void few_kernel(Few F) {
  few_part<F16, D, RT>(F, blockIdx.x);
}

// The shared part's narrow items beside them: 32 requests decoding behind 4096 tokens (32 heads of 128,
// up to 1024 own) 18.5 us and 5.3 of the join, 23 in all; as two launches 31.
template <bool F16, int D, int RT>
__global__ __launch_bounds__(256, narrow_per_cu(D)) void beside_kernel(Few F) {
  const int items = F.a.Hkv * F.a.tiles_sh * F.a.s_sh;
  if ((int)blockIdx.x < items)
    attend_item<F16, D, kNarrow, narrow_step(D, true), true>(F.a, blockIdx.x);
  else
    few_part<F16, D, RT>(F, blockIdx.x - items);
}

// Joins the slots of a pair that was cut, and the shared items' of every pair, in rows of the pairs (or
// of those that begin in a part and go on, where there are more pairs than parts and no shared items).
// J groups of threads take every J-th slot of a row; a workgroup has 256 / (J D / 4) rows at a time, or
// with J = 4096 / D one and 1024 threads, where a few pairs were cut into very many slots.
template <bool F16, int D, int J>
__global__ __launch_bounds__(J * D > 1024 ? 1024 : 256) void join_kernel(Few F) {
  constexpr int LPR = D / 4, RPB = J * D > 1024 ? 1 : 256 / (LPR * J);
  const Args& A = F.a;
  Cut cut{(int)blockIdx.x, 0, 0, 0};
  if (F.parts) {
    cut = cut_inside(F.cut[blockIdx.x], A.N * A.Hkv, F.parts);
    if (F.by_pair) cut.pair = blockIdx.x;
  }
  if (cut.slots == 0 && A.slots_sh == 0) return;
  const int R = A.B * A.G, d = threadIdx.x % LPR * 4;
  const int group = threadIdx.x / LPR % J, r = blockIdx.y * RPB + threadIdx.x / (LPR * J);
  const int request = cut.pair / A.Hkv, hk = cut.pair % A.Hkv;
  const int n_sh =
      A.slots_sh && own_begin(list_len(A, request), A.B, A.shared) > 0 ? A.slots_sh : 0;
  const int n = r < R ? n_sh + max(cut.slots, 1) : 0;
  const int64_t rows = (int64_t)A.N * A.B * A.Hq;
  const int64_t token = (int64_t)request * A.B + r / A.G;
  const int hq = hk * A.G + r % A.G;
  const int64_t row = token * A.Hq + hq;
  Joined all{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = group; s0 < n; s0 += 4 * J) {  // four slots' loads in flight
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = min(s0 + j * J, n - 1), own = s - n_sh;
      const bool part = own >= 0 && cut.slots;
      const int64_t from = part ? (own == 0 ? cut.slot : 2 * ((int64_t)cut.part + own)) * R + r
                                : (own >= 0 ? A.slots_sh : s) * rows + row;
      ml[j] = (part ? F.pml : A.pml)[from];
      x[j] = *reinterpret_cast<const float4*>((part ? F.po : A.po) + from * D + d);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s0 + j * J < n && ml[j].y != 0.f) all.add(ml[j].x, ml[j].y, x[j]);
  }
  __shared__ Joined s_part[RPB * J * LPR];
  s_part[threadIdx.x] = all;
  __syncthreads();
  if (group || r >= R) return;
#pragma unroll 8
  for (int g = 1; g < J; ++g) {
    const Joined& p = s_part[threadIdx.x + g * LPR];
    if (p.l != 0.f) all.add(p.m, p.l, p.o);
  }
  const float inv = all.l == 0.f ? 0.f : 1.f / all.l;
  uint2 w;
  w.x = pack2<F16>(all.o.x * inv, all.o.y * inv);
  w.y = pack2<F16>(all.o.z * inv, all.o.w * inv);
  *reinterpret_cast<uint2*>(A.out + token * A.out_ld + (int64_t)hq * D + d) = w;
  if (A.lse && d == 0)
    A.lse[row] = all.l == 0.f ? -INFINITY : (all.m + log2f(all.l)) * 0.69314718056f;
}

template <bool F16, int D> hipError_t launch_few(Few F, bool wide, bool beside, hipStream_t s) {
  Args& A = F.a;
  const int64_t shared = (int64_t)A.Hkv * A.tiles_sh * A.s_sh;
  A.slots_sh = A.s_sh;
  A.step_own = narrow_step(D, true);
  A.direct = false;
  const int R = A.B * A.G;
  const int64_t own = ceil_div(F.parts ? F.parts : (int64_t)A.N * A.Hkv, 4 / F.waves);
  const bool one = few_row_tiles(D, R) == 1;
  if (beside) {
    const dim3 grid((unsigned)(shared + own));
    if constexpr (D != 256) {
      if (one)
        hipLaunchKernelGGL((beside_kernel<F16, D, 1>), grid, dim3(256), 0, s, F);
      else
        hipLaunchKernelGGL((beside_kernel<F16, D, 2>), grid, dim3(256), 0, s, F);
    }
  } else {
    if (shared > 0) {
      if constexpr (D == 128)
        if (wide)
          hipLaunchKernelGGL((attend_kernel<F16, D, kWide, kWideStep, true>), dim3((unsigned)shared),
                             dim3(kWide * 64), 0, s, A);
      if (!wide)
        hipLaunchKernelGGL((attend_kernel<F16, D, kNarrow, narrow_step(D, true), true>),
                           dim3((unsigned)shared), dim3(kNarrow * 64), 0, s, A);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (one)
      hipLaunchKernelGGL((few_kernel<F16, D, 1>), dim3((unsigned)own), dim3(256), 0, s, F);
    else if constexpr (D != 256)
      hipLaunchKernelGGL((few_kernel<F16, D, 2>), dim3((unsigned)own), dim3(256), 0, s, F);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (F.parts == 0 && shared == 0)) return e;
  const int64_t joined = F.parts == 0 || F.by_pair ? (int64_t)A.N * A.Hkv : F.parts;
  // few rows may have many slots each
  const int64_t tiles = ceil_div((int64_t)A.ld << A.shift, kFewTile);
  if (joined * R <= kCUs && tiles / F.least > 32) {
    hipLaunchKernelGGL((join_kernel<F16, D, 4096 / D>), dim3((unsigned)joined, (unsigned)R), dim3(1024),
                       0, s, F);
  } else if (joined * R <= 8 * kCUs) {
    hipLaunchKernelGGL((join_kernel<F16, D, 1024 / D>), dim3((unsigned)joined, (unsigned)R), dim3(256),
                       0, s, F);
  } else {
    constexpr int J = 2, RPB = 1024 / (D * J);
    hipLaunchKernelGGL((join_kernel<F16, D, J>), dim3((unsigned)joined, (unsigned)ceil_div(R, RPB)),
                       dim3(256), 0, s, F);
  }
  return hipGetLastError();
}

}  // namespace

size_t few_scratch_bytes(const xpress_cache& c, int N, int B, int Hq) {
  const int R = B * (Hq / c.Hkv);
  if (R > kFewRows4) return 0;
  const size_t parts = few_parts(c.D, R), pairs = (size_t)std::min(N, kFewRequests) * c.Hkv;
  return parts * 2 * R * (c.D * sizeof(float) + sizeof(float2)) + std::max(parts, pairs) * sizeof(Cut);
}

hipError_t launch_block_attention4(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                   const int32_t* seq, int N, int B, int Hq, float scale, int shared,
                                   void* out, int64_t out_ld, float* lse, void* ws, hipStream_t s) {
  shared = shared / kTile * kTile;
  const AttendPlan p = plan_of(c, N, B, Hq, shared);
  Args A = args_of(c, p, layer, q, q_ld, seq, N, B, Hq, scale, shared, out, out_ld, lse, ws);
  const bool f16 = value_type(c) == XPRESS_F16;
  const int R = B * A.G;
  if (!few_rows(c, N, R, shared)) return launch_values<true>(A, c.D, f16, p.wide, s);
  Few F{A, 0, 2, few_waves(c.D, R), false, nullptr, nullptr, nullptr};
  const bool beside = p.s_sh && !p.wide && c.D != 256;
  if (N <= kFewRequests) {
    const int items = c.Hkv * p.tiles_sh * p.s_sh;
    F.parts = few_parts(c.D, R);
    if (beside)
      F.parts = 4 / F.waves * std::max(kCUs, kCUs * narrow_per_cu(c.D) - items);
    F.by_pair = p.s_sh || N * c.Hkv <= F.parts;
  }
  // the shared part's slots and one of every row, then the parts' (attention_scratch_bytes has room)
  const size_t rows = (size_t)N * B * Hq, slots = rows * (p.s_sh ? p.s_sh + 1 : 0);
  F.a.po = static_cast<float*>(ws);
  F.a.pml = reinterpret_cast<float2*>(F.a.po + slots * c.D);
  F.po = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                  up16(slots * (c.D * sizeof(float) + sizeof(float2))));
  F.cut = reinterpret_cast<Cut*>(F.po + 2 * (size_t)F.parts * R * c.D);
  const size_t cuts = F.by_pair ? (size_t)N * c.Hkv : F.parts;
  F.pml = reinterpret_cast<float2*>(F.cut + (F.parts ? cuts : 0));
  switch (c.D) {
    case 64:
      return f16 ? launch_few<true, 64>(F, p.wide, beside, s)
                 : launch_few<false, 64>(F, p.wide, beside, s);
    case 128:
      return f16 ? launch_few<true, 128>(F, p.wide, beside, s)
                 : launch_few<false, 128>(F, p.wide, beside, s);
    default:
      return f16 ? launch_few<true, 256>(F, p.wide, beside, s)
                 : launch_few<false, 256>(F, p.wide, beside, s);
  }
}

}  // namespace xpress
