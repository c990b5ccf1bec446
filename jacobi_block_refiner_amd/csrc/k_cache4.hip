// Tokens written into a cache of 4 bits, and tokens of a cache read back (gfx950).
//
// Both go through the cache by tiles of 16 tokens of a row: a workgroup takes one tile of positions of
// one row, K or V, and its heads in steps of 256 pieces of 8 channels, a thread each. K's bytes lie as
// the pieces do. V's lie by pairs of channels and four tokens: between a piece (a token's four pairs) and
// a word (a pair's four tokens) the bytes pass through LDS, so that both sides are read and written in
// whole lines. (A thread with a piece of its own and V's bytes one by one took 128 us instead of 77 for
// 8 x 8192 tokens of 8 heads of 128 read, whose bytes a copy passes in 65 to 71.)
#include "serve.hpp"
#include "cache_mx4.hpp"
#include "xpress_common.hpp"

#include <type_traits>

namespace xpress {

namespace {

struct Lines {
  const int32_t *table, *len, *seq;
  int rows, ld, n_pages, shift, N, B, Hkv;
  int64_t head_bytes;  // of a head's part of a page
  int tiles;           // of an entry of the list
  int steps, per;      // of 256 pieces in a tile of all heads; of a workgroup
};

// The tile of positions of this workgroup, and what of it the call is about.
struct Tile {
  int entry, row, len;
  int64_t start, pos;  // of the call's first token of the row; of the tile's
  int id;              // page (clamped; -1: none)
};

__device__ __forceinline__ Tile tile_of(const Lines& L, const int32_t* first) {
  Tile t;
  t.entry = blockIdx.x / (unsigned)L.tiles;
  const int r = L.seq ? L.seq[t.entry] : t.entry;
  t.row = (unsigned)r < (unsigned)L.rows ? r : -1;
  t.len = t.row < 0 ? 0 : clamp_len(L.len[t.row], L.ld, L.shift);
  t.start = first ? (int64_t)first[t.entry] : (int64_t)t.len - L.B;
  t.pos = ((t.start >> 4) + blockIdx.x % (unsigned)L.tiles) << 4;
  t.id = -1;
  if (t.pos >= 0 && t.pos < t.len) t.id = L.table[(int64_t)t.row * L.ld + (t.pos >> L.shift)];
  return t;
}
// Token of the call at position `pos`, or -1.
__device__ __forceinline__ int64_t token_at(const Lines& L, const Tile& t, int64_t pos) {
  const int64_t b = pos - t.start;
  return b >= 0 && b < L.B ? (int64_t)t.entry * L.B + b : -1;
}

template <bool F16> __device__ __forceinline__ float2 two(uint32_t u) {
  if constexpr (F16) {
    const mx4_f16x2 h = __builtin_bit_cast(mx4_f16x2, u);
    return make_float2((float)h.x, (float)h.y);
  } else {
    return make_float2(bf16_lo(u), bf16_hi(u));
  }
}

// Where a thread's piece lies in a step: head, token of the tile, channel; and its word of V, pairs i of
// group g of the tokens 4q...
template <int D> struct Place {
  int head, token, c, q, i, g;
  __device__ __forceinline__ Place(int step) {
    const int u = step * 256 + threadIdx.x, w = u % (2 * D);
    head = u / (2 * D);
    token = w / (D / 8);
    c = w % (D / 8) * 8;
    q = w / (D / 2);
    i = w / (D / 32) % 16;
    g = w % (D / 32);
  }
  // The thread of this step that has the piece of channels 32 g + 8 p.. of a token.
  static __device__ __forceinline__ int piece_thread(int head, int token, int g, int p) {
    return (head * 2 * D + token * (D / 8) + g * 4 + p) % 256;
  }
  // The thread that has the word of pair i of group g of a token's four.
  static __device__ __forceinline__ int word_thread(int head, int token, int g, int i) {
    return (head * 2 * D + (token / 4 * 16 + i) * (D / 32) + g) % 256;
  }
};

// The four threads of a group share its scale; NaN counts as 0. Bound by latency for a few tokens (32 rows
// of 16 tokens 3.3 us) and by HBM for many (8192 tokens 14 us). Loads of two or four steps ahead changed
// nothing: other workgroups of the CU fill the time.
template <bool F16, int D>
__global__ __launch_bounds__(256) void append4_kernel(Lines L, const int32_t* lacking, uint8_t* k,
                                                      uint8_t* v, const uint16_t* k_new,
                                                      const uint16_t* v_new, int64_t ld_new) {
  __shared__ uint32_t s_code[2][256];
  const int no = lacking ? *lacking : 0;
  const Tile t = tile_of(L, nullptr);
  if (no || !page_ok(t.id, L.n_pages)) return;
  const bool is_v = blockIdx.y & 1;
  const uint16_t* fresh = is_v ? v_new : k_new;
  uint8_t* page = (is_v ? v : k) + (int64_t)t.id * L.Hkv * L.head_bytes +
                  ((t.pos & ((1 << L.shift) - 1)) >> 4) * mx4_tile_bytes(D);
  const int step0 = (blockIdx.y >> 1) * L.per, step1 = min(step0 + L.per, L.steps);
  for (int step = step0; step < step1; ++step) {
    const Place<D> at(step);
    const bool is_head = at.head < L.Hkv;
    const int64_t token = is_head ? token_at(L, t, t.pos + at.token) : -1;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (token >= 0) x = *reinterpret_cast<const uint4*>(fresh + token * ld_new + at.head * D + at.c);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    float y[8], top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 w = two<F16>(u[j / 2]);
      const float z = j % 2 ? w.y : w.x;
      y[j] = z != z ? 0.f : z;
      top = fmaxf(top, fabsf(y[j]));
    }
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    const int s = mx4_scale_byte(__float_as_uint(top), F16);
    const float scale = __uint_as_float((uint32_t)s << 23);
    uint32_t code = 0;
    code = mx4_code<0>(code, y[0], y[1], scale);
    code = mx4_code<1>(code, y[2], y[3], scale);
    code = mx4_code<2>(code, y[4], y[5], scale);
    code = mx4_code<3>(code, y[6], y[7], scale);
    uint8_t* tile = page + at.head * L.head_bytes;
    if (token >= 0 && at.c % 32 == 0)
      tile[is_v ? mx4_v_scale(D, at.token, at.c / 32) : mx4_k_scale(D, at.token, at.c / 32)] = (uint8_t)s;
    if (!is_v) {
      if (token >= 0) *reinterpret_cast<uint32_t*>(tile + mx4_k_code(D, at.token, at.c)) = code;
      continue;
    }
    // (two buffers: the words of two steps ago were read before the last meeting)
    s_code[step & 1][threadIdx.x] = code;
    __syncthreads();
    if (!is_head) continue;
    uint32_t word = 0;
    int inside = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int piece = Place<D>::piece_thread(at.head, 4 * at.q + j, at.g, at.i / 4);
      word |= (s_code[step & 1][piece] >> at.i % 4 * 8 & 255) << 8 * j;
      inside |= (token_at(L, t, t.pos + 4 * at.q + j) >= 0) << j;
    }
    uint8_t* to = tile + mx4_v_code(D, 4 * at.q, 32 * at.g + 2 * at.i);
    if (inside == 15) {
      *reinterpret_cast<uint32_t*>(to) = word;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (inside >> j & 1) to[j] = (uint8_t)(word >> 8 * j);
    }
  }
}

// Tokens outside a row are 0. Bound by HBM for many tokens.
constexpr int kAhead = 4;  // steps whose loads are in flight (two: 82 us instead of 77)

template <bool F16, int D>
__global__ __launch_bounds__(256) void read4_kernel(Lines L, const uint8_t* k, const uint8_t* v,
                                                    const int32_t* first, uint16_t* k_out,
                                                    uint16_t* v_out, int64_t ld_out) {
  __shared__ uint32_t s_code[2][256];
  const Tile t = tile_of(L, first);
  const bool is_v = blockIdx.y & 1, held = t.pos >= 0 && t.pos < t.len;
  uint16_t* to = is_v ? v_out : k_out;
  const uint8_t* page = (is_v ? v : k) + (int64_t)clamp_page(t.id, L.n_pages) * L.Hkv * L.head_bytes +
                        ((t.pos & ((1 << L.shift) - 1)) >> 4) * mx4_tile_bytes(D);
  const int step0 = (blockIdx.y >> 1) * L.per, step1 = min(step0 + L.per, L.steps);
  for (int from = step0; from < step1; from += kAhead) {
    uint32_t code[kAhead], scale[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const Place<D> at(min(from + a, step1 - 1));
      const uint8_t* tile = page + min(at.head, L.Hkv - 1) * L.head_bytes;
      code[a] = scale[a] = 0;
      if (held) {
        code[a] = *reinterpret_cast<const uint32_t*>(
            tile + (is_v ? mx4_v_code(D, 4 * at.q, 32 * at.g + 2 * at.i) : mx4_k_code(D, at.token, at.c)));
        scale[a] = tile[is_v ? mx4_v_scale(D, at.token, at.c / 32) : mx4_k_scale(D, at.token, at.c / 32)];
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int step = from + a;
      if (step >= step1) break;
      const Place<D> at(step);
      uint32_t word = code[a];
      if (is_v) {
        s_code[a & 1][threadIdx.x] = word;
        __syncthreads();
        word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int from_thread =
              Place<D>::word_thread(at.head, at.token, at.c / 32, at.c % 32 / 2 + j);
          word |= (s_code[a & 1][from_thread] >> at.token % 4 * 8 & 255) << 8 * j;
        }
      }
      const int64_t pos = t.pos + at.token, token = token_at(L, t, pos);
      if (at.head >= L.Hkv || token < 0) continue;
      const float s = mx4_scale<0>(scale[a]);
      uint4 out = make_uint4(mx4_pair<F16, 0>(word, s), mx4_pair<F16, 1>(word, s),
                             mx4_pair<F16, 2>(word, s), mx4_pair<F16, 3>(word, s));
      if (pos < 0 || pos >= t.len) out = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(to + token * ld_out + at.head * D + at.c) = out;
    }
  }
}

// Of a cache of 16 bits: copies, at the rate of one (8 x 8192 tokens of 8 heads of 128, 537 MB, 102 us, 5.2
// TB/s; 8191 tokens 11.8 us; 16 tokens 2.5).
template <int D>
__global__ __launch_bounds__(256) void read16_kernel(Lines L, const uint8_t* k, const uint8_t* v,
                                                     const int32_t* first, uint16_t* k_out,
                                                     uint16_t* v_out, int64_t ld_out) {
  const Tile t = tile_of(L, first);
  const bool is_v = blockIdx.y & 1;
  const uint8_t* page = (is_v ? v : k) + (int64_t)clamp_page(t.id, L.n_pages) * L.Hkv * L.head_bytes;
  const int step0 = (blockIdx.y >> 1) * L.per, step1 = min(step0 + L.per, L.steps);
#pragma unroll 4
  for (int step = step0; step < step1; ++step) {
    const Place<D> at(step);
    const int64_t pos = t.pos + at.token, token = token_at(L, t, pos);
    if (at.head >= L.Hkv || token < 0) continue;
    uint4 out = make_uint4(0, 0, 0, 0);
    if (pos >= 0 && pos < t.len)
      out = *reinterpret_cast<const uint4*>(page + at.head * L.head_bytes +
                                            ((pos & ((1 << L.shift) - 1)) * D + at.c) * 2);
    *reinterpret_cast<uint4*>((is_v ? v_out : k_out) + token * ld_out + at.head * D + at.c) = out;
  }
}

Lines lines(const xpress_cache& c, const int32_t* seq, int N, int B, dim3* grid) {
  const int shift = __builtin_ctz((unsigned)c.page), steps = (c.Hkv * 2 * c.D + 255) / 256;
  const int64_t tiles = ((int64_t)B + 30) / 16;  // that B tokens can touch
  // a workgroup takes all heads of a tile where there are tiles enough to fill the card
  int per = 1;
  while (per < steps && tiles * N * (steps / per) > 2048) per *= 2;
  *grid = dim3((unsigned)(tiles * N), 2 * (unsigned)((steps + per - 1) / per));
  return Lines{c.table, c.len, seq,   c.rows, c.table_ld, c.n_pages, shift,
               N,       B,     c.Hkv, cache_page_bytes(c) / c.Hkv, (int)tiles, steps, per};
}

template <class F> hipError_t for_heads(int D, F&& f) {
  switch (D) {
    case 64: f(std::integral_constant<int, 64>{}); break;
    case 128: f(std::integral_constant<int, 128>{}); break;
    default: f(std::integral_constant<int, 256>{});
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append4(const xpress_cache& c, const int32_t* lacking, int layer,
                                const void* k_new, const void* v_new, int64_t ld_new,
                                const int32_t* seq, int N, int B, hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * cache_page_bytes(c);
  dim3 grid;
  const Lines L = lines(c, seq, N, B, &grid);
  return for_heads(c.D, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const auto kernel =
        value_type(c) == XPRESS_F16 ? append4_kernel<true, D> : append4_kernel<false, D>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, L, lacking, static_cast<uint8_t*>(c.k) + at,
                       static_cast<uint8_t*>(c.v) + at, static_cast<const uint16_t*>(k_new),
                       static_cast<const uint16_t*>(v_new), ld_new);
  });
}

hipError_t launch_cache_read(const xpress_cache& c, int layer, const int32_t* first, void* k_out,
                             void* v_out, int64_t ld_out, const int32_t* seq, int N, int B,
                             hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * cache_page_bytes(c);
  dim3 grid;
  const Lines L = lines(c, seq, N, B, &grid);
  return for_heads(c.D, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const auto kernel = !cache_in_4_bits(c)           ? read16_kernel<D>
                        : value_type(c) == XPRESS_F16 ? read4_kernel<true, D>
                                                      : read4_kernel<false, D>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, L, static_cast<const uint8_t*>(c.k) + at,
                       static_cast<const uint8_t*>(c.v) + at, first, static_cast<uint16_t*>(k_out),
                       static_cast<uint16_t*>(v_out), ld_out);
  });
}

}  // namespace xpress
