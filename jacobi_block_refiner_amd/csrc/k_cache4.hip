// Tokens written into a cache of 4 bits, and tokens of a cache read back (gfx950).
#include "serve.hpp"
#include "cache_mx4.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

// What a thread's piece of 8 channels of a token needs of the cache.
struct Lines {
  const int32_t *table, *len, *seq;
  int rows, ld, n_pages, shift, N, B, Hkv, D;
  int64_t head_bytes;  // of a head's part of a page
};

Lines lines(const xpress_cache& c, const int32_t* seq, int N, int B) {
  const int shift = __builtin_ctz((unsigned)c.page);
  return Lines{c.table, c.len, seq, c.rows, c.table_ld, c.n_pages, shift, N, B, c.Hkv, c.D,
               cache_page_bytes(c) / c.Hkv};
}

// Row of list entry e, or -1.
__device__ __forceinline__ int row_of(const Lines& L, int e) {
  const int r = L.seq ? L.seq[e] : e;
  return (unsigned)r < (unsigned)L.rows ? r : -1;
}

template <bool F16> __device__ __forceinline__ float2 two(uint32_t u) {
  if constexpr (F16) {
    const mx4_f16x2 h = __builtin_bit_cast(mx4_f16x2, u);
    return make_float2((float)h.x, (float)h.y);
  } else {
    return make_float2(bf16_lo(u), bf16_hi(u));
  }
}

// A thread 8 channels of a token; the four threads of a group share its scale. NaN counts as 0.
template <bool F16>
__global__ __launch_bounds__(256) void append4_kernel(Lines L, const int32_t* lacking, uint8_t* k,
                                                      uint8_t* v, const uint16_t* k_new,
                                                      const uint16_t* v_new, int64_t ld_new) {
  const unsigned per = L.Hkv * L.D / 8;
  const unsigned i = blockIdx.x * 256u + threadIdx.x;  // (below 2^31: N*B*Hkv is below 2^26)
  if (i >= (unsigned)L.N * L.B * per) return;
  const unsigned token = i / per, piece = i % per;
  const int e = token / (unsigned)L.B, b = token % (unsigned)L.B;
  const uint4 x = *reinterpret_cast<const uint4*>((blockIdx.y ? v_new : k_new) +
                                                  (int64_t)token * ld_new + piece * 8);
  const int no = lacking ? *lacking : 0;
  const int r = row_of(L, e);
  if (r < 0 || no) return;
  const int pos = in_sight(clamp_len(L.len[r], L.ld, L.shift), L.B, b) - 1;
  if (pos < 0) return;
  const int id = L.table[(int64_t)r * L.ld + (pos >> L.shift)];
  if (!page_ok(id, L.n_pages)) return;
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
  const int h = piece * 8 / (unsigned)L.D, c = piece * 8 % (unsigned)L.D, t = pos & 15;
  const int line = pos & ((1 << L.shift) - 1);
  uint8_t* tile = (blockIdx.y ? v : k) + ((int64_t)id * L.Hkv + h) * L.head_bytes +
                  (line >> 4) * mx4_tile_bytes(L.D);
  if (blockIdx.y) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      tile[mx4_v_code(L.D, t, c + 2 * j)] = (uint8_t)(code >> 8 * j);
    if (c % 32 == 0) tile[mx4_v_scale(L.D, t, c / 32)] = (uint8_t)s;
  } else {
    *reinterpret_cast<uint32_t*>(tile + mx4_k_code(L.D, t, c)) = code;
    if (c % 32 == 0) tile[mx4_k_scale(L.D, t, c / 32)] = (uint8_t)s;
  }
}

// The same pieces the other way; tokens outside a row are 0.
template <bool F16, bool MX4>
__global__ __launch_bounds__(256) void read_kernel(Lines L, const uint8_t* k, const uint8_t* v,
                                                   const int32_t* first, uint16_t* k_out,
                                                   uint16_t* v_out, int64_t ld_out) {
  const unsigned per = L.Hkv * L.D / 8;
  const unsigned i = blockIdx.x * 256u + threadIdx.x;
  if (i >= (unsigned)L.N * L.B * per) return;
  const unsigned token = i / per, piece = i % per;
  const int e = token / (unsigned)L.B, b = token % (unsigned)L.B;
  uint4 out = make_uint4(0, 0, 0, 0);
  const int r = row_of(L, e);
  if (r >= 0) {
    const int len = clamp_len(L.len[r], L.ld, L.shift);
    const int64_t pos = (first ? (int64_t)first[e] : (int64_t)len - L.B) + b;
    if (pos >= 0 && pos < len) {
      const int id = clamp_page(L.table[(int64_t)r * L.ld + (pos >> L.shift)], L.n_pages);
      const int h = piece * 8 / (unsigned)L.D, c = piece * 8 % (unsigned)L.D, t = pos & 15;
      const int line = (int)pos & ((1 << L.shift) - 1);
      const uint8_t* head = (blockIdx.y ? v : k) + ((int64_t)id * L.Hkv + h) * L.head_bytes;
      if constexpr (!MX4) {
        out = *reinterpret_cast<const uint4*>(head + ((int64_t)line * L.D + c) * 2);
      } else {
        const uint8_t* tile = head + (line >> 4) * mx4_tile_bytes(L.D);
        uint32_t code = 0, s;
        if (blockIdx.y) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            code |= (uint32_t)tile[mx4_v_code(L.D, t, c + 2 * j)] << 8 * j;
          s = tile[mx4_v_scale(L.D, t, c / 32)];
        } else {
          code = *reinterpret_cast<const uint32_t*>(tile + mx4_k_code(L.D, t, c));
          s = tile[mx4_k_scale(L.D, t, c / 32)];
        }
        const float scale = mx4_scale<0>(s);
        out = make_uint4(mx4_pair<F16, 0>(code, scale), mx4_pair<F16, 1>(code, scale),
                         mx4_pair<F16, 2>(code, scale), mx4_pair<F16, 3>(code, scale));
      }
    }
  }
  *reinterpret_cast<uint4*>((blockIdx.y ? v_out : k_out) + (int64_t)token * ld_out + piece * 8) = out;
}

dim3 pieces_grid(const xpress_cache& c, int N, int B) {
  const int64_t n = (int64_t)N * B * (c.Hkv * c.D / 8);
  return dim3((unsigned)((n + 255) / 256), 2);
}

}  // namespace

hipError_t launch_cache_append4(const xpress_cache& c, const int32_t* lacking, int layer,
                                const void* k_new, const void* v_new, int64_t ld_new,
                                const int32_t* seq, int N, int B, hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * cache_page_bytes(c);
  const auto kernel = value_type(c) == XPRESS_F16 ? append4_kernel<true> : append4_kernel<false>;
  hipLaunchKernelGGL(kernel, pieces_grid(c, N, B), dim3(256), 0, s, lines(c, seq, N, B), lacking,
                     static_cast<uint8_t*>(c.k) + at, static_cast<uint8_t*>(c.v) + at,
                     static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new), ld_new);
  return hipGetLastError();
}

hipError_t launch_cache_read(const xpress_cache& c, int layer, const int32_t* first, void* k_out,
                             void* v_out, int64_t ld_out, const int32_t* seq, int N, int B,
                             hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * cache_page_bytes(c);
  const auto kernel = !cache_in_4_bits(c)              ? read_kernel<false, false>
                      : value_type(c) == XPRESS_F16 ? read_kernel<true, true>
                                                    : read_kernel<false, true>;
  hipLaunchKernelGGL(kernel, pieces_grid(c, N, B), dim3(256), 0, s, lines(c, seq, N, B),
                     static_cast<const uint8_t*>(c.k) + at, static_cast<const uint8_t*>(c.v) + at,
                     first, static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out), ld_out);
  return hipGetLastError();
}

}  // namespace xpress
