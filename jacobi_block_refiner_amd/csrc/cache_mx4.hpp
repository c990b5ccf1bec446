// A paged cache in 4 bits: where its codes and scales lie, and how they turn into 16-bit values and
// back (gfx950 converts pairs in one instruction, at the rate of an addition).
//
// 16 tokens of a page and head are a tile: 8 D bytes of codes, then D / 2 of scales, one for 32
// channels of a token. K lies as a row a token. V lies as the second product takes it: the lane that
// holds a pair of channels of each group and four tokens finds its bytes in one piece.
#pragma once

#include "cache_index.hpp"

namespace xpress {

XP_HD constexpr int mx4_tile_bytes(int D) { return 17 * D / 2; }
// Bytes of one side of a head's tiles of a page of 2^shift tokens.
XP_HD constexpr int64_t mx4_tiles_bytes(int D, int shift) {
  return (int64_t)mx4_tile_bytes(D) << (shift - 4);
}
// Bytes inside a tile: channels c and c + 1 (c even) of token t, and the scale of group g.
XP_HD constexpr int mx4_k_code(int D, int t, int c) { return t * (D / 2) + c / 2; }
XP_HD constexpr int mx4_k_scale(int D, int t, int g) { return 8 * D + t * (D / 32) + g; }
XP_HD constexpr int mx4_v_code(int D, int t, int c) {
  return ((t / 4 * 16 + c % 32 / 2) * (D / 32) + c / 32) * 4 + t % 4;
}
XP_HD constexpr int mx4_v_scale(int D, int t, int g) {
  return 8 * D + (t / 4 * (D / 32) + g) * 4 + t % 4;
}

// Exponents (with the byte's offset of 127) of the scales that an append writes: the smallest turns
// every 16-bit subnormal into 0 or, for fp16, into itself; with the largest, 6 times it is finite.
XP_HD constexpr int mx4_lowest(bool f16) { return f16 ? 127 - 23 : 127 - 123; }
XP_HD constexpr int mx4_highest(bool f16) { return f16 ? 127 + 13 : 127 + 125; }

// The scale's byte for a group whose largest magnitude has these bits (32-bit float, no NaN): 4 to 6
// times the scale hold it, and up to 7 times, which 6 is as near to as 8 would be.
XP_HD int mx4_scale_byte(uint32_t top_bits, bool f16) {
  const int e = (int)((top_bits + (1u << 21)) >> 23) - 2;
  return e < mx4_lowest(f16) ? mx4_lowest(f16) : e > mx4_highest(f16) ? mx4_highest(f16) : e;
}

#if defined(__HIPCC__)

typedef _Float16 mx4_f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx4_bf16x2 __attribute__((ext_vector_type(2)));

// Byte I of four scales as a factor. (The conversions take the exponent alone; the bits round it are
// of no consequence.)
template <int I> __device__ __forceinline__ float mx4_scale(uint32_t four) {
  return __uint_as_float(I == 3 ? four >> 1 : four << (23 - 8 * I));
}

// The two values of byte I of eight codes, 16 bits each, the low half's in the low bits. Exact.
template <bool F16, int I> __device__ __forceinline__ uint32_t mx4_pair(uint32_t codes, float scale) {
  if constexpr (F16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, I));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
}

// Byte I of `codes` from two values: to nearest, ties to the even code, beyond 6 scales 6.
template <int I>
__device__ __forceinline__ uint32_t mx4_code(uint32_t codes, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, scale, I);
}

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302);
}

#endif

}  // namespace xpress
