// Rows of logits of any type and alignment, read in 16-byte pieces (gfx950).
#pragma once

#include "xpress_common.hpp"

namespace xpress {

namespace {

template <class T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
template <> __device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
template <> __device__ __forceinline__ float to_f32(float x) { return x; }

template <class T> __device__ __forceinline__ T lowest();  // -inf
template <> __device__ __forceinline__ uint16_t lowest() { return 0xff80; }
template <> __device__ __forceinline__ _Float16 lowest() { return (_Float16)-INFINITY; }
template <> __device__ __forceinline__ float lowest() { return -INFINITY; }

// 16 bytes of a row.
template <class T> struct Piece {
  T e[16 / sizeof(T)];
  __device__ __forceinline__ float operator[](int i) const { return to_f32<T>(e[i]); }
};

// Chunks of a row: its first 16-byte boundary at or before the row begins chunk 0, so that all but
// the row's two ends are read in whole 16-byte pieces whatever the row's alignment.
template <class T> struct Row {
  static constexpr int E = 16 / sizeof(T);  // ids of a piece
  const T* x;
  int V, off;
  __device__ Row(const T* x_, int V_) : x(x_), V(V_), off((int)((uintptr_t)x_ % 16 / sizeof(T))) {}
  __device__ __forceinline__ int first(int64_t j) const { return (int)(j * E - off); }
  // The logits of piece j (ids outside the row: -inf).
  __device__ __forceinline__ Piece<T> load(int64_t j) const {
    const int64_t v0 = j * E - off;
    if (v0 >= 0 && v0 + E <= V)
      return __builtin_bit_cast(Piece<T>, *reinterpret_cast<const uint4*>(x + v0));
    Piece<T> p;
#pragma unroll
    for (int i = 0; i < E; ++i) p.e[i] = v0 + i >= 0 && v0 + i < V ? x[v0 + i] : lowest<T>();
    return p;
  }
};

}  // namespace
}  // namespace xpress
