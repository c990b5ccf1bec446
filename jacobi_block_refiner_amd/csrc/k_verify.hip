// Verification of drafted blocks against the target's logits (gfx950).
//
// A row's weights are w(v) = 2^((x_v - m) c), c = log2(e) / T, m the row's maximum. Rows are cut into
// chunks of kChunk ids; stats_kernel leaves each chunk's maximum, its id and the sum of its weights
// (relative to the chunk's own maximum), and the last chunk of a row joins them and tests the row's
// draft. For the one row of each block where a token is drawn, sums_kernel forms the chunks' sums
// once more in 64 bits (left_kernel what the drafts' probabilities leave of them), and the block's
// last chunk finds the token: first the chunk whose running sum passes u * total, then the id in it.
//
// Precision. A draw from V ids has borders 1/V apart: weights that are off by 2^-24 would shift a
// border of a flat distribution of 151,936 ids by several percent of their distance and change that
// share of the tokens; at 2e-12 it is one in 10^6. A test u q S < w has one border and takes 32-bit
// weights; where the two sides are within 1e-5 of each other the row is summed anew in 64 bits.
// (64 bits for all rows: 74 against 37 us at 512 rows of 151,936 ids.)
//
// Rows after a block's first refusal do not matter. Chunks go by slot, all blocks' first slots
// first, and a chunk whose block is known to have been refused earlier returns at once. How many
// do depends on timing; the result does not, since rows up to the first refusal are never left out.
#include "serve.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // ids of a chunk: 32 a thread

template <class T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
template <> __device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
template <> __device__ __forceinline__ float to_f32(float x) { return x; }

// 2^t for t <= 0 (NaN and below -1075: 0), relative error 2.2e-12: 2^f = 1 + f p(f) for the fraction
// f in [-1/2, 1/2], p fitted at Chebyshev nodes; adding 3 * 2^51 rounds t to an integer that stands
// in the sum's low word.
__device__ __forceinline__ double pow2(double t) {
  const double c = fmax(t, -1100.0);
  const double big = c + 6755399441055744.0;
  const double f = c - (big - 6755399441055744.0);
  double p = 1.3255215184459522e-06;
  p = fma(p, f, 1.530370229370019e-05);
  p = fma(p, f, 0.0001540345588901354);
  p = fma(p, f, 0.001333347846767389);
  p = fma(p, f, 0.009618129159364436);
  p = fma(p, f, 0.055504109063315425);
  p = fma(p, f, 0.24022650695813097);
  p = fma(p, f, 0.6931471805568313);
  p = fma(p, f, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)(uint32_t)(uint64_t)__double_as_longlong(big));
}

// A logit's weight relative to the maximum m: 0 for -inf and NaN; at m = +inf the ids that hold it
// share all.
__device__ __forceinline__ double weight(float x, float m, double c) {
  return pow2((x == m ? 0.0 : (double)x - (double)m) * c);
}

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

// What a chunk leaves: the sum of its weights relative to its maximum m, and the lowest id of m
// (INT_MAX where the chunk has no weight).
struct Part {
  double sum;
  float m;
  int arg;
};

struct Args {
  const void* logits;
  int64_t ld, q_ld;
  const int64_t* blk;
  const int32_t* draft_len;
  const void* q;
  uint32_t q_dtype;
  const float *temperature, *u;
  int N, B, V, chunks, draws;
  int64_t* out;
  int32_t *accepted, *drop;
  Part* part;     // [N*B, chunks]
  Part* row;      // [N*B]: the rows' own
  double* sums;   // [N, chunks]: the row of the draw (without a refused point draft)
  double* left;   // [N, chunks]: what is left of it beside the drafts' probabilities
  int32_t* done;  // [N*B]: chunks that are in
  int32_t* stop;  // [N]: first refused slot so far (B: none)
  int32_t* drawn; // [N]: chunks of the row of the draw that are in
};

// An element of q by its type code.
__device__ __forceinline__ float q_at(const Args& A, int64_t i) {
  if (A.q_dtype == XPRESS_BF16) return bf16_to_f32(static_cast<const uint16_t*>(A.q)[i]);
  if (A.q_dtype == XPRESS_F16) return (float)static_cast<const _Float16*>(A.q)[i];
  return static_cast<const float*>(A.q)[i];
}

// n of them, where they lie inside q's row and on a 16-byte boundary in whole 16-byte pieces.
template <int N> __device__ __forceinline__ void q_piece(const Args& A, int64_t row, int64_t v0, float (&q)[N]) {
  const int size = A.q_dtype == XPRESS_F32 ? 4 : 2;
  const char* at = static_cast<const char*>(A.q) + (row + v0) * size;
  if (v0 >= 0 && v0 + N <= A.V && ((uintptr_t)at & 15) == 0 && N * size % 16 == 0) {
    if (size == 4) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        *reinterpret_cast<float4*>(q + 4 * i) = reinterpret_cast<const float4*>(at)[i];
    } else if constexpr (N == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(at);
      const auto b = __builtin_bit_cast(Piece<uint16_t>, u);
      const auto h = __builtin_bit_cast(Piece<_Float16>, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = A.q_dtype == XPRESS_BF16 ? b[i] : h[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = v0 + i >= 0 && v0 + i < A.V ? q_at(A, row + v0 + i) : 0.f;
}

__device__ __forceinline__ int limit_of(const Args& A, int n) {
  return A.draft_len ? min(max(A.draft_len[n], 0), A.B - 1) : A.B - 1;
}
// log2(e) / T, or 0 for greedy (an infinite T: every finite logit weighs the same).
__device__ __forceinline__ double scale_of(const Args& A, int n) {
  const float t = A.temperature ? A.temperature[n] : 0.f;
  return t > 0.f ? fmax(1.4426950408889634 / (double)t, 1e-300) : 0.0;
}

// Chunks travel between workgroups of different XCDs: stores and loads at the card's scope, which
// neither leave a value in an L2 nor take one from it.
__device__ __forceinline__ void put(Part* at, const Part& p) {
  uint64_t* w = reinterpret_cast<uint64_t*>(at);
  const uint64_t lo = (uint64_t)__double_as_longlong(p.sum);
  const uint64_t hi = (uint64_t)__float_as_uint(p.m) | (uint64_t)(uint32_t)p.arg << 32;
  __hip_atomic_store(w, lo, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(w + 1, hi, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Part get(const Part* at) {
  const uint64_t* w = reinterpret_cast<const uint64_t*>(at);
  const uint64_t lo = __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t hi = __hip_atomic_load(w + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return Part{__longlong_as_double((int64_t)lo), __uint_as_float((uint32_t)hi), (int)(hi >> 32)};
}

// Counts a chunk in, after its stores: they go through the caches to the card's point of coherence,
// and the wait is for their acknowledgement. (A release at the card's scope also writes back the
// whole L2 of the XCD and an acquire empties it, once a chunk: 278 against 74 us at 512 rows of
// 151,936 ids.) Returns how many were in before. What the last chunk then reads with get() must not be
// read before the add has returned: the branch on its result keeps the loads behind it on the card,
// and the compiler, which may move relaxed loads above a relaxed add, is kept from it here.
__device__ __forceinline__ int count_in(int32_t* counter) {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  asm volatile("" ::: "memory");
  const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("" ::: "memory");
  return before;
}
__device__ __forceinline__ void put(double* at, double v) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(at), (uint64_t)__double_as_longlong(v),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get(const double* at) {
  return __longlong_as_double((int64_t)__hip_atomic_load(
      reinterpret_cast<const uint64_t*>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One chunk of one row. Bound by HBM: 16 KiB of bf16 a workgroup, eight workgroups a CU. 16 rows of
// 151,936 ids 9 us, 32 blocks of 16 rows 38, 256 blocks 125.
template <class T>
__global__ __launch_bounds__(kThreads, 8) void stats_kernel(Args A) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;
  const int c = blockIdx.x % A.chunks, y = blockIdx.x / A.chunks, t = threadIdx.x;
  const int n = y % A.N, s = y / A.N, limit = limit_of(A, n);
  if (s > limit) return;
  __shared__ int s_stop;  // one thread's look: the whole workgroup goes or stays
  if (t == 0) s_stop = __hip_atomic_load(A.stop + n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (s > s_stop) return;
  const int64_t r = (int64_t)n * A.B + s;
  const Row<T> row(static_cast<const T*>(A.logits) + r * A.ld, A.V);
  float x[K][E];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Piece<T> p = row.load((int64_t)c * (kChunk / E) + k * kThreads + t);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[k][e] = p[e];
      asm("" : "+v"(x[k][e]));  // (fp16: or both the halves and their values stay live, and spill)
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, x[k][e]);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const double scale = scale_of(A, n);
  const float c32 = (float)fmin(scale, 1e37);
  float sum = 0;
  int arg = INT_MAX;
  if (scale == 0.0) {
#pragma unroll
    for (int k = K - 1; k >= 0; --k)
#pragma unroll
      for (int e = E - 1; e >= 0; --e)
        if (x[k][e] == m) arg = row.first((int64_t)c * (kChunk / E) + k * kThreads + t) + e;
#pragma unroll
    for (int d = 32; d; d >>= 1) arg = min(arg, __shfl_xor(arg, d));
    if (m == -INFINITY) arg = INT_MAX;
  } else if (m > -INFINITY) {
    arg = 0;
    if (m == INFINITY) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) sum += x[k][e] == m ? 1.f : 0.f;
    } else {
      // (x - m first: near the maximum, where the weight is, the product then has no large terms
      // that cancel; the maximum with -1e30 turns NaN and -inf into no weight)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e)
          sum += __builtin_amdgcn_exp2f(fmaxf((x[k][e] - m) * c32, -1e30f));
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  }
  // The waves' parts go to the first wave; the others are done.
  __shared__ Part s_part[kThreads / 64];
  if ((t & 63) == 0) s_part[t >> 6] = Part{sum, m, arg};
  __syncthreads();
  if (t >= 64) return;
  Part p = t < kThreads / 64 ? s_part[t] : Part{0, -INFINITY, INT_MAX};
  {
    float top = p.m;
#pragma unroll
    for (int i = kThreads / 128; i; i >>= 1) top = fmaxf(top, __shfl_xor(top, i));
    float part = p.sum;
    if (p.m != top) {
      part = scale != 0.0 && top != INFINITY ? part * __builtin_amdgcn_exp2f(fmaxf((p.m - top) * c32, -1e30f)) : 0.f;
      p.arg = INT_MAX;
    }
#pragma unroll
    for (int i = kThreads / 128; i; i >>= 1) {
      part += __shfl_xor(part, i);
      p.arg = min(p.arg, __shfl_xor(p.arg, i));
    }
    p.m = top;
    p.sum = part;
  }
  int last = 0;
  if (t == 0) {
    put(A.part + r * A.chunks + c, p);
    last = count_in(A.done + r) == A.chunks - 1;
  }
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  // the row's last chunk: join them, test the draft
  int64_t d = s < limit ? A.blk[r + 1] : -1;
  if (d < 0 || d >= A.V) d = -1;
  double test = 0;  // u q
  if (scale != 0.0 && d >= 0)
    test = (double)A.u[r] * (A.q ? q_at(A, ((int64_t)n * (A.B - 1) + s) * A.q_ld + d) : 1.f);
  const Part* part = A.part + r * A.chunks;
  Part w{0, -INFINITY, INT_MAX};
  const Part mine = t < A.chunks ? get(part + t) : w;
  for (int i = t; i < A.chunks; i += 64) {
    const Part o = i == t ? mine : get(part + i);
    if (o.arg != INT_MAX) argmax_merge(w.m, w.arg, o.m, o.arg);
  }
#pragma unroll
  for (int x = 32; x; x >>= 1) argmax_merge(w.m, w.arg, __shfl_xor(w.m, x), __shfl_xor(w.arg, x));
  bool ok = false;
  if (w.arg != INT_MAX && d >= 0) {
    if (scale == 0.0) {
      ok = d == w.arg;
    } else {
      const double drafted = weight(to_f32<T>(row.x[d]), w.m, scale);
      double all = 0;
      for (int i = t; i < A.chunks; i += 64) {
        const Part o = i == t ? mine : get(part + i);
        if (o.arg != INT_MAX) all += o.sum * weight(o.m, w.m, scale);
      }
      all = wave_sum(all);
      if (fabs(test * all - drafted) <= 1e-5 * drafted) {
        all = 0;
        const int64_t pieces = ((int64_t)A.V + row.off + E - 1) / E;
#pragma unroll 1
        for (int64_t j = t; j < pieces; j += 64) {
          const Piece<T> y = row.load(j);
#pragma unroll
          for (int e = 0; e < E; ++e) all += weight(y[e], w.m, scale);
        }
        all = wave_sum(all);
      }
      ok = test * all < drafted;
    }
  }
  if (t == 0) {
    A.row[r] = w;
    if (s < limit && !ok) atomicMin(A.stop + n, s);
  }
}

// What a block's rows say.
struct Verdict {
  int a;         // drafts that stand
  bool refused;  // the draft of slot a + 1 was tested and refused
  Part row;      // row a's maximum, its id (INT_MAX: no weight), and the sum of its weights
};

__device__ __forceinline__ Verdict verdict_of(const Args& A, int n) {
  const int limit = limit_of(A, n), stop = A.stop[n];
  Verdict v;
  v.refused = stop < limit;
  v.a = min(stop, limit);
  v.row = A.row[(int64_t)n * A.B + v.a];
  return v;
}

__global__ __launch_bounds__(kThreads) void clear_kernel(Args A) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < A.N * A.B) A.done[i] = 0;
  if (i < A.N) {
    A.stop[i] = A.B;
    A.drawn[i] = 0;
  }
}

// The row of the draw: weights p = 2^((x - m) c); where the draft d was refused, what it leaves of
// them: p without d, or (`drawn`) max(p / sum - q, 0).
template <class T> struct Weights {
  const Args& A;
  const T* x;
  float m;
  double scale, inv_sum;
  bool drawn;
  int d;
  int64_t q_row;

  __device__ __forceinline__ double kept(float xv, float q) const {
    const double p = pow2(((double)xv - (double)m) * scale);
    return drawn ? fmax(fma(p, inv_sum, -(double)q), 0.0) : p;
  }
  // The piece's logits as kept() takes them: the point draft's is -inf, and where the maximum is +inf
  // (a difference of infinities is no number) the ids that hold it are 0 and the others -inf.
  __device__ __forceinline__ void load(const Row<T>& row, int64_t j, float (&out)[Row<T>::E]) const {
    const Piece<T> p = row.load(j);
    const int v0 = row.first(j);
#pragma unroll
    for (int e = 0; e < Row<T>::E; ++e) out[e] = p[e];
    if (!drawn && d >= v0 && d < v0 + Row<T>::E) {
#pragma unroll
      for (int e = 0; e < Row<T>::E; ++e) out[e] = d == v0 + e ? -INFINITY : out[e];
    }
    if (infinite) {
#pragma unroll
      for (int e = 0; e < Row<T>::E; ++e) out[e] = out[e] == INFINITY ? 0.f : -INFINITY;
    }
  }
  bool infinite;
};

// With the target's own weights, without a refused point draft.
template <class T>
__device__ Weights<T> weights_of(const Args& A, int n, const Verdict& v, double scale) {
  const int64_t r = (int64_t)n * A.B + v.a;
  const int64_t d = v.refused && !A.q ? A.blk[r + 1] : -1;
  const bool infinite = v.row.m == INFINITY;
  return Weights<T>{A, static_cast<const T*>(A.logits) + r * A.ld, infinite ? 0.f : v.row.m, scale,
                    0, false, d >= 0 && d < A.V ? (int)d : -1,
                    ((int64_t)n * (A.B - 1) + v.a) * A.q_ld, infinite};
}

// Running sums over a wave's lanes, this lane's included.
__device__ __forceinline__ double wave_scan(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Sum over the workgroup, in every thread; s_sum is the caller's and used once.
__device__ __forceinline__ double block_sum(double v, double* s_sum) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) t += s_sum[i];
  return t;
}

// Picks the first unit whose running sum passes the goal, one unit a lane in order, *before the sum
// before lane 0's. Where none does (the sums' last roundings) it is the last unit with weight, and
// *goal is lifted so that the levels below do the same. Uniform in the wave.
__device__ __forceinline__ int pick_lane(double unit, double* before, double* goal) {
  const double to_here = *before + wave_scan(unit);
  const uint64_t some = __ballot(unit > 0), pass = __ballot(unit > 0 && to_here > *goal);
  if (!pass) *goal = INFINITY;
  const int lane = pass ? __builtin_ctzll(pass) : 63 - __builtin_clzll(some | 1);
  *before = __shfl(to_here - unit, lane);
  return lane;
}

// The block's answer, by one wave; `next` is blk[n, lane + 1].
__device__ __forceinline__ void finish(const Args& A, int n, const Verdict& v, int64_t next, int token) {
  const int lane = threadIdx.x;
  if (lane < A.B) A.out[(int64_t)n * A.B + lane] = lane < v.a ? next : lane == v.a ? token : -1;
  if (lane == 0) {
    A.accepted[n] = v.a;
    if (A.drop) A.drop[n] = A.B - 1 - v.a;
  }
}
__device__ __forceinline__ int64_t next_of(const Args& A, int n) {
  return (int)threadIdx.x < A.B - 1 ? A.blk[(int64_t)n * A.B + threadIdx.x + 1] : -1;
}

// One chunk's sum of what the draw takes from; in the block's last chunk (`draw`) also the draw: the
// lowest id whose running sum passes u * total. First the chunk (every wave for itself), then the
// piece in it, then the id (the first wave). Bound by latency: a chain of a dozen dependent reads,
// scans and barriers.
template <class T>
__device__ void sum_and_draw(const Args& A, int n, int c, const Verdict& v, Weights<T> left,
                             double* sums, bool draw) {
  constexpr int E = Row<T>::E, P = kChunk / E, K = P / kThreads;
  constexpr int R = P / 64;  // pieces in a row that a lane of the first wave adds up
  __shared__ double s_piece[P + P / R], s_sum[kThreads / 64];
  __shared__ int s_draw;
  const int t = threadIdx.x, lane = t & 63;
  const Row<T> row(left.x, A.V);
  const double u = A.u[(int64_t)n * A.B + A.B - 1];
  const int64_t next = next_of(A, n);
  double goal = 0, before = 0;
  // pass 0: this chunk; pass 1: the draw's chunk, its pieces' sums kept
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    const int64_t j0 = (int64_t)c * P + t;
    float x[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) left.load(row, j0 + k * kThreads, x[k]);
    float q[K][E] = {};
    if (left.drawn) {
#pragma unroll
      for (int k = 0; k < K; ++k) q_piece<E>(A, left.q_row, row.first(j0 + k * kThreads), q[k]);
    }
    double mine = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      double w = 0;
#pragma unroll
      for (int e = 0; e < E; ++e)
        w += left.kept(x[k][e], q[k][e]);
      if (pass) s_piece[k * kThreads + t + (k * kThreads + t) / R] = w;
      mine += w;
    }
    if (pass) break;
    const double total = block_sum(mine, s_sum);
    if (t == 0) {
      put(sums + c, total);
      s_draw = draw && count_in(A.drawn + n) == A.chunks - 1;
    }
    __syncthreads();
    if (!s_draw) return;
    // the chunk: the lanes' ranges of chunks, then the range's chunks
    const int per = (A.chunks + 63) / 64, c0 = min(lane * per, A.chunks), c1 = min(c0 + per, A.chunks);
    double range, all;
#pragma unroll 1
    for (;;) {
      range = 0;
      for (int i = c0; i < c1; ++i) range += get(sums + i);
      all = wave_sum(range);
      if (all > 0) break;
      if (!left.drawn) {  // nothing beside the point draft: it holds all the weight
        if (t < 64) finish(A, n, v, next, (int)left.d);
        return;
      }
      left.drawn = false;  // nothing is left: the target itself
      sums = A.sums + (int64_t)n * A.chunks;
    }
    goal = u * all;
    c = pick_lane(range, &before, &goal);
    if (per > 1) {
      const int first = c * per, end = min(first + per, A.chunks);
      double run = before;
      int last = first;
#pragma unroll 1
      for (int i = first; i < end; ++i) {
        const double w = get(sums + i);
        if (w > 0) {
          last = i;
          before = run;
          if (run + w > goal) break;
        }
        run += w;
      }
      c = last;
    }
  }
  __syncthreads();
  if (t >= 64) return;
  double mine = 0;
#pragma unroll
  for (int k = 0; k < R; ++k) mine += s_piece[lane * (R + 1) + k];
  const int range = pick_lane(mine, &before, &goal);
  const int piece = range * R + pick_lane(lane < R ? s_piece[range * (R + 1) + lane] : 0.0, &before, &goal);
  // one id a lane (every lane reads the piece and takes its own)
  const int64_t j = (int64_t)c * P + piece;
  float x[E], q[E] = {};
  left.load(row, j, x);
  if (left.drawn) q_piece<E>(A, left.q_row, row.first(j), q);
  float xv = -INFINITY, qv = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    xv = lane == e ? x[e] : xv;
    qv = lane == e ? q[e] : qv;
  }
  const int at = pick_lane(left.kept(xv, qv), &before, &goal);
  finish(A, n, v, next, row.first(j) + at);
}

// The row of the draw in 64 bits: each chunk's sum (A.draws workgroups a block: all its chunks, or
// one where every block is greedy). One block 10 us, 32 blocks 17, 256 blocks 45 (151,936 ids).
template <class T>
__global__ __launch_bounds__(kThreads) void sums_kernel(Args A) {
  const int n = blockIdx.x / A.draws, c = blockIdx.x % A.draws;
  const double scale = scale_of(A, n);
  const Verdict v = verdict_of(A, n);
  if (scale == 0.0 || v.row.arg == INT_MAX) {
    if (c == 0 && threadIdx.x < 64)
      finish(A, n, v, next_of(A, n), v.row.arg == INT_MAX ? -1 : v.row.arg);
    return;
  }
  sum_and_draw<T>(A, n, c, v, weights_of<T>(A, n, v, scale), A.sums + (int64_t)n * A.chunks,
                  !(A.q && v.refused));
}

// With the drafts' probabilities: what they leave of each chunk of a refused row. 32 blocks 18 us.
template <class T>
__global__ __launch_bounds__(kThreads) void left_kernel(Args A) {
  const int n = blockIdx.x / A.chunks, c = blockIdx.x % A.chunks;
  const double scale = scale_of(A, n);
  if (scale == 0.0) return;
  const Verdict v = verdict_of(A, n);
  if (!v.refused || v.row.arg == INT_MAX) return;
  Weights<T> left = weights_of<T>(A, n, v, scale);
  left.drawn = true;
  double mine = 0;
  for (int i = threadIdx.x; i < A.chunks; i += kThreads) mine += A.sums[(int64_t)n * A.chunks + i];
  __shared__ double s_sum[kThreads / 64];
  left.inv_sum = 1.0 / block_sum(mine, s_sum);
  sum_and_draw<T>(A, n, c, v, left, A.left + (int64_t)n * A.chunks, true);
}

template <class T> hipError_t launch_t(const Args& A, hipStream_t s) {
  hipLaunchKernelGGL(clear_kernel, dim3((A.N * A.B + kThreads - 1) / kThreads), dim3(kThreads), 0,
                     s, A);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(stats_kernel<T>, dim3((unsigned)A.chunks * A.N * A.B), dim3(kThreads), 0, s, A);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sums_kernel<T>, dim3((unsigned)A.draws * A.N), dim3(kThreads), 0, s, A);
  e = hipGetLastError();
  if (e != hipSuccess || A.q == nullptr || A.temperature == nullptr) return e;
  hipLaunchKernelGGL(left_kernel<T>, dim3((unsigned)A.chunks * A.N), dim3(kThreads), 0, s, A);
  return hipGetLastError();
}

int chunks_of(int64_t V) { return (int)((V + 7 + kChunk - 1) / kChunk); }

}  // namespace

int64_t verify_items(int N, int B, int64_t V) { return (int64_t)N * B * chunks_of(V); }

size_t verify_scratch_bytes(int N, int B, int64_t V) {
  return (size_t)N * chunks_of(V) * (B * sizeof(Part) + 2 * sizeof(double)) +
         (size_t)N * B * (sizeof(Part) + sizeof(int32_t)) + 2 * (size_t)N * sizeof(int32_t);
}

hipError_t launch_verify_draft(const void* logits, uint32_t logits_dtype, int64_t ld,
                               const int64_t* blk, const int32_t* draft_len, const void* q,
                               uint32_t q_dtype, int64_t q_ld, const float* temperature,
                               const float* u, int N, int B, int64_t V, int64_t* out,
                               int32_t* accepted, int32_t* drop, void* ws, hipStream_t s) {
  Args A{};
  A.logits = logits;
  A.ld = ld;
  A.q_ld = q_ld;
  A.blk = blk;
  A.draft_len = draft_len;
  A.q = q;
  A.q_dtype = q_dtype;
  A.temperature = temperature;
  A.u = u;
  A.N = N;
  A.B = B;
  A.V = (int)V;
  A.chunks = chunks_of(V);
  A.draws = temperature != nullptr ? A.chunks : 1;
  A.out = out;
  A.accepted = accepted;
  A.drop = drop;
  A.part = static_cast<Part*>(ws);
  A.row = A.part + (size_t)N * B * A.chunks;
  A.sums = reinterpret_cast<double*>(A.row + (size_t)N * B);
  A.left = A.sums + (size_t)N * A.chunks;
  A.done = reinterpret_cast<int32_t*>(A.left + (size_t)N * A.chunks);
  A.stop = A.done + (size_t)N * B;
  A.drawn = A.stop + N;
  return logits_dtype == XPRESS_BF16  ? launch_t<uint16_t>(A, s)
         : logits_dtype == XPRESS_F16 ? launch_t<_Float16>(A, s)
                                      : launch_t<float>(A, s);
}

}  // namespace xpress
