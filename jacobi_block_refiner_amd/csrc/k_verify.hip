// Verification of drafted blocks against the target's logits (gfx950).
//
// A row's weights are w(v) = 2^((x_v - m) c), c = log2(e) / T, m the row's maximum. Rows are cut into
// chunks of kChunk ids; stats_kernel leaves each chunk's maximum, its id and the sum of its weights
// (relative to the chunk's own maximum), and the last chunk of a row joins them and tests the row's
// draft. For the one row of each block where a token is drawn, sums_kernel forms the chunks' sums
// once more in 64 bits (left_kernel what the drafts' probabilities leave of them), and draw_kernel
// finds the token: first the chunk whose running sum passes u * total, then the id inside it.
//
// Precision. A draw from V ids has borders 1/V apart: weights that are off by 2^-24 would shift a
// border of a flat distribution of 151,936 ids by several percent of their distance and change that
// share of the tokens; at 2e-12 it is one in 10^6. A test u q S < w has one border and takes 32-bit
// weights; where the two sides are within 1e-5 of each other the row is summed anew in 64 bits.
// (64 bits for all rows: 74 against MEASURED_STATS us at 512 rows of 151,936 ids.)
//
// Rows after a block's first refusal do not matter. Chunks go by slot, all blocks' first slots
// first, and a chunk whose block is known to have been refused earlier returns at once. How many
// do depends on timing; the result does not, since rows up to the first refusal are never left out.
#include "serve.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

constexpr int kThreads = 256;
constexpr int kDraw = 1024;  // threads of draw_kernel: one workgroup a block, bound by latency
constexpr int kChunk = 8192;  // ids of a chunk: 32 a thread

template <class T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
template <> __device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
template <> __device__ __forceinline__ float to_f32(float x) { return x; }

// 2^t for t <= 0 (NaN: 0), relative error 2.2e-12: 2^f = 1 + f p(f) for the fraction f in
// [-1/2, 1/2], p fitted at Chebyshev nodes; adding 3 * 2^51 rounds t to an integer that stands in
// the sum's low word.
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
  const int64_t bits = __double_as_longlong(p) + ((int64_t)(uint64_t)__double_as_longlong(big) << 52);
  return c < -1000.0 ? 0.0 : __longlong_as_double(bits);
}

// A logit's weight relative to the maximum m: 0 for -inf and NaN; at m = +inf the ids that hold it
// share all.
__device__ __forceinline__ double weight(float x, float m, double c) {
  return m == INFINITY ? (x == INFINITY ? 1.0 : 0.0) : pow2(((double)x - (double)m) * c);
}

// Chunks of a row: its first 16-byte boundary at or before the row begins chunk 0, so that all but
// the row's two ends are read in whole 16-byte pieces whatever the row's alignment.
template <class T> struct Row {
  static constexpr int E = 16 / sizeof(T);  // ids of a piece
  const T* x;
  int V, off;
  __device__ Row(const T* x_, int V_) : x(x_), V(V_), off((int)((uintptr_t)x_ % 16 / sizeof(T))) {}
  // The ids of piece j (ids outside the row: -inf).
  __device__ __forceinline__ int first(int64_t j) const { return (int)(j * E - off); }
  __device__ __forceinline__ void load(int64_t j, float* out) const {
    const int64_t v0 = j * E - off;
    if (v0 >= 0 && v0 + E <= V) {
      const uint4 u = *reinterpret_cast<const uint4*>(x + v0);
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < E; ++i) out[i] = to_f32<T>(e[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        out[i] = v0 + i >= 0 && v0 + i < V ? to_f32<T>(x[v0 + i]) : -INFINITY;
    }
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
  int N, B, V, chunks;
  int64_t* out;
  int32_t *accepted, *drop;
  Part* part;     // [N*B, chunks]
  Part* row;      // [N*B]: the rows' own
  double* sums;   // [N, chunks]: the row of the draw (without a refused point draft)
  double* left;   // [N, chunks]: what is left of it beside the drafts' probabilities
  int32_t* done;  // [N*B]: chunks that are in
  int32_t* stop;  // [N]: first refused slot so far (B: none)
};

// An element of q by its type code.
__device__ __forceinline__ float q_at(const Args& A, int64_t i) {
  if (A.q_dtype == XPRESS_BF16) return bf16_to_f32(static_cast<const uint16_t*>(A.q)[i]);
  if (A.q_dtype == XPRESS_F16) return (float)static_cast<const _Float16*>(A.q)[i];
  return static_cast<const float*>(A.q)[i];
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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

template <int NT> __device__ double block_sum(double v) {
  __shared__ double s_sum[NT / 64];
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) t += s_sum[i];
  return t;  // the same in every thread
}

// One chunk of one row. Bound by HBM: 16 KiB of bf16 a workgroup, eight workgroups a CU.
template <class T>
__global__ __launch_bounds__(kThreads) void stats_kernel(Args A) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;
  const int c = blockIdx.x % A.chunks, y = blockIdx.x / A.chunks, t = threadIdx.x;
  const int n = y % A.N, s = y / A.N, limit = limit_of(A, n);
  if (s > limit || s > __hip_atomic_load(A.stop + n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
    return;
  const int64_t r = (int64_t)n * A.B + s;
  const Row<T> row(static_cast<const T*>(A.logits) + r * A.ld, A.V);
  float x[K][E];
#pragma unroll
  for (int k = 0; k < K; ++k) row.load((int64_t)c * (kChunk / E) + k * kThreads + t, x[k]);
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, x[k][e]);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const double scale = scale_of(A, n);
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
      const float c32 = (float)fmin(scale, 1e37);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e)
          sum += __builtin_amdgcn_exp2f(fmaxf((x[k][e] - m) * c32, -1e30f));
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  }
  __shared__ Part s_part[kThreads / 64];
  __shared__ int s_last, s_again;
  if ((t & 63) == 0) s_part[t >> 6] = Part{sum, m, arg};
  __syncthreads();
  if (t == 0) {
    Part p = s_part[0];
    for (int i = 1; i < kThreads / 64; ++i) p.m = fmaxf(p.m, s_part[i].m);
    p.sum = 0;
    p.arg = INT_MAX;
    for (int i = 0; i < kThreads / 64; ++i) {
      const Part& o = s_part[i];
      if (o.arg == INT_MAX) continue;
      if (scale != 0.0) p.sum += o.sum * weight(o.m, p.m, scale);
      if (o.m == p.m) p.arg = min(p.arg, o.arg);
    }
    put(A.part + r * A.chunks + c, p);
    // The chunk is in memory before it is counted: its stores go through the caches to the card's
    // point of coherence, and the wait is for their acknowledgement. (A release at the card's scope
    // also writes back the whole L2 of the XCD and an acquire empties it, once a chunk: 278 against
    // 74 us at 512 rows of 151,936 ids.)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    asm volatile("" ::: "memory");
    s_last = __hip_atomic_fetch_add(A.done + r, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             A.chunks - 1;
    s_again = 0;
  }
  __syncthreads();
  if (!s_last) return;
  // the row's last chunk: join them, test the draft
  const Part* part = A.part + r * A.chunks;
  Part w{0, -INFINITY, INT_MAX};
  bool ok = false;
  int64_t d = -1;
  double test = 0, drafted = 0;  // u q, and the draft's weight
  if (t < 64) {
    if (s < limit) {
      d = A.blk[r + 1];
      if (d < 0 || d >= A.V) d = -1;
      if (scale != 0.0 && d >= 0) {
        const double qd = A.q ? q_at(A, ((int64_t)n * (A.B - 1) + s) * A.q_ld + d) : 1.0;
        test = (double)A.u[r] * qd;
      }
    }
    for (int i = t; i < A.chunks; i += 64) {
      const Part o = get(part + i);
      if (o.arg != INT_MAX) argmax_merge(w.m, w.arg, o.m, o.arg);
    }
#pragma unroll
    for (int x = 32; x; x >>= 1) argmax_merge(w.m, w.arg, __shfl_xor(w.m, x), __shfl_xor(w.arg, x));
    if (scale == 0.0) {
      ok = w.arg != INT_MAX && d == w.arg;
    } else if (w.arg != INT_MAX && d >= 0) {
      for (int i = t; i < A.chunks; i += 64) {
        const Part o = get(part + i);
        if (o.arg != INT_MAX) w.sum += o.sum * weight(o.m, w.m, scale);
      }
      w.sum = wave_sum(w.sum);
      drafted = weight(to_f32<T>(row.x[d]), w.m, scale);
      ok = test * w.sum < drafted;
      if (t == 0) s_again = fabs(test * w.sum - drafted) <= 1e-5 * drafted;
    }
    if (t == 0) s_part[0] = w;
  }
  __syncthreads();
  if (s_again) {
    const float top = s_part[0].m;
    double all = 0;
    for (int v = t; v < A.V; v += kThreads) all += weight(to_f32<T>(row.x[v]), top, scale);
    all = block_sum<kThreads>(all);
    ok = test * all < drafted;
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

__global__ __launch_bounds__(kThreads) void clear_kernel(int32_t* done, int rows, int32_t* stop,
                                                         int N, int B) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < rows) done[i] = 0;
  if (i < N) stop[i] = B;
}

// The row of the draw: weights p = 2^((x - m) c); where the draft d was refused, what it leaves of
// them: p without d, or (`drawn`) max(p / sum - q, 0).
template <class T> struct Weights {
  const Args& A;
  const T* x;
  float m;
  double scale, sum;
  bool drawn;
  int64_t d, q_row;
};

// With the target's own weights, without a refused point draft.
template <class T>
__device__ Weights<T> weights_of(const Args& A, int n, const Verdict& v, double scale) {
  const int64_t r = (int64_t)n * A.B + v.a;
  return Weights<T>{A, static_cast<const T*>(A.logits) + r * A.ld, v.row.m, scale, 0, false,
                    v.refused && !A.q ? A.blk[r + 1] : -1, ((int64_t)n * (A.B - 1) + v.a) * A.q_ld};
}

// The weights that this thread's ids of chunk c keep, in `w`: pieces a thread apart (coalesced),
// or with `in_order` one after the other, so that threads hold ascending ranges of ids. All loads
// are in flight before the first weight is formed. Returns the first piece.
template <class T, int NT, bool in_order>
__device__ __forceinline__ int64_t chunk_weights(const Row<T>& row, const Weights<T>& left, int c,
                                                 double (&w)[kChunk / NT]) {
  constexpr int E = Row<T>::E, K = kChunk / NT / E;
  const int64_t j0 = (int64_t)c * (kChunk / E) + threadIdx.x * (in_order ? K : 1);
  constexpr int step = in_order ? 1 : NT;
  float x[K][E], q[K][E];
#pragma unroll
  for (int k = 0; k < K; ++k) row.load(j0 + k * step, x[k]);
  if (left.drawn) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int64_t v = (j0 + k * step) * E - row.off + e;
        q[k][e] = v >= 0 && v < row.V ? q_at(left.A, left.q_row + v) : 0.f;
      }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const double p = weight(x[k][e], left.m, left.scale);
      const int64_t v = (j0 + k * step) * E - row.off + e;
      w[k * E + e] = left.drawn    ? fmax(p / left.sum - (double)q[k][e], 0.0)
                     : v == left.d ? 0.0
                                   : p;
    }
  return j0;
}

// Sum of the values of the threads before this one.
template <int NT> __device__ double block_before(double v) {
  __shared__ double s_wave[NT / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) s_wave[w] = x;
  __syncthreads();
  double before = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) before += i < w ? s_wave[i] : 0.0;
  const double up = __shfl_up(x, 1);
  return before + (lane ? up : 0.0);
}

// The row of the draw in 64 bits: each chunk's sum.
template <class T>
__global__ __launch_bounds__(kThreads) void sums_kernel(Args A) {
  const int n = blockIdx.x / A.chunks, c = blockIdx.x % A.chunks;
  const double scale = scale_of(A, n);
  if (scale == 0.0) return;
  const Verdict v = verdict_of(A, n);
  if (v.row.arg == INT_MAX) return;
  const Weights<T> left = weights_of<T>(A, n, v, scale);
  double w[kChunk / kThreads], sum = 0;
  chunk_weights<T, kThreads, false>(Row<T>(left.x, A.V), left, c, w);
#pragma unroll
  for (int i = 0; i < kChunk / kThreads; ++i) sum += w[i];
  sum = block_sum<kThreads>(sum);
  if (threadIdx.x == 0) A.sums[(int64_t)n * A.chunks + c] = sum;
}

template <int NT> __device__ double total_of(const double* sums, int chunks) {
  double mine = 0;
  for (int c = threadIdx.x; c < chunks; c += NT) mine += sums[c];
  return block_sum<NT>(mine);
}

// With the drafts' probabilities: what they leave of each chunk of a refused row.
template <class T>
__global__ __launch_bounds__(kThreads) void left_kernel(Args A) {
  const int n = blockIdx.x / A.chunks, c = blockIdx.x % A.chunks;
  const double scale = scale_of(A, n);
  if (scale == 0.0) return;
  const Verdict v = verdict_of(A, n);
  if (!v.refused || v.row.arg == INT_MAX) return;
  Weights<T> left = weights_of<T>(A, n, v, scale);
  left.drawn = true;
  left.sum = total_of<kThreads>(A.sums + (int64_t)n * A.chunks, A.chunks);
  double w[kChunk / kThreads], sum = 0;
  chunk_weights<T, kThreads, false>(Row<T>(left.x, A.V), left, c, w);
#pragma unroll
  for (int i = 0; i < kChunk / kThreads; ++i) sum += w[i];
  sum = block_sum<kThreads>(sum);
  if (threadIdx.x == 0) A.left[(int64_t)n * A.chunks + c] = sum;
}

// The lowest id whose running sum passes u * total.
template <class T>
__device__ int draw_token(const Args& A, int n, const Verdict& v, double scale) {
  const int t = threadIdx.x;
  Weights<T> left = weights_of<T>(A, n, v, scale);
  const double* sums = A.sums + (int64_t)n * A.chunks;
  double total = total_of<kDraw>(sums, A.chunks);
  if (total == 0) return (int)left.d;  // nothing beside the point draft: it holds all the weight
  if (v.refused && A.q) {
    const double* rest = A.left + (int64_t)n * A.chunks;
    const double what = total_of<kDraw>(rest, A.chunks);
    if (what > 0) {  // else nothing is left: the target itself
      left.drawn = true;
      left.sum = total;
      sums = rest;
      total = what;
    }
  }
  const double goal = (double)A.u[(int64_t)n * A.B + A.B - 1] * total;
  const int per = (A.chunks + kDraw - 1) / kDraw;
  const int c0 = min(t * per, A.chunks), c1 = min(c0 + per, A.chunks);
  double mine = 0;
  for (int c = c0; c < c1; ++c) mine += sums[c];
  __shared__ int s_chunk, s_last, s_token, s_end;
  __shared__ double s_before;
  if (t == 0) {
    s_chunk = s_token = INT_MAX;
    s_last = s_end = -1;
  }
  double run = block_before<kDraw>(mine);  // (its barriers order the lines above)
  double before = run;
  int hit = INT_MAX, last = -1;
  for (int c = c0; c < c1; ++c) {
    const double w = sums[c];
    if (w > 0) {
      last = c;
      if (hit == INT_MAX && run + w > goal) {
        hit = c;
        before = run;
      }
    }
    run += w;
  }
  if (hit != INT_MAX) atomicMin(&s_chunk, hit);
  if (last >= 0) atomicMax(&s_last, last);
  __syncthreads();
  const bool rounded = s_chunk == INT_MAX;  // the sums' last roundings: take the last weight
  const int chunk = rounded ? s_last : s_chunk;
  if (!rounded && hit == chunk) s_before = before;
  constexpr int K = kChunk / kDraw;
  double w[K];
  const Row<T> row(left.x, A.V);
  const int64_t v0 = chunk_weights<T, kDraw, true>(row, left, chunk, w) * Row<T>::E - row.off;
  mine = 0;
#pragma unroll
  for (int i = 0; i < K; ++i) mine += w[i];
  run = block_before<kDraw>(mine);
  run += rounded ? 0.0 : s_before;
  int end = -1, first = INT_MAX;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    run += w[i];
    if (w[i] > 0) {
      end = (int)(v0 + i);
      if (!rounded && first == INT_MAX && run > goal) first = end;
    }
  }
  if (first != INT_MAX) atomicMin(&s_token, first);
  if (end >= 0) atomicMax(&s_end, end);
  __syncthreads();
  return s_token == INT_MAX ? s_end : s_token;
}

// The verdict on one block, and its token.
template <class T>
__global__ __launch_bounds__(kDraw) void draw_kernel(Args A) {
  const int n = blockIdx.x, t = threadIdx.x;
  const double scale = scale_of(A, n);
  const Verdict v = verdict_of(A, n);
  const int token = v.row.arg == INT_MAX ? -1 : scale == 0.0 ? v.row.arg : draw_token<T>(A, n, v, scale);
  for (int s = t; s < A.B; s += kDraw)
    A.out[(int64_t)n * A.B + s] = s < v.a ? A.blk[(int64_t)n * A.B + s + 1] : s == v.a ? token : -1;
  if (t == 0) {
    A.accepted[n] = v.a;
    if (A.drop) A.drop[n] = A.B - 1 - v.a;
  }
}

template <class T> hipError_t launch_t(const Args& A, hipStream_t s) {
  const int rows = A.N * A.B;
  hipLaunchKernelGGL(clear_kernel, dim3((rows + kThreads - 1) / kThreads), dim3(kThreads), 0, s,
                     A.done, rows, A.stop, A.N, A.B);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(stats_kernel<T>, dim3((unsigned)A.chunks * A.N * A.B), dim3(kThreads), 0, s, A);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (A.temperature != nullptr) {
    hipLaunchKernelGGL(sums_kernel<T>, dim3((unsigned)A.chunks * A.N), dim3(kThreads), 0, s, A);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (A.q != nullptr && A.temperature != nullptr) {
    hipLaunchKernelGGL(left_kernel<T>, dim3((unsigned)A.chunks * A.N), dim3(kThreads), 0, s, A);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(draw_kernel<T>, dim3(A.N), dim3(kDraw), 0, s, A);
  return hipGetLastError();
}

int chunks_of(int64_t V) { return (int)((V + 7 + kChunk - 1) / kChunk); }

}  // namespace

int64_t verify_items(int N, int B, int64_t V) { return (int64_t)N * B * chunks_of(V); }

size_t verify_scratch_bytes(int N, int B, int64_t V) {
  return (size_t)N * chunks_of(V) * (B * sizeof(Part) + 2 * sizeof(double)) +
         (size_t)N * B * (sizeof(Part) + sizeof(int32_t)) + (size_t)N * sizeof(int32_t);
}

hipError_t launch_verify_draft(const void* logits, uint32_t logits_dtype, int64_t ld,
                               const int64_t* blk, const int32_t* draft_len, const void* q,
                               uint32_t q_dtype, int64_t q_ld, const float* temperature,
                               const float* u, int N, int B, int64_t V, int64_t* out,
                               int32_t* accepted, int32_t* drop, void* ws, hipStream_t s) {
  Args A{logits, ld, q_ld, blk, draft_len, q, q_dtype, temperature, u, N, B, (int)V, chunks_of(V),
         out, accepted, drop, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  A.part = static_cast<Part*>(ws);
  A.row = A.part + (size_t)N * B * A.chunks;
  A.sums = reinterpret_cast<double*>(A.row + (size_t)N * B);
  A.left = A.sums + (size_t)N * A.chunks;
  A.done = reinterpret_cast<int32_t*>(A.left + (size_t)N * A.chunks);
  A.stop = A.done + (size_t)N * B;
  return logits_dtype == XPRESS_BF16  ? launch_t<uint16_t>(A, s)
         : logits_dtype == XPRESS_F16 ? launch_t<_Float16>(A, s)
                                      : launch_t<float>(A, s);
}

}  // namespace xpress
