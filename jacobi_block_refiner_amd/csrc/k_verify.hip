// Verification of drafted blocks against the target's logits (gfx950).
//
// A row's weights are w(v) = 2^((x_v - m) c), c = log2(e) / T, m the row's maximum. Rows are cut into
// chunks of kChunk ids; stats_kernel leaves each chunk's maximum, its id and the sum of its weights
// (relative to the chunk's own maximum), and draw_kernel joins the chunks of a block's rows, tests
// the drafts, and finds the token: first the chunk whose running sum passes u * total, then the id
// inside it, the only part of the row that is read again.
//
// Weights and sums are kept in 64 bits. A draw from V ids has borders 1/V apart: weights that are
// off by 2^-24 would shift a border of a flat distribution of 151,936 ids by several percent of
// their distance and change that share of the tokens; at 2e-12 it is one in 10^6.
#include "serve.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // ids of a chunk: 32 a thread
constexpr int kMaxB = 64;

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
  double* left;   // [N, chunks]: what is left of the refused row's chunks (with q)
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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One chunk of one row. Bound by HBM: 16 KiB of bf16 a workgroup, eight workgroups a CU; the 18
// operations of 64 bits a weight are about as long as its two bytes' way from HBM.
template <class T>
__global__ __launch_bounds__(kThreads) void stats_kernel(Args A) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;
  const int c = blockIdx.x % A.chunks, y = blockIdx.x / A.chunks, t = threadIdx.x;
  const int n = y % A.N, s = y / A.N;
  if (s > limit_of(A, n)) return;
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
  double sum = 0;
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
        for (int e = 0; e < E; ++e) sum += x[k][e] == m ? 1.0 : 0.0;
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) sum += pow2(((double)x[k][e] - (double)m) * scale);
    }
    sum = wave_sum(sum);
  }
  __shared__ Part s_part[kThreads / 64];
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
    A.part[r * A.chunks + c] = p;
  }
}

// What a block's rows say, in every thread of the workgroup.
struct Verdict {
  int a;          // drafts that stand
  bool refused;   // the draft of slot a + 1 was tested and refused
  float m;        // row a's maximum, its id (INT_MAX: no weight), and the sum of its weights
  int arg;
  double sum;
};

template <class T>
__device__ Verdict decide(const Args& A, int n, double scale) {
  __shared__ Part s_row[kMaxB];
  __shared__ int s_ok[kMaxB];
  const int lane = threadIdx.x & 63, limit = limit_of(A, n);
  for (int s = threadIdx.x >> 6; s <= limit; s += kThreads / 64) {
    const int64_t r = (int64_t)n * A.B + s;
    const Part* part = A.part + r * A.chunks;
    float m = -INFINITY;
    int arg = INT_MAX;
    for (int c = lane; c < A.chunks; c += 64) {
      const Part p = part[c];
      if (p.arg != INT_MAX) argmax_merge(m, arg, p.m, p.arg);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) argmax_merge(m, arg, __shfl_xor(m, d), __shfl_xor(arg, d));
    double sum = 0;
    if (scale != 0.0 && arg != INT_MAX) {
      for (int c = lane; c < A.chunks; c += 64) {
        const Part p = part[c];
        if (p.arg != INT_MAX) sum += p.sum * weight(p.m, m, scale);
      }
      sum = wave_sum(sum);
    }
    bool ok = false;
    if (s < limit && arg != INT_MAX) {
      const int64_t d = A.blk[r + 1];
      if (scale == 0.0) {
        ok = d == arg;
      } else if (d >= 0 && d < A.V) {
        const float x = to_f32<T>(static_cast<const T*>(A.logits)[r * A.ld + d]);
        const double qd = A.q ? q_at(A, ((int64_t)n * (A.B - 1) + s) * A.q_ld + d) : 1.0;
        ok = (double)A.u[r] * qd * sum < weight(x, m, scale);
      }
    }
    if (lane == 0) {
      s_row[s] = Part{sum, m, arg};
      s_ok[s] = ok;
    }
  }
  __syncthreads();
  Verdict v;
  v.a = 0;
  while (v.a < limit && s_ok[v.a]) ++v.a;
  v.refused = v.a < limit;
  v.m = s_row[v.a].m;
  v.arg = s_row[v.a].arg;
  v.sum = s_row[v.a].sum;
  return v;
}

// The row of the draw: weights p = 2^((x - m) c); with `residual` what the refused draft d leaves
// of them, max(p / sum - q, 0), or p without d for a point draft.
template <class T> struct Weights {
  const Args& A;
  const T* x;
  float m;
  double scale, sum;
  bool residual;
  int64_t d, q_row;
};

template <class T>
__device__ Weights<T> weights_of(const Args& A, int n, const Verdict& v, double scale) {
  const int64_t r = (int64_t)n * A.B + v.a;
  return Weights<T>{A, static_cast<const T*>(A.logits) + r * A.ld, v.m, scale, v.sum, v.refused,
                    v.refused ? A.blk[r + 1] : -1, ((int64_t)n * (A.B - 1) + v.a) * A.q_ld};
}

// The weights that this thread's ids of chunk c keep, in `w`: pieces a thread apart (coalesced),
// or with `in_order` one after the other, so that threads hold ascending ranges of ids. All loads
// are in flight before the first weight is formed. Returns the first piece.
template <class T, bool in_order>
__device__ __forceinline__ int64_t chunk_weights(const Row<T>& row, const Weights<T>& left, int c,
                                                 double (&w)[kChunk / kThreads]) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;
  const int64_t j0 = (int64_t)c * (kChunk / E) + threadIdx.x * (in_order ? K : 1);
  constexpr int step = in_order ? 1 : kThreads;
  float x[K][E], q[K][E];
#pragma unroll
  for (int k = 0; k < K; ++k) row.load(j0 + k * step, x[k]);
  const bool drawn = left.residual && left.A.q;
  if (drawn) {
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
      w[k * E + e] = drawn                            ? fmax(p / left.sum - (double)q[k][e], 0.0)
                     : left.residual && v == left.d ? 0.0
                                                    : p;
    }
  return j0;
}

// Sum over the workgroup, the same in every thread.
__device__ double block_sum(double v) {
  __shared__ double s_sum[kThreads / 64];
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) t += s_sum[i];
  return t;
}

// Sum of the values of the threads before this one.
__device__ double block_before(double v) {
  __shared__ double s_wave[kThreads / 64];
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
  for (int i = 0; i < kThreads / 64; ++i) before += i < w ? s_wave[i] : 0.0;
  const double up = __shfl_up(x, 1);
  return before + (lane ? up : 0.0);
}

// With the drafts' probabilities: what is left of each chunk of the refused row.
template <class T>
__global__ __launch_bounds__(kThreads) void left_kernel(Args A) {
  const int n = blockIdx.x / A.chunks, c = blockIdx.x % A.chunks;
  const double scale = scale_of(A, n);
  if (scale == 0.0) return;
  const Verdict v = decide<T>(A, n, scale);
  if (!v.refused || v.arg == INT_MAX) return;
  const Weights<T> left = weights_of<T>(A, n, v, scale);
  double w[kChunk / kThreads], sum = 0;
  chunk_weights<T, false>(Row<T>(left.x, A.V), left, c, w);
#pragma unroll
  for (int i = 0; i < kChunk / kThreads; ++i) sum += w[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) A.left[(int64_t)n * A.chunks + c] = sum;
}

// The verdict on one block, and its token.
template <class T>
__global__ __launch_bounds__(kThreads) void draw_kernel(Args A) {
  const int n = blockIdx.x, t = threadIdx.x;
  const double scale = scale_of(A, n);
  const Verdict v = decide<T>(A, n, scale);
  int token = -1;
  if (v.arg != INT_MAX && scale == 0.0) token = v.arg;
  if (v.arg != INT_MAX && scale != 0.0) {
    Weights<T> left = weights_of<T>(A, n, v, scale);
    const Row<T> row(left.x, A.V);
    const Part* part = A.part + ((int64_t)n * A.B + v.a) * A.chunks;
    // a point draft's chunk is summed anew without it (a difference of sums would lose what is
    // left beside a draft that holds nearly all the weight)
    int point_chunk = -1;
    double point_sum = 0;
    if (v.refused && !A.q && left.d >= 0 && left.d < A.V) {
      point_chunk = (int)((left.d + row.off) / kChunk);
      double w[kChunk / kThreads];
      chunk_weights<T, false>(row, left, point_chunk, w);
#pragma unroll
      for (int i = 0; i < kChunk / kThreads; ++i) point_sum += w[i];
      point_sum = block_sum(point_sum);
    }
    auto chunk_sum = [&](int c) {
      if (left.residual && A.q) return A.left[(int64_t)n * A.chunks + c];
      if (left.residual && c == point_chunk) return point_sum;
      return part[c].arg == INT_MAX ? 0.0 : part[c].sum * weight(part[c].m, v.m, scale);
    };
    const int per = (A.chunks + kThreads - 1) / kThreads;
    const int c0 = min(t * per, A.chunks), c1 = min(c0 + per, A.chunks);
    double mine = 0, total = 0;
    for (int round = 0; round < 2; ++round) {
      mine = 0;
      for (int c = c0; c < c1; ++c) mine += chunk_sum(c);
      total = block_sum(mine);
      if (!left.residual || total > 0) break;
      left.residual = false;  // nothing is left: the target itself
    }
    const double goal = (double)A.u[(int64_t)n * A.B + A.B - 1] * total;
    __shared__ int s_chunk, s_last, s_token, s_end;
    __shared__ double s_before;
    if (t == 0) {
      s_chunk = INT_MAX;
      s_last = s_end = -1;
      s_token = INT_MAX;
    }
    double run = block_before(mine);  // (its barriers order the lines above)
    double before = run;
    int hit = INT_MAX, last = -1;
    for (int c = c0; c < c1; ++c) {
      const double w = chunk_sum(c);
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
    __syncthreads();
    constexpr int K = kChunk / kThreads;
    double w[K];
    const int64_t v0 = chunk_weights<T, true>(row, left, chunk, w) * Row<T>::E - row.off;
    mine = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) mine += w[i];
    run = block_before(mine) + (rounded ? 0.0 : s_before);
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
    token = s_token == INT_MAX ? s_end : s_token;
  }
  for (int s = t; s < A.B; s += kThreads)
    A.out[(int64_t)n * A.B + s] = s < v.a ? A.blk[(int64_t)n * A.B + s + 1] : s == v.a ? token : -1;
  if (t == 0) {
    A.accepted[n] = v.a;
    if (A.drop) A.drop[n] = A.B - 1 - v.a;
  }
}

template <class T> hipError_t launch_t(const Args& A, hipStream_t s) {
  hipLaunchKernelGGL(stats_kernel<T>, dim3((unsigned)A.chunks * A.N * A.B), dim3(kThreads), 0, s, A);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (A.q != nullptr && A.temperature != nullptr) {
    hipLaunchKernelGGL(left_kernel<T>, dim3((unsigned)A.chunks * A.N), dim3(kThreads), 0, s, A);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(draw_kernel<T>, dim3(A.N), dim3(kThreads), 0, s, A);
  return hipGetLastError();
}

int chunks_of(int64_t V) { return (int)((V + 7 + kChunk - 1) / kChunk); }

}  // namespace

int64_t verify_items(int N, int B, int64_t V) { return (int64_t)N * B * chunks_of(V); }

size_t verify_scratch_bytes(int N, int B, int64_t V) {
  return (size_t)N * chunks_of(V) * (B * sizeof(Part) + sizeof(double));
}

hipError_t launch_verify_draft(const void* logits, uint32_t logits_dtype, int64_t ld,
                               const int64_t* blk, const int32_t* draft_len, const void* q,
                               uint32_t q_dtype, int64_t q_ld, const float* temperature,
                               const float* u, int N, int B, int64_t V, int64_t* out,
                               int32_t* accepted, int32_t* drop, void* ws, hipStream_t s) {
  Args A{logits, ld, q_ld, blk, draft_len, q, q_dtype, temperature, u, N, B, (int)V, chunks_of(V),
         out, accepted, drop, nullptr, nullptr};
  A.part = static_cast<Part*>(ws);
  A.left = reinterpret_cast<double*>(A.part + (size_t)N * B * A.chunks);
  return logits_dtype == XPRESS_BF16  ? launch_t<uint16_t>(A, s)
         : logits_dtype == XPRESS_F16 ? launch_t<_Float16>(A, s)
                                      : launch_t<float>(A, s);
}

}  // namespace xpress
