// Verification of drafted blocks against the target's logits (gfx950).
#include "serve.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

template <class T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
template <> __device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
template <> __device__ __forceinline__ float to_f32(float x) { return x; }

// An element of q by its type code.
__device__ __forceinline__ float q_at(const void* q, uint32_t dtype, int64_t i) {
  if (dtype == XPRESS_BF16) return bf16_to_f32(static_cast<const uint16_t*>(q)[i]);
  if (dtype == XPRESS_F16) return (float)static_cast<const _Float16*>(q)[i];
  return static_cast<const float*>(q)[i];
}

// Weight of a logit relative to the row's maximum m: exp((x - m) / T); 0 for NaN and -inf, 1 where
// x == m (also at +inf).
__device__ __forceinline__ double weight(float x, float m, double inv_t) {
  return x == m ? 1.0 : x < m ? exp(((double)x - (double)m) * inv_t) : 0.0;
}

constexpr int kThreads = 1024;

struct Best {
  float v;
  int i;
};

__device__ __forceinline__ double block_sum(double v, double* s_d) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_d[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
  for (int i = 0; i < kThreads / 64; ++i) t += s_d[i];
  return t;
}

// One workgroup per block of drafts: row by row, the maximum and the sum of weights, the test,
// and at the end the draw from the row where it stopped.
template <class T>
__global__ __launch_bounds__(kThreads) void verify_kernel(
    const T* logits, int64_t ld, const int64_t* blk, const int32_t* draft_len, const void* q,
    uint32_t q_dtype, int64_t q_ld, const float* temperature, const float* u, int B, int V,
    int64_t* out, int32_t* accepted, int32_t* drop) {
  __shared__ float s_v[kThreads / 64];
  __shared__ int s_i[kThreads / 64];
  __shared__ double s_d[kThreads / 64];
  const int n = blockIdx.x, t = threadIdx.x;
  const float temp = temperature ? temperature[n] : 0.f;
  const bool greedy = !(temp > 0.f);
  const double inv_t = greedy ? 1.0 : 1.0 / (double)temp;
  const int limit = draft_len ? min(max(draft_len[n], 0), B - 1) : B - 1;
  int a = 0;
  int64_t token = -1;
  for (;; ++a) {
    const T* x = logits + ((int64_t)n * B + a) * ld;
    float bv = -INFINITY;
    int bi = INT_MAX;
    for (int v = t; v < V; v += kThreads) {
      const float f = to_f32<T>(x[v]);
      if (f > bv) { bv = f; bi = v; }
    }
    for (int d = 32; d; d >>= 1) argmax_merge(bv, bi, __shfl_xor(bv, d), __shfl_xor(bi, d));
    __syncthreads();
    if ((t & 63) == 0) { s_v[t >> 6] = bv; s_i[t >> 6] = bi; }
    __syncthreads();
    for (int i = 0; i < kThreads / 64; ++i) argmax_merge(bv, bi, s_v[i], s_i[i]);
    if (bi == INT_MAX) break;  // a row without any weight
    const int64_t d = a < limit ? blk[(int64_t)n * B + a + 1] : -1;
    if (greedy) {
      if (a < limit && d == bi) continue;
      token = bi;
      break;
    }
    double sum = 0;
    for (int v = t; v < V; v += kThreads) sum += weight(to_f32<T>(x[v]), bv, inv_t);
    sum = block_sum(sum, s_d);
    const bool known = d >= 0 && d < V;
    const int64_t qrow = ((int64_t)n * (B - 1) + a) * q_ld;
    if (a < limit && known) {
      const double qd = q ? (double)q_at(q, q_dtype, qrow + d) : 1.0;
      if ((double)u[(int64_t)n * B + a] * qd * sum < weight(to_f32<T>(x[d]), bv, inv_t)) continue;
    }
    // the draw: left(v) for what is left of the row, or all of it
    auto left = [&](int v, bool residual) {
      const double w = weight(to_f32<T>(x[v]), bv, inv_t);
      if (!residual) return w;
      if (!q) return v == d ? 0.0 : w;
      return fmax(w / sum - (double)q_at(q, q_dtype, qrow + v), 0.0);
    };
    const int chunk = (V + kThreads - 1) / kThreads, v0 = min(t * chunk, V), v1 = min(v0 + chunk, V);
    bool residual = a < limit;
    double mine = 0, all = 0;
    for (int round = 0; round < 2; ++round) {
      mine = 0;
      for (int v = v0; v < v1; ++v) mine += left(v, residual);
      all = block_sum(mine, s_d);
      if (!residual || all > 0) break;
      residual = false;
    }
    // running sums in id order: an exclusive scan of the threads' sums
    __shared__ double s_run[kThreads];
    __shared__ int s_tok, s_last;
    if (t == 0) { s_tok = INT_MAX; s_last = -1; }
    s_run[t] = mine;
    __syncthreads();
    if (t == 0) {
      double run = 0;
      for (int i = 0; i < kThreads; ++i) {
        const double w = s_run[i];
        s_run[i] = run;
        run += w;
      }
      s_d[0] = run;
    }
    __syncthreads();
    const double goal = (double)u[(int64_t)n * B + B - 1] * s_d[0];
    double run = s_run[t];
    int last = -1;
    for (int v = v0; v < v1; ++v) {
      const double w = left(v, residual);
      run += w;
      if (w > 0) last = v;
      if (run > goal && w > 0) {
        atomicMin(&s_tok, v);
        break;
      }
    }
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
    token = s_tok == INT_MAX ? s_last : s_tok;
    break;
  }
  for (int s = t; s < B; s += kThreads)
    out[(int64_t)n * B + s] = s < a ? blk[(int64_t)n * B + s + 1] : s == a ? token : -1;
  if (t == 0) {
    accepted[n] = a;
    if (drop) drop[n] = B - 1 - a;
  }
}

template <class T>
hipError_t launch_t(const void* logits, int64_t ld, const int64_t* blk, const int32_t* draft_len,
                    const void* q, uint32_t q_dtype, int64_t q_ld, const float* temperature,
                    const float* u, int N, int B, int64_t V, int64_t* out, int32_t* accepted,
                    int32_t* drop, hipStream_t s) {
  hipLaunchKernelGGL(verify_kernel<T>, dim3(N), dim3(kThreads), 0, s,
                     static_cast<const T*>(logits), ld, blk, draft_len, q, q_dtype, q_ld,
                     temperature, u, B, (int)V, out, accepted, drop);
  return hipGetLastError();
}

}  // namespace

size_t verify_scratch_bytes(int N, int B, int64_t V) { return 256; }

hipError_t launch_verify_draft(const void* logits, uint32_t logits_dtype, int64_t ld,
                               const int64_t* blk, const int32_t* draft_len, const void* q,
                               uint32_t q_dtype, int64_t q_ld, const float* temperature,
                               const float* u, int N, int B, int64_t V, int64_t* out,
                               int32_t* accepted, int32_t* drop, void* ws, hipStream_t s) {
  const auto go = logits_dtype == XPRESS_BF16 ? launch_t<uint16_t>
                  : logits_dtype == XPRESS_F16 ? launch_t<_Float16> : launch_t<float>;
  return go(logits, ld, blk, draft_len, q, q_dtype, q_ld, temperature, u, N, B, V, out, accepted,
            drop, s);
}

}  // namespace xpress
