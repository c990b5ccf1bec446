// Log probabilities of given tokens, with entropy, rank and the most likely alternatives (gfx950).
//
// With c = log2(e) / T, m the row's maximum and z_v = (x_v - m) c, a row's sums are S = sum 2^z and
// Z = sum z 2^z: log p(v) = (x_v - m) / T - ln S, entropy ln 2 (log2 S - Z / S). Rows are cut into
// chunks of kChunk ids; chunks_kernel reads each once and leaves its maximum, its sums, how many ids
// lie above the token, and the maxima of its groups of 32 ids. finish_kernel, a workgroup a row, joins
// the sums and finds the alternatives: the ids in front of the others, by value and then by id, lie
// in the groups whose own best ids are in front of the other groups'. So it takes the best groups by
// their maxima, and then the best ids of those groups.
//
// To find the best K of n keys without sorting them: each thread's best of the keys that it holds, of
// these the K-th; keys that are not below it are a few more than K, and their places are counted.
#include "serve.hpp"
#include "logit_rows.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;          // ids of a chunk: 32 a thread
constexpr int kGroup = 32;            // ids of a group
constexpr int kGroups = kChunk / kGroup;
constexpr int kList = kMostTop * kGroup;  // keys whose places are counted, at most

struct Part {
  float m, sum, zsum;
  int above;
};

struct Args {
  const void* logits;
  int64_t ld;
  const int64_t* token;
  const float* temperature;
  int B, V, top, chunks;
  float *logprob, *entropy;
  int32_t* rank;
  int64_t* top_ids;
  float* top_logprobs;
  Part* part;     // [rows, chunks]
  float* groups;  // [rows, chunks, kGroups]
};

// 1 / T of a row, or 0 for greedy; without temperatures 1.
__device__ __forceinline__ double inverse_of(const Args& A, int64_t row) {
  const float t = A.temperature ? A.temperature[row / A.B] : 1.f;
  return t > 0.f ? fmax(1.0 / (double)t, 1e-300) : 0.0;
}

// A logit as it is ordered: NaN as -inf, and -0 as +0.
__device__ __forceinline__ float plain(float x) { return x != x ? -INFINITY : x + 0.f; }
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(plain(x));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Larger keys are in front: by value, then the lower index. (Never 0: an index is below 2^31.)
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  return (uint64_t)order_of(x) << 32 | (0xffffffffu - (uint32_t)index);
}
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

template <int N> __device__ __forceinline__ float max_of_lanes(float x) {
#pragma unroll
  for (int d = 1; d < N; d *= 2) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}

template <class T> __global__ __launch_bounds__(kThreads, 8) void chunks_kernel(Args A) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;  // K loads; as many lanes hold a group
  static_assert(K * E == kGroup, "a thread's ids are as many as a group's");
  const int c = blockIdx.x % A.chunks, t = threadIdx.x;
  const int64_t r = blockIdx.x / A.chunks;
  const int64_t token = A.token ? A.token[r] : 0;
  if (token < 0) return;
  const Row<T> row(static_cast<const T*>(A.logits) + r * A.ld, A.V);
  const float mine = A.token && token < A.V ? plain(to_f32<T>(row.x[token])) : INFINITY;
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
  int above = 0;
  float best = -INFINITY, m = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float g = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      g = fmaxf(g, x[k][e]);
      above += x[k][e] > mine ? 1 : 0;
    }
    m = fmaxf(m, g);
    g = max_of_lanes<K>(g);
    best = t % K == k ? g : best;
  }
  A.groups[(r * A.chunks + c) * kGroups + t % K * (kGroups / K) + t / K] = best;
  m = max_of_lanes<64>(m);
  const double inverse = inverse_of(A, r);
  const float c32 = (float)fmin(inverse * 1.4426950408889634, 1e37);
  float sum = 0.f, zsum = 0.f;
  if (m == INFINITY) {  // the ids that hold it share all
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) sum += x[k][e] == m ? 1.f : 0.f;
  } else if (m > -INFINITY && inverse != 0.0) {
    // (x - m first: near the maximum, where the weight is, the product then has no large terms that
    // cancel; the maximum with -1e30 turns NaN and -inf into no weight)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float z = fmaxf((x[k][e] - m) * c32, -1e30f), w = __builtin_amdgcn_exp2f(z);
        sum += w;
        zsum = fmaf(w, z, zsum);
      }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    sum += __shfl_xor(sum, d);
    zsum += __shfl_xor(zsum, d);
    above += __shfl_xor(above, d);
  }
  __shared__ Part s_part[kThreads / 64];
  if ((t & 63) == 0) s_part[t >> 6] = Part{m, sum, zsum, above};
  __syncthreads();
  if (t != 0) return;
  Part all = s_part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) all.m = fmaxf(all.m, s_part[i].m);
  all.sum = all.zsum = 0.f;
  all.above = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    const Part& p = s_part[i];
    all.above += p.above;
    if (p.m == -INFINITY || (all.m == INFINITY && p.m != INFINITY)) continue;
    const float z = p.m == all.m ? 0.f : fmaxf((p.m - all.m) * c32, -1e30f);
    const float f = __builtin_amdgcn_exp2f(z);
    all.sum += f * p.sum;
    all.zsum += f * fmaf(z, p.sum, p.zsum);
  }
  A.part[r * A.chunks + c] = all;
}

// Places of the n keys in `list` (all different); take(place, key) for the first `count` of them.
template <class F>
__device__ __forceinline__ void in_order(const uint64_t* list, int n, int count, F&& take) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = list[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += list[j] > key ? 1 : 0;
    if (place < count) take(place, key);
  }
}

template <class T> __global__ __launch_bounds__(kThreads) void finish_kernel(Args A) {
  const int64_t r = blockIdx.x;
  const int t = threadIdx.x;
  const int64_t token = A.token ? A.token[r] : 0;
  if (token < 0) {  // a slot without a token
    for (int k = t; k < A.top; k += kThreads) {
      A.top_ids[r * A.top + k] = -1;
      A.top_logprobs[r * A.top + k] = -INFINITY;
    }
    if (t == 0) {
      if (A.logprob) A.logprob[r] = 0.f;
      if (A.entropy) A.entropy[r] = 0.f;
      if (A.rank) A.rank[r] = -1;
    }
    return;
  }
  const Row<T> row(static_cast<const T*>(A.logits) + r * A.ld, A.V);
  const double inverse = inverse_of(A, r);
  const bool greedy = inverse == 0.0;
  // the row's sums, in every wave
  float m = -INFINITY;
  double sum = 0, zsum = 0;
  int above = 0;
  const Part* part = A.part + r * A.chunks;
  for (int i = t & 63; i < A.chunks; i += 64) m = fmaxf(m, part[i].m);
  m = max_of_lanes<64>(m);
  const double c = fmin(inverse * 1.4426950408889634, 1e37);
  for (int i = t & 63; i < A.chunks; i += 64) {
    const Part p = part[i];
    above += p.above;
    if (p.m == -INFINITY || (m == INFINITY && p.m != INFINITY)) continue;
    const double z = p.m == m ? 0.0 : ((double)p.m - (double)m) * c, f = exp2(z);
    sum += f * p.sum;
    if (f > 0) zsum += f * (z * p.sum + p.zsum);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    sum += __shfl_xor(sum, d);
    zsum += __shfl_xor(zsum, d);
    above += __shfl_xor(above, d);
  }
  const double log_sum = log(sum);
  // log p of a logit (greedy: of one that is not the first best)
  auto logp = [&](float x) {
    if (greedy || m == -INFINITY || x == -INFINITY || (m == INFINITY && x != m)) return -INFINITY;
    return (float)((x == m ? 0.0 : ((double)x - (double)m) * inverse) - log_sum);
  };

  __shared__ uint64_t s_list[kList];
  __shared__ int s_group[kMostTop];
  __shared__ uint64_t s_floor;
  __shared__ int s_n, s_first;
  const int n_groups = (int)(((int64_t)A.V + row.off + kGroup - 1) / kGroup);
  const int count = min(max(A.top, greedy ? 1 : 0), A.V), of_groups = min(count, n_groups);
  if (count > 0) {
    const float* groups = A.groups + r * A.chunks * kGroups;
    uint64_t best = 0;
    for (int g = t; g < n_groups; g += kThreads) best = max(best, key_of(groups[g], g));
    s_list[t] = best;
    if (t == 0) {
      s_floor = 0;
      s_n = 0;
    }
    __syncthreads();
    {
      int place = 0;
      for (int j = 0; j < kThreads; ++j) place += s_list[j] > best ? 1 : 0;
      if (best != 0 && place == of_groups - 1) s_floor = best;
    }
    __syncthreads();
    const uint64_t least = s_floor;
    for (int g = t; g < n_groups; g += kThreads) {
      const uint64_t key = key_of(groups[g], g);
      if (key < least) continue;
      const int at = atomicAdd(&s_n, 1);
      if (at < kList) s_list[at] = key;
    }
    __syncthreads();
    if (s_n <= kList) {
      in_order(s_list, s_n, of_groups, [&](int place, uint64_t key) {
        s_group[place] = index_of(key);
        if (place == of_groups - 1) s_floor = key;
      });
    } else {
      // more than the list holds, of very many groups whose best lie with few threads: one after the
      // other
      uint64_t last = ~0ull;
      for (int k = 0; k < of_groups; ++k) {
        best = 0;
        for (int g = t; g < n_groups; g += kThreads) {
          const uint64_t key = key_of(groups[g], g);
          if (key < last) best = max(best, key);
        }
        __syncthreads();
        s_list[t] = best;
        __syncthreads();
        for (int j = 0; j < kThreads; ++j) best = max(best, s_list[j]);
        last = best;
        if (t == 0) s_group[k] = index_of(best);
      }
      if (t == 0) s_floor = last;
    }
    __syncthreads();
    // ids below the last of as many groups as there are places are not among the first
    const uint32_t cut = of_groups == count ? (uint32_t)(s_floor >> 32) : 0u;
    if (t == 0) s_n = 0;
    __syncthreads();
    for (int i = t; i < of_groups * kGroup; i += kThreads) {
      const int64_t id = (int64_t)s_group[i / kGroup] * kGroup + i % kGroup - row.off;
      if (id < 0 || id >= A.V) continue;
      const float x = to_f32<T>(row.x[id]);
      if (order_of(x) >= cut) s_list[atomicAdd(&s_n, 1)] = key_of(x, (int)id);
    }
    __syncthreads();
    in_order(s_list, s_n, count, [&](int place, uint64_t key) {
      if (place == 0) s_first = index_of(key);
      if (place >= A.top) return;
      const float x = value_of((uint32_t)(key >> 32));
      A.top_ids[r * A.top + place] = index_of(key);
      A.top_logprobs[r * A.top + place] = greedy && place == 0 && m > -INFINITY ? 0.f : logp(x);
    });
    for (int k = count + t; k < A.top; k += kThreads) {
      A.top_ids[r * A.top + k] = -1;
      A.top_logprobs[r * A.top + k] = -INFINITY;
    }
    __syncthreads();
  }
  if (t != 0) return;
  if (A.entropy) {
    const bool none = greedy || m == -INFINITY;
    A.entropy[r] = none ? 0.f : (float)(log_sum - zsum / sum * 0.69314718055994531);
  }
  const bool inside = token < A.V;
  if (A.token && A.rank) A.rank[r] = inside ? above : -1;
  if (A.token && A.logprob) {
    float l = -INFINITY;
    if (inside) {
      if (greedy)
        l = token == s_first && m > -INFINITY ? 0.f : -INFINITY;
      else
        l = logp(plain(to_f32<T>(row.x[token])));
    }
    A.logprob[r] = l;
  }
}

template <class T> hipError_t launch_t(const Args& A, int rows, hipStream_t s) {
  hipLaunchKernelGGL(chunks_kernel<T>, dim3((unsigned)(rows * A.chunks)), dim3(kThreads), 0, s, A);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(finish_kernel<T>, dim3((unsigned)rows), dim3(kThreads), 0, s, A);
  return hipGetLastError();
}

int64_t chunks_of(int64_t V) { return (V + 7 + kChunk - 1) / kChunk; }

}  // namespace

int64_t logprobs_items(int64_t rows, int64_t V) { return rows * chunks_of(V); }

size_t logprobs_scratch_bytes(int64_t rows, int64_t V) {
  return (size_t)(rows * chunks_of(V)) * (sizeof(Part) + kGroups * sizeof(float));
}

hipError_t launch_token_logprobs(const void* logits, uint32_t dtype, int64_t ld, const int64_t* token,
                                 const float* temperature, int N, int B, int64_t V, int top,
                                 float* logprob, float* entropy, int32_t* rank, int64_t* top_ids,
                                 float* top_logprobs, void* ws, hipStream_t s) {
  const int rows = N * B;
  Args A{logits, ld, token, temperature, B, (int)V, top, (int)chunks_of(V), logprob, entropy, rank,
         top_ids, top_logprobs, static_cast<Part*>(ws), nullptr};
  A.groups = reinterpret_cast<float*>(A.part + (size_t)rows * A.chunks);
  switch (dtype) {
    case XPRESS_BF16: return launch_t<uint16_t>(A, rows, s);
    case XPRESS_F16: return launch_t<_Float16>(A, rows, s);
    default: return launch_t<float>(A, rows, s);
  }
}

}  // namespace xpress
