// Log probabilities of given tokens, with entropy, rank and the most likely alternatives (gfx950).
//
// With c = log2(e) / T, m the row's maximum and z_v = x_v c - m c, a row's sums are S = sum 2^z and
// Z = sum z 2^z: log p(v) = ln 2 (z_v - log2 S), entropy ln 2 (log2 S - Z / S). Rows are cut into
// chunks of kChunk ids; chunks_kernel reads each once and leaves its maximum, its sums, how many ids
// lie above the token, and the maxima of its groups of 32 ids. finish_kernel, a workgroup a row, joins
// the sums and finds the alternatives: the ids in front of the others, by value and then by id, lie
// in the groups whose own best ids are in front of the other groups'. So it takes the best groups by
// their maxima, and then the best ids of those groups.
//
// To find the best K of n values without sorting them: of the threads' own best ones the K-th, by a
// search over its bits; values that are not below it are a few more than K, and their places are
// counted.
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
  Part* part;    // [rows, chunks]
  void* groups;  // [rows, chunks, kGroups], of the logits' type
};

// What a row's temperature makes of its logits.
struct Scale {
  double inverse;  // 1 / T, 0 for greedy; without temperatures 1
  float c;         // log2(e) / T
  __device__ __forceinline__ Scale(const Args& A, int64_t row) {
    const float t = A.temperature ? A.temperature[row / A.B] : 1.f;
    inverse = t > 0.f ? fmax(1.0 / (double)t, 1e-300) : 0.0;
    c = (float)fmin(inverse * 1.4426950408889634, 1e37);
  }
  // Whether exponents are x c - unit in one operation, with the unit m c rounded: what its rounding is
  // off by is the same for all, and the sums' unit is what it was rounded to. Where m c is large, or c at
  // its limit, x - m comes first: the product then has no large terms that cancel, or overflow.
  __device__ __forceinline__ bool plain(float m) const { return fabsf(m * c) <= 0x1p20f && c < 1e30f; }
  __device__ __forceinline__ double unit(float m) const {
    return plain(m) ? (double)(m * c) : (double)m * (double)c;
  }
};

// A logit as it is ordered: NaN as -inf, and -0 as +0.
__device__ __forceinline__ float ordered(float x) { return x != x ? -INFINITY : x + 0.f; }
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(ordered(x));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Larger keys are in front: by value, then the lower index. (Never 0: an index is below 2^31.)
__device__ __forceinline__ uint64_t key_of(uint32_t order, int index) {
  return (uint64_t)order << 32 | (0xffffffffu - (uint32_t)index);
}
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

// Lanes d away (d a power of two) inside groups of eight, without the LDS's help.
template <int D> __device__ __forceinline__ float lane_xor(float x) {
  constexpr int P = D == 1 ? 0xB1 : D == 2 ? 0x4E : 0x141;  // quad_perm [1,0,3,2], [2,3,0,1]; half mirror
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), P, 0xf, 0xf, false));
}
// The maximum over N = 4 or 8 neighbouring lanes (of eight the second four, mirrored, have one value).
template <int N> __device__ __forceinline__ float max_of_group(float x) {
  x = fmaxf(x, lane_xor<1>(x));
  x = fmaxf(x, lane_xor<2>(x));
  return N == 4 ? x : fmaxf(x, lane_xor<4>(x));
}
template <int FROM> __device__ __forceinline__ float max_of_lanes(float x) {
#pragma unroll
  for (int d = FROM; d < 64; d *= 2) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}

template <class T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ uint16_t narrow(float x) { return __float_as_uint(x) >> 16; }
template <> __device__ __forceinline__ _Float16 narrow(float x) { return (_Float16)x; }
template <> __device__ __forceinline__ float narrow(float x) { return x; }

// Bound by HBM: 16 KiB of 16-bit logits a workgroup, eight workgroups a CU.
template <class T> __global__ __launch_bounds__(kThreads, 8) void chunks_kernel(Args A) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;  // K loads; as many lanes hold a group
  static_assert(K * E == kGroup, "a thread's ids are as many as a group's");
  const int c = blockIdx.x % A.chunks, t = threadIdx.x;
  const int64_t r = blockIdx.x / A.chunks;
  const int64_t token = A.token ? A.token[r] : 0;
  if (token < 0) return;
  const Row<T> row(static_cast<const T*>(A.logits) + r * A.ld, A.V);
  const float mine = A.token && token < A.V ? ordered(to_f32<T>(row.x[token])) : INFINITY;
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
    for (int e = 0; e < E; ++e) g = fmaxf(g, x[k][e]);
    if (__ballot(g > mine)) {  // (most pieces hold no id above a likely token)
#pragma unroll
      for (int e = 0; e < E; ++e) above += x[k][e] > mine ? 1 : 0;
    }
    g = max_of_group<K>(g);
    m = fmaxf(m, g);
    best = t % K == k ? g : best;
  }
  static_cast<T*>(A.groups)[(r * A.chunks + c) * kGroups + t % K * (kGroups / K) + t / K] =
      narrow<T>(best);
  m = max_of_lanes<K>(m);
  const Scale scale(A, r);
  float sum = 0.f, zsum = 0.f;
  if (m == INFINITY) {  // the ids that hold it share all
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) sum += x[k][e] == m ? 1.f : 0.f;
  } else if (m > -INFINITY && scale.inverse != 0.0) {
    // (the maximum with -1e30 turns NaN and -inf into no weight)
    auto add = [&](auto exponent) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float z = fmaxf(exponent(x[k][e]), -1e30f), w = __builtin_amdgcn_exp2f(z);
          sum += w;
          zsum = fmaf(w, z, zsum);
        }
    };
    if (scale.plain(m)) {
      const float unit = m * scale.c;
      add([&](float v) { return fmaf(v, scale.c, -unit); });
    } else {
      add([&](float v) { return (v - m) * scale.c; });
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
    const float z =
        p.m == all.m ? 0.f : fmaxf((float)(scale.unit(p.m) - scale.unit(all.m)), -1e30f);
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
#pragma unroll 8
    for (int j = 0; j < n; ++j) place += list[j] > key ? 1 : 0;
    if (place < count) take(place, key);
  }
}

// A 16-byte piece of the groups' maxima, E of them; past the last -inf's order and below all keys: 0.
template <class T> struct Best {
  static constexpr int E = Row<T>::E;
  uint32_t o[E];
  __device__ __forceinline__ void load(const void* groups, int64_t piece, int n) {
    const Piece<T> p =
        __builtin_bit_cast(Piece<T>, static_cast<const uint4*>(groups)[piece]);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = piece * E + e < n ? order_of(p[e]) : 0u;
  }
};

template <class T> __global__ __launch_bounds__(kThreads) void finish_kernel(Args A) {
  constexpr int E = Row<T>::E, HOLD = 32 / E;  // pieces that stay in a thread's registers
  const int64_t r = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63;
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
  const Scale scale(A, r);
  const bool greedy = scale.inverse == 0.0;
  const int n_groups = (int)(((int64_t)A.V + row.off + kGroup - 1) / kGroup);
  const int count = min(max(A.top, greedy ? 1 : 0), A.V), of_groups = min(count, n_groups);
  const int pieces = (n_groups + E - 1) / E;
  const T* groups = static_cast<const T*>(A.groups) + r * A.chunks * kGroups;
  Best<T> held[HOLD];
  if (count > 0) {
#pragma unroll
    for (int i = 0; i < HOLD; ++i) held[i].load(groups, min(t + i * kThreads, pieces - 1), n_groups);
  }
  // the row's sums, in every wave
  const float given = A.token && token < A.V ? ordered(to_f32<T>(row.x[token])) : -INFINITY;
  float m = -INFINITY;
  double sum = 0, zsum = 0;
  int above = 0;
  const Part* part = A.part + r * A.chunks;
  const Part mine = lane < A.chunks ? part[lane] : Part{-INFINITY, 0.f, 0.f, 0};
  for (int i = lane; i < A.chunks; i += 64) m = fmaxf(m, i == lane ? mine.m : part[i].m);
  m = max_of_lanes<1>(m);
  for (int i = lane; i < A.chunks; i += 64) {
    const Part p = i == lane ? mine : part[i];
    above += p.above;
    if (p.m == -INFINITY || (m == INFINITY && p.m != INFINITY)) continue;
    const double z = p.m == m ? 0.0 : scale.unit(p.m) - scale.unit(m), f = exp2(z);
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
  // of the sum relative to the maximum's own weight
  const double log_top =
      m == INFINITY ? log_sum
                    : log_sum - ((double)m * scale.c - scale.unit(m)) * 0.69314718055994531;
  // log p of a logit (greedy: of one that is not the first best)
  auto logp = [&](float x) {
    if (greedy || m == -INFINITY || x == -INFINITY || (m == INFINITY && x != m)) return -INFINITY;
    return (float)((x == m ? 0.0 : ((double)x - (double)m) * scale.inverse) - log_top);
  };

  __shared__ uint64_t s_list[kList];
  __shared__ uint32_t s_best[kThreads];
  __shared__ int s_group[kMostTop];
  __shared__ uint64_t s_floor;
  __shared__ int s_n, s_first;
  if (count > 0) {
    // all of this thread's maxima: f(order, index) of each
    auto each = [&](auto&& f) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (t + i * kThreads < pieces)
#pragma unroll
          for (int e = 0; e < E; ++e) f(held[i].o[e], (t + i * kThreads) * E + e);
      for (int i = t + HOLD * kThreads; i < pieces; i += kThreads) {
        Best<T> b;
        b.load(groups, i, n_groups);
#pragma unroll
        for (int e = 0; e < E; ++e) f(b.o[e], i * E + e);
      }
    };
    uint32_t top = 0;
    each([&](uint32_t o, int) { top = max(top, o); });
    s_best[t] = top;
    if (t == 0) s_n = 0;
    __syncthreads();
    // The largest value that as many threads' best ones reach as there are places (0: fewer threads
    // have any), one bit after the other, in every wave.
    uint32_t least = 0;
    {
      uint32_t b[kThreads / 64];
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) b[i] = s_best[lane + 64 * i];
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t next = least | 1u << bit;
        int n = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) n += __popcll(__ballot(b[i] >= next));
        if (n >= of_groups) least = next;
        if (n == of_groups) break;  // (no more than needed: what is above is as good)
      }
    }
    each([&](uint32_t o, int g) {
      if (o < least || o == 0) return;
      const int at = atomicAdd(&s_n, 1);
      if (at < kList) s_list[at] = key_of(o, g);
    });
    __syncthreads();
    if (s_n <= kList) {
      in_order(s_list, s_n, of_groups, [&](int place, uint64_t key) {
        s_group[place] = index_of(key);
        if (place == of_groups - 1) s_floor = key;
      });
    } else {
      // more than the list holds, as in a row of equal logits: one after the other
      uint64_t last = ~0ull;
      for (int k = 0; k < of_groups; ++k) {
        uint64_t best = 0;
        each([&](uint32_t o, int g) {
          const uint64_t key = o ? key_of(o, g) : 0;
          if (key < last) best = max(best, key);
        });
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
    for (int i0 = t; i0 < of_groups * kGroup; i0 += 4 * kThreads) {  // four loads in flight
      float x[4];
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * kThreads, g = s_group[min(i / kGroup, of_groups - 1)];
        const int64_t v = (int64_t)g * kGroup + i % kGroup - row.off;
        id[j] = i < of_groups * kGroup && v >= 0 && v < A.V ? (int)v : -1;
        x[j] = to_f32<T>(row.x[max(id[j], 0)]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (id[j] >= 0 && order_of(x[j]) >= cut)
          s_list[atomicAdd(&s_n, 1)] = key_of(order_of(x[j]), id[j]);
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
        l = logp(given);
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
  return (size_t)(rows * chunks_of(V)) * (sizeof(Part) + kGroups * sizeof(float));  // (of any type)
}

hipError_t launch_token_logprobs(const void* logits, uint32_t dtype, int64_t ld, const int64_t* token,
                                 const float* temperature, int N, int B, int64_t V, int top,
                                 float* logprob, float* entropy, int32_t* rank, int64_t* top_ids,
                                 float* top_logprobs, void* ws, hipStream_t s) {
  const int rows = N * B;
  Args A{logits, ld, token, temperature, B, (int)V, top, (int)chunks_of(V), logprob, entropy, rank,
         top_ids, top_logprobs, static_cast<Part*>(ws), nullptr};
  A.groups = A.part + (size_t)rows * A.chunks;
  switch (dtype) {
    case XPRESS_BF16: return launch_t<uint16_t>(A, rows, s);
    case XPRESS_F16: return launch_t<_Float16>(A, rows, s);
    default: return launch_t<float>(A, rows, s);
  }
}

}  // namespace xpress
