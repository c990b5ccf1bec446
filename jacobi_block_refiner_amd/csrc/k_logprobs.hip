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
// counted. Where they are very many, as in rows that are masked but for a few ids, values above it come
// first, then the first by index of those that equal it.
#include "serve.hpp"
#include "logit_rows.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;          // ids of a chunk: 32 a thread
constexpr int kGroup = 32;            // ids of a group
constexpr int kGroups = kChunk / kGroup;
constexpr int kWaves = kThreads / 64;  // of a chunk, each with sums of its own
constexpr int kFinish = 8;            // workgroups of finish_kernel on a CU
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
  Part* part;    // [rows, chunks, kWaves]
  void* groups;  // [rows, chunks, kGroups], of the logits' type
};

// What a row's temperature makes of its logits.
struct Scale {
  float t;  // 0 for greedy; without temperatures 1
  float c;  // log2(e) / t
  __device__ __forceinline__ Scale(const Args& A, int64_t row) {
    t = A.temperature ? A.temperature[(uint32_t)row / (uint32_t)A.B] : 1.f;  // (below 2^24 rows)
    t = t > 0.f ? t : 0.f;
    c = fminf(1.44269504f / t, 1e37f);
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

// Maxima of numbers. (fmaxf quiets what could be a signalling NaN first, an operation more for each.)
__device__ __forceinline__ float max_of(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ float max_of(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
// A neighbouring lane's value, without the LDS's help.
template <int P> __device__ __forceinline__ float lane_by(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), P, 0xf, 0xf, false));
}
// The maximum over N = 4 or 8 neighbouring lanes.
template <int N> __device__ __forceinline__ float max_of_group(float x) {
  x = max_of(x, lane_by<0xB1>(x));                        // quad_perm 1 0 3 2
  x = max_of(x, lane_by<0x4E>(x));                        // quad_perm 2 3 0 1
  return N == 4 ? x : max_of(x, lane_by<0x141>(x));  // half mirror
}
// f(x, y) of all lanes: neighbours by DPP, whole rows of 16 through the LDS's crossbar.
template <class F> __device__ __forceinline__ uint32_t of_wave(uint32_t x, F&& f) {
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0xB1, 0xf, 0xf, false));   // quad_perm 1 0 3 2
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x4E, 0xf, 0xf, false));   // quad_perm 2 3 0 1
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x141, 0xf, 0xf, false));  // half mirror
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x140, 0xf, 0xf, false));  // mirror
  x = f(x, (uint32_t)__shfl_xor((int)x, 16));
  return f(x, (uint32_t)__shfl_xor((int)x, 32));
}
__device__ __forceinline__ float wave_max(float x) {
  return __uint_as_float(of_wave(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(max_of(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float x) {
  return __uint_as_float(of_wave(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ int wave_sum(int x) {
  return (int)of_wave((uint32_t)x, [](uint32_t a, uint32_t b) { return a + b; });
}

template <class T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ uint16_t narrow(float x) { return __float_as_uint(x) >> 16; }
template <> __device__ __forceinline__ _Float16 narrow(float x) { return (_Float16)x; }
template <> __device__ __forceinline__ float narrow(float x) { return x; }

// One chunk of one row, 16 KiB of 16-bit logits; each wave leaves sums of its own. Bound by HBM, close to
// the vector unit's 290 operations a wave: 2048 rows of 151,936 ids 118 us, at the rate of a copy 120 to
// 130 (which writes too). With quieted maxima, a join of the waves and bounds checks of every piece 430
// operations, and 14 us more. Workgroups that go on from chunk to chunk and ask for the next one's logits
// ahead were slower by half.
template <class T> __global__ __launch_bounds__(kThreads, 8) void chunks_kernel(Args A) {
  constexpr int E = Row<T>::E, K = kChunk / kThreads / E;  // K loads; as many lanes hold a group
  static_assert(K * E == kGroup, "a thread's ids are as many as a group's");
  const int c = blockIdx.x % A.chunks, t = threadIdx.x;
  const int64_t r = blockIdx.x / A.chunks;
  const int64_t token = A.token ? A.token[r] : 0;
  if (token < 0) return;
  const Row<T> row(static_cast<const T*>(A.logits) + r * A.ld, A.V);
  const float mine = A.token && token < A.V ? ordered(to_f32<T>(row.x[token])) : INFINITY;
  Piece<T> p[K];
  const int64_t first = (int64_t)c * kChunk - row.off;
  if (first >= 0 && first + kChunk <= A.V) {
    const uint4* from = reinterpret_cast<const uint4*>(row.x + first) + t;
#pragma unroll
    for (int k = 0; k < K; ++k) p[k] = __builtin_bit_cast(Piece<T>, from[k * kThreads]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) p[k] = row.load((int64_t)c * (kChunk / E) + k * kThreads + t);
  }
  float x[K][E];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[k][e] = p[k][e];
      asm("" : "+v"(x[k][e]));  // (fp16: or both the halves and their values stay live, and spill)
    }
  const Scale scale(A, r);
  int above;
  float m, sum, zsum;
  // What the chunk leaves, of x as it is: numbers.
  auto maxima = [&]() __attribute__((always_inline)) {
    above = 0;
    m = -INFINITY;
    float best = -INFINITY;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g = max_of(x[k][0], x[k][1]);
#pragma unroll
      for (int e = 2; e < E; e += 2) g = max_of(g, x[k][e], x[k][e + 1]);
      if (__ballot(g > mine)) {  // (most pieces hold no id above a likely token)
#pragma unroll
        for (int e = 0; e < E; ++e) above += x[k][e] > mine ? 1 : 0;
      }
      g = max_of_group<K>(g);
      m = max_of(m, g);
      best = t % K == k ? g : best;
    }
    static_cast<T*>(A.groups)[(r * A.chunks + c) * kGroups + t % K * (kGroups / K) + t / K] =
        narrow<T>(best);
    m = wave_max(m);
  };
  auto sums = [&](auto exponent) __attribute__((always_inline)) {
    sum = zsum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float z = exponent(x[k][e]), w = __builtin_amdgcn_exp2f(z);
        sum += w;
        zsum = fmaf(w, fmaxf(z, -1e30f), zsum);  // (-inf: no weight, and no NaN of it)
      }
  };
  maxima();
  bool care = !scale.plain(m) || scale.t == 0.f;
  if (!care) {
    const float unit = m * scale.c;
    sums([&](float v) { return fmaf(v, scale.c, -unit); });
    // (a NaN is in the sum. Asked of both, or the second is formed behind the branch and its terms kept
    // until then: twice the registers.)
    care = __ballot(!(sum >= zsum)) != 0;
  }
  // Once more with care for NaN, an infinite maximum, and where the scale asks for it.
  if (care) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) x[k][e] = ordered(x[k][e]);
    maxima();
    sum = zsum = 0.f;
    if (m == INFINITY) {  // the ids that hold it share all
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) sum += x[k][e] == m ? 1.f : 0.f;
    } else if (m > -INFINITY && scale.t != 0.f) {
      const float unit = m * scale.c;
      // (-1e30 for what an infinite temperature makes of -inf)
      if (scale.plain(m))
        sums([&](float v) { return fmaxf(fmaf(v, scale.c, -unit), -1e30f); });
      else
        sums([&](float v) { return fmaxf((v - m) * scale.c, -1e30f); });
    }
  }
  sum = wave_sum(sum);
  zsum = wave_sum(zsum);
  above = wave_sum(above);
  if (t % 64 == 0) A.part[(r * A.chunks + c) * kWaves + t / 64] = Part{m, sum, zsum, above};
}

// Places of the n keys in `list` (all different); take(place, key) for the first `count` of them. Four
// threads a key.
template <class F>
__device__ __forceinline__ void in_order(const uint64_t* list, int n, int count, F&& take) {
  const int part = threadIdx.x & 3;
  for (int i = threadIdx.x >> 2; i < n; i += kThreads / 4) {
    const uint64_t key = list[i];
    int place = 0;
#pragma unroll 4
    for (int j = part; j < n; j += 4) place += list[j] > key ? 1 : 0;
    place += __builtin_amdgcn_update_dpp(0, place, 0xB1, 0xf, 0xf, false);  // quad_perm 1 0 3 2
    place += __builtin_amdgcn_update_dpp(0, place, 0x4E, 0xf, 0xf, false);  // quad_perm 2 3 0 1
    if (part == 0 && place < count) take(place, key);
  }
}

// The best `count` of the n keys in `list` (all different, n >= count): take(place, key). Of many, the least
// that counts is searched for first, by its bits: 256 keys are as quick without.
template <class F>
__device__ __forceinline__ void best_of(const uint64_t* list, int n, int count, F&& take) {
  __shared__ uint64_t s_keep[kMostTop];
  __shared__ int s_count[2][kWaves], s_kept;
  if (n <= kThreads) return in_order(list, n, count, take);
  const int t = threadIdx.x;
  if (t == 0) s_kept = 0;
  uint64_t mine[kList / kThreads], least = 0;
#pragma unroll
  for (int i = 0; i < kList / kThreads; ++i) mine[i] = t + i * kThreads < n ? list[t + i * kThreads] : 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t next = least | 1ull << bit;
    int above = 0;
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i) above += __popcll(__ballot(mine[i] >= next));
    // (two sets: the last but one was read before the last meeting)
    if (t % 64 == 0) s_count[bit & 1][t / 64] = above;
    __syncthreads();
    above = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) above += s_count[bit & 1][w];
    if (above >= count) least = next;
    if (above == count) break;
  }
#pragma unroll
  for (int i = 0; i < kList / kThreads; ++i)
    if (mine[i] >= least && mine[i]) s_keep[atomicAdd(&s_kept, 1)] = mine[i];
  __syncthreads();
  in_order(s_keep, count, count, take);
}

// A row's end: dependent loads and meetings of about 9 us, so few registers, for many rows at a time. The
// sums, in 64 bits, are one wave's work beside the search of another (in every wave, before the search:
// 9.7 us instead of 9.2 for one row of 151,936 ids with 20 alternatives, 20 instead of 17.2 for 2048 rows
// with 5). The maxima held in registers between their two uses spill: 24 us for the 2048 rows.
template <class T> __global__ __launch_bounds__(kThreads, kFinish) void finish_kernel(Args A) {
  constexpr int E = Row<T>::E;
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
  const bool greedy = scale.t == 0.f;
  const int n_groups = (int)(((int64_t)A.V + row.off + kGroup - 1) / kGroup);
  const int count = min(max(A.top, greedy ? 1 : 0), A.V), of_groups = min(count, n_groups);
  const int pieces = (n_groups + E - 1) / E;
  const uint4* groups = reinterpret_cast<const uint4*>(static_cast<const T*>(A.groups) +
                                                       r * A.chunks * kGroups);
  const float given = A.token && token < A.V ? ordered(to_f32<T>(row.x[token])) : -INFINITY;
  __shared__ double s_sums[3];  // maximum, log of the sum, entropy
  __shared__ int s_above;
  // The row's sums, by the second wave (while the first looks for the best groups).
  auto join = [&] {
    const Part* part = A.part + r * A.chunks * kWaves;
    const int parts = A.chunks * kWaves;
    const Part mine = lane < parts ? part[lane] : Part{-INFINITY, 0.f, 0.f, 0};
    float m = -INFINITY;
    double sum = 0, zsum = 0;
    int above = 0;
    for (int i = lane; i < parts; i += 64) m = fmaxf(m, i == lane ? mine.m : part[i].m);
    m = wave_max(m);
    for (int i = lane; i < parts; i += 64) {
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
    }
    above = wave_sum(above);
    if (lane) return;
    const double log_sum = log(sum);
    s_sums[0] = m;
    // of the sum relative to the maximum's own weight
    s_sums[1] = m == INFINITY
                    ? log_sum
                    : log_sum - ((double)m * scale.c - scale.unit(m)) * 0.69314718055994531;
    s_sums[2] = log_sum - zsum / sum * 0.69314718055994531;
    s_above = above;
  };
  // log p of a logit (greedy: of one that is not the first best). Where one id has nearly all, the rounding
  // of its 32-bit weight is all that is left of the sum's logarithm, of either sign: no p is above 1.
  auto logp = [&](float x) {
    const float m = (float)s_sums[0];
    if (greedy || m == -INFINITY || x == -INFINITY || (m == INFINITY && x != m)) return -INFINITY;
    return fminf((float)((x == m ? 0.0 : ((double)x - (double)m) / scale.t) - s_sums[1]), 0.f);
  };

  __shared__ uint64_t s_list[kList];
  __shared__ uint32_t s_best[kThreads];
  __shared__ int s_group[kMostTop];
  __shared__ uint64_t s_floor;
  __shared__ int s_n, s_ids, s_first;
  __shared__ uint32_t s_least;
  __shared__ int s_part[kWaves];
  if (count > 0) {
    // all of this thread's maxima: f(order, index) of each
    auto piece = [&](const uint4& u, int i, auto&& f) {
      const Piece<T> p = __builtin_bit_cast(Piece<T>, u);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (i * E + e < n_groups) f(order_of(p[e]), i * E + e);
    };
    auto each = [&](auto&& f) {
      for (int i0 = t; i0 < pieces; i0 += 4 * kThreads) {  // four loads in flight
        uint4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = groups[min(i0 + i * kThreads, pieces - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i0 + i * kThreads < pieces) piece(u[i], i0 + i * kThreads, f);
      }
    };
    uint32_t top = 0;
    each([&](uint32_t o, int) { top = max(top, o); });
    s_best[t] = top;
    if (t == 0) s_n = s_ids = 0;
    __syncthreads();
    // The largest value that as many threads' best ones reach as there are places (0: fewer threads
    // have any), one bit after the other, by the first wave.
    if (t < 64) {
      uint32_t b[kThreads / 64], least = 0;
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
      s_least = least;
    } else if (t < 128) {
      join();
    }
    __syncthreads();
    const uint32_t least = s_least;
    each([&](uint32_t o, int g) {
      if (o < least) return;
      const int at = atomicAdd(&s_n, 1);
      if (at < kList) s_list[at] = key_of(o, g);
    });
    __syncthreads();
    int n = s_n;
    if (n > kList) {
      // once more without those that equal it, of which the first are then looked for in their order
      __syncthreads();
      if (t == 0) s_n = 0;
      __syncthreads();
      each([&](uint32_t o, int g) {
        if (o <= least) return;
        const int at = atomicAdd(&s_n, 1);
        if (at < kList) s_list[at] = key_of(o, g);
      });
      __syncthreads();
      n = s_n;
      for (int i0 = 0; n < of_groups && i0 < pieces; i0 += kThreads) {
        uint32_t equal = 0;
        if (i0 + t < pieces)
          piece(groups[i0 + t], i0 + t, [&](uint32_t o, int g) { equal |= (o == least) << g % E; });
        int before = __popc(equal);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const int y = __shfl_up(before, d);
          if (lane >= d) before += y;
        }
        if (lane == 63) s_part[t / 64] = before;
        __syncthreads();
        before -= __popc(equal);
        int all = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          if (w < t / 64) before += s_part[w];
          all += s_part[w];
        }
        for (; equal && n + before < of_groups; equal &= equal - 1, ++before)
          s_list[n + before] = key_of(least, (i0 + t) * E + __ffs(equal) - 1);
        n = min(n + all, of_groups);
        __syncthreads();
      }
    }
    if (n <= kList) {
      best_of(s_list, n, of_groups, [&](int place, uint64_t key) {
        s_group[place] = index_of(key);
        if (place == of_groups - 1) s_floor = key;
      });
    } else {
      // more than the list holds: one after the other
      uint64_t last = ~0ull;
      for (int k = 0; k < of_groups; ++k) {
        uint64_t best = 0;
        each([&](uint32_t o, int g) {
          const uint64_t key = key_of(o, g);
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
    const int n_ids = of_groups * kGroup;
    for (int i0 = t; i0 < n_ids; i0 += 4 * kThreads) {  // four loads in flight
      float x[4];
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * kThreads, g = s_group[min(i / kGroup, of_groups - 1)];
        const int64_t v = (int64_t)g * kGroup + i % kGroup - row.off;
        id[j] = i < n_ids && v >= 0 && v < A.V ? (int)v : -1;
        x[j] = to_f32<T>(row.x[max(id[j], 0)]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (id[j] >= 0 && order_of(x[j]) >= cut)
          s_list[atomicAdd(&s_ids, 1)] = key_of(order_of(x[j]), id[j]);
    }
    __syncthreads();
    best_of(s_list, s_ids, count, [&](int place, uint64_t key) {
      if (place == 0) s_first = index_of(key);
      if (place >= A.top) return;
      const float x = value_of((uint32_t)(key >> 32));
      A.top_ids[r * A.top + place] = index_of(key);
      A.top_logprobs[r * A.top + place] = greedy && place == 0 && s_sums[0] > -INFINITY ? 0.f : logp(x);
    });
    for (int k = count + t; k < A.top; k += kThreads) {
      A.top_ids[r * A.top + k] = -1;
      A.top_logprobs[r * A.top + k] = -INFINITY;
    }
    __syncthreads();
  } else {
    if (t >= 64 && t < 128) join();
    __syncthreads();
  }
  if (t != 0) return;
  if (A.entropy) {
    const bool none = greedy || s_sums[0] == -INFINITY;
    A.entropy[r] = none ? 0.f : fmaxf((float)s_sums[2], 0.f);  // (as a log p's end at 0)
  }
  const bool inside = token < A.V;
  if (A.token && A.rank) A.rank[r] = inside ? s_above : -1;
  if (A.token && A.logprob) {
    float l = -INFINITY;
    if (inside) {
      if (greedy)
        l = token == s_first && s_sums[0] > -INFINITY ? 0.f : -INFINITY;
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
  return (size_t)(rows * chunks_of(V)) * (kWaves * sizeof(Part) + kGroups * sizeof(float));  // (of any type)
}

hipError_t launch_token_logprobs(const void* logits, uint32_t dtype, int64_t ld, const int64_t* token,
                                 const float* temperature, int N, int B, int64_t V, int top,
                                 float* logprob, float* entropy, int32_t* rank, int64_t* top_ids,
                                 float* top_logprobs, void* ws, hipStream_t s) {
  const int rows = N * B;
  Args A{logits, ld, token, temperature, B, (int)V, top, (int)chunks_of(V), logprob, entropy, rank,
         top_ids, top_logprobs, static_cast<Part*>(ws), nullptr};
  A.groups = A.part + (size_t)rows * A.chunks * kWaves;
  switch (dtype) {
    case XPRESS_BF16: return launch_t<uint16_t>(A, rows, s);
    case XPRESS_F16: return launch_t<_Float16>(A, rows, s);
    default: return launch_t<float>(A, rows, s);
  }
}

}  // namespace xpress
