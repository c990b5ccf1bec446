// Pages of the K/V cache (gfx950): fork, extension with copy on write, append, freeing and
// compaction. The metadata (tables, lengths, counts) is integer work of a few KB, so its kernels take
// the time of a launch and of the loads that wait for one another (row -> length -> table entry ->
// holders, close to 1 us each): what does not depend on such a load is asked for before it. The
// copies are plain 16-byte streams. 32 rows of about 8600 tokens, 6 of them forks, in pages of 64
// tokens of 4 layers of 8 heads of 128: fork 3.9 us, extension 6.0 and its copies (a dozen pages of 1
// MiB at most) 6.4, append of 16 tokens 3.2 a layer, trim 2.3. A launch takes 3 to 4 us on the host,
// so a turn that is not captured into a graph is bound by its launches.
#include "serve.hpp"
#include "cache_index.hpp"

#include <algorithm>

#include <limits.h>

namespace xpress {

namespace {

constexpr int kPlan = 1024;  // threads of the single workgroup that plans an allocation
constexpr int kScan = 4;     // counts of a thread in a step of a walk over the pool

int shift_of(int page) { return __builtin_ctz((unsigned)page); }

// What the kernels need of an xpress_cache.
struct Pages {
  int32_t *table, *len, *ref;
  int rows, ld, n_pages, shift;
};

Pages pages(const xpress_cache& c) {
  return Pages{c.table, c.len, c.ref, c.rows, c.table_ld, c.n_pages, shift_of(c.page)};
}

__device__ __forceinline__ int row_of(const int32_t* seq, int i, int rows) {
  const int r = seq ? seq[i] : i;
  return (unsigned)r < (unsigned)rows ? r : -1;
}

// Exclusive prefix sum over the workgroup's kPlan threads; *total gets the sum.
__device__ int block_scan(int v, int* total) {
  __shared__ int s_part[kPlan / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the previous call's s_part has been read
  if (lane == 63) s_part[w] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlan / 64; ++i) {
    const int p = s_part[i];
    before += i < w ? p : 0;
    all += p;
  }
  *total = all;
  return before + x - v;
}

// Sum of v over the waves before this one (v is the same in a wave's lanes); *total gets the sum.
__device__ __forceinline__ int waves_before(int v, int* total) {
  __shared__ int s_part[kPlan / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  __syncthreads();  // the previous call's s_part has been read
  if (lane == 0) s_part[w] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlan / 64; ++i) {
    const int p = s_part[i];
    before += i < w ? p : 0;
    all += p;
  }
  *total = all;
  return before;
}

// A walk over the pool's counts takes kPlan * kScan pages a step; a wave has kScan * 64 of them in a
// row, each lane every 64th, so that a ballot gives the ranks in id order. Pages past the pool count -1.
__device__ __forceinline__ int walk_at(int p0, int i) {
  return p0 + (threadIdx.x >> 6) * kScan * 64 + i * 64 + (threadIdx.x & 63);
}
__device__ __forceinline__ void counts_at(const Pages& P, int p0, int* ref) {
#pragma unroll
  for (int i = 0; i < kScan; ++i) {
    const int p = walk_at(p0, i);
    ref[i] = p < P.n_pages ? holders(P.ref[p]) : -1;
  }
}
__device__ __forceinline__ int lanes_before(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// One workgroup a row; a thread an entry. The lengths are needed for the counts alone, so the entries
// are read beside them.
__global__ __launch_bounds__(256) void fork_kernel(Pages P, const int32_t* src, const int32_t* dst) {
  const int from = row_of(src, blockIdx.x, P.rows), to = row_of(dst, blockIdx.x, P.rows);
  if (from < 0 || to < 0 || from == to) return;
  const int old_len = clamp_len(P.len[to], P.ld, P.shift);
  const int new_len = clamp_len(P.len[from], P.ld, P.shift);
  const int old_pages = pages_of(old_len, P.shift), new_pages = pages_of(new_len, P.shift);
  const int32_t* a = P.table + (int64_t)from * P.ld;
  int32_t* b = P.table + (int64_t)to * P.ld;
  for (int j = threadIdx.x; j < P.ld; j += blockDim.x) {
    const int old = b[j], id = a[j];  // (the first of these loads do not wait for the lengths)
    if (j < old_pages && page_ok(old, P.n_pages)) atomicSub(&P.ref[old], 1);
    if (j < new_pages && page_ok(id, P.n_pages)) atomicAdd(&P.ref[id], 1);
    b[j] = id;
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) P.len[to] = new_len;
}

__global__ __launch_bounds__(256) void trim_kernel(Pages P, const int32_t* lacking,
                                                   const int32_t* seq, const int32_t* drop) {
  const int no = lacking ? *lacking : 0;
  const int r = row_of(seq, blockIdx.x, P.rows);
  if (r < 0 || no) return;
  const int len = clamp_len(P.len[r], P.ld, P.shift);
  const int d = drop ? min(max(drop[blockIdx.x], 0), len) : len;
  __syncthreads();  // every thread has read the length
  int32_t* t = P.table + (int64_t)r * P.ld;
  const int keep = pages_of(len - d, P.shift), had = pages_of(len, P.shift);
  for (int j = keep + threadIdx.x; j < had; j += blockDim.x) {
    const int id = t[j];
    if (page_ok(id, P.n_pages)) atomicSub(&P.ref[id], 1);
    t[j] = -1;
  }
  if (threadIdx.x == 0) P.len[r] = len - d;
}

// What a row asks for: whether its partly filled last page is shared (cow), and its pages.
struct Need {
  int len, after, first, count;  // new pages go to table entries first .. first+count-1
  bool cow;
};
__device__ Need need_of(const Pages& P, const int32_t* seq, const int32_t* add, int add_all, int i,
                        int* r_out) {
  Need n{0, 0, 0, 0, false};
  const int r = row_of(seq, i, P.rows);
  *r_out = r;
  if (r < 0) return n;
  n.len = clamp_len(P.len[r], P.ld, P.shift);
  const int64_t after = (int64_t)n.len + max(add ? add[i] : add_all, 0);
  if (after > ((int64_t)P.ld << P.shift)) {
    n.count = -1;
    return n;
  }
  n.after = (int)after;
  n.first = pages_of(n.len, P.shift);
  if (after > n.len && (n.len & ((1 << P.shift) - 1))) {
    const int id = P.table[(int64_t)r * P.ld + n.first - 1];
    n.cow = page_ok(id, P.n_pages) && P.ref[id] > 1;
  }
  n.first -= n.cow;
  n.count = pages_of(after, P.shift) - n.first;
  return n;
}

// Scratch of an extension: how many copies there are at most (0 where nothing is changed); by list
// entry the copy's source (-1: none) and target, the first table entry and the number of the new
// pages and their offset in the list of free pages; that list.
struct ExtendScratch {
  int32_t *ncopy, *from, *to, *first, *count, *offset, *free_ids;
};
constexpr int kExtendPerRow = 5;
__host__ __device__ inline ExtendScratch extend_scratch(void* ws, int N) {
  int32_t* p = static_cast<int32_t*>(ws);
  const int64_t n = N;
  return ExtendScratch{p,         p + 4,         p + 4 + n,     p + 4 + 2 * n, p + 4 + 3 * n,
                       p + 4 + 4 * n, p + 4 + 5 * n};
}

// The copies are a launch of their own: they need the plan of all rows, and a flag to wait for it
// would need a workspace that the caller has cleared.
// One workgroup: the rows' needs in list order (prefix sums), the first `total` free pages in id
// order, then the tables. The whole plan is made before anything is written.
__global__ __launch_bounds__(kPlan) void extend_kernel(Pages P, const int32_t* seq, int N,
                                                       const int32_t* add, int add_all,
                                                       int32_t* lacking, void* ws) {
  const ExtendScratch S = extend_scratch(ws, N);
  const int t = threadIdx.x;
  int ref[kScan];
  counts_at(P, 0, ref);  // in flight beside the rows' loads
  __shared__ int s_over;
  if (t == 0) s_over = 0;
  __syncthreads();
  int64_t total = 0;
  for (int i0 = 0; i0 < N; i0 += kPlan) {
    const int i = i0 + t;
    int r, all;
    const Need n = i < N ? need_of(P, seq, add, add_all, i, &r) : Need{0, 0, 0, 0, false};
    if (n.count < 0) s_over = 1;
    const int at = block_scan(max(n.count, 0), &all);
    if (i < N) {
      S.offset[i] = (int)min(total + at, (int64_t)P.n_pages);
      S.first[i] = n.first;
      S.count[i] = n.count;
      S.from[i] = n.cow ? P.table[(int64_t)r * P.ld + n.first] : -1;
    }
    total += all;
  }
  __syncthreads();
  int found = 0;
  const int want = (int)min(total, (int64_t)P.n_pages);
  if (!s_over)
    for (int p0 = 0; p0 < P.n_pages && found < want; p0 += kPlan * kScan) {
      if (p0) counts_at(P, p0, ref);
      uint64_t is_free[kScan];
      int mine = 0, all;
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        is_free[i] = __ballot(ref[i] == 0);
        mine += __popcll(is_free[i]);
      }
      int k = found + waves_before(mine, &all);
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        const int at = k + lanes_before(is_free[i]);
        if (ref[i] == 0 && at < want) S.free_ids[at] = walk_at(p0, i);
        k += __popcll(is_free[i]);
      }
      found += all;
    }
  const bool no = s_over || found < total;
  if (t == 0) {
    *lacking = s_over ? -1 : pages_missing(total, found);
    *S.ncopy = no ? 0 : N;
  }
  if (no) return;
  __syncthreads();
  for (int i0 = 0; i0 < N; i0 += kPlan) {
    const int i = i0 + t;
    if (i >= N) continue;
    const int r = row_of(seq, i, P.rows);
    if (r < 0) continue;
    const int old = S.from[i], first = S.first[i], count = S.count[i];
    int32_t* row = P.table + (int64_t)r * P.ld;
    for (int j = 0; j < count; ++j) {
      const int id = S.free_ids[S.offset[i] + j];
      row[first + j] = id;
      P.ref[id] = 1;
    }
    if (old >= 0) {
      atomicSub(&P.ref[old], 1);
      S.to[i] = row[first];
    }
    const int64_t after = (int64_t)clamp_len(P.len[r], P.ld, P.shift) + max(add ? add[i] : add_all, 0);
    P.len[r] = clamp_len((int)min(after, (int64_t)INT_MAX), P.ld, P.shift);
  }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kCopy = 8;  // loads of a thread in flight: 32 KB a workgroup (with one, a
                           // dozen pages of 1 MiB took 9.2 us instead of 6.4, 512 of them 221
                           // instead of 213)

// Page copies from[i] -> to[i], i < *count, in every layer of K and V.
struct Copies {
  const int32_t *count, *from, *to;
  u32x4 *k, *v;
  int n_layers;
  int64_t n_pages, chunks;  // 16-byte pieces of a page
};

// One workgroup per (page, layer and side) at a time. 537 MB read and as much written: 213 us, 5.0
// TB/s, the rate of a copy of 4 GiB.
__device__ __forceinline__ void copy_pages(const Copies& C, unsigned first, unsigned step) {
  const int64_t items = (int64_t)*C.count * C.n_layers * 2;
  for (int64_t it = first; it < items; it += step) {
    const int i = (int)(it / (C.n_layers * 2)), side = (int)(it % (C.n_layers * 2));
    const int a = C.from[i];
    if (a < 0) continue;
    u32x4* pool = (side & 1 ? C.v : C.k) + (int64_t)(side >> 1) * C.n_pages * C.chunks;
    const u32x4* x = pool + a * C.chunks;
    u32x4* y = pool + C.to[i] * C.chunks;
    int j = threadIdx.x;
    for (; j + 256 * (kCopy - 1) < C.chunks; j += 256 * kCopy) {
      u32x4 c[kCopy];
#pragma unroll
      for (int u = 0; u < kCopy; ++u) c[u] = x[j + u * 256];
#pragma unroll
      for (int u = 0; u < kCopy; ++u) y[j + u * 256] = c[u];
    }
    for (; j < C.chunks; j += 256) y[j] = x[j];
  }
}
__global__ __launch_bounds__(256) void copy_pages_kernel(Copies C) {
  copy_pages(C, blockIdx.x, gridDim.x);
}

// A thread a 16-byte piece of a token. The new values and `lacking` are read beside the row's length
// and table.
__global__ __launch_bounds__(256) void append_kernel(Pages P, const int32_t* lacking, uint16_t* k,
                                                     uint16_t* v,
                                                     const uint16_t* __restrict__ k_new,
                                                     const uint16_t* __restrict__ v_new,
                                                     int64_t ld_new, const int32_t* seq, int N,
                                                     int B, int Hkv, int D) {
  const unsigned per = Hkv * D / 8;  // 16-byte pieces of a token
  const unsigned i = blockIdx.x * 256u + threadIdx.x;  // (below 2^31: N*B*Hkv is below 2^26)
  if (i >= (unsigned)N * B * per) return;
  const unsigned token = i / per, piece = i % per;
  const int e = token / (unsigned)B, b = token % (unsigned)B;
  const uint4 x = *reinterpret_cast<const uint4*>((blockIdx.y ? v_new : k_new) +
                                                  (int64_t)token * ld_new + piece * 8);
  const int no = lacking ? *lacking : 0;
  const int r = row_of(seq, e, P.rows);
  if (r < 0 || no) return;
  const int pos = in_sight(clamp_len(P.len[r], P.ld, P.shift), B, b) - 1;
  if (pos < 0) return;
  const int id = P.table[(int64_t)r * P.ld + (pos >> P.shift)];
  if (!page_ok(id, P.n_pages)) return;
  const int h = piece * 8 / (unsigned)D, d = piece * 8 % (unsigned)D;
  const int64_t to = line_offset(id, h, pos & ((1 << P.shift) - 1), Hkv, P.shift, D) + d;
  *reinterpret_cast<uint4*>((blockIdx.y ? v : k) + to) = x;
}

// Scratch of a compaction: the number of moves, the moves, and where each page goes.
struct CompactScratch {
  int32_t *nmove, *from, *to, *place;
};
__host__ __device__ inline CompactScratch compact_scratch(void* ws, int n_pages) {
  int32_t* p = static_cast<int32_t*>(ws);
  return CompactScratch{p, p + 4, p + 4 + n_pages, p + 4 + 2 * (int64_t)n_pages};
}

// One workgroup, two walks over the counts: how many pages live (L), then the live ones from L on and
// the free ones before it, which pair up in id order. 4.8 us for 2048 pages.
__global__ __launch_bounds__(kPlan) void compact_plan_kernel(Pages P, int32_t* live, void* ws) {
  const CompactScratch S = compact_scratch(ws, P.n_pages);
  const int t = threadIdx.x;
  int ref[kScan];
  int L = 0, all;
  for (int p0 = 0; p0 < P.n_pages; p0 += kPlan * kScan) {
    counts_at(P, p0, ref);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kScan; ++i) mine += __popcll(__ballot(ref[i] > 0));
    waves_before(mine, &all);
    L += all;
  }
  int nfrom = 0, nto = 0;
  for (int p0 = 0; p0 < P.n_pages; p0 += kPlan * kScan) {
    if (P.n_pages > kPlan * kScan) counts_at(P, p0, ref);
    // live pages from L on and free ones before it, both counts in one word (4096 a step at most)
    uint64_t out[kScan], in[kScan];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int p = walk_at(p0, i);
      out[i] = __ballot(moves_out(ref[i], p, L));
      in[i] = __ballot(takes_in(ref[i], p, L));
      mine += __popcll(out[i]) + (__popcll(in[i]) << 16);
    }
    const int before = waves_before(mine, &all);
    int a = nfrom + (before & 0xffff), b = nto + (before >> 16);
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int p = walk_at(p0, i);
      if (moves_out(ref[i], p, L)) S.from[a + lanes_before(out[i])] = p;
      if (takes_in(ref[i], p, L)) S.to[b + lanes_before(in[i])] = p;
      if (p >= L && p < P.n_pages) S.place[p] = p;  // unless it moves
      a += __popcll(out[i]);
      b += __popcll(in[i]);
    }
    nfrom += all & 0xffff;
    nto += all >> 16;
  }
  __syncthreads();
  // (the two sides are equal unless another stream changes counts between the walks)
  const int nmove = min(nfrom, nto);
  for (int i = t; i < nmove; i += kPlan) {
    const int a = S.from[i], b = S.to[i];
    S.place[a] = b;
    P.ref[b] = P.ref[a];
    P.ref[a] = 0;
  }
  if (t == 0) {
    *live = L;
    *S.nmove = nmove;
  }
}

// The tables (a workgroup a row) and the copies, which need the plan alone, in one launch.
__global__ __launch_bounds__(256) void compact_move_kernel(Pages P, const int32_t* live,
                                                           const int32_t* place, Copies C) {
  const int r = blockIdx.x, L = *live;
  if (r >= P.rows) {
    copy_pages(C, r - P.rows, gridDim.x - P.rows);
    return;
  }
  const int n = pages_of(clamp_len(P.len[r], P.ld, P.shift), P.shift);
  int32_t* t = P.table + (int64_t)r * P.ld;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int id = t[j];
    if (page_ok(id, P.n_pages) && id >= L) t[j] = place[id];
  }
}

Copies copies(const xpress_cache& c, const int32_t* count, const int32_t* from, const int32_t* to) {
  return Copies{count, from, to, static_cast<u32x4*>(c.k), static_cast<u32x4*>(c.v), c.n_layers,
                c.n_pages, cache_page_bytes(c) / 16};
}
// Workgroups for `most` page copies.
unsigned copy_grid(const xpress_cache& c, int64_t most) {
  return (unsigned)std::min<int64_t>(most * c.n_layers * 2, 2048);
}

}  // namespace

size_t cache_scratch_bytes(const xpress_cache& c, int n_max) {
  const size_t extend = 4 * (4 + kExtendPerRow * (size_t)n_max + c.n_pages);
  const size_t compact = 4 * (4 + 3 * (size_t)c.n_pages);
  return extend > compact ? extend : compact;
}

hipError_t launch_cache_fork(const xpress_cache& c, const int32_t* src, const int32_t* dst, int n,
                             hipStream_t s) {
  hipLaunchKernelGGL(fork_kernel, dim3(n), dim3(256), 0, s, pages(c), src, dst);
  return hipGetLastError();
}

hipError_t launch_cache_extend(const xpress_cache& c, const int32_t* seq, int N,
                               const int32_t* add, int add_all, int32_t* lacking, void* ws,
                               hipStream_t s) {
  hipLaunchKernelGGL(extend_kernel, dim3(1), dim3(kPlan), 0, s, pages(c), seq, N, add, add_all,
                     lacking, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const ExtendScratch S = extend_scratch(ws, N);
  hipLaunchKernelGGL(copy_pages_kernel, dim3(copy_grid(c, N)), dim3(256), 0, s,
                     copies(c, S.ncopy, S.from, S.to));
  return hipGetLastError();
}

hipError_t launch_cache_append(const xpress_cache& c, const int32_t* lacking, int layer,
                               const void* k_new, const void* v_new, int64_t ld_new,
                               const int32_t* seq, int N, int B, hipStream_t s) {
  if (cache_in_4_bits(c))
    return launch_cache_append4(c, lacking, layer, k_new, v_new, ld_new, seq, N, B, s);
  const int64_t n = (int64_t)N * B * (c.Hkv * c.D / 8);
  const int64_t layer_elems = (int64_t)c.n_pages * c.Hkv * c.page * c.D;
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, s,
                     pages(c), lacking, static_cast<uint16_t*>(c.k) + layer * layer_elems,
                     static_cast<uint16_t*>(c.v) + layer * layer_elems,
                     static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new),
                     ld_new, seq, N, B, c.Hkv, c.D);
  return hipGetLastError();
}

hipError_t launch_cache_trim(const xpress_cache& c, const int32_t* lacking, const int32_t* seq, int N,
                             const int32_t* drop, hipStream_t s) {
  hipLaunchKernelGGL(trim_kernel, dim3(N), dim3(256), 0, s, pages(c), lacking, seq, drop);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const xpress_cache& c, int32_t* live, void* ws, hipStream_t s) {
  hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(kPlan), 0, s, pages(c), live, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const CompactScratch S = compact_scratch(ws, c.n_pages);
  hipLaunchKernelGGL(compact_move_kernel, dim3(c.rows + copy_grid(c, (c.n_pages + 1) / 2)), dim3(256),
                     0, s, pages(c), static_cast<const int32_t*>(live), S.place,
                     copies(c, S.nmove, S.from, S.to));
  return hipGetLastError();
}

}  // namespace xpress
