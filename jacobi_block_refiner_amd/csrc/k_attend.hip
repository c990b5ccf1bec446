// Attention of drafted blocks over the paged cache (gfx950).
//
// Per kv head h the query rows of a batch are the N*B*G vectors q[token, h*G + g]. The keys fall in
// two parts: the `shared` first tokens, which are the same for every request, and each request's
// own. Work items are (head, tile of 32*NW query rows, range of keys): tiles over all requests'
// rows for the shared part (its K and V are read once per tile of 256 rows instead of once per
// request), tiles over one request's rows for its own part. Each item runs the softmax in one pass
// over its keys with a running maximum and sum; where a row has more than one item, they leave
// (sum of weighted values, maximum, sum) in the workspace and merge_kernel joins them.
#include "serve.hpp"
#include "cache_index.hpp"
#include "xpress_common.hpp"

#include <algorithm>

namespace xpress {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

constexpr int kIds = 2048;  // table entries an item keeps in LDS: bounds its range of keys

struct Args {
  const uint16_t *q, *k, *v;  // k, v of the layer
  int64_t q_ld, out_ld;
  const int32_t *table, *len, *seq;
  int rows, ld, n_pages, shift;
  int N, B, G, Hq, Hkv, shared;
  float c;  // scale * log2(e)
  // shared items: tiles of rows x splits of keys; own items the same per request
  int tiles_sh, s_sh, chunk_sh, tiles_own, s_own;
  uint16_t* out;
  float* lse;
  float* po;   // [slots, N*B, Hq, D]
  float2* pml; // [slots, N*B, Hq]: maximum (log2 units), sum
};

// Two weights rounded to the type (to nearest even) in one register: the matrix core takes them as
// bf16 or fp16. Relative error half a step each, against the 32-bit sum of the unrounded weights.
template <bool F16> __device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2 x = {a, b};
  return F16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2))
             : __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
}

template <bool F16>
__device__ __forceinline__ f32x16 mfma(const s16x8& a, const s16x8& b, const f32x16& c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The value of the lane 32 further (round the wave), beside this lane's own.
__device__ __forceinline__ float2 both_halves(float x) {
  const u32x2v r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
  return make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
}

// Range of a request's own keys that split s of s_own covers.
__device__ __forceinline__ int2 own_range(int len, int shared, int s, int s_own, int step) {
  const int n = max(len - shared, 0);
  const int chunk = ((n + s_own - 1) / s_own + step - 1) / step * step;
  const int64_t a = (int64_t)s * chunk;
  return make_int2(shared + (int)min(a, (int64_t)n), shared + (int)min(a + chunk, (int64_t)n));
}

__device__ __forceinline__ int list_row(const Args& A, int i) {
  const int r = A.seq ? A.seq[i] : i;
  return (unsigned)r < (unsigned)A.rows ? r : -1;
}
__device__ __forceinline__ int list_len(const Args& A, int i) {
  const int r = list_row(A, i);
  return r < 0 ? 0 : clamp_len(A.len[r], A.ld, A.shift);
}

// One work item. Scores are formed transposed, S^T = K Q^T (32 keys x 32 queries a tile of the
// matrix core), so a lane holds scores of one query only: maxima and sums stay in the lane up to
// one exchange with the lane 32 further. The weights P^T leave the accumulator in the order in which
// the second product O^T = V^T P^T takes its right operand, once V^T's keys are taken in the same
// order: lane half h, element j of a step of 16 keys is key 8*(j/4) + 4*h + j%4. V^T comes from the
// row-major V tile with transposing LDS reads of 4 keys x 16 channels.
//
// K and V tiles of KT keys go from HBM straight into an LDS ring of three stages, two tiles in
// flight while one is used; one barrier a tile. 16-byte pieces of a row are placed with an XOR of
// the key's low bits, so that both kinds of reads are free of bank conflicts.
template <bool F16, int D, int NW, int KT>
__global__ __launch_bounds__(NW * 64) void attend_kernel(Args A) {
  constexpr int CPR = D / 8;               // 16-byte pieces of a row
  constexpr int KPC = 64 / CPR;            // keys of a 1 KiB copy
  constexpr int CW = KT / KPC / NW;        // copies of K (and of V) a wave issues per tile
  constexpr int NS = 3;
  constexpr int SIDE = KT * CPR * 16;      // bytes of a K or V tile
  constexpr int KH = KT / 32, KK = KT / 16, DT = D / 32, DS = D / 16;
  static_assert(CW * KPC * NW == KT, "copies divide evenly");
  __shared__ uint4 s_tile[NS * 2 * SIDE / 16];
  __shared__ int s_ids[kIds];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;

  // the item
  int id = blockIdx.x;
  const int n_sh = A.Hkv * A.tiles_sh * A.s_sh;
  const bool is_shared = id < n_sh;
  int hk, tile, slot, req, kbeg, kend, nrows, trow;
  if (is_shared) {
    hk = id % A.Hkv;
    id /= A.Hkv;
    tile = id % A.tiles_sh;
    slot = id / A.tiles_sh;
    req = 0;
    kbeg = slot * A.chunk_sh;
    kend = min(kbeg + A.chunk_sh, A.shared);
    nrows = A.N * A.B * A.G;
  } else {
    id -= n_sh;
    hk = id % A.Hkv;
    id /= A.Hkv;
    const int s = id % A.s_own;
    id /= A.s_own;
    tile = id % A.tiles_own;
    req = id / A.tiles_own;
    slot = A.s_sh + s;
    const int2 r = own_range(list_len(A, req), A.shared, s, A.s_own, KT);
    kbeg = r.x;
    kend = r.y;
    nrows = A.B * A.G;
  }
  const bool direct = A.s_sh + A.s_own == 1;
  if (kend <= kbeg && !direct) return;
  trow = max(list_row(A, req), 0);

  // this lane's query
  const int rl = (tile * NW + wave) * 32 + col;
  const bool valid = rl < nrows;
  const int token = (is_shared ? 0 : req * A.B) + min(rl, nrows - 1) / A.G;
  const int hq = hk * A.G + min(rl, nrows - 1) % A.G;
  const int sight = min(in_sight(list_len(A, token / A.B), A.B, token % A.B), kend);
  const int vis = valid ? sight : INT_MAX;
  int vmin = vis, vmax = valid ? sight : 0;
  for (int x = 16; x; x >>= 1) {
    vmin = min(vmin, __shfl_xor(vmin, x));
    vmax = max(vmax, __shfl_xor(vmax, x));
  }
  vmin = __builtin_amdgcn_readfirstlane(vmin);
  vmax = __builtin_amdgcn_readfirstlane(vmax);

  s16x8 qf[DS];
  {
    const uint16_t* qp = A.q + token * A.q_ld + (int64_t)hq * D + 8 * h;
#pragma unroll
    for (int s = 0; s < DS; ++s) qf[s] = *reinterpret_cast<const s16x8*>(qp + 16 * s);
  }

  const int pfirst = kbeg >> A.shift;
  {
    const int n = kend > kbeg ? ((kend - 1) >> A.shift) - pfirst + 1 : 0;
    const int32_t* t = A.table + (int64_t)trow * A.ld + pfirst;
    for (int j = threadIdx.x; j < n; j += NW * 64) s_ids[j] = clamp_page(t[j], A.n_pages);
  }
  __syncthreads();

  const uint32_t sbase = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint4*)s_tile;
  const int nt = (kend - kbeg + KT - 1) / KT;
  // lane's piece of each copy: its key's line, and which 16 bytes of it (keys past the range read
  // the last one: their weights are masked)
  auto copy_tile = [&](int t, int stage) {
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      const int ci = wave + NW * c, key = ci * KPC + lane / CPR, piece = lane % CPR;
      const int pos = min(kbeg + t * KT + key, kend - 1);
      const int page_id = s_ids[(pos >> A.shift) - pfirst];
      const int64_t off = line_offset(page_id, hk, pos & ((1 << A.shift) - 1), A.Hkv, A.shift, D);
      const int fk = D == 64 ? (key >> 1) & 7 : key & 15;
      const int fv = D == 64 ? ((key >> 1) & 1) << 2 | ((key >> 2) & 3) : (key & 3) << 2 | ((key >> 2) & 3);
      const uint32_t to = sbase + stage * 2 * SIDE + ci * 1024;
      lds_copy16_at(A.k + off + ((piece ^ fk) * 8), to);
      lds_copy16_at(A.v + off + ((piece ^ fv) * 8), to + SIDE);
    }
  };

  // LDS byte offsets of this lane's fragment reads inside a stage
  const int fk = D == 64 ? (col >> 1) & 7 : col & 15;
  const int i16 = lane & 15, vkey = 4 * h + (i16 >> 2);           // key of the transposing read
  const int vpiece = ((lane >> 4) & 1) * 2 + ((i16 >> 1) & 1);    // 16-byte piece inside 32 channels
  auto k_frag = [&](int stage, int kh, int s) {
    const int byte = stage * 2 * SIDE + (kh * 32 + col) * D * 2 + (((2 * s + h) ^ fk) * 16);
    return *reinterpret_cast<const s16x8*>(reinterpret_cast<const char*>(s_tile) + byte);
  };
  auto v_frag = [&](int stage, int kk, int dt) {
    s16x4 part[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int key = kk * 16 + 8 * x + vkey;
      const int fv = D == 64 ? ((key >> 1) & 1) << 2 | ((key >> 2) & 3) : (key & 3) << 2 | ((key >> 2) & 3);
      const int byte = stage * 2 * SIDE + SIDE + key * D * 2 + (((dt * 4 + vpiece) ^ fv) * 16) + (i16 & 1) * 8;
      part[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(reinterpret_cast<char*>(s_tile) + byte));
    }
    return __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
  };

  float m = -1e30f, l = 0.f;
  f32x16 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) o[dt] = f32x16{};

  // Start of a tile: its copies have landed in every wave, and tile t-1's stage is free again.
  int stage = 0;
  auto enter = [&](int t) {
    // this wave's copies of tile t (those of tile t+1 may be in flight) and its reads of tile t-1:
    // vmcnt, lgkmcnt(0)
    if (t + 1 < nt)
      __builtin_amdgcn_s_waitcnt(0x0070 | (2 * CW));
    else
      __builtin_amdgcn_s_waitcnt(0x0070);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t + 2 < nt) copy_tile(t + 2, stage == 0 ? 2 : stage - 1);
  };
  auto leave = [&] { stage = stage == NS - 1 ? 0 : stage + 1; };
  f32x16 s[KH];
  s16x8 pf[KK];
  auto scores = [&] {
#pragma unroll
    for (int d = 0; d < DS; ++d)
#pragma unroll
      for (int kh = 0; kh < KH; ++kh)
        s[kh] = mfma<F16>(k_frag(stage, kh, d), qf[d], d == 0 ? f32x16{} : s[kh]);
  };
  auto weights = [&] {
    float top = s[0][0];
#pragma unroll
    for (int kh = 0; kh < KH; ++kh)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kh][i]);
    const float2 tops = both_halves(top);
    top = fmaxf(tops.x, tops.y);
    // The sums are rescaled only when some row's maximum grew by more than 2^8 in weight: weights
    // stay below 2^8, which 32-bit sums and the rounded weights' relative precision do not feel.
    if (__any((top - m) * A.c > 8.f)) {
      const float mn = fmaxf(m, top);
      const float alpha = __builtin_amdgcn_exp2f((m - mn) * A.c);
      l *= alpha;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] *= alpha;
      m = mn;
    }
    const float mc = -m * A.c;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = __builtin_amdgcn_exp2f(fmaf(s[kk / 2][8 * (kk % 2) + 2 * j], A.c, mc));
        const float b = __builtin_amdgcn_exp2f(fmaf(s[kk / 2][8 * (kk % 2) + 2 * j + 1], A.c, mc));
        l += a + b;
        w[j] = pack2<F16>(a, b);
      }
      pf[kk] = __builtin_bit_cast(s16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }
  };

  if (nt > 0) copy_tile(0, 0);
  if (nt > 1) copy_tile(1, 1);
  int t = 0;
  // tiles that every row of the wave sees whole
  for (; t < nt && kbeg + t * KT + KT <= vmin; ++t) {
    enter(t);
    scores();
    weights();
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] = mfma<F16>(v_frag(stage, kk, dt), pf[kk], o[dt]);
    leave();
  }
  // the others
  for (; t < nt; ++t) {
    enter(t);
    const int t0 = kbeg + t * KT;
    if (t0 < vmax) {
      scores();
#pragma unroll
      for (int kh = 0; kh < KH; ++kh)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[kh][i] = t0 + kh * 32 + 8 * (i / 4) + 4 * h + i % 4 < vis ? s[kh][i] : -INFINITY;
      weights();
      // Values in masked places must not reach a row: 0 * inf would. Keys with a value that is not
      // finite are taken out of the product and added one by one to the rows that see them.
      uint64_t bad;
      {
        const uint4* row = s_tile + (stage * 2 * SIDE + SIDE) / 16 + lane % KT * CPR;
        constexpr uint32_t E = F16 ? 0x7c00u : 0x7f80u;
        bool found = false;
#pragma unroll 4
        for (int x = 0; x < CPR; ++x) {
          const uint4 u = row[x];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) found |= (w[y] & E) == E || ((w[y] >> 16) & E) == E;
        }
        bad = __ballot(found);
        if (KT < 64) bad &= (uint64_t(1) << (KT & 63)) - 1;
      }
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        s16x8 keep;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          keep[j] = (bad >> (kk * 16 + 8 * (j / 4) + 4 * h + j % 4)) & 1 ? 0 : -1;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
          o[dt] = mfma<F16>(v_frag(stage, kk, dt) & keep, pf[kk], o[dt]);
      }
#pragma unroll 1
      for (uint64_t left = bad; left; left &= left - 1) {
        const int key = __builtin_ctzll(left);
        const bool sees = t0 + key < vis;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          if (key / 16 != kk) continue;
          s16x8 keep;
#pragma unroll
          for (int j = 0; j < 8; ++j) keep[j] = kk * 16 + 8 * (j / 4) + 4 * h + j % 4 == key ? -1 : 0;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) {
            const f32x16 one = mfma<F16>(v_frag(stage, kk, dt) & keep, pf[kk] & keep, f32x16{});
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] += sees ? one[i] : 0.f;
          }
        }
      }
    }
    leave();
  }

  const float2 ls = both_halves(l);
  l = ls.x + ls.y;
  if (!valid) return;
  const int64_t row = (int64_t)token * A.Hq + hq;
  if (direct) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* op = A.out + token * A.out_ld + (int64_t)hq * D + 4 * h;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint2 w;
        w.x = pack2<F16>(o[dt][4 * i] * inv, o[dt][4 * i + 1] * inv);
        w.y = pack2<F16>(o[dt][4 * i + 2] * inv, o[dt][4 * i + 3] * inv);
        *reinterpret_cast<uint2*>(op + dt * 32 + 8 * i) = w;
      }
    if (A.lse && h == 0)
      A.lse[row] = l == 0.f ? -INFINITY : (m * A.c + log2f(l)) * 0.69314718056f;
    return;
  }
  const int64_t at = (int64_t)slot * A.N * A.B * A.Hq + row;
  float* op = A.po + at * D + 4 * h;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(op + dt * 32 + 8 * i) =
          make_float4(o[dt][4 * i], o[dt][4 * i + 1], o[dt][4 * i + 2], o[dt][4 * i + 3]);
  if (h == 0) A.pml[at] = make_float2(m * A.c, l);
}

// Joins a row's items: weights relative to the largest maximum, in slot order.
template <bool F16, int D, int KT>
__global__ __launch_bounds__(256) void merge_kernel(Args A) {
  constexpr int LPR = D / 4;  // lanes of a row
  const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int64_t n = (int64_t)A.N * A.B * A.Hq;
  if (row >= n) return;
  const int d = threadIdx.x % LPR * 4;
  const int token = (int)(row / A.Hq), hq = (int)(row % A.Hq);
  const int len = list_len(A, token / A.B);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < A.s_sh + A.s_own; ++s) {
    if (s >= A.s_sh) {
      const int2 r = own_range(len, A.shared, s - A.s_sh, A.s_own, KT);
      if (r.y <= r.x) break;
    }
    const int64_t at = s * n + row;
    const float2 ml = A.pml[at];
    if (ml.y == 0.f) continue;
    const float4 x = *reinterpret_cast<const float4*>(A.po + at * D + d);
    const float mn = fmaxf(m, ml.x);
    const float a = __builtin_amdgcn_exp2f(m - mn), b = __builtin_amdgcn_exp2f(ml.x - mn);
    l = l * a + ml.y * b;
    o.x = o.x * a + x.x * b;
    o.y = o.y * a + x.y * b;
    o.z = o.z * a + x.z * b;
    o.w = o.w * a + x.w * b;
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 w;
  w.x = pack2<F16>(o.x * inv, o.y * inv);
  w.y = pack2<F16>(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(A.out + token * A.out_ld + (int64_t)hq * D + d) = w;
  if (A.lse && d == 0) A.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
}

// How a call is cut into items.
struct Plan {
  int tiles_sh, s_sh, chunk_sh, tiles_own, s_own;
  int slots() const { return s_sh + s_own; }
};

constexpr int waves_of(int D) { return D == 256 ? 4 : 8; }
constexpr int step_of(int D) { return D == 256 ? 32 : 64; }
constexpr int kItems = 512;   // items a call is cut into where its rows alone give fewer
constexpr int kSplits = 64;   // splits of one row's keys at most (more where ids do not fit in LDS)

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Keys of one item at most: its table entries have to fit in LDS.
int64_t most_keys(const xpress_cache& c) { return (int64_t)(kIds - 2) * c.page / 64 * 64; }

Plan plan_of(const xpress_cache& c, int N, int B, int Hq, int shared) {
  const int NW = waves_of(c.D), KT = step_of(c.D), G = Hq / c.Hkv;
  const int64_t own = (int64_t)c.table_ld * c.page - shared, most = most_keys(c);
  Plan p{};
  p.tiles_own = (int)ceil_div((int64_t)B * G, NW * 32);
  int64_t s = ceil_div(kItems, (int64_t)N * c.Hkv * p.tiles_own);
  s = std::max<int64_t>(1, std::min({s, ceil_div(own, 2 * KT), (int64_t)kSplits}));
  p.s_own = (int)std::max(s, ceil_div(own, most));
  if (shared > 0) {
    p.tiles_sh = (int)ceil_div((int64_t)N * B * G, NW * 32);
    s = ceil_div(kItems, (int64_t)c.Hkv * p.tiles_sh);
    s = std::max<int64_t>(1, std::min({s, ceil_div(shared, 4 * KT), (int64_t)kSplits}));
    s = std::max(s, ceil_div(shared, most));
    p.chunk_sh = (int)(ceil_div(ceil_div(shared, s), KT) * KT);
    p.s_sh = (int)ceil_div(shared, p.chunk_sh);
  }
  return p;
}

// Largest number of (row of the batch, slot) pairs of any N <= n and any shared: with A items
// wanted for n requests, n * ceil(A / n) <= A + n; every bound grows with n.
int64_t most_row_slots(const xpress_cache& c, int n, int B, int Hq) {
  const int rows = waves_of(c.D) * 32, KT = step_of(c.D), G = Hq / c.Hkv;
  const int64_t cap = (int64_t)c.table_ld * c.page, ids = ceil_div(cap, most_keys(c));
  const int64_t tiles = ceil_div((int64_t)B * G, rows);
  const int64_t own = std::min({ceil_div(kItems, c.Hkv * tiles) + n, n * ceil_div(cap, 2 * KT),
                                (int64_t)n * kSplits});
  const int64_t sh = std::min({ceil_div((int64_t)kItems * rows, (int64_t)c.Hkv * B * G) + n,
                               n * ceil_div(cap, 4 * KT), (int64_t)n * kSplits});
  return std::max<int64_t>(own, n * ids) + std::max<int64_t>(sh, n * ids);
}

template <bool F16, int D>
hipError_t launch_t(const Args& A, hipStream_t s) {
  constexpr int NW = waves_of(D), KT = step_of(D);
  const int64_t items = (int64_t)A.Hkv * A.tiles_sh * A.s_sh + (int64_t)A.Hkv * A.s_own * A.tiles_own * A.N;
  hipLaunchKernelGGL((attend_kernel<F16, D, NW, KT>), dim3((unsigned)items), dim3(NW * 64), 0, s, A);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || A.s_sh + A.s_own == 1) return e;
  const int64_t rows = (int64_t)A.N * A.B * A.Hq;
  const int per = 256 / (D / 4);
  hipLaunchKernelGGL((merge_kernel<F16, D, KT>), dim3((unsigned)((rows + per - 1) / per)), dim3(256),
                     0, s, A);
  return hipGetLastError();
}

}  // namespace

size_t attention_scratch_bytes(const xpress_cache& c, int N, int B, int Hq) {
  return (size_t)most_row_slots(c, N, B, Hq) * B * Hq * (c.D * sizeof(float) + sizeof(float2));
}

int64_t attention_items(const xpress_cache& c, int N, int B, int Hq, int shared) {
  const Plan p = plan_of(c, N, B, Hq, shared);
  return c.Hkv * ((int64_t)p.tiles_sh * p.s_sh + (int64_t)p.tiles_own * p.s_own * N);
}

hipError_t launch_block_attention(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                  const int32_t* seq, int N, int B, int Hq, float scale,
                                  int shared, void* out, int64_t out_ld, float* lse, void* ws,
                                  hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * c.Hkv * c.page * c.D;
  const Plan p = plan_of(c, N, B, Hq, shared);
  Args A;
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(c.k) + at;
  A.v = static_cast<const uint16_t*>(c.v) + at;
  A.q_ld = q_ld;
  A.out_ld = out_ld;
  A.table = c.table;
  A.len = c.len;
  A.seq = seq;
  A.rows = c.rows;
  A.ld = c.table_ld;
  A.n_pages = c.n_pages;
  A.shift = __builtin_ctz((unsigned)c.page);
  A.N = N;
  A.B = B;
  A.G = Hq / c.Hkv;
  A.Hq = Hq;
  A.Hkv = c.Hkv;
  A.shared = shared;
  A.c = scale * 1.44269504089f;
  A.tiles_sh = p.tiles_sh;
  A.s_sh = p.s_sh;
  A.chunk_sh = p.chunk_sh;
  A.tiles_own = p.tiles_own;
  A.s_own = p.s_own;
  A.out = static_cast<uint16_t*>(out);
  A.lse = lse;
  A.po = static_cast<float*>(ws);
  A.pml = reinterpret_cast<float2*>(A.po + (size_t)p.slots() * N * B * Hq * c.D);
  const bool f16 = c.dtype == XPRESS_F16;
  switch (c.D) {
    case 64: return f16 ? launch_t<true, 64>(A, s) : launch_t<false, 64>(A, s);
    case 128: return f16 ? launch_t<true, 128>(A, s) : launch_t<false, 128>(A, s);
    default: return f16 ? launch_t<true, 256>(A, s) : launch_t<false, 256>(A, s);
  }
}

}  // namespace xpress
