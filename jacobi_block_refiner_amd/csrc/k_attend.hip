// Attention of drafted blocks over the paged cache (gfx950).
//
// Per kv head h the query rows of a batch are the N*B*G vectors q[token, h*G + g]. The keys fall in
// two parts: the first tokens, which are the same for every request, and each request's own. Work
// items are (head, tile of query rows, range of keys): tiles over all requests' rows for the shared
// part (its K and V are read once per tile of 128 or 256 rows instead of once per request), tiles
// over one request's rows for its own part. Each item runs the softmax in one pass over its keys with
// a running maximum and sum; where a row has more than one item, they leave (sum of weighted values,
// unit of the weights, sum) in the workspace and merge_kernel joins them.
//
// The shared part is cut to whole tiles of 64 keys; what is left of it goes with the requests' own.
// A request whose queries do not all see the whole shared part (a short or an empty row) takes all
// its keys as its own. So no shared item has a mask.
#include "serve.hpp"
#include "attend_plan.hpp"
#include "cache_index.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

struct Args {
  const uint16_t *q, *k, *v;  // k, v of the layer
  int64_t q_ld, out_ld;
  const int32_t *table, *len, *seq;
  int rows, ld, n_pages, shift;
  int N, B, G, Hq, Hkv, shared;
  float c;  // scale * log2(e)
  // shared items: tiles of rows x splits of keys; own items the same per request
  int tiles_sh, s_sh, chunk_sh, tiles_own, s_own;
  int slots_sh;  // slots of the shared part (items of this launch or of one before it)
  int step_own;  // own ranges are multiples of it
  bool direct;   // own items are their rows' last and write the result
  uint16_t* out;
  float* lse;
  float* po;   // [slots, N*B, Hq, D]
  float2* pml; // [slots, N*B, Hq]: log2 of the weights' unit, their sum in it
};

// Two weights rounded to the type (to nearest even) in one register: the matrix core takes 16-bit
// operands at its full rate, while the sum of the weights and the sums of weighted values have 32 bits.
// The rounding is off by half a step of each weight: as much again as that of the result itself.
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

// Keys of one split of a request's n own keys.
__device__ __forceinline__ int own_chunk(int n, int s_own, int step) {
  return ((n + s_own - 1) / s_own + step - 1) / step * step;
}
// First of a request's own keys: 0 where some query of it does not see the whole shared part.
__device__ __forceinline__ int own_begin(int len, int B, int shared) {
  return in_sight(len, B, 0) >= shared ? shared : 0;
}
// Range of a request's own keys that split s of s_own covers.
__device__ __forceinline__ int2 own_range(int len, int first, int s, int s_own, int step) {
  const int n = len - first, chunk = own_chunk(n, s_own, step);
  const int64_t a = (int64_t)s * chunk;
  return make_int2(first + (int)min(a, (int64_t)n), first + (int)min(a + chunk, (int64_t)n));
}

__device__ __forceinline__ int list_row(const Args& A, int i) {
  const int r = A.seq ? A.seq[i] : i;
  return (unsigned)r < (unsigned)A.rows ? r : -1;
}
__device__ __forceinline__ int list_len(const Args& A, int i) {
  const int r = list_row(A, i);
  return r < 0 ? 0 : clamp_len(A.len[r], A.ld, A.shift);
}

// A wave's 32 queries against tiles of KT keys in LDS. Scores are formed transposed, S^T = K Q^T (32
// keys x 32 queries a tile of the matrix core), so a lane holds scores of one query only: maxima and
// sums stay in the lane up to one exchange with the lane 32 further. The weights P^T leave the
// accumulator in the order in which the second product O^T = V^T P^T takes its right operand, once
// V^T's keys are taken in the same order: lane half h, element j of a step of 16 keys is key
// 8*(j/4) + 4*h + j%4. V^T comes from the row-major V tile with transposing LDS reads of 4 keys x 16
// channels. 16-byte pieces of a K or V row are placed with an XOR of the key's low bits, so that both
// kinds of reads are free of bank conflicts.
template <bool F16, int D, int KT> struct Core {
  static constexpr int CPR = D / 8;           // 16-byte pieces of a row
  static constexpr int KPC = 64 / CPR;        // keys of a 1 KiB copy
  static constexpr int SIDE = KT * CPR * 16;  // bytes of a K or V tile
  static constexpr int KH = KT / 32, KK = KT / 16, DT = D / 32, DS = D / 16;
  // Weights are 2^kLift times those relative to the running maximum, which they pass by 2^8 at most
  // (rise). fp16 has whole precision from 2^-14 to 2^16 only: without the factor a weight below 2^-14
  // of the maximum lost bits and one below 2^-25 vanished, and 60,000 of them 17 nats under one key
  // were off by 44%. With it steps are coarser from 2^-21 on and nothing is left from 2^-32 on: half a
  // step of 2^21 such keys is 2^-11 of the row, the result's own rounding.
  static constexpr float kLift = F16 ? 7.f : 0.f;

  char* lds;
  int lane, h, col;
  float c;
  s16x8 qf[DS];
  f32x16 s[KH], o[DT];
  s16x8 pf[KK];
  float m, l;
  float shift;    // of the weights' exponents: 2^(s c + shift)
  uint64_t huge;  // lanes whose unit is past kHuge

  __device__ static int k_swizzle(int key) { return D == 64 ? (key >> 1) & 7 : key & 15; }
  __device__ static int v_swizzle(int key) {
    return D == 64 ? ((key >> 1) & 1) << 2 | ((key >> 2) & 3) : (key & 3) << 2 | ((key >> 2) & 3);
  }

  __device__ __forceinline__ void begin(void* tiles, const uint16_t* q, float scale) {
    lds = static_cast<char*>(tiles);
    lane = threadIdx.x & 63;
    h = lane >> 5;
    col = lane & 31;
    c = scale;
#pragma unroll
    for (int x = 0; x < DS; ++x) qf[x] = *reinterpret_cast<const s16x8*>(q + 16 * x + 8 * h);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[dt] = f32x16{};
    m = -1e30f;
    l = 0.f;
    huge = ~0ull;
  }

  // Scores of the K tile at byte kb.
  __device__ __forceinline__ void scores(int kb) {
    const int fk = k_swizzle(col);
#pragma unroll
    for (int d = 0; d < DS; ++d)
#pragma unroll
      for (int kh = 0; kh < KH; ++kh) {
        const s16x8 k = *reinterpret_cast<const s16x8*>(lds + kb + (kh * 32 + col) * D * 2 +
                                                        (((2 * d + h) ^ fk) * 16));
        s[kh] = mfma<F16>(k, qf[d], d == 0 ? f32x16{} : s[kh]);
      }
  }

  static constexpr float kHuge = 0x1p20f;

  // log2 of the weights' unit.
  __device__ __forceinline__ float unit() const { return fmaf(m, c, -kLift); }

  // Keys t0.. of which this lane's query sees those below vis.
  __device__ __forceinline__ void mask(int t0, int vis) {
#pragma unroll
    for (int kh = 0; kh < KH; ++kh)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[kh][i] = t0 + kh * 32 + 8 * (i / 4) + 4 * h + i % 4 < vis ? s[kh][i] : -INFINITY;
  }

  // Takes the tile's maximum in.
  // The exponents are s c - unit in one operation: the unit is rounded, but the weights are relative to
  // what it was rounded to. Where half a step of it is no longer small beside the factor of 2 that
  // fp16's range has left, the scores become s - m first.
  // The sums are rescaled only when some row's maximum grew by more than
  // 2^8 in weight: weights relative to it stay below 2^8, which 32-bit sums and the rounded weights'
  // relative precision do not feel.
  __device__ __forceinline__ void rise() {
    float top = s[0][0];
#pragma unroll
    for (int kh = 0; kh < KH; ++kh)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kh][i]);
    const float2 tops = both_halves(top);
    top = fmaxf(tops.x, tops.y);
    if ((__ballot((top - m) * c > 8.f) | huge) != 0) {
      const float mn = fmaxf(m, top);
      const float alpha = __builtin_amdgcn_exp2f((m - mn) * c);
      l *= alpha;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] *= alpha;
      m = mn;
      shift = -unit();
      huge = __ballot(fabsf(shift) > kHuge);
      if (huge != 0) {
#pragma unroll
        for (int kh = 0; kh < KH; ++kh) s[kh] -= m;
        shift = kLift;
      }
    }
  }

  __device__ __forceinline__ void weights() {
    float sum[4] = {l, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = __builtin_amdgcn_exp2f(fmaf(s[kk / 2][8 * (kk % 2) + 2 * j], c, shift));
        const float b = __builtin_amdgcn_exp2f(fmaf(s[kk / 2][8 * (kk % 2) + 2 * j + 1], c, shift));
        sum[j] += a + b;
        w[j] = pack2<F16>(a, b);
      }
      pf[kk] = __builtin_bit_cast(s16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }
    l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }

  // V^T of 32 channels dt for the 16 keys kk of the tile at byte vb.
  __device__ __forceinline__ s16x8 v_frag(int vb, int kk, int dt) const {
    const int i16 = lane & 15, vkey = 4 * h + (i16 >> 2);         // key of the transposing read
    const int vpiece = ((lane >> 4) & 1) * 2 + ((i16 >> 1) & 1);  // 16-byte piece of 32 channels
    s16x4 part[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int key = kk * 16 + 8 * x + vkey;
      part[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(lds + vb + key * D * 2 +
                                                     (((dt * 4 + vpiece) ^ v_swizzle(key)) * 16) +
                                                     (i16 & 1) * 8));
    }
    return __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }

  // Adds the weights times the V tile at byte vb.
  __device__ __forceinline__ void values(int vb) {
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] = mfma<F16>(v_frag(vb, kk, dt), pf[kk], o[dt]);
  }
};

// The 16-bit values of u that are not finite set to 0; whether there were any.
template <bool F16> __device__ __forceinline__ bool tame(uint32_t& u) {
  constexpr uint32_t E = F16 ? 0x7c00u : 0x7f80u;
  const bool lo = (u & E) == E, hi = ((u >> 16) & E) == E;
  u &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
  return lo || hi;
}
template <bool F16> __device__ __forceinline__ float value(uint32_t x) {
  return F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)x) : bf16_to_f32((uint16_t)x);
}

// Where an item's K and V come from: a range of one row's tokens, its table entries in LDS. A lane
// copies 16 bytes of one key's line at a time; keys past the range copy the last one (their weights
// are masked, or nothing reads them). Page ids are read a tile ahead: the chain from LDS to an address
// took a thousand cycles of every tile when it stood before each copy.
template <int D, int KT, int NW> struct Source {
  using C = Core<false, D, KT>;
  static constexpr int CW = KT / C::KPC / NW;  // copies of K (and of V) a wave issues per tile
  static_assert(CW * C::KPC * NW == KT, "copies divide evenly");
  const uint16_t *k, *v;  // of the head
  const int* ids;
  int kbeg, kend, shift, key0;
  uint32_t base, page_elems;  // LDS address of this wave's first copy; elements of a page
  int64_t off[CW], off_before[CW];
  int id[CW], line[CW];

  __device__ __forceinline__ void begin(const Args& A, int hk, const int* ids_, int kbeg_, int kend_,
                                        uint32_t lds) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    ids = ids_;
    kbeg = kbeg_;
    kend = kend_;
    shift = A.shift;
    key0 = wave * C::KPC + lane / C::CPR;
    base = lds + wave * 1024;
    page_elems = (uint32_t)(A.Hkv * D) << A.shift;
    const int64_t head = (int64_t)hk * D << A.shift;
    k = A.k + head;
    v = A.v + head;
    ask(0);
  }
  // Page ids and lines of tile t's keys are under way.
  __device__ __forceinline__ void ask(int t) {
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      const int pos = min(kbeg + t * KT + key0 + i * NW * C::KPC, kend - 1);
      id[i] = ids[(pos >> shift) - (kbeg >> shift)];
      line[i] = pos & ((1 << shift) - 1);
    }
  }
  // Turns to the tile asked for, and asks for tile `next`.
  __device__ __forceinline__ void turn(int next) {
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      off_before[i] = off[i];
      off[i] = (int64_t)((uint64_t)(uint32_t)id[i] * page_elems) + line[i] * D;
    }
    ask(next);
  }
  __device__ __forceinline__ void copy_k(int to) const {
    const int piece = threadIdx.x % C::CPR;
#pragma unroll
    for (int i = 0; i < CW; ++i)
      lds_copy16_at(k + off[i] + (piece ^ C::k_swizzle(key0 + i * NW * C::KPC)) * 8,
                    base + to + i * NW * 1024);
  }
  // V of the tile turned to, or of the one before it.
  template <bool BEFORE> __device__ __forceinline__ void copy_v(int to) const {
    const int piece = threadIdx.x % C::CPR;
#pragma unroll
    for (int i = 0; i < CW; ++i)
      lds_copy16_at(v + (BEFORE ? off_before[i] : off[i]) +
                        (piece ^ C::v_swizzle(key0 + i * NW * C::KPC)) * 8,
                    base + to + i * NW * 1024);
  }
};

// Waits until at most N of this wave's copies are under way and all its LDS reads are done, then for
// the other waves.
template <int N> __device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// Waits for this wave's LDS reads, then for the other waves.
__device__ __forceinline__ void meet_reads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Order of a wide item's products (N/2 of each kind) and their LDS reads: eight reads ahead of the
// first product, and every read about eight products ahead of its own, so that none waits for LDS.
// (Left to itself the compiler reads two fragments, waits for both and multiplies: 1450-1850 cycles
// a tile where the products alone take 1024.)
template <int N> __device__ __forceinline__ void feed() {
  __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);  // LDS reads
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix core
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
}

// One work item: NW waves of 32 query rows each; K and V tiles of KT keys go from HBM straight into an
// LDS ring of two to four stages.
//
// Narrow (NW = 4): for items that wait for HBM. Tiles are taken one after the other with one barrier
// each; the workgroups of a CU (three at D 64, two at 128, one at 256) fill each other's waits. At D
// 128 a tile is 16 KB, and two workgroups that ask three tiles ahead read faster than three that ask
// two ahead: 256 requests decoding up to 1024 tokens each (8 heads, 4 queries each, 555 MB) 111 us (5.0
// TB/s) and 136, 32 decoding behind 4096 shared ones 32 and 35. At D 64 three are faster (32 requests of
// 16 tokens x 32 heads, 8192 shared tokens and up to 512 own: 66 and 70 us).
//
// Slim (NW = 2, D 256): items of a request's own keys alone, at most 64 query rows, where they fill
// more than one round of the card. A narrow item at D 256 keeps a CU to itself (its registers, and 96
// KB of tiles), and with one row of queries three of its four waves only copy; two slim ones share a
// CU. 64 requests decoding up to 1024 tokens each (8 heads, 4 queries each) 73 us and 105 narrow, 256
// requests 225 and 348. Beside shared items they would be a launch of their own: 168 and 100 us for 64
// requests behind 4096 tokens, so there the narrow ones stay.
//
// Wide (NW = 8, one workgroup a CU): shared items that the matrix core bounds. The two waves of a SIMD
// are half a tile apart: while one multiplies (scores of tile t, values of tile t-1) the other forms
// weights, and after each such half they meet and change roles. A tile needs about as many cycles of
// the matrix core as of the vector unit; with both waves in step, each unit waited for the other.
// 20480 rows a head, 16384 keys, 8 heads: 1310 to 1400 us, 1.0 PFLOP/s at 1.9 to 2.0 GHz (the power
// limit takes the rest of 2.3), the matrix core busy 47% of the cycles; 2560 rows, 8192 keys: 104 us, 0.8
// PFLOP/s on 240 CUs.
template <bool F16, int D, int NW, int KT>
__global__ __launch_bounds__(NW * 64, D == 256 ? 1 : D == 128 ? 2 : 3) void attend_kernel(
    Args A) {
  using C = Core<F16, D, KT>;
  using S = Source<D, KT, NW>;
  constexpr bool WIDE = NW == kWide;
  constexpr int NS = NW == kSlim ? 2 : WIDE || D == 128 ? 4 : 3, STAGE = 2 * C::SIDE, CW = S::CW;
  __shared__ uint4 s_tile[NS * STAGE / 16];
  __shared__ int s_ids[kIds];
  __shared__ int s_req;
  __shared__ int s_wild[2];  // first and last masked tile with V values that are not finite

  const int lane = threadIdx.x & 63, h = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // the item
  int id = blockIdx.x;
  const int n_sh = A.Hkv * A.tiles_sh * A.s_sh;
  const bool is_shared = WIDE || id < n_sh;
  int hk, tile, slot, req, kbeg, kend, nrows;
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
    slot = A.slots_sh + s;
    const int len = list_len(A, req);
    const int2 r = own_range(len, own_begin(len, A.B, A.shared), s, A.s_own, A.step_own);
    kbeg = r.x;
    kend = r.y;
    nrows = A.B * A.G;
  }
  const bool direct = !WIDE && A.direct;
  if (kend <= kbeg && !direct) return;

  // this lane's query; `blind`: it sees nothing here (what it computes is dropped)
  const int rl = (tile * NW + wave) * 32 + col;
  const bool valid = rl < nrows;
  const int token = (is_shared ? 0 : req * A.B) + min(rl, nrows - 1) / A.G;
  const int hq = hk * A.G + min(rl, nrows - 1) % A.G;
  const int len = list_len(A, token / A.B);
  const int sight = min(in_sight(len, A.B, token % A.B), kend);
  const bool blind =
      !valid || sight <= kbeg || (is_shared && own_begin(len, A.B, A.shared) < A.shared);
  // Whose table leads to the shared part: the first request's, unless it ends inside it (a short or an
  // empty row); then that of any request whose rows are here. Where there is none, all is dropped.
  if (is_shared && own_begin(list_len(A, 0), A.B, A.shared) < A.shared) {
    if (threadIdx.x == 0) s_req = INT_MAX;
    __syncthreads();
    if (!blind) atomicMin(&s_req, token / A.B);
    __syncthreads();
    req = __builtin_amdgcn_readfirstlane(s_req);
    if (req == INT_MAX) req = 0;
  }
  C w;
  w.begin(s_tile, A.q + token * A.q_ld + (int64_t)hq * D, A.c);
  {
    const int first = kbeg >> A.shift, n = kend > kbeg ? ((kend - 1) >> A.shift) - first + 1 : 0;
    const int32_t* t = A.table + (int64_t)max(list_row(A, req), 0) * A.ld + first;
    for (int j = threadIdx.x; j < n; j += NW * 64) s_ids[j] = clamp_page(t[j], A.n_pages);
    if (threadIdx.x == 0) {
      s_wild[0] = INT_MAX;
      s_wild[1] = -1;
    }
  }
  __syncthreads();
  // q has to be in before the first copies: the compiler waits for it at its first use by a count of
  // loads in flight, in which the copies, which it does not know, would take the loads' places
#pragma unroll
  for (int x = 0; x < C::DS; ++x) asm volatile("" : "+v"(w.qf[x]));
  const int nt = (kend - kbeg + KT - 1) / KT;
  S src;
  if (nt > 0)
    src.begin(A, hk, s_ids, kbeg, kend,
              (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint4*)s_tile);
  if constexpr (WIDE) {
    // Copies by group: group t is K(t+3) and V(t+2), issued in half-step 2t or 2t+1, when the last
    // readers of their stages (those of tile t-1 in half-step 2t-1) are done. From half-step 2t+1 on
    // the groups up to t-2 are in, so K(t+1) and V(t). (Tiles past the end are read by no one.)
    auto step = [](int& at, int first) { at = at == first + (NS - 1) * STAGE ? first : at + STAGE; };
    int kto = 0, vto = C::SIDE;
    auto group = [&](int t) {
      src.turn(t + 4);
      src.copy_k(kto);
      step(kto, 0);
      src.template copy_v<true>(vto);
      step(vto, C::SIDE);
    };
    src.turn(1);
    src.copy_k(kto);
    step(kto, 0);
    group(-2);
    group(-1);
    const bool second = wave >= 4;
    meet<4 * CW>();
    if (second) {
      group(0);
      meet<4 * CW>();
    }
    int kb = 0, vb = (NS - 1) * STAGE + C::SIDE;  // K(t), V(t-1)
    auto half = [&](int t) {  // what follows the products of tile t: weights, and the two meetings
      if (second)
        meet_reads();
      else
        meet<2 * CW>();
      group(t + second);
      w.rise();
      w.weights();
      if (second)
        meet<4 * CW>();
      else
        meet_reads();
      step(kb, 0);
      step(vb, C::SIDE);
    };
    w.scores(kb);
    half(0);
    for (int t = 1; t < nt; ++t) {
      w.scores(kb);
      w.values(vb);
      feed<C::KH * C::DS + C::KK * C::DT>();
      half(t);
    }
    w.values(vb);
    if (!second) meet_reads();
    meet<0>();
  } else {
    const int vis = blind ? INT_MAX : sight;
    // no rows, no products: only copies and meetings
    const bool idle = __ballot(!blind) == 0;
    // tiles that every row sees whole: all of a shared item's, else up to the reach of the request's
    // first query
    const int len0 = is_shared ? 0 : list_len(A, req);
    const int whole = is_shared ? nt : max(min(in_sight(len0, A.B, 0), kend) - kbeg, 0) / KT;
    int t = 0, at = 0, to = 0;
    auto copy_both = [&](int next) {
      src.turn(next);
      src.copy_k(to);
      src.template copy_v<false>(to + C::SIDE);
      to = to == (NS - 1) * STAGE ? 0 : to + STAGE;
    };
    auto enter = [&] {
      if (t + NS - 2 < nt)
        meet<2 * CW * (NS - 2)>();
      else if (NS > 3 && t + 1 < nt)
        meet<2 * CW>();
      else
        meet<0>();
      if (t + NS - 1 < nt) copy_both(t + NS);
    };
    auto leave = [&] {
      at = at == (NS - 1) * STAGE ? 0 : at + STAGE;
      ++t;
    };
#pragma unroll
    for (int i = 1; i < NS; ++i)
      if (nt >= i) copy_both(i);
    while (t < min(nt, whole)) {
      enter();
      if (!idle) {
        w.scores(at);
        w.rise();
        w.weights();
        w.values(at + C::SIDE);
      }
      leave();
    }
    // The others. Values in masked places must not reach a row, and 0 * inf would: V values that are
    // not finite are set to 0 in LDS here, and added to the rows that see them at the end.
    while (t < nt) {
      enter();
      bool wild = false;
      for (int x = threadIdx.x; x < KT * C::CPR; x += NW * 64) {
        uint4& v = s_tile[(at + C::SIDE) / 16 + x];
        uint4 u = v;
        if (tame<F16>(u.x) | tame<F16>(u.y) | tame<F16>(u.z) | tame<F16>(u.w)) {
          v = u;
          wild = true;
        }
      }
      if (wild) {
        atomicMin(&s_wild[0], t);
        atomicMax(&s_wild[1], t);
      }
      meet_reads();
      if (!idle) {
        w.scores(at);
        w.mask(kbeg + t * KT, vis);
        w.rise();
        w.weights();
        w.values(at + C::SIDE);
      }
      leave();
    }
    if (s_wild[1] >= 0 && !idle) {
#pragma unroll 1
      for (int pos = kbeg + s_wild[0] * KT; pos < min(kbeg + (s_wild[1] + 1) * KT, kend); ++pos) {
        const int64_t from = line_offset(s_ids[(pos >> A.shift) - (kbeg >> A.shift)], hk,
                                         pos & ((1 << A.shift) - 1), A.Hkv, A.shift, D);
#pragma unroll
        for (int i = 0; i < C::DT * 4; ++i) {
          const uint2 v = *reinterpret_cast<const uint2*>(A.v + from + 4 * h + 8 * i);
          const uint32_t x[4] = {v.x & 0xffff, v.x >> 16, v.y & 0xffff, v.y >> 16};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t tamed = x[j];
            // (a weight is never 0 in exact arithmetic: the value itself reaches the sum)
            w.o[i / 4][i % 4 * 4 + j] += tame<F16>(tamed) && pos < vis ? value<F16>(x[j]) : 0.f;
          }
        }
      }
    }
  }

  const float2 ls = both_halves(w.l);
  float l = blind ? 0.f : ls.x + ls.y;
  if (!valid) return;
  const int64_t row = (int64_t)token * A.Hq + hq, rows = (int64_t)A.N * A.B * A.Hq;
  if (direct) {
    // the shared items' parts of this row, from the launch before this one (0 times what a row that
    // sees nothing here holds, tokens that it must not see among it, would be no number)
    if (l == 0.f) {
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt) w.o[dt] = f32x16{};
    }
    float m = l == 0.f ? -INFINITY : w.unit();
    for (int s = 0; s < A.slots_sh; ++s) {
      const int64_t at = s * rows + row;
      const float2 ml = A.pml[at];
      float4 x[C::DT * 4];
#pragma unroll
      for (int i = 0; i < C::DT * 4; ++i)
        x[i] = *reinterpret_cast<const float4*>(A.po + at * D + 4 * h + 8 * i);
      if (ml.y == 0.f) continue;
      const float mn = fmaxf(m, ml.x);
      const float a = __builtin_amdgcn_exp2f(m - mn), b = __builtin_amdgcn_exp2f(ml.x - mn);
      m = mn;
      l = l * a + ml.y * b;
#pragma unroll
      for (int i = 0; i < C::DT * 4; ++i) {
        f32x16& o = w.o[i / 4];
        o[i % 4 * 4] = o[i % 4 * 4] * a + x[i].x * b;
        o[i % 4 * 4 + 1] = o[i % 4 * 4 + 1] * a + x[i].y * b;
        o[i % 4 * 4 + 2] = o[i % 4 * 4 + 2] * a + x[i].z * b;
        o[i % 4 * 4 + 3] = o[i % 4 * 4 + 3] * a + x[i].w * b;
      }
    }
    const float inv = 1.f / l;
    uint16_t* op = A.out + token * A.out_ld + (int64_t)hq * D + 4 * h;
#pragma unroll
    for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint2 u;
        u.x = pack2<F16>(w.o[dt][4 * i] * inv, w.o[dt][4 * i + 1] * inv);
        u.y = pack2<F16>(w.o[dt][4 * i + 2] * inv, w.o[dt][4 * i + 3] * inv);
        *reinterpret_cast<uint2*>(op + dt * 32 + 8 * i) = l == 0.f ? make_uint2(0, 0) : u;
      }
    if (A.lse && h == 0)
      A.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
    return;
  }
  const int64_t at = slot * rows + row;
  float* op = A.po + at * D + 4 * h;
#pragma unroll
  for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(op + dt * 32 + 8 * i) =
          make_float4(w.o[dt][4 * i], w.o[dt][4 * i + 1], w.o[dt][4 * i + 2], w.o[dt][4 * i + 3]);
  if (h == 0) A.pml[at] = make_float2(w.unit(), l);
}

// Joins a row's items: weights relative to the largest maximum. J groups of threads take every J-th
// four slots each, then the first joins the groups. Few rows have many slots, and one after the other
// each four cost the latency of a load (32 requests decoding, 1024 rows of 18 slots: 41 us a call with
// one group, 35 with four); many rows have enough loads in flight (4096 rows: 41 against 46 us).

struct Joined {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float m2, float l2, const float4& x) {
    const float mn = fmaxf(m, m2);
    const float a = __builtin_amdgcn_exp2f(m - mn), b = __builtin_amdgcn_exp2f(m2 - mn);
    l = l * a + l2 * b;
    o.x = o.x * a + x.x * b;
    o.y = o.y * a + x.y * b;
    o.z = o.z * a + x.z * b;
    o.w = o.w * a + x.w * b;
    m = mn;
  }
};

template <bool F16, int D, int J>
__global__ __launch_bounds__(256) void merge_kernel(Args A) {
  constexpr int LPR = D / 4, RPB = 256 / (LPR * J);  // lanes of a row and group; rows
  const int64_t n = (int64_t)A.N * A.B * A.Hq;
  const int local = threadIdx.x / LPR, group = local % J, d = threadIdx.x % LPR * 4;
  const int64_t row = min((int64_t)blockIdx.x * RPB + local / J, n - 1);
  const int token = (int)(row / A.Hq), hq = (int)(row % A.Hq);
  const int len = list_len(A, token / A.B);
  const int own = len - own_begin(len, A.B, A.shared);
  const int slots = A.slots_sh + (own ? (own - 1) / own_chunk(own, A.s_own, A.step_own) + 1 : 0);
  Joined all{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = group * 4; s0 < slots; s0 += 4 * J) {  // four slots' loads in flight
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = (int64_t)min(s0 + j, slots - 1) * n + row;
      ml[j] = A.pml[at];
      x[j] = *reinterpret_cast<const float4*>(A.po + at * D + d);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s0 + j < slots && ml[j].y != 0.f) all.add(ml[j].x, ml[j].y, x[j]);
  }
  __shared__ Joined s_part[256];
  s_part[threadIdx.x] = all;
  __syncthreads();
  if (group) return;
#pragma unroll
  for (int g = 1; g < J; ++g) {
    const Joined& p = s_part[threadIdx.x + g * LPR];
    if (p.l != 0.f) all.add(p.m, p.l, p.o);
  }
  const float inv = all.l == 0.f ? 0.f : 1.f / all.l;
  uint2 w;
  w.x = pack2<F16>(all.o.x * inv, all.o.y * inv);
  w.y = pack2<F16>(all.o.z * inv, all.o.w * inv);
  *reinterpret_cast<uint2*>(A.out + token * A.out_ld + (int64_t)hq * D + d) = w;
  if (A.lse && d == 0)
    A.lse[row] = all.l == 0.f ? -INFINITY : (all.m + log2f(all.l)) * 0.69314718056f;
}

template <bool F16, int D>
hipError_t launch_t(Args A, bool wide, hipStream_t s) {
  const int64_t own = (int64_t)A.Hkv * A.s_own * A.tiles_own * A.N;
  int64_t shared = (int64_t)A.Hkv * A.tiles_sh * A.s_sh;
  A.slots_sh = A.s_sh;
  A.step_own = narrow_step(D);
  A.direct = A.s_own == 1 && (wide || A.s_sh == 0);
  if constexpr (D == 128) if (wide) {
    hipLaunchKernelGGL((attend_kernel<F16, D, kWide, kWideStep>), dim3((unsigned)shared),
                       dim3(kWide * 64), 0, s, A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    shared = A.tiles_sh = A.s_sh = 0;  // done
  }
  bool slim = false;
  if constexpr (D == 256) slim = shared == 0 && A.B * A.G <= kSlim * 32 && own > kCUs;
  if (slim) {
    if constexpr (D == 256)
      hipLaunchKernelGGL((attend_kernel<F16, D, kSlim, narrow_step(D)>), dim3((unsigned)own),
                         dim3(kSlim * 64), 0, s, A);
  } else {
    hipLaunchKernelGGL((attend_kernel<F16, D, kNarrow, narrow_step(D)>),
                       dim3((unsigned)(shared + own)), dim3(kNarrow * 64), 0, s, A);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || A.direct) return e;
  const int64_t rows = (int64_t)A.N * A.B * A.Hq;
  const int groups = rows <= kFewRows ? 4 : 1, per = 256 / (D / 4 * groups);
  const dim3 grid((unsigned)((rows + per - 1) / per));
  if (groups == 4)
    hipLaunchKernelGGL((merge_kernel<F16, D, 4>), grid, dim3(256), 0, s, A);
  else
    hipLaunchKernelGGL((merge_kernel<F16, D, 1>), grid, dim3(256), 0, s, A);
  return hipGetLastError();
}

}  // namespace

size_t attention_scratch_bytes(const xpress_cache& c, int N, int B, int Hq) {
  return (size_t)most_row_slots(c, N, B, Hq) * B * Hq * (c.D * sizeof(float) + sizeof(float2));
}

int64_t attention_items(const xpress_cache& c, int N, int B, int Hq, int shared) {
  const AttendPlan p = plan_of(c, N, B, Hq, shared / kTile * kTile);
  return c.Hkv * ((int64_t)p.tiles_sh * p.s_sh + (int64_t)p.tiles_own * p.s_own * N);
}

hipError_t launch_block_attention(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                  const int32_t* seq, int N, int B, int Hq, float scale,
                                  int shared, void* out, int64_t out_ld, float* lse, void* ws,
                                  hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * c.Hkv * c.page * c.D;
  shared = shared / kTile * kTile;
  const AttendPlan p = plan_of(c, N, B, Hq, shared);
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
    case 64: return f16 ? launch_t<true, 64>(A, p.wide, s) : launch_t<false, 64>(A, p.wide, s);
    case 128: return f16 ? launch_t<true, 128>(A, p.wide, s) : launch_t<false, 128>(A, p.wide, s);
    default: return f16 ? launch_t<true, 256>(A, p.wide, s) : launch_t<false, 256>(A, p.wide, s);
  }
}

}  // namespace xpress
