// Attention of drafted blocks over the paged cache (gfx950).
#include "serve.hpp"
#include "cache_index.hpp"
#include "xpress_common.hpp"

namespace xpress {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Args {
  const uint16_t *q, *k, *v;  // k, v of the layer
  int64_t q_ld, out_ld;
  const int32_t *table, *len, *seq;
  int rows, ld, n_pages, shift;
  int N, B, Hq, Hkv, shared;
  float c;  // scale * log2(e)
  uint16_t* out;
  float* lse;
};

template <bool F16> __device__ __forceinline__ float value(uint16_t x) {
  return F16 ? (float)__builtin_bit_cast(_Float16, x) : bf16_to_f32(x);
}
template <bool F16> __device__ __forceinline__ uint16_t round_to(float x) {
  return F16 ? __builtin_bit_cast(uint16_t, (_Float16)x) : __builtin_bit_cast(uint16_t, (__bf16)x);
}

// One wave per query row (token, head): 64 keys at a time, a key a lane for the scores, D/64
// channels a lane for the sum.
template <bool F16, int D>
__global__ __launch_bounds__(64) void attend_kernel(Args A) {
  const int h = blockIdx.x % A.Hq, token = blockIdx.x / A.Hq, i = token / A.B, b = token % A.B;
  const int lane = threadIdx.x, hk = h / (A.Hq / A.Hkv);
  constexpr int E = D / 64;
  __shared__ float s_q[D];
  const int r = A.seq ? A.seq[i] : i, r0 = A.seq ? A.seq[0] : 0;
  const bool ok = (unsigned)r < (unsigned)A.rows;
  const int see = ok ? in_sight(clamp_len(A.len[r], A.ld, A.shift), A.B, b) : 0;
  for (int d = lane; d < D; d += 64) s_q[d] = value<F16>(A.q[token * A.q_ld + h * D + d]);
  __syncthreads();
  const int32_t* own = A.table + (int64_t)(ok ? r : 0) * A.ld;
  const int32_t* first = (unsigned)r0 < (unsigned)A.rows ? A.table + (int64_t)r0 * A.ld : own;
  float m = -1e30f, l = 0, o[E] = {};
  for (int t0 = 0; t0 < see; t0 += 64) {
    const int t = t0 + lane;
    const int at = min(t, see - 1);
    const int id = clamp_page((at < A.shared ? first : own)[at >> A.shift], A.n_pages);
    const int64_t off = line_offset(id, hk, at & ((1 << A.shift) - 1), A.Hkv, A.shift, D);
    float s = 0;
    for (int d = 0; d < D; ++d) s += s_q[d] * value<F16>(A.k[off + d]);
    s = t < see ? s * A.c : -INFINITY;
    float top = s;
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float mn = fmaxf(m, top), scale = exp2f(m - mn), p = exp2f(s - mn);
    l = l * scale + p;
    m = mn;
    for (int e = 0; e < E; ++e) o[e] *= scale;
    const int n = min(64, see - t0);
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl(p, j);
      const int64_t oj = __shfl(off, j);
      for (int e = 0; e < E; ++e) o[e] += pj * value<F16>(A.v[oj + lane * E + e]);
    }
  }
  for (int x = 32; x; x >>= 1) l += __shfl_xor(l, x);
  const float inv = l > 0 || l != l ? 1.f / l : 0.f;
  for (int e = 0; e < E; ++e)
    A.out[token * A.out_ld + h * D + lane * E + e] = round_to<F16>(o[e] * inv);
  if (A.lse && lane == 0)
    A.lse[(int64_t)token * A.Hq + h] = l == 0 ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
}

template <bool F16>
hipError_t launch_t(const Args& A, int D, hipStream_t s) {
  const dim3 grid((unsigned)(A.N * A.B * A.Hq));
  if (D == 64)
    hipLaunchKernelGGL((attend_kernel<F16, 64>), grid, dim3(64), 0, s, A);
  else if (D == 128)
    hipLaunchKernelGGL((attend_kernel<F16, 128>), grid, dim3(64), 0, s, A);
  else
    hipLaunchKernelGGL((attend_kernel<F16, 256>), grid, dim3(64), 0, s, A);
  return hipGetLastError();
}

}  // namespace

size_t attention_scratch_bytes(const xpress_cache& c, int N, int B, int Hq) { return 256; }

hipError_t launch_block_attention(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                  const int32_t* seq, int N, int B, int Hq, float scale,
                                  int shared, void* out, int64_t out_ld, float* lse, void* ws,
                                  hipStream_t s) {
  const int64_t at = (int64_t)layer * c.n_pages * c.Hkv * c.page * c.D;
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
  A.Hq = Hq;
  A.Hkv = c.Hkv;
  A.shared = shared;
  A.c = scale * 1.44269504089f;
  A.out = static_cast<uint16_t*>(out);
  A.lse = lse;
  return c.dtype == XPRESS_F16 ? launch_t<true>(A, c.D, s) : launch_t<false>(A, c.D, s);
}

}  // namespace xpress
