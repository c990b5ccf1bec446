// Attention of drafted blocks over a paged cache of 16-bit values (gfx950): the kernels of
// attend_kernel.hpp for it, and what the calls over either cache share on the host.
#include "attend_kernel.hpp"

namespace xpress {

size_t attention_scratch_bytes(const xpress_cache& c, int N, int B, int Hq) {
  const size_t slots =
      (size_t)most_row_slots(c, N, B, Hq) * B * Hq * (c.D * sizeof(float) + sizeof(float2));
  return cache_in_4_bits(c) ? up16(slots) + few_scratch_bytes(c, N, B, Hq) : slots;
}

int64_t attention_items(const xpress_cache& c, int N, int B, int Hq, int shared) {
  const AttendPlan p = plan_of(c, N, B, Hq, shared / kTile * kTile);
  return c.Hkv * ((int64_t)p.tiles_sh * p.s_sh + (int64_t)p.tiles_own * p.s_own * N);
}

hipError_t launch_block_attention(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                  const int32_t* seq, int N, int B, int Hq, float scale,
                                  int shared, void* out, int64_t out_ld, float* lse, void* ws,
                                  hipStream_t s) {
  if (cache_in_4_bits(c))
    return launch_block_attention4(c, layer, q, q_ld, seq, N, B, Hq, scale, shared, out, out_ld, lse,
                                   ws, s);
  shared = shared / kTile * kTile;
  const AttendPlan p = plan_of(c, N, B, Hq, shared);
  const Args A =
      args_of(c, p, layer, q, q_ld, seq, N, B, Hq, scale, shared, out, out_ld, lse, ws);
  return launch_values<false>(A, c.D, value_type(c) == XPRESS_F16, p.wide, s);
}

}  // namespace xpress
