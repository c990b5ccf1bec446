// Attention of drafted blocks over a paged cache of 4 bits (gfx950).
#include "attend_kernel.hpp"

namespace xpress {

hipError_t launch_block_attention4(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                   const int32_t* seq, int N, int B, int Hq, float scale, int shared,
                                   void* out, int64_t out_ld, float* lse, void* ws, hipStream_t s) {
  shared = shared / kTile * kTile;
  const AttendPlan p = plan_of(c, N, B, Hq, shared);
  const Args A =
      args_of(c, p, layer, q, q_ld, seq, N, B, Hq, scale, shared, out, out_ld, lse, ws);
  return launch_values<true>(A, c.D, value_type(c) == XPRESS_F16, p.wide, s);
}

}  // namespace xpress
