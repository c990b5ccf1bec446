// Host-side launchers of the target's side of a draft step (paged cache, block attention, draft
// verification). Arguments are validated by the C-ABI layer (serve_api.hip); each launcher only
// enqueues work on its stream.
#pragma once

#include "xpress.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace xpress {

size_t cache_scratch_bytes(const xpress_cache& c, int n_max);
hipError_t launch_cache_fork(const xpress_cache& c, const int32_t* src, const int32_t* dst, int n,
                             hipStream_t s);
hipError_t launch_cache_extend(const xpress_cache& c, const int32_t* seq, int N,
                               const int32_t* add, int add_all, int32_t* lacking, void* ws,
                               hipStream_t s);
hipError_t launch_cache_append(const xpress_cache& c, const int32_t* lacking, int layer,
                               const void* k_new, const void* v_new, int64_t ld_new,
                               const int32_t* seq, int N, int B, hipStream_t s);
hipError_t launch_cache_trim(const xpress_cache& c, const int32_t* lacking, const int32_t* seq, int N,
                             const int32_t* drop, hipStream_t s);
hipError_t launch_cache_compact(const xpress_cache& c, int32_t* live, void* ws, hipStream_t s);

size_t attention_scratch_bytes(const xpress_cache& c, int N, int B, int Hq);
int64_t attention_items(const xpress_cache& c, int N, int B, int Hq, int shared);  // workgroups
hipError_t launch_block_attention(const xpress_cache& c, int layer, const void* q, int64_t q_ld,
                                  const int32_t* seq, int N, int B, int Hq, float scale,
                                  int shared, void* out, int64_t out_ld, float* lse, void* ws,
                                  hipStream_t s);

size_t verify_scratch_bytes(int N, int B, int64_t V);
int64_t verify_items(int N, int B, int64_t V);  // workgroups
hipError_t launch_verify_draft(const void* logits, uint32_t logits_dtype, int64_t ld,
                               const int64_t* blk, const int32_t* draft_len, const void* q,
                               uint32_t q_dtype, int64_t q_ld, const float* temperature,
                               const float* u, int N, int B, int64_t V, int64_t* out,
                               int32_t* accepted, int32_t* drop, void* ws, hipStream_t s);

}  // namespace xpress
