// C ABI of the target's side of a draft step: argument checks of the paged cache, the block
// attention, the draft verification and the log probabilities of tokens. Every entry point validates
// on the host, then only enqueues kernels on the caller's stream.
#include "api_common.hpp"
#include "serve.hpp"

namespace {

using xpress::aligned_to;
using xpress::fail;
using xpress::up256;

hipStream_t hip_stream(xpress_stream s) { return reinterpret_cast<hipStream_t>(s); }

#define XP_WORDS(p)                                                                       \
  do {                                                                                    \
    if ((p) == nullptr) return fail(XPRESS_ERR_ARG, "%s is NULL", #p);                    \
    if (!aligned_to((p), 4)) return fail(XPRESS_ERR_ARG, "%s is not 4-byte aligned", #p); \
  } while (0)
#define XP_WORDS_OR_NULL(p) \
  do {                      \
    if ((p) != nullptr) XP_WORDS(p); \
  } while (0)

// Sizes of a cache; with `pools` its K and V pointers, with `tables` its metadata pointers.
xpress_status check_cache(const xpress_cache* c, bool pools, bool tables) {
  if (c == nullptr) return fail(XPRESS_ERR_ARG, "cache struct is NULL");
  if (c->n_layers < 1 || c->n_layers > 1 << 16)
    return fail(XPRESS_ERR_ARG, "n_layers=%d outside [1, 2^16]", c->n_layers);
  if (c->n_pages < 1 || c->n_pages > 1 << 24)
    return fail(XPRESS_ERR_ARG, "n_pages=%d outside [1, 2^24]", c->n_pages);
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
    return fail(XPRESS_ERR_ARG, "page=%d not in {16,32,64,128,256}", c->page);
  if (c->Hkv < 1 || c->Hkv > 256) return fail(XPRESS_ERR_ARG, "Hkv=%d outside [1, 256]", c->Hkv);
  if (c->D != 64 && c->D != 128 && c->D != 256)
    return fail(XPRESS_ERR_ARG, "D=%d not in {64,128,256}", c->D);
  if (c->rows < 1 || c->rows > 1 << 20)
    return fail(XPRESS_ERR_ARG, "rows=%d outside [1, 2^20]", c->rows);
  if (c->table_ld < 1 || c->table_ld > 1 << 20)
    return fail(XPRESS_ERR_ARG, "table_ld=%d outside [1, 2^20]", c->table_ld);
  if (c->dtype != XPRESS_BF16 && c->dtype != XPRESS_F16 && c->dtype != XPRESS_BF16_MX4 &&
      c->dtype != XPRESS_F16_MX4)
    return fail(XPRESS_ERR_ARG, "dtype=%u is not XPRESS_BF16, _F16, _BF16_MX4 or _F16_MX4", c->dtype);
  if (pools) {
    XP_PTR(c->k);
    XP_PTR(c->v);
  }
  if (tables) {
    XP_WORDS(c->table);
    XP_WORDS(c->len);
    XP_WORDS(c->ref);
  }
  return XPRESS_OK;
}

xpress_status check_rows(const xpress_cache* c, const int32_t* seq, int32_t N) {
  if (N < 0) return fail(XPRESS_ERR_ARG, "N=%d < 0", N);
  if (N > c->rows) return fail(XPRESS_ERR_ARG, "N=%d > rows=%d", N, c->rows);
  XP_WORDS_OR_NULL(seq);
  return XPRESS_OK;
}

// B tokens of each of N rows in one layer, a token every `ld` elements.
xpress_status check_block(const xpress_cache* c, int32_t layer, int32_t N, int32_t B, int64_t ld,
                          const char* name) {
  if (layer < 0 || layer >= c->n_layers)
    return fail(XPRESS_ERR_ARG, "layer=%d outside [0, %d)", layer, c->n_layers);
  if (B < 0) return fail(XPRESS_ERR_ARG, "B=%d < 0", B);
  if ((int64_t)N * B * c->Hkv >= (int64_t)1 << 26)
    return fail(XPRESS_ERR_ARG, "N*B*Hkv = %d*%d*%d is not below 2^26", N, B, c->Hkv);
  if (ld < (int64_t)c->Hkv * c->D || ld % 8)
    return fail(XPRESS_ERR_ARG, "%s=%lld must be >= Hkv*D=%d and a multiple of 8", name, (long long)ld,
                c->Hkv * c->D);
  return XPRESS_OK;
}

xpress_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  XP_PTR(ws);
  if (ws_bytes < need)
    return fail(XPRESS_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
  return XPRESS_OK;
}

xpress_status check_attention(const xpress_cache* c, int32_t N, int32_t B, int32_t Hq) {
  if (N < 0) return fail(XPRESS_ERR_ARG, "N=%d < 0", N);
  if (N > c->rows) return fail(XPRESS_ERR_ARG, "N=%d > rows=%d", N, c->rows);
  if (B < 1) return fail(XPRESS_ERR_ARG, "B=%d < 1", B);
  if (Hq < 1 || Hq % c->Hkv)
    return fail(XPRESS_ERR_ARG, "Hq=%d not a positive multiple of Hkv=%d", Hq, c->Hkv);
  if ((int64_t)N * B >= (int64_t)1 << 26 || (int64_t)N * B * Hq >= (int64_t)1 << 26)
    return fail(XPRESS_ERR_ARG, "N*B*Hq = %d*%d*%d is not below 2^26", N, B, Hq);
  return XPRESS_OK;
}

xpress_status check_verify(int32_t N, int32_t B, int64_t V) {
  if (N < 0) return fail(XPRESS_ERR_ARG, "N=%d < 0", N);
  if (B < 1 || B > 64) return fail(XPRESS_ERR_ARG, "B=%d outside [1, 64]", B);
  if (V < 1 || V >= (int64_t)1 << 31)
    return fail(XPRESS_ERR_ARG, "V=%lld outside [1, 2^31)", (long long)V);
  if ((int64_t)N * B >= (int64_t)1 << 24 || xpress::verify_items(N, B, V) >= (int64_t)1 << 24)
    return fail(XPRESS_ERR_ARG, "N=%d, B=%d, V=%lld is too large a launch", N, B, (long long)V);
  return XPRESS_OK;
}

xpress_status check_logprobs(int64_t rows, int64_t V, int32_t top) {
  if (rows < 0) return fail(XPRESS_ERR_ARG, "%lld rows < 0", (long long)rows);
  if (V < 1 || V >= (int64_t)1 << 31)
    return fail(XPRESS_ERR_ARG, "V=%lld outside [1, 2^31)", (long long)V);
  if (top < 0 || top > xpress::kMostTop)
    return fail(XPRESS_ERR_ARG, "top=%d outside [0, %d]", top, xpress::kMostTop);
  if (rows >= (int64_t)1 << 24 || xpress::logprobs_items(rows, V) >= (int64_t)1 << 24)
    return fail(XPRESS_ERR_ARG, "%lld rows of V=%lld are too large a launch", (long long)rows,
                (long long)V);
  return XPRESS_OK;
}

// Rows of V values of type code `dtype`, `ld` elements apart.
xpress_status check_values(const void* p, const char* name, uint32_t dtype, int64_t ld, int64_t V) {
  if (p == nullptr) return fail(XPRESS_ERR_ARG, "%s is NULL", name);
  if (dtype > XPRESS_F32) return fail(XPRESS_ERR_ARG, "%s: unknown type code %u", name, dtype);
  if (!aligned_to(p, dtype == XPRESS_F32 ? 4 : 2))
    return fail(XPRESS_ERR_ARG, "%s is not aligned to its elements", name);
  if (ld < V || ld >= (int64_t)1 << 31)
    return fail(XPRESS_ERR_ARG, "%s: row stride %lld outside [V=%lld, 2^31)", name, (long long)ld,
                (long long)V);
  return XPRESS_OK;
}

}  // namespace

extern "C" {

xpress_status xpress_cache_workspace_size(const xpress_cache* c, int32_t n_max, size_t* bytes) {
  if (bytes == nullptr) return fail(XPRESS_ERR_ARG, "bytes is NULL");
  xpress_status st = check_cache(c, false, false);
  if (st != XPRESS_OK) return st;
  if (n_max < 0) return fail(XPRESS_ERR_ARG, "n_max=%d < 0", n_max);
  *bytes = up256(xpress::cache_scratch_bytes(*c, n_max));
  return XPRESS_OK;
}

xpress_status xpress_cache_fork(const xpress_cache* c, const int32_t* src, const int32_t* dst,
                                int32_t n, xpress_stream stream) {
  xpress_status st = check_cache(c, false, true);
  if (st != XPRESS_OK) return st;
  if (n < 0 || n > c->rows) return fail(XPRESS_ERR_ARG, "n=%d outside [0, rows=%d]", n, c->rows);
  if (n == 0) return XPRESS_OK;
  XP_WORDS(src);
  XP_WORDS(dst);
  XP_TRY(xpress::launch_cache_fork(*c, src, dst, n, hip_stream(stream)), "cache fork");
  return XPRESS_OK;
}

xpress_status xpress_cache_extend(const xpress_cache* c, const int32_t* seq, int32_t N,
                                  const int32_t* add, int32_t add_all, int32_t* lacking, void* ws,
                                  size_t ws_bytes, xpress_stream stream) {
  xpress_status st = check_cache(c, true, true);
  if (st != XPRESS_OK) return st;
  st = check_rows(c, seq, N);
  if (st != XPRESS_OK) return st;
  if (add == nullptr && add_all < 0) return fail(XPRESS_ERR_ARG, "add_all=%d < 0", add_all);
  if (N == 0) return XPRESS_OK;
  XP_WORDS_OR_NULL(add);
  XP_WORDS(lacking);
  st = check_ws(ws, ws_bytes, xpress::cache_scratch_bytes(*c, N));
  if (st != XPRESS_OK) return st;
  XP_TRY(xpress::launch_cache_extend(*c, seq, N, add, add_all, lacking, ws, hip_stream(stream)),
         "cache extension");
  return XPRESS_OK;
}

xpress_status xpress_cache_append_if(const xpress_cache* c, const int32_t* lacking, int32_t layer,
                                     const void* k_new, const void* v_new, int64_t ld_new,
                                     const int32_t* seq, int32_t N, int32_t B,
                                     xpress_stream stream) {
  xpress_status st = check_cache(c, true, true);
  if (st != XPRESS_OK) return st;
  st = check_rows(c, seq, N);
  if (st != XPRESS_OK) return st;
  st = check_block(c, layer, N, B, ld_new, "ld_new");
  if (st != XPRESS_OK) return st;
  XP_WORDS_OR_NULL(lacking);
  if (N == 0 || B == 0) return XPRESS_OK;
  XP_PTR(k_new);
  XP_PTR(v_new);
  XP_TRY(xpress::launch_cache_append(*c, lacking, layer, k_new, v_new, ld_new, seq, N, B,
                                     hip_stream(stream)),
         "cache append");
  return XPRESS_OK;
}

xpress_status xpress_cache_append(const xpress_cache* c, int32_t layer, const void* k_new,
                                  const void* v_new, int64_t ld_new, const int32_t* seq, int32_t N,
                                  int32_t B, xpress_stream stream) {
  return xpress_cache_append_if(c, nullptr, layer, k_new, v_new, ld_new, seq, N, B, stream);
}

xpress_status xpress_cache_read(const xpress_cache* c, int32_t layer, const int32_t* seq, int32_t N,
                                const int32_t* first, int32_t B, void* k_out, void* v_out,
                                int64_t ld_out, xpress_stream stream) {
  xpress_status st = check_cache(c, true, true);
  if (st != XPRESS_OK) return st;
  st = check_rows(c, seq, N);
  if (st != XPRESS_OK) return st;
  st = check_block(c, layer, N, B, ld_out, "ld_out");
  if (st != XPRESS_OK) return st;
  XP_WORDS_OR_NULL(first);
  if (N == 0 || B == 0) return XPRESS_OK;
  XP_PTR(k_out);
  XP_PTR(v_out);
  XP_TRY(xpress::launch_cache_read(*c, layer, first, k_out, v_out, ld_out, seq, N, B,
                                   hip_stream(stream)),
         "cache read");
  return XPRESS_OK;
}

xpress_status xpress_cache_trim_if(const xpress_cache* c, const int32_t* lacking, const int32_t* seq,
                                   int32_t N, const int32_t* drop, xpress_stream stream) {
  xpress_status st = check_cache(c, false, true);
  if (st != XPRESS_OK) return st;
  st = check_rows(c, seq, N);
  if (st != XPRESS_OK) return st;
  XP_WORDS_OR_NULL(lacking);
  if (N == 0) return XPRESS_OK;
  XP_WORDS_OR_NULL(drop);
  XP_TRY(xpress::launch_cache_trim(*c, lacking, seq, N, drop, hip_stream(stream)), "cache trim");
  return XPRESS_OK;
}

xpress_status xpress_cache_trim(const xpress_cache* c, const int32_t* seq, int32_t N,
                                const int32_t* drop, xpress_stream stream) {
  return xpress_cache_trim_if(c, nullptr, seq, N, drop, stream);
}

xpress_status xpress_cache_compact(const xpress_cache* c, int32_t* live, void* ws, size_t ws_bytes,
                                   xpress_stream stream) {
  xpress_status st = check_cache(c, true, true);
  if (st != XPRESS_OK) return st;
  XP_WORDS(live);
  st = check_ws(ws, ws_bytes, xpress::cache_scratch_bytes(*c, 0));
  if (st != XPRESS_OK) return st;
  XP_TRY(xpress::launch_cache_compact(*c, live, ws, hip_stream(stream)), "cache compaction");
  return XPRESS_OK;
}

xpress_status xpress_attention_workspace_size(const xpress_cache* c, int32_t n_max, int32_t B,
                                              int32_t Hq, size_t* bytes) {
  if (bytes == nullptr) return fail(XPRESS_ERR_ARG, "bytes is NULL");
  xpress_status st = check_cache(c, false, false);
  if (st != XPRESS_OK) return st;
  st = check_attention(c, n_max, B, Hq);
  if (st != XPRESS_OK) return st;
  *bytes = up256(xpress::attention_scratch_bytes(*c, n_max, B, Hq));
  return XPRESS_OK;
}

xpress_status xpress_block_attention(const xpress_cache* c, int32_t layer, const void* q,
                                     int64_t q_ld, const int32_t* seq, int32_t N, int32_t B,
                                     int32_t Hq, float scale, int32_t shared, void* out,
                                     int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                     xpress_stream stream) {
  xpress_status st = check_cache(c, true, true);
  if (st != XPRESS_OK) return st;
  st = check_attention(c, N, B, Hq);
  if (st != XPRESS_OK) return st;
  XP_WORDS_OR_NULL(seq);
  if (layer < 0 || layer >= c->n_layers)
    return fail(XPRESS_ERR_ARG, "layer=%d outside [0, %d)", layer, c->n_layers);
  const int64_t width = (int64_t)Hq * c->D;
  if (q_ld < width || q_ld % 8 || out_ld < width || out_ld % 8)
    return fail(XPRESS_ERR_ARG, "q_ld=%lld and out_ld=%lld must be >= Hq*D=%lld and multiples of 8",
                (long long)q_ld, (long long)out_ld, (long long)width);
  if (!(scale > 0.f && scale <= 1e6f))
    return fail(XPRESS_ERR_ARG, "scale=%g outside (0, 1e6]", (double)scale);
  if (shared < 0 || shared > (int64_t)c->table_ld * c->page)
    return fail(XPRESS_ERR_ARG, "shared=%d outside [0, table_ld*page=%lld]", shared,
                (long long)c->table_ld * c->page);
  if (N == 0) return XPRESS_OK;
  if (xpress::attention_items(*c, N, B, Hq, shared) >= (int64_t)1 << 23)
    return fail(XPRESS_ERR_ARG, "N=%d, B=%d, Hq=%d over tables of %lld tokens is too large a launch",
                N, B, Hq, (long long)c->table_ld * c->page);
  XP_PTR(q);
  XP_PTR(out);
  XP_WORDS_OR_NULL(lse);
  st = check_ws(ws, ws_bytes, xpress::attention_scratch_bytes(*c, N, B, Hq));
  if (st != XPRESS_OK) return st;
  XP_TRY(xpress::launch_block_attention(*c, layer, q, q_ld, seq, N, B, Hq, scale, shared, out,
                                        out_ld, lse, ws, hip_stream(stream)),
         "block attention");
  return XPRESS_OK;
}

xpress_status xpress_verify_workspace_size(int32_t n_max, int32_t B, int64_t V, size_t* bytes) {
  if (bytes == nullptr) return fail(XPRESS_ERR_ARG, "bytes is NULL");
  xpress_status st = check_verify(n_max, B, V);
  if (st != XPRESS_OK) return st;
  *bytes = up256(xpress::verify_scratch_bytes(n_max, B, V));
  return XPRESS_OK;
}

xpress_status xpress_verify_draft(const void* logits, uint32_t logits_dtype, int64_t ld,
                                  const int64_t* blk, const int32_t* draft_len, const void* q,
                                  uint32_t q_dtype, int64_t q_ld, const float* temperature,
                                  const float* u, int32_t N, int32_t B, int64_t V, int64_t* out,
                                  int32_t* accepted, int32_t* drop, void* ws, size_t ws_bytes,
                                  xpress_stream stream) {
  xpress_status st = check_verify(N, B, V);
  if (st != XPRESS_OK) return st;
  if (N == 0) return XPRESS_OK;
  st = check_values(logits, "logits", logits_dtype, ld, V);
  if (st != XPRESS_OK) return st;
  if (q != nullptr) {
    st = check_values(q, "q", q_dtype, q_ld, V);
    if (st != XPRESS_OK) return st;
  }
  if (blk == nullptr || out == nullptr || !aligned_to(blk, 8) || !aligned_to(out, 8))
    return fail(XPRESS_ERR_ARG, "blk or out is NULL or not 8-byte aligned");
  XP_WORDS_OR_NULL(draft_len);
  XP_WORDS_OR_NULL(temperature);
  XP_WORDS_OR_NULL(drop);
  XP_WORDS(accepted);
  if (temperature != nullptr) XP_WORDS(u);
  st = check_ws(ws, ws_bytes, xpress::verify_scratch_bytes(N, B, V));
  if (st != XPRESS_OK) return st;
  XP_TRY(xpress::launch_verify_draft(logits, logits_dtype, ld, blk, draft_len, q, q_dtype, q_ld,
                                     temperature, u, N, B, V, out, accepted, drop, ws,
                                     hip_stream(stream)),
         "draft verification");
  return XPRESS_OK;
}

xpress_status xpress_logprobs_workspace_size(int32_t rows_max, int64_t V, int32_t top,
                                             size_t* bytes) {
  if (bytes == nullptr) return fail(XPRESS_ERR_ARG, "bytes is NULL");
  xpress_status st = check_logprobs(rows_max, V, top);
  if (st != XPRESS_OK) return st;
  *bytes = up256(xpress::logprobs_scratch_bytes(rows_max, V));
  return XPRESS_OK;
}

xpress_status xpress_token_logprobs(const void* logits, uint32_t logits_dtype, int64_t ld,
                                    const int64_t* token, const float* temperature, int32_t N,
                                    int32_t B, int64_t V, int32_t top, float* logprob,
                                    float* entropy, int32_t* rank, int64_t* top_ids,
                                    float* top_logprobs, void* ws, size_t ws_bytes,
                                    xpress_stream stream) {
  if (N < 0) return fail(XPRESS_ERR_ARG, "N=%d < 0", N);
  if (B < 1) return fail(XPRESS_ERR_ARG, "B=%d < 1", B);
  const int64_t rows = (int64_t)N * B;
  xpress_status st = check_logprobs(rows, V, top);
  if (st != XPRESS_OK) return st;
  if (N == 0) return XPRESS_OK;
  st = check_values(logits, "logits", logits_dtype, ld, V);
  if (st != XPRESS_OK) return st;
  if (!aligned_to(token, 8)) return fail(XPRESS_ERR_ARG, "token is not 8-byte aligned");
  XP_WORDS_OR_NULL(temperature);
  XP_WORDS_OR_NULL(logprob);
  XP_WORDS_OR_NULL(entropy);
  XP_WORDS_OR_NULL(rank);
  if (token == nullptr && (logprob != nullptr || rank != nullptr))
    return fail(XPRESS_ERR_ARG, "token is NULL: there is no logprob and no rank without it");
  if (top > 0) {
    if (top_ids == nullptr || !aligned_to(top_ids, 8))
      return fail(XPRESS_ERR_ARG, "top_ids is NULL or not 8-byte aligned");
    XP_WORDS(top_logprobs);
  }
  st = check_ws(ws, ws_bytes, xpress::logprobs_scratch_bytes(rows, V));
  if (st != XPRESS_OK) return st;
  XP_TRY(xpress::launch_token_logprobs(logits, logits_dtype, ld, token, temperature, N, B, V, top,
                                       logprob, entropy, rank, top_ids, top_logprobs, ws,
                                       hip_stream(stream)),
         "token log probabilities");
  return XPRESS_OK;
}

}  // extern "C"
