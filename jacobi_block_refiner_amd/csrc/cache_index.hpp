// Index arithmetic of the paged cache, shared by its kernels and the attention that reads it.
// Plain integer functions (no device built-ins), so they compile for the host too.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define XP_HD __host__ __device__ __forceinline__
#else
#define XP_HD inline
#endif

namespace xpress {

// Pages that hold n tokens (n >= 0).
XP_HD int pages_of(int64_t n, int page_shift) {
  return (int)((n + ((int64_t)1 << page_shift) - 1) >> page_shift);
}

// A row's token count as the kernels use it: inside what its table can hold, whatever the buffer
// says.
XP_HD int clamp_len(int len, int64_t table_ld, int page_shift) {
  const int64_t most = table_ld << page_shift;
  const int64_t v = len < 0 ? 0 : len;
  return (int)(v < most ? v : most);
}

// A page id as the kernels use it for an address: inside the pool.
XP_HD int clamp_page(int id, int n_pages) {
  return id < 0 ? 0 : (id < n_pages ? id : n_pages - 1);
}
XP_HD bool page_ok(int id, int n_pages) { return id >= 0 && id < n_pages; }

// Rows that hold a page, by its count. A list that names a row twice may give its pages back twice and
// leave a count below 0: nobody holds such a page.
XP_HD int holders(int ref) { return ref > 0 ? ref : 0; }

// What an extension says of `total` pages wanted (up to 2^40) and `found` free ones: the pages that are
// missing, as far as an int holds them.
XP_HD int pages_missing(int64_t total, int64_t found) {
  const int64_t n = total > found ? total - found : 0;
  return (int)(n < INT32_MAX ? n : INT32_MAX);
}

// The two sides of a compaction to `live` pages (those with holders): a page that moves out of the
// pool's rest, and a free one of the front that takes it in. There are as many of one side as of the
// other, since all live pages fit in the front.
XP_HD bool moves_out(int ref, int p, int live) { return holders(ref) > 0 && p >= live; }
XP_HD bool takes_in(int ref, int p, int live) { return holders(ref) == 0 && p < live; }

// Element offset of line `line` of page `id`, head `h`, inside one layer of K or V. 64 bits: a
// layer of 2^16 pages of 64 tokens, 8 heads of 128 already holds 2^32 elements.
XP_HD int64_t line_offset(int id, int h, int line, int Hkv, int page_shift, int D) {
  return ((((int64_t)id * Hkv + h) << page_shift) + line) * D;
}

// Tokens in the sight of query b of a block of B that ends its row of `len` tokens.
XP_HD int in_sight(int len, int B, int b) {
  const int64_t v = (int64_t)len - B + b + 1;
  return v < 0 ? 0 : (int)v;
}

}  // namespace xpress
