// paged_common.h -- the batch plan over a paged FP8 cache as the kernels see
// it.  The plan's integers live on the device and are not trusted: every index
// that comes from them is clamped here, once.
#pragma once

#include "device_common.h"
#include "internal.h"

namespace fp8rt {

// One sequence's new tokens and positions.
struct SeqSpan {
  int64_t tok0;   // its first new token
  int32_t n;      // new tokens taken (at most max_new)
  int64_t first;  // position of its first new token (negative: kv_len below the number of new tokens)
  int64_t len;    // positions that exist: kv_len, at most the table's pages, at least 0
};

__device__ __forceinline__ SeqSpan seq_span(const PagedArgs& p, int64_t b) {
  SeqSpan s;
  int64_t t0 = p.seq_start[b], t1 = p.seq_start[b + 1];
  t0 = t0 < 0 ? 0 : t0 > p.tokens ? p.tokens : t0;
  t1 = t1 < t0 ? t0 : t1 > p.tokens ? p.tokens : t1;
  const int64_t len = p.kv_len[b];
  s.tok0 = t0;
  s.first = len - (t1 - t0);
  s.n = static_cast<int32_t>(t1 - t0 < p.max_new ? t1 - t0 : p.max_new);
  // positions stay 32-bit with room for a tile past the end
  const int64_t cap = p.width * p.page < 0x7FFF0000 ? p.width * p.page : 0x7FFF0000;
  s.len = len < 0 ? 0 : len < cap ? len : cap;
  return s;
}

// The page that holds logical page i of sequence b, or -1.
__device__ __forceinline__ int32_t page_of(const PagedArgs& p, int64_t b, int64_t i) {
  const int32_t pg = p.table[b * p.ld_table + i];
  return pg >= 0 && pg < p.pages ? pg : -1;
}

}  // namespace fp8rt
