// sdpa_operands.h -- what the front ends of the paged cache's operators share:
// checks of their operands, and where these overlap.
#pragma once
#include "../../include/sdpa.h"

#include <cstdint>
#include <utility>

#include "sdpa_internal.h"

namespace sdpa_host {

constexpr int64_t kIntMax = 0x7fffffffLL;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// An operand's memory: runs of `run` bytes at every combination of up to three
// steps (in bytes, positive).  `bytes`: from its first byte to behind its last one,
// 0 for an operand that is not there.
struct Block {
  uintptr_t p = 0;
  uint64_t run = 0, bytes = 0;
  int n = 0;
  int64_t extent[3], step[3];

  void add(int64_t ext, int64_t st) {
    if (ext <= 1) return;
    extent[n] = ext, step[n++] = st;
    bytes += static_cast<uint64_t>(ext - 1) * static_cast<uint64_t>(st);
  }
  void sort() {   // the largest step first
    for (int i = 1; i < n; ++i)
      for (int j = i; j > 0 && step[j - 1] < step[j]; --j) {
        std::swap(step[j - 1], step[j]);
        std::swap(extent[j - 1], extent[j]);
      }
  }
};

inline Block block_of(const void* p, uint64_t bytes) {
  Block b;
  b.p = reinterpret_cast<uintptr_t>(p);
  b.run = b.bytes = p ? bytes : 0;
  return b;
}

// Whether a's steps from ia on and b's from ib on reach a byte in common, b's
// beginning `shift` bytes behind a's; span_a, span_b: the bytes that they span.
// Operands cut from one buffer (queries, keys and values side by side, key and
// value pages of one pool) interleave without sharing: with s the larger step,
// places i s + x of a and shift + j s + y of b (x, y: below s) meet only where
// shift + (j - i) s is one of the two remainders between -s and s.  unknown: the
// answer where a step's inner part is longer than the step.
inline bool shares(const Block& a, int ia, int64_t span_a, const Block& b, int ib, int64_t span_b, int64_t shift, bool unknown) {
  if (shift >= span_a || -shift >= span_b) return false;
  if (ia == a.n && ib == b.n) return true;
  const int64_t sa = ia < a.n ? a.step[ia] : 0, sb = ib < b.n ? b.step[ib] : 0, s = sa > sb ? sa : sb;
  const int64_t na = sa == s ? a.extent[ia++] : 1, nb = sb == s ? b.extent[ib++] : 1;
  span_a -= (na - 1) * s;
  span_b -= (nb - 1) * s;
  if (span_a > s || span_b > s) return unknown;
  int64_t k = shift / s, r = shift % s;
  if (r < 0) r += s, --k;
  // j - i = -k, or -k - 1
  const auto possible = [&](int64_t d) { return d > -na && d < nb; };
  return (possible(-k) && shares(a, ia, span_a, b, ib, span_b, r, unknown)) ||
         (possible(-k - 1) && shares(a, ia, span_a, b, ib, span_b, r - s, unknown));
}
inline bool shares(Block a, Block b, bool unknown) {
  // (no operand of a program spans 2^62 bytes)
  if ((a.bytes | b.bytes) >> 62) return unknown;
  a.sort();
  b.sort();
  return shares(a, 0, static_cast<int64_t>(a.bytes), b, 0, static_cast<int64_t>(b.bytes),
                static_cast<int64_t>(b.p) - static_cast<int64_t>(a.p), unknown);
}
inline bool overlap(const Block& a, const Block& b, bool unknown = true) {
  return a.bytes != 0 && b.bytes != 0 && a.p < b.p + b.bytes && b.p < a.p + a.bytes && shares(a, b, unknown);
}

// [tokens, heads, D] of 16-bit elements with (token, head) strides.
struct Rows {
  const void* p;
  int64_t tokens, heads, dim, st, sh;

  Block block() const {
    Block b = block_of(p, 2ull * static_cast<uint64_t>(dim));
    if (p) b.add(tokens, 2 * st), b.add(heads, 2 * sh);
    return b;
  }
};

inline sdpa_status check_rows(const void* p, int64_t tokens, int64_t heads, int64_t dim,
                       const int64_t* stride, Rows* r) {
  *r = {p, tokens, heads, dim, tokens > 1 ? stride[0] : 0, heads > 1 ? stride[1] : 0};
  if (!aligned(p, 16)) return SDPA_ERR_LAYOUT;
  if (tokens > 1 && (r->st <= 0 || r->st % 8 != 0)) return SDPA_ERR_LAYOUT;
  if (heads > 1 && (r->sh <= 0 || r->sh % 8 != 0)) return SDPA_ERR_LAYOUT;
  if (r->st >= (int64_t(1) << 38) || r->sh >= (int64_t(1) << 38)) return SDPA_ERR_LAYOUT;
  return SDPA_OK;
}

inline bool in_16_to_1024(int64_t page_size) {
  return page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0;
}

inline sdpa_status check_cache(const sdpa_paged_cache* c, sdpa_dtype dtype) {
  if (!c || !c->k || !c->v) return SDPA_ERR_NULL;
  if (dtype != SDPA_BF16 && dtype != SDPA_FP16) return SDPA_ERR_DTYPE;
  const bool e4m3 = c->elem == SDPA_CACHE_E4M3;
  if (!e4m3 && c->elem != (dtype == SDPA_BF16 ? SDPA_CACHE_BF16 : SDPA_CACHE_FP16)) return SDPA_ERR_DTYPE;
  if (e4m3 && (!c->k_scale || !c->v_scale)) return SDPA_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128) return SDPA_ERR_SHAPE;
  if (!in_16_to_1024(c->page_size) || c->n_pages < 1 || c->n_pages > kIntMax || c->n_kv_heads < 1 ||
      c->n_kv_heads > kIntMax)
    return SDPA_ERR_SHAPE;
  const int64_t unit = e4m3 ? 16 : 8;  // elements of 16 bytes
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SDPA_ERR_LAYOUT;
  if (e4m3 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return SDPA_ERR_LAYOUT;
  const int64_t ext[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  for (const int64_t* st : {c->k_stride, c->v_stride})
    for (int i = 0; i < 3; ++i)
      if (ext[i] > 1 && (st[i] <= 0 || st[i] % unit != 0 || st[i] >= (int64_t(1) << 38))) return SDPA_ERR_LAYOUT;
  return SDPA_OK;
}

inline Block cache_block(const sdpa_paged_cache* c, const void* p, const int64_t* st) {
  const int64_t ext[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  const int64_t bytes = c->elem == SDPA_CACHE_E4M3 ? 1 : 2;
  Block b = block_of(p, static_cast<uint64_t>(c->head_dim * bytes));
  for (int i = 0; i < 3; ++i) b.add(ext[i], st[i] * bytes);
  return b;
}

// The batch's index arrays.
inline sdpa_status check_batch(const sdpa_paged_cache* c, int64_t total, const int32_t* table,
                        int64_t table_stride, int64_t max_pages, const int32_t* kv_lens,
                        const int32_t* cu, int64_t n_seqs) {
  if (!table || !kv_lens) return SDPA_ERR_NULL;
  if (total < 1 || n_seqs < 1 || max_pages < 1 || n_seqs > kIntMax - 1 || max_pages > kIntMax / c->page_size)
    return SDPA_ERR_SHAPE;
  if (!cu && total % n_seqs != 0) return SDPA_ERR_SHAPE;
  if (!aligned(table, 4) || !aligned(kv_lens, 4) || !aligned(cu, 4) || (n_seqs > 1 && table_stride < max_pages))
    return SDPA_ERR_LAYOUT;
  return SDPA_OK;
}

inline int log2_of(int64_t page_size) {
  int s = 0;
  while ((int64_t(1) << s) < page_size) ++s;
  return s;
}

// n / by = n mul >> shift for 0 <= n < 2^31: mul = floor(2^(31+s) / by) + 1 with
// 2^s >= by, so n mul is off from n 2^(31+s) / by by at most n < 2^31 parts of by
// <= 2^s, too little to reach the next multiple.
inline void divisor(int64_t by, unsigned int* mul, int* shift) {
  *shift = 31;
  while ((int64_t(1) << (*shift - 31)) < by) ++*shift;
  *mul = static_cast<unsigned int>((uint64_t(1) << *shift) / static_cast<uint64_t>(by) + 1);
}

// Byte strides (page, token, head); a dimension of one has none.
inline void byte_strides(const sdpa_paged_cache* c, const int64_t* st, int64_t* sp, int64_t* stok, int64_t* sh) {
  const int64_t bytes = c->elem == SDPA_CACHE_E4M3 ? 1 : 2;
  *sp = c->n_pages > 1 ? st[0] * bytes : 0;
  *stok = st[1] * bytes;
  *sh = c->n_kv_heads > 1 ? st[2] * bytes : 0;
}

}  // namespace sdpa_host
