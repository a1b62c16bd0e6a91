// sdpa_paged_api.cpp -- C-ABI front end of the paged cache's operators:
// argument checks (all on the host, before any CUDA call) and launches.
#include "../../include/sdpa.h"

#include <cfloat>
#include <cmath>
#include <cstring>
#include <utility>

#include "sdpa_internal.h"

namespace {

constexpr int64_t kIntMax = 0x7fffffffLL;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

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

Block block_of(const void* p, uint64_t bytes) {
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
bool shares(const Block& a, int ia, int64_t span_a, const Block& b, int ib, int64_t span_b, int64_t shift, bool unknown) {
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
bool shares(Block a, Block b, bool unknown) {
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

sdpa_status check_rows(const void* p, int64_t tokens, int64_t heads, int64_t dim,
                       const int64_t* stride, Rows* r) {
  *r = {p, tokens, heads, dim, tokens > 1 ? stride[0] : 0, heads > 1 ? stride[1] : 0};
  if (!aligned(p, 16)) return SDPA_ERR_LAYOUT;
  if (tokens > 1 && (r->st <= 0 || r->st % 8 != 0)) return SDPA_ERR_LAYOUT;
  if (heads > 1 && (r->sh <= 0 || r->sh % 8 != 0)) return SDPA_ERR_LAYOUT;
  if (r->st >= (int64_t(1) << 38) || r->sh >= (int64_t(1) << 38)) return SDPA_ERR_LAYOUT;
  return SDPA_OK;
}

bool in_16_to_1024(int64_t page_size) {
  return page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0;
}

sdpa_status check_cache(const sdpa_paged_cache* c, sdpa_dtype dtype) {
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

Block cache_block(const sdpa_paged_cache* c, const void* p, const int64_t* st) {
  const int64_t ext[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  const int64_t bytes = c->elem == SDPA_CACHE_E4M3 ? 1 : 2;
  Block b = block_of(p, static_cast<uint64_t>(c->head_dim * bytes));
  for (int i = 0; i < 3; ++i) b.add(ext[i], st[i] * bytes);
  return b;
}

// The batch's index arrays.
sdpa_status check_batch(const sdpa_paged_cache* c, int64_t total, const int32_t* table,
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

int log2_of(int64_t page_size) {
  int s = 0;
  while ((int64_t(1) << s) < page_size) ++s;
  return s;
}

// Byte strides (page, token, head); a dimension of one has none.
void byte_strides(const sdpa_paged_cache* c, const int64_t* st, int64_t* sp, int64_t* stok, int64_t* sh) {
  const int64_t bytes = c->elem == SDPA_CACHE_E4M3 ? 1 : 2;
  *sp = c->n_pages > 1 ? st[0] * bytes : 0;
  *stok = st[1] * bytes;
  *sh = c->n_kv_heads > 1 ? st[2] * bytes : 0;
}

uint64_t workspace_bytes(const sdpa_impl::PagedForm& f, int64_t head_dim) {
  return static_cast<uint64_t>(f.ctas) *
         (sdpa_impl::kJoinNoteBytes + 2u * static_cast<uint64_t>(f.heads) * static_cast<uint64_t>(f.rows) * static_cast<uint64_t>(head_dim + 2) * 4u);
}

}  // namespace

extern "C" {

sdpa_status sdpa_cache_append(const sdpa_paged_cache* cache, const void* k, const void* v,
                              sdpa_dtype dtype, int64_t total, const int64_t* k_stride,
                              const int64_t* v_stride, const int32_t* page_table,
                              int64_t page_table_stride, int64_t max_pages,
                              const int32_t* kv_lens, const int32_t* cu_seqlens, int64_t n_seqs,
                              const float* cos, const float* sin, int64_t n_pos, int64_t rot_dim,
                              int interleaved, const void* q, void* q_out, int64_t n_heads,
                              const int64_t* q_stride, const int64_t* q_out_stride,
                              void* stream) {
  sdpa_status s = check_cache(cache, dtype);
  if (s != SDPA_OK) return s;
  if (!k || !v || !k_stride || !v_stride) return SDPA_ERR_NULL;
  if ((cos == nullptr) != (sin == nullptr)) return SDPA_ERR_NULL;
  if ((q == nullptr) != (q_out == nullptr)) return SDPA_ERR_NULL;
  if (q && (!q_stride || !q_out_stride)) return SDPA_ERR_NULL;
  if ((s = check_batch(cache, total, page_table, page_table_stride, max_pages, kv_lens, cu_seqlens, n_seqs)) !=
      SDPA_OK)
    return s;
  const int64_t D = cache->head_dim, hkv = cache->n_kv_heads;
  if (cos && (rot_dim < 8 || rot_dim > D || rot_dim % 8 != 0 || n_pos < 1)) return SDPA_ERR_SHAPE;
  if (q && (n_heads < 1 || n_heads > kIntMax)) return SDPA_ERR_SHAPE;
  // (the kernel counts page slots, total / page_size + 2 n_seqs, and shares of
  // heads in 32 bits)
  if (total > kIntMax / 2 || n_seqs > kIntMax / 8 || hkv > 65535 || (q && n_heads > kIntMax / 32))
    return SDPA_ERR_SHAPE;
  if (cos && (!aligned(cos, 16) || !aligned(sin, 16))) return SDPA_ERR_LAYOUT;
  Rows rk, rv, rq{}, ro{};
  if ((s = check_rows(k, total, hkv, D, k_stride, &rk)) != SDPA_OK) return s;
  if ((s = check_rows(v, total, hkv, D, v_stride, &rv)) != SDPA_OK) return s;
  if (q) {
    if ((s = check_rows(q, total, n_heads, D, q_stride, &rq)) != SDPA_OK) return s;
    if ((s = check_rows(q_out, total, n_heads, D, q_out_stride, &ro)) != SDPA_OK) return s;
  }
  {
    const bool e4m3 = cache->elem == SDPA_CACHE_E4M3;
    const uint64_t sb = 4ull * static_cast<uint64_t>(cache->n_pages) * static_cast<uint64_t>(hkv);
    const Block outs[4] = {cache_block(cache, cache->k, cache->k_stride), cache_block(cache, cache->v, cache->v_stride),
                           block_of(e4m3 ? cache->k_scale : nullptr, sb), block_of(e4m3 ? cache->v_scale : nullptr, sb)};
    const uint64_t tb = cos ? 4ull * static_cast<uint64_t>(n_pos) * static_cast<uint64_t>(rot_dim / 2) : 0;
    const Block ins[5] = {block_of(page_table, 4ull * static_cast<uint64_t>((n_seqs - 1) * page_table_stride + max_pages)),
                          block_of(kv_lens, 4ull * static_cast<uint64_t>(n_seqs)),
                          block_of(cu_seqlens, 4ull * static_cast<uint64_t>(n_seqs + 1)), block_of(cos, tb), block_of(sin, tb)};
    const Block bk = rk.block(), bv = rv.block(), bq = rq.block(), bo = ro.block();
    for (const Block& o : outs) {
      for (const Block& i : ins)
        if (overlap(o, i)) return SDPA_ERR_ARG;
      for (const Block* r : {&bk, &bv, &bq, &bo})
        if (overlap(o, *r)) return SDPA_ERR_ARG;
    }
    // keys' pages apart from the values' (refused where that is certain), scales
    // from the codes and from each other
    if (overlap(outs[0], outs[1], false) || overlap(outs[0], outs[2]) || overlap(outs[0], outs[3]) || overlap(outs[1], outs[2]) ||
        overlap(outs[1], outs[3]) || overlap(outs[2], outs[3]))
      return SDPA_ERR_ARG;
    if (q) {
      for (const Block& i : ins)
        if (overlap(bo, i)) return SDPA_ERR_ARG;
      const bool in_place = q == q_out && rq.st == ro.st && rq.sh == ro.sh;
      if ((!in_place && overlap(bo, bq)) || overlap(bo, bk) || overlap(bo, bv)) return SDPA_ERR_ARG;
    }
  }
  int dev = 0, sms = 0;
  s = static_cast<sdpa_status>(sdpa_impl::current_device(&dev, &sms));
  if (s != SDPA_OK) return s;
  sdpa_impl::AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = k;
  p.v = v;
  p.q = q;
  p.q_out = q_out;
  p.k_st = rk.st, p.k_sh = rk.sh, p.v_st = rv.st, p.v_sh = rv.sh;
  p.q_st = rq.st, p.q_sh = rq.sh, p.qo_st = ro.st, p.qo_sh = ro.sh;
  p.ck = static_cast<uint8_t*>(cache->k);
  p.cv = static_cast<uint8_t*>(cache->v);
  byte_strides(cache, cache->k_stride, &p.ck_sp, &p.ck_st, &p.ck_sh);
  byte_strides(cache, cache->v_stride, &p.cv_sp, &p.cv_st, &p.cv_sh);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.cos = cos;
  p.sin = sin;
  p.table = page_table;
  p.table_st = n_seqs > 1 ? page_table_stride : 0;
  p.kv_lens = kv_lens;
  p.cu = cu_seqlens;
  p.total = static_cast<int>(total);
  p.n_seqs = static_cast<int>(n_seqs);
  p.n_kv = static_cast<int>(hkv);
  p.H = q ? static_cast<int>(n_heads) : 0;
  p.n_pages = static_cast<int>(cache->n_pages);
  p.max_len = static_cast<int>(max_pages * cache->page_size);
  p.n_pos = cos ? static_cast<int>(n_pos < kIntMax ? n_pos : kIntMax) : 0;
  p.rot = cos ? static_cast<int>(rot_dim) : 0;
  p.interleaved = interleaved ? 1 : 0;
  p.page_shift = log2_of(cache->page_size);
  return sdpa_impl::launch_cache_append(p, static_cast<int>(D), dtype == SDPA_BF16,
                                        cache->elem == SDPA_CACHE_E4M3, sms,
                                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SDPA_OK
             : SDPA_ERR_CUDA;
}

uint64_t sdpa_paged_workspace_bytes(int64_t head_dim, int64_t n_heads, int64_t n_kv_heads,
                                    int64_t max_seqlen_q) {
  if ((head_dim != 64 && head_dim != 128) || n_kv_heads < 1 || n_heads < n_kv_heads ||
      n_heads % n_kv_heads != 0 || n_heads > kIntMax || max_seqlen_q < 1 || max_seqlen_q > kIntMax)
    return 0;
  int dev = 0, sms = 0;
  if (sdpa_impl::current_device(&dev, &sms) != SDPA_OK) return 0;
  // enough for a cache of either kind, and for the forms that fewer rows take
  const int64_t rows = max_seqlen_q * (n_heads / n_kv_heads);
  uint64_t most = 0;
  for (const bool e4m3 : {false, true})
    for (const int64_t r : {rows < 16 ? rows : 16, rows < 64 ? rows : 64, rows}) {
      const uint64_t n =
          workspace_bytes(sdpa_impl::paged_form(r, static_cast<int>(head_dim), e4m3, n_kv_heads, sms), head_dim);
      most = n > most ? n : most;
    }
  return most;
}

sdpa_status sdpa_paged_forward(const void* q, void* out, float* lse, sdpa_dtype dtype,
                               const sdpa_paged_cache* cache, int64_t total_q, int64_t n_heads,
                               const int64_t* q_stride, const int64_t* o_stride,
                               const int64_t* lse_stride, const int32_t* page_table,
                               int64_t page_table_stride, int64_t max_pages,
                               const int32_t* kv_lens, const int32_t* cu_seqlens_q,
                               int64_t n_seqs, int64_t max_seqlen_q, int is_causal, float scale,
                               void* workspace, uint64_t workspace_size, void* stream) {
  sdpa_status s = check_cache(cache, dtype);
  if (s != SDPA_OK) return s;
  if (!q || !out || !q_stride || !o_stride || !workspace || (lse && !lse_stride)) return SDPA_ERR_NULL;
  if ((s = check_batch(cache, total_q, page_table, page_table_stride, max_pages, kv_lens, cu_seqlens_q,
                       n_seqs)) != SDPA_OK)
    return s;
  const int64_t D = cache->head_dim, hkv = cache->n_kv_heads;
  if (n_heads < 1 || n_heads % hkv != 0 || max_seqlen_q < 1) return SDPA_ERR_SHAPE;
  const int64_t G = n_heads / hkv;
  if (total_q > (kIntMax - 1024) / G || max_pages * cache->page_size > kIntMax - 4096) return SDPA_ERR_SHAPE;
  Rows rq, ro;
  if ((s = check_rows(q, total_q, n_heads, D, q_stride, &rq)) != SDPA_OK) return s;
  if ((s = check_rows(out, total_q, n_heads, D, o_stride, &ro)) != SDPA_OK) return s;
  if (!aligned(workspace, 16)) return SDPA_ERR_LAYOUT;
  Block ls;
  int64_t lt = 0, lh = 0;
  if (lse) {
    lt = total_q > 1 ? lse_stride[0] : 0;
    lh = n_heads > 1 ? lse_stride[1] : 0;
    if (!aligned(lse, 4) || (total_q > 1 && lt <= 0) || (n_heads > 1 && lh <= 0)) return SDPA_ERR_LAYOUT;
    if (lt >= (int64_t(1) << 38) || lh >= (int64_t(1) << 38)) return SDPA_ERR_LAYOUT;
    ls = block_of(lse, 4);
    ls.add(total_q, 4 * lt), ls.add(n_heads, 4 * lh);
  }
  if (std::isinf(scale)) return SDPA_ERR_ARG;
  const bool e4m3 = cache->elem == SDPA_CACHE_E4M3;
  {
    const uint64_t sb = 4ull * static_cast<uint64_t>(cache->n_pages) * static_cast<uint64_t>(hkv);
    const Block ins[8] = {rq.block(),
                          cache_block(cache, cache->k, cache->k_stride),
                          cache_block(cache, cache->v, cache->v_stride),
                          block_of(e4m3 ? cache->k_scale : nullptr, sb),
                          block_of(e4m3 ? cache->v_scale : nullptr, sb),
                          block_of(page_table, 4ull * static_cast<uint64_t>((n_seqs - 1) * page_table_stride + max_pages)),
                          block_of(kv_lens, 4ull * static_cast<uint64_t>(n_seqs)),
                          block_of(cu_seqlens_q, 4ull * static_cast<uint64_t>(n_seqs + 1))};
    const Block outs[3] = {ro.block(), ls, block_of(workspace, workspace_size)};
    for (const Block& o : outs)
      for (const Block& i : ins)
        if (overlap(o, i)) return SDPA_ERR_ARG;
    if (overlap(outs[0], outs[1]) || overlap(outs[0], outs[2]) || overlap(outs[1], outs[2])) return SDPA_ERR_ARG;
  }
  int dev = 0, sms = 0;
  s = static_cast<sdpa_status>(sdpa_impl::current_device(&dev, &sms));
  if (s != SDPA_OK) return s;
  const int64_t max_rows = (max_seqlen_q < total_q ? max_seqlen_q : total_q) * G;
  const sdpa_impl::PagedForm form = sdpa_impl::paged_form(max_rows, static_cast<int>(D), e4m3, hkv, sms);
  {
    // the kernels count their steps in 31 bits
    const double units = static_cast<double>(total_q) * static_cast<double>(G) / form.rows + static_cast<double>(n_seqs);
    const double steps = static_cast<double>((max_pages * cache->page_size) >> form.step_shift) + 1.0;
    if (units * static_cast<double>(hkv / form.heads) * steps > 2.0e9) return SDPA_ERR_SHAPE;
  }
  if (workspace_size < workspace_bytes(form, D)) return SDPA_ERR_ARG;
  sdpa_impl::PagedParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q;
  p.q_st = rq.st, p.q_sh = rq.sh;
  p.out = out;
  p.o_st = ro.st, p.o_sh = ro.sh;
  p.out_sectors = aligned(out, 32) && ro.st % 16 == 0 && ro.sh % 16 == 0;
  p.lse = lse;
  p.lse_st = lt, p.lse_sh = lh;
  p.k = static_cast<const uint8_t*>(cache->k);
  p.v = static_cast<const uint8_t*>(cache->v);
  byte_strides(cache, cache->k_stride, &p.k_sp, &p.k_st, &p.k_sh);
  byte_strides(cache, cache->v_stride, &p.v_sp, &p.v_st, &p.v_sh);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.table = page_table;
  p.table_st = n_seqs > 1 ? page_table_stride : 0;
  p.kv_lens = kv_lens;
  p.cu = cu_seqlens_q;
  p.total_q = static_cast<int>(total_q);
  p.n_seqs = static_cast<int>(n_seqs);
  p.n_kv = static_cast<int>(hkv);
  p.G = static_cast<int>(G);
  // m = floor(2^(31+s) / G) + 1 with 2^s >= G: n m is off from n 2^(31+s) / G by
  // at most n < 2^31 parts of G <= 2^s, too little to reach the next multiple
  p.g_shift = 31;
  while ((int64_t(1) << (p.g_shift - 31)) < G) ++p.g_shift;
  p.g_mul = static_cast<unsigned int>((uint64_t(1) << p.g_shift) / static_cast<uint64_t>(G) + 1);
  p.seq_q = static_cast<int>(total_q / n_seqs);
  p.n_pages = static_cast<int>(cache->n_pages);
  p.max_len = static_cast<int>(max_pages * cache->page_size);
  p.page_shift = log2_of(cache->page_size);
  p.is_causal = is_causal ? 1 : 0;
  const double sc = std::isnan(scale) ? 1.0 / std::sqrt(static_cast<double>(D)) : static_cast<double>(scale);
  p.scale_log2 = static_cast<float>(sc * 1.4426950408889634);  // log2(e)
  p.part = static_cast<float*>(workspace);
  p.n_ctas = form.ctas;
  p.max_rows = static_cast<int>(max_rows);
  p.unit_heads = form.heads;
  p.n_groups = static_cast<int>(hkv) / form.heads;
  p.step_shift = form.step_shift;
  p.min_steps = form.min_steps;
  p.min_steps_shift = log2_of(form.min_steps);
  p.device = dev;
  cudaError_t e;
  if (form.tc) {
    // a zero scale: the smallest normal multiplier rounds every finite score
    // to 0 and keeps a removed one infinite (its sign does not matter)
    if (p.scale_log2 == 0.0f) p.scale_log2 = FLT_MIN;
    p.debug_withhold_q = sdpa_impl::withhold_q();
    p.wait_limit_ns = sdpa_impl::wait_limit_ns();
    CUtensorMap tm_k, tm_v;
    const int64_t ext[4] = {D, cache->page_size, hkv, cache->n_pages};
    const int64_t ks[3] = {p.k_st, p.k_sh, p.k_sp}, vs[3] = {p.v_st, p.v_sh, p.v_sp};
    const int box = static_cast<int>(cache->page_size < 128 ? cache->page_size : 128);
    const bool bf16 = dtype == SDPA_BF16;
    s = static_cast<sdpa_status>(sdpa_impl::encode_pages(cache->k, e4m3, bf16, ext, ks, box,
                                                         e4m3 ? static_cast<int>(D) : 128, &tm_k));
    if (s == SDPA_OK)
      s = static_cast<sdpa_status>(sdpa_impl::encode_pages(cache->v, e4m3, bf16, ext, vs, box, e4m3 ? 0 : 128, &tm_v));
    if (s != SDPA_OK) return s;
    e = sdpa_impl::launch_paged_tc(p, static_cast<int>(D), dtype == SDPA_BF16, e4m3, form.rows, tm_k, tm_v,
                                   static_cast<cudaStream_t>(stream));
  } else {
    e = sdpa_impl::launch_paged(p, static_cast<int>(D), dtype == SDPA_BF16, e4m3, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // extern "C"
