// sdpa_pages_api.cpp -- C-ABI front end of the operators on whole pages of a
// cache: argument checks (all on the host, before any CUDA call) and launches.
#include <cstring>

#include "sdpa_operands.h"

namespace {

using namespace sdpa_host;

sdpa_status check_pages(const sdpa_paged_cache* cache) {
  if (!cache) return SDPA_ERR_NULL;
  // (the cache's own type: nothing else is given)
  const sdpa_status s = check_cache(cache, cache->elem == SDPA_CACHE_FP16 ? SDPA_FP16 : SDPA_BF16);
  if (s != SDPA_OK) return s;
  return cache->n_kv_heads > 65535 ? SDPA_ERR_SHAPE : SDPA_OK;
}

sdpa_impl::PageBytes page_bytes(const sdpa_paged_cache* c) {
  sdpa_impl::PageBytes b;
  std::memset(&b, 0, sizeof(b));
  const bool e4m3 = c->elem == SDPA_CACHE_E4M3;
  b.p[0] = static_cast<uint8_t*>(c->k);
  b.p[1] = static_cast<uint8_t*>(c->v);
  b.scale[0] = e4m3 ? c->k_scale : nullptr;
  b.scale[1] = e4m3 ? c->v_scale : nullptr;
  byte_strides(c, c->k_stride, &b.sp[0], &b.st[0], &b.sh[0]);
  byte_strides(c, c->v_stride, &b.sp[1], &b.st[1], &b.sh[1]);
  b.n_pages = static_cast<int>(c->n_pages);
  b.n_kv = static_cast<int>(c->n_kv_heads);
  b.page_shift = log2_of(c->page_size);
  b.row_shift = log2_of(c->head_dim * (e4m3 ? 1 : 2) / 16);
  divisor(c->n_kv_heads, &b.h_mul, &b.h_shift);
  return b;
}

// Whether the cache's pages or scales (all written) meet one another or one of the
// operands.
bool cache_meets(const sdpa_paged_cache* c, const Block* ins, int n) {
  const bool e4m3 = c->elem == SDPA_CACHE_E4M3;
  const uint64_t sb = 4ull * static_cast<uint64_t>(c->n_pages) * static_cast<uint64_t>(c->n_kv_heads);
  const Block outs[4] = {cache_block(c, c->k, c->k_stride), cache_block(c, c->v, c->v_stride),
                         block_of(e4m3 ? c->k_scale : nullptr, sb), block_of(e4m3 ? c->v_scale : nullptr, sb)};
  for (const Block& o : outs)
    for (int i = 0; i < n; ++i)
      if (overlap(o, ins[i])) return true;
  return overlap(outs[0], outs[1], false) || overlap(outs[0], outs[2]) || overlap(outs[0], outs[3]) || overlap(outs[1], outs[2]) ||
         overlap(outs[1], outs[3]) || overlap(outs[2], outs[3]);
}

Block ints(const int32_t* p, int64_t n) { return block_of(p, 4ull * static_cast<uint64_t>(n)); }
Block rows_of(const int32_t* p, int64_t rows, int64_t columns, int64_t stride) {
  Block b = ints(p, columns);
  if (p) b.add(rows, 4 * stride);
  return b;
}

// A table of `rows` rows, row stride `stride` where there are several.
sdpa_status check_table(const int32_t* table, int64_t rows, int64_t columns, int64_t stride) {
  if (rows < 1 || columns < 1 || rows > kIntMax - 1 || columns > kIntMax) return SDPA_ERR_SHAPE;
  if (!aligned(table, 4) || (rows > 1 && (stride < columns || stride >= (int64_t(1) << 38)))) return SDPA_ERR_LAYOUT;
  return SDPA_OK;
}

sdpa_status check_accounts(const int32_t* refs, int64_t n_pages, const int32_t* table, int64_t rows, int64_t columns, int64_t stride,
                           int64_t page_size) {
  if (!refs || !table) return SDPA_ERR_NULL;
  if (n_pages < 1 || n_pages > (int64_t(1) << 30) || !in_16_to_1024(page_size)) return SDPA_ERR_SHAPE;
  const sdpa_status s = check_table(table, rows, columns, stride);
  if (s != SDPA_OK) return s;
  if (columns > kIntMax / page_size) return SDPA_ERR_SHAPE;
  return aligned(refs, 16) ? SDPA_OK : SDPA_ERR_LAYOUT;
}

sdpa_impl::PageTable table_of(int32_t* refs, int64_t n_pages, int32_t* table, int64_t rows, int64_t columns, int64_t stride,
                              int64_t page_size) {
  sdpa_impl::PageTable t;
  t.refs = refs;
  t.table = table;
  t.st = rows > 1 ? stride : 0;
  t.n_pages = static_cast<int>(n_pages);
  t.rows = static_cast<int>(rows);
  t.max_pages = static_cast<int>(columns);
  t.page_shift = log2_of(page_size);
  return t;
}

// Whether one of the outputs meets another operand.
bool any_meets(const Block* outs, int n_outs, const Block* ins, int n_ins) {
  for (int o = 0; o < n_outs; ++o) {
    for (int i = 0; i < n_ins; ++i)
      if (overlap(outs[o], ins[i])) return true;
    for (int i = o + 1; i < n_outs; ++i)
      if (overlap(outs[o], outs[i])) return true;
  }
  return false;
}

sdpa_status device_of(int* dev) {
  int sms = 0;
  return static_cast<sdpa_status>(sdpa_impl::current_device(dev, &sms));
}
sdpa_status launched(cudaError_t e) { return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA; }

}  // namespace

extern "C" {

sdpa_status sdpa_cache_copy_pages(const sdpa_paged_cache* cache, const int32_t* src, const int32_t* dst, const int32_t* rows,
                                  int64_t n, void* stream) {
  sdpa_status s = check_pages(cache);
  if (s != SDPA_OK) return s;
  if (!src || !dst) return SDPA_ERR_NULL;
  if (n < 1 || n > kIntMax / 2) return SDPA_ERR_SHAPE;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(rows, 4)) return SDPA_ERR_LAYOUT;
  sdpa_impl::CopyPagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = page_bytes(cache);
  const int64_t pieces = (cache->page_size * cache->n_kv_heads) << p.c.row_shift;
  p.slabs = static_cast<int>((pieces + sdpa_impl::kSlabPieces - 1) / sdpa_impl::kSlabPieces);
  if (n > kIntMax / 2 / p.slabs) return SDPA_ERR_SHAPE;
  const Block ins[3] = {ints(src, n), ints(dst, n), ints(rows, n)};
  if (cache_meets(cache, ins, 3)) return SDPA_ERR_ARG;
  int dev = 0;
  if ((s = device_of(&dev)) != SDPA_OK) return s;
  p.src = src;
  p.dst = dst;
  p.rows = rows;
  p.n = static_cast<int>(n);
  return launched(sdpa_impl::launch_copy_pages(p, static_cast<cudaStream_t>(stream)));
}

sdpa_status sdpa_cache_compact(const sdpa_paged_cache* cache, const int32_t* page_table, int64_t page_table_stride,
                               int64_t max_pages, const int32_t* kept, int64_t kept_stride, int64_t max_kept,
                               const int32_t* kept_lens, const int32_t* new_table, int64_t new_table_stride,
                               int64_t new_max_pages, int64_t n_seqs, void* stream) {
  sdpa_status s = check_pages(cache);
  if (s != SDPA_OK) return s;
  if (!page_table || !kept || !new_table) return SDPA_ERR_NULL;
  if ((s = check_table(page_table, n_seqs, max_pages, page_table_stride)) != SDPA_OK) return s;
  if ((s = check_table(kept, n_seqs, max_kept, kept_stride)) != SDPA_OK) return s;
  if ((s = check_table(new_table, n_seqs, new_max_pages, new_table_stride)) != SDPA_OK) return s;
  if (max_pages > kIntMax / cache->page_size || new_max_pages > kIntMax / cache->page_size) return SDPA_ERR_SHAPE;
  if (!aligned(kept_lens, 4)) return SDPA_ERR_LAYOUT;
  sdpa_impl::CompactPagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = page_bytes(cache);
  // a block takes as many heads as make 64 KB of a full page, at most 16 (8 x about
  // 7400 of 16384 tokens, us: 16 KB 49.7, its look at the lists weighs more; 32 KB 42.7; 64 KB 41.9)
  const int64_t head_bytes = cache->page_size << (p.c.row_shift + 4);
  while (p.unit_shift < 4 && (int64_t(1) << p.unit_shift) < cache->n_kv_heads && (head_bytes << p.unit_shift) < 65536)
    ++p.unit_shift;
  p.groups = static_cast<int>((cache->n_kv_heads + (1 << p.unit_shift) - 1) >> p.unit_shift);
  const int64_t pages = (max_kept + cache->page_size - 1) / cache->page_size;
  p.entries = static_cast<int>(pages < new_max_pages ? pages : new_max_pages);
  if (n_seqs > kIntMax / 2 / p.groups / p.entries) return SDPA_ERR_SHAPE;
  const Block ins[4] = {rows_of(page_table, n_seqs, max_pages, page_table_stride), rows_of(kept, n_seqs, max_kept, kept_stride),
                        ints(kept_lens, n_seqs), rows_of(new_table, n_seqs, new_max_pages, new_table_stride)};
  if (cache_meets(cache, ins, 4)) return SDPA_ERR_ARG;
  int dev = 0;
  if ((s = device_of(&dev)) != SDPA_OK) return s;
  p.table = page_table;
  p.table_st = n_seqs > 1 ? page_table_stride : 0;
  p.kept = kept;
  p.kept_st = n_seqs > 1 ? kept_stride : 0;
  p.kept_lens = kept_lens;
  p.new_table = new_table;
  p.new_st = n_seqs > 1 ? new_table_stride : 0;
  p.n_seqs = static_cast<int>(n_seqs);
  p.max_kept = static_cast<int>(max_kept);
  p.max_len = static_cast<int>(max_pages * cache->page_size);
  return launched(sdpa_impl::launch_compact_pages(p, cache->elem == SDPA_CACHE_E4M3, static_cast<cudaStream_t>(stream)));
}

sdpa_status sdpa_pages_fork(int32_t* refs, int64_t n_pages, const int32_t* page_table, int64_t page_table_stride, int64_t n_rows,
                            int32_t* new_table, int64_t new_table_stride, int64_t n_new_rows, int64_t max_pages,
                            int64_t page_size, const int32_t* kv_lens, const int32_t* src, const int32_t* dst, int64_t n,
                            int32_t* copy_src, int32_t* copy_dst, int32_t* copy_rows, int32_t* missing, void* stream) {
  sdpa_status s = check_accounts(refs, n_pages, page_table, n_rows, max_pages, page_table_stride, page_size);
  if (s != SDPA_OK) return s;
  if (!new_table || !kv_lens || !src || !dst || !copy_src || !copy_dst || !copy_rows || !missing) return SDPA_ERR_NULL;
  if ((s = check_table(new_table, n_new_rows, max_pages, new_table_stride)) != SDPA_OK) return s;
  if (n < 1 || n > sdpa_impl::kMostRequests) return SDPA_ERR_SHAPE;
  for (const void* p : {static_cast<const void*>(kv_lens), static_cast<const void*>(src), static_cast<const void*>(dst),
                        static_cast<const void*>(copy_src), static_cast<const void*>(copy_dst), static_cast<const void*>(copy_rows),
                        static_cast<const void*>(missing)})
    if (!aligned(p, 4)) return SDPA_ERR_LAYOUT;
  const bool same = new_table == page_table;
  // one table has one layout
  if (same && (n_new_rows != n_rows || (n_rows > 1 && new_table_stride != page_table_stride))) return SDPA_ERR_ARG;
  const Block table = rows_of(page_table, n_rows, max_pages, page_table_stride);
  const Block outs[6] = {ints(refs, n_pages), rows_of(new_table, n_new_rows, max_pages, new_table_stride), ints(copy_src, n),
                         ints(copy_dst, n), ints(copy_rows, n), ints(missing, 1)};
  const Block ins[4] = {ints(kv_lens, n_rows), ints(src, n), ints(dst, n), same ? Block{} : table};
  if (any_meets(outs, 6, ins, 4)) return SDPA_ERR_ARG;
  int dev = 0;
  if ((s = device_of(&dev)) != SDPA_OK) return s;
  sdpa_impl::ForkParams p;
  std::memset(&p, 0, sizeof(p));
  p.t = table_of(refs, n_pages, const_cast<int32_t*>(page_table), n_rows, max_pages, page_table_stride, page_size);
  p.new_table = new_table;
  p.new_st = n_new_rows > 1 ? new_table_stride : 0;
  p.new_rows = static_cast<int>(n_new_rows);
  p.same = same ? 1 : 0;
  p.lens = kv_lens;
  p.src = src;
  p.dst = dst;
  p.n = static_cast<int>(n);
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.copy_rows = copy_rows;
  p.missing = missing;
  return launched(sdpa_impl::launch_fork(p, dev, static_cast<cudaStream_t>(stream)));
}

sdpa_status sdpa_pages_take(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t page_table_stride, int64_t n_rows,
                            int64_t max_pages, int64_t page_size, const int32_t* from_lens, const int32_t* to_lens,
                            int32_t* missing, void* stream) {
  sdpa_status s = check_accounts(refs, n_pages, page_table, n_rows, max_pages, page_table_stride, page_size);
  if (s != SDPA_OK) return s;
  if (!from_lens || !to_lens || !missing) return SDPA_ERR_NULL;
  // (requests are counted in 31 bits)
  if (n_rows > sdpa_impl::kMostRequests || max_pages > kIntMax / n_rows) return SDPA_ERR_SHAPE;
  if (!aligned(from_lens, 4) || !aligned(to_lens, 4) || !aligned(missing, 4)) return SDPA_ERR_LAYOUT;
  const Block outs[3] = {ints(refs, n_pages), rows_of(page_table, n_rows, max_pages, page_table_stride), ints(missing, 1)};
  const Block ins[2] = {ints(from_lens, n_rows), ints(to_lens, n_rows)};
  if (any_meets(outs, 3, ins, 2)) return SDPA_ERR_ARG;
  int dev = 0;
  if ((s = device_of(&dev)) != SDPA_OK) return s;
  sdpa_impl::TakeParams p;
  std::memset(&p, 0, sizeof(p));
  p.t = table_of(refs, n_pages, page_table, n_rows, max_pages, page_table_stride, page_size);
  p.from = from_lens;
  p.to = to_lens;
  p.missing = missing;
  return launched(sdpa_impl::launch_take(p, dev, static_cast<cudaStream_t>(stream)));
}

sdpa_status sdpa_pages_release(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t page_table_stride, int64_t n_rows,
                               int64_t max_pages, int64_t page_size, const int32_t* rows, const int32_t* from_lens,
                               const int32_t* to_lens, int64_t n, void* stream) {
  sdpa_status s = check_accounts(refs, n_pages, page_table, n_rows, max_pages, page_table_stride, page_size);
  if (s != SDPA_OK) return s;
  if (n < 1 || (!rows && n > n_rows) || n > kIntMax / ((max_pages + 1023) / 1024)) return SDPA_ERR_SHAPE;
  if (!aligned(rows, 4) || !aligned(from_lens, 4) || !aligned(to_lens, 4)) return SDPA_ERR_LAYOUT;
  const Block outs[2] = {ints(refs, n_pages), rows_of(page_table, n_rows, max_pages, page_table_stride)};
  const Block ins[3] = {ints(rows, n), ints(from_lens, n), ints(to_lens, n)};
  if (any_meets(outs, 2, ins, 3)) return SDPA_ERR_ARG;
  int dev = 0;
  if ((s = device_of(&dev)) != SDPA_OK) return s;
  sdpa_impl::ReleaseParams p;
  std::memset(&p, 0, sizeof(p));
  p.t = table_of(refs, n_pages, page_table, n_rows, max_pages, page_table_stride, page_size);
  p.which = rows;
  p.from = from_lens;
  p.to = to_lens;
  p.n = static_cast<int>(n);
  return launched(sdpa_impl::launch_release(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
