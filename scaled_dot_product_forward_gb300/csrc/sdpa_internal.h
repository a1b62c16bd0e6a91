// sdpa_internal.h -- shared between the C-ABI front end and the kernel
// translation unit.  Not part of the public interface.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sdpa_impl {

// Kernel arguments; passed by value as a __grid_constant__ parameter so the
// TMA descriptors live in parameter space (no device allocation per call).
struct FwdParams {
  CUtensorMap tm_q;  // 4-D maps over (D, and L/H/B in stride order); box 64 x 128 rows
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  void* out;          // [B, H, L, D] with element strides below (inner stride 1)
  int64_t o_sb, o_sh, o_sl;
  const uint8_t* mask;  // [L, L] row-major bytes, nonzero = removed; null unless mask mode
  float* lse;           // optional [B, H, L] fp32 log-sum-exp per row (element strides below)
  int64_t lse_sb, lse_sh, lse_sl;
  int B, H, L;          // packed sequences: B = 1 and L = total rows
  int n_tiles;          // ceil(L / 128)
  // Packed sequences (null: dense [B, H, L, D]): sequence i is rows
  // [cu_seqlens[i], cu_seqlens[i+1]) of the L axis, attended on its own.
  const int* cu_seqlens;
  int n_seqs;
  long long max_units;  // upper bound on the number of work units (grid size)
  int snake;            // dense only: 1 = jobs by falling cost in snake order (small problems)
  float scale_log2;     // scale * log2(e)
  int pos_q[3], pos_k[3], pos_v[3];  // tensor-map coordinate slot (1..3) of L, H, B
  int mask_vec16;       // 1: mask rows may be read as 16-byte vectors (L % 16 == 0, aligned)
  // Optional tile summary of the explicit mask (both null: read the mask
  // bytes).  Tile (qt, kt) of the n_tiles x n_tiles grid of 128 x 128 tiles:
  // class byte tile_class[qt * n_tiles + kt] (kTileKept / kTileMixed /
  // kTileRemoved) and 128 rows of 128 bits at tile_bits[(qt * n_tiles + kt) *
  // 128 + row] (bit c of word w = key 32w + c removed; keys and rows past L
  // read as removed).
  const uint4* tile_bits;
  const uint8_t* tile_class;
  int debug_withhold_q; // test hook: 1 = never load Q, so every consumer wait runs out
  uint64_t wait_limit_ns;  // bound on any single barrier wait
};

// Tile classes of a mask summary, counting only entries inside [L, L].
enum TileClass : uint8_t { kTileKept = 0, kTileMixed = 1, kTileRemoved = 2 };

// Mask summary: one CTA per 128 x 128 tile of an [L, L] byte mask.
struct MaskTilesParams {
  const uint8_t* mask;  // [L, L] row-major, nonzero = removed
  int L, n_tiles;
  int vec16;            // rows may be read as 16-byte vectors
  uint16_t* bits;       // [n_tiles^2][128 rows][8] 16-bit words (the tile_bits layout)
  uint8_t* tile_class;  // [n_tiles^2]
};

// Sparse top-k attention: query row i (all heads of head group g) attends to
// the key rows idx[i, 0 .. len_i) of one shared key/value head.
struct SparseParams {
  CUtensorMap tm_q;  // 3-D (D, H, total_q), box 64 x min(H, 128) x 1 (one head group)
  void* out;                // [total_q, H, D]
  int64_t o_st, o_sh;
  float* lse;               // optional [total_q, H]
  int64_t lse_st, lse_sh;
  const int* idx;           // [total_q, topk] global key rows
  int64_t idx_st;
  const int* topk_length;   // [total_q] valid leading entries, or null (all topk)
  int total_q, total_k, H, topk, n_groups;
  int q_rows;               // heads of a group: min(H, 128)
  // 1 (H <= 64): M = 64 products, which put head h in TMEM lane
  // 32 (h / 16) + h % 16, and two softmax threads share each row; 0: M = 128
  // products, one thread a row
  int q_half;
  int kv_shared;            // 1: k and v are one tensor (gather once, use twice)
  const void* k;            // [total_k, D] rows for the gathers
  const void* v;
  int64_t k_row_bytes, v_row_bytes;
  float scale_log2;
  int debug_withhold_q;     // test hook: 1 = never load Q, so every consumer wait runs out
  uint64_t wait_limit_ns;
};

// Index preparation: per-document key positions -> global rows, holes removed.
struct CompactParams {
  const int* idx_local;
  int64_t in_st;
  int* idx_global;
  int64_t out_st;
  int* length;
  const int* cu_q;
  const int* cu_k;
  int total_q, topk, n_docs, is_causal;
};

cudaError_t launch_sparse(const SparseParams& p, int head_dim, bool bf16, int max_ctas,
                          cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);
// Reads and clears the sparse kernel's status word (its own translation unit).
cudaError_t read_and_clear_sparse_status(unsigned int* status);

enum MaskMode : int { kMaskNone = 0, kMaskCausal = 1, kMaskExplicit = 2 };

// Launches the persistent forward kernel for (head_dim, mask mode, dtype) on
// `stream` with at most max_ctas CTAs (one per SM: pass the device's SM
// count).  Returns the CUDA error of the launch.
cudaError_t launch_forward(const FwdParams& p, int head_dim, int mask_mode, bool bf16,
                           int max_ctas, cudaStream_t stream);
// The head-size-64 kernel (its own translation unit; launch_forward calls it).
cudaError_t launch_forward64(const FwdParams& p, int mask_mode, bool bf16, int max_ctas,
                             cudaStream_t stream);
// Reads and clears the head-size-64 kernel's status word.
cudaError_t read_and_clear_fwd64_status(unsigned int* status);

// Writes the tile summary of p.mask (PDL launch: waits for the previous
// kernel in the stream before reading the mask).
cudaError_t launch_mask_tiles(const MaskTilesParams& p, cudaStream_t stream);

// sdpa_forward_masked_noalloc: the mask summary lives in a fixed array in
// the library, enough for n_tiles <= kNoAllocMaxTiles.  Returns the device
// addresses of its bits and class parts for `device`, which must be current
// (looked up once per device with cudaGetSymbolAddress, then cached).
constexpr int kNoAllocMaxTiles = 32;
constexpr int kNoAllocMaxDevices = 64;
cudaError_t noalloc_mask_tiles(int device, const uint4** tile_bits, const uint8_t** tile_class);

// Attention over a paged cache (e4m3 or 16-bit).
struct PagedParams {
  const void* q;            // [total_q, H, D], element strides below
  int64_t q_st, q_sh;
  void* out;                // [total_q, H, D]
  int64_t o_st, o_sh;
  float* lse;               // optional [total_q, H]
  int64_t lse_st, lse_sh;
  const uint8_t* k;         // pages, BYTE strides below
  const uint8_t* v;
  int64_t k_sp, k_st, k_sh, v_sp, v_st, v_sh;
  const float* k_scale;     // e4m3: [n_pages, n_kv] (null for 16-bit caches)
  const float* v_scale;
  const int* table;         // [n_seqs, max_pages]
  int64_t table_st;
  const int* kv_lens;       // [n_seqs]
  const int* cu;            // [n_seqs + 1], or null: total_q / n_seqs tokens each
  int total_q, n_seqs, n_kv, G, n_pages, max_len;
  unsigned int g_mul;       // n / G = n g_mul >> g_shift, for 31-bit n (by_G)
  int g_shift;
  int seq_q;                // total_q / n_seqs
  int unit_heads, n_groups; // key/value heads of a unit, groups of them
  int step_shift;           // keys a step = 1 << step_shift
  int min_steps, min_steps_shift;  // at most one range for as many steps; a power of two
  int page_shift;           // page size = 1 << page_shift
  int is_causal;
  float scale_log2;
  int out_sectors;          // rows of out begin on 32-byte boundaries
  int max_rows;             // the caller's bound on a sequence's rows a head (>= 1)
  float* part;              // workspace: n_ctas notes, [n_ctas][2][unit_heads][rows of a unit][D + 2] floats
  int n_ctas;               // ranges of the division (grid of the main kernel)
  int device;               // the current device (below 64)
  int debug_withhold_q;     // test hook: 1 = no products are issued, so the waits run out
  uint64_t wait_limit_ns;
};

// Appending to a paged cache.
struct AppendParams {
  const void* k;            // [total, n_kv, D] 16-bit, element strides
  const void* v;
  const void* q;            // optional [total, H, D]
  void* q_out;
  int64_t k_st, k_sh, v_st, v_sh, q_st, q_sh, qo_st, qo_sh;
  uint8_t* ck;              // pages, BYTE strides
  uint8_t* cv;
  int64_t ck_sp, ck_st, ck_sh, cv_sp, cv_st, cv_sh;
  float* k_scale;           // e4m3: [n_pages, n_kv]
  float* v_scale;
  const float* cos;         // [n_pos, rot / 2], null: no rotation
  const float* sin;
  const int* table;
  int64_t table_st;
  const int* kv_lens;
  const int* cu;
  int total, n_seqs, n_kv, H, n_pages, max_len, n_pos, rot, interleaved, page_shift;
};

// The scales a cache may hold: positive, 2^-50 .. 2^50 (others are taken as
// the nearest of these, NaN and zero as the least).
constexpr int kScaleMinExp = -50, kScaleMaxExp = 50;

cudaError_t launch_cache_append(const AppendParams& p, int head_dim, bool bf16, bool e4m3, int sms,
                                cudaStream_t stream);
constexpr int kJoinNoteBytes = 32;  // a CTA's note at the workspace's start

// How a launch is divided: CTAs, rows and key/value heads of a unit, keys of
// a step, and whether it is the form for many rows (paged_tc).
struct PagedForm {
  int ctas, rows, heads, step_shift, min_steps;
  bool tc;
};
// CTAs an SM of the form for few rows.  They hide each other's latencies (a
// step is a chain of loads, conversions, two products and an exponential), as
// many as the registers and the rings leave room for.
constexpr int paged_per_sm(int head_dim, bool e4m3) { return head_dim == 64 ? 4 : e4m3 ? 3 : 2; }
// Up to 16 rows a head go to the form for few rows (sdpa_paged_sm103a.cu), up
// to 64 to the half-tile form of the other (sdpa_paged_tc_sm103a.cu), more to
// its full tiles.  16 sequences of 8192 tokens, 8 heads, us in the first form and
// in the second:
//                          8 rows      16 rows     24 rows
//   D 128, e4m3, bf16      72, 77      80, 78      103, 80
//   D 128, e4m3, fp16      67, 79      76, 80
//   D 128, 16-bit pages    91, 94      94, 95
//   D 64, e4m3             41, 60      45, 59      66, 60
//   D 64, 16-bit pages     55, 58      60, 58
// (24 rows are two tiles in the first form).  At 16 rows neither form is ahead
// throughout; one limit serves all of them, and is off by 2 us at most.
// 64 rows take 85 / 63 us in half tiles, 72 rows 101 / 87 in full ones (e4m3).
// The form for few rows has four warps, for up to four heads of a unit (as
// many as divide the heads; tokens' rows of neighbouring heads lie together,
// so reading them together keeps DRAM pages open), which share a head's keys
// when there are fewer: 16 keys of a head each a step.
inline PagedForm paged_form(int64_t max_rows, int head_dim, bool e4m3, int64_t n_kv, int sms) {
  if (max_rows > 16) return {sms, max_rows <= 64 ? 64 : 256, 1, 7, 2, true};
  const int heads = n_kv % 4 == 0 ? 4 : n_kv % 2 == 0 ? 2 : 1;
  return {paged_per_sm(head_dim, e4m3) * sms, 16, heads, heads == 4 ? 4 : heads == 2 ? 5 : 6, heads == 4 ? 4 : 2, false};
}
cudaError_t launch_paged(const PagedParams& p, int head_dim, bool bf16, bool e4m3, cudaStream_t stream);
// The form for many rows; tm_k, tm_v: 4-D maps of the pages (D, token, head,
// page), box min(page size, 128) tokens by 64 16-bit elements with the 128-byte
// swizzle, or by D codes, the keys' with the swizzle of D bytes, the values'
// without.
cudaError_t launch_paged_tc(const PagedParams& p, int head_dim, bool bf16, bool e4m3, int tile_rows,
                            const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream);
// Joins the units that the division cut.
cudaError_t launch_paged_join(const PagedParams& p, int head_dim, bool bf16, int tile_rows,
                                 cudaStream_t stream);
cudaError_t read_and_clear_paged_status(unsigned int* status);

// Tiled map of a cache's pages (the driver's encoder); an sdpa_status as an int.
int encode_pages(const void* ptr, bool e4m3, bool bf16, const int64_t* extents, const int64_t* byte_strides,
                 int box_tokens, int swizzle, CUtensorMap* map);
// The test hooks' settings.
uint64_t wait_limit_ns();
int withhold_q();

// The current device and its SM count; the status of the check that it is an
// sm_103 GPU (an sdpa_status as an int).
int current_device(int* device, int* sms);

// Reads and clears the device status word (nonzero = a barrier wait timed out).
cudaError_t read_and_clear_device_status(cudaStream_t stream, unsigned int* status);

}  // namespace sdpa_impl
