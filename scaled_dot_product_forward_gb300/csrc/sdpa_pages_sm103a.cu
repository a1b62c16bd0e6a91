// sdpa_pages_sm103a.cu -- pages of a key/value cache as a whole: copying them,
// moving the tokens of a sequence that are kept together into new ones, and the
// accounts of who holds which, for sm_103a.
//
// Copies and compaction are bound by memory: each kept byte is read once and
// written once, in 16-byte pieces of a head's row, several in flight a thread.
//
// The accounts are a count of references a page and the page tables themselves.
// Counts are raised and lowered by atomic additions, whose sum does not depend
// on their order, and free pages (no references) are given out in rising order of
// their numbers to the requests in their order, so nothing depends on timing.
#include <cuda_fp8.h>

#include <atomic>

#include "sdpa_paged.cuh"

using namespace sdpa_dev;
using namespace sdpa_paged;
using sdpa_impl::CompactPagesParams;
using sdpa_impl::CopyPagesParams;
using sdpa_impl::ForkParams;
using sdpa_impl::PageBytes;
using sdpa_impl::PageTable;
using sdpa_impl::ReleaseParams;
using sdpa_impl::TakeParams;

namespace {

constexpr int kThreads = 256;

// Byte offset within a page of 16-byte piece u of its tokens' rows (token by
// token, head by head).
__device__ __forceinline__ int64_t piece_offset(const PageBytes& c, int which, int u) {
  const int r = u >> c.row_shift;
  const int token = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(r)) * c.h_mul) >> c.h_shift);
  const int head = r - token * c.n_kv;
  return token * c.st[which] + head * c.sh[which] + ((u & ((1 << c.row_shift) - 1)) << 4);
}

// A block: kSlabPieces pieces of one page's keys or values, eight a thread, all
// asked for before the first is written (2048 pages of 64 tokens, 8 heads of 128
// codes: 80 us, 6.7 TB/s, 99% of the measured copy rate).
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p) {
  constexpr int kPer = sdpa_impl::kSlabPieces / kThreads;
  grid_dependency_wait();
  grid_launch_dependents();
  const PageBytes& c = p.c;
  const unsigned block = blockIdx.x / static_cast<unsigned>(p.slabs);
  const int slab = static_cast<int>(blockIdx.x - block * p.slabs);
  const int i = static_cast<int>(block >> 1), which = static_cast<int>(block & 1);
  const int src = __ldg(p.src + i), dst = __ldg(p.dst + i);
  if (src < 0 || src >= c.n_pages || dst < 0 || dst >= c.n_pages || src == dst) return;
  const int P = 1 << c.page_shift;
  const int rows = p.rows != nullptr ? min(max(__ldg(p.rows + i), 0), P) : P;
  if (rows == 0) return;
  const int pieces = (rows * c.n_kv) << c.row_shift;
  const int first = slab * sdpa_impl::kSlabPieces + static_cast<int>(threadIdx.x);
  const uint8_t* from = c.p[which] + src * c.sp[which];
  uint8_t* to = c.p[which] + dst * c.sp[which];
  uint4 x[kPer];
  int64_t at[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int u = first + k * kThreads;
    at[k] = u < pieces ? piece_offset(c, which, u) : -1;
    if (at[k] >= 0) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (at[k] >= 0) *reinterpret_cast<uint4*>(to + at[k]) = x[k];
  if (slab == 0 && c.scale[which] != nullptr)
    for (int h = threadIdx.x; h < c.n_kv; h += kThreads)
      c.scale[which][static_cast<int64_t>(dst) * c.n_kv + h] = c.scale[which][static_cast<int64_t>(src) * c.n_kv + h];
}

// Sixteen e4m3 codes times a factor <= 1, each rounded once: in fp16, where a
// power of two down to 2^-14 makes no other rounding (a product that fp16 does not
// hold is far below half of e4m3's least step), else in fp32.
__device__ __forceinline__ uint4 scaled16(const uint4& x, float f) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const bool exact = (__float_as_uint(f) & 0x7fffffu) == 0 && f >= 6.103515625e-5f;
  const __half2 f2 = __float2half2_rn(f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 h(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((w[e] >> (16 * i)) & 0xffffu), __NV_E4M3)));
      uint32_t two;
      if (exact) {
        two = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(h, f2)), __NV_SATFINITE, __NV_E4M3);
      } else {
        const float2 v = __half22float2(h);
        two = __nv_cvt_float2_to_fp8x2(make_float2(v.x * f, v.y * f), __NV_SATFINITE, __NV_E4M3);
      }
      out |= two << (16 * i);
    }
    w[e] = out;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void copy_16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// A block: the tokens of one new page, 1 << unit_shift of their key or value
// heads, of which a thread has one 16-byte piece of every so many tokens.  e4m3:
// the new scale of a (page, head) is the largest of those under which its tokens
// came, so that no value grows; each block finds it for its heads, codes that
// came under that very scale are moved as they are.
//
// Bound by latency before memory: a row's place is behind two lists (a third for
// its scale), so what counts is that much is asked for at once.  The lists are
// read together, then eight pieces a thread go to shared memory by asynchronous
// copies, while the scales are compared.  8 x about 7400 of 16384 tokens, 8 heads of
// 128 codes: 42 us, 5.8 TB/s (47 with a batch of pieces in registers; without any
// conversion the same).
constexpr int kMove = 8;        // pieces of a thread at a time
struct CompactSmem {
  int data, from, old, total;   // byte offsets
  __host__ __device__ CompactSmem(bool e4m3, int tokens, int unit_shift) {
    data = 64;
    from = data + kMove * kThreads * 16;
    old = from + tokens * 8;
    total = old + (e4m3 ? (tokens << unit_shift) * 4 : 0);
  }
};
template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 6) compact_pages_kernel(const __grid_constant__ CompactPagesParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const PageBytes& c = p.c;
  const CompactSmem at(E4M3, 1 << c.page_shift, p.unit_shift);
  float* const s_scale = reinterpret_cast<float*>(smem);                 // [16] new scales
  int2* const s_from = reinterpret_cast<int2*>(smem + at.from);          // each token's old page (-1: none) and row
  float* const s_old = reinterpret_cast<float*>(smem + at.old);          // its scales, by head
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x);
  unsigned block = blockIdx.x;
  const int group = static_cast<int>(block % static_cast<unsigned>(p.groups));
  block /= static_cast<unsigned>(p.groups);
  const int which = static_cast<int>(block & 1);
  block >>= 1;
  const int entry = static_cast<int>(block % static_cast<unsigned>(p.entries));
  const int b = static_cast<int>(block / static_cast<unsigned>(p.entries));
  const int P = 1 << c.page_shift;
  const int* const kept = p.kept + b * p.kept_st + (static_cast<int64_t>(entry) << c.page_shift);
  const int* const table = p.table + b * p.table_st;
  const int listed = min(P, p.max_kept - (entry << c.page_shift));
  auto place = [&](int pos) { return pos >= 0 && pos < p.max_len ? __ldg(table + (pos >> c.page_shift)) : -1; };
  int pos = tid < listed ? __ldg(kept + tid) : -1;
  const int n = p.kept_lens != nullptr ? min(max(__ldg(p.kept_lens + b), 0), p.max_kept) : p.max_kept;
  const int page = __ldg(p.new_table + b * p.new_st + entry);
  int from = place(pos);
  const int count = min(P, n - (entry << c.page_shift));
  if (count <= 0 || page < 0 || page >= c.n_pages) return;
  const int unit = 1 << p.unit_shift, h0 = group << p.unit_shift, heads = min(unit, c.n_kv - h0);
  if (E4M3 && tid < 16) s_scale[tid] = 0.0f;
  for (int i = tid; i < count; i += kThreads) {
    if (i != tid) {
      pos = __ldg(kept + i);
      from = place(pos);
    }
    if (from >= c.n_pages) from = -1;
    s_from[i] = make_int2(from, pos & (P - 1));
  }
  __syncthreads();
  // this thread's piece of a token, and its tokens (a token has at most 256 pieces)
  const int per_token = p.unit_shift + c.row_shift;
  const int h = (tid >> c.row_shift) & (unit - 1);
  const int64_t piece = (h0 + h) * c.sh[which] + ((tid & ((1 << c.row_shift) - 1)) << 4);
  const uint8_t* const from0 = c.p[which] + piece;
  const int first = tid >> per_token, step = kThreads >> per_token;
  const int tokens = h < heads ? count : 0;
  uint8_t* const mine = smem + at.data + tid * 16;   // (a thread reads what it has asked for)
  const uint32_t mine_at = smem_addr(mine);
  auto ask = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kMove; ++k) {
      const int i = i0 + k * step;
      const int2 o = i < tokens ? s_from[i] : make_int2(-1, 0);
      if (o.x >= 0) copy_16(mine_at + k * (kThreads * 16), from0 + (o.x * c.sp[which] + o.y * c.st[which]));
    }
    cp_async_commit();
  };
  ask(first);
  if constexpr (E4M3) {
    // (a warp's lanes: as many tokens, head by head)
    for (int i0 = tid & ~31; i0 < count; i0 += kThreads) {
      const int i = i0 + (tid & 31), page_i = i < count ? s_from[i].x : -1;
      const float* const scales = c.scale[which] + static_cast<int64_t>(max(page_i, 0)) * c.n_kv + h0;
#pragma unroll 4
      for (int e = 0; e < heads; ++e) {
        const float y = page_i >= 0 ? clamp_scale(__ldg(scales + e)) : 0.0f;
        if (i < count) s_old[(i << p.unit_shift) + e] = y;
        // (positive: ordered as their bits are)
        const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(y));
        if ((tid & 31) == 0) atomicMax(reinterpret_cast<unsigned*>(s_scale + e), top);
      }
    }
    __syncthreads();
    if (tid < heads && s_scale[tid] > 0.0f)
      c.scale[which][static_cast<int64_t>(page) * c.n_kv + h0 + tid] = s_scale[tid];
  }
  uint8_t* to = c.p[which] + piece + page * c.sp[which] + first * c.st[which];
  const int64_t to_step = step * c.st[which];
  const float now = E4M3 ? s_scale[h] : 1.0f;
#pragma unroll 1
  for (int i0 = first; i0 < tokens; i0 += kMove * step) {
    if (i0 != first) ask(i0);
    cp_async_wait<0>();
#pragma unroll 4
    for (int k = 0; k < kMove; ++k) {
      const int i = i0 + k * step;
      if (i < tokens && s_from[i].x >= 0) {
        uint4 x = *reinterpret_cast<const uint4*>(mine + k * (kThreads * 16));
        if constexpr (E4M3) {
          const float old = s_old[(i << p.unit_shift) + h];
          if (old != now) x = scaled16(x, old / now);
        }
        *reinterpret_cast<uint4*>(to) = x;
      }
      to += to_step;
    }
  }
}

// ------------------------------------------------------------ accounts

__device__ __forceinline__ bool is_page(const PageTable& t, int page) { return page >= 0 && page < t.n_pages; }

// Entries of a sequence's full pages, and tokens of the one that is begun.
__device__ __forceinline__ void pages_of(const PageTable& t, int len, int& full, int& begun) {
  const int most = static_cast<int>(min(static_cast<int64_t>(t.max_pages) << t.page_shift, static_cast<int64_t>(0x7fffffff)));
  const int n = min(max(len, 0), most);
  full = n >> t.page_shift;
  begun = n & ((1 << t.page_shift) - 1);
}

// A fork's rows, or false where the pair names none (a row forked to itself is
// left as it is).
__device__ __forceinline__ bool fork_rows(const ForkParams& p, int i, int& src, int& dst) {
  src = __ldg(p.src + i);
  dst = __ldg(p.dst + i);
  return src >= 0 && src < p.t.rows && dst >= 0 && dst < p.new_rows && !(p.same && src == dst);
}

constexpr int kEntries = 4 * kThreads;   // of a block

// Entries e0, e0 + step, .. (four of them, below the row's end) of fork i's new
// row, which lose what they held and share the source's full pages.
__device__ __forceinline__ void fork_entries(const ForkParams& p, int i, int e0, int step) {
  int src, dst, full, begun;
  if (!fork_rows(p, i, src, dst)) return;
  pages_of(p.t, __ldg(p.lens + src), full, begun);
  const int* const from = p.t.table + src * p.t.st;
  int* const to = p.new_table + dst * p.new_st;
  int old[4], now[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int e = e0 + k * step;
    old[k] = now[k] = -1;
    if (e >= p.t.max_pages) continue;
    old[k] = to[e];
    if (e < full) now[k] = from[e];
    if (!is_page(p.t, now[k])) now[k] = -1;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int e = e0 + k * step;
    if (e >= p.t.max_pages || now[k] == old[k]) continue;
    if (is_page(p.t, old[k])) atomicAdd(p.t.refs + old[k], -1);
    if (now[k] >= 0) atomicAdd(p.t.refs + now[k], 1);
    to[e] = now[k];
  }
}

// A block: kEntries entries of a fork's new row.
__global__ void __launch_bounds__(kThreads) fork_entries_kernel(const __grid_constant__ ForkParams p, int slabs) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int i = static_cast<int>(blockIdx.x / static_cast<unsigned>(slabs));
  const int slab = static_cast<int>(blockIdx.x % static_cast<unsigned>(slabs));
  fork_entries(p, i, slab * kEntries + static_cast<int>(threadIdx.x), kThreads);
}

// A block: kEntries entries of a row; those of pages wholly within [from, to) are
// given up.
__global__ void __launch_bounds__(kThreads) release_kernel(const __grid_constant__ ReleaseParams p, int slabs) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int i = static_cast<int>(blockIdx.x / static_cast<unsigned>(slabs));
  const int slab = static_cast<int>(blockIdx.x % static_cast<unsigned>(slabs));
  const int row = p.which != nullptr ? __ldg(p.which + i) : i;
  if (row < 0 || row >= p.t.rows) return;
  const int shift = p.t.page_shift;
  const int from = p.from != nullptr ? max(__ldg(p.from + i), 0) : 0;
  const int e0 = (from >> shift) + ((from & ((1 << shift) - 1)) != 0 ? 1 : 0);
  const int e1 = p.to != nullptr ? min(max(__ldg(p.to + i), 0) >> shift, p.t.max_pages) : p.t.max_pages;
  int* const entries = p.t.table + row * p.t.st;
#pragma unroll
  for (int k = 0; k < kEntries / kThreads; ++k) {
    const int e = slab * kEntries + k * kThreads + static_cast<int>(threadIdx.x);
    if (e < e0 || e >= e1) continue;
    // (a row that is named twice gives up its pages once)
    const int page = atomicExch(entries + e, -1);
    if (is_page(p.t, page)) atomicAdd(p.t.refs + page, -1);
  }
}

// Giving out free pages.  Requests (FORK: the begun page of each pair; else the
// entries of each row) stand in a row, prefix sums over them in shared memory;
// the r-th free page goes to the r-th request.  One cluster of kCtas blocks walks
// over the counts, each thread 16 of them a round, and the blocks tell each other
// how many free ones they have found, and at first how many are wanted: whatever
// else writes to the tables meanwhile, all leave after the same round.  Bound by
// latency: a round is one trip to memory and one barrier of the cluster (taking
// pages for 128 rows from 32000: 3.8 us as a graph's node; the begun pages of 96
// forks, whose places are behind two more lists, 10).
constexpr int kCtas = 8, kPickThreads = 1024, kPickPages = 16;

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit word to the same place in block `rank`'s shared memory.
__device__ __forceinline__ void store_remote(const int* at, int rank, int value) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(smem_addr(at)),
      "r"(rank), "r"(value)
      : "memory");
}

// Exclusive sum over the block, and the block's total.
__device__ __forceinline__ int block_sum(int x, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  const int ws = scratch[lane];
  total = __reduce_add_sync(0xffffffffu, ws);
  return incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
}

__device__ __forceinline__ void entries_to_take(const TakeParams& p, int i, int& e0, int& n) {
  int f0, b0, f1, b1;
  pages_of(p.t, __ldg(p.from + i), f0, b0);
  pages_of(p.t, __ldg(p.to + i), f1, b1);
  e0 = f0 + (b0 != 0 ? 1 : 0);
  n = max(f1 + (b1 != 0 ? 1 : 0) - e0, 0);
}

// FUSED: the forks' other entries too, a warp's 128 at a time.
template <bool FORK, bool FUSED, class Params>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kPickThreads)
    pick_kernel(const __grid_constant__ Params p, int n) {
  extern __shared__ int prefix[];   // [n + 1]
  __shared__ int scratch[32];
  __shared__ int found[2][kCtas], wants[kCtas];
  const int tid = static_cast<int>(threadIdx.x), cta = static_cast<int>(blockIdx.x);
  const PageTable& t = p.t;
  if constexpr (!FUSED) cluster_arrive();
  grid_dependency_wait();
  grid_launch_dependents();
  if constexpr (FUSED) {
    const unsigned runs = static_cast<unsigned>((t.max_pages + 127) / 128);
    for (unsigned w = cta * (kPickThreads / 32) + (tid >> 5); w < runs * n; w += kCtas * (kPickThreads / 32))
      fork_entries(p, static_cast<int>(w / runs), static_cast<int>(w % runs) * 128 + (tid & 31), 32);
    __threadfence();
    cluster_arrive();   // (waited for below, before the counts are read)
  }
  // the requests
  auto request = [&](int i) -> int {
    if constexpr (FORK) {
      int src, dst, full, begun;
      if (!fork_rows(p, i, src, dst)) return 0;
      pages_of(t, __ldg(p.lens + src), full, begun);
      return begun != 0 && is_page(t, t.table[src * t.st + full]) ? 1 : 0;
    } else {
      int e0, m;
      entries_to_take(p, i, e0, m);
      return m;
    }
  };
  int wanted = 0;
  if (tid == 0) prefix[0] = 0;
  for (int i0 = 0; i0 < n; i0 += kPickThreads) {
    const int i = i0 + tid, m = i < n ? request(i) : 0;
    int total;
    const int before = block_sum(m, scratch, total);
    if (i < n) prefix[i + 1] = wanted + before + m;
    wanted += total;
  }
  __syncthreads();
  // request r gets a page (-1: none is left)
  auto give = [&](int r, int page) {
    int lo = 0, hi = n;   // prefix[lo] <= r < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= r)
        lo = mid;
      else
        hi = mid;
    }
    if constexpr (FORK) {
      int src, dst, full, begun;
      fork_rows(p, lo, src, dst);
      pages_of(t, __ldg(p.lens + src), full, begun);
      p.new_table[dst * p.new_st + full] = page;
      p.copy_src[lo] = t.table[src * t.st + full];
      p.copy_dst[lo] = page;
      p.copy_rows[lo] = begun;
    } else {
      int e0, m;
      entries_to_take(p, lo, e0, m);
      t.table[lo * t.st + e0 + (r - prefix[lo])] = page;
    }
  };
  cluster_wait();   // (all blocks are there)
  if (tid < kCtas) store_remote(&wants[cta], tid, wanted);
  int got = 0, most = wanted;
  for (int round = 0; ; ++round) {
    const int64_t page0 = (static_cast<int64_t>(round) * kCtas * kPickThreads + cta * kPickThreads + tid) * kPickPages;
    unsigned free_pages = 0;
    if (page0 + kPickPages <= t.n_pages) {
#pragma unroll
      for (int k = 0; k < kPickPages / 4; ++k) {
        const int4 x = __ldcg(reinterpret_cast<const int4*>(t.refs + page0) + k);
        free_pages |= ((x.x <= 0 ? 1u : 0u) | (x.y <= 0 ? 2u : 0u) | (x.z <= 0 ? 4u : 0u) | (x.w <= 0 ? 8u : 0u)) << (4 * k);
      }
    } else {
      for (int k = 0; k < kPickPages; ++k)
        if (page0 + k < t.n_pages && __ldcg(t.refs + page0 + k) <= 0) free_pages |= 1u << k;
    }
    int total;
    int r = got + block_sum(__popc(free_pages), scratch, total);
    if (tid < kCtas) store_remote(&found[round & 1][cta], tid, total);
    cluster_arrive();
    cluster_wait();
    int all = 0;
#pragma unroll
    for (int k = 0; k < kCtas; ++k) {
      if (round == 0) most = max(most, wants[k]);
      const int m = found[round & 1][k];
      if (k < cta) r += m;
      all += m;
    }
    got += all;
    for (; free_pages != 0 && r < wanted; ++r, free_pages &= free_pages - 1) {
      const int page = static_cast<int>(page0) + __ffs(static_cast<int>(free_pages)) - 1;
      t.refs[page] = 1;
      give(r, page);
    }
    if (got >= most || static_cast<int64_t>(round + 1) * kCtas * kPickThreads * kPickPages >= t.n_pages) break;
  }
  got = min(got, wanted);
  const int at = cta * kPickThreads + tid;
  if (at == 0) p.missing[0] = wanted - got;
  if constexpr (FORK) {
    // pairs that have nothing to copy
    for (int i = at; i < n; i += kCtas * kPickThreads)
      if (prefix[i + 1] == prefix[i] || prefix[i] >= got) p.copy_src[i] = -1, p.copy_dst[i] = -1, p.copy_rows[i] = 0;
  } else {
    for (int r = got + at; r < wanted; r += kCtas * kPickThreads) give(r, -1);
  }
}

template <class K, class... A>
cudaError_t launch_pdl(K kern, long long blocks, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool FORK, bool FUSED, class Params>
cudaError_t launch_pick(const Params& p, int n, int device, cudaStream_t stream) {
  auto kern = pick_kernel<FORK, FUSED, Params>;
  static std::atomic<uint64_t> configured{0};  // a bit a device
  const uint64_t bit = 1ull << device;
  if ((configured.load(std::memory_order_relaxed) & bit) == 0) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (sdpa_impl::kMostRequests + 1) * 4);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_pdl(kern, kCtas, kPickThreads, static_cast<size_t>(n + 1) * 4, stream, p, n);
}

// Forks with so many table entries at most are one launch, by eight blocks (as a graph
// 4 rows of 63 entries 7.2 us, in two launches 7.5, and 3 us less of the host's; 96
// rows of 515 13.7 and 12.6).
constexpr long long kFusedEntries = 16384;

int slabs_of(int max_pages) { return (max_pages + kEntries - 1) / kEntries; }

}  // namespace

namespace sdpa_impl {

cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t stream) {
  return launch_pdl(copy_pages_kernel, 2LL * p.n * p.slabs, kThreads, 0, stream, p);
}

cudaError_t launch_compact_pages(const CompactPagesParams& p, bool e4m3, cudaStream_t stream) {
  const long long blocks = 2LL * p.n_seqs * p.entries * p.groups;
  const CompactSmem at(e4m3, 1 << p.c.page_shift, p.unit_shift);
  return e4m3 ? launch_pdl(compact_pages_kernel<true>, blocks, kThreads, at.total, stream, p)
              : launch_pdl(compact_pages_kernel<false>, blocks, kThreads, at.total, stream, p);
}

cudaError_t launch_fork(const ForkParams& p, int device, cudaStream_t stream) {
  if (static_cast<long long>(p.n) * p.t.max_pages <= kFusedEntries) return launch_pick<true, true>(p, p.n, device, stream);
  const int slabs = slabs_of(p.t.max_pages);
  const cudaError_t e = launch_pdl(fork_entries_kernel, static_cast<long long>(p.n) * slabs, kThreads, 0, stream, p, slabs);
  return e != cudaSuccess ? e : launch_pick<true, false>(p, p.n, device, stream);
}

cudaError_t launch_take(const TakeParams& p, int device, cudaStream_t stream) {
  return launch_pick<false, false>(p, p.t.rows, device, stream);
}

cudaError_t launch_release(const ReleaseParams& p, cudaStream_t stream) {
  const int slabs = slabs_of(p.t.max_pages);
  return launch_pdl(release_kernel, static_cast<long long>(p.n) * slabs, kThreads, 0, stream, p, slabs);
}

}  // namespace sdpa_impl
