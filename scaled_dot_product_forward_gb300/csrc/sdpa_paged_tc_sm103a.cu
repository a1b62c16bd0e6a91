// sdpa_paged_tc_sm103a.cu -- attention of many new tokens a sequence over a
// paged key/value cache, on the fifth-generation tensor cores (sm_103a): the
// rows of a key/value head (tokens times the query heads that share it) are
// more than the few that sdpa_paged_sm103a.cu is made for.
//
// Same mathematics as there, tiles as in the dense forward: a step is 128
// keys; S = Q K^T and O += P V are M = 128 tcgen05 products with S, P and O
// in tensor memory, two softmax warpgroups (one row a thread) alternate on
// the tensor core.  A unit is up to 256 rows of a sequence and head:
//   * more than 128: warpgroup t owns rows 128 t .. of the unit, both read
//     every key tile;
//   * at most 128: both own the same rows and take the key tiles in turn
//     (even steps, odd steps), so that a unit with few rows, bound by memory
//     or by the softmax's latency, still keeps both at work; their sums are
//     joined at the end through tensor memory, each thread of one reading the
//     other's lane.
// When no sequence has more than 64 rows a head, units have 64 and take the
// second way with M = 64 products, which put row h in lane 32 (h / 16) + h % 16;
// two threads share a row, each half of a step's keys and of the columns
// (HALF; five tokens of 16 sequences, 40 rows a head: 119 -> 97 us).
// Pages arrive by TMA (one box a page and 128-byte column chunk; an entry that
// is no page lies out of the map's bounds and reads as zeros).  16-bit pages
// land in the 128-byte-swizzled layout that the products read.  e4m3 pages
// land as they are in a small ring; the keys' are multiplied as they are, with
// the queries split into 8-bit terms, and a warpgroup turns the values' into
// fp16 tiles (exact); a key's weight carries its page's value scale, so the
// scales touch eight constants a row and step, not the elements.
//
// The steps of all units are divided equally over the CTAs (one an SM), the
// two cut units of a CTA joined by a second kernel (sdpa_paged.cuh).  Every
// wait is bounded in time; on expiry the CTA records a status bit, stops, lets
// what it issued land and frees its tensor memory.
#include <atomic>

#include <cuda_fp8.h>

#include "sdpa_paged.cuh"
#include "sdpa_sched.cuh"

using namespace sdpa_dev;
using namespace sdpa_paged;

__device__ unsigned int g_sdpa_paged_status = 0;

namespace {

constexpr int KT = 128;        // keys a step
// Rows of a unit, and of a softmax warpgroup's tile.  HALF: see below.
__host__ __device__ constexpr int unit_rows(bool half) { return half ? 64 : 256; }
__host__ __device__ constexpr int tile_rows(bool half) { return half ? 64 : 128; }
// Warp 0 loads the keys and writes the notes on each step, warp 2 loads the
// values, warp 1 issues the products; warpgroups 1 and 2 are the softmax; with
// e4m3 pages warpgroup 3 converts.  The register splits exhaust the launch's
// 64K.
template <bool E4M3>
struct Split {
  static constexpr int kThreads = E4M3 ? 512 : 384;
  static constexpr uint32_t kLaunch = E4M3 ? 128 : 168;
  static constexpr uint32_t kControl = E4M3 ? 64 : 80;   // and conversion
  static constexpr uint32_t kSoftmax = E4M3 ? 192 : 208;
  static_assert((kThreads - 256) * kControl + 256 * kSoftmax <= kThreads * kLaunch,
                "register split exceeds the launch allocation");
};
constexpr int kConvertWarps = 4;
constexpr uint32_t kSuspendNs = 4000;  // a waiting thread may sleep this long between its looks
constexpr uint32_t kTmemCols = 512;  // S_0 [0,128), S_1 [128,256), O_0 [256,384), O_1 [384,512)
constexpr int kGroups = KT / 16;     // 16 keys lie in one page

// Terms of a query row for products with e4m3 keys, the first in e4m3 (four
// significant bits), the others in e5m2 (three, and the sign of what is left is
// one more): two carry a bf16 value, three an fp16 one.
__host__ __device__ constexpr int q_terms(bool e4m3, bool bf16) { return !e4m3 ? 1 : bf16 ? 2 : 3; }

template <int D, bool E4M3, bool BF16, bool HALF>
struct Lay {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = KT * 128;
  static constexpr int kTile = kChunks * kChunkBytes;      // 128 rows of 16-bit elements
  static constexpr int kCodes = KT * D;                    // 128 rows of codes
  static constexpr int kQRows = tile_rows(HALF);
  static constexpr int kQChunk = kQRows * (E4M3 ? D : 128);   // a term, or 64 columns
  static constexpr int kQTile = (E4M3 ? q_terms(E4M3, BF16) : kChunks) * kQChunk;
  static constexpr int kKTile = E4M3 ? kCodes : kTile;
  static constexpr int kKStages = D == 64 ? 4 : !E4M3 ? 3 : (BF16 ? 3 : 2) + (HALF ? 1 : 0);
  static constexpr int kVStages = D == 64 ? (E4M3 ? 3 : 4) : !E4M3 && HALF ? 3 : 2;
  static constexpr int kRawStages = !E4M3 ? 0 : D == 64 || HALF ? 4 : BF16 ? 3 : 2;  // V's codes
  // Notes on a step (its pages' scales), written when step x's keys have been
  // asked for: S of step x - K stages is complete then, and so (S is issued
  // behind the product that needs the weights of two steps before, at most)
  // the softmax of every step up to x - K stages - 2.
  static constexpr int kNotes = 8;
  static_assert(kNotes >= kKStages + 2, "notes are rewritten before they are read");
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kQTile;
  static constexpr int kV = kK + kKStages * kKTile;
  static constexpr int kRaw = kV + kVStages * kTile;
  static constexpr int kNote = kRaw + kRawStages * kCodes;
  static constexpr int kBar = kNote + (E4M3 ? kNotes * kGroups * 16 : 0);
  static constexpr int kCursors = kBar + 512;   // the softmax warps' places (8 x 64 bytes)
  static constexpr int kTotal = kCursors + 512 + 1024;
  static_assert(kTotal <= 227 * 1024, "shared memory over the per-CTA limit");
};

struct Bars {
  uint64_t q_full[2];   // a warpgroup's Q is written, its last unit's rows are read out
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t sums, read;  // alternating steps: both warpgroups' sums are in tensor memory; are read
  uint64_t fin;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], raw_full[4], raw_empty[4];
  uint64_t note[8];
  int valid[4];         // a raw tile's rows before the sequence's end
  uint32_t bad[8];      // a step's groups of 16 keys without a page
  uint32_t tmem_base, abort_flag;
};

enum Site : unsigned int {
  kSiteQ = 1u << 1, kSiteK = 1u << 2, kSiteEmpty = 1u << 3, kSiteS = 1u << 4, kSiteP = 1u << 5,
  kSiteO = 1u << 6, kSiteDrain = 1u << 7, kSiteV = 1u << 8, kSiteNote = 1u << 9, kSiteSums = 1u << 10,
};

// mbar_try_wait with a hint how long (ns) the thread may be suspended meanwhile.
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(ns)
      : "memory");
  return done != 0;
}

// All roles' loops together have to fit the instruction cache, and this stands in
// each of them at every wait: a wait that gives up only raises the flag, which
// thread 0 reports at the end (with that, rolled loops where little runs, and
// divisions by multiplication, 106 -> 96 KB of code with e4m3 pages: a chunk of
// 2048 tokens behind 14336 445 -> 441 us, with 16-bit pages 424 -> 392; uneven
// prompts, 16-bit 597 -> 541, e4m3 742 -> 661).
__device__ __forceinline__ bool wait_any(uint64_t* bar, uint32_t parity, Bars* bars, uint64_t limit,
                                         unsigned int site, bool honour_abort = true) {
  uint64_t t0 = 0;
  while (!mbar_try_wait_for(bar, parity, kSuspendNs)) {
    volatile uint32_t* const flag = &bars->abort_flag;
    if (honour_abort && *flag != 0) return false;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit) {
      *flag = 1u | site;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars* bars, uint64_t limit,
                                          unsigned int site) {
  return __all_sync(0xffffffffu, wait_any(bar, parity, bars, limit, site));
}

// A position in a ring of N slots.
template <int N>
struct RingAt {
  int idx = 0;
  uint32_t phase = 0;
  bool lapped = false;
  __device__ __forceinline__ void next() {
    if (++idx == N) {
      idx = 0;
      phase ^= 1u;
      lapped = true;
    }
  }
};

// One CTA's share of one unit: steps [s0, s1) of c's unit.
struct Segment {
  int s0, s1, rows;
  bool whole, split, first;
};

// tma_load_4d to a shared-memory address.
__device__ __forceinline__ void tma_load_4d_at(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                               int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}

template <int RT>
__device__ __forceinline__ Segment segment_of(const PagedParams& p, const Cursor& c, int v, int v_end,
                                              bool first) {
  const int steps = unit_steps(p, c.s, c.t, RT);
  Segment g;
  g.s0 = v - c.u0;
  g.s1 = min(steps, v_end - c.u0);
  g.rows = min(RT, c.s.nq * p.G - c.t * RT);
  g.whole = g.s0 == 0 && g.s1 == steps;
  g.split = g.rows <= 128;
  g.first = first;
  return g;
}

// Calls f(cursor, segment) for the CTA's segments in order until it returns
// false.
template <int RT, class F>
__device__ __forceinline__ void for_each_segment(const PagedParams& p, Cursor c, int v,
                                                 int v_end, F&& f) {
  bool first = true;
  while (v < v_end) {
    const Segment g = segment_of<RT>(p, c, v, v_end, first);
    if (!f(c, g)) return;
    first = false;
    v = c.u0 + g.s1;
    if (v < v_end) advance(p, RT, c);
  }
}

// A softmax warp's place in the division, in shared memory: its registers
// hold a row of scores.
struct Place {
  Cursor c;
  int v, v_end;
};
static_assert(sizeof(Place) <= 64, "place");

// Four e4m3 codes as four fp16 values, in the arithmetic units: the code's
// exponent and mantissa bits moved to fp16's place are the value times 2^-8,
// subnormals too.  (The conversion instruction shares the unit of the base-2
// exponential, which the softmax fills.)  Codes of NaN come out as +-480.
__device__ __forceinline__ uint2 halves_of(uint32_t w) {
  const __half2 up = __float2half2_rn(256.0f);
  const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
  const uint32_t x = (a & 0x80008000u) | ((a >> 1) & 0x3f803f80u);
  const uint32_t y = (b & 0x80008000u) | ((b >> 1) & 0x3f803f80u);
  const __half2 hx = __hmul2(*reinterpret_cast<const __half2*>(&x), up);
  const __half2 hy = __hmul2(*reinterpret_cast<const __half2*>(&y), up);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&hx), *reinterpret_cast<const uint32_t*>(&hy));
}
// Bytes of w that are NaN codes (0x7f, 0xff): their top bits.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// +-480 back to NaN where code e of w was one.
__device__ __forceinline__ uint2 with_nan(uint2 h, uint32_t w) {
  const uint32_t n = nan_codes(w);
  if (n & 0x00000080u) h.x = (h.x & 0xffff0000u) | 0x7fffu;
  if (n & 0x00008000u) h.x = (h.x & 0x0000ffffu) | 0x7fff0000u;
  if (n & 0x00800000u) h.y = (h.y & 0xffff0000u) | 0x7fffu;
  if (n & 0x80000000u) h.y = (h.y & 0x0000ffffu) | 0x7fff0000u;
  return h;
}

// Converter warp w: its quarter of a value tile's 128 rows from codes to
// fp16 in the swizzled layout; rows from `valid` on become zeros.  Eight lanes
// take two rows at a time, so that both the 16-byte reads and the writes of
// each eight touch all banks.  TAIL: rows may be past `valid` and codes may be
// NaN; otherwise returns whether a NaN code was met (the tile is then done
// again with TAIL, so that the loop that always runs has no branch in it).
template <int D, bool TAIL>
__device__ __forceinline__ bool convert_rows(const uint8_t* raw, uint8_t* tile, int w, int lane, int valid) {
  constexpr int kUnits = D / 16;  // 16-byte units of a raw row
  constexpr int kChunkBytes = KT * 128;
  constexpr int kIters = KT / kConvertWarps * kUnits / 32, kBatch = 2;
  // lane's row and unit in iteration 0; in the odd ones (D = 128) the unit is
  // the other half's
  const int sub = lane & 7;
  const int row0 = w * (KT / kConvertWarps) + (lane >> 3) * 2 + (sub >> 2);
  const int unit0 = D == 128 ? sub : (sub & 3);
  uint32_t nan = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < kIters; i0 += kBatch) {
    // a batch's loads first: they may not pass the stores of the one before
    uint4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k, row = row0 + (D == 128 ? (i >> 1) : i) * 8;
      const int unit = D == 128 && (i & 1) ? unit0 ^ 4 : unit0;
      x[k] = *reinterpret_cast<const uint4*>(raw + row * D + unit * 16);
      if (TAIL && row >= valid) x[k] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k, row = row0 + (D == 128 ? (i >> 1) : i) * 8;
      const int unit = D == 128 && (i & 1) ? unit0 ^ 4 : unit0;
      uint2 h0 = halves_of(x[k].x), h1 = halves_of(x[k].y), h2 = halves_of(x[k].z), h3 = halves_of(x[k].w);
      if constexpr (TAIL) {
        h0 = with_nan(h0, x[k].x);
        h1 = with_nan(h1, x[k].y);
        h2 = with_nan(h2, x[k].z);
        h3 = with_nan(h3, x[k].w);
      } else {
        nan |= nan_codes(x[k].x) | nan_codes(x[k].y) | nan_codes(x[k].z) | nan_codes(x[k].w);
      }
      uint8_t* dst = tile + (unit >> 2) * kChunkBytes + row * 128;
      const int q = (unit & 3) * 2;
      *reinterpret_cast<uint4*>(dst + ((q ^ (row & 7)) << 4)) = make_uint4(h0.x, h0.y, h1.x, h1.y);
      *reinterpret_cast<uint4*>(dst + (((q + 1) ^ (row & 7)) << 4)) = make_uint4(h2.x, h2.y, h3.x, h3.y);
    }
  }
  return nan != 0;
}
template <int D>
__device__ __forceinline__ void convert_tile(const uint8_t* raw, uint8_t* tile, int w, int lane, int valid) {
  if (valid >= KT && !__any_sync(0xffffffffu, convert_rows<D, false>(raw, tile, w, lane, valid))) return;
  convert_rows<D, true>(raw, tile, w, lane, valid);
}

// A row's 128 scores (raw, in s; -inf: removed) to weights: 2^(f s - m), and
// with groups of 16 keys that have scales of their own 2^(f ks s + log2 vs -
// m).  f >= 0.  Returns the factor that the earlier sums have to take (need:
// it is not 1).
// With N = 64 a row's other half is the partner thread's (lane ^ 16): both take
// the same maximum, and l is this half's sum.
template <bool E4M3, bool MBF, int N>
__device__ __forceinline__ float weights(float (&s)[N], float f, const float4* note, float& m, float& l,
                                         bool& need, uint32_t (&pk)[N / 2]) {
  float top = -INFINITY;
  // never zero: a removed score, an infinity, has to stay one
  auto mul = [&](int g) { return fmaxf(f * note[g].x, 1.17549435e-38f); };
  if constexpr (E4M3) {
#pragma unroll
    for (int g = 0; g < N / 16; ++g) {
      const float* x = s + g * 16;
      const float a = max3f(x[0], x[1], x[2]), b = max3f(x[3], x[4], x[5]), c = max3f(x[6], x[7], x[8]);
      const float d = max3f(x[9], x[10], x[11]), e = max3f(x[12], x[13], x[14]);
      top = fmaxf(top, fmaf(fmaxf(max3f(a, b, c), max3f(d, e, x[15])), mul(g), note[g].y));
    }
  } else {
    float e8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e8[i] = s[i];
#pragma unroll
    for (int c = 8; c < N; c += 16)
#pragma unroll
      for (int i = 0; i < 8; ++i) e8[i] = max3f(e8[i], s[c + i], s[c + 8 + i < N ? c + 8 + i : c + i]);
    e8[0] = fmaxf(max3f(e8[0], e8[1], e8[2]), max3f(e8[3], e8[4], e8[5]));
    top = max3f(e8[0], e8[6], e8[7]) * f;
  }
  if constexpr (N < KT) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
  need = top > m + WeightRange<MBF>::kRoom;
  float alpha = 1.0f;
  if (need) {
    const float base = top - WeightRange<MBF>::kTop;
    alpha = ex2(m - base);
    m = base;
    l *= alpha;
  }
  const float neg_m = m == -INFINITY ? 0.0f : -m;
  if constexpr (E4M3) {
#pragma unroll
    for (int g = 0; g < N / 16; ++g) {
      const float a = mul(g), b = note[g].y + neg_m;
#pragma unroll
      for (int c = 16 * g; c < 16 * g + 16; c += 2) fma2_bcast(s[c], s[c + 1], s[c], s[c + 1], a, b);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 2) fma2_bcast(s[c], s[c + 1], s[c], s[c + 1], f, neg_m);
  }
#pragma unroll
  for (int c = 0; c < N; ++c) s[c] = ex2(s[c]);
  if constexpr (E4M3) {
#pragma unroll
    for (int g = 0; g < N / 16; ++g) {
      float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int e = 16 * g + 2 * c;
        add2_acc(r[2 * (c & 1)], r[2 * (c & 1) + 1], s[e], s[e + 1]);
        pk[e / 2] = pack2<MBF>(s[e], s[e + 1]);
      }
      add2_acc(r[0], r[1], r[2], r[3]);
      l = fmaf(r[0] + r[1], note[g].z, l);
    }
  } else {
    float rs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rs[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
      add2_acc(rs[2 * (c & 3)], rs[2 * (c & 3) + 1], s[2 * c], s[2 * c + 1]);
      pk[c] = pack2<MBF>(s[2 * c], s[2 * c + 1]);
    }
    add2_acc(rs[0], rs[1], rs[2], rs[3]);
    add2_acc(rs[4], rs[5], rs[6], rs[7]);
    add2_acc(rs[0], rs[1], rs[4], rs[5]);
    l += rs[0] + rs[1];
  }
  return alpha;
}

// Where 16-byte piece c of row r of a tile of ROW_BYTES-wide rows lies: the
// 128-byte swizzle, or the 64-byte one.
template <int ROW_BYTES>
__device__ __forceinline__ int swizzled(int r, int c) {
  return ROW_BYTES == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4);
}

// Two codes' values (a conversion instruction: not for the inner loops).
template <__nv_fp8_interpretation_t TYPE>
__device__ __forceinline__ float2 codes_value2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), TYPE);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// v to codes of one term, and what they leave.
template <__nv_fp8_interpretation_t TYPE, bool LAST>
__device__ __forceinline__ uint32_t take_term(float (&v)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, TYPE);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, TYPE);
  if constexpr (!LAST) {
    const float2 g0 = codes_value2<TYPE>(lo), g1 = codes_value2<TYPE>(hi);
    v[0] -= g0.x, v[1] -= g0.y, v[2] -= g1.x, v[3] -= g1.y;
  }
  return lo | (hi << 16);
}

// Where 16-byte piece i of row r of a query tile waits as it lies in memory.
// 16-bit: its own place.  8-bit terms: pieces 2u and 2u + 1 become piece u of
// every term, and wait in that piece's places of the first two.
template <int D, bool E4M3, int QCHUNK>
__device__ __forceinline__ int query_piece(int r, int i) {
  if constexpr (!E4M3) return (i >> 3) * QCHUNK + swizzled<128>(r, i & 7);
  return (i & 1) * QCHUNK + swizzled<D>(r, i >> 1);
}
// Asks for the row's pieces [i0, i1); finished by cp_async_wait<0>().
template <int D, bool E4M3, int N, int QCHUNK>
__device__ __forceinline__ void ask_query(const uint16_t* src, uint8_t* tile, int r, int i0) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    cp_async_16(tile + query_piece<D, E4M3, QCHUNK>(r, i0 + k), src + (i0 + k) * 8);
  cp_async_commit();
}

// N pieces of the row from i0 on (not live: zeros) to the tile as the products
// read it, negated for a negative scale; returns the (positive) multiplier of
// the scores, |scale| * log2(e).  For e4m3 keys the row is brought by a power of
// two to a largest element in [2^7, 2^8) (the factor goes into the multiplier)
// and split into terms, each what the earlier ones leave.  Where the first term
// is a normal e4m3 (from 2^-6, 2^-13 of the row's largest element) all of a bf16
// value is in two, of an fp16 one in three: the first leaves a multiple of the
// value's last place, at most 8 of them (fp16: 64, of which the next leaves at
// most 4), and an e5m2 holds any of these, its least step being 2^-16.  Below,
// the first leaves up to 2^-10, and the last is off by half a step of e5m2: 2^-14
// (fp16: 2^-17), 2^-21 (2^-24) of the row's largest.  HALF: a row is two threads' (lane ^ 16).  The whole
// warp calls it.  (Rolled loops over pieces that are rewritten in place: with
// the row in registers this was 16 to 24 KB of code between the softmax's loops;
// uneven prompts with e4m3 pages 660 -> 625 us.)
template <int D, bool E4M3, bool BF16, bool HALF, int N, int QCHUNK>
__device__ __forceinline__ float put_query(const PagedParams& p, bool live, uint8_t* tile, int r, int i0) {
  const float f = fabsf(p.scale_log2);
  const uint32_t sign = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
  auto at = [&](int i) { return reinterpret_cast<uint4*>(tile + query_piece<D, E4M3, QCHUNK>(r, i)); };
  if constexpr (!E4M3) {
    if (live && sign == 0u) return f;
#pragma unroll 1
    for (int i = i0; i < i0 + N; ++i) {
      const uint4 w = *at(i);
      *at(i) = live ? make_uint4(w.x ^ sign, w.y ^ sign, w.z ^ sign, w.w ^ sign) : make_uint4(0u, 0u, 0u, 0u);
    }
    return f;
  } else {
    const uint32_t keep = live ? 0xffffffffu : 0u;
    float top = 0.0f;
#pragma unroll 2
    for (int i = i0; i < i0 + N; ++i) {
      const uint4 w = *at(i);
      const uint32_t x[4] = {w.x & keep, w.y & keep, w.z & keep, w.w & keep};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = unpack2<BF16>(x[k]);
        top = max3f(top, fabsf(a.x), fabsf(a.y));
      }
    }
    if (HALF) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -110);
    // (an infinite element makes the row NaN)
    float up = top < INFINITY ? __int_as_float((127 + 7 - e) << 23) : NAN;
    if (sign != 0u) up = -up;
#pragma unroll 1
    for (int i = i0; i < i0 + N; i += 2) {
      const uint4 w0 = *at(i), w1 = *at(i + 1);
      const uint32_t x[8] = {w0.x & keep, w0.y & keep, w0.z & keep, w0.w & keep,
                             w1.x & keep, w1.y & keep, w1.z & keep, w1.w & keep};
      uint32_t term[3][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = unpack2<BF16>(x[2 * k]), b = unpack2<BF16>(x[2 * k + 1]);
        float v[4] = {a.x * up, a.y * up, b.x * up, b.y * up};
        term[0][k] = take_term<__NV_E4M3, false>(v);
        if constexpr (q_terms(E4M3, BF16) == 3) term[1][k] = take_term<__NV_E5M2, false>(v);
        term[q_terms(E4M3, BF16) - 1][k] = take_term<__NV_E5M2, true>(v);
      }
#pragma unroll
      for (int n = 0; n < q_terms(E4M3, BF16); ++n)
        *reinterpret_cast<uint4*>(tile + n * QCHUNK + swizzled<D>(r, i >> 1)) =
            make_uint4(term[n][0], term[n][1], term[n][2], term[n][3]);
    }
    return f * __int_as_float((127 - 7 + e) << 23);
  }
}

// 32 bytes, on a 32-byte boundary.  (A thread stores its own row, so that a warp's
// store touches 32 sectors: halves of them, 16 bytes at a time, took 0.9 us more
// of a unit of 256 rows; turning four rows between lanes first won no more.)
__device__ __forceinline__ void store_sector(void* to, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A thread's part of 32 (HALF: two times 32, SPLIT columns apart) accumulator
// columns.
template <bool HALF, int SPLIT>
__device__ __forceinline__ void acc_load(uint32_t at, uint32_t* r) {
  if constexpr (HALF)
    tmem_ld16x2_32<SPLIT>(at, r);
  else
    tmem_ld32(at, r);
}
template <bool HALF, int SPLIT>
__device__ __forceinline__ void acc_store(uint32_t at, const uint32_t* r) {
  if constexpr (HALF)
    tmem_st16x2_32<SPLIT>(at, r);
  else
    tmem_st32(at, r);
}

// Two consecutive K-steps (32 codes each) of D[tmem] (+)= A[smem] * B[smem]^T
// with 8-bit operands (each of a type of its own), in one elected issue; see
// mma_ss_x4.
template <uint32_t HI>
__device__ __forceinline__ void mma_codes_x2(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                             uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e, q;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, %4, %4;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t"
      "add.u32 a, %1, 2;\n\t"
      "add.u32 b, %2, 2;\n\t"
      "mov.b64 da, {a, %5};\n\t"
      "mov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, q;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(HI)
      : "memory");
}

template <int D, bool E4M3, bool BF16, bool HALF>
__global__ void __launch_bounds__(Split<E4M3>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
  using L = Lay<D, E4M3, BF16, HALF>;
  constexpr bool MBF = BF16 && !E4M3;
  constexpr int RT = unit_rows(HALF);
  constexpr int kPer = HALF ? KT / 2 : KT;   // a step's keys a softmax thread takes
  constexpr int kQPieces = D / 8 / (HALF ? 2 : 1);   // 16-byte pieces of the queries
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem + L::kQ;
  uint8_t* sK = smem + L::kK;
  uint8_t* sV = smem + L::kV;
  float4* notes = reinterpret_cast<float4*>(smem + L::kNote);
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBar);
  static_assert(sizeof(Bars) <= 512, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 4);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_ready[t], 4);
      mbar_init(&bars->o_done[t], 1);
    }
    mbar_init(&bars->sums, 8);
    mbar_init(&bars->read, 8);
    mbar_init(&bars->fin, 1);
    for (int i = 0; i < L::kKStages; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < L::kVStages; ++i) {
      mbar_init(&bars->v_full[i], E4M3 ? kConvertWarps : 1);
      mbar_init(&bars->v_empty[i], 1);
    }
    for (int i = 0; i < L::kRawStages; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], kConvertWarps);
    }
    for (int i = 0; i < L::kNotes; ++i) mbar_init(&bars->note[i], 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  const uint32_t tmem = bars->tmem_base;

  // the division, in the scratch of the Q tiles
  const int cta = static_cast<int>(blockIdx.x);
  int total;
  Cursor c0{};
  const int v0 = divide<Split<E4M3>::kThreads>(
      p, RT, reinterpret_cast<DivideScratch*>(sQ),
      [&](int all) {
        const int n = range_count(p, all);
        return cta < n ? range_start(all, cta, n) : all;
      },
      total, c0);
  const int n_ranges = range_count(p, total);
  const int v1 = v0 < 0 ? v0 : range_start(total, cta + 1, n_ranges);
  // nothing to join, until the last segment says otherwise: a CTA that stops
  // early leaves no note that the join would follow out of the workspace
  if (threadIdx.x == 0) reinterpret_cast<JoinNote*>(p.part)[cta].pieces = 0;
  __syncthreads();

  if (warp >= 4 && warp < 12) {
    // -------------------------------------------------------- softmax
    regs_increase<Split<E4M3>::kSoftmax>();
    const int t = (warp - 4) >> 2, wq = warp & 3;
    // row of the tile, and which half of it
    const int half = HALF ? lane >> 4 : 0;
    const int r = HALF ? wq * 16 + (lane & 15) : wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + (t ? 128u : 0u) + lane_off;
    const uint32_t tO = tmem + (t ? 384u : 256u) + lane_off;
    uint32_t n_s = 0, n_sums = 0;   // completions consumed
    RingAt<L::kNotes> note_at;
    volatile Place* vplace = reinterpret_cast<volatile Place*>(smem + L::kCursors) + (warp - 4);
    auto save = [&](const Cursor& c, int v) {
      if (lane == 0) {
        vplace->c.b = c.b, vplace->c.h = c.h, vplace->c.t = c.t, vplace->c.u0 = c.u0;
        vplace->c.s.q0 = c.s.q0, vplace->c.s.nq = c.s.nq, vplace->c.s.len = c.s.len, vplace->c.s.nt = c.s.nt;
        vplace->v = v, vplace->v_end = v1;
      }
      __syncwarp();
    };
    auto load = [&](Cursor& c, int& v, int& v_end) {
      c.b = vplace->c.b, c.h = vplace->c.h, c.t = vplace->c.t, c.u0 = vplace->c.u0;
      c.s.q0 = vplace->c.s.q0, c.s.nq = vplace->c.s.nq, c.s.len = vplace->c.s.len, c.s.nt = vplace->c.s.nt;
      v = vplace->v, v_end = vplace->v_end;
    };
    // the row's token and query head
    auto place = [&](const Cursor& c, int ru, int64_t& token, int64_t& head) {
      const int rr = c.t * RT + ru, tok = by_G(p, rr);
      token = static_cast<int64_t>(c.s.q0) + tok;
      head = static_cast<int64_t>(c.h) * p.G + (rr - tok * p.G);
      return tok;
    };
    // the row of a segment's unit, and its query
    auto row_of = [&](const Segment& g) { return HALF || g.split ? r : t * 128 + r; };
    auto ask = [&](const Cursor& c, const Segment& g) {
      int64_t token, head;
      const int ru = row_of(g);
      place(c, ru, token, head);
      if (ru < g.rows)
        ask_query<D, E4M3, kQPieces, L::kQChunk>(reinterpret_cast<const uint16_t*>(p.q) + token * p.q_st + head * p.q_sh,
                                             sQ + t * L::kQTile, r, half * kQPieces);
    };
    save(c0, v0);
    bool first = true;
    if (v0 < v1) ask(c0, segment_of<RT>(p, c0, v0, v1, true));
    for (bool ok = v0 < v1; ok;) {
      float f = 0.0f;
      int seen, s0, s1;
      bool split, idle;
      {
        Cursor c;
        int v, v_end;
        load(c, v, v_end);
        const Segment g = segment_of<RT>(p, c, v, v_end, first);
        s0 = g.s0, s1 = g.s1, split = HALF || g.split;
        const int ru = row_of(g);
        int64_t token, head;
        const int tok = place(c, ru, token, head);
        // rows that the unit has not: nothing of theirs is removed (a removed
        // key costs the whole warp), and a warp of them alone only keeps step
        idle = ru - (HALF ? lane & 15 : lane) >= g.rows;
        seen = ru >= g.rows ? 0x7fffffff : p.is_causal ? min(max(c.s.len - c.s.nq + tok + 1, 0), c.s.len) : c.s.len;
        cp_async_wait<0>();
        if (!idle) {
          __syncwarp();
          f = put_query<D, E4M3, BF16, HALF, kQPieces, L::kQChunk>(p, ru < g.rows, sQ + t * L::kQTile, r, half * kQPieces);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_full[t]);
      float m = -INFINITY, l = 0.0f;
      int mine = 0;
      for (int s = s0; s < s1; ++s) {
        const int slot = note_at.idx;
        const uint32_t note_phase = note_at.phase;
        note_at.next();
        if (split && ((s - s0) & 1) != t) continue;
        if (!warp_wait(&bars->note[slot], note_phase, bars, limit, kSiteNote)) {
          ok = false;
          break;
        }
        const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&bars->bad[slot]);
        if (!warp_wait(&bars->s_full[t], n_s & 1, bars, limit, kSiteS)) {
          ok = false;
          break;
        }
        ++n_s;
        if (idle) {
          // (its rows of P are whatever is there: their products are not read)
          if (lane == 0) mbar_arrive(&bars->p_ready[t]);
          ++mine;
          continue;
        }
        tc_fence_after();
        float x[kPer];
        {
          uint32_t u[kPer];
#pragma unroll
          for (int i = 0; i < kPer / 32; ++i) acc_load<HALF, KT / 2>(tS + i * 32, u + i * 32);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] = __uint_as_float(u[i]);
        }
        const int left = seen - s * KT;   // keys of this tile that the row sees
        if (__any_sync(0xffffffffu, left < KT) || bad != 0u) {
          const int mine_left = left - half * kPer;
          const uint32_t mine_bad = bad >> (half * (kPer / 16));
          uint32_t keep[kPer / 32];
#pragma unroll
          for (int i = 0; i < kPer / 32; ++i) {
            const int n = min(max(mine_left - 32 * i, 0), 32);
            keep[i] = n == 32 ? 0xffffffffu : (1u << n) - 1u;
            if ((mine_bad >> (2 * i)) & 1u) keep[i] &= 0xffff0000u;
            if ((mine_bad >> (2 * i)) & 2u) keep[i] &= 0x0000ffffu;
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] = ((keep[i >> 5] >> (i & 31)) & 1u) ? x[i] : -INFINITY;
        }
        bool need;
        uint32_t pk[kPer / 2];
        const float alpha = weights<E4M3, MBF, kPer>(x, f, notes + slot * kGroups + half * (kPer / 16), m, l, need, pk);
        if (mine > 0 && __any_sync(0xffffffffu, need)) {
          // the earlier products of this tile are complete: S of this step was
          // issued behind them (rolled, as whatever seldom runs)
#pragma unroll 1
          for (int i = 0; i < D / (HALF ? 64 : 32); ++i) {
            uint32_t o[32];
            acc_load<HALF, D / 2>(tO + i * 32, o);
            tmem_ld_wait();
            float* of = reinterpret_cast<float*>(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) mul2_bcast(of[e], of[e + 1], alpha);
            acc_store<HALF, D / 2>(tO + i * 32, o);
          }
        }
#pragma unroll
        for (int i = 0; i < kPer / 64; ++i) acc_store<HALF, KT / 4>(tS + i * 32, pk + i * 32);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_ready[t]);
        ++mine;
      }
      if (!ok) break;
      Cursor c;
      int v, v_end;
      load(c, v, v_end);
      const Segment g = segment_of<RT>(p, c, v, v_end, first);
      Cursor next = c;
      const int v_next = c.u0 + g.s1;
      if (v_next < v_end) {
        advance(p, RT, next);
        // its query, while this one's rows are written (S of this tile is complete)
        ask(next, segment_of<RT>(p, next, v_next, v_end, false));
      }
      // n_s completions of s_full[t] so far, as many of o_done[t]
      if (mine > 0 && !warp_wait(&bars->o_done[t], (n_s - 1) & 1, bars, limit, kSiteO)) break;
      tc_fence_after();
      float fa = 1.0f, fb = 0.0f;
      if (HALF) l += __shfl_xor_sync(0xffffffffu, l, 16);   // the row's sum
      if (split) {
        // join the two warpgroups' sums: each leaves (m, l) behind its P and
        // writes half of the columns
        uint32_t ml[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) ml[i] = 0u;
        ml[0] = __float_as_uint(m);
        ml[1] = __float_as_uint(l);
        // (HALF: a copy for each of a row's threads)
        acc_store<HALF, 32>(tS + (HALF ? 64 : 96), ml);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->sums);
        if (!warp_wait(&bars->sums, n_sums & 1, bars, limit, kSiteSums)) {
          ok = false;
          break;
        }
        ++n_sums;
        tc_fence_after();
        acc_load<HALF, 32>(tmem + (t ? 0u : 128u) + lane_off + (HALF ? 64 : 96), ml);
        tmem_ld_wait();
        const float mo = __uint_as_float(ml[0]), lo = __uint_as_float(ml[1]);
        const float mx = fmaxf(m, mo), base = mx == -INFINITY ? 0.0f : mx;
        fa = ex2(m - base);
        fb = ex2(mo - base);
        l = l * fa + lo * fb;
        m = mx;
      }
      const int ru = row_of(g);
      const bool live = ru < g.rows;
      int64_t token, head;
      place(c, ru, token, head);
      // O is undefined where no step was taken; otherwise (no key seen) zeros
      const bool own = mine > 0, other = split && (t == 0 ? g.s1 - g.s0 > 1 : true);
      const float inv = !g.whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      fa *= inv;
      fb *= inv;
      uint16_t* orow = reinterpret_cast<uint16_t*>(p.out) + token * p.o_st + head * p.o_sh;
      float* prow = part_rows<D>(p, blockIdx.x, g.first ? 0 : 1, RT) + static_cast<int64_t>(ru) * (D + 2);
      // this thread's runs of 32 columns: all, or half of them (HALF: of its
      // half row's; where that is one run, the first warpgroup's)
      constexpr int kRuns = HALF ? D / 64 : D / 32;
      const int i0 = split ? t * (kRuns / 2) : 0;
      const int i1 = !split ? kRuns : kRuns == 1 ? 1 - t : i0 + kRuns / 2;
      const int col0 = half * (D / 2);
#pragma unroll 1
      for (int i = i0; i < i1 && !idle; ++i) {
        uint32_t o[32];
        acc_load<HALF, D / 2>(tO + i * 32, o);
        tmem_ld_wait();
        float* of = reinterpret_cast<float*>(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) of[e] = own ? of[e] * fa : 0.0f;
        if (other) {
          uint32_t o2[32];
          acc_load<HALF, D / 2>(tmem + (t ? 256u : 384u) + lane_off + i * 32, o2);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) of[e] = fmaf(__uint_as_float(o2[e]), fb, of[e]);
        }
        if (live) {
          if (g.whole) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2<BF16>(of[2 * e], of[2 * e + 1]);
            uint16_t* to = orow + col0 + i * 32;
            if (p.out_sectors) {
              store_sector(to, w);
              store_sector(to + 16, w + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(to + e * 8) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              *reinterpret_cast<float2*>(prow + col0 + i * 32 + e) = make_float2(of[e], of[e + 1]);
          }
        }
      }
      if (split) {
        // this warpgroup's sums stay until the other has read them
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->read);
        if (!warp_wait(&bars->read, (n_sums - 1) & 1, bars, limit, kSiteSums)) break;
      }
      if (live && half == 0 && (!split || t == 0)) {
        if (!g.whole) {
          *reinterpret_cast<float2*>(prow + D) = make_float2(m, l);
        } else if (p.lse != nullptr) {
          constexpr float kLn2 = 0.693147180559945309f;
          p.lse[token * p.lse_st + head * p.lse_sh] = l == 0.0f ? -INFINITY : (log2f(l) + m) * kLn2;
        }
      }
      tc_fence_before();
      if (v_next >= v_end) {
        grid_launch_dependents();
        if (t == 0 && r == 0) leave_note(p, blockIdx.x, total, n_ranges, RT, c, g.s0, g.s1, first);
        break;
      }
      first = false;
      __syncwarp();
      save(next, v_next);
    }
    cp_async_wait<0>();
    tc_fence_before();
  } else {
    regs_decrease<Split<E4M3>::kControl>();
    const int P = 1 << p.page_shift;
    // A window of 32 of a sequence's page entries in the lanes, the next one
    // behind it; an entry that is no page becomes n_pages, out of the maps'
    // bounds.
    struct Window {
      const int* row;
      int n, at, ids, next;
    };
    auto entries = [&](const Window& w, int from) {
      const int id = from + lane < w.n ? __ldg(w.row + from + lane) : -1;
      return id >= 0 && id < p.n_pages ? id : p.n_pages;
    };
    auto open_window = [&](const Cursor& c, int s) {
      Window w;
      w.row = p.table + static_cast<int64_t>(c.b) * p.table_st;
      w.n = (c.s.len + P - 1) >> p.page_shift;
      w.at = (s * KT) >> p.page_shift;
      w.ids = entries(w, w.at);
      w.next = entries(w, w.at + 32);
      return w;
    };
    // (a step's entries lie in one window: their number divides 32)
    auto reach = [&](Window& w, int s) {
      const int e = (s * KT) >> p.page_shift;
      if (e - w.at >= 32) {
        w.at += 32;
        w.ids = w.next;
        w.next = entries(w, w.at + 32);
      }
      return e;
    };
    if (warp == 0 || warp == 2) {
      // ----------------------------------------------------------- loads
      constexpr int kVRing = E4M3 ? L::kRawStages : L::kVStages;
      const bool is_k = warp == 0;
      const int ring = is_k ? L::kKStages : kVRing;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      uint64_t* const full0 = is_k ? bars->k_full : E4M3 ? bars->raw_full : bars->v_full;
      uint64_t* const empty0 = is_k ? bars->k_empty : E4M3 ? bars->raw_empty : bars->v_empty;
      const uint32_t dst0 = smem_addr(is_k ? sK : E4M3 ? smem + L::kRaw : sV);
      const int box = P < KT ? P : KT, per_step = KT / box;
      int at = 0, issued = 0;   // ring slot, tiles issued
      uint32_t phase = 0;
      bool lapped = false;
      RingAt<L::kNotes> note_at;
      for_each_segment<RT>(p, c0, v0, v1, [&](const Cursor& c, const Segment& g) -> bool {
        Window w = open_window(c, g.s0);
        // keys' warp: lane i < 8 looks after keys 16 i .. of a step; its page's
        // scales are asked for a step ahead (the entry may lie in the window
        // behind)
        int id = 0;
        float ks = 1.0f, vs = 1.0f;
        auto ask = [&](int s) {
          const int e = ((s * KT + (lane & 7) * 16) >> p.page_shift) - w.at;
          const int a = __shfl_sync(0xffffffffu, w.ids, e & 31), b = __shfl_sync(0xffffffffu, w.next, e & 31);
          id = e < 32 ? a : b;
          if (E4M3 && lane < 8 && id < p.n_pages) {
            const int64_t at = static_cast<int64_t>(id) * p.n_kv + c.h;
            ks = __ldg(p.k_scale + at);
            vs = __ldg(p.v_scale + at);
          }
        };
        if (is_k) ask(g.s0);
        for (int s = g.s0; s < g.s1; ++s) {
          const int e0 = reach(w, s), row0 = (s * KT) & (P - 1);
          if (lapped && !warp_wait(empty0 + at, phase ^ 1u, bars, limit, kSiteEmpty)) return false;
          uint64_t* full = full0 + at;
          const uint32_t dst = dst0 + static_cast<uint32_t>(at) * (E4M3 ? L::kCodes : L::kTile);
          // one elected lane issues the tile's boxes
          const bool leader = elect_one();
          if (leader) {
            if (E4M3 && !is_k) *reinterpret_cast<volatile int*>(&bars->valid[at]) = c.s.len - s * KT;
            mbar_arrive_expect_tx(full, E4M3 ? L::kCodes : L::kTile);
          }
#pragma unroll 2
          for (int i = 0; i < per_step; ++i) {
            const int id = __shfl_sync(0xffffffffu, w.ids, e0 - w.at + i);
            if (leader) {
              if constexpr (E4M3) {
                tma_load_4d_at(dst + i * box * D, map, full, 0, row0, c.h, id);
              } else {
#pragma unroll
                for (int ch = 0; ch < L::kChunks; ++ch)
                  tma_load_4d_at(dst + ch * L::kChunkBytes + i * box * 128, map, full, ch * 64, row0, c.h, id);
              }
            }
          }
          __syncwarp();
          if (is_k) {
            const uint32_t bad = __ballot_sync(0xffffffffu, id >= p.n_pages) & 0xffu;
            if (E4M3 && lane < 8) {
              vs = clamp_scale(vs);
              notes[note_at.idx * kGroups + lane] = make_float4(clamp_scale(ks), __log2f(vs), __fdividef(1.0f, vs), 0.0f);
            }
            if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&bars->bad[note_at.idx]) = bad;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->note[note_at.idx]);
            note_at.next();
            if (s + 1 < g.s1) ask(s + 1);
          }
          ++issued;
          if (++at == ring) {
            at = 0;
            phase ^= 1u;
            lapped = true;
          }
        }
        return true;
      });
      // what was issued must land before shared memory is released
      for (int j = max(0, issued - ring); j < issued; ++j)
        wait_any(full0 + j % ring, (j / ring) & 1, bars, limit, kSiteDrain, false);
    } else if (warp == 1) {
      // -------------------------------------------------------- products
      constexpr uint32_t kM = tile_rows(HALF);
      constexpr uint32_t idS = idesc_f16_f32acc(MBF, false, kM, KT);
      constexpr uint32_t idPV = idesc_f16_f32acc(MBF, true, kM, D);
      constexpr uint32_t kHi = desc_hi_sw128(1024);
      // e4m3 operands (type 0 in the descriptor's fields, D = fp32), rows of D
      // bytes: the 128-byte swizzle, or the 64-byte one (mode 4)
      constexpr uint32_t idCodes = (1u << 4) | ((KT >> 3) << 17) | ((kM >> 4) << 24);
      constexpr uint32_t kQueryE5m2 = 1u << 7;   // the later terms' type
      constexpr uint32_t kHiCodes = D == 128 ? kHi : ((512u >> 4) | (1u << 14) | (4u << 29));
      const uint32_t q_lo = desc_lo_sw128(smem_addr(sQ), 16);
      const uint32_t k_lo = desc_lo_sw128(smem_addr(sK), 16);
      const uint32_t v_lo = desc_lo_sw128(smem_addr(sV), L::kChunkBytes);
      RingAt<L::kKStages> k_at;
      RingAt<L::kVStages> v_at;
      uint32_t p_phase = 0, n_seg = 0;   // p_phase: a bit a warpgroup
      bool issued = false;
      auto issue_s = [&](int t) {
        const uint32_t a0 = q_lo + static_cast<uint32_t>(t * (L::kQTile >> 4));
        const uint32_t b0 = k_lo + static_cast<uint32_t>(k_at.idx * (L::kKTile >> 4));
        if constexpr (E4M3) {
#pragma unroll
          for (int n = 0; n < q_terms(E4M3, BF16); ++n)
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
              mma_codes_x2<kHiCodes>(tmem + (t ? 128u : 0u), a0 + n * (L::kQChunk >> 4) + 4 * k, b0 + 4 * k,
                                     n > 0 ? idCodes | kQueryE5m2 : idCodes, n + k > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int ch = 0; ch < L::kChunks; ++ch) {
            const uint32_t off = static_cast<uint32_t>(ch * L::kChunkBytes) >> 4;
            mma_ss_x4<kHi, kHi>(tmem + (t ? 128u : 0u), a0 + ((ch * L::kQChunk) >> 4), b0 + off, 2u, 2u, idS, ch > 0 ? 1u : 0u);
          }
        }
        mma_commit_elect(&bars->s_full[t]);
      };
      auto issue_pv = [&](int t, bool more) {
        const uint32_t b0 = v_lo + static_cast<uint32_t>(v_at.idx * (L::kTile >> 4));
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          mma_ts_x4<kHi>(tmem + (t ? 384u : 256u), tmem + (t ? 128u : 0u) + hf * 32,
                         b0 + hf * ((64 * 128) >> 4), 8u, (16 * 128) >> 4, idPV, (more || hf > 0) ? 1u : 0u);
        mma_commit_elect(&bars->o_done[t]);
      };
      auto next_k = [&]() {
        if (!warp_wait(&bars->k_full[k_at.idx], k_at.phase, bars, limit, kSiteK)) return false;
        tc_fence_after();
        return true;
      };
      auto done_k = [&]() {
        mma_commit_elect(&bars->k_empty[k_at.idx]);
        k_at.next();
      };
      // V of the step: rows past the sequence's end are made zeros (their
      // weights are, but a stale NaN must not meet them)
      auto next_v = [&](int valid) {
        if (!warp_wait(&bars->v_full[v_at.idx], v_at.phase, bars, limit, kSiteV)) return false;
        if (!E4M3 && valid < KT) {
          uint8_t* tile = sV + v_at.idx * L::kTile;
#pragma unroll 1
          for (int i = max(valid, 0) * 8 + lane; i < KT * 8; i += 32)
#pragma unroll
            for (int ch = 0; ch < L::kChunks; ++ch)
              *reinterpret_cast<uint4*>(tile + ch * L::kChunkBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        return true;
      };
      auto next_p = [&](int t) {
        if (!warp_wait(&bars->p_ready[t], (p_phase >> t) & 1u, bars, limit, kSiteP)) return false;
        p_phase ^= 1u << t;
        tc_fence_after();
        return true;
      };
      for_each_segment<RT>(p, c0, v0, v1, [&](const Cursor& c, const Segment& g) -> bool {
        if (p.debug_withhold_q) return false;
        const int n = g.s1 - g.s0;
        issued = true;
        // One place each for the two products, whatever the mode (the code of
        // all roles together is what the instruction cache has to hold):
        // event e is warpgroup t = e & 1's product of its step j and S of its
        // next one, the first two only the latter.
        const int events = HALF || g.split ? n : 2 * n;
#pragma unroll 1
        for (int e = -2; e < events; ++e) {
          const bool split = HALF || g.split;
          const int t = e & 1, j = split ? e : e >> 1;
          const int ahead = j + (split ? 2 : 1);
          const bool head = split || t == 0, tail = split || t == 1;   // of the step's events
          if (e >= 0) {
            if (head && !next_v(c.s.len - (g.s0 + j) * KT)) return false;
            if (!next_p(t)) return false;
            issue_pv(t, j > (split ? 1 : 0));
            if (tail) {
              mma_commit_elect(&bars->v_empty[v_at.idx]);
              v_at.next();
            }
          }
          if (e < 0) {
            // each warpgroup's Q on its own: one may still be writing the last
            // unit's rows
            if (!warp_wait(&bars->q_full[t], n_seg & 1, bars, limit, kSiteQ)) return false;
            tc_fence_after();
          }
          if (ahead < n) {
            if (head && !next_k()) return false;
            issue_s(t);
            if (tail) done_k();
          }
        }
        ++n_seg;
        return true;
      });
      if (issued) {
        mma_commit_elect(&bars->fin);
        wait_any(&bars->fin, 0, bars, limit, kSiteDrain, false);
      }
    } else if (E4M3 && warp >= 12) {
      // ------------------------------------------------------ conversion
     if constexpr (E4M3) {
      RingAt<L::kVStages> v_at;
      RingAt<L::kRawStages> raw_at;
      // the CTA's steps, whatever units they belong to
      for (int left = v1 - v0; left > 0; --left) {
        if (!warp_wait(&bars->raw_full[raw_at.idx], raw_at.phase, bars, limit, kSiteK)) break;
        const int valid = *reinterpret_cast<volatile int*>(&bars->valid[raw_at.idx]);
        if (v_at.lapped && !warp_wait(&bars->v_empty[v_at.idx], v_at.phase ^ 1u, bars, limit, kSiteEmpty)) break;
        convert_tile<D>(smem + L::kRaw + raw_at.idx * L::kCodes, sV + v_at.idx * L::kTile, warp - 12, lane, valid);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->raw_empty[raw_at.idx]);
          mbar_arrive(&bars->v_full[v_at.idx]);
        }
        raw_at.next();
        v_at.next();
      }
     }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && bars->abort_flag != 0) atomicOr(&g_sdpa_paged_status, bars->abort_flag);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool E4M3, bool BF16, bool HALF>
cudaError_t launch_one(const PagedParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream) {
  auto kern = paged_tc_kernel<D, E4M3, BF16, HALF>;
  static std::atomic<uint64_t> configured{0};  // a bit a device
  const uint64_t bit = 1ull << p.device;
  cudaError_t e = cudaSuccess;
  if ((configured.load(std::memory_order_relaxed) & bit) == 0) {
    // the register split assumes kLaunch a thread at launch: never start a
    // build where that does not hold (setmaxnreg would wait)
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != static_cast<int>(Split<E4M3>::kLaunch)) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, E4M3, BF16, HALF>::kTotal);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_ctas));
  cfg.blockDim = dim3(Split<E4M3>::kThreads);
  cfg.dynamicSmemBytes = Lay<D, E4M3, BF16, HALF>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p, tm_k, tm_v);
  if (e != cudaSuccess) return e;
  return sdpa_impl::launch_paged_join(p, D, BF16, unit_rows(HALF), stream);
}

template <int D, bool HALF>
cudaError_t launch_dim(const PagedParams& p, bool bf16, bool e4m3, const CUtensorMap& k, const CUtensorMap& v,
                       cudaStream_t s) {
  if (e4m3) return bf16 ? launch_one<D, true, true, HALF>(p, k, v, s) : launch_one<D, true, false, HALF>(p, k, v, s);
  return bf16 ? launch_one<D, false, true, HALF>(p, k, v, s) : launch_one<D, false, false, HALF>(p, k, v, s);
}

}  // namespace

namespace sdpa_impl {

cudaError_t launch_paged_tc(const PagedParams& p, int head_dim, bool bf16, bool e4m3, int tile, const CUtensorMap& tm_k,
                            const CUtensorMap& tm_v, cudaStream_t stream) {
  if (tile == unit_rows(true))
    return head_dim == 64 ? launch_dim<64, true>(p, bf16, e4m3, tm_k, tm_v, stream)
                          : launch_dim<128, true>(p, bf16, e4m3, tm_k, tm_v, stream);
  return head_dim == 64 ? launch_dim<64, false>(p, bf16, e4m3, tm_k, tm_v, stream)
                        : launch_dim<128, false>(p, bf16, e4m3, tm_k, tm_v, stream);
}

cudaError_t read_and_clear_paged_status(unsigned int* status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_sdpa_paged_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  if (*status != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_sdpa_paged_status, &zero, sizeof(unsigned int));
  }
  return e;
}

}  // namespace sdpa_impl
