// sdpa_paged_sm103a.cu -- attention of a few new tokens a sequence over a
// paged key/value cache (16-bit, or e4m3 with a scale a page and head), for
// sm_103a.
//
// For the rows of one key/value head (a token's G query heads share it) and
// key j, s_j = scale * ks_j * (q . kcode_j) and out = sum_j p_j vs_j vcode_j /
// sum_j p_j.  One pass over the pages, online: with a = scale * log2(e), each
// key's weight is w_j = 2^(a ks_j q.kcode_j + log2 vs_j - m), m the running
// maximum of that exponent, so that the value's scale is inside the weight
// before it is rounded to 16 bits (w <= 2^15 whatever the scales are: m is the
// maximum less a constant, see WeightRange), and
//     out = sum_j w_j vcode_j / sum_j w_j / vs_j,
// the sums in fp32.  e4m3 codes are exact in fp16, so products of an 8-bit
// cache run in fp16 whatever the query's type: a bf16 query row is brought to
// fp16 by a power of two that takes its largest element to 2^14 .. 2^15 (exact
// for elements down to 2^-29 of it; the factor goes into the score's).
//
// Bound by memory while few rows share the keys: 2 D bytes (e4m3) a key and
// head against 4 G D operations.  Each of a CTA's four warps has a key/value
// head of its own (with fewer than four heads, a share of one's keys) and reads
// 16 keys of it a step (they lie in one page, whose entry and scales the warp
// needs once) into its own ring of stages with asynchronous 16-byte copies and
// multiplies from there: no block barrier, and no exchange between warps but
// for a shared head's sums at the end.  The next unit's first stages are asked
// for before this one's rows are written.  The tensor work is one 16 x 16
// tile a step (mma.sync; the rows of one head seldom fill it): a tcgen05 tile
// of 128 rows would be 7/8 padding here.  The order of D inside both products
// is free, so each thread takes 16 consecutive bytes of a key's row as they
// lie in memory, and the output's columns come out in runs of D / 4.
//
// With a window (WIN; a kernel of its own, since the loop is bound by its issue
// slots) a unit's steps are those that hold the sinks and those from its first
// row's window on; keys of these that a row does not see are removed as those
// behind its causal limit are.  64 sequences in a window of 4096 (H 32/8, D 128,
// e4m3): 102 us, 20 of which are the start, uneven ends and the join (2048 more
// keys of a window cost 40.6, 97% of the measured copy rate).
#include <atomic>

#include "sdpa_paged.cuh"

using namespace sdpa_dev;
using namespace sdpa_paged;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWarpKeys = 16;
constexpr int RT = 16;                 // rows a unit: one tile of the products

template <int D, bool E4M3>
struct Ring {
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kTile = kWarpKeys * kRowBytes;  // 16 keys of K or of V
  static constexpr int kStages = kTile == 1024 ? 6 : E4M3 ? 4 : 3;
  static constexpr int kWarpBytes = kStages * 2 * kTile;
};

// Where 16-byte piece c of row r of a 16-row tile lies, so that the reads of
// eight threads at a time touch all banks once (see load order in step()).
template <int ROW_BYTES, bool IS_V>
__device__ __forceinline__ int piece_at(int r, int c) {
  if constexpr (ROW_BYTES == 64) {
    const int half = (r ^ (r >> 2)) & 1, q = c ^ (r & 2);
    return (r >> 1) * 128 + half * 64 + q * 16;
  } else if constexpr (IS_V) {
    return r * ROW_BYTES + ((c ^ (r & 6)) << 4);
  } else {
    return r * ROW_BYTES + ((c ^ ((r & 1) << 2)) << 4);
  }
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes (low 16 bits of w) as two fp16 values.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t codes_to_half2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct WarpScratch {      // a warp's notes on its stages
  float k_scale[6], v_scale[6];
  int ok[6];              // 0: the stage's page is not one of the cache's
};

template <int D, bool E4M3>
struct Smem {
  using R = Ring<D, E4M3>;
  static constexpr int kJoinRow = D + 4;                        // floats
  static constexpr int kJoin = kWarps * RT * kJoinRow * 4;      // over the rings
  static constexpr int kRings = kWarps * R::kWarpBytes;
  static constexpr int kBulk = kRings > kJoin ? kRings : kJoin;
  static constexpr int kNotes = kBulk;
  static constexpr int kMl = kNotes + static_cast<int>(sizeof(WarpScratch)) * kWarps;
  static constexpr int kDivide = (kMl + kWarps * RT * 8 + 15) / 16 * 16;
  // Exactly kPerSm CTAs an SM: with room for more, the kernel's equal shares
  // would land on some SMs one more at a time and on others one fewer.
  static constexpr int kPerSm = sdpa_impl::paged_per_sm(D, E4M3);
  static constexpr int kNeed = kDivide + static_cast<int>(sizeof(DivideScratch));
  static constexpr int kLeast = 227 * 1024 / (kPerSm + 1);
  static constexpr int kTotal = kNeed > kLeast ? kNeed : kLeast;
  static_assert(kPerSm * (kTotal + 1024) <= 228 * 1024, "CTAs an SM");
};

// Row r of a sequence's rows for key/value head h: its place in out, and its
// log-sum-exp.
__device__ __forceinline__ uint16_t* out_row(const PagedParams& p, int q0, int h, int r) {
  const int i = by_G(p, r), g = r - i * p.G;
  return reinterpret_cast<uint16_t*>(p.out) + (static_cast<int64_t>(q0) + i) * p.o_st +
         (static_cast<int64_t>(h) * p.G + g) * p.o_sh;
}
__device__ __forceinline__ void store_lse(const PagedParams& p, int q0, int h, int r, float m, float l) {
  const int i = by_G(p, r), g = r - i * p.G;
  constexpr float kLn2 = 0.693147180559945309f;
  p.lse[(static_cast<int64_t>(q0) + i) * p.lse_st + (static_cast<int64_t>(h) * p.G + g) * p.lse_sh] =
      l == 0.0f ? -INFINITY : (log2f(l) + m) * kLn2;
}
template <int D, bool BF16>
__device__ __forceinline__ void store_out4(uint16_t* at, const float4& o, float inv) {
  *reinterpret_cast<uint2*>(at) = make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
}

template <int D, bool E4M3, bool BF16, bool WIN>
__global__ void __launch_bounds__(kThreads, sdpa_impl::paged_per_sm(D, E4M3))
    paged_kernel(const __grid_constant__ PagedParams p) {
  using S = Smem<D, E4M3>;
  using R = Ring<D, E4M3>;
  constexpr int NK = D / 16;              // k-steps of S
  constexpr int NV = D / 8;               // column groups of O
  constexpr int RB = R::kRowBytes;
  constexpr bool MBF = BF16 && !E4M3;     // type of the products
  using W = WeightRange<MBF>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  uint8_t* const ring = smem + warp * R::kWarpBytes;
  const uint32_t ring_addr = smem_addr(ring);
  WarpScratch* notes = reinterpret_cast<WarpScratch*>(smem + S::kNotes) + warp;
  float* ml = reinterpret_cast<float*>(smem + S::kMl);  // [warp][RT][2]
  DivideScratch* sc = reinterpret_cast<DivideScratch*>(smem + S::kDivide);

  grid_dependency_wait();

  const int cta = static_cast<int>(blockIdx.x);
  int total;
  Cursor c;
  int v = divide<kThreads, WIN>(
      p, RT, sc,
      [&](int all) {
        const int n = range_count(p, all);
        return cta < n ? range_start(all, cta, n) : all;
      },
      total, c);
  const int n_ranges = range_count(p, total);
  if (v < 0) {
    // more CTAs than steps
    if (threadIdx.x == 0) reinterpret_cast<JoinNote*>(p.part)[cta].pieces = 0;
    return;
  }
  const int v_end = range_start(total, cta + 1, n_ranges);
  // this warp's head of a unit's, and its share of the head's keys
  const int hsub = warp % p.unit_heads, slice = warp / p.unit_heads;
  const int slices = kWarps / p.unit_heads;
  const int page_mask = (1 << p.page_shift) - 1;

  // a lane's share of a 16-row tile: piece cc of rows r0, r0 + kRowsAtOnce, ..
  constexpr int kPieces = RB / 16;
  constexpr int kRowsAtOnce = 32 / kPieces;
  const int r0 = lane / kPieces, cc = lane % kPieces;
  const int64_t k_step = kRowsAtOnce * p.k_st, v_step = kRowsAtOnce * p.v_st;

  // The warp's loads: a segment's steps [s0, s1) of a unit's keys.
  struct Loads {
    const int* trow;
    const uint8_t *kh, *vh;
    int64_t scale_at;
    int s0, s1, keys, len;
    int skip, from;              // WIN: steps left out, first key of the rows' windows
    int ids_at, ids, ids_next;   // lane i: the page entry of step ids_at + i
  };
  auto key_of = [&](int skip, int s) { return (step_run<WIN>(p, skip, s) << p.step_shift) + slice * kWarpKeys; };
  // (16 keys that no row sees may lie in a page that is gone: they are taken for
  // keys without a page)
  auto load_ids = [&](const Loads& a, int s) {
    const int key0 = key_of(a.skip, s + lane);
    const bool seen = !WIN || key0 + kWarpKeys > a.from || key0 < p.sinks;
    return (s + lane < a.s1 && key0 < a.keys && seen) ? __ldg(a.trow + (key0 >> p.page_shift)) : -1;
  };
  auto issue = [&](Loads& a, int s, int stage) {
    if (s < a.s1) {
      if (s - a.ids_at == 32) {
        a.ids = a.ids_next;
        a.ids_at += 32;
        a.ids_next = load_ids(a, a.ids_at + 32);
      }
      const int page = __shfl_sync(0xffffffffu, a.ids, s - a.ids_at);
      const int key0 = key_of(a.skip, s);
      const bool ok = page >= 0 && page < p.n_pages;
      const int64_t pg = ok ? page : 0;
      const int tok = key0 & page_mask;
      if (key0 < a.keys) {
        const uint8_t* ks = a.kh + (pg * p.k_sp + tok * p.k_st);
        const uint8_t* vs = a.vh + (pg * p.v_sp + tok * p.v_st);
        const uint32_t dst = ring_addr + stage * 2 * R::kTile;
        if (ok && key0 + kWarpKeys <= a.len) {
#pragma unroll
          for (int i = 0; i < kWarpKeys / kRowsAtOnce; ++i) {
            cp_async_16_at(dst + piece_at<RB, false>(r0 + i * kRowsAtOnce, cc), ks);
            cp_async_16_at(dst + R::kTile + piece_at<RB, true>(r0 + i * kRowsAtOnce, cc), vs);
            ks += k_step;
            vs += v_step;
          }
        } else {
          // rows past the sequence's end, and a page that is none, read as
          // zeros: their weights are zero, and a stale NaN there must not
          // meet them
#pragma unroll
          for (int i = 0; i < kWarpKeys / kRowsAtOnce; ++i) {
            const int r = r0 + i * kRowsAtOnce;
            const bool in = ok && key0 + r < a.len;
            cp16(dst + piece_at<RB, false>(r, cc), ks, in);
            cp16(dst + R::kTile + piece_at<RB, true>(r, cc), vs, in);
            ks += k_step;
            vs += v_step;
          }
        }
        if (lane < 2) {
          if constexpr (E4M3) {
            const float* src = (lane == 0 ? p.k_scale : p.v_scale) + pg * p.n_kv + a.scale_at;
            cp4(smem_addr(lane == 0 ? &notes->k_scale[stage] : &notes->v_scale[stage]), src);
          }
          if (lane == 0) notes->ok[stage] = ok ? 1 : 0;
        }
      }
    }
    cp_async_commit();
  };
  auto open = [&](const Cursor& cu, int from) {
    Loads a;
    const int h = cu.h * p.unit_heads + hsub;
    a.trow = p.table + static_cast<int64_t>(cu.b) * p.table_st;
    a.kh = p.k + h * p.k_sh + r0 * p.k_st + cc * 16;   // this lane's piece
    a.vh = p.v + h * p.v_sh + r0 * p.v_st + cc * 16;
    a.scale_at = h;
    a.keys = unit_keys(p, cu.s, cu.t, RT);
    a.len = cu.s.len;
    a.s0 = from - cu.u0;
    a.s1 = min(unit_steps<WIN>(p, cu.s, cu.t, RT), v_end - cu.u0);
    a.skip = unit_skip<WIN>(p, cu.s, cu.t, RT);
    a.from = WIN ? unit_from(p, cu.s, cu.t, RT) : 0;
    a.ids_at = a.s0;
    a.ids = load_ids(a, a.s0);
    a.ids_next = load_ids(a, a.s0 + 32);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < R::kStages - 1; ++i) issue(a, a.s0 + i, i);
    return a;
  };

  Loads ld = open(c, v);
  bool first_segment = true;
  while (true) {
    const int s0 = ld.s0, s1 = ld.s1, keys = ld.keys;
    const bool whole = s0 == 0 && s1 == unit_steps<WIN>(p, c.s, c.t, RT);
    const int rows = min(RT, c.s.nq * p.G - c.t * RT);
    const int head = c.h * p.unit_heads + hsub;

    // the rows' queries as operand fragments, and how many keys each sees
    uint32_t qf[NK][4];
    float mul[2];
    int lim[2];
    int lim_min = keys, lim_max = 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = hf * 8 + g8;
      const bool live = r < rows;
      const int rr = c.t * RT + r;
      const int i = by_G(p, rr), g = rr - i * p.G;
      lim[hf] = live ? (p.is_causal ? min(max(c.s.len - c.s.nq + i + 1, 0), c.s.len) : c.s.len) : 0;
      if (live) lim_min = min(lim_min, lim[hf]);
      if (WIN) lim_max = max(lim_max, lim[hf]);
      const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) +
                            (static_cast<int64_t>(c.s.q0) + i) * p.q_st +
                            (static_cast<int64_t>(head) * p.G + g) * p.q_sh;
      uint2 w[NK];
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const int d = E4M3 ? 16 * (t4 + 4 * (ks / 4)) + 4 * (ks % 4)
                           : 8 * (t4 + 4 * (ks / 2)) + 4 * (ks % 2);
        w[ks] = live ? __ldg(reinterpret_cast<const uint2*>(src + d)) : make_uint2(0u, 0u);
      }
      float f = p.scale_log2;
      if constexpr (E4M3 && BF16) {
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
          top = max(top, max(w[ks].x & 0x7fffu, (w[ks].x >> 16) & 0x7fffu));
          top = max(top, max(w[ks].y & 0x7fffu, (w[ks].y >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - exponent of the row's largest element), itself within fp32
        const int e = max(static_cast<int>(top >> 7) - 127, -110);
        const float up = __int_as_float((127 + 14 - e) << 23);
        f *= __int_as_float((127 - 14 + e) << 23);
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
          const float2 a = unpack2<true>(w[ks].x), b = unpack2<true>(w[ks].y);
          w[ks].x = pack2<false>(a.x * up, a.y * up);
          w[ks].y = pack2<false>(b.x * up, b.y * up);
        }
      }
      mul[hf] = f;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        qf[ks][hf] = w[ks].x;
        qf[ks][2 + hf] = w[ks].y;
      }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    if (WIN) lim_max = __reduce_max_sync(0xffffffffu, lim_max);

    float o[NV][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

    int stage = 0;
    for (int s = s0; s < s1; ++s) {
      cp_async_wait<R::kStages - 2>();
      __syncwarp();
      issue(ld, s + R::kStages - 1, stage == 0 ? R::kStages - 1 : stage - 1);
      const int key0 = key_of(ld.skip, s);
      if (key0 < keys && notes->ok[stage] != 0) {
        const uint8_t* kt = ring + stage * 2 * R::kTile;
        const uint8_t* vt = kt + R::kTile;
        // S = Q K^T: thread (g8, t4) reads pieces t4, t4 + 4, .. of keys g8
        // and 8 + g8
        float acc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int cc = 0; cc < RB / 64; ++cc) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(
                kt + piece_at<RB, false>(n * 8 + g8, t4 + 4 * cc));
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            if constexpr (E4M3) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t b0 = codes_to_half2(w[e]), b1 = codes_to_half2_hi(w[e]);
                mma16816<MBF>(acc[n], qf[cc * 4 + e], b0, b1);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                mma16816<MBF>(acc[n], qf[cc * 2 + e], w[2 * e], w[2 * e + 1]);
            }
          }
        float ksc = 1.0f, lv = 0.0f, ivs = 1.0f;
        if constexpr (E4M3) {
          ksc = clamp_scale(notes->k_scale[stage]);
          const float vsc = clamp_scale(notes->v_scale[stage]);
          lv = lg2(vsc);
          ivs = rcp(vsc);
        }
        bool grow = false;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float f = mul[hf] * ksc;
          float* x = acc[0] + 2 * hf;
          float* y = acc[1] + 2 * hf;
          x[0] = fmaf(x[0], f, lv);
          x[1] = fmaf(x[1], f, lv);
          y[0] = fmaf(y[0], f, lv);
          y[1] = fmaf(y[1], f, lv);
        }
        if (key0 + kWarpKeys > lim_min || (WIN && key0 < lim_max - p.window && key0 + kWarpKeys > p.sinks)) {
          // some row does not see some of these keys
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + n * 8 + t4 * 2 + (e & 1);
              if (key >= lim[e >> 1] || (WIN && key < lim[e >> 1] - p.window && key >= p.sinks)) acc[n][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          grow |= fmaxf(max3f(acc[0][2 * hf], acc[0][2 * hf + 1], acc[1][2 * hf]),
                        acc[1][2 * hf + 1]) > m[hf] + W::kRoom;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float x = fmaxf(fmaxf(acc[0][2 * hf], acc[0][2 * hf + 1]),
                            fmaxf(acc[1][2 * hf], acc[1][2 * hf + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            x -= W::kTop;
            if (x > m[hf]) {
              const float alpha = ex2(m[hf] - x);
              m[hf] = x;
              l[hf] *= alpha;
#pragma unroll
              for (int j = 0; j < NV; ++j) {
                o[j][2 * hf] *= alpha;
                o[j][2 * hf + 1] *= alpha;
              }
            }
          }
        }
        // weights, rounded to 16 bits for the second product (the sum keeps
        // them in fp32)
        uint32_t pf[4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float mm = m[hf] == -INFINITY ? 0.0f : m[hf];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float w0 = ex2(acc[n][2 * hf] - mm), w1 = ex2(acc[n][2 * hf + 1] - mm);
            l[hf] = fmaf(w0 + w1, ivs, l[hf]);
            pf[2 * n + hf] = pack2<MBF>(w0, w1);
          }
        }
        // O += P V: thread (g8, t4) reads its run of columns of keys 2 t4,
        // 2 t4 + 1, 8 + 2 t4, 9 + 2 t4, and pairs neighbouring keys' elements
        auto columns = [&](int piece, int sub, int j0) {
          uint4 x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint8_t* at = vt + piece_at<RB, true>(2 * t4 + (e & 1) + 8 * (e >> 1), piece);
            if constexpr (RB == 64) {
              const uint2 y = *reinterpret_cast<const uint2*>(at + sub * 8);
              x[e] = make_uint4(y.x, y.y, 0u, 0u);
            } else {
              x[e] = *reinterpret_cast<const uint4*>(at);
            }
          }
#pragma unroll
          for (int e = 0; e < (RB == 64 ? 2 : 4); ++e) {
            auto word = [&](int k) { return e == 0 ? x[k].x : e == 1 ? x[k].y : e == 2 ? x[k].z : x[k].w; };
            const uint32_t a = word(0), b = word(1), cw = word(2), d = word(3);
            if constexpr (E4M3) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const uint32_t lo = __byte_perm(a, b, hh ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(cw, d, hh ? 0x7362 : 0x5140);
                const uint32_t l0 = codes_to_half2(lo), l1 = codes_to_half2_hi(lo);
                const uint32_t h0 = codes_to_half2(hi), h1 = codes_to_half2_hi(hi);
                mma16816<MBF>(o[j0 + e * 4 + hh * 2], pf, l0, h0);
                mma16816<MBF>(o[j0 + e * 4 + hh * 2 + 1], pf, l1, h1);
              }
            } else {
              const uint32_t l0 = __byte_perm(a, b, 0x5410), l1 = __byte_perm(a, b, 0x7632);
              const uint32_t h0 = __byte_perm(cw, d, 0x5410), h1 = __byte_perm(cw, d, 0x7632);
              mma16816<MBF>(o[j0 + e * 2], pf, l0, h0);
              mma16816<MBF>(o[j0 + e * 2 + 1], pf, l1, h1);
            }
          }
        };
        if constexpr (RB == 64) {
          columns(g8 >> 1, g8 & 1, 0);
        } else if constexpr (RB == 128) {
          columns(g8, 0, 0);
        } else {
          columns(g8, 0, 0);
          columns(g8 + 8, 0, 8);
        }
      }
      stage = stage + 1 == R::kStages ? 0 : stage + 1;
    }

    // the next unit
    const int v_next = c.u0 + s1;
    const bool more = v_next < v_end;
    // The join may start only now: its blocks, waiting early, would take the
    // place of CTAs of the next call's kernel on some SMs and leave those
    // behind (64 sequences up to 4096 tokens: 110 us a call, so 72).
    if (!more) grid_launch_dependents();
    Cursor next = c;
    if (more) {
      advance<WIN>(p, RT, next);
      if (slices == 1) ld = open(next, v_next);
    } else if (threadIdx.x == 0) {
      leave_note<WIN>(p, cta, total, n_ranges, RT, c, s0, s1, first_segment);
    }

    // Accumulator columns 2 t4 and 2 t4 + 1 of group j are elements j of the
    // runs 2 t4 and 2 t4 + 1; column of element j of run n:
    auto column = [](int n, int j) {
      return (E4M3 || D == 64) ? n * NV + j : (j < 8 ? 8 * n + j : 64 + 8 * n + j - 8);
    };
    float* part = part_rows<D>(p, cta, first_segment ? 0 : 1, RT);
    if (slices > 1) {
      // join the head's warps: each leaves its rows' maximum, sum and O (over
      // its own ring, which holds no copies in flight any more)
      cp_async_wait<0>();
      __syncthreads();
    }
    float* join = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float ls = l[hf];
      ls += __shfl_xor_sync(0xffffffffu, ls, 1);
      ls += __shfl_xor_sync(0xffffffffu, ls, 2);
      const float mx = m[hf];
      const int r = hf * 8 + g8;
      if (slices > 1) {
        if (t4 == 0) {
          ml[(warp * RT + r) * 2] = mx;
          ml[(warp * RT + r) * 2 + 1] = ls;
        }
      }
      if (r >= rows) continue;
      if (slices > 1 || !whole) {
        float* row = slices > 1 ? join + (warp * RT + r) * S::kJoinRow : part + (hsub * RT + r) * D;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NV; j += 2)
            *reinterpret_cast<float2*>(row + column(2 * t4 + e, j)) =
                make_float2(o[j][2 * hf + e], o[j + 1][2 * hf + e]);
        if (slices == 1 && t4 == 0) *part_sums<D>(part, p.unit_heads, RT, hsub * RT + r) = make_float2(mx, ls);
      } else {
        const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NV; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack2<BF16>(o[j + 2 * k][2 * hf + e] * inv, o[j + 2 * k + 1][2 * hf + e] * inv);
            *reinterpret_cast<uint4*>(out_row(p, c.s.q0, head, c.t * RT + r) + column(2 * t4 + e, j)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        if (t4 == 0 && p.lse != nullptr) store_lse(p, c.s.q0, head, c.t * RT + r, mx, ls);
      }
    }
    if (slices > 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < p.unit_heads * rows * (D / 4); i += kThreads) {
        const int d = (i % (D / 4)) * 4, hr = i / (D / 4);
        const int hs = hr / rows, r = hr - hs * rows;
        float mx = -INFINITY;
        for (int w = hs; w < kWarps; w += p.unit_heads) mx = fmaxf(mx, ml[(w * RT + r) * 2]);
        const float base = mx == -INFINITY ? 0.0f : mx;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float ls = 0.0f;
        for (int w = hs; w < kWarps; w += p.unit_heads) {
          const float a = ex2(ml[(w * RT + r) * 2] - base);
          const float4 x = *reinterpret_cast<const float4*>(join + (w * RT + r) * S::kJoinRow + d);
          sum.x = fmaf(x.x, a, sum.x);
          sum.y = fmaf(x.y, a, sum.y);
          sum.z = fmaf(x.z, a, sum.z);
          sum.w = fmaf(x.w, a, sum.w);
          ls = fmaf(ml[(w * RT + r) * 2 + 1], a, ls);
        }
        const int hd = c.h * p.unit_heads + hs;
        if (whole) {
          store_out4<D, BF16>(out_row(p, c.s.q0, hd, c.t * RT + r) + d, sum, ls == 0.0f ? 0.0f : 1.0f / ls);
          if (d == 0 && p.lse != nullptr) store_lse(p, c.s.q0, hd, c.t * RT + r, mx, ls);
        } else {
          *reinterpret_cast<float4*>(part + (hs * RT + r) * D + d) = sum;
          if (d == 0) *part_sums<D>(part, p.unit_heads, RT, hs * RT + r) = make_float2(mx, ls);
        }
      }
      __syncthreads();
    }
    if (!more) break;
    first_segment = false;
    c = next;
    v = v_next;
    if (slices > 1) ld = open(c, v);
  }
}

// Joins a unit that several CTAs worked on, by the note of the CTA where it
// begins (blockIdx.x).  A warp takes a row: lane k reads piece k's maximum and
// sum, then each lane four columns of one piece after the other (head size 64:
// half the lanes every second piece), DEEP pieces asked for at once: one sequence of
// 1000 tokens 12.4 -> 11.0 us with eight (one behind the other where they were fewer);
// many rows want many blocks, four (chunks 305 us, with eight 310).
template <int D, bool BF16, int DEEP>
__global__ void __launch_bounds__(kThreads)
    paged_join_kernel(const __grid_constant__ PagedParams p, int rt) {
  grid_dependency_wait();
  const int i = static_cast<int>(blockIdx.x);
  const JoinNote note = reinterpret_cast<const JoinNote*>(p.part)[i];
  if (note.pieces == 0) return;
  constexpr int kCols = D / 4, kSplit = 32 / kCols;
  const int lane = threadIdx.x & 31, d = (lane % kCols) * 4, first = lane / kCols;
  const int64_t step = static_cast<int64_t>(2) * note.heads * rt * (D + 2);   // the next CTA's first piece
  // (the grid has rows for the caller's bound on them, which may be too small)
  for (int hr = static_cast<int>(blockIdx.y * kWarps + (threadIdx.x >> 5)); hr < note.heads * note.rows;
       hr += static_cast<int>(gridDim.y) * kWarps) {
    const int hs = hr / note.rows, r = hr - hs * note.rows;
    float* const rows0 = part_rows<D>(p, i, note.slot, rt);
    float* const rows1 = part_rows<D>(p, i + 1, 0, rt);
    auto piece = [&](int k) { return k == 0 ? rows0 : rows1 + (k - 1) * step; };
    float mx = -INFINITY, ls = 0.0f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < note.pieces; k0 += 32) {
      const int n = min(note.pieces - k0, 32);
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (lane < n) ml = *part_sums<D>(piece(k0 + lane), note.heads, rt, hs * rt + r);
      float top = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (top > mx) {
        const float f = ex2(mx - top);   // 0 for the first pieces
        sum.x *= f, sum.y *= f, sum.z *= f, sum.w *= f;
        ls *= f;
        mx = top;
      }
      const float f = ex2(ml.x - (mx == -INFINITY ? 0.0f : mx));
      float l = ml.y * f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      ls += l;
#pragma unroll 1
      for (int k = 0; k < n; k += DEEP * kSplit) {
        float4 x[DEEP];
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
          const int kk = k + u * kSplit + first;
          x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (kk < n) x[u] = *reinterpret_cast<const float4*>(piece(k0 + kk) + (hs * rt + r) * D + d);
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
          const int kk = k + u * kSplit + first;
          const float fk = __shfl_sync(0xffffffffu, f, kk & 31);
          if (kk < n) {
            sum.x = fmaf(x[u].x, fk, sum.x);
            sum.y = fmaf(x[u].y, fk, sum.y);
            sum.z = fmaf(x[u].z, fk, sum.z);
            sum.w = fmaf(x[u].w, fk, sum.w);
          }
        }
      }
    }
    if (kSplit == 2) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, 16);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, 16);
      sum.z += __shfl_xor_sync(0xffffffffu, sum.z, 16);
      sum.w += __shfl_xor_sync(0xffffffffu, sum.w, 16);
    }
    const int h = note.kv_head0 + hs;
    if (first == 0)
      store_out4<D, BF16>(out_row(p, note.q0, h, note.row0 + r) + d, sum, ls == 0.0f ? 0.0f : 1.0f / ls);
    if (lane == 0 && p.lse != nullptr) store_lse(p, note.q0, h, note.row0 + r, mx, ls);
  }
}

template <class K, class... A>
cudaError_t launch_pdl(K kern, dim3 grid, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool BF16>
cudaError_t launch_join(const PagedParams& p, int rt, cudaStream_t stream) {
  if (p.n_ctas < 2) return cudaSuccess;
  // a row a warp, or four when there are many
  const int rows = (p.max_rows < rt ? p.max_rows : rt) * p.unit_heads;
  const int block_rows = rows <= 64 ? kWarps : 4 * kWarps;
  const dim3 grid(static_cast<unsigned>(p.n_ctas - 1), static_cast<unsigned>((rows + block_rows - 1) / block_rows));
  return rt <= RT ? launch_pdl(paged_join_kernel<D, BF16, 8>, grid, 0, stream, p, rt)
                  : launch_pdl(paged_join_kernel<D, BF16, 4>, grid, 0, stream, p, rt);
}

template <int D, bool E4M3, bool BF16, bool WIN>
cudaError_t launch_one(const PagedParams& p, cudaStream_t stream) {
  using S = Smem<D, E4M3>;
  auto kern = paged_kernel<D, E4M3, BF16, WIN>;
  static std::atomic<uint64_t> configured{0};  // a bit a device
  const uint64_t bit = 1ull << p.device;
  cudaError_t e = cudaSuccess;
  if ((configured.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kTotal);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_pdl(kern, dim3(static_cast<unsigned>(p.n_ctas)), S::kTotal, stream, p);
  if (e != cudaSuccess) return e;
  return launch_join<D, BF16>(p, RT, stream);
}

template <int D, bool WIN>
cudaError_t launch_dim(const PagedParams& p, bool bf16, bool e4m3, cudaStream_t s) {
  if (e4m3) return bf16 ? launch_one<D, true, true, WIN>(p, s) : launch_one<D, true, false, WIN>(p, s);
  return bf16 ? launch_one<D, false, true, WIN>(p, s) : launch_one<D, false, false, WIN>(p, s);
}

}  // namespace

namespace sdpa_impl {

cudaError_t launch_paged(const PagedParams& p, int head_dim, bool bf16, bool e4m3, cudaStream_t stream) {
  if (p.window != 0)
    return head_dim == 64 ? launch_dim<64, true>(p, bf16, e4m3, stream) : launch_dim<128, true>(p, bf16, e4m3, stream);
  return head_dim == 64 ? launch_dim<64, false>(p, bf16, e4m3, stream) : launch_dim<128, false>(p, bf16, e4m3, stream);
}

cudaError_t launch_paged_join(const PagedParams& p, int head_dim, bool bf16, int rt, cudaStream_t stream) {
  if (head_dim == 64)
    return bf16 ? launch_join<64, true>(p, rt, stream) : launch_join<64, false>(p, rt, stream);
  return bf16 ? launch_join<128, true>(p, rt, stream) : launch_join<128, false>(p, rt, stream);
}

}  // namespace sdpa_impl
