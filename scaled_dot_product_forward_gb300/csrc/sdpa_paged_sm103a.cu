// sdpa_paged_sm103a.cu -- attention of a few new tokens a sequence over a
// paged key/value cache (16-bit, or e4m3 with a scale a page and head), for
// sm_103a.
//
// For the rows of one key/value head (a token's G query heads share it) and
// key j, s_j = scale * ks_j * (q . kcode_j) and out = sum_j p_j vs_j vcode_j /
// sum_j p_j.  One pass over the pages, online: with a = scale * log2(e), each
// key's weight is w_j = 2^(a ks_j q.kcode_j + log2 vs_j - m), m the running
// maximum of that exponent, so that the value's scale is inside the weight
// before it is rounded to 16 bits (w <= 2^8 whatever the scales are), and
//     out = sum_j w_j vcode_j / sum_j w_j / vs_j,
// the sums in fp32.  e4m3 codes are exact in fp16, so products of an 8-bit
// cache run in fp16 whatever the query's type: a bf16 query row is brought to
// fp16 by a power of two that takes its largest element to 2^14 .. 2^15 (exact
// for elements down to 2^-29 of it; the factor goes into the score's).
//
// Bound by memory while few rows share the keys: 2 D bytes (e4m3) a key and
// head against 4 G D operations.  Each of a CTA's four warps reads its own 16
// keys of every 64 (16 keys lie in one page, whose entry and scales the warp
// needs once) into its own ring of stages with asynchronous 16-byte copies and
// multiplies from there: no block barrier and no exchange between warps until
// the unit ends, when their sums are joined.  The tensor work is one 16 x 16
// tile a step (mma.sync; the rows of one head seldom fill it): a tcgen05 tile
// of 128 rows would be 7/8 padding here.  The order of D inside both products
// is free, so each thread takes 16 consecutive bytes of a key's row as they
// lie in memory, and the output's columns come out in runs of D / 4.
#include <atomic>

#include "sdpa_paged.cuh"

using namespace sdpa_dev;
using namespace sdpa_paged;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWarpKeys = 16;
constexpr int KT = kWarps * kWarpKeys;  // keys a step
constexpr float kRescaleLog2 = 8.0f;

template <int D, bool E4M3>
struct Ring {
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kTile = kWarpKeys * kRowBytes;  // 16 keys of K or of V
  static constexpr int kStages = kTile == 4096 ? 3 : 4;
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

struct WarpScratch {      // a warp's notes on its stages
  float k_scale[4], v_scale[4];
  int ok[4];              // 0: the stage's page is not one of the cache's
};

template <int D, bool E4M3, bool BF16, int MT>
struct Smem {
  static constexpr int RT = 16 * MT;
  using R = Ring<D, E4M3>;
  static constexpr int kJoinRow = D + 4;                        // floats
  static constexpr int kJoin = kWarps * RT * kJoinRow * 4;      // over the rings
  static constexpr int kRings = kWarps * R::kWarpBytes;
  static constexpr int kBulk = kRings > kJoin ? kRings : kJoin;
  static constexpr int kNotes = kBulk;
  static constexpr int kMl = kNotes + static_cast<int>(sizeof(WarpScratch)) * kWarps;
  static constexpr int kDivide = (kMl + kWarps * RT * 8 + 15) / 16 * 16;
  // Not below 80 KB: two CTAs an SM and never three, or the kernel's equal
  // shares land on some SMs three at a time and on others one.
  static constexpr int kNeed = kDivide + static_cast<int>(sizeof(DivideScratch));
  static constexpr int kTotal = kNeed > 80 * 1024 ? kNeed : 80 * 1024;
  static_assert(2 * (kTotal + 1024) <= 227 * 1024, "two CTAs an SM");
};

// Writes a finished element group (4 values of row r from column d) of a unit.
template <int D, bool BF16>
__device__ __forceinline__ void store_out4(const PagedParams& p, const Cursor& c, int row, int d,
                                           const float4& o, float inv) {
  const int i = row / p.G, g = row - i * p.G;
  uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (static_cast<int64_t>(c.s.q0) + i) * p.o_st +
                  (static_cast<int64_t>(c.h) * p.G + g) * p.o_sh + d;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
}
__device__ __forceinline__ void store_lse(const PagedParams& p, const Cursor& c, int row, float m,
                                          float l) {
  const int i = row / p.G, g = row - i * p.G;
  constexpr float kLn2 = 0.693147180559945309f;
  p.lse[(static_cast<int64_t>(c.s.q0) + i) * p.lse_st +
        (static_cast<int64_t>(c.h) * p.G + g) * p.lse_sh] =
      l == 0.0f ? -INFINITY : (log2f(l) + m) * kLn2;
}

template <int D, bool E4M3, bool BF16, int MT>
__global__ void __launch_bounds__(kThreads)
    paged_kernel(const __grid_constant__ PagedParams p) {
  using S = Smem<D, E4M3, BF16, MT>;
  using R = Ring<D, E4M3>;
  constexpr int RT = 16 * MT;
  constexpr int NK = D / 16;              // k-steps of S
  constexpr int NV = D / 8;               // column groups of O
  constexpr int RB = R::kRowBytes;
  constexpr bool MBF = BF16 && !E4M3;     // type of the products
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + warp * R::kWarpBytes;
  const uint32_t ring_addr = smem_addr(ring);
  WarpScratch* notes = reinterpret_cast<WarpScratch*>(smem + S::kNotes) + warp;
  float* ml = reinterpret_cast<float*>(smem + S::kMl);  // [warp][RT][2]
  DivideScratch* sc = reinterpret_cast<DivideScratch*>(smem + S::kDivide);

  grid_dependency_wait();
  grid_launch_dependents();

  const int cta = static_cast<int>(blockIdx.x);
  long long total;
  Cursor c;
  long long v = divide<KT, kThreads>(
      p, RT, sc,
      [&](long long all) {
        const int n = range_count(all, p.n_ctas);
        return cta < n ? range_start(all, cta, n) : all;
      },
      total, c);
  const int n_ranges = range_count(total, p.n_ctas);
  if (v < 0) {
    // more CTAs than steps
    if (threadIdx.x == 0) reinterpret_cast<JoinNote*>(p.part)[cta].pieces = 0;
    return;
  }
  const long long v_end = range_start(total, cta + 1, n_ranges);
  bool first_segment = true;

  while (true) {
    const int steps = unit_steps<KT>(p, c.s, c.t, RT);
    const int s0 = static_cast<int>(v - c.u0);
    const int s1 = static_cast<int>(min(static_cast<long long>(steps), v_end - c.u0));
    const int rows = min(RT, c.s.nq * p.G - c.t * RT);
    const int keys = unit_keys(p, c.s, c.t, RT);

    // the rows' queries as operand fragments, and how many keys each sees
    uint32_t qf[MT][NK][4];
    float mul[MT][2];
    int lim[MT][2];
    int lim_min = keys;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = mt * 16 + hf * 8 + g8;
        const bool live = r < rows;
        const int rr = c.t * RT + r;
        const int i = rr / p.G, g = rr - i * p.G;
        lim[mt][hf] = live ? (p.is_causal ? min(max(c.s.len - c.s.nq + i + 1, 0), c.s.len) : c.s.len) : 0;
        if (live) lim_min = min(lim_min, lim[mt][hf]);
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) +
                              (static_cast<int64_t>(c.s.q0) + i) * p.q_st +
                              (static_cast<int64_t>(c.h) * p.G + g) * p.q_sh;
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
        mul[mt][hf] = f;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
          qf[mt][ks][hf] = w[ks].x;
          qf[mt][ks][2 + hf] = w[ks].y;
        }
      }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[MT][NV][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.0f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.0f;
    }

    // Page entries: lane i holds the entry of step `ids_at + i`'s 16 keys.
    const int* trow = p.table + static_cast<int64_t>(c.b) * p.table_st;
    auto load_ids = [&](int s) {
      const int key0 = (s + lane) * KT + warp * kWarpKeys;
      return (s + lane < s1 && key0 < keys) ? __ldg(trow + (key0 >> p.page_shift)) : -1;
    };
    int ids_at = s0;
    int ids = load_ids(s0), ids_next = load_ids(s0 + 32);
    const int page_mask = (1 << p.page_shift) - 1;
    const uint8_t* kh = p.k + c.h * p.k_sh;
    const uint8_t* vh = p.v + c.h * p.v_sh;

    auto issue = [&](int s, int stage) {
      if (s < s1) {
        if (s - ids_at == 32) {
          ids = ids_next;
          ids_at += 32;
          ids_next = load_ids(ids_at + 32);
        }
        const int page = __shfl_sync(0xffffffffu, ids, s - ids_at);
        const int key0 = s * KT + warp * kWarpKeys;
        const bool ok = page >= 0 && page < p.n_pages;
        const int64_t pg = ok ? page : 0;
        const int tok = key0 & page_mask;
        if (key0 < keys) {
          constexpr int kPieces = RB / 16;
          constexpr int kRowsAtOnce = 32 / kPieces;
          const int r0 = lane / kPieces, cc = lane % kPieces;
          const uint8_t* ks = kh + pg * p.k_sp + (tok + r0) * p.k_st + cc * 16;
          const uint8_t* vs = vh + pg * p.v_sp + (tok + r0) * p.v_st + cc * 16;
          const uint32_t dst = ring_addr + stage * 2 * R::kTile;
#pragma unroll
          for (int i = 0; i < kWarpKeys / kRowsAtOnce; ++i) {
            const int r = r0 + i * kRowsAtOnce;
            // rows past the sequence's end read as zeros: their weights are
            // zero, and a stale NaN there must not meet them
            const bool in = ok && key0 + r < c.s.len;
            cp16(dst + piece_at<RB, false>(r, cc), ks + i * kRowsAtOnce * p.k_st, in);
            cp16(dst + R::kTile + piece_at<RB, true>(r, cc), vs + i * kRowsAtOnce * p.v_st, in);
          }
          if (lane < 2) {
            if constexpr (E4M3) {
              const float* src = (lane == 0 ? p.k_scale : p.v_scale) + pg * p.n_kv + c.h;
              cp4(smem_addr(lane == 0 ? &notes->k_scale[stage] : &notes->v_scale[stage]), src);
            }
            if (lane == 0) notes->ok[stage] = ok ? 1 : 0;
          }
        }
      }
      cp_async_commit();
    };

#pragma unroll
    for (int i = 0; i < R::kStages - 1; ++i) issue(s0 + i, i);
    int stage = 0;
    for (int s = s0; s < s1; ++s) {
      cp_async_wait<R::kStages - 2>();
      __syncwarp();
      {
        const int ahead = stage == 0 ? R::kStages - 1 : stage - 1;
        issue(s + R::kStages - 1, ahead);
      }
      const int key0 = s * KT + warp * kWarpKeys;
      if (key0 < keys && notes->ok[stage] != 0) {
        const uint8_t* kt = ring + stage * 2 * R::kTile;
        const uint8_t* vt = kt + R::kTile;
        // S = Q K^T: thread (g8, t4) reads pieces t4, t4 + 4, .. of keys g8
        // and 8 + g8
        float acc[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][n][e] = 0.0f;
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
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma16816<MBF>(acc[mt][n], qf[mt][cc * 4 + e], b0, b1);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  mma16816<MBF>(acc[mt][n], qf[mt][cc * 2 + e], w[2 * e], w[2 * e + 1]);
            }
          }
        float ksc = 1.0f, lv = 0.0f, ivs = 1.0f;
        if constexpr (E4M3) {
          ksc = clamp_scale(notes->k_scale[stage]);
          const float vsc = clamp_scale(notes->v_scale[stage]);
          lv = lg2(vsc);
          ivs = 1.0f / vsc;
        }
        const bool all_seen = key0 + kWarpKeys <= lim_min;
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float f = mul[mt][hf] * ksc;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& x = acc[mt][n][2 * hf + e];
                x = fmaf(x, f, lv);
                if (!all_seen && key0 + n * 8 + t4 * 2 + e >= lim[mt][hf]) x = -INFINITY;
                grow |= x > m[mt][hf] + kRescaleLog2;
              }
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float x = fmaxf(fmaxf(acc[mt][0][2 * hf], acc[mt][0][2 * hf + 1]),
                              fmaxf(acc[mt][1][2 * hf], acc[mt][1][2 * hf + 1]));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              if (x > m[mt][hf]) {
                const float alpha = ex2(m[mt][hf] - x);
                m[mt][hf] = x;
                l[mt][hf] *= alpha;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                  o[mt][j][2 * hf] *= alpha;
                  o[mt][j][2 * hf + 1] *= alpha;
                }
              }
            }
        }
        // weights, rounded to 16 bits for the second product (the sum keeps
        // them in fp32)
        uint32_t pf[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float mm = m[mt][hf] == -INFINITY ? 0.0f : m[mt][hf];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float w0 = ex2(acc[mt][n][2 * hf] - mm), w1 = ex2(acc[mt][n][2 * hf + 1] - mm);
              l[mt][hf] = fmaf(w0 + w1, ivs, l[mt][hf]);
              pf[mt][2 * n + hf] = pack2<MBF>(w0, w1);
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
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  mma16816<MBF>(o[mt][j0 + e * 4 + hh * 2], pf[mt], l0, h0);
                  mma16816<MBF>(o[mt][j0 + e * 4 + hh * 2 + 1], pf[mt], l1, h1);
                }
              }
            } else {
              const uint32_t l0 = __byte_perm(a, b, 0x5410), l1 = __byte_perm(a, b, 0x7632);
              const uint32_t h0 = __byte_perm(cw, d, 0x5410), h1 = __byte_perm(cw, d, 0x7632);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<MBF>(o[mt][j0 + e * 2], pf[mt], l0, h0);
                mma16816<MBF>(o[mt][j0 + e * 2 + 1], pf[mt], l1, h1);
              }
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

    // Join the warps: each leaves its rows' maximum, sum and O (over its own
    // ring, which holds no copies in flight any more).
    cp_async_wait<0>();
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float x = l[mt][hf];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const int r = mt * 16 + hf * 8 + g8;
        if (t4 == 0) {
          ml[(warp * RT + r) * 2] = m[mt][hf];
          ml[(warp * RT + r) * 2 + 1] = x;
        }
        if (r < rows) {
          float* row = join + (warp * RT + r) * S::kJoinRow;
          // accumulator columns 2 t4 and 2 t4 + 1 of group j are elements j of
          // the runs g8 = 2 t4 and 2 t4 + 1
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int run = 2 * t4 + e;
#pragma unroll
            for (int j = 0; j < NV; j += 4) {
              const int d = (E4M3 || D == 64) ? run * NV + j : (j < 8 ? 8 * run + j : 64 + 8 * run + j - 8);
              *reinterpret_cast<float4*>(row + d) =
                  make_float4(o[mt][j][2 * hf + e], o[mt][j + 1][2 * hf + e],
                              o[mt][j + 2][2 * hf + e], o[mt][j + 3][2 * hf + e]);
            }
          }
        }
      }
    __syncthreads();
    const bool whole = s0 == 0 && s1 == steps;
    float* part = part_rows<D>(p, blockIdx.x, first_segment ? 0 : 1, RT);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float mx = ml[r * 2];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, ml[(w * RT + r) * 2]);
      const float base = mx == -INFINITY ? 0.0f : mx;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = ex2(ml[(w * RT + r) * 2] - base);
        const float4 x = *reinterpret_cast<const float4*>(join + (w * RT + r) * S::kJoinRow + d);
        sum.x = fmaf(x.x, a, sum.x);
        sum.y = fmaf(x.y, a, sum.y);
        sum.z = fmaf(x.z, a, sum.z);
        sum.w = fmaf(x.w, a, sum.w);
        ls = fmaf(ml[(w * RT + r) * 2 + 1], a, ls);
      }
      if (whole) {
        store_out4<D, BF16>(p, c, c.t * RT + r, d, sum, ls == 0.0f ? 0.0f : 1.0f / ls);
        if (d == 0 && p.lse != nullptr) store_lse(p, c, c.t * RT + r, mx, ls);
      } else {
        float* row = part + r * (D + 2);
        *reinterpret_cast<float2*>(row + d) = make_float2(sum.x, sum.y);
        *reinterpret_cast<float2*>(row + d + 2) = make_float2(sum.z, sum.w);
        if (d == 0) *reinterpret_cast<float2*>(row + D) = make_float2(mx, ls);
      }
    }
    v = c.u0 + s1;
    if (v >= v_end) {
      if (threadIdx.x == 0) leave_note<KT>(p, cta, total, n_ranges, RT, c, s0, s1, first_segment);
      break;
    }
    first_segment = false;
    __syncthreads();
    advance<KT>(p, RT, c);
  }
}

// Joins a unit that several CTAs worked on, by the note of the CTA where it
// begins (blockIdx.x); a thread takes four columns of a row, a block
// kThreads * 4 / D rows.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
    paged_join_kernel(const __grid_constant__ PagedParams p, int rt) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int i = static_cast<int>(blockIdx.x);
  const JoinNote note = reinterpret_cast<const JoinNote*>(p.part)[i];
  if (note.pieces == 0) return;
  const int64_t step = static_cast<int64_t>(2) * rt * (D + 2);   // the next CTA's first piece
  // (the grid has rows for the caller's bound on them, which may be too small)
  for (int e = static_cast<int>(blockIdx.y * kThreads + threadIdx.x); e < note.rows * (D / 4);
       e += static_cast<int>(gridDim.y) * kThreads) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    const float* row0 = part_rows<D>(p, i, note.slot, rt) + r * (D + 2);
    const float* row1 = part_rows<D>(p, i + 1, 0, rt) + r * (D + 2);
    auto piece = [&](int k) { return k == 0 ? row0 : row1 + (k - 1) * step; };
    float mx = -INFINITY;
#pragma unroll 4
    for (int k = 0; k < note.pieces; ++k) mx = fmaxf(mx, piece(k)[D]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.0f;
#pragma unroll 4
    for (int k = 0; k < note.pieces; ++k) {
      const float* row = piece(k);
      const float2 x0 = *reinterpret_cast<const float2*>(row + d);
      const float2 x1 = *reinterpret_cast<const float2*>(row + d + 2);
      const float2 y = *reinterpret_cast<const float2*>(row + D);
      const float f = ex2(y.x - base);
      sum.x = fmaf(x0.x, f, sum.x);
      sum.y = fmaf(x0.y, f, sum.y);
      sum.z = fmaf(x1.x, f, sum.z);
      sum.w = fmaf(x1.y, f, sum.w);
      ls = fmaf(y.y, f, ls);
    }
    Cursor c{};
    c.s.q0 = note.q0;
    c.h = note.head0 / p.G;
    store_out4<D, BF16>(p, c, note.row0 + r, d, sum, ls == 0.0f ? 0.0f : 1.0f / ls);
    if (d == 0 && p.lse != nullptr) store_lse(p, c, note.row0 + r, mx, ls);
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
  const int rows = p.max_rows < rt ? p.max_rows : rt, block_rows = kThreads * 4 / D;
  return launch_pdl(paged_join_kernel<D, BF16>,
                    dim3(static_cast<unsigned>(p.n_ctas - 1), static_cast<unsigned>((rows + block_rows - 1) / block_rows)),
                    0, stream, p, rt);
}

template <int D, bool E4M3, bool BF16, int MT>
cudaError_t launch_one(const PagedParams& p, cudaStream_t stream) {
  using S = Smem<D, E4M3, BF16, MT>;
  auto kern = paged_kernel<D, E4M3, BF16, MT>;
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
  return launch_join<D, BF16>(p, S::RT, stream);
}

template <int D, bool E4M3, bool BF16>
cudaError_t launch_rows(const PagedParams& p, int rt, cudaStream_t stream) {
  return rt == 16 ? launch_one<D, E4M3, BF16, 1>(p, stream) : launch_one<D, E4M3, BF16, 2>(p, stream);
}

template <int D>
cudaError_t launch_dim(const PagedParams& p, int rt, bool bf16, bool e4m3, cudaStream_t s) {
  if (e4m3)
    return bf16 ? launch_rows<D, true, true>(p, rt, s) : launch_rows<D, true, false>(p, rt, s);
  return bf16 ? launch_rows<D, false, true>(p, rt, s) : launch_rows<D, false, false>(p, rt, s);
}

}  // namespace

namespace sdpa_impl {

cudaError_t launch_paged(const PagedParams& p, int head_dim, bool bf16, bool e4m3, int rt,
                         cudaStream_t stream) {
  return head_dim == 64 ? launch_dim<64>(p, rt, bf16, e4m3, stream)
                        : launch_dim<128>(p, rt, bf16, e4m3, stream);
}

cudaError_t launch_paged_join(const PagedParams& p, int head_dim, bool bf16, int rt, cudaStream_t stream) {
  if (head_dim == 64)
    return bf16 ? launch_join<64, true>(p, rt, stream) : launch_join<64, false>(p, rt, stream);
  return bf16 ? launch_join<128, true>(p, rt, stream) : launch_join<128, false>(p, rt, stream);
}

}  // namespace sdpa_impl
