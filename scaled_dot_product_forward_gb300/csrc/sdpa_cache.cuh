// sdpa_cache.cuh -- appending new tokens' keys and values to a paged cache,
// rotated by their positions, for sm_103a (the kernels without norms are
// compiled in sdpa_cache_sm103a.cu, those with them in sdpa_norm_sm103a.cu and
// sdpa_norm64_sm103a.cu).
//
// Token i of a sequence with n new tokens and len cached ones (the new ones
// among them) has position len - n + i; it goes to row pos % P of page
// table[pos / P].  Its key (and, if given, its queries) is rotated on the way:
// pair (x1, x2) of a head becomes (x1 c - x2 s, x2 c + x1 s) with (c, s) the
// position's table entries, each product and each sum rounded to fp32 on its
// own (no contraction), then rounded once to the cache's type.
//
// 8-bit caches hold e4m3 codes under one power-of-two scale a page and head:
// the least one under which every finite value fits in +-448.  e4m3 has its
// own exponent, so a finer scale would not round values any better, and a
// power of two makes raising it later exact but for codes that fall below the
// type's least normal: when a token arrives that does not fit, the page's
// earlier codes are multiplied by old / new in place.
//
// With norms (NORM) a key's or query's head is first divided by the root mean
// square of its D elements and multiplied by the weights, x rsqrt(sum x^2 / D +
// eps) w, in fp32: the row's lanes add up their squares by log2(D / 8) exchanges,
// and nothing is rounded before the rotation's end.  norm_rotate_kernel does the
// same to rows that go to no cache.  8 x 4096 tokens (H 32/8, D 128, e4m3): 127 us,
// 5.8 TB/s; 17700 rows of 16 + 16 heads of 64: 26 us, 5.6 TB/s.
//
// Bound by memory: each new row is read once and written once.  Two kinds of
// work share one launch:
//   * rows without a scale (the queries; 16-bit keys and values): a warp takes a
//     token's heads, or a share of them when tokens are few, four rows a lane
//     at a time, with the token's angles read once;
//   * 8-bit pages: one page's new rows of one head are one unit, of a warp (few
//     rows) or of several, so the scale of a (page, head) has one owner and needs
//     no atomics.  The rows wait in registers, four a lane, while their
//     largest value is found.
// Lane j of a row's D / 8 holds pairs 4j .. 4j + 3, both halves of each, so the
// rotation needs no exchange.
#pragma once
#include <cuda_fp8.h>

#include <type_traits>

#include "sdpa_paged.cuh"

using namespace sdpa_dev;
using namespace sdpa_paged;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitHeads = 4;   // of a unit of several warps, at most
constexpr int kPerSm = 4;   // blocks an SM: the loads' latency is hidden by warps, not by registers

// Where lane j of a row keeps its eight elements: a[0..3] from `ea`, b[0..3]
// from `eb`; pairs (a[e], b[e]) in the half-split form, (a0,a1), (a2,a3),
// (b0,b1), (b2,b3) when neighbours are paired.  rotated: the pairs have
// angles 4j .. 4j + 3.
struct Lane {
  int ea, eb;
  bool rotated;
};

__device__ __forceinline__ Lane lane_of(int j, int rot, int interleaved) {
  Lane l;
  if (8 * j < rot) {
    l.rotated = true;
    if (interleaved) {
      l.ea = 8 * j;
      l.eb = 8 * j + 4;
    } else {
      l.ea = 4 * j;
      l.eb = rot / 2 + 4 * j;
    }
  } else {
    l.rotated = false;
    l.ea = 8 * j;
    l.eb = 8 * j + 4;
  }
  return l;
}

// TOGETHER: the lane's eight elements are one run (nothing is rotated).
template <bool BF16, bool TOGETHER = false>
__device__ __forceinline__ void load8(const uint16_t* row, const Lane& l, float (&x)[8]) {
  // (plain loads: the queries may be rotated in place)
  uint2 a, b;
  if constexpr (TOGETHER) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + l.ea);
    a = make_uint2(w.x, w.y), b = make_uint2(w.z, w.w);
  } else {
    a = *reinterpret_cast<const uint2*>(row + l.ea);
    b = *reinterpret_cast<const uint2*>(row + l.eb);
  }
  const float2 f0 = unpack2<BF16>(a.x), f1 = unpack2<BF16>(a.y);
  const float2 f2 = unpack2<BF16>(b.x), f3 = unpack2<BF16>(b.y);
  x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
  x[4] = f2.x, x[5] = f2.y, x[6] = f3.x, x[7] = f3.y;
}

template <bool BF16, bool TOGETHER = false>
__device__ __forceinline__ void store8(uint16_t* row, const Lane& l, const float (&x)[8]) {
  const uint2 a = make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
  const uint2 b = make_uint2(pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
  if constexpr (TOGETHER) {
    *reinterpret_cast<uint4*>(row + l.ea) = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<uint2*>(row + l.ea) = a;
    *reinterpret_cast<uint2*>(row + l.eb) = b;
  }
}

// Two fp32 values an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// (x1, x2) of two pairs turned by (c, s): x1 c - x2 s, x2 c + x1 s.  (The sums
// one by one: a packed sum behind a packed product is made one operation,
// without the product's rounding.)
__device__ __forceinline__ void turn2(float& a1, float& b1, float& a2, float& b2, float c0, float c1, float s0,
                                      float s1) {
  const uint64_t x1 = pair(a1, b1), x2 = pair(a2, b2), c = pair(c0, c1), s = pair(s0, s1);
  float p0, p1, q0, q1, r0, r1, t0, t1;
  unpair(mul2(x1, c), p0, p1);
  unpair(mul2(x2, s), q0, q1);
  unpair(mul2(x2, c), r0, r1);
  unpair(mul2(x1, s), t0, t1);
  a1 = __fsub_rn(p0, q0);
  b1 = __fsub_rn(p1, q1);
  a2 = __fadd_rn(r0, t0);
  b2 = __fadd_rn(r1, t1);
}

__device__ __forceinline__ void rotate8(float (&x)[8], const float4& c, const float4& s,
                                        int interleaved) {
  if (interleaved) {
    turn2(x[0], x[2], x[1], x[3], c.x, c.y, s.x, s.y);
    turn2(x[4], x[6], x[5], x[7], c.z, c.w, s.z, s.w);
  } else {
    turn2(x[0], x[1], x[4], x[5], c.x, c.y, s.x, s.y);
    turn2(x[2], x[3], x[6], x[7], c.z, c.w, s.z, s.w);
  }
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The lane's weights (of elements ea .. ea + 3, eb .. eb + 3).
__device__ __forceinline__ void load_weights(const float* weight, const Lane& l, float (&w)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(weight + l.ea));
  const float4 b = __ldg(reinterpret_cast<const float4*>(weight + l.eb));
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// Sum over a row's LANES lanes, the same in each of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float square_sum(const uint64_t (&v)[4]) {
  float a, b;
  unpair(fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0])))), a, b);
  return a + b;
}

// 1 / sqrt(mean of squares + eps) of rows v[0 .. N), LANES lanes a row; the whole
// warp calls it.  Squares below 2^-126 do not matter beside eps >= 2^-100; those of
// values above 2^60 (bf16) may overflow: such a row becomes 2^-70 times as large
// and is summed again, without eps (nothing beside squares above 2^120).
template <int LANES, int N>
__device__ __forceinline__ void row_factors(uint64_t (&v)[N][4], float eps, float (&r)[N]) {
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) r[k] = square_sum(v[k]);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    r[k] = row_sum<LANES>(r[k]);
    most = fmaxf(most, r[k]);   // (drops a NaN)
  }
  if (__any_sync(0xffffffffu, most == INFINITY)) {
    const float down = 8.470329472543003e-22f;   // 2^-70
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const bool large = r[k] == INFINITY;
      const float f = large ? down : 1.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k][e] = mul2(v[k][e], pair(f, f));
      r[k] = rsqrtf(fmaf(row_sum<LANES>(square_sum(v[k])), 1.0f / (8 * LANES), large ? 0.0f : eps));
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = rsqrtf(fmaf(r[k], 1.0f / (8 * LANES), eps));
  }
}

// Rows x[0 .. N) normalised.
template <int LANES, int N>
__device__ __forceinline__ void normalise(float (&x)[N][8], const float (&w)[8], float eps) {
  uint64_t v[N][4];
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[k][e] = pair(x[k][2 * e], x[k][2 * e + 1]);
  float r[N];
  row_factors<LANES, N>(v, eps, r);
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      unpair(mul2(mul2(v[k][e], pair(r[k], r[k])), pair(w[2 * e], w[2 * e + 1])), x[k][2 * e], x[k][2 * e + 1]);
}

// The page's new tokens: positions [lo, hi), the first being row t0 of k, v, q.
struct PageTokens {
  int lo, hi, t0;
};

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float2 values2(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// What a scale has to cover: infinities and NaN are left out (an infinity is
// stored as +-448 codes, a NaN as NaN).
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}
__device__ __forceinline__ float abs_max(float m, float a, float b) {   // drops NaN, keeps infinities
  return max3f(m, fabsf(a), fabsf(b));
}

// The least power of two s with amax <= 448 s = 1.75 * 2^8 s, in range.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, sdpa_impl::kScaleMinExp), sdpa_impl::kScaleMaxExp);
  return __int_as_float((e + 127) << 23);
}

// Rows r, r + stride, .. (kBatch of them) of a unit of n rows, normalised (NORM)
// and rotated (ROT), in registers; rows from n on are zeros.  src, cos, sin: this
// lane's part of row r; steps in elements.
constexpr int kBatch = 4;
template <int D, bool BF16, bool ROT, bool NORM>
__device__ __forceinline__ void load_rows(const uint16_t* src, int64_t src_step, const float* cos, const float* sin,
                                          int64_t angle_step, const Lane& at, int interleaved, int r, int stride, int n,
                                          const float* weight, float eps, float (&x)[kBatch][8]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    if (r + k * stride < n) {
      load8<BF16, !ROT>(src, at, x[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = 0.0f;
    }
    src += src_step;
  }
  if (NORM && weight != nullptr) {
    float w[8];
    load_weights(weight, at, w);
    normalise<D / 8, kBatch>(x, w, eps);
  }
  if (ROT && at.rotated) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r + k * stride < n)
        rotate8(x[k], __ldg(reinterpret_cast<const float4*>(cos)), __ldg(reinterpret_cast<const float4*>(sin)), interleaved);
      cos += angle_step;
      sin += angle_step;
    }
  }
}

template <bool TOGETHER>
__device__ __forceinline__ void store_codes(uint8_t* to, int64_t step, const Lane& at, int r, int stride, int n, float inv,
                                            const float (&x)[kBatch][8]) {
  const uint64_t f = pair(inv, inv);
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    if (r + k * stride < n) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) unpair(mul2(pair(x[k][e], x[k][e + 1]), f), y[e], y[e + 1]);
      const uint32_t a = codes4(y[0], y[1], y[2], y[3]), b = codes4(y[4], y[5], y[6], y[7]);
      if constexpr (TOGETHER) {
        *reinterpret_cast<uint2*>(to + at.ea) = make_uint2(a, b);
      } else {
        *reinterpret_cast<uint32_t*>(to + at.ea) = a;
        *reinterpret_cast<uint32_t*>(to + at.eb) = b;
      }
    }
    to += step;
  }
}

// A unit: the page's new rows of one head, quantised under the page's scale, by
// WARPS warps (part: this one's number, red: their shared scratch); with several
// warps, of `heads` heads after one another, so that the page is looked up once
// for them.  8 x 4096 tokens with norms, 8 heads, pages of 64: one a unit 138 us, two
// 131, four 127, eight 125 but 63 without queries, where four take 56; pages of 32
// 151 and 133, of 16 151 and 139.  (Units of one warp gain 1%, a single token's
// append loses 5.)
template <int D, bool BF16, bool ROT, bool NORM, int WARPS>
__device__ __forceinline__ void append_codes(const sdpa_impl::AppendParams& p, const PageTokens& pt,
                                             const uint16_t* src, int64_t src_st, int64_t src_sh, uint8_t* dst,
                                             int64_t dst_st, int64_t dst_sh, float* scale_at, int heads, int part,
                                             float* red) {
  constexpr int kLanes = D / 8;                  // lanes a row
  constexpr int kStride = WARPS * 32 / kLanes;   // rows a step
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes, first = part * (32 / kLanes) + lane / kLanes;
  const Lane at = lane_of(j, ROT ? p.rot : 0, p.interleaved);
  const int n = pt.hi - pt.lo;
  const int row0 = pt.lo & ((1 << p.page_shift) - 1);
  // this lane's part of its first row, and from one of its rows to the next
  const uint16_t* rows = src + (static_cast<int64_t>(pt.t0) + first) * src_st;
  const int64_t row_step = kStride * src_st, angle_step = static_cast<int64_t>(kStride) * (p.rot / 2);
  const int64_t angle = (static_cast<int64_t>(pt.lo) + first) * (p.rot / 2) + 4 * j;
  const float* const cos = ROT ? p.cos + angle : nullptr;
  const float* const sin = ROT ? p.sin + angle : nullptr;
  auto load = [&](int batch, float (&x)[kBatch][8]) {
    load_rows<D, BF16, ROT, NORM>(rows + batch * (kBatch * row_step), row_step, cos + batch * (kBatch * angle_step),
                         sin + batch * (kBatch * angle_step), angle_step, at, p.interleaved,
                         first + batch * kBatch * kStride, kStride, n, p.k_norm, p.eps, x);
  };
  // (more rows than the registers hold are read again below)
  const int batches = (n + kBatch * kStride - 1) / (kBatch * kStride);
#pragma unroll 1
  for (int h = 0; h < (WARPS > 1 ? heads : 1); ++h) {
    // the page's scale, if earlier rows have made one
    float old = 0.0f;
    if (row0 > 0) old = clamp_scale(*scale_at);
    float x[kBatch][8];
    float amax = 0.0f;
#pragma unroll 1
    for (int i = 0; i < batches; ++i) {
      load(i, x);
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int e = 0; e < 8; e += 2) top = abs_max(top, x[k][e], x[k][e + 1]);
      if (top == INFINITY) {
        top = 0.0f;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_abs(x[k][e]));
      }
      amax = fmaxf(amax, top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (WARPS > 1) {
      // (heads in turn use two places: one barrier a head)
      float* const tops = red + (h & 1) * kWarps;
      if (lane == 0) tops[part] = amax;
      // the unit's warps (also: all have read the old scale)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / (WARPS * 32)), "n"(WARPS * 32) : "memory");
#pragma unroll
      for (int w = 0; w < WARPS; ++w) amax = fmaxf(amax, tops[w]);
    } else {
      __syncwarp();
    }
    float scale = scale_for(amax);
    if (row0 > 0) {
      if (scale > old) {
        // raise the scale: the page's earlier codes of this head
        const float ratio = old / scale;
        for (int i = part * 32 + lane; i < row0 * (D / 16); i += WARPS * 32) {
          uint4* at16 = reinterpret_cast<uint4*>(dst + (i / (D / 16)) * dst_st + (i % (D / 16)) * 16);
          const uint4 w = *at16;
          uint32_t in[4] = {w.x, w.y, w.z, w.w}, res[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = values2(in[e]), b = values2(in[e] >> 16);
            res[e] = codes4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
          }
          *at16 = make_uint4(res[0], res[1], res[2], res[3]);
        }
      } else {
        scale = old;
      }
    }
    if (part == 0 && lane == 0) *scale_at = scale;
    const float inv = 1.0f / scale;
    uint8_t* const to = dst + (row0 + first) * dst_st;
    const int64_t to_step = kStride * dst_st;
#pragma unroll 1
    for (int i = 0; i < batches; ++i) {
      if (batches > 1) load(i, x);
      store_codes<!ROT>(to + i * (kBatch * to_step), to_step, at, first + i * kBatch * kStride, kStride, n, inv, x);
    }
    rows += src_sh;
    dst += dst_sh;
    ++scale_at;
  }
}

// One warp: heads [h0, h1) of one token, rotated (ROT) or copied, four rows a
// lane at a time.  (c, s): the lane's angles.
template <int D, bool BF16, bool ROT>
__device__ __forceinline__ void token_rows(int interleaved, const Lane& at, const float4& c, const float4& s,
                                           const uint16_t* src, int64_t src_sh, uint8_t* dst, int64_t dst_sh_bytes,
                                           int h0, int h1) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  int h = h0 + static_cast<int>(threadIdx.x & 31) / kLanes;
  src += h * src_sh;
  dst += h * dst_sh_bytes;
  const int64_t src_step = kRows * src_sh, dst_step = kRows * dst_sh_bytes;
#pragma unroll 1
  for (; h < h1; h += kBatch * kRows) {
    float x[kBatch][8];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (h + u * kRows < h1) load8<BF16, !ROT>(src, at, x[u]);
      src += src_step;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (h + u * kRows < h1) {
        if (ROT && at.rotated) rotate8(x[u], c, s, interleaved);
        store8<BF16, !ROT>(reinterpret_cast<uint16_t*>(dst), at, x[u]);
      }
      dst += dst_step;
    }
  }
}

// The same heads normalised, then rotated.  The weights go into the angles, once a
// token, and a row's factor comes last: an element is (x m + x' n) r, m and n the
// products of its weight and its pair's with cosine and sine, x' the pair's other
// element (as many roundings as with the factor first).  The next rows are on
// their way while these are turned, and the first before the token's place is
// known: angles(c, s) looks it up, false for a token that is left out.
// PAIRED: neighbours are pairs.  ALL: all of a head is rotated.
constexpr int kNormBatch = 2;
template <int D, bool BF16, bool PAIRED, bool ALL, class Angles>
__device__ __forceinline__ void norm_rows_as(const Lane& at, Angles&& angles, const uint16_t* src, int64_t src_sh,
                                             uint8_t* dst, int64_t dst_sh_bytes, const float* weight, float eps, int h0, int h1) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  const int sub = static_cast<int>(threadIdx.x & 31) / kLanes;
  // from a lane's first four elements to its others (bytes)
  const int apart = PAIRED ? 8 : ALL ? D : 2 * (at.eb - at.ea);
  const uint8_t* from = reinterpret_cast<const uint8_t*>(src + (h0 + sub) * src_sh + at.ea);
  const int64_t from_step = kRows * src_sh * 2, to_step = kRows * dst_sh_bytes;
  uint2 raw[kNormBatch][2];
  auto ask = [&](int h) {
    // (plain loads: the queries may be rotated in place)
    if (h + kNormBatch * kRows <= h1) {
#pragma unroll
      for (int u = 0; u < kNormBatch; ++u) {
        raw[u][0] = *reinterpret_cast<const uint2*>(from);
        raw[u][1] = *reinterpret_cast<const uint2*>(from + apart);
        from += from_step;
      }
    } else {
#pragma unroll
      for (int u = 0; u < kNormBatch; ++u) {
        raw[u][0] = raw[u][1] = make_uint2(0u, 0u);
        if (h + sub + u * kRows < h1) {
          raw[u][0] = *reinterpret_cast<const uint2*>(from);
          raw[u][1] = *reinterpret_cast<const uint2*>(from + apart);
        }
        from += from_step;
      }
    }
  };
  ask(h0);
  float w[8];
  load_weights(weight, at, w);
  float4 c, s;
  if (!angles(c, s)) return;
  uint64_t m[4], n[4];
  if (!ALL && !at.rotated) {
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = pair(w[2 * e], w[2 * e + 1]), n[e] = 0;
  } else if (PAIRED) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = pair(w[2 * e] * cc[e], w[2 * e + 1] * cc[e]);
      n[e] = pair(-w[2 * e + 1] * ss[e], w[2 * e] * ss[e]);
    }
  } else {
    const uint64_t cc[2] = {pair(c.x, c.y), pair(c.z, c.w)}, ss[2] = {pair(s.x, s.y), pair(s.z, s.w)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = mul2(pair(w[2 * e], w[2 * e + 1]), cc[e]);
      n[2 + e] = mul2(pair(w[2 * e], w[2 * e + 1]), ss[e]);
      m[2 + e] = mul2(pair(w[4 + 2 * e], w[5 + 2 * e]), cc[e]);
      n[e] = mul2(pair(-w[4 + 2 * e], -w[5 + 2 * e]), ss[e]);
    }
  }
  uint8_t* to = dst + (h0 + sub) * dst_sh_bytes + 2 * at.ea;
  // (the sums are exchanged: the warp stays together)
#pragma unroll 1
  for (int h = h0; h < h1; h += kNormBatch * kRows) {
    uint64_t v[kNormBatch][4];
    float r[kNormBatch];
#pragma unroll
    for (int u = 0; u < kNormBatch; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint2 x = raw[u][e >> 1];
        const float2 f = unpack2<BF16>((e & 1) ? x.y : x.x);
        v[u][e] = pair(f.x, f.y);
      }
    if (h + kNormBatch * kRows < h1) ask(h + kNormBatch * kRows);
    row_factors<kLanes, kNormBatch>(v, eps, r);
#pragma unroll
    for (int u = 0; u < kNormBatch; ++u) {
      uint64_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t other = v[u][e ^ 2];
        if (PAIRED) {
          float a, b;
          unpair(v[u][e], a, b);
          other = pair(b, a);
        }
        // (an infinite element has no part in one that it is no pair of)
        y[e] = !ALL && !at.rotated ? mul2(v[u][e], m[e]) : fma2(v[u][e], m[e], mul2(other, n[e]));
      }
      uint32_t out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        unpair(mul2(y[e], pair(r[u], r[u])), a, b);
        out[e] = pack2<BF16>(a, b);
      }
      if (h + sub + u * kRows < h1) {
        *reinterpret_cast<uint2*>(to) = make_uint2(out[0], out[1]);
        *reinterpret_cast<uint2*>(to + apart) = make_uint2(out[2], out[3]);
      }
      to += to_step;
    }
  }
}
// (Knowing the form saves instructions: 8 x 4096 tokens of 32 + 8 heads 142 -> 139 us,
// 17700 rows of 16 + 16 heads of 64 29.2 -> 27.7; kernels of their own for them 26,
// sdpa_norm.cuh.  Two rows a lane at a time and four
// blocks an SM: with four rows and three blocks 144 and 30.5, with one row 160 and
// 34.5; without the next rows on their way 145 and 29.4.  Rows by asynchronous
// copies into a ring in shared memory, eight a lane on their way: 136 and 27.6, with
// twice the code and spills: not kept.)
template <int D, bool BF16, class Angles>
__device__ __forceinline__ void norm_rows(int rot, int interleaved, const Lane& at, Angles&& angles, const uint16_t* src,
                                          int64_t src_sh, uint8_t* dst, int64_t dst_sh_bytes, const float* weight, float eps,
                                          int h0, int h1) {
  auto go = [&](auto paired, auto all) {
    norm_rows_as<D, BF16, paired.value, all.value>(at, angles, src, src_sh, dst, dst_sh_bytes, weight, eps, h0, h1);
  };
  using std::false_type;
  using std::true_type;
  if (interleaved)
    rot == D ? go(true_type{}, true_type{}) : go(true_type{}, false_type{});
  else
    rot == D ? go(false_type{}, true_type{}) : go(false_type{}, false_type{});
}

// The last of n values, f(0) <= f(1) <= .., that is at most x (-1: none); the
// whole warp calls it.
template <class F>
__device__ __forceinline__ int last_at_most(int n, int x, F&& f) {
  int count = 0;
#pragma unroll 4
  for (int b0 = 0; b0 < n; b0 += 32) {
    const int i = b0 + static_cast<int>(threadIdx.x & 31);
    count += __popc(__ballot_sync(0xffffffffu, i < n && f(i) <= x));
  }
  return count - 1;
}

// Blocks [0, kv_blocks): units of 8-bit pages, UNIT_WARPS warps each.  (Evenly among
// the others, they are no faster: 8 x 4096 tokens with norms 130 us against 127.)  A slot
// stands for a (sequence, page with new tokens): sequence b has the slots
// [f(b), f(b+1)), f(b) = cu[b] / P + 2 b, at least as many as the pages its new
// tokens can touch, so a slot finds its sequence without a prefix sum over
// lengths; a slot's units are its value and key heads.  The other blocks: a
// warp takes a share (1 / parts) of one token's rows.
template <int D, bool BF16, bool E4M3, bool ROT, bool NORM, int UNIT_WARPS>
__global__ void __launch_bounds__(kThreads, kPerSm)
    append_kernel(const __grid_constant__ sdpa_impl::AppendParams p, int kv_blocks, int parts) {
  __shared__ float red[2 * kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int P = 1 << p.page_shift;
  const int uniform = p.total / p.n_seqs;
  const int warp = threadIdx.x >> 5;
  auto first_token = [&](int b) {
    return p.cu != nullptr ? min(max(__ldg(p.cu + b), 0), p.total) : b * uniform;
  };
  if constexpr (E4M3) {
    if (static_cast<int>(blockIdx.x) < kv_blocks) {
      const int part = warp % UNIT_WARPS;
      PageTokens pt;
      int hv = 0, page = -1;
      // the unit's page (-1: nothing to do) and its new tokens
      auto look_up = [&]() {
        const unsigned unit = blockIdx.x * (kWarps / UNIT_WARPS) + warp / UNIT_WARPS;
        const int unit_heads = UNIT_WARPS > 1 ? p.unit_heads : 1;
        const unsigned each = 2u * p.n_kv / unit_heads;   // units of a slot
        const int slot = static_cast<int>(unit / each);
        hv = static_cast<int>(unit - slot * each) * unit_heads;
        auto first_slot = [&](int b) { return (first_token(b) >> p.page_shift) + 2 * b; };
        const int b = last_at_most(p.n_seqs, slot, first_slot);
        if (b < 0) return;
        const int q0 = first_token(b), q1 = max(first_token(b + 1), q0);
        const int len = __ldg(p.kv_lens + b), n = q1 - q0;
        const int p0 = max(len - n, 0);          // position of the first token that has one
        const int page_i = (p0 >> p.page_shift) + (slot - first_slot(b));
        if (page_i < 0 || page_i > (p.max_len - 1) >> p.page_shift) return;
        pt.lo = max(p0, page_i << p.page_shift);
        // a position past the table's pages or the angles' table is left out
        pt.hi = min(min(len, p.max_len), (page_i << p.page_shift) + P);
        if (p.cos != nullptr) pt.hi = min(pt.hi, p.n_pos);
        if (pt.lo >= pt.hi) return;
        pt.t0 = q0 + (pt.lo - (len - n));
        page = __ldg(p.table + b * p.table_st + page_i);
      };
      if constexpr (UNIT_WARPS > 1) {
        // (the first of the unit's warps looks for all of them)
        __shared__ int4 found[kWarps / UNIT_WARPS];
        __shared__ int found_hv[kWarps / UNIT_WARPS];
        const int u = warp / UNIT_WARPS;
        if (part == 0) {
          look_up();
          if ((threadIdx.x & 31) == 0) found[u] = make_int4(pt.lo, pt.hi, pt.t0, page), found_hv[u] = hv;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + u), "n"(UNIT_WARPS * 32) : "memory");
        const int4 f = found[u];
        pt.lo = f.x, pt.hi = f.y, pt.t0 = f.z, page = f.w, hv = found_hv[u];
      } else {
        look_up();
      }
      if (page < 0 || page >= p.n_pages) return;
      const int h = hv < p.n_kv ? hv : hv - p.n_kv;
      const int64_t at = static_cast<int64_t>(page) * p.n_kv + h;
      if (hv < p.n_kv)
        append_codes<D, BF16, false, false, UNIT_WARPS>(p, pt, reinterpret_cast<const uint16_t*>(p.v) + h * p.v_sh, p.v_st, p.v_sh,
                                                 p.cv + page * p.cv_sp + h * p.cv_sh, p.cv_st, p.cv_sh, p.v_scale + at,
                                                 p.unit_heads, part, red + warp - part);
      else
        append_codes<D, BF16, ROT, NORM, UNIT_WARPS>(p, pt, reinterpret_cast<const uint16_t*>(p.k) + h * p.k_sh, p.k_st, p.k_sh,
                                               p.ck + page * p.ck_sp + h * p.ck_sh, p.ck_st, p.ck_sh, p.k_scale + at,
                                               p.unit_heads, part, red + warp - part);
      return;
    }
  }
  const unsigned w = (blockIdx.x - kv_blocks) * kWarps + warp;
  const int64_t tok = w / static_cast<unsigned>(parts);
  const int share = static_cast<int>(w % static_cast<unsigned>(parts));
  if (tok >= p.total) return;
  const int j = (threadIdx.x & 31) % (D / 8);
  const Lane at = lane_of(j, ROT ? p.rot : 0, p.interleaved);
  int b = -1, pos = -1;
  // the token's sequence and position; false: it is left out
  auto look_up = [&]() {
    b = last_at_most(p.n_seqs, static_cast<int>(tok), first_token);
    if (b < 0) return false;
    const int q0 = first_token(b), q1 = first_token(b + 1);
    if (tok >= q1) return false;   // behind the last sequence
    pos = __ldg(p.kv_lens + b) - (q1 - q0) + (static_cast<int>(tok) - q0);
    return pos >= 0 && pos < p.max_len && (p.cos == nullptr || pos < p.n_pos);
  };
  auto angles = [&](float4& c, float4& s) {
    c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ROT && at.rotated) {
      const int64_t o = static_cast<int64_t>(pos) * (p.rot / 2) + 4 * j;
      c = __ldg(reinterpret_cast<const float4*>(p.cos + o));
      s = __ldg(reinterpret_cast<const float4*>(p.sin + o));
    }
  };
  float4 c, s;
  const uint16_t* const q = reinterpret_cast<const uint16_t*>(p.q) + tok * p.q_st;
  uint8_t* const q_out = reinterpret_cast<uint8_t*>(p.q_out) + tok * p.qo_st * 2;
  const int qh0 = p.H * share / parts, qh1 = p.H * (share + 1) / parts;
  if (NORM && p.q_norm != nullptr) {
    bool there = false;
    norm_rows<D, BF16>(
        p.rot, p.interleaved, at,
        [&](float4& cc, float4& ss) {
          there = look_up();
          if (there) angles(cc, ss);
          return there;
        },
        q, p.q_sh, q_out, p.qo_sh * 2, p.q_norm, p.eps, qh0, qh1);
    if (!there) return;
  } else {
    if (!look_up()) return;
    angles(c, s);
    if (p.q != nullptr) token_rows<D, BF16, ROT>(p.interleaved, at, c, s, q, p.q_sh, q_out, p.qo_sh * 2, qh0, qh1);
  }
  if constexpr (!E4M3) {
    const int page = __ldg(p.table + b * p.table_st + (pos >> p.page_shift));
    if (page < 0 || page >= p.n_pages) return;
    const int row = pos & (P - 1), h0 = p.n_kv * share / parts, h1 = p.n_kv * (share + 1) / parts;
    const uint16_t* const k = reinterpret_cast<const uint16_t*>(p.k) + tok * p.k_st;
    uint8_t* const ck = p.ck + page * p.ck_sp + row * p.ck_st;
    if (NORM && p.k_norm != nullptr) {
      norm_rows<D, BF16>(
          p.rot, p.interleaved, at,
          [&](float4& cc, float4& ss) {
            angles(cc, ss);
            return true;
          },
          k, p.k_sh, ck, p.ck_sh, p.k_norm, p.eps, h0, h1);
    } else {
      if (NORM) angles(c, s);   // (the queries' norm did not leave them)
      token_rows<D, BF16, ROT>(p.interleaved, at, c, s, k, p.k_sh, ck, p.ck_sh, h0, h1);
    }
    // (plain copies: every lane takes eight elements that lie together)
    token_rows<D, BF16, false>(0, lane_of(j, 0, 0), c, s, reinterpret_cast<const uint16_t*>(p.v) + tok * p.v_st, p.v_sh,
                               p.cv + page * p.cv_sp + row * p.cv_st, p.cv_sh, h0, h1);
  }
}

// Warps a token: one, or several that share its heads where tokens are few.
inline int token_parts(long long total, int heads, int sms) {
  int parts = 1;
  while (parts < 16 && total * parts < 16LL * sms && parts * 2 <= heads) parts *= 2;
  return parts;
}

template <class K, class... A>
cudaError_t launch_pdl(K kern, long long blocks, cudaStream_t stream, const A&... args) {
  if (blocks > 0x7fffffffLL / kWarps) return cudaErrorInvalidValue;   // (units and warps are counted in 32 bits)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool BF16, bool E4M3, bool ROT, bool NORM, int UNIT_WARPS>
cudaError_t launch_one(sdpa_impl::AppendParams p, int sms, cudaStream_t stream) {
  long long kv_blocks = 0;
  p.unit_heads = 1;
  if (E4M3) {
    long long units = ((p.total >> p.page_shift) + 2LL * p.n_seqs) * 2 * p.n_kv;
    // (while they still fill the SMs twice over)
    while (UNIT_WARPS > 1 && p.unit_heads < kUnitHeads && p.n_kv % (2 * p.unit_heads) == 0 &&
           units * UNIT_WARPS / kWarps >= 8LL * sms)
      p.unit_heads *= 2, units /= 2;
    kv_blocks = (units + kWarps / UNIT_WARPS - 1) / (kWarps / UNIT_WARPS);
  }
  // Tokens' rows: a warp a token, or a share of its heads each where that
  // leaves SMs without work.
  const int parts = token_parts(p.total, p.H > p.n_kv ? p.H : p.n_kv, sms);
  const bool rows = !E4M3 || p.q != nullptr;
  const long long row_blocks = rows ? (static_cast<long long>(p.total) * parts + kWarps - 1) / kWarps : 0;
  return launch_pdl(append_kernel<D, BF16, E4M3, ROT, NORM, UNIT_WARPS>, kv_blocks + row_blocks, stream, p,
                    static_cast<int>(kv_blocks), parts);
}

template <int D, bool BF16, bool ROT, bool NORM>
cudaError_t launch_typed(const sdpa_impl::AppendParams& p, bool e4m3, int sms, cudaStream_t s) {
  if (!e4m3) return launch_one<D, BF16, false, ROT, NORM, 1>(p, sms, s);
  // as many warps a unit as hold its rows in registers (the most it can have:
  // a page's, or about a sequence's when those are fewer)
  const int P = 1 << p.page_shift, n = p.total / p.n_seqs, rows = P < n ? P : n;
  const int warp_rows = kBatch * 32 / (D / 8);
  if (rows <= warp_rows) return launch_one<D, BF16, true, ROT, NORM, 1>(p, sms, s);
  if (rows <= 2 * warp_rows) return launch_one<D, BF16, true, ROT, NORM, 2>(p, sms, s);
  if (rows <= 4 * warp_rows) return launch_one<D, BF16, true, ROT, NORM, 4>(p, sms, s);
  return launch_one<D, BF16, true, ROT, NORM, 8>(p, sms, s);
}

}  // namespace
