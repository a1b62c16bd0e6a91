// sdpa_cache_sm103a.cu -- appending new tokens' keys and values to a paged
// cache, rotated by their positions, for sm_103a.
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
// Bound by memory: each new row is read once and written once.  A block takes
// one page's new tokens (one sequence) and a share of the heads, so the
// scale of a (page, head) has one owner, a warp, and needs no atomics; lane
// j of a row's D / 8 holds pairs 4j .. 4j + 3, both halves of each, so the
// rotation needs no exchange either.
#include <cuda_fp8.h>

#include "sdpa_paged.cuh"

using namespace sdpa_dev;
using namespace sdpa_paged;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

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

template <bool BF16>
__device__ __forceinline__ void load8(const uint16_t* row, const Lane& l, float (&x)[8]) {
  // (plain loads: the queries may be rotated in place)
  const uint2 a = *reinterpret_cast<const uint2*>(row + l.ea);
  const uint2 b = *reinterpret_cast<const uint2*>(row + l.eb);
  const float2 f0 = unpack2<BF16>(a.x), f1 = unpack2<BF16>(a.y);
  const float2 f2 = unpack2<BF16>(b.x), f3 = unpack2<BF16>(b.y);
  x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
  x[4] = f2.x, x[5] = f2.y, x[6] = f3.x, x[7] = f3.y;
}

template <bool BF16>
__device__ __forceinline__ void store8(uint16_t* row, const Lane& l, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(row + l.ea) =
      make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
  *reinterpret_cast<uint2*>(row + l.eb) =
      make_uint2(pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
}

__device__ __forceinline__ void turn(float& x1, float& x2, float c, float s) {
  const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  const float y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = y1;
  x2 = y2;
}

__device__ __forceinline__ void rotate8(float (&x)[8], const float4& c, const float4& s,
                                        int interleaved) {
  if (interleaved) {
    turn(x[0], x[1], c.x, s.x);
    turn(x[2], x[3], c.y, s.y);
    turn(x[4], x[5], c.z, s.z);
    turn(x[6], x[7], c.w, s.w);
  } else {
    turn(x[0], x[4], c.x, s.x);
    turn(x[1], x[5], c.y, s.y);
    turn(x[2], x[6], c.z, s.z);
    turn(x[3], x[7], c.w, s.w);
  }
}

// The page's new tokens: positions [lo, hi), the first being row t0 of k, v, q.
struct PageTokens {
  int lo, hi, t0;
  int page;       // -1: the table has no page here (its rows are not written)
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

// The largest |x| that a scale has to cover: infinities and NaN are left out
// (an infinity is stored as +-448 codes, a NaN as NaN).
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}

// The least power of two s with amax <= 448 s = 1.75 * 2^8 s, in range.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, sdpa_impl::kScaleMinExp), sdpa_impl::kScaleMaxExp);
  return __int_as_float((e + 127) << 23);
}

// One warp: the page's new rows of one head, quantised under the page's scale.
template <int D, bool BF16, bool ROT>
__device__ __forceinline__ void append_codes(const sdpa_impl::AppendParams& p, const PageTokens& pt,
                                             const uint16_t* src, int64_t src_st, uint8_t* dst,
                                             int64_t dst_st, float* scale_at) {
  constexpr int kLanes = D / 8;       // lanes a row
  constexpr int kRows = 32 / kLanes;  // rows a step
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int rot = ROT ? p.rot : 0;
  const Lane at = lane_of(j, rot, p.interleaved);
  const int n = pt.hi - pt.lo;
  auto row_values = [&](int r, float (&x)[8]) {
    load8<BF16>(src + static_cast<int64_t>(pt.t0 + r) * src_st, at, x);
    if (ROT && at.rotated) {
      const int64_t o = static_cast<int64_t>(pt.lo + r) * (rot / 2) + 4 * j;
      const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + o));
      const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + o));
      rotate8(x, c, s, p.interleaved);
    }
  };
  float amax = 0.0f;
#pragma unroll 4
  for (int r = sub; r < n; r += kRows) {
    float x[8];
    row_values(r, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(x[e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int row0 = pt.lo & ((1 << p.page_shift) - 1);
  float scale = scale_for(amax);
  if (row0 > 0) {
    const float old = clamp_scale(*scale_at);
    if (scale > old) {
      // raise the scale: the page's earlier codes of this head
      const float ratio = old / scale;
      for (int i = lane; i < row0 * (D / 16); i += 32) {
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
  __syncwarp();
  if (lane == 0) *scale_at = scale;
  const float inv = 1.0f / scale;
#pragma unroll 4
  for (int r = sub; r < n; r += kRows) {
    float x[8];
    row_values(r, x);
    uint8_t* row = dst + (row0 + r) * dst_st;
    *reinterpret_cast<uint32_t*>(row + at.ea) =
        codes4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    *reinterpret_cast<uint32_t*>(row + at.eb) =
        codes4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
  }
}

// One warp: heads [h0, h1) of one token, rotated (ROT) or copied, in steps of
// four rows a lane group so that the token's angles are read once for them.
template <int D, bool BF16, bool ROT>
__device__ __forceinline__ void token_rows(const sdpa_impl::AppendParams& p, int pos,
                                           const uint16_t* src, int64_t src_sh, uint8_t* dst,
                                           int64_t dst_sh_bytes, int h0, int h1) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int rot = ROT ? p.rot : 0;
  const Lane at = lane_of(j, rot, p.interleaved);
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ROT && at.rotated) {
    const int64_t o = static_cast<int64_t>(pos) * (rot / 2) + 4 * j;
    c = __ldg(reinterpret_cast<const float4*>(p.cos + o));
    s = __ldg(reinterpret_cast<const float4*>(p.sin + o));
  }
  float x[4][8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int h = h0 + sub + u * kRows;
    if (h < h1) load8<BF16>(src + h * src_sh, at, x[u]);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int h = h0 + sub + u * kRows;
    if (h < h1) {
      if (ROT && at.rotated) rotate8(x[u], c, s, p.interleaved);
      store8<BF16>(reinterpret_cast<uint16_t*>(dst + h * dst_sh_bytes), at, x[u]);
    }
  }
}

// grid.x: slots of (sequence, page with new tokens); sequence b has the slots
// [f(b), f(b+1)), f(b) = cu[b] / P + 2 b, which is at least the pages its new
// tokens can touch, so a slot finds its sequence without a prefix sum over
// lengths.  grid.y: shares of the heads.
template <int D, bool BF16, bool E4M3, bool ROT>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const __grid_constant__ sdpa_impl::AppendParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int P = 1 << p.page_shift;
  const int slot = static_cast<int>(blockIdx.x);
  const int uniform = p.total / p.n_seqs;
  auto first_token = [&](int b) {
    return p.cu != nullptr ? min(max(__ldg(p.cu + b), 0), p.total) : b * uniform;
  };
  auto first_slot = [&](int b) { return (first_token(b) >> p.page_shift) + 2 * b; };
  int b = -1;
  for (int b0 = 0; b0 < p.n_seqs; b0 += kThreads) {
    const int i = b0 + static_cast<int>(threadIdx.x);
    const int c = __syncthreads_count(i < p.n_seqs && first_slot(i) <= slot);
    b += c;
    if (c < kThreads) break;
  }
  if (b < 0) return;
  const int q0 = first_token(b), q1 = max(first_token(b + 1), q0);
  const int len = __ldg(p.kv_lens + b), n = q1 - q0;
  const int p0 = max(len - n, 0);          // position of the first token that has one
  const int page_i = (p0 >> p.page_shift) + (slot - first_slot(b));
  PageTokens pt;
  pt.lo = max(p0, page_i << p.page_shift);
  // a position past the table's pages or the angles' table is left out
  pt.hi = min(min(len, p.max_len), (page_i << p.page_shift) + P);
  if (p.cos != nullptr) pt.hi = min(pt.hi, p.n_pos);
  if (pt.lo >= pt.hi) return;
  pt.t0 = q0 + (pt.lo - (len - n));
  pt.page = __ldg(p.table + b * p.table_st + page_i);
  if (pt.page < 0 || pt.page >= p.n_pages) pt.page = -1;

  const int y = static_cast<int>(blockIdx.y), Y = static_cast<int>(gridDim.y);
  const int kv0 = p.n_kv * y / Y, kv1 = p.n_kv * (y + 1) / Y, n_kv = kv1 - kv0;
  const int hq0 = p.q != nullptr ? p.H * y / Y : 0, hq1 = p.q != nullptr ? p.H * (y + 1) / Y : 0;
  const int tokens = pt.hi - pt.lo;
  const int row0 = pt.lo & (P - 1);
  const int warp = threadIdx.x >> 5;
  constexpr int kGroup = 4 * (32 / (D / 8));  // heads a warp takes of a token
  const int q_units = ((hq1 - hq0 + kGroup - 1) / kGroup) * tokens;
  const int kv_groups = (n_kv + kGroup - 1) / kGroup;
  const int kv_units = pt.page < 0 ? 0 : (E4M3 ? 2 * n_kv : 2 * kv_groups * tokens);
  for (int u = warp; u < kv_units + q_units; u += kWarps) {
    if (u < kv_units) {
      if constexpr (E4M3) {
        const int h = kv0 + (u >> 1);
        float* scale_at = ((u & 1) ? p.v_scale : p.k_scale) + static_cast<int64_t>(pt.page) * p.n_kv + h;
        if (u & 1)
          append_codes<D, BF16, false>(p, pt, reinterpret_cast<const uint16_t*>(p.v) + h * p.v_sh,
                                       p.v_st, p.cv + pt.page * p.cv_sp + h * p.cv_sh, p.cv_st,
                                       scale_at);
        else
          append_codes<D, BF16, ROT>(p, pt, reinterpret_cast<const uint16_t*>(p.k) + h * p.k_sh,
                                     p.k_st, p.ck + pt.page * p.ck_sp + h * p.ck_sh, p.ck_st,
                                     scale_at);
      } else {
        const int r = u / (2 * kv_groups), g = u - r * 2 * kv_groups;
        const int64_t tok = pt.t0 + r;
        const int h0 = kv0 + (g >> 1) * kGroup, h1 = min(h0 + kGroup, kv1);
        if (g & 1)
          token_rows<D, BF16, false>(p, pt.lo + r, reinterpret_cast<const uint16_t*>(p.v) + tok * p.v_st,
                                     p.v_sh, p.cv + pt.page * p.cv_sp + (row0 + r) * p.cv_st, p.cv_sh,
                                     h0, h1);
        else
          token_rows<D, BF16, ROT>(p, pt.lo + r, reinterpret_cast<const uint16_t*>(p.k) + tok * p.k_st,
                                   p.k_sh, p.ck + pt.page * p.ck_sp + (row0 + r) * p.ck_st, p.ck_sh,
                                   h0, h1);
      }
    } else {
      const int groups = (hq1 - hq0 + kGroup - 1) / kGroup;
      const int w = u - kv_units, r = w / groups, g = w - r * groups;
      const int64_t tok = pt.t0 + r;
      const int h0 = hq0 + g * kGroup, h1 = min(h0 + kGroup, hq1);
      token_rows<D, BF16, ROT>(p, pt.lo + r, reinterpret_cast<const uint16_t*>(p.q) + tok * p.q_st, p.q_sh,
                               reinterpret_cast<uint8_t*>(p.q_out) + tok * p.qo_st * 2, p.qo_sh * 2, h0,
                               h1);
    }
  }
}

template <int D, bool BF16, bool E4M3, bool ROT>
cudaError_t launch_one(const sdpa_impl::AppendParams& p, int sms, cudaStream_t stream) {
  const long long slots = (p.total >> p.page_shift) + 2LL * p.n_seqs;
  // enough blocks for about twelve an SM, by sharing out the heads
  long long y = (12LL * sms + slots - 1) / slots;
  y = y < p.n_kv ? y : p.n_kv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(slots), static_cast<unsigned>(y));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<D, BF16, E4M3, ROT>, p);
}

template <int D, bool BF16>
cudaError_t launch_typed(const sdpa_impl::AppendParams& p, bool e4m3, int sms, cudaStream_t s) {
  if (e4m3)
    return p.cos ? launch_one<D, BF16, true, true>(p, sms, s) : launch_one<D, BF16, true, false>(p, sms, s);
  return p.cos ? launch_one<D, BF16, false, true>(p, sms, s) : launch_one<D, BF16, false, false>(p, sms, s);
}

}  // namespace

namespace sdpa_impl {

cudaError_t launch_cache_append(const AppendParams& p, int head_dim, bool bf16, bool e4m3, int sms,
                                cudaStream_t stream) {
  if (head_dim == 64)
    return bf16 ? launch_typed<64, true>(p, e4m3, sms, stream) : launch_typed<64, false>(p, e4m3, sms, stream);
  return bf16 ? launch_typed<128, true>(p, e4m3, sms, stream) : launch_typed<128, false>(p, e4m3, sms, stream);
}

}  // namespace sdpa_impl
