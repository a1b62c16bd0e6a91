// sdpa_paged.cuh -- what the paged-cache kernels share: the launch arguments,
// the division of a batch of uneven sequences into equal shares of key
// tiles, and small conversions.
//
// A unit is (sequence, key/value head, tile of query rows); row r of a
// sequence's nq * G rows for one key/value head is token r / G, query head
// h * G + r % G, so the G query heads that share the head's keys sit in one
// tile and its pages are read once for all of them.  A unit costs as many
// steps as its rows see tiles of kt keys (at least one, which writes the
// rows).  The units' steps, laid end to end, are cut into n equal ranges, one
// a CTA, whatever the lengths are: the host knows none of them, they stay on
// the device.  A range begins and ends inside a unit, so each CTA leaves at
// most two partial units (its first and its last), kept in the workspace as
// unnormalised rows with their maximum and sum and joined by a second small
// kernel, in the order of the CTAs: the result does not depend on timing.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa_paged {

using sdpa_impl::PagedParams;

__device__ __forceinline__ float clamp_scale(float s) {
  // fmaxf drops a NaN
  return fminf(fmaxf(s, __int_as_float((127 + sdpa_impl::kScaleMinExp) << 23)),
               __int_as_float((127 + sdpa_impl::kScaleMaxExp) << 23));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<__half2*>(&w));
}

struct Seq {
  int q0, nq, len, nt;
};

__device__ __forceinline__ Seq load_seq(const PagedParams& p, int b, int rt) {
  Seq s;
  int q1;
  if (p.cu != nullptr) {
    s.q0 = min(max(__ldg(p.cu + b), 0), p.total_q);
    q1 = min(max(__ldg(p.cu + b + 1), s.q0), p.total_q);
  } else {
    const int n = p.total_q / p.n_seqs;
    s.q0 = b * n;
    q1 = s.q0 + n;
  }
  s.nq = q1 - s.q0;
  s.len = min(max(__ldg(p.kv_lens + b), 0), p.max_len);
  const int rows = s.nq * p.G;
  s.nt = (rows > p.min_rows && rows <= p.max_rows) ? (rows + rt - 1) / rt : 0;
  return s;
}

// Keys that the rows of tile t see (the last row sees the most).
__device__ __forceinline__ int unit_keys(const PagedParams& p, const Seq& s, int t, int rt) {
  if (!p.is_causal) return s.len;
  const int last = (min((t + 1) * rt, s.nq * p.G) - 1) / p.G;
  return min(max(s.len - s.nq + last + 1, 0), s.len);
}
template <int KT>
__device__ __forceinline__ int unit_steps(const PagedParams& p, const Seq& s, int t, int rt) {
  return max((unit_keys(p, s, t, rt) + KT - 1) / KT, 1);
}
template <int KT>
__device__ __forceinline__ long long head_steps(const PagedParams& p, const Seq& s, int rt) {
  if (s.nt == 0) return 0;
  if (!p.is_causal) return static_cast<long long>(s.nt) * unit_steps<KT>(p, s, 0, rt);
  long long sum = 0;
  for (int t = 0; t < s.nt; ++t) sum += unit_steps<KT>(p, s, t, rt);
  return sum;
}

// A position in the division: unit (b, h, t), whose steps begin at u0.
struct Cursor {
  int b, h, t;
  long long u0;
  Seq s;
};

// Shared scratch of locate().
struct LocateScratch {
  long long warp_sum[16];
  long long total;
  int found_b;
  long long found_u0;
};

// Total steps of the batch; every thread of the block calls it.
template <int KT, int NT>
__device__ __forceinline__ long long batch_steps(const PagedParams& p, int rt, LocateScratch* sc) {
  long long sum = 0;
  for (int b = threadIdx.x; b < p.n_seqs; b += NT)
    sum += head_steps<KT>(p, load_seq(p, b, rt), rt);
  sum *= p.n_kv;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sc->warp_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) total += sc->warp_sum[w];
  return total;
}

// The unit that holds step v (v < the batch's total); every thread of the
// block calls it.
template <int KT, int NT>
__device__ __forceinline__ Cursor locate(const PagedParams& p, int rt, long long v,
                                         LocateScratch* sc) {
  long long base = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += NT) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    long long mine = 0;
    if (b < p.n_seqs) mine = head_steps<KT>(p, load_seq(p, b, rt), rt) * p.n_kv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (static_cast<int>(threadIdx.x & 31) >= o) incl += x;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 31) sc->warp_sum[threadIdx.x >> 5] = incl;
    __syncthreads();
    long long before = base, all = base;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < static_cast<int>(threadIdx.x >> 5)) before += sc->warp_sum[w];
      all += sc->warp_sum[w];
    }
    const long long u = before + incl - mine;
    if (mine > 0 && v >= u && v < u + mine) {
      sc->found_b = b;
      sc->found_u0 = u;
    }
    base = all;
    if (v < all) break;
  }
  __syncthreads();
  Cursor c;
  c.b = sc->found_b;
  c.s = load_seq(p, c.b, rt);
  const long long per_head = head_steps<KT>(p, c.s, rt);
  const long long off = v - sc->found_u0;
  c.h = static_cast<int>(off / per_head);
  c.u0 = sc->found_u0 + c.h * per_head;
  c.t = 0;
  while (true) {
    const int n = unit_steps<KT>(p, c.s, c.t, rt);
    if (v < c.u0 + n) break;
    c.u0 += n;
    ++c.t;
  }
  return c;
}

// The next unit (its steps begin where this one's end).
template <int KT>
__device__ __forceinline__ void advance(const PagedParams& p, int rt, Cursor& c) {
  c.u0 += unit_steps<KT>(p, c.s, c.t, rt);
  if (++c.t < c.s.nt) return;
  c.t = 0;
  if (++c.h < p.n_kv) return;
  c.h = 0;
  do {
    ++c.b;
    if (c.b >= p.n_seqs) return;
    c.s = load_seq(p, c.b, rt);
  } while (c.s.nt == 0);
}

// First step of range i of the n equal ones of `total` steps.
__device__ __forceinline__ long long range_start(long long total, int i, int n) {
  return total * i / n;
}

// Partial rows of slot s of CTA i.
template <int D>
__device__ __forceinline__ float* part_rows(const PagedParams& p, int i, int slot, int rt) {
  return p.part + (static_cast<int64_t>(i) * 2 + slot) * rt * (D + 2);
}

}  // namespace sdpa_paged
