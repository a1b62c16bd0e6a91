// sdpa_paged.cuh -- what the paged-cache kernels share: the launch arguments,
// the division of a batch of uneven sequences into equal shares of key
// tiles, and small conversions.
//
// A unit is (sequence, group of key/value heads, tile of query rows); row r of
// a sequence's nq * G rows for one key/value head is token r / G, query head
// h * G + r % G, so the G query heads that share the head's keys sit in one
// tile and its pages are read once for all of them.  A unit costs as many
// steps as its rows see runs of 2^step_shift keys (at least one, which writes
// the rows).  The units' steps, laid end to end, are cut into n equal ranges, one
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

// Where a row's weights 2^(exponent - base) lie.  The base follows the running
// maximum of the exponents: it is moved when one exceeds it by kRoom, to kTop
// below that one.  bf16 weights reach from 1 (or, until the next move, 2^8) down
// to 2^-126.  fp16 ones end at 2^-24: a base kTop below the maximum leaves each
// weight an error of at most 2^-(25 + kTop) of the row's largest, whatever that
// one's value is (many small weights beside one large one, whose value may be
// zero, add up), and kRoom keeps the largest at 2^15.
template <bool BF16>
struct WeightRange {
  static constexpr float kTop = BF16 ? 0.0f : 11.0f;
  static constexpr float kRoom = BF16 ? 8.0f : 15.0f;
};

// n / G for 0 <= n < 2^31 (the quotients of a unit's rows are wanted in many
// places, whose code would be a division's each).
__device__ __forceinline__ int by_G(const PagedParams& p, int n) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * p.g_mul) >> p.g_shift);
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
    s.q0 = b * p.seq_q;
    q1 = s.q0 + p.seq_q;
  }
  s.nq = q1 - s.q0;
  s.len = min(max(__ldg(p.kv_lens + b), 0), p.max_len);
  s.nt = (s.nq * p.G + rt - 1) / rt;
  return s;
}

// Keys that the rows of tile t see (the last row sees the most).
__device__ __forceinline__ int unit_keys(const PagedParams& p, const Seq& s, int t, int rt) {
  if (!p.is_causal) return s.len;
  const int last = by_G(p, min((t + 1) * rt, s.nq * p.G) - 1);
  return min(max(s.len - s.nq + last + 1, 0), s.len);
}
// With a window (WIN, causal): first key of the window of tile t's first row, which
// reaches back the farthest.  The unit's rows see no key between the sinks and it.
__device__ __forceinline__ int unit_from(const PagedParams& p, const Seq& s, int t, int rt) {
  const int seen = min(max(s.len - s.nq + by_G(p, t * rt) + 1, 0), s.len);
  return max(seen - p.window, 0);
}
// Steps without a key that the unit's rows see, between the sinks' steps and the
// window's: step s of the unit stands for run step_run(..) of its keys.
template <bool WIN>
__device__ __forceinline__ int unit_skip(const PagedParams& p, const Seq& s, int t, int rt) {
  if constexpr (!WIN) return 0;
  return max((unit_from(p, s, t, rt) >> p.step_shift) - p.sink_steps, 0);
}
template <bool WIN>
__device__ __forceinline__ int step_run(const PagedParams& p, int skip, int s) {
  if constexpr (!WIN) return s;
  return s < p.sink_steps ? s : s + skip;
}
template <bool WIN>
__device__ __forceinline__ int unit_steps(const PagedParams& p, const Seq& s, int t, int rt) {
  return max(((unit_keys(p, s, t, rt) + (1 << p.step_shift) - 1) >> p.step_shift) - unit_skip<WIN>(p, s, t, rt), 1);
}

// A position in the division: unit (b, h, t) (h: the group of heads), whose
// steps begin at u0.  (The host has checked that all steps fit 31 bits.)
struct Cursor {
  int b, h, t, u0;
  Seq s;
};

// Shared scratch of divide().
struct DivideScratch {
  int warp_sum[16];
  int found_b, found_u0, found_steps;
  Seq found;
};

// Ranges of a division: at most one a CTA, and at most one for p.min_steps steps
// or what is left of them (joining many short pieces costs more than it saves;
// being equal, ranges of a few steps in all may have fewer, never none).
__device__ __forceinline__ int range_count(const PagedParams& p, int total) {
  return min((total + p.min_steps - 1) >> p.min_steps_shift, p.n_ctas);
}
// First step of range i of the n equal ones of `total` steps.
__device__ __forceinline__ int range_start(int total, int i, int n) {
  const int q = total / n;
  return q * i + (total - q * n) * i / n;   // (both factors below n)
}

// The batch's total of steps, and the unit that holds step `at(total)` when
// that is below the total (returns it; -1 otherwise).  Every thread of the
// block calls it.  A group of W lanes adds up a sequence's units, as many
// sequences at a time as the block has groups; a batch of at most that many is
// read once.
template <int NT, bool WIN, class At>
__device__ __forceinline__ int divide(const PagedParams& p, int rt, DivideScratch* sc, At&& at, int& total,
                                      Cursor& c) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  int w_shift = 0;
  if (p.is_causal && p.max_rows > rt)   // (else a sequence has one unit a group)
    while (w_shift < 5 && p.n_seqs * (2 << w_shift) <= NT) ++w_shift;
  const int w = 1 << w_shift, per = NT >> w_shift, sub = tid & (w - 1);
  // this thread's part of sequence b0 + tid / w; inclusive sum over the block
  // of the sequences' steps, at each group's first lane
  int mine, incl, all;
  Seq seq{};
  auto chunk = [&](int b0) {
    const int b = b0 + (tid >> w_shift);
    mine = 0;
    if (b < p.n_seqs) {
      seq = load_seq(p, b, rt);
      if (!p.is_causal)
        mine = seq.nt == 0 ? 0 : seq.nt * unit_steps<WIN>(p, seq, 0, rt);
      else
#pragma unroll 1
        for (int t = sub; t < seq.nt; t += w) mine += unit_steps<WIN>(p, seq, t, rt);
    }
    for (int o = 1; o < w; o <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    incl = sub == 0 ? mine * p.n_groups : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sc->warp_sum[warp] = incl;
    __syncthreads();
    // each lane one warp's sum
    const int ws = lane < NT / 32 ? sc->warp_sum[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, ws);
    incl += __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
  };
  total = 0;
  const int chunks = (p.n_seqs + per - 1) / per;
  for (int k = 0; k < chunks; ++k) {
    chunk(k * per);
    total += all;
  }
  const int v = at(total);
  if (v >= total) return -1;
  int base = 0;
  for (int k = 0; k < chunks; ++k) {
    if (chunks > 1) chunk(k * per);
    const int u1 = base + incl, u0 = u1 - mine * p.n_groups;
    if (sub == 0 && mine > 0 && v >= u0 && v < u1) {
      sc->found_b = k * per + (tid >> w_shift);
      sc->found_u0 = u0;
      sc->found_steps = mine;
      sc->found = seq;
    }
    base += all;
    if (v < base) break;
  }
  __syncthreads();
  c.b = sc->found_b;
  c.s = sc->found;
  c.h = (v - sc->found_u0) / sc->found_steps;
  c.u0 = sc->found_u0 + c.h * sc->found_steps;
  c.t = 0;
#pragma unroll 1
  while (c.s.nt > 1) {
    const int n = c.t + lane < c.s.nt ? unit_steps<WIN>(p, c.s, c.t + lane, rt) : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, v < c.u0 + sum);
    if (hit != 0 || c.t + 32 >= c.s.nt) {
      const int k = hit != 0 ? __ffs(static_cast<int>(hit)) - 1 : 31;
      c.t += k;
      c.u0 += __shfl_sync(0xffffffffu, sum - n, k);
      break;
    }
    c.t += 32;
    c.u0 += __shfl_sync(0xffffffffu, sum, 31);
  }
  return v;
}

// The next unit (its steps begin where this one's end).
template <bool WIN>
__device__ __forceinline__ void advance(const PagedParams& p, int rt, Cursor& c) {
  c.u0 += unit_steps<WIN>(p, c.s, c.t, rt);
  if (++c.t < c.s.nt) return;
  c.t = 0;
  if (++c.h < p.n_groups) return;
  c.h = 0;
  do {
    ++c.b;
    if (c.b >= p.n_seqs) return;
    c.s = load_seq(p, c.b, rt);
  } while (c.s.nt == 0);
}

// The workspace: what to join, a note of each CTA's, then the partial units,
// two a CTA: rt rows a head of D sums, behind them the rows' maxima and sums (so
// that a row begins where a sector does).
struct JoinNote {
  int pieces;        // 0: no unit begins in this CTA's range and ends behind it
  int slot;          // of its piece here; the following CTAs' pieces are their first
  int rows, row0;    // the unit's rows a head, the first one's number in the sequence
  int q0, kv_head0;  // the sequence's first row of q, the unit's first key/value head
  int heads;         // key/value heads of a unit
  int unused;
};
static_assert(sizeof(JoinNote) == sdpa_impl::kJoinNoteBytes, "workspace layout");

template <int D>
__device__ __forceinline__ float* part_rows(const PagedParams& p, int i, int slot, int rt) {
  return p.part + static_cast<int64_t>(p.n_ctas) * (sizeof(JoinNote) / 4) +
         (static_cast<int64_t>(i) * 2 + slot) * p.unit_heads * rt * (D + 2);
}
// Of the piece at `rows`: row hr's maximum and sum.
template <int D>
__device__ __forceinline__ float2* part_sums(float* rows, int heads, int rt, int hr) {
  return reinterpret_cast<float2*>(rows + heads * rt * D) + hr;
}

// CTA i's note: its last unit, if that begins here (with its first or a later
// segment) and goes on behind its range.
template <bool WIN>
__device__ __forceinline__ void leave_note(const PagedParams& p, int i, int total, int n, int rt,
                                           const Cursor& c, int s0, int s1, bool first) {
  JoinNote j{};
  const int steps = unit_steps<WIN>(p, c.s, c.t, rt);
  if (s0 == 0 && s1 < steps) {
    // the range that holds the unit's last step
    const long long last = (static_cast<long long>(c.u0 + steps) * n - 1) / total;
    j.pieces = static_cast<int>(last) - i + 1;
    j.slot = first ? 0 : 1;
    j.rows = min(rt, c.s.nq * p.G - c.t * rt);
    j.row0 = c.t * rt;
    j.q0 = c.s.q0;
    j.kv_head0 = c.h * p.unit_heads;
    j.heads = p.unit_heads;
  }
  reinterpret_cast<JoinNote*>(p.part)[i] = j;
}

}  // namespace sdpa_paged
