// sdpa_norm.cuh -- query and key heads normalised and rotated without a cache, and
// how the kernels with norms are launched.
#pragma once
#include "sdpa_cache.cuh"

namespace {

// As token_rows, two rows a lane at a time with the next ones on their way: 32768
// rows of 32 heads of 128 85 us, 103 with four and none (in the append, behind
// the look at the sequences, the four are ahead, 128 against 130).
template <int D, bool BF16>
__device__ __forceinline__ void turned_rows(int interleaved, const Lane& at, const float4& c, const float4& s,
                                            const uint16_t* src, int64_t src_sh, uint8_t* dst, int64_t dst_sh_bytes, int h0,
                                            int h1) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kTwo = 2;
  int h = h0 + static_cast<int>(threadIdx.x & 31) / kLanes;
  src += h * src_sh;
  dst += h * dst_sh_bytes;
  const int64_t src_step = kRows * src_sh, dst_step = kRows * dst_sh_bytes;
  float x[kTwo][8], next[kTwo][8];
  auto ask = [&](int from) {
#pragma unroll
    for (int u = 0; u < kTwo; ++u) {
      if (from + u * kRows < h1) load8<BF16>(src, at, next[u]);
      src += src_step;
    }
  };
  ask(h);
#pragma unroll 1
  for (; h < h1; h += kTwo * kRows) {
#pragma unroll
    for (int u = 0; u < kTwo; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = next[u][e];
    ask(h + kTwo * kRows);
#pragma unroll
    for (int u = 0; u < kTwo; ++u) {
      if (h + u * kRows < h1) {
        if (at.rotated) rotate8(x[u], c, s, interleaved);
        store8<BF16>(reinterpret_cast<uint16_t*>(dst), at, x[u]);
      }
      dst += dst_step;
    }
  }
}

// Rows without a cache: a warp takes a share (1 / 2^parts_shift) of one token's query
// and key heads.  Bound by its instructions and by latency together: a warp's life
// is a few trips to memory (positions, angles, rows), a third of its instructions
// are its own token's.  17700 rows of 16 + 16 heads of 64, fp16, 32 of 64 rotated: 26
// us, 5.6 TB/s of the rows' bytes; a kernel for each form of rotation (27.7 with one).
template <int D, bool BF16, bool PAIRED, bool ALL>
__global__ void __launch_bounds__(kThreads, kPerSm)
    norm_rotate_kernel(const __grid_constant__ sdpa_impl::RowsParams p, int parts_shift) {
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t tok = w >> parts_shift;
  const int share = static_cast<int>(w & ((1u << parts_shift) - 1u));
  if (tok >= p.total) return;
  const int j = (threadIdx.x & 31) % (D / 8);
  const Lane at = lane_of(j, ALL ? D : p.rot, PAIRED);
  // the row's position (before: none yet), and its angles; false: it is left out
  int pos = -1;
  auto angles = [&](float4& c, float4& s) {
    c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.rot == 0) return true;
    if (pos < 0) pos = p.positions != nullptr ? __ldg(p.positions + tok) : static_cast<int>(tok);
    if (pos < 0 || pos >= p.n_pos) return false;
    if (at.rotated) {
      const int64_t o = static_cast<int64_t>(pos) * (p.rot / 2) + 4 * j;
      c = __ldg(reinterpret_cast<const float4*>(p.cos + o));
      s = __ldg(reinterpret_cast<const float4*>(p.sin + o));
    }
    return true;
  };
  auto rows = [&](const void* x, int64_t st, int64_t sh, void* out, int64_t ost, int64_t osh, const float* weight, int heads) {
    const uint16_t* const from = reinterpret_cast<const uint16_t*>(x) + tok * st;
    uint8_t* const to = reinterpret_cast<uint8_t*>(out) + tok * ost * 2;
    const int h0 = (heads * share) >> parts_shift, h1 = (heads * (share + 1)) >> parts_shift;
    bool there = true;
    if (weight != nullptr) {
      norm_rows_as<D, BF16, PAIRED, ALL>(
          at, [&](float4& c, float4& s) { return there = angles(c, s); }, from, sh, to, osh * 2, weight, p.eps, h0, h1);
    } else {
      float4 c, s;
      there = angles(c, s);
      if (there) turned_rows<D, BF16>(PAIRED, at, c, s, from, sh, to, osh * 2, h0, h1);
    }
    return there;
  };
  if (rows(p.q, p.q_st, p.q_sh, p.q_out, p.qo_st, p.qo_sh, p.q_norm, p.H) && p.k != nullptr)
    rows(p.k, p.k_st, p.k_sh, p.k_out, p.ko_st, p.ko_sh, p.k_norm, p.n_kv);
}

template <int D, bool BF16>
cudaError_t launch_rows(const sdpa_impl::RowsParams& p, int sms, cudaStream_t stream) {
  const int parts = token_parts(p.total, p.H > p.n_kv ? p.H : p.n_kv, sms);
  int shift = 0;
  while ((1 << shift) < parts) ++shift;
  const long long blocks = (static_cast<long long>(p.total) * parts + kWarps - 1) / kWarps;
  const bool all = p.rot == D;
  if (p.interleaved)
    return all ? launch_pdl(norm_rotate_kernel<D, BF16, true, true>, blocks, stream, p, shift)
               : launch_pdl(norm_rotate_kernel<D, BF16, true, false>, blocks, stream, p, shift);
  return all ? launch_pdl(norm_rotate_kernel<D, BF16, false, true>, blocks, stream, p, shift)
             : launch_pdl(norm_rotate_kernel<D, BF16, false, false>, blocks, stream, p, shift);
}

// (There is one form for rotated rows and others: rot = 0.)
template <int D>
cudaError_t launch_append_norm(const sdpa_impl::AppendParams& p, bool bf16, bool e4m3, int sms, cudaStream_t s) {
  return bf16 ? launch_typed<D, true, true, true>(p, e4m3, sms, s) : launch_typed<D, false, true, true>(p, e4m3, sms, s);
}

}  // namespace
