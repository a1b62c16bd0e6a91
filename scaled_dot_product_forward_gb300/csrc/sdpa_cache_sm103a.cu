// sdpa_cache_sm103a.cu -- the append's kernels without norms (sdpa_cache.cuh).
#include "sdpa_cache.cuh"

namespace {

template <int D, bool BF16>
cudaError_t launch_dim(const sdpa_impl::AppendParams& p, bool e4m3, int sms, cudaStream_t s) {
  if (p.cos != nullptr) return launch_typed<D, BF16, true, false>(p, e4m3, sms, s);
  return launch_typed<D, BF16, false, false>(p, e4m3, sms, s);
}

}  // namespace

namespace sdpa_impl {

cudaError_t launch_cache_append(const AppendParams& p, int head_dim, bool bf16, bool e4m3, int sms,
                                cudaStream_t stream) {
  if (p.q_norm != nullptr || p.k_norm != nullptr)
    return head_dim == 64 ? launch_append_norm64(p, bf16, e4m3, sms, stream) : launch_append_norm128(p, bf16, e4m3, sms, stream);
  if (head_dim == 64) return bf16 ? launch_dim<64, true>(p, e4m3, sms, stream) : launch_dim<64, false>(p, e4m3, sms, stream);
  return bf16 ? launch_dim<128, true>(p, e4m3, sms, stream) : launch_dim<128, false>(p, e4m3, sms, stream);
}

cudaError_t launch_norm_rotate(const RowsParams& p, int head_dim, bool bf16, int sms, cudaStream_t stream) {
  return head_dim == 64 ? launch_norm_rotate64(p, bf16, sms, stream) : launch_norm_rotate128(p, bf16, sms, stream);
}

}  // namespace sdpa_impl
