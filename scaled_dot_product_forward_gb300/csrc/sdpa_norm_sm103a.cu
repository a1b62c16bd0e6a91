// sdpa_norm_sm103a.cu -- the kernels with norms of head size 128.
#include "sdpa_norm.cuh"

namespace sdpa_impl {

cudaError_t launch_append_norm128(const AppendParams& p, bool bf16, bool e4m3, int sms, cudaStream_t stream) {
  return launch_append_norm<128>(p, bf16, e4m3, sms, stream);
}
cudaError_t launch_norm_rotate128(const RowsParams& p, bool bf16, int sms, cudaStream_t stream) {
  return bf16 ? launch_rows<128, true>(p, sms, stream) : launch_rows<128, false>(p, sms, stream);
}

}  // namespace sdpa_impl
