// Few-row attention over a paged fp16 cache.
#include "paged_decode.cuh"

namespace attn {
namespace paged {

cudaError_t launch_decode_f16(const Args& a, int rows, int sms, cudaStream_t st) {
  return launch_dims<kCacheF16>(a, rows, sms, st);
}

}  // namespace paged
}  // namespace attn
