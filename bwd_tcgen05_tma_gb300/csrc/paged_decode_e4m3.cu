// Few-row attention over a paged E4M3 cache.
#include "paged_decode.cuh"

namespace attn {
namespace paged {

cudaError_t launch_decode_e4m3(const Args& a, int rows, int sms, cudaStream_t st) {
  return launch_dims<kCacheE4m3>(a, rows, sms, st);
}

}  // namespace paged
}  // namespace attn
