// Many-row attention over a paged E4M3 cache.
#include "paged_chunk.cuh"

namespace attn {
namespace paged {

cudaError_t launch_chunk_e4m3(const Args& a, int sms, cudaStream_t st) {
  return chunk_dims<kCacheE4m3>(a, sms, st);
}

}  // namespace paged
}  // namespace attn
