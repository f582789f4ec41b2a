// Many-row attention over a paged fp16 cache.
#include "paged_chunk.cuh"

namespace attn {
namespace paged {

cudaError_t launch_chunk_f16(const Args& a, int sms, cudaStream_t st) {
  return chunk_dims<kCacheF16>(a, sms, st);
}

}  // namespace paged
}  // namespace attn
