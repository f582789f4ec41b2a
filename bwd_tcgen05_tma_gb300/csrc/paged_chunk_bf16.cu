// Many-row attention over a paged bf16 cache.
#include "paged_chunk.cuh"

namespace attn {
namespace paged {

cudaError_t launch_chunk_bf16(const Args& a, int sms, cudaStream_t st) {
  return chunk_dims<kCacheBf16>(a, sms, st);
}

}  // namespace paged
}  // namespace attn
