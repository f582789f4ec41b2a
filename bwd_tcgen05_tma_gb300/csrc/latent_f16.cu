// Attention over a paged latent cache of fp16 rows.
#include "latent_attend.cuh"

namespace attn {
namespace paged {

cudaError_t launch_latent_f16(const LatentArgs& l, int rows, int sms, cudaStream_t st) {
  return launch_latent<true>(l, rows, sms, st);
}

}  // namespace paged
}  // namespace attn
