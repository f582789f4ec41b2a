// Shared by the kernels of the paged latent cache: the device view of one call.
#pragma once
#include "rotate.cuh"

namespace attn {
namespace paged {

// The part that sequences, tables and pages need is that of the paged cache with
// one KV head: `kc` is the cache, `group` the query heads.
struct LatentArgs {
  Args a;
  int d_c;
  int pair;  // attention: blocks work in pairs on row blocks of twice the rows (0 or 1)
  uint64_t wait_ns;  // attention: limit of the waits that may last for whole pieces
  const uint16_t* c_new;
  const uint16_t* k_rope;
  const uint16_t* q_rope;
  const uint16_t* q_lat;
  uint16_t* q_rot;
  // strides in elements, of tokens and of heads
  int64_t c_new_stride, k_rope_stride;
  int64_t q_rope_tok, q_rope_head, q_lat_tok, q_lat_head, q_rot_tok, q_rot_head;
};

constexpr int kLatentRope = 64;  // width of the rotated part

// Rows (tokens x heads) the attention's kernel takes at once, and its blocks.
constexpr int kLatentMaxCtas = 152;
inline int latent_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
// Tensor map over the cache, [page][64 coordinates][slot][coordinate]: boxes of
// `slots` slots and `chunks` times 64 coordinates, 128-byte swizzle.
bool latent_map(CUtensorMap* m, const LatentArgs& l, int slots, int chunks);

cudaError_t launch_latent_append(const LatentArgs& a, cudaStream_t st);
cudaError_t launch_latent_bf16(const LatentArgs& a, int rows, int sms, cudaStream_t st);
cudaError_t launch_latent_f16(const LatentArgs& a, int rows, int sms, cudaStream_t st);

}  // namespace paged
}  // namespace attn
