// Appending new tokens to the paged latent cache.
//
// One warp a job: a token's cache row (its latent vector copied, its rotated
// part behind it) and the rotated parts of its first sixteen query heads, or of the
// next sixteen.  A row is
// 16-byte units side by side, so a warp's accesses are whole lines, and all of a
// job's loads are on their way before the token's place is known.  Bound by HBM
// for prompts (17349 tokens, 16 heads, 98 MB: 18.0 us, 5.4 TB/s); for single tokens by
// the launch and the chain of reads lengths -> table -> store (64 tokens: 2.4 us in a
// graph, 3.9 as the host launches them).
#include "latent.cuh"

namespace attn {
namespace paged {
namespace {

constexpr int kWarps = 4;
constexpr int kUnits = kLatentRope / 8;  // 16-byte units of the rotated part
constexpr int kHeadsJob = 16, kPer = 32 / kUnits;

// Unit u of a rotated part, turned: a lane each.  (Halves: the other of each pair
// is kUnits / 2 lanes away.)
__device__ __forceinline__ uint4 turn_unit(uint4 v, int u, const float* cos, const float* sin,
                                           int interleaved, int f16) {
  float x[8];
  unpack8(v, x, f16);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn_pair(x[2 * i], x[2 * i + 1], cos[i], sin[i]);
  } else {
    const bool second = u >= kUnits / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __shfl_xor_sync(0xffffffffu, x[i], kUnits / 2);
      float p = second ? y : x[i], q = second ? x[i] : y;
      turn_pair(p, q, cos[i], sin[i]);
      x[i] = second ? q : p;
    }
  }
  return make_uint4(pack2(x[0], x[1], f16), pack2(x[2], x[3], f16), pack2(x[4], x[5], f16),
                    pack2(x[6], x[7], f16));
}

template <int kC>  // 16-byte units of the latent vector a lane
__global__ void __launch_bounds__(kWarps * 32)
    latent_append_kernel(const __grid_constant__ LatentArgs l, int jobs_token) {
  sm103::grid_dep_wait();
  const Args& a = l.a;
  const int lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t tok = job / jobs_token;
  if (tok >= a.num_tokens) {
    const int64_t jobs = static_cast<int64_t>(a.num_tokens) * jobs_token;
    check_seqs(a, static_cast<int>(blockIdx.x - (jobs + kWarps - 1) / kWarps));
    return;
  }
  const int t = static_cast<int>(tok), part = static_cast<int>(job - tok * jobs_token);
  if (a.cu && behind_last(a.cu, a.num_seqs, t)) return;  // padding: its row is not even read
  const int u = lane % kUnits, first = lane / kUnits;

  // the job's loads
  uint4 c[kC], pe, r[kHeadsJob / kPer];
  const int h0 = part * kHeadsJob + first, heads = l.q_rope ? a.Hq : 0;
  if (part == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(l.c_new + t * l.c_new_stride);
#pragma unroll
    for (int i = 0; i < kC; ++i) c[i] = src[lane + 32 * i];
    pe = *reinterpret_cast<const uint4*>(l.k_rope + t * l.k_rope_stride + 8 * u);
  }
#pragma unroll
  for (int j = 0; j < kHeadsJob / kPer; ++j) {
    const int h = h0 + j * kPer;
    r[j] = h < heads ? *reinterpret_cast<const uint4*>(l.q_rope + t * l.q_rope_tok +
                                                       h * l.q_rope_head + 8 * u)
                     : make_uint4(0, 0, 0, 0);
  }

  const int s = a.cu ? segment_of(a.cu, a.num_seqs, t) : t;
  const Seq q = load_seq(a, s);
  if (t < q.row0 || t >= q.row0 + q.n || q.len <= 0) return;  // padding
  const int pos = q.len - q.n + t - q.row0;
  const int row = a.rope_pos ? a.rope_pos[t] : pos;
  if (row < 0 || row >= a.rope_len) {
    flag_bounds(a);
    return;
  }
  float cs[8], sn[8];
  {
    const int n = a.interleaved ? 4 : 8, col = a.interleaved ? 4 * u : 8 * (u % (kUnits / 2));
    const float4* cp =
        reinterpret_cast<const float4*>(a.cos + int64_t{row} * (kLatentRope / 2) + col);
    const float4* sp =
        reinterpret_cast<const float4*>(a.sin + int64_t{row} * (kLatentRope / 2) + col);
    *reinterpret_cast<float4*>(cs) = __ldg(cp);
    *reinterpret_cast<float4*>(sn) = __ldg(sp);
    if (n == 8) {
      *reinterpret_cast<float4*>(cs + 4) = __ldg(cp + 1);
      *reinterpret_cast<float4*>(sn + 4) = __ldg(sp + 1);
    }
  }
  if (part == 0) {
    const int page = page_of(a, s, pos);
    if (page >= 0) {
      char* dst = a.kc + page * a.k_page + (pos & ((1 << a.page_shift) - 1)) * a.k_tok;
      const uint4 o = turn_unit(pe, u, cs, sn, a.interleaved, a.f16);
#pragma unroll
      for (int i = 0; i < kC; ++i) reinterpret_cast<uint4*>(dst)[lane + 32 * i] = c[i];
      if (first == 0) reinterpret_cast<uint4*>(dst)[32 * kC + u] = o;
    }
  }
#pragma unroll
  for (int j = 0; j < kHeadsJob / kPer; ++j) {
    const uint4 o = turn_unit(r[j], u, cs, sn, a.interleaved, a.f16);
    const int h = h0 + j * kPer;
    if (h < heads)
      *reinterpret_cast<uint4*>(l.q_rot + t * l.q_rot_tok + h * l.q_rot_head + 8 * u) = o;
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentArgs& l, cudaStream_t st) {
  const int per = l.q_rope ? (l.a.Hq + kHeadsJob - 1) / kHeadsJob : 1;
  const int64_t blocks = (static_cast<int64_t>(l.a.num_tokens) * per + kWarps - 1) / kWarps +
                         check_blocks(l.a, kWarps * 32);
  if (blocks >= 1ll << 31) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kWarps * 32);
  return l.d_c == 512 ? launch_early(latent_append_kernel<2>, grid, block, 0, st, l, per)
                      : launch_early(latent_append_kernel<1>, grid, block, 0, st, l, per);
}

}  // namespace paged
}  // namespace attn
