// Attention over the paged cache, the plain way: one block per (new token,
// query head), one warp per key at a time with the head's dims over its lanes,
// the softmax's running maximum and sum in fp32, and the warps' states joined
// at the end.
#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

constexpr int kWarps = 4;

template <int kKind>
__device__ __forceinline__ float cache_elem(const char* p, int i) {
  if (kKind == kCacheE4m3) return e4m3_value(reinterpret_cast<const uint8_t*>(p)[i]);
  return elem(reinterpret_cast<const uint16_t*>(p)[i], kKind == kCacheF16);
}

template <int kKind>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(Args a) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][128];
  const int row = blockIdx.x, h = blockIdx.y, hk = h / a.group;
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32;
  int seq = row;
  Seq q;
  if (a.cu) {
    for (seq = 0; seq < a.num_seqs; ++seq) {
      q = load_seq(a, seq);
      if (row >= q.row0 && row < q.row0 + q.n) break;
    }
    if (seq == a.num_seqs) return;
  } else {
    q = load_seq(a, seq);
  }
  const int pos = q.len - q.n + (row - q.row0);
  const int lo = a.window >= 0 ? max(0, pos - a.window) : 0;
  const int hi = a.causal ? min(q.len, pos + 1) : q.len;
  const uint16_t* qp = a.q + row * a.q_stride + h * a.d_qk;
  float qv[6], o[4] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 6; ++i)
    qv[i] = lane + 32 * i < a.d_qk ? elem(qp[lane + 32 * i], a.f16) : 0.f;
  for (int j = lo + w; j < hi; j += kWarps) {
    const int page = page_of(a, seq, j);
    if (page < 0) continue;
    const int slot = j & ((1 << a.page_shift) - 1);
    const char* kp = a.kc + page * a.k_page + hk * a.k_head + slot * a.k_tok;
    const char* vp = a.vc + page * a.v_page + hk * a.v_head + slot * a.v_tok;
    float s = 0.f;
    for (int i = 0; lane + 32 * i < a.d_qk; ++i) s += qv[i] * cache_elem<kKind>(kp, lane + 32 * i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale;
    float vs = 1.f;
    if (kKind == kCacheE4m3) {
      s *= a.k_scale[static_cast<int64_t>(page) * a.Hkv + hk];
      vs = a.v_scale[static_cast<int64_t>(page) * a.Hkv + hk];
    }
    const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
    const float c = expf(m - mu), p = expf(s - mu);
    l = l * c + p;
    for (int i = 0; lane + 32 * i < a.d_v; ++i)
      o[i] = o[i] * c + p * vs * cache_elem<kKind>(vp, lane + 32 * i);
    m = mn;
  }
  s_m[w] = m;
  s_l[w] = l;
  for (int i = 0; lane + 32 * i < a.d_v; ++i) s_o[w][lane + 32 * i] = o[i];
  __syncthreads();
  float mt = a.sink ? a.sink[h] : -INFINITY;
  for (int i = 0; i < kWarps; ++i) mt = fmaxf(mt, s_m[i]);
  const float mu = mt == -INFINITY ? 0.f : mt;
  float lt = a.sink ? expf(a.sink[h] - mu) : 0.f;
  for (int i = 0; i < kWarps; ++i) lt += s_l[i] * expf(s_m[i] - mu);
  for (int d = threadIdx.x; d < a.d_v; d += kWarps * 32) {
    float x = 0.f;
    for (int i = 0; i < kWarps; ++i) x += s_o[i][d] * expf(s_m[i] - mu);
    a.o[(static_cast<int64_t>(row) * a.Hq + h) * a.d_v + d] =
        round16(lt > 0.f ? x / lt : (lt == 0.f ? 0.f : lt), a.f16);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[static_cast<int64_t>(h) * a.num_tokens + row] = lt == 0.f ? -INFINITY : mt + logf(lt);
}

}  // namespace

cudaError_t launch_attend(const Args& a, int kind, cudaStream_t st) {
  const dim3 grid(a.num_tokens, a.Hq);
  if (kind == kCacheE4m3) attend_kernel<kCacheE4m3><<<grid, kWarps * 32, 0, st>>>(a);
  else if (kind == kCacheF16) attend_kernel<kCacheF16><<<grid, kWarps * 32, 0, st>>>(a);
  else attend_kernel<kCacheBf16><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace attn
