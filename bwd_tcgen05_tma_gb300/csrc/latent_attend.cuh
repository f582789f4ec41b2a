// Attention over the paged latent cache: one block a (token, head), a plain
// kernel.  Four warps take a sequence's keys in turn, a lane a slice of the
// coordinates, with a running maximum and sum each, and join their states.
#pragma once
#include "latent.cuh"

namespace attn {
namespace paged {
namespace {

using sm103::ex2_approx;

template <bool F16, int DC>
__global__ void __launch_bounds__(128) latent_plain_kernel(const __grid_constant__ LatentArgs l) {
  constexpr int kV = DC / 32;
  __shared__ float s_o[4][DC];
  __shared__ float s_m[4], s_l[4];
  sm103::grid_dep_wait();
  const Args& a = l.a;
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int s = t;
  if (a.cu) {
    if (t >= a.cu[a.num_seqs]) return;
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    s = lo;
  }
  const Seq q = load_seq(a, s);
  if (t < q.row0 || t >= q.row0 + q.n) return;
  if (outside(a, q)) flag_bounds(a);
  const int pos = q.len - q.n + t - q.row0, cap = a.max_pages << a.page_shift;
  const int lo = a.window >= 0 ? max(0, pos - a.window) : 0;
  const int hi = min(a.causal ? min(q.len, pos + 1) : q.len, cap);
  float ql[kV], qr[2];
  for (int i = 0; i < kV; ++i)
    ql[i] = elem(l.q_lat[t * l.q_lat_tok + h * l.q_lat_head + lane + 32 * i], F16);
  for (int i = 0; i < 2; ++i)
    qr[i] = elem(l.q_rot[t * l.q_rot_tok + h * l.q_rot_head + lane + 32 * i], F16);
  float o[kV], m = -INFINITY, sum = 0.f;
  for (int i = 0; i < kV; ++i) o[i] = 0.f;
  for (int j = lo + w; j < hi; j += 4) {
    const int page = page_of(a, s, j);
    if (page < 0) continue;
    const uint16_t* c = reinterpret_cast<const uint16_t*>(
        a.kc + page * a.k_page + (j & ((1 << a.page_shift) - 1)) * a.k_tok);
    float v[kV], d = 0.f;
    for (int i = 0; i < kV; ++i) {
      v[i] = elem(c[lane + 32 * i], F16);
      d += v[i] * ql[i];
    }
    for (int i = 0; i < 2; ++i) d += elem(c[DC + lane + 32 * i], F16) * qr[i];
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    d *= a.scale * kLog2e;
    const float mn = fmaxf(m, d), mu = mn == -INFINITY ? 0.f : mn;
    const float f = ex2_approx(m - mu), p = ex2_approx(d - mu);
    sum = sum * f + p;
    for (int i = 0; i < kV; ++i) o[i] = o[i] * f + (p == 0.f ? 0.f : p * v[i]);
    m = mn;
  }
  for (int i = 0; i < kV; ++i) s_o[w][lane + 32 * i] = o[i];
  if (lane == 0) s_m[w] = m, s_l[w] = sum;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float s2 = a.sink ? a.sink[h] * kLog2e : -INFINITY, mt = fmaxf(m, s2);
  const float mu = mt == -INFINITY ? 0.f : mt;
  float keys = 0.f;
  for (int i = 0; i < 4; ++i) keys += s_l[i] * ex2_approx(s_m[i] - mu);
  const float lt = keys + ex2_approx(s2 - mu);
  const bool none = no_key(m, keys);
  uint16_t* out = a.o + (static_cast<int64_t>(t) * a.Hq + h) * DC;
  for (int d = threadIdx.x; d < DC; d += 128) {
    float x = 0.f;
    for (int i = 0; i < 4; ++i) x += s_o[i][d] * ex2_approx(s_m[i] - mu);
    out[d] = static_cast<uint16_t>(pack2(none ? 0.f : x / lt, 0.f, F16));
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[static_cast<int64_t>(h) * a.num_tokens + t] =
        none ? (a.sink ? a.sink[h] : -INFINITY) : mt * kLn2 + logf(lt);
}

template <bool F16>
cudaError_t launch_latent(const LatentArgs& l, cudaStream_t st) {
  const dim3 grid(l.a.num_tokens, l.a.Hq);
  return l.d_c == 512 ? launch_early(latent_plain_kernel<F16, 512>, grid, dim3(128), 0, st, l)
                      : launch_early(latent_plain_kernel<F16, 256>, grid, dim3(128), 0, st, l);
}

}  // namespace
}  // namespace paged
}  // namespace attn
