// Latent attention, expanded form: keys and values from the up-projected latent
// vectors, and the gradients back.
//
// One warp a token.  The per-head parts are copied in 16-byte units, lane after
// lane, so that a warp's accesses are whole lines; the shared rotated part is
// turned once a token and lies in registers while it is written to every head
// (forward), or is summed over the heads in registers, lanes meeting in a fixed
// order, and turned back once (gradient).  Bound by HBM: nothing is read or
// written twice (8192 tokens of 16 heads, 128 + 64 and 128 wide, 153 MB: 25.3 us
// forward, 25.8 back, 6.0 TB/s).
#include "rotate.cuh"

namespace attn {
namespace paged {
namespace {

constexpr int kWarps = 4;
constexpr int kAtOnce = 6;  // loads in flight a lane

struct ExpandArgs {
  Places w;
  int H, d_n, d_r, d_v, interleaved, f16;
  const float* cos;
  const float* sin;
  uint16_t* kv;
  uint16_t* pe;
  uint16_t* k;
  uint16_t* v;
  int64_t kv_stride, pe_stride, k_stride, v_stride;
};

// The eight coordinates of unit u of the shared part, turned: units are 16 bytes,
// a lane each (lanes u, u + units, ... hold the same).
template <int kUnits>
__device__ __forceinline__ void turn_shared(const ExpandArgs& a, int u, int row, bool back,
                                            float (&x)[8]) {
  constexpr int kHalf = 4 * kUnits;  // pairs
  if (a.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(a.cos + int64_t{row} * kHalf + 4 * u);
    float4 s = *reinterpret_cast<const float4*>(a.sin + int64_t{row} * kHalf + 4 * u);
    if (back) s = make_float4(-s.x, -s.y, -s.z, -s.w);
    turn_pair(x[0], x[1], c.x, s.x);
    turn_pair(x[2], x[3], c.y, s.y);
    turn_pair(x[4], x[5], c.z, s.z);
    turn_pair(x[6], x[7], c.w, s.w);
    return;
  }
  // the other of each pair is kUnits / 2 lanes away
  const bool second = u >= kUnits / 2;
  const int col = 8 * (u - (second ? kUnits / 2 : 0));
  const float* cp = a.cos + int64_t{row} * kHalf + col;
  const float* sp = a.sin + int64_t{row} * kHalf + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = cp[i], s = back ? -sp[i] : sp[i];
    const float y = __shfl_xor_sync(0xffffffffu, x[i], kUnits / 2);
    float p = second ? y : x[i], q = second ? x[i] : y;
    turn_pair(p, q, c, s);
    x[i] = second ? q : p;
  }
}

// kUnits: 16-byte units of the shared part.
template <int kUnits, bool kBack>
__global__ void __launch_bounds__(kWarps * 32) expand_kernel(const __grid_constant__ ExpandArgs a) {
  sm103::grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.w.num_tokens) {
    const int block = blockIdx.x - (a.w.num_tokens + kWarps - 1) / kWarps;
    if (block >= 0) check_offsets(a.w, block);
    return;
  }
  const int row = place_of(a.w, t);
  if (row < 0) return;
  uint16_t *kv = a.kv + t * a.kv_stride, *k = a.k + t * a.k_stride, *v = a.v + t * a.v_stride;
  uint16_t* pe = a.pe + t * a.pe_stride;
  const int u = lane % kUnits, first = lane / kUnits;
  constexpr int kPer = 32 / kUnits;
  const int k_head = a.d_n + a.d_r;

  // the heads' own parts
  const int nu = a.d_n / 8, units = (a.d_n + a.d_v) / 8, step = 32 / units, odd = 32 % units;
  int h = lane / units, x = lane % units;
  auto next = [&](int& hh, int& xx) {
    hh += step;
    xx += odd;
    if (xx >= units) {
      xx -= units;
      ++hh;
    }
  };
  auto packed = [&](int hh, int xx) { return kv + (hh * units + xx) * 8; };
  auto apart = [&](int hh, int xx) {
    return xx < nu ? k + hh * k_head + xx * 8 : v + hh * a.d_v + (xx - nu) * 8;
  };
  while (h < a.H) {
    uint4 r[kAtOnce];
    int hh = h, xx = x;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (hh < a.H)
        r[j] = ld16(kBack ? apart(hh, xx) : packed(hh, xx));
      next(hh, xx);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (h < a.H) st16(kBack ? packed(h, x) : apart(h, x), r[j]);
      next(h, x);
    }
  }

  // the shared part
  float y[8];
  if constexpr (!kBack) {
    unpack8(*reinterpret_cast<const uint4*>(pe + 8 * u), y, a.f16);
    turn_shared<kUnits>(a, u, row, false, y);
    const uint4 o = pack8(y, a.f16);
    for (int hh = first; hh < a.H; hh += kPer)
      st16(k + hh * k_head + a.d_n + 8 * u, o);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.f;
    for (int h0 = first; h0 < a.H; h0 += kPer * kAtOnce) {
      uint4 r[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (h0 + j * kPer < a.H)
          r[j] = ld16(k + (h0 + j * kPer) * k_head + a.d_n + 8 * u);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (h0 + j * kPer >= a.H) break;
        float z[8];
        unpack8(r[j], z, a.f16);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += z[i];
      }
    }
    __syncwarp();
#pragma unroll
    for (int m = kUnits; m < 32; m <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += __shfl_xor_sync(0xffffffffu, y[i], m);
    turn_shared<kUnits>(a, u, row, true, y);
    if (first == 0) *reinterpret_cast<uint4*>(pe + 8 * u) = pack8(y, a.f16);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status_t check(const attn_latent_expand_params_t* p) {
  if (!p || p->struct_version != ATTN_LATENT_EXPAND_PARAMS_VERSION) return ATTN_ERR_INVALID_ARG;
  if (p->dtype != ATTN_DTYPE_BF16 && p->dtype != ATTN_DTYPE_FP16) return ATTN_ERR_INVALID_ARG;
  if (p->H <= 0 || p->d_n <= 0 || p->d_v <= 0 || p->d_r <= 0) return ATTN_ERR_INVALID_ARG;
  if (p->H > 1024 || p->d_n % 8 || p->d_v % 8 || p->d_n > 256 || p->d_v > 256 ||
      (p->d_r != 32 && p->d_r != 64 && p->d_r != 128))
    return ATTN_ERR_UNSUPPORTED;
  const attn_status_t s = check_places(p);
  if (s != ATTN_OK) return s;
  const int64_t H = p->H;
  struct {
    const void* ptr;
    int64_t stride, width;
  } const all[4] = {{p->kv, p->kv_stride, H * (p->d_n + p->d_v)},
                    {p->k_rope, p->k_rope_stride, p->d_r},
                    {p->k, p->k_stride, H * (p->d_n + p->d_r)},
                    {p->v, p->v_stride, H * p->d_v}};
  for (const auto& x : all) {
    if (p->num_tokens > 0 && !x.ptr) return ATTN_ERR_INVALID_ARG;
    if (!aligned(x.ptr, 16) || x.stride < x.width || x.stride % 8) return ATTN_ERR_INVALID_ARG;
  }
  return ATTN_OK;
}

template <bool kBack>
attn_status_t run(const attn_latent_expand_params_t* p, void* stream) {
  const attn_status_t s = check(p);
  if (s != ATTN_OK) return s;
  if (p->num_tokens == 0) return ATTN_OK;
  ExpandArgs a = {};
  a.w = places(p);
  a.H = p->H;
  a.d_n = p->d_n;
  a.d_r = p->d_r;
  a.d_v = p->d_v;
  a.interleaved = p->rot_interleaved != 0;
  a.f16 = p->dtype == ATTN_DTYPE_FP16;
  a.cos = p->rope_cos;
  a.sin = p->rope_sin;
  a.kv = static_cast<uint16_t*>(p->kv);
  a.pe = static_cast<uint16_t*>(p->k_rope);
  a.k = static_cast<uint16_t*>(p->k);
  a.v = static_cast<uint16_t*>(p->v);
  a.kv_stride = p->kv_stride;
  a.pe_stride = p->k_rope_stride;
  a.k_stride = p->k_stride;
  a.v_stride = p->v_stride;
  const dim3 grid(token_blocks(p, kWarps)), block(kWarps * 32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->d_r == 32   ? launch_early(expand_kernel<4, kBack>, grid, block, 0, st, a)
                        : p->d_r == 64 ? launch_early(expand_kernel<8, kBack>, grid, block, 0, st, a)
                                       : launch_early(expand_kernel<16, kBack>, grid, block, 0, st, a);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace paged
}  // namespace attn

extern "C" {

attn_status_t attn_latent_expand(const attn_latent_expand_params_t* p, void* stream) {
  return attn::paged::run<false>(p, stream);
}
attn_status_t attn_latent_expand_bwd(const attn_latent_expand_params_t* p, void* stream) {
  return attn::paged::run<true>(p, stream);
}

}  // extern "C"
