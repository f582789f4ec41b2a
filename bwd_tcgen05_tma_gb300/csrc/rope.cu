// Rotary positions: the tables, and turning queries and keys (or their
// gradients) in the layouts the attention reads.
#include <cmath>

#include "rotate.cuh"

namespace attn {
namespace paged {
namespace {

// ---------------------------------------------------------------- tables
// Angles in turns, modulo 1, as fixed-point fractions: position times frequency is
// an integer product whose overflow is the modulo, exact whatever the position (an
// error of half a unit of a frequency, 2^-65 turns, grows to 2^-35 at position 2^30).
// Of the product's 64 bits the upper 32 are kept, 2^-32 turns or 1.5e-9 radians, an
// eightieth of what the angle's roundings to float make of it.  The nearest quarter is
// taken off first, so that those are relative to an angle below pi/4.  (In fp64 the same
// products and reductions would run at a sixty-fourth of the fp32 rate here.)  Bound by
// its stores and a launch's 2 us (131072 positions of 32 pairs, 33.5 MB: 6.1 us; with
// all 64 bits turned to float 8.7, and with sincospif in place of the series 9.8; 4
// positions a thread 6.3, blocks of 256 threads 6.4); small tables by the
// launch (8192 positions of 64 pairs: 2.3 us in a graph, 4.5 as the host launches them).
constexpr int kTableThreads = 128;
constexpr int kTableRows = 8;  // positions a thread takes

struct TableArgs {
  int rope_len, half;
  float magnitude;
  float* cos;
  float* sin;
  uint64_t freq[128];  // turns a position, times 2^64
};

// Taylor's series of cos x and sin x for |x| <= pi/4, cut where the next term is
// below 2e-9.  (x itself comes with three roundings, 2^-22.8 together at pi/4; the
// values are off by less than 2^-22.)
__device__ __forceinline__ void sincos_eighth(float x, float& c, float& s) {
  const float z = x * x;
  float p = fmaf(z, -1.f / 3628800, 1.f / 40320);
  p = fmaf(z, p, -1.f / 720);
  p = fmaf(z, p, 1.f / 24);
  p = fmaf(z, p, -0.5f);
  c = fmaf(z, p, 1.f);
  float q = fmaf(z, 1.f / 362880, -1.f / 5040);
  q = fmaf(z, q, 1.f / 120);
  q = fmaf(z, q, -1.f / 6);
  s = fmaf(x * z, q, x);
}

__global__ void __launch_bounds__(kTableThreads) table_kernel(const __grid_constant__ TableArgs a) {
  const int groups = a.half / 4, per = kTableThreads / groups;  // positions of a block at once
  const int g = threadIdx.x % groups, i = threadIdx.x / groups;
  if (i >= per) return;
  uint64_t f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = a.freq[4 * g + k];
  sm103::grid_dep_wait();
  const int j0 = blockIdx.x * per * kTableRows + i;
#pragma unroll
  for (int r = 0; r < kTableRows; ++r) {
    const int j = j0 + r * per;
    if (j >= a.rope_len) return;
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t turn = static_cast<uint32_t>(f[k] >> 32) * j +
                            __umulhi(static_cast<uint32_t>(f[k]), static_cast<uint32_t>(j));
      const uint32_t q = (turn + (1u << 29)) >> 30;
      const int32_t rest = static_cast<int32_t>(turn - (q << 30));
      float cc, ss;
      sincos_eighth(__int2float_rn(rest) * (6.2831853f * 0x1p-32f), cc, ss);
      const float x = (q & 1) ? ss : cc, y = (q & 1) ? cc : ss;
      // quarters: (c, s), (-s, c), (-c, -s), (s, -c)
      c[k] = (((q + 1) & 2) ? -x : x) * a.magnitude;
      s[k] = ((q & 2) ? -y : y) * a.magnitude;
    }
    const int64_t at = static_cast<int64_t>(j) * a.half + 4 * g;
    *reinterpret_cast<float4*>(a.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(a.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// ---------------------------------------------------------------- turning
// One warp a token: its lanes take the units of several heads side by side, so
// that a warp's accesses are whole lines, and each lane keeps its unit's cosines
// and sines for all heads.  Bound by HBM, two bytes an element each way: 2 x 8192
// tokens of 32 + 8 heads, d 128, 52.1 us, 6.5 TB/s; 8192 tokens of 16 + 16 heads, d
// 192 of which 64 turn, 32.2 us, 6.3 TB/s.  (Blocks of 4 warps instead of 8, so that
// they leave one by one, 58 -> 54 and 42 -> 36; accesses that leave the caches first
// 52 and 34.5; eight copies in flight 32.2.)
constexpr int kWarps = 4;
constexpr int kAtOnce = 4;  // units in flight a lane
constexpr int kCopies = 8;

struct RopeArgs {
  Places w;
  int Hq, heads, d, start, rot, interleaved, inverse, f16, copy;
  const float* cos;
  const float* sin;
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
};

__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeArgs a) {
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
  const uint16_t *q = a.q + t * a.q_stride, *k = a.k + t * a.k_stride;
  uint16_t *qo = a.q_out + t * a.q_out_stride, *ko = a.k_out + t * a.k_out_stride;
  auto src = [&](int h) { return h < a.Hq ? q + h * a.d : k + (h - a.Hq) * a.d; };
  auto dst = [&](int h) { return h < a.Hq ? qo + h * a.d : ko + (h - a.Hq) * a.d; };

  const int units = a.rot / 16, per = 32 / units;
  const int u = lane % units, first = lane / units;
  if (first < per) {
    int2 at = unit_at(u, a.rot, a.interleaved);
    at.x += a.start;
    at.y += a.start;
    Turn cs;
    load_turn(a.cos, a.sin, a.rot, u, row, cs);
    if (a.inverse) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs.s[i] = -cs.s[i];
    }
    for (int h0 = first; h0 < a.heads; h0 += per * kAtOnce) {
      Raw raw[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (h0 + j * per < a.heads)
          raw[j] = {ld16(src(h0 + j * per) + at.x), ld16(src(h0 + j * per) + at.y)};
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (h0 + j * per >= a.heads) break;
        Unit r;
        unpack(raw[j], r, a.f16);
        turn(r, cs, a.interleaved);
        uint16_t* const to = dst(h0 + j * per);
        st16(to + at.x, pack8(r.x, a.f16));
        st16(to + at.y, pack8(r.x + 8, a.f16));
      }
    }
  }
  const int rest = (a.d - a.rot) / 8;  // 16-byte units of a head that pass
  if (!a.copy || rest == 0) return;
  const int before = a.start / 8, skip = a.rot / 8, step = 32 / rest, odd = 32 % rest;
  int h = lane / rest, x = lane % rest;
  while (h < a.heads) {
    uint4 v[kCopies];
    int hh = h, xx = x;
    auto next = [&]() {
      hh += step;
      xx += odd;
      if (xx >= rest) {
        xx -= rest;
        ++hh;
      }
    };
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int e = (xx < before ? xx : xx + skip) * 8;
      if (hh < a.heads) v[j] = ld16(src(hh) + e);
      next();
    }
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int e = (x < before ? x : x + skip) * 8;
      if (h < a.heads) st16(dst(h) + e, v[j]);
      h += step;
      x += odd;
      if (x >= rest) {
        x -= rest;
        ++h;
      }
    }
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status_t check_table(const attn_rope_table_params_t* p) {
  if (!p || p->struct_version != ATTN_ROPE_TABLE_PARAMS_VERSION) return ATTN_ERR_INVALID_ARG;
  if (p->scaling < ATTN_ROPE_NONE || p->scaling > ATTN_ROPE_TURNS) return ATTN_ERR_INVALID_ARG;
  if (p->rope_len < 0 || p->rot_dim <= 0) return ATTN_ERR_INVALID_ARG;
  if (p->rope_len > (1 << 30) || p->rot_dim % 16 || p->rot_dim > 256) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(p->base) || p->base < 1 || !std::isfinite(p->magnitude))
    return ATTN_ERR_INVALID_ARG;
  if (p->scaling != ATTN_ROPE_NONE && (!std::isfinite(p->factor) || p->factor < 1))
    return ATTN_ERR_INVALID_ARG;
  if (p->scaling == ATTN_ROPE_TURNS &&
      (!std::isfinite(p->turns_low) || !std::isfinite(p->turns_high) ||
       !(p->turns_low < p->turns_high) || p->trained_len < 1))
    return ATTN_ERR_INVALID_ARG;
  if (p->rope_len > 0 && (!p->rope_cos || !p->rope_sin)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->rope_cos, 16) || !aligned(p->rope_sin, 16)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t check_rope(const attn_rope_params_t* p) {
  if (!p || p->struct_version != ATTN_ROPE_PARAMS_VERSION) return ATTN_ERR_INVALID_ARG;
  if (p->dtype != ATTN_DTYPE_BF16 && p->dtype != ATTN_DTYPE_FP16) return ATTN_ERR_INVALID_ARG;
  if (p->Hq < 0 || p->Hkv < 0 || p->Hq + int64_t{p->Hkv} == 0 || p->d <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (p->Hq > 1024 || p->Hkv > 1024 || p->d > 256 || p->d % 16) return ATTN_ERR_UNSUPPORTED;
  if (p->rot_start < 0 || p->rot_dim <= 0 || int64_t{p->rot_start} + p->rot_dim > p->d)
    return ATTN_ERR_INVALID_ARG;
  if (p->rot_start % 8 || p->rot_dim % 16) return ATTN_ERR_UNSUPPORTED;
  const attn_status_t s = check_places(p);
  if (s != ATTN_OK) return s;
  struct {
    const void* in;
    const void* out;
    int64_t in_stride, out_stride;
    int heads;
  } const both[2] = {{p->q, p->q_out, p->q_stride, p->q_out_stride, p->Hq},
                     {p->k, p->k_out, p->k_stride, p->k_out_stride, p->Hkv}};
  for (const auto& x : both) {
    if (x.heads == 0) continue;
    const int64_t width = static_cast<int64_t>(x.heads) * p->d;
    if (p->num_tokens > 0 && (!x.in || !x.out)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(x.in, 16) || !aligned(x.out, 16) || x.in_stride < width || x.out_stride < width ||
        x.in_stride % 8 || x.out_stride % 8)
      return ATTN_ERR_INVALID_ARG;
    // in place a row is turned where it lies
    if (x.in && x.in == x.out && x.in_stride != x.out_stride && p->num_tokens > 1)
      return ATTN_ERR_INVALID_ARG;
  }
  return ATTN_OK;
}

}  // namespace
}  // namespace paged
}  // namespace attn

using namespace attn::paged;

extern "C" {

attn_status_t attn_rope_table(const attn_rope_table_params_t* p, void* stream) {
  const attn_status_t s = check_table(p);
  if (s != ATTN_OK) return s;
  TableArgs a = {};
  a.rope_len = p->rope_len;
  a.half = p->rot_dim / 2;
  a.magnitude = p->magnitude;
  a.cos = p->rope_cos;
  a.sin = p->rope_sin;
  const double pi2 = 6.283185307179586476925286766559;
  double base = p->base;
  if (p->scaling == ATTN_ROPE_BASE) {
    base *= std::pow(p->factor, p->rot_dim / (p->rot_dim - 2.0));
    if (!std::isfinite(base)) return ATTN_ERR_INVALID_ARG;
  }
  // powers by eights: two factors, three roundings of 2^-53 a frequency
  double low[8], high = 1;
  for (int i = 0; i < 8; ++i) low[i] = std::pow(base, -2.0 * i / p->rot_dim);
  for (int i = 0; i < a.half; ++i) {
    if (i % 8 == 0) high = std::pow(base, -2.0 * i / p->rot_dim);
    double f = high * low[i % 8];
    if (p->scaling == ATTN_ROPE_LINEAR) f /= p->factor;
    if (p->scaling == ATTN_ROPE_TURNS) {
      const double turns = p->trained_len * f / pi2;
      double w = (turns - p->turns_low) / (p->turns_high - p->turns_low);
      w = w < 0 ? 0 : w > 1 ? 1 : w;
      f *= w + (1 - w) / p->factor;
    }
    a.freq[i] = static_cast<uint64_t>(std::ldexp(f / pi2, 64) + 0.5);
  }
  if (p->rope_len == 0) return ATTN_OK;
  const int rows = kTableThreads / (a.half / 4) * kTableRows;
  const unsigned blocks = static_cast<unsigned>((int64_t{p->rope_len} + rows - 1) / rows);
  return launch_early(table_kernel, dim3(blocks), dim3(kTableThreads), 0,
                      static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

attn_status_t attn_rope(const attn_rope_params_t* p, void* stream) {
  const attn_status_t s = check_rope(p);
  if (s != ATTN_OK) return s;
  if (p->num_tokens == 0) return ATTN_OK;
  RopeArgs a = {};
  a.w = places(p);
  a.Hq = p->Hq;
  a.heads = p->Hq + p->Hkv;
  a.d = p->d;
  a.start = p->rot_start;
  a.rot = p->rot_dim;
  a.interleaved = p->rot_interleaved != 0;
  a.inverse = p->inverse != 0;
  a.f16 = p->dtype == ATTN_DTYPE_FP16;
  a.copy = (p->Hq && p->q != p->q_out) || (p->Hkv && p->k != p->k_out);
  a.cos = p->rope_cos;
  a.sin = p->rope_sin;
  a.q = static_cast<const uint16_t*>(p->q);
  a.k = static_cast<const uint16_t*>(p->k);
  a.q_out = static_cast<uint16_t*>(p->q_out);
  a.k_out = static_cast<uint16_t*>(p->k_out);
  a.q_stride = p->q_stride;
  a.k_stride = p->k_stride;
  a.q_out_stride = p->q_out_stride;
  a.k_out_stride = p->k_out_stride;
  const unsigned blocks = token_blocks(p, kWarps);
  return launch_early(rope_kernel, dim3(blocks), dim3(kWarps * 32), 0,
                      static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // extern "C"
