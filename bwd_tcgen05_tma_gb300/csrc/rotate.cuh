// Rotary positions: the arithmetic shared by the kernels that turn queries and
// keys, in units of 16 elements (two 16-byte halves of a head's row).
#pragma once
#include "paged.cuh"

namespace attn {
namespace paged {

struct Unit {
  float x[16];  // first eight, second eight
};

// Element offsets of a unit's two halves inside a head of width d.
__device__ __forceinline__ int2 unit_at(int u, int rot, int interleaved) {
  if (!interleaved && u < rot / 16) return make_int2(8 * u, rot / 2 + 8 * u);
  return make_int2(16 * u, 16 * u + 8);
}

__device__ __forceinline__ void unpack8(uint4 v, float* x, int f16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (f16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The two 16-byte halves of a unit as they lie in memory.
struct Raw {
  uint4 lo, hi;
};
__device__ __forceinline__ Raw load_raw(const uint16_t* src, int2 at) {
  return {*reinterpret_cast<const uint4*>(src + at.x), *reinterpret_cast<const uint4*>(src + at.y)};
}
__device__ __forceinline__ void unpack(const Raw& v, Unit& r, int f16) {
  unpack8(v.lo, r.x, f16);
  unpack8(v.hi, r.x + 8, f16);
}

// A unit's cosines and sines: row `cs` of the tables, columns 8 u .. 8 u + 7.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(const float* cos, const float* sin, int rot, int u,
                                          int64_t cs, Turn& t) {
  const float4* cp = reinterpret_cast<const float4*>(cos + cs * (rot / 2) + 8 * u);
  const float4* sp = reinterpret_cast<const float4*>(sin + cs * (rot / 2) + 8 * u);
  *reinterpret_cast<float4*>(t.c) = __ldg(cp);
  *reinterpret_cast<float4*>(t.c + 4) = __ldg(cp + 1);
  *reinterpret_cast<float4*>(t.s) = __ldg(sp);
  *reinterpret_cast<float4*>(t.s + 4) = __ldg(sp + 1);
}
// a' = a c - b s and b' = b c + a s, each product and the sum rounded in fp32.
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = x, b = y;
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ void turn(Unit& r, const Turn& t, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(r.x[2 * i], r.x[2 * i + 1], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(r.x[i], r.x[i + 8], t.c[i], t.s[i]);
  }
}

__device__ __forceinline__ void store16(uint16_t* dst, int2 at, const Unit& r, int f16) {
  uint4 lo, hi;
  lo.x = pack2(r.x[0], r.x[1], f16);
  lo.y = pack2(r.x[2], r.x[3], f16);
  lo.z = pack2(r.x[4], r.x[5], f16);
  lo.w = pack2(r.x[6], r.x[7], f16);
  hi.x = pack2(r.x[8], r.x[9], f16);
  hi.y = pack2(r.x[10], r.x[11], f16);
  hi.z = pack2(r.x[12], r.x[13], f16);
  hi.w = pack2(r.x[14], r.x[15], f16);
  *reinterpret_cast<uint4*>(dst + at.x) = lo;
  *reinterpret_cast<uint4*>(dst + at.y) = hi;
}

// 16 bytes that are read, or written, once: first to leave the caches.
__device__ __forceinline__ uint4 ld16(const void* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void st16(void* p, uint4 v) { __stcs(reinterpret_cast<uint4*>(p), v); }

__device__ __forceinline__ uint4 pack8(const float* x, int f16) {
  return make_uint4(pack2(x[0], x[1], f16), pack2(x[2], x[3], f16), pack2(x[4], x[5], f16),
                    pack2(x[6], x[7], f16));
}

// Where a packed token stands: its row of the tables.
struct Places {
  int num_tokens, seq_len, num_segments, rope_len;
  const int32_t* positions;
  const int32_t* cu;
  int32_t* status;
};
// Blocks behind those of the tokens look all offsets over, so that a bad one is
// reported wherever it stands.
constexpr int kOffsetsThread = 4;
__device__ __forceinline__ void check_offsets(const Places& w, int block) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kOffsetsThread; ++k) {
    const int64_t i = (int64_t{block} * kOffsetsThread + k) * blockDim.x + threadIdx.x;
    if (i > w.num_segments) break;
    const int x = w.cu[i];
    bad |= x < 0 || x > w.num_tokens || (i < w.num_segments && w.cu[i + 1] < x);
  }
  if (bad && w.status) *w.status = ATTN_ERR_DEVICE_BOUNDS;
}
// -1: padding, or (reported) offsets or a position that may not be used.
__device__ __forceinline__ int place_of(const Places& w, int t) {
  int pos;
  if (w.positions) {
    pos = w.positions[t];
  } else if (w.cu) {
    if (w.num_segments == 0 || behind_last(w.cu, w.num_segments, t)) return -1;
    const int s = segment_of(w.cu, w.num_segments, t);
    const int a = w.cu[s], b = w.cu[s + 1];
    if (a < 0 || b > w.num_tokens || t < a || t >= b) return -1;  // (check_offsets reports it)
    pos = t - a;
  } else {
    pos = t % w.seq_len;
  }
  if (pos < 0 || pos >= w.rope_len) {
    if (w.status) *w.status = ATTN_ERR_DEVICE_BOUNDS;
    return -1;
  }
  return pos;
}

// What a call that turns packed tokens says about their places, checked.
template <class P>
attn_status_t check_places(const P* p) {
  auto aligned = [](const void* x, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0;
  };
  if (p->num_tokens < 0 || p->rope_len < 0) return ATTN_ERR_INVALID_ARG;
  if (p->num_tokens > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  if (p->positions && p->cu_seqlens) return ATTN_ERR_INVALID_ARG;
  if (p->cu_seqlens ? p->num_segments < 0 : !p->positions && p->seq_len < 1)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->positions, 4) || !aligned(p->cu_seqlens, 4) || !aligned(p->status, 4) ||
      !aligned(p->rope_cos, 16) || !aligned(p->rope_sin, 16))
    return ATTN_ERR_INVALID_ARG;
  if (p->num_tokens > 0 && p->rope_len > 0 && (!p->rope_cos || !p->rope_sin))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}
// Blocks of `warps` warps, a token each, and those that check the offsets.
template <class P>
unsigned token_blocks(const P* p, int warps) {
  const int64_t each = int64_t{32} * warps * kOffsetsThread;
  return static_cast<unsigned>((p->num_tokens + warps - 1) / warps +
                               (p->cu_seqlens ? (p->num_segments + each) / each : 0));
}
template <class P>
Places places(const P* p) {
  return {p->num_tokens, p->seq_len,    p->num_segments, p->rope_len,
          p->positions,  p->cu_seqlens, p->status};
}

}  // namespace paged
}  // namespace attn
