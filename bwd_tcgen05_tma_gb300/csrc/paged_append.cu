// Appending new tokens to the paged cache.
//
// Two kinds of blocks in one launch.
//
// Keys and values: one block per (run of new tokens inside one page, KV head).
// With an E4M3 cache it owns the page's two scales of that head, so the scale,
// the codes already there and the new ones are settled in one place without
// atomics: the result does not depend on the order of blocks.  The values stay
// in registers from the load over the block's maximum to the store (up to
// kHold units a thread; pages of more read them twice).
//
// Queries: a thread takes one unit of a token (its cosines and sines stay in
// registers) through several heads, four in flight.
//
// Work goes in units of 16 elements, two 16-byte loads: the eight pairs of a
// rotation (halves rot/2 apart, or neighbours), or sixteen values that pass.
// Bound by HBM: two bytes a query element each way, a key or value element
// read as two bytes and written as one or two (17349 tokens of 32 query and 8
// KV heads, d 128, into E4M3: 82 us, 4.9 TB/s).
#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kHold = 4;

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
__device__ __forceinline__ void load_turn(const Args& a, int u, int64_t cs, Turn& t) {
  const float4* cp = reinterpret_cast<const float4*>(a.cos + cs * (a.rot / 2) + 8 * u);
  const float4* sp = reinterpret_cast<const float4*>(a.sin + cs * (a.rot / 2) + 8 * u);
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

__device__ __forceinline__ void store8(uint8_t* dst, int2 at, Unit r, float inv) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) m = sm103::fmax3(m, fabsf(r.x[i]), fabsf(r.x[i + 1]));
  if (m == __int_as_float(0x7f800000)) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (fabsf(r.x[i]) == __int_as_float(0x7f800000)) r.x[i] = __int_as_float(0x7fc00000);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = f32x2_e4m3x2(r.x[4 * i] * inv, r.x[4 * i + 1] * inv);
    const uint32_t hi = f32x2_e4m3x2(r.x[4 * i + 2] * inv, r.x[4 * i + 3] * inv);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(dst + at.x) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(dst + at.y) = make_uint2(w[2], w[3]);
}

// Largest finite magnitude (infinities and NaN become NaN codes and are left
// out; fmax leaves NaN out by itself).
__device__ __forceinline__ float unit_amax(const Unit& r) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) m = sm103::fmax3(m, fabsf(r.x[i]), fabsf(r.x[i + 1]));
  if (m < __int_as_float(0x7f800000)) return m;
  m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x = fabsf(r.x[i]);
    m = x < __int_as_float(0x7f800000) ? fmaxf(m, x) : m;
  }
  return m;
}

// The run of new tokens a block works on.
struct Run {
  int seq, col, slot0, n, row0, pos0;  // sequence, page's column of the table, slots, rows, position
};

// Block `c`'s run: the runs of all sequences in order, each sequence's new
// positions cut at page borders.  With one token per sequence run c is
// sequence c; otherwise every block sums the sequences' run counts, and the
// thread that finds run c among its sequence's hands it to the others.
__device__ __forceinline__ bool find_run(const Args& a, int c, Run* out) {
  __shared__ int s_sum[kThreads / 32];
  __shared__ Run s_run;
  auto cut = [&](int s, const Seq& q, int left) -> Run {
    const int first = q.len - q.n, lo = max(0, first);  // first < 0: those tokens have no slot
    if (first < 0) flag_bounds(a);
    const int col = (lo >> a.page_shift) + left;
    const int p0 = max(lo, col << a.page_shift), p1 = min(q.len, (col + 1) << a.page_shift);
    return {s, col, p0 & ((1 << a.page_shift) - 1), p1 - p0, q.row0 + (p0 - first), p0};
  };
  if (!a.cu) {
    const Seq q = load_seq(a, c);
    if (q.len <= 0) return false;  // length 0: the row is padding
    *out = cut(c, q, 0);
    return true;
  }
  if (threadIdx.x == 0) s_run.seq = -1;
  int base = 0;
  for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    Seq q = {0, 0, 0};
    int cnt = 0;
    if (s < a.num_seqs) {
      q = load_seq(a, s);
      if (q.n > 0 && q.len > 0)
        cnt = ((q.len - 1) >> a.page_shift) - (max(0, q.len - q.n) >> a.page_shift) + 1;
    }
    int x = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if ((threadIdx.x & 31) >= d) x += y;
    }
    if ((threadIdx.x & 31) == 31) s_sum[threadIdx.x / 32] = x;
    __syncthreads();
    int before = base;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int t = s_sum[w];
      if (w < static_cast<int>(threadIdx.x) / 32) before += t;
      base += t;
    }
    before += x - cnt;
    if (c >= before && c < before + cnt) s_run = cut(s, q, c - before);
    __syncthreads();
    if (s_run.seq >= 0 || c < base) break;
  }
  *out = s_run;
  return out->seq >= 0;
}

// Row of the rotation tables for a token, or -1 (reported).
__device__ __forceinline__ int table_row(const Args& a, int row, int pos) {
  const int p = a.rope_pos ? a.rope_pos[row] : pos;
  if (p < 0 || p >= a.rope_len) {
    flag_bounds(a);
    return -1;
  }
  return p;
}

// Queries: this block's tokens and eight heads.
constexpr int kHeads = 8;
template <int units>
__device__ __forceinline__ void turn_queries(const Args& a, int block) {
  constexpr int tokens = kThreads / units;
  const int groups = (a.Hq + kHeads - 1) / kHeads;
  const int u = threadIdx.x % units, i = threadIdx.x / units;
  const int t = (block / groups) * tokens + i, h0 = (block % groups) * kHeads;
  if (i >= tokens || t >= a.num_tokens) return;
  if (a.cu && t >= a.cu[a.num_seqs]) return;  // padding: its row is not even read
  const int2 at = unit_at(u, a.rot, a.interleaved);
  const int heads = min(kHeads, a.Hq - h0);
  const uint16_t* src = a.q + t * a.q_stride + h0 * a.d_qk;
  uint16_t* dst = a.q_rot + t * a.q_rot_stride + h0 * a.d_qk;
  Raw raw[4];  // on their way while the token's place is looked up
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < heads) raw[j] = load_raw(src + j * a.d_qk, at);
  // the token's sequence: the last one that starts at or before it
  int s = t;
  if (a.cu) {
    int lo = 0, hi = a.num_seqs;  // cu[lo] <= t < cu[hi], where it is anywhere
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    s = lo;
  }
  const Seq q = load_seq(a, s);
  if (t < q.row0 || t >= q.row0 + q.n || q.len <= 0) return;  // padding
  const bool turns = u < a.rot / 16;
  Turn cs;
  if (a.rot > 0) {
    const int row = table_row(a, t, q.len - q.n + t - q.row0);
    if (row < 0) return;
    if (turns) load_turn(a, u, row, cs);
  }
#pragma unroll
  for (int b = 0; b < kHeads; b += 4) {
    if (b > 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (b + j < heads) raw[j] = load_raw(src + (b + j) * a.d_qk, at);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (b + j >= heads) continue;
      uint16_t* const to = dst + (b + j) * a.d_qk;
      if (turns) {
        Unit r;
        unpack(raw[j], r, a.f16);
        turn(r, cs, a.interleaved);
        store16(to, at, r, a.f16);
      } else {
        *reinterpret_cast<uint4*>(to + at.x) = raw[j].lo;
        *reinterpret_cast<uint4*>(to + at.y) = raw[j].hi;
      }
    }
  }
}

// Blocks [0, runs * groups) write keys and values, of `per_block` heads (one
// with an E4M3 cache), the others turn queries.
template <int kKind, int uk, int uv>
__global__ void __launch_bounds__(kThreads, 3)
    append_kernel(const __grid_constant__ Args a, int runs, int per_block) {
  sm103::grid_dep_wait();
  const int groups = (a.Hkv + per_block - 1) / per_block;
  if (static_cast<int>(blockIdx.x) >= runs * groups) {
    turn_queries<uk>(a, blockIdx.x - runs * groups);
    return;
  }
  Run run;
  if (!find_run(a, blockIdx.x / groups, &run)) return;
  const int h = (blockIdx.x % groups) * per_block, tid = threadIdx.x;
  const int nk = run.n * uk, each = nk + run.n * uv;
  const int nkv = each * min(per_block, a.Hkv - h);
  char *kdst, *vdst;  // the run's first slot of head h

  // Unit e of the run's keys, then values.
  struct Place {
    int h, i, u;
    bool key;
  };
  auto place = [&](int e) -> Place {
    int hh = 0;
    if (kKind != kCacheE4m3) {
      hh = e / each;
      e -= hh * each;
    }
    const bool key = e < nk;
    const int i = key ? e / uk : (e - nk) / uv;
    return {hh, i, key ? e - i * uk : e - nk - i * uv, key};
  };
  auto fetch = [&](const Place& p) -> Raw {
    const int64_t t = run.row0 + p.i;
    return p.key ? load_raw(a.k_new + t * a.k_new_stride + (h + p.h) * a.d_qk,
                            unit_at(p.u, a.rot, a.interleaved))
                 : load_raw(a.v_new + t * a.v_new_stride + (h + p.h) * a.d_v, unit_at(p.u, 0, 0));
  };
  // its values, turned; false if the token is not to be written
  auto finish = [&](const Place& p, const Raw& raw, Unit& r) -> bool {
    int row = 0;
    if (a.rot > 0 && (row = table_row(a, run.row0 + p.i, run.pos0 + p.i)) < 0) return false;
    unpack(raw, r, a.f16);
    if (p.key && p.u < a.rot / 16) {
      Turn cs;
      load_turn(a, p.u, row, cs);
      turn(r, cs, a.interleaved);
    }
    return true;
  };
  auto store = [&](const Place& p, const Unit& r, float inv_k, float inv_v) {
    char* dst = p.key ? kdst + p.h * a.k_head + p.i * a.k_tok : vdst + p.h * a.v_head + p.i * a.v_tok;
    const int2 at = unit_at(p.u, p.key ? a.rot : 0, a.interleaved);
    if (kKind == kCacheE4m3)
      store8(reinterpret_cast<uint8_t*>(dst), at, r, p.key ? inv_k : inv_v);
    else
      store16(reinterpret_cast<uint16_t*>(dst), at, r, kKind == kCacheF16);
  };

  // The first units are on their way while the page is looked up.
  Raw raw[kHold];
  auto fetch_from = [&](int e0) {
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if (e0 + j * kThreads < nkv) raw[j] = fetch(place(e0 + j * kThreads));
  };
  fetch_from(tid);
  const int page = page_of(a, run.seq, run.pos0);
  if (page < 0) return;
  kdst = a.kc + page * a.k_page + h * a.k_head + run.slot0 * a.k_tok;
  vdst = a.vc + page * a.v_page + h * a.v_head + run.slot0 * a.v_tok;

  if (kKind != kCacheE4m3) {
    for (int e0 = tid; e0 < nkv; e0 += kHold * kThreads) {
      if (e0 != tid) fetch_from(e0);
#pragma unroll
      for (int j = 0; j < kHold; ++j) {
        const int e = e0 + j * kThreads;
        Unit r;
        if (e < nkv && finish(place(e), raw[j], r)) store(place(e), r, 1.f, 1.f);
      }
    }
    return;
  }

  // E4M3: the maxima first.  What is held is the unit as loaded; it is turned
  // again at the store (its cosines are in L1 by then), which leaves the
  // registers to a third block.
  float mk = 0.f, mv = 0.f;
  unsigned ok = 0;
  bool any = false;  // some token is written
  auto largest = [&](const Place& p, const Unit& r) {
    const float m = unit_amax(r);
    if (p.key) mk = fmaxf(mk, m);
    else mv = fmaxf(mv, m);
    any = true;
  };
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int e = tid + j * kThreads;
    Unit r;
    if (e < nkv && finish(place(e), raw[j], r)) {
      ok |= 1u << j;
      largest(place(e), r);
    }
  }
  for (int e = tid + kHold * kThreads; e < nkv; e += kThreads) {
    Unit r;
    if (finish(place(e), fetch(place(e)), r)) largest(place(e), r);
  }
  __shared__ float s_mk[kThreads / 32], s_mv[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, d));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, d));
  }
  if ((tid & 31) == 0) {
    s_mk[tid / 32] = mk;
    s_mv[tid / 32] = mv;
  }
  float* pk = a.k_scale + static_cast<int64_t>(page) * a.Hkv + h;
  float* pv = a.v_scale + static_cast<int64_t>(page) * a.Hkv + h;
  const float old_k = run.slot0 ? *pk : 0.f, old_v = run.slot0 ? *pv : 0.f;
  if (!__syncthreads_or(any)) return;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    mk = fmaxf(mk, s_mk[w]);
    mv = fmaxf(mv, s_mv[w]);
  }
  const float new_k = fmaxf(page_scale(mk), old_k), new_v = fmaxf(page_scale(mv), old_v);
  // codes of earlier tokens again under a grown scale
  auto again = [&](char* base, int64_t tok, int d, float ratio) {
    const int per = d / 16;
    for (int e = tid; e < run.slot0 * per; e += kThreads) {
      uint4* at = reinterpret_cast<uint4*>(base + (e / per - run.slot0) * tok + (e % per) * 16);
      uint4 v = *at;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t r = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t f2 = e4m3x2_f16x2(static_cast<uint16_t>(w[i] >> (16 * b)));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
          r |= static_cast<uint32_t>(f32x2_e4m3x2(f.x * ratio, f.y * ratio)) << (16 * b);
        }
        w[i] = r;
      }
      *at = v;
    }
  };
  if (new_k > old_k && run.slot0) again(kdst, a.k_tok, a.d_qk, old_k / new_k);
  if (new_v > old_v && run.slot0) again(vdst, a.v_tok, a.d_v, old_v / new_v);
  // scales are powers of two of at least 2^-64, but a caller's own may be
  // anything: the quotient is exact for the former
  const float inv_k = 1.f / new_k, inv_v = 1.f / new_v;
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (ok >> j & 1) {
      const Place p = place(tid + j * kThreads);
      Unit r;
      finish(p, raw[j], r);
      store(p, r, inv_k, inv_v);
    }
  for (int e = tid + kHold * kThreads; e < nkv; e += kThreads) {
    Unit r;
    if (finish(place(e), fetch(place(e)), r)) store(place(e), r, inv_k, inv_v);
  }
  if (tid == 0) {
    *pk = new_k;
    *pv = new_v;
  }
}

template <int kKind, int uk>
cudaError_t launch_width(const Args& a, dim3 grid, int runs, int per_block, cudaStream_t st) {
  return a.d_v == 64
             ? launch_early(append_kernel<kKind, uk, 4>, grid, dim3(kThreads), 0, st, a, runs,
                            per_block)
             : launch_early(append_kernel<kKind, uk, 8>, grid, dim3(kThreads), 0, st, a, runs,
                            per_block);
}
template <int kKind>
cudaError_t launch_dims(const Args& a, dim3 grid, int runs, int per_block, cudaStream_t st) {
  return a.d_qk == 64    ? launch_width<kKind, 4>(a, grid, runs, per_block, st)
         : a.d_qk == 128 ? launch_width<kKind, 8>(a, grid, runs, per_block, st)
                         : launch_width<kKind, 12>(a, grid, runs, per_block, st);
}

}  // namespace

cudaError_t launch_append(const Args& a, int kind, cudaStream_t st) {
  // runs of one sequence: one per page its new tokens touch
  int64_t runs = a.num_seqs;
  if (a.cu) {
    runs = (static_cast<int64_t>(a.num_tokens) >> a.page_shift) + 2ll * a.num_seqs;
    if (runs > a.num_tokens) runs = a.num_tokens;
  }
  // heads of a 16-bit cache's block: about 1024 units of a whole page
  int per_block = 1;
  if (kind != kCacheE4m3)
    while (per_block < a.Hkv &&
           (2 * per_block * (a.d_qk + a.d_v) / 16 << (a.cu ? a.page_shift : 0)) <= 1024)
      per_block *= 2;
  int64_t blocks = runs * ((a.Hkv + per_block - 1) / per_block);
  if (a.q) {
    const int tokens = kThreads / (a.d_qk / 16);
    blocks += (static_cast<int64_t>(a.num_tokens) + tokens - 1) / tokens *
              ((a.Hq + kHeads - 1) / kHeads);
  }
  if (blocks >= 1ll << 31) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  const int n = static_cast<int>(runs);
  return kind == kCacheE4m3  ? launch_dims<kCacheE4m3>(a, grid, n, per_block, st)
         : kind == kCacheF16 ? launch_dims<kCacheF16>(a, grid, n, per_block, st)
                             : launch_dims<kCacheBf16>(a, grid, n, per_block, st);
}

}  // namespace paged
}  // namespace attn
