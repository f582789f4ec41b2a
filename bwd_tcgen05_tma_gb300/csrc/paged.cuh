// Shared by the paged-cache kernels: the device view of one call, and the
// arithmetic of pages, positions and E4M3 scales.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Element kinds of a cache.
enum CacheKind { kCacheBf16 = 0, kCacheF16 = 1, kCacheE4m3 = 2 };

struct Args {
  int num_seqs, num_tokens, Hq, Hkv, group;
  uint32_t group_mul;  // multiplier and shift of a division by `group`
  int group_shift;
  int page_shift, num_pages, max_pages;
  int f16;     // 16-bit tensors are fp16 (else bf16)
  int causal;  // attention: keys behind the row's position are masked
  int window;  // attention: keys more than this before it are masked (< 0: none)
  float scale;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu;
  int64_t table_stride;
  char* kc;  // cache bases; strides in bytes
  char* vc;
  int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;
  float* k_scale;
  float* v_scale;
  int32_t* status;
  // new tokens (strides in elements)
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint16_t* q_rot;
  int64_t q_stride, k_new_stride, v_new_stride, q_rot_stride;
  int rot, interleaved, rope_len, d_qk, d_v;
  const float* cos;
  const float* sin;
  const int32_t* rope_pos;
  // attention outputs and split partials
  const float* sink;
  uint16_t* o;
  float* lse;
  float* part;       // [2 * ctas][rows][d_v] unnormalised O
  float2* part_ml;   // [2 * ctas][rows] (max in log2 units, sum)
  int4* split_desc;  // [ctas] of an item's first piece: pieces (0: none), sequence, head, rows
  int part_rows;
  int o_st32;  // O may be stored 32 bytes at a time
};

// One sequence: its new rows and its length.
struct Seq {
  int row0, n, len;
};

__device__ __forceinline__ void flag_bounds(const Args& a) {
  if (a.status) *a.status = ATTN_ERR_DEVICE_BOUNDS;
}

// n / group for n >= 0 (multiplication by a rounded-up reciprocal of 33 bits,
// after Granlund and Montgomery's division by invariant integers).
__device__ __forceinline__ int div_group(const Args& a, int n) {
  const uint32_t u = static_cast<uint32_t>(n), t = __umulhi(a.group_mul, u);
  return a.group == 1 ? n : static_cast<int>((t + ((u - t) >> 1)) >> (a.group_shift - 1));
}

// Is packed token t behind the last of n > 0 segments?  Their end is taken for it only
// where the last segment's offsets are in order.
__device__ __forceinline__ bool behind_last(const int32_t* cu, int n, int t) {
  const int end = cu[n];
  return t >= end && end >= 0 && end >= cu[n - 1];
}
// The segment that holds packed token t, if one does: cu[s] <= t < cu[s + 1], but for
// the first, which may begin behind t, and the last, which may end before it.
__device__ __forceinline__ int segment_of(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;  // (hi + lo may pass 32 bits)
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Rows and length of sequence s.  Offsets outside [0, num_tokens] or
// decreasing, and negative lengths, are reported and read as empty.
__device__ __forceinline__ Seq load_seq(const Args& a, int s) {
  Seq q;
  q.len = a.seq_lens[s];
  q.row0 = s;
  q.n = 1;
  if (a.cu) {
    q.row0 = a.cu[s];
    const int end = a.cu[s + 1];
    q.n = end - q.row0;
    if (q.row0 < 0 || end > a.num_tokens || q.n < 0) {
      flag_bounds(a);
      q.row0 = 0;
      q.n = 0;
    }
  }
  if (q.len < 0) {
    flag_bounds(a);
    q.len = 0;
    q.n = 0;
  }
  return q;
}

// A token's place is looked up from the token, so that a call may meet few of its
// sequences: where there are offsets, blocks behind the others (of `threads` threads)
// go through all of them, and report what is bad wherever it stands.  (Out of line: the
// append of 64 tokens to a cache of heads takes 7.0 us, inlined 7.2.)
constexpr int kSeqsThread = 4;
inline int64_t check_blocks(const Args& a, int threads) {
  const int64_t each = int64_t{kSeqsThread} * threads;
  return a.cu ? (a.num_seqs + each - 1) / each : 0;
}
inline __device__ __noinline__ void check_seqs(const Args& a, int block) {
  if (!a.cu || block < 0) return;
#pragma unroll
  for (int k = 0; k < kSeqsThread; ++k) {
    const int64_t s = (int64_t{block} * kSeqsThread + k) * blockDim.x + threadIdx.x;
    if (s < a.num_seqs) load_seq(a, static_cast<int>(s));
  }
}

// Has a sequence positions outside the table's row, or new rows below position
// 0?  (One of length 0 has padding for rows.)
__device__ __forceinline__ bool outside(const Args& a, const Seq& q) {
  return q.len > a.max_pages << a.page_shift || (q.len > 0 && q.len < q.n);
}

// Page of position j of sequence s, or -1 (reported) when the table cannot
// give one.
__device__ __forceinline__ int page_of(const Args& a, int s, int j) {
  const int c = j >> a.page_shift;
  if (j < 0 || c >= a.max_pages) {
    flag_bounds(a);
    return -1;
  }
  const int p = a.table[s * a.table_stride + c];
  if (p < 0 || p >= a.num_pages) {
    flag_bounds(a);
    return -1;
  }
  return p;
}

__device__ __forceinline__ float elem(uint16_t x, int f16) {
  return f16 ? __half2float(__ushort_as_half(x)) : __uint_as_float(uint32_t(x) << 16);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int f16) {
  return f16 ? sm103::pack_f16x2(lo, hi) : sm103::pack_bf16x2(lo, hi);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint64_t* bar, int x,
                                            int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(sm103::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(p)
               : "memory");
  return v;
}

// Two E4M3 codes (low byte first) to a pair of fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t c) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(c));
  return d;
}
__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(e4m3x2_f16x2(c))));
}
// Top bits of a word's elements that are not finite.  (E4M3 has only NaN.)
template <int KIND>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if (KIND == kCacheE4m3) return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  if (KIND == kCacheF16) return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// The word with zeros in their place.
template <int KIND>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  const uint32_t f = not_finite<KIND>(w);
  return w & ~(KIND == kCacheE4m3 ? (f >> 7) * 255u : (f >> 15) * 65535u);
}
// Two values of at most 448 in magnitude, or NaN, to E4M3 codes, nearest even.
__device__ __forceinline__ uint16_t f32x2_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The larger of two, or NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Did a row (or a part of it) keep no key?  Its running maximum alone does not
// tell: maxima leave NaN out, so a row of NaN scores has -inf there too, but
// NaN in its sum.
__device__ __forceinline__ bool no_key(float max, float sum) {
  return max == -INFINITY && sum == 0.f;
}

// Launches a kernel that may be put in place while the one before it on the
// stream still runs; it waits for that one (grid_dep_wait) before it reads
// anything.
template <class... P, class... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

constexpr int kMinExp = -64;
// Smallest V scale the attention tells from 0: its inverse times the largest P
// (2^15) times the most keys (2^30) is still a number in the normaliser.
constexpr float kMinVScale = 0x1p-80f;
// Smallest power of two s >= 2^-64 with amax <= 448 s (amax finite): with
// amax = 1.f * 2^x, 448 = 1.75 * 2^8, so e = x - 8, or one more if 1.f > 1.75.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kMinExp ? kMinExp : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

cudaError_t launch_append(const Args& a, int kind, cudaStream_t st);

// Few rows per KV head: `rows` is the expected number of query rows of one
// KV head (tokens x group); sms the device's SM count.
constexpr int kMaxCtas = 304;
inline int decode_rows(int64_t rows) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32;
}
struct CacheMaps {
  CUtensorMap k, v;
};
// Tensor map over a cache, [page][head][slot][dim] by its strides in bytes:
// boxes of `slots` slots of one head and `width` bytes of their dims, in the
// swizzle of that many bytes (0: in the order of memory).
bool cache_map(CUtensorMap* m, int kind, const void* base, int d, const Args& a, int64_t tok,
               int64_t head, int64_t page, int slots, int width, int swizzle);
cudaError_t launch_decode_e4m3(const Args& a, int rows, int sms, cudaStream_t st);
cudaError_t launch_decode_f16(const Args& a, int rows, int sms, cudaStream_t st);
cudaError_t launch_decode_bf16(const Args& a, int rows, int sms, cudaStream_t st);

// Many rows per KV head.
constexpr int kMaxChunkCtas = 152;
constexpr int kChunkPartRows = 256;
cudaError_t launch_chunk_e4m3(const Args& a, int sms, cudaStream_t st);
cudaError_t launch_chunk_f16(const Args& a, int sms, cudaStream_t st);
cudaError_t launch_chunk_bf16(const Args& a, int sms, cudaStream_t st);

}  // namespace paged
}  // namespace attn
