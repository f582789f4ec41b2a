// Host side of the paged-cache calls: argument validation, workspace layout
// and launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

int64_t cache_bytes(const attn_paged_params_t* p) {
  return p->cache_dtype == ATTN_DTYPE_FP8_E4M3 ? 1 : 2;
}

int kind_of(const attn_paged_params_t* p) {
  if (p->cache_dtype == ATTN_DTYPE_FP8_E4M3) return kCacheE4m3;
  return p->cache_dtype == ATTN_DTYPE_FP16 ? kCacheF16 : kCacheBf16;
}

bool row_stride_ok(const void* ptr, int64_t stride, int64_t width) {
  return !ptr || (aligned(ptr, 16) && stride >= width && stride % 8 == 0);
}

// What both calls require.
attn_status_t validate(const attn_paged_params_t* p) {
  if (!p || p->struct_version != ATTN_PAGED_PARAMS_VERSION) return ATTN_ERR_INVALID_ARG;
  if (p->dtype != ATTN_DTYPE_BF16 && p->dtype != ATTN_DTYPE_FP16) return ATTN_ERR_INVALID_ARG;
  if (p->cache_dtype != p->dtype && p->cache_dtype != ATTN_DTYPE_FP8_E4M3)
    return ATTN_ERR_INVALID_ARG;
  if (p->mask != ATTN_MASK_NONE && p->mask != ATTN_MASK_CAUSAL) return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs < 0 || p->num_tokens < 0 || p->max_q_len < 1 || p->Hq <= 0 || p->Hkv <= 0 ||
      p->num_pages < 0 || p->max_pages < 0)
    return ATTN_ERR_INVALID_ARG;
  if (p->Hq % p->Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (p->Hq > 256) return ATTN_ERR_UNSUPPORTED;
  if (p->d_qk != 64 && p->d_qk != 128 && p->d_qk != 192) return ATTN_ERR_UNSUPPORTED;
  if (p->d_v != 64 && p->d_v != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)))
    return ATTN_ERR_UNSUPPORTED;
  // positions, packed rows and sequences are 32-bit, with room for a window, a tile or
  // a block's sequences beyond
  if (p->num_seqs > (1 << 30) || static_cast<int64_t>(p->max_pages) * p->page_size > (1ll << 30) ||
      static_cast<int64_t>(p->num_tokens) * (p->Hq / p->Hkv) > (1ll << 30))
    return ATTN_ERR_UNSUPPORTED;
  if (!p->cu_seqlens_q && p->num_tokens != p->num_seqs) return ATTN_ERR_SHAPE_MISMATCH;
  const bool none = p->num_seqs == 0 || p->num_tokens == 0;
  if (!none && (!p->seq_lens || (!p->page_table && p->max_pages > 0) ||
                ((!p->k_cache || !p->v_cache) && p->num_pages > 0)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->seq_lens, 4) || !aligned(p->page_table, 4) || !aligned(p->cu_seqlens_q, 4) ||
      !aligned(p->status, 4) || !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4) ||
      !aligned(p->k_cache, 16) || !aligned(p->v_cache, 16))
    return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs > 1 && p->table_stride < p->max_pages) return ATTN_ERR_INVALID_ARG;
  const int64_t per16 = 16 / cache_bytes(p);
  for (int i = 0; i < 3; ++i)
    if (p->k_cache_stride[i] <= 0 || p->k_cache_stride[i] % per16 || p->v_cache_stride[i] <= 0 ||
        p->v_cache_stride[i] % per16)
      return ATTN_ERR_INVALID_ARG;
  const bool scales = p->k_scale && p->v_scale, any = p->k_scale || p->v_scale;
  if (p->cache_dtype == ATTN_DTYPE_FP8_E4M3 ? (!none && !scales && p->num_pages > 0) : any)
    return ATTN_ERR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(p->Hq) * p->d_qk;
  if (!row_stride_ok(p->q, p->q_stride, wq) || !row_stride_ok(p->q_rot, p->q_rot_stride, wq))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t validate_append(const attn_paged_params_t* p) {
  const attn_status_t s = validate(p);
  if (s != ATTN_OK) return s;
  if (!p->k_new != !p->v_new) return ATTN_ERR_INVALID_ARG;
  if (!p->k_new && p->num_tokens > 0) return ATTN_ERR_INVALID_ARG;
  if (p->q && !p->q_rot) return ATTN_ERR_INVALID_ARG;
  // in place a row is turned where it lies
  if (p->q && p->q == p->q_rot && p->q_stride != p->q_rot_stride && p->num_tokens > 1)
    return ATTN_ERR_INVALID_ARG;
  if (!row_stride_ok(p->k_new, p->k_new_stride, static_cast<int64_t>(p->Hkv) * p->d_qk) ||
      !row_stride_ok(p->v_new, p->v_new_stride, static_cast<int64_t>(p->Hkv) * p->d_v))
    return ATTN_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > p->d_qk) return ATTN_ERR_INVALID_ARG;
  if (p->rot_dim % 16) return ATTN_ERR_UNSUPPORTED;
  if (p->rot_dim > 0 && (!p->rope_cos || !p->rope_sin || !aligned(p->rope_cos, 16) ||
                         !aligned(p->rope_sin, 16) || p->rope_len <= 0))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->rope_pos, 4)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t validate_fwd(const attn_paged_params_t* p) {
  const attn_status_t s = validate(p);
  if (s != ATTN_OK) return s;
  if (!p->q && !p->q_rot && p->num_tokens > 0) return ATTN_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->sink, 4)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

void fill(Args& a, const attn_paged_params_t* p) {
  std::memset(&a, 0, sizeof(a));
  const int64_t cb = cache_bytes(p);
  a.num_seqs = p->num_seqs;
  a.num_tokens = p->num_tokens;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.group = p->Hq / p->Hkv;
  while ((1 << a.group_shift) < a.group) ++a.group_shift;
  a.group_mul = static_cast<uint32_t>(
      ((1ull << 32) * ((1ull << a.group_shift) - a.group)) / a.group + 1);
  while ((1 << a.page_shift) < p->page_size) ++a.page_shift;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages;
  a.f16 = p->dtype == ATTN_DTYPE_FP16;
  a.causal = p->mask == ATTN_MASK_CAUSAL;
  a.window = p->window_left < 0 ? -1 : p->window_left < (1 << 30) ? p->window_left : 1 << 30;
  a.scale = p->scale;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.seq_lens = p->seq_lens;
  a.cu = p->cu_seqlens_q;
  a.kc = static_cast<char*>(p->k_cache);
  a.vc = static_cast<char*>(p->v_cache);
  a.k_page = p->k_cache_stride[0] * cb;
  a.k_head = p->k_cache_stride[1] * cb;
  a.k_tok = p->k_cache_stride[2] * cb;
  a.v_page = p->v_cache_stride[0] * cb;
  a.v_head = p->v_cache_stride[1] * cb;
  a.v_tok = p->v_cache_stride[2] * cb;
  a.k_scale = p->k_scale;
  a.v_scale = p->v_scale;
  a.status = p->status;
  a.d_qk = p->d_qk;
  a.d_v = p->d_v;
}

// Which kernel, by the rows expected for a KV head and the keys a row can see.
// The many-row kernel's time hardly depends on the rows up to 256, the few-row
// kernel's grows with them.  d 128, 8 KV heads, us, few against many rows:
//   16 x 4096 keys, E4M3: 32 rows 80 : 96, 48 rows 136 : 96, 128 rows 257 : 97;
//     bf16: 88 : 85, 148 : 85, 279 : 87.
//   1 x 32768 keys, E4M3: 32 rows 45 : 60, 48 rows 67 : 61; bf16: 51 : 56,
//     75 : 56.
// With few keys a row block's start weighs more than a second pass, and more
// so in E4M3, whose pages are converted.  64 rows of each of 64 sequences:
//   E4M3: 256 keys 46 : 68, 512 keys 76 : 84, 1024 keys 132 : 120;
//   bf16: 256 keys 51 : 52, 512 keys 85 : 69; a window of 10 keys 20 : 44.
// (Of 16 sequences of 256 keys: E4M3 43 : 30, bf16 40 : 22; the batch's size
// moves the point, the keys a row sees move it more.)
// 96 rows of 64 x 512 keys: E4M3 142 : 85, bf16 158 : 70.
// One kernel serves the whole call, so a prompt's chunk brings the single tokens
// beside it to the many-row kernel: a chunk of 512 tokens over 2048 cached ones
// (32 query heads) and 64 tokens over 251 k keys take 329 us together in E4M3
// (bf16 277), in calls of their own 42 and 94 (36 and 160).
bool many_rows(const attn_paged_params_t* p) {
  const int64_t rows = static_cast<int64_t>(p->max_q_len) * (p->Hq / p->Hkv);
  int64_t keys = static_cast<int64_t>(p->max_pages) * p->page_size;
  if (p->window_left >= 0) keys = std::min<int64_t>(keys, int64_t{p->window_left} + p->max_q_len);
  const int64_t few_keys = p->cache_dtype == ATTN_DTYPE_FP8_E4M3 ? 768 : 192;
  return p->num_pages > 0 && (rows > 64 || (rows > 32 && keys > few_keys));
}

// Workspace: descriptors of split items, then their partial states.
struct Plan {
  size_t desc, ml, part, total;
};
Plan make_plan(const attn_paged_params_t* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int64_t expected = static_cast<int64_t>(p->max_q_len) * (p->Hq / p->Hkv);
  // partial states: two a block, of all its rows
  const size_t rows = many_rows(p) ? 2 * kMaxChunkCtas * kChunkPartRows
                                   : 2 * kMaxCtas * decode_rows(expected);
  Plan pl;
  pl.desc = 0;
  pl.ml = up(kMaxCtas * sizeof(int4));
  pl.part = pl.ml + up(rows * sizeof(float2));
  pl.total = pl.part + rows * p->d_v * sizeof(float);
  return pl;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

}  // namespace

bool cache_map(CUtensorMap* m, int kind, const void* base, int d, const Args& a, int64_t tok,
               int64_t head, int64_t page, int slots, int width, int swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool codes = kind == kCacheE4m3;
  // a pool without pages has no memory; no box of it is ever asked for
  const void* mem = a.num_pages > 0 ? base : static_cast<const void*>(a.q);
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)1 << a.page_shift, (cuuint64_t)a.Hkv,
                              (cuuint64_t)(a.num_pages > 0 ? a.num_pages : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)tok, (cuuint64_t)head, (cuuint64_t)page};
  const cuuint32_t box[4] = {(cuuint32_t)(codes ? width : width / 2), (cuuint32_t)slots, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = codes                ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : kind == kCacheF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = swizzle == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_NONE;
  return fn(m, type, 4, const_cast<void*>(mem), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace paged
}  // namespace attn

using namespace attn::paged;

extern "C" {

size_t attn_paged_workspace_size(const attn_paged_params_t* p) {
  if (validate_fwd(p) != ATTN_OK) return 0;
  return make_plan(p).total;
}

attn_status_t attn_paged_append(const attn_paged_params_t* p, void* stream) {
  const attn_status_t s = validate_append(p);
  if (s != ATTN_OK) return s;
  if (p->num_seqs == 0 || p->num_tokens == 0) return ATTN_OK;
  Args a;
  fill(a, p);
  a.q = static_cast<const uint16_t*>(p->q);
  a.q_stride = p->q_stride;
  a.k_new = static_cast<const uint16_t*>(p->k_new);
  a.v_new = static_cast<const uint16_t*>(p->v_new);
  a.q_rot = static_cast<uint16_t*>(p->q_rot);
  a.k_new_stride = p->k_new_stride;
  a.v_new_stride = p->v_new_stride;
  a.q_rot_stride = p->q_rot_stride;
  a.rot = p->rot_dim;
  a.interleaved = p->rot_interleaved != 0;
  a.rope_len = p->rope_len;
  a.cos = p->rope_cos;
  a.sin = p->rope_sin;
  a.rope_pos = p->rope_pos;
  return launch_append(a, kind_of(p), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

attn_status_t attn_paged_fwd(const attn_paged_params_t* p, void* o, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  const attn_status_t s = validate_fwd(p);
  if (s != ATTN_OK) return s;
  if (p->num_seqs == 0 || p->num_tokens == 0) return ATTN_OK;
  if (!o || !aligned(o, 16) || !aligned(lse, 4) || !ws || !aligned(ws, 256))
    return ATTN_ERR_INVALID_ARG;
  const Plan pl = make_plan(p);
  if (ws_bytes < pl.total) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  Args a;
  fill(a, p);
  a.q = static_cast<const uint16_t*>(p->q_rot ? p->q_rot : p->q);
  a.q_stride = p->q_rot ? p->q_rot_stride : p->q_stride;
  a.sink = p->sink;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.o_st32 = aligned(o, 32);
  char* w = static_cast<char*>(ws);
  a.split_desc = reinterpret_cast<int4*>(w + pl.desc);
  a.part_ml = reinterpret_cast<float2*>(w + pl.ml);
  a.part = reinterpret_cast<float*>(w + pl.part);
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  const int rows = decode_rows(static_cast<int64_t>(p->max_q_len) * a.group);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kind = kind_of(p);
  cudaError_t e;
  if (many_rows(p))
    e = kind == kCacheE4m3  ? launch_chunk_e4m3(a, sms, st)
        : kind == kCacheF16 ? launch_chunk_f16(a, sms, st)
                            : launch_chunk_bf16(a, sms, st);
  else
    e = kind == kCacheE4m3  ? launch_decode_e4m3(a, rows, sms, st)
        : kind == kCacheF16 ? launch_decode_f16(a, rows, sms, st)
                            : launch_decode_bf16(a, rows, sms, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
