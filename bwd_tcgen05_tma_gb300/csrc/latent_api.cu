// Host side of the paged latent cache's calls: argument validation, workspace
// layout and launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "latent.cuh"

namespace attn {
namespace paged {
namespace {

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
bool rows_ok(const void* ptr, int64_t stride, int64_t width) {
  return !ptr || (aligned(ptr, 16) && stride >= width && stride % 8 == 0);
}
// token and head strides of [tokens, H, width]
bool heads_ok(const void* ptr, const int64_t* stride, int64_t width) {
  return rows_ok(ptr, stride[0], width) && rows_ok(ptr, stride[1], width);
}

// What both calls require.
attn_status_t validate(const attn_latent_params_t* p) {
  if (!p || p->struct_version != ATTN_LATENT_PARAMS_VERSION) return ATTN_ERR_INVALID_ARG;
  if (p->dtype != ATTN_DTYPE_BF16 && p->dtype != ATTN_DTYPE_FP16) return ATTN_ERR_INVALID_ARG;
  if (p->mask != ATTN_MASK_NONE && p->mask != ATTN_MASK_CAUSAL) return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs < 0 || p->num_tokens < 0 || p->max_q_len < 1 || p->H <= 0 ||
      p->num_pages < 0 || p->max_pages < 0)
    return ATTN_ERR_INVALID_ARG;
  if (p->H > 256) return ATTN_ERR_UNSUPPORTED;
  if ((p->d_c != 256 && p->d_c != 512) || p->d_r != kLatentRope) return ATTN_ERR_UNSUPPORTED;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)))
    return ATTN_ERR_UNSUPPORTED;
  // positions, packed rows and sequences are 32-bit, with room for a window, a tile or
  // the sequences of a lane beyond
  if (p->num_seqs > (1 << 30) || static_cast<int64_t>(p->max_pages) * p->page_size > (1ll << 30) ||
      static_cast<int64_t>(p->num_tokens) * p->H > (1ll << 30))
    return ATTN_ERR_UNSUPPORTED;
  if (!p->cu_seqlens_q && p->num_tokens != p->num_seqs) return ATTN_ERR_SHAPE_MISMATCH;
  const bool none = p->num_seqs == 0 || p->num_tokens == 0;
  if (!none && (!p->seq_lens || (!p->page_table && p->max_pages > 0) ||
                (!p->cache && p->num_pages > 0)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->seq_lens, 4) || !aligned(p->page_table, 4) || !aligned(p->cu_seqlens_q, 4) ||
      !aligned(p->status, 4) || !aligned(p->cache, 16))
    return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs > 1 && p->table_stride < p->max_pages) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    if (p->cache_stride[i] < p->d_c + p->d_r || p->cache_stride[i] % 8)
      return ATTN_ERR_INVALID_ARG;
  if (!heads_ok(p->q_rot, p->q_rot_stride, p->d_r)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t validate_append(const attn_latent_params_t* p) {
  const attn_status_t s = validate(p);
  if (s != ATTN_OK) return s;
  if ((!p->c_new || !p->k_rope) && p->num_tokens > 0) return ATTN_ERR_INVALID_ARG;
  if (!rows_ok(p->c_new, p->c_new_stride, p->d_c) ||
      !rows_ok(p->k_rope, p->k_rope_stride, p->d_r) ||
      !heads_ok(p->q_rope, p->q_rope_stride, p->d_r))
    return ATTN_ERR_INVALID_ARG;
  if (p->q_rope && !p->q_rot) return ATTN_ERR_INVALID_ARG;
  // in place a head's part is turned where it lies
  if (p->q_rope && p->q_rope == p->q_rot &&
      ((p->q_rope_stride[0] != p->q_rot_stride[0] && p->num_tokens > 1) ||
       (p->q_rope_stride[1] != p->q_rot_stride[1] && p->H > 1)))
    return ATTN_ERR_INVALID_ARG;
  if (p->rope_len < 0 || !aligned(p->rope_cos, 16) || !aligned(p->rope_sin, 16) ||
      !aligned(p->rope_pos, 4))
    return ATTN_ERR_INVALID_ARG;
  if (p->num_tokens > 0 && p->rope_len > 0 && (!p->rope_cos || !p->rope_sin))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t validate_fwd(const attn_latent_params_t* p) {
  const attn_status_t s = validate(p);
  if (s != ATTN_OK) return s;
  if ((!p->q_lat || !p->q_rot) && p->num_tokens > 0) return ATTN_ERR_INVALID_ARG;
  if (!heads_ok(p->q_lat, p->q_lat_stride, p->d_c)) return ATTN_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(p->sink, 4)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

void fill(LatentArgs& l, const attn_latent_params_t* p) {
  std::memset(&l, 0, sizeof(l));
  Args& a = l.a;
  a.num_seqs = p->num_seqs;
  a.num_tokens = p->num_tokens;
  a.Hq = a.group = p->H;
  a.Hkv = 1;
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
  a.kc = static_cast<char*>(p->cache);
  a.k_page = p->cache_stride[0] * 2;
  a.k_tok = p->cache_stride[1] * 2;
  a.status = p->status;
  a.d_qk = p->d_c + p->d_r;
  a.d_v = l.d_c = p->d_c;
  a.rot = p->d_r;
  a.interleaved = p->rot_interleaved != 0;
  a.rope_len = p->rope_len;
  a.cos = p->rope_cos;
  a.sin = p->rope_sin;
  a.rope_pos = p->rope_pos;
  a.sink = p->sink;
  l.c_new = static_cast<const uint16_t*>(p->c_new);
  l.k_rope = static_cast<const uint16_t*>(p->k_rope);
  l.q_rope = static_cast<const uint16_t*>(p->q_rope);
  l.q_lat = static_cast<const uint16_t*>(p->q_lat);
  l.q_rot = static_cast<uint16_t*>(p->q_rot);
  l.c_new_stride = p->c_new_stride;
  l.k_rope_stride = p->k_rope_stride;
  l.q_rope_tok = p->q_rope_stride[0];
  l.q_rope_head = p->q_rope_stride[1];
  l.q_lat_tok = p->q_lat_stride[0];
  l.q_lat_head = p->q_lat_stride[1];
  l.q_rot_tok = p->q_rot_stride[0];
  l.q_rot_head = p->q_rot_stride[1];
}

// Workspace: descriptors of split row blocks, then their partial states, two a
// block of all its rows.
struct Plan {
  size_t desc, ml, part, total;
};
int rows_of(const attn_latent_params_t* p) {
  return latent_rows(static_cast<int64_t>(p->max_q_len) * p->H);
}
// Blocks in pairs: two row blocks of a sequence go through its tiles side by side, so
// that they come from HBM once.  By the rows of the mean sequence (the largest may be
// alone): always for two row blocks (128 heads: 4 contexts of 100-131 k keys 184 -> 150
// us, 256 of up to 256 keys 60 -> 53); for more where the caches, at their longest,
// exceed the L2 cache (three chunks over up to 16 k keys: 232 us without, 239 with;
// shares are coarser); not for few and odd, where the last pair has one at work.
bool pairs(const attn_latent_params_t* p, int sms) {
  const int64_t rows = std::min(static_cast<int64_t>(p->max_q_len) * p->H,
                                (static_cast<int64_t>(p->num_tokens) * p->H + p->num_seqs - 1) /
                                    p->num_seqs);
  const int64_t blocks = (rows + 63) / 64;
  if (sms < 2 || blocks < 2 || (blocks % 2 && blocks < 7)) return false;
  constexpr double kL2 = 100e6;
  return blocks == 2 || static_cast<double>(p->num_seqs) * p->max_pages * p->page_size *
                                (p->d_c + p->d_r) * 2 > kL2;
}
Plan make_plan(const attn_latent_params_t* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = size_t{2} * kLatentMaxCtas * rows_of(p);
  Plan pl;
  pl.desc = 0;
  pl.ml = up(kLatentMaxCtas * sizeof(int4));
  pl.part = pl.ml + up(rows * sizeof(float2));
  pl.total = pl.part + rows * p->d_c * sizeof(float);
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

bool latent_map(CUtensorMap* m, const LatentArgs& l, int slots, int chunks) {
  auto fn = encode_fn();
  if (!fn) return false;
  const Args& a = l.a;
  // a pool without pages has no memory; no box of it is ever asked for
  const void* mem = a.num_pages > 0 ? static_cast<const void*>(a.kc) : l.q_lat;
  const cuuint64_t dims[4] = {64, cuuint64_t{1} << a.page_shift,
                              static_cast<cuuint64_t>(a.d_qk / 64),
                              static_cast<cuuint64_t>(a.num_pages > 0 ? a.num_pages : 1)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.k_tok), 128,
                                 static_cast<cuuint64_t>(a.k_page)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(slots), static_cast<cuuint32_t>(chunks),
                             1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(mem), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace paged
}  // namespace attn

using namespace attn::paged;

extern "C" {

size_t attn_latent_workspace_size(const attn_latent_params_t* p) {
  if (validate_fwd(p) != ATTN_OK) return 0;
  return make_plan(p).total;
}

attn_status_t attn_latent_append(const attn_latent_params_t* p, void* stream) {
  const attn_status_t s = validate_append(p);
  if (s != ATTN_OK) return s;
  if (p->num_seqs == 0 || p->num_tokens == 0) return ATTN_OK;
  LatentArgs l;
  fill(l, p);
  return launch_latent_append(l, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

attn_status_t attn_latent_fwd(const attn_latent_params_t* p, void* o, float* lse, void* ws,
                              size_t ws_bytes, void* stream) {
  const attn_status_t s = validate_fwd(p);
  if (s != ATTN_OK) return s;
  if (p->num_seqs == 0 || p->num_tokens == 0) return ATTN_OK;
  if (!o || !aligned(o, 16) || !aligned(lse, 4) || !ws || !aligned(ws, 256))
    return ATTN_ERR_INVALID_ARG;
  const Plan pl = make_plan(p);
  if (ws_bytes < pl.total) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  LatentArgs l;
  fill(l, p);
  l.a.o = static_cast<uint16_t*>(o);
  l.a.lse = lse;
  char* w = static_cast<char*>(ws);
  l.a.split_desc = reinterpret_cast<int4*>(w + pl.desc);
  l.a.part_ml = reinterpret_cast<float2*>(w + pl.ml);
  l.a.part = reinterpret_cast<float*>(w + pl.part);
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rows = rows_of(p);
  l.pair = rows == 64 && pairs(p, sms);
  // Queries are copied, and pieces handed out, up to four pieces ahead of the softmax: a
  // piece has at most the keys of a table's row, of which 64 take 1 to 2 us (4 us are
  // allowed them), and its search passes empty sequences in some 10 ns each (64).
  l.wait_ns = sm103::kWaitNs + 64ull * p->num_seqs + 250ull * p->max_pages * p->page_size;
  const cudaError_t e =
      l.a.f16 ? launch_latent_f16(l, rows, sms, st) : launch_latent_bf16(l, rows, sms, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
