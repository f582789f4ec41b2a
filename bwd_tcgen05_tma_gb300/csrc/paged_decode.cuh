// Attention over the paged cache for few query rows per KV head: single
// tokens, drafted tokens, short chunks.
//
// Mathematics.  The query rows of one KV head (tokens x heads of the group)
// are the columns of transposed products, so a group of 4 or 8 heads fills
// the N = 8 side of an MMA instead of a sixteenth of its M = 128 side:
//   S^T [16 keys x 8 rows] = K [16 x d] Q^T,   O^T [d_v x 8] += V^T [d_v x 16] P^T
// with the softmax's running maximum and sum per column (fp32, base 2).
//
// What bounds it: every K and V byte is read once from HBM and used for 8
// rows, 16 or 32 FLOP a byte, so the HBM rate (450 k keys of 8 heads in E4M3,
// 922 MB: 150 us, 6.1 TB/s); mma.sync runs far below its peak here and no
// tensor-memory round trip pays.  More rows are bound by the products and their
// softmax (16 x 4096 keys, 32 rows, E4M3: 80 us where the bytes take 20).
//
// Layout.  One warp takes 16 keys a step, alone: no barrier between warps
// until their states are joined.  A step's 16 slots of K and of V come by TMA
// into the warp's ring in shared memory, 64-128 KB of them on their way on each
// SM.  (With copies of 16 bytes a lane, 64 bytes of a K row together, the
// loads alone took 180 us.)  The order of dims inside S's sum and of rows
// inside V^T is free, so a lane's MMA fragments are whole 16-byte units, chosen
// so that eight lanes meet eight bank groups under the TMA's swizzle.
//   K: lane (g = lane / 4, t = lane % 4) holds keys g and g + 8, dims by t
//   V: lane (g, t) holds keys 2t, 2t+1, 2t+8, 2t+9, dims by g; pairs of keys
//      are interleaved by byte permutes (a transpose without shared memory)
//   P^T: the C fragment of S^T, rounded and transposed 8x8 (movmatrix), is
//      the B fragment of the second product.
// E4M3 codes become fp16 exactly; the K scale multiplies the scores, the V
// scale is added to them as its logarithm (P V s_v = 2^(s + log2 s_v) V) and
// taken out of the normaliser again, so both cost one multiply-add.
//
// Work split.  A tile is one step of each of a block's warps, of one (sequence,
// KV head, block of rows).  All tiles of the batch, in order, are cut into
// equal shares, one per block of a grid that fills the SMs: long and short
// sequences balance without a host-side plan, and a single sequence spreads
// over the whole chip.  A share that covers a whole item writes O; others write
// partial states (at most two a block), which a second kernel joins in a fixed
// order.
#pragma once
#include <climits>

#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

using sm103::ex2_approx;
using sm103::smem_u32;

template <int KIND, int DQK, int DV, int NT>
struct Cfg {
  static constexpr int kCb = KIND == kCacheE4m3 ? 1 : 2;
  static constexpr int kKch = DQK * kCb / 64;  // 16-byte units of K per lane and key
  static constexpr int kVb = DV * kCb / 8;     // bytes of V per lane and key
  // boxes of 16 slots, this many bytes wide, in the swizzle of that width
  static constexpr int kKw = DQK * kCb % 128 ? 64 : 128, kVw = DV * kCb % 128 ? 64 : 128;
  static constexpr int kStageK = 16 * DQK * kCb;
  static constexpr int kStageV = 16 * DV * kCb;
  static constexpr int kStage = kStageK + kStageV;
  // Steps a warp takes together: with one tile of rows a step is a chain of
  // dependent short operations, and two chains hide each other's latency (and
  // share the maximum's shuffles); more rows are independent work already.
  // (One step at a time from the same ring: 4 contexts of 100-131 k keys 155 us
  // against 150, 32 ragged ones 59 against 60, 256 short ones 32 against 32.6.)
  static constexpr int kTogether = NT == 1 ? 2 : 1;
  // blocks per SM: two where a stage is small, so that one streams while the
  // other joins its warps' states
  static constexpr int kBlocks = NT == 1 && kStage <= 4096 ? 2 : 1;
  static constexpr int kBudget = kBlocks == 2 ? 100 * 1024 : 200 * 1024;
  static constexpr int kKs = DQK / 16;  // K slices of S^T
  static constexpr int kMt = DV / 16;   // row tiles of O^T
  static constexpr int kRows = 8 * NT;
  // queries of more rows than registers hold, a copy for each warp
  static constexpr bool kQSmem = NT > 2;
  static constexpr int kQBytes = kQSmem ? NT * kKs * 256 : 0;
  // the steps in hand, and as many on their way
  static constexpr int kFitWarps = kBudget / (2 * kTogether * kStage + kQBytes);
  static constexpr int kWarps = kFitWarps > 8 ? 8 : kFitWarps;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTileKeys = 16 * kWarps;
  static constexpr int kFit = (kBudget - kWarps * kQBytes) / (kWarps * kStage);
  static constexpr int kStages = kFit > 4 * kTogether ? 4 * kTogether : kFit;
  static_assert(kStages >= 2 * kTogether && kWarps >= 4, "ring");
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = kWarps * 8 * DV * 4;
  static constexpr int kBody = (kRing > kMerge ? kRing : kMerge);
  static constexpr int kSmem = 1024 + kBody + kWarps * kQBytes;  // the ring starts at a multiple of 1024
};

__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four dims of slice ks that lane t holds, in the order of its 16-byte units
// (two neighbouring ones of each 128-byte box, or one of each 64-byte box).
template <class C>
__device__ __forceinline__ constexpr int k_dim(int ks, int t) {
  constexpr int kE = 16 / C::kCb, kPer = kE / 4;  // elements, slices of a unit
  const int c = ks / kPer;
  return (C::kKw == 128 ? (c / 2) * (8 * kE) + (2 * t + c % 2) * kE : c * (4 * kE) + t * kE) +
         4 * (ks % kPer);
}

// An item costs its tiles and about as much as this many more (its queries, a
// pipeline to fill, a state to join): shares are cut by that sum.
constexpr int kStart = 3;

// What a sequence asks for: row blocks, first key, end.
struct Need {
  Seq q;
  int nrb, k0, hi;
  __device__ __forceinline__ int tiles(int tile_keys) const {
    return max(1, (hi - k0 + tile_keys - 1) / tile_keys);
  }
};
__device__ __forceinline__ Need need_of(const Args& a, int s, int rows_per) {
  Need d;
  d.q = load_seq(a, s);
  const int cap = a.max_pages << a.page_shift;
  d.hi = min(d.q.len, cap);
  int lo = 0;
  if (a.window >= 0) lo = max(0, d.q.len - d.q.n - a.window);
  d.k0 = lo & ~15;
  d.nrb = (d.q.n * a.group + rows_per - 1) / rows_per;
  return d;
}

// A block's or a warp's share of the batch: units [begin, end) of all, the
// first one unit `off` of sequence `s`.
struct Share {
  int64_t off, begin, end, total;
  int64_t base;  // units of a share; the first `more` shares have one more
  int s, more;
  bool solo;
  __device__ __forceinline__ int64_t start(int64_t k) const {
    return k * base + (k < more ? k : more);
  }
  // the share that unit x is in
  __device__ __forceinline__ int of(int64_t x) const {
    const int64_t cut = more * (base + 1);
    return static_cast<int>(x < cut ? x / (base + 1) : more + (x - cut) / base);
  }
};

// Every thread of the block (solo: of the warp) returns the same values.
//
// Solo: a warp takes whole items alone and nothing is joined.  That is the
// better half where no item is much larger than a warp's average share (many
// short sequences: 256 of up to 256 keys take 62 us when a block's warps share
// each item, 33 us so); otherwise blocks share items, cut anywhere.
template <class C>
__device__ __forceinline__ Share find_share(const Args& a) {
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  __shared__ int64_t s_sum[2][kWarps], s_off[kWarps];
  __shared__ int s_max[kWarps], s_seq[kWarps];
  const int w = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int first = threadIdx.x * per, last = min(a.num_seqs, first + per);
  int64_t mine[2] = {0, 0}, sum[2];
  int most = 0;
  for (int s = first; s < last; ++s) {
    const Need d = need_of(a, s, C::kRows);
    if (outside(a, d.q)) flag_bounds(a);
    const int64_t items = static_cast<int64_t>(d.nrb) * a.Hkv;
    const int steps = d.tiles(16);
    mine[0] += items * (kStart + d.tiles(C::kTileKeys));
    mine[1] += items * (kStart + steps);
    if (items) most = max(most, kStart + steps);
  }
  sum[0] = mine[0];
  sum[1] = mine[1];
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t y0 = __shfl_up_sync(0xffffffffu, sum[0], i);
    const int64_t y1 = __shfl_up_sync(0xffffffffu, sum[1], i);
    if (lane >= i) {
      sum[0] += y0;
      sum[1] += y1;
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    s_sum[0][w] = sum[0];
    s_sum[1][w] = sum[1];
    s_max[w] = most;
  }
  __syncthreads();
  int64_t total[2] = {0, 0}, before[2] = {sum[0] - mine[0], sum[1] - mine[1]};
#pragma unroll
  for (int x = 0; x < kWarps; ++x) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (x < w) before[m] += s_sum[m][x];
      total[m] += s_sum[m][x];
    }
    most = max(most, s_max[x]);
  }
  Share sh;
  sh.solo = static_cast<int64_t>(most) * gridDim.x * kWarps <= 2 * total[1];
  sh.total = total[sh.solo];
  const int64_t lo = before[sh.solo], hi = lo + mine[sh.solo];
  const int workers =
      static_cast<int>(min(static_cast<int64_t>(gridDim.x) * (sh.solo ? kWarps : 1), sh.total));
  const int me = sh.solo ? blockIdx.x * kWarps + w : blockIdx.x;
  sh.base = 0;
  sh.more = 0;
  if (workers > 0) {
    sh.base = (sh.total >> 31) ? sh.total / workers
                               : static_cast<uint32_t>(sh.total) / static_cast<uint32_t>(workers);
    sh.more = static_cast<int>(sh.total - sh.base * workers);
  }
#pragma unroll 1
  for (int x = 0; x < (sh.solo ? kWarps : 1); ++x) {
    const int k = sh.solo ? blockIdx.x * kWarps + x : blockIdx.x;
    if (k >= workers) break;
    const int64_t begin = sh.start(k);
    if (begin >= lo && begin < hi) {
      int s = first;
      int64_t off = begin - lo;
      for (;; ++s) {
        const Need d = need_of(a, s, C::kRows);
        const int64_t c = static_cast<int64_t>(d.nrb) * a.Hkv *
                          (kStart + d.tiles(sh.solo ? 16 : C::kTileKeys));
        if (off < c) break;
        off -= c;
      }
      s_seq[x] = s;
      s_off[x] = off;
    }
  }
  __syncthreads();
  sh.begin = sh.end = 0;
  if (me < workers) {
    sh.begin = sh.start(me);
    sh.end = sh.start(me + 1);
  }
  sh.s = s_seq[sh.solo ? w : 0];
  sh.off = s_off[sh.solo ? w : 0];
  return sh;
}

template <int KIND, int DQK, int DV, int NT>
__global__ void __launch_bounds__(Cfg<KIND, DQK, DV, NT>::kThreads, Cfg<KIND, DQK, DV, NT>::kBlocks)
    decode_kernel(const __grid_constant__ Args a, const __grid_constant__ CacheMaps maps) {
  using C = Cfg<KIND, DQK, DV, NT>;
  constexpr bool kBf = KIND == kCacheBf16;
  constexpr int kWarps = C::kWarps, U = C::kTogether;
  // fp16 P is kept at up to 2^14 so that weights down to 2^-28 of the row's
  // largest are normal numbers
  constexpr float kShift = kBf ? 0.f : 14.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
  const int tid = threadIdx.x, w = tid / 32, lane = tid & 31, g = lane >> 2, t = lane & 3;
  // a barrier for each warp's each stage
  __shared__ uint64_t s_full[kWarps][C::kStages];
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) sm103::mbar_init(&s_full[w][i], 1);
    sm103::mbar_fence_init();
    sm103::prefetch_tensormap(&maps.k);
    sm103::prefetch_tensormap(&maps.v);
  }
  sm103::grid_dep_wait();
  const Share sh = find_share<C>(a);
  if (tid == 0 && a.split_desc) a.split_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  sm103::grid_dep_launch();  // the joining kernel may be put in place
  if (sh.begin >= sh.end) return;

  uint8_t* const body = smem + (-smem_u32(smem) & 1023u);
  const uint32_t ring = smem_u32(body) + w * (C::kStages * C::kStage);
  const uint32_t qs = smem_u32(body) + C::kBody + w * C::kQBytes;
  float* const s_o = reinterpret_cast<float*>(body);
  // the ring runs on from item to item: stage and phase of the next copy, and
  // of the next step to compute
  int in_stage = 0, out_stage = 0;
  uint32_t out_phase = 0;
  bool dead = false;
  const int page_mask = (1 << a.page_shift) - 1;

  // the warps that share an item, and this one among them
  const int nw = sh.solo ? 1 : kWarps, wi = sh.solo ? 0 : w;
  const int tile_keys = 16 * nw;
  int seq = sh.s;
  int64_t off = sh.off, at = sh.begin;
  Need nd = need_of(a, seq, C::kRows);
  while (at < sh.end) {
    const int tiles = nd.tiles(tile_keys), cost = kStart + tiles;
    if (off >= static_cast<int64_t>(nd.nrb) * a.Hkv * cost) {
      off -= static_cast<int64_t>(nd.nrb) * a.Hkv * cost;
      nd = need_of(a, ++seq, C::kRows);
      continue;
    }
    const int item = static_cast<int>((off >> 31) ? off / cost
                                                  : static_cast<uint32_t>(off) / static_cast<uint32_t>(cost));
    const int u0 = static_cast<int>(off - static_cast<int64_t>(item) * cost);
    // units [u0, u1): an item's start, then its tiles [t0, t1)
    const int u1 = sh.solo ? cost
                           : static_cast<int>(min(static_cast<int64_t>(cost), u0 + (sh.end - at)));
    const int t0 = max(0, u0 - kStart), t1 = max(0, u1 - kStart);
    const int64_t here = at;
    at += u1 - u0;
    off += u1 - u0;
    // solo, an item is its first unit's; a share may end inside a start
    if (sh.solo ? u0 > 0 : t1 <= t0) continue;
    const int hk = item / nd.nrb, rb = item % nd.nrb;
    const int rows = nd.q.n * a.group, r0 = rb * C::kRows;
    const int pos0 = nd.q.len - nd.q.n;  // position of the sequence's first new row
    const int tok_lo = div_group(a, r0), tok_hi = div_group(a, min(rows - 1, r0 + C::kRows - 1));
    // keys some row of the block keeps, and keys all of them keep
    const int klo = a.window >= 0 ? max(0, pos0 + tok_lo - a.window) : 0;
    const int khi = a.causal ? min(nd.hi, pos0 + tok_hi + 1) : nd.hi;
    const int all_lo = a.window >= 0 ? max(0, pos0 + tok_hi - a.window) : 0;
    const int all_hi = a.causal ? min(nd.hi, pos0 + tok_lo + 1) : nd.hi;
    // this piece's 16-key steps
    const int b_lo = max(nd.k0 + t0 * tile_keys, klo) >> 4;
    const int b_hi = (min(nd.k0 + t1 * tile_keys, khi) + 15) >> 4;
    const int ns = b_hi - b_lo > wi ? (b_hi - b_lo - wi + nw - 1) / nw : 0;

    // ---- page ids and scales: lane i holds those of step (window * 32 + i).
    // Ids are read two windows of 32 steps ahead and scales one, so that no
    // load waits for another in the loop.
    auto load_ids = [&](int window) -> int {
      const int i = window * 32 + lane;
      if (i >= ns) return -1;
      const int col = (b_lo + wi + nw * i) >> (a.page_shift - 4);
      int id = col < a.max_pages ? a.table[seq * a.table_stride + col] : -1;
      if (id < 0 || id >= a.num_pages) {
        flag_bounds(a);
        id = -1;
      }
      return id;
    };
    struct Scales {
      float k, v;
    };
    auto load_scales = [&](int id) -> Scales {
      Scales r = {1.f, 1.f};
      if (KIND == kCacheE4m3 && id >= 0) {
        r.k = a.k_scale[static_cast<int64_t>(id) * a.Hkv + hk];
        r.v = fmaxf(a.v_scale[static_cast<int64_t>(id) * a.Hkv + hk], kMinVScale);
      }
      return r;
    };
    int ids = load_ids(0), ids1 = ns > 32 ? load_ids(1) : -1, ids2 = ns > 64 ? load_ids(2) : -1;
    Scales sc = load_scales(ids), sc1 = load_scales(ids1);
    // of the window being computed: K scale, log2 of the V scale, its inverse,
    // and whether the page exists
    float w_k = 1.f, w_lg = 0.f, w_inv = 1.f;
    int w_id = ids;
    // Step i's 16 slots of K and V, by TMA: whole boxes, whatever the mask
    // keeps of them; nothing where there is no page.
    auto issue = [&](int i) {
      if (i >= ns || dead) return;
      if (i > 0 && (i & 31) == 0) {
        ids = ids1;
        ids1 = ids2;
        ids2 = load_ids((i >> 5) + 2);
      }
      const int page = __shfl_sync(0xffffffffu, ids, i & 31);
      if (lane == 0) {
        uint64_t* const bar = &s_full[w][in_stage];
        if (page >= 0) {
          const int slot = ((b_lo + wi + nw * i) << 4) & page_mask;
          const uint32_t dst = ring + in_stage * C::kStage;
          sm103::mbar_arrive_expect_tx(bar, C::kStage);
#pragma unroll
          for (int c = 0; c < DQK * C::kCb / C::kKw; ++c)
            tma_load_4d(dst + c * 16 * C::kKw, &maps.k, bar, c * C::kKw / C::kCb, slot, hk, page);
#pragma unroll
          for (int c = 0; c < DV * C::kCb / C::kVw; ++c)
            tma_load_4d(dst + C::kStageK + c * 16 * C::kVw, &maps.v, bar, c * C::kVw / C::kCb, slot,
                        hk, page);
        } else {
          sm103::mbar_arrive(bar);
        }
      }
      in_stage = in_stage + 1 == C::kStages ? 0 : in_stage + 1;
    };
#pragma unroll
    for (int i = 0; i < C::kStages - U; ++i) issue(i);

    // ---- queries: column g of each tile as B fragments; factors of columns
    // 2t and 2t + 1 (base-2 softmax scale, and the row's power of two)
    uint32_t qf[C::kQSmem ? 1 : NT][C::kKs][2];
    float fac[NT][2];
    int cpos[NT][2];  // positions of columns 2t and 2t + 1 (INT_MIN: no row)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g;
      const bool real = r < rows;
      const uint16_t* qp = a.q;
      if (real) {
        const int tok = div_group(a, r);
        qp += (nd.q.row0 + tok) * a.q_stride + (hk * a.group + r - tok * a.group) * DQK;
      }
      uint32_t raw[C::kKs][2];
#pragma unroll
      for (int ks = 0; ks < C::kKs; ++ks) {
        const int d = k_dim<C>(ks, t);
        uint2 v = make_uint2(0, 0);
        if (real) v = *reinterpret_cast<const uint2*>(qp + d);
        raw[ks][0] = v.x;
        raw[ks][1] = v.y;
      }
      float back = 1.f;
      if (KIND == kCacheE4m3 && !a.f16) {
        // bf16 row to fp16: its largest element to [2^14, 2^15)
        uint32_t mx = 0;
#pragma unroll
        for (int ks = 0; ks < C::kKs; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx = max(mx, max(raw[ks][i] & 0x7fffu, (raw[ks][i] >> 16) & 0x7fffu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int e = static_cast<int>(mx >> 7);  // biased exponent
        e = e == 255 ? 127 + 14 : max(e, 27);
        const float to = __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
        back = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
        for (int ks = 0; ks < C::kKs; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            raw[ks][i] = sm103::pack_f16x2(__uint_as_float(raw[ks][i] << 16) * to,
                                           __uint_as_float(raw[ks][i] & 0xffff0000u) * to);
      }
      if constexpr (C::kQSmem) {
        // (a lane reads back what it wrote itself)
#pragma unroll
        for (int ks = 0; ks < C::kKs; ++ks)
          asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(qs + (nt * C::kKs + ks) * 256 +
                                                              lane * 8),
                       "r"(raw[ks][0]), "r"(raw[ks][1])
                       : "memory");
      } else {
#pragma unroll
        for (int ks = 0; ks < C::kKs; ++ks) {
          qf[nt][ks][0] = raw[ks][0];
          qf[nt][ks][1] = raw[ks][1];
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fac[nt][c] = a.scale * kLog2e * __shfl_sync(0xffffffffu, back, (2 * t + c) * 4);
        const int rr = r0 + nt * 8 + 2 * t + c;
        cpos[nt][c] = rr < rows ? pos0 + div_group(a, rr) : INT_MIN;
      }
    }

    float o[NT][C::kMt][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    auto kept = [&](int nt, int c, int key) -> bool {
      const int p = cpos[nt][c];
      return p != INT_MIN && key < nd.hi && (!a.causal || key <= p) &&
             (a.window < 0 || key >= p - a.window);
    };

    // this lane's places in a stage: K rows g (and g + 8, 8 rows on) for its
    // units of a box, V rows 2t, 2t + 1 (and 8 rows on)
    uint32_t k_at[2], v_at[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      k_at[c] = C::kKw == 128 ? g * 128 + (((2 * t + c) ^ g) << 4) : g * 64 + ((t ^ (g >> 1)) << 4);
      v_at[c] = C::kStageK + (C::kVw == 128 ? (2 * t + c) * 128 + ((g ^ (2 * t + c)) << 4)
                                            : (2 * t + c) * 64 + (((g >> 1) ^ t) << 4) + 8 * (g & 1));
    }
    for (int i = 0; i < ns; i += U) {
      if ((i & 31) == 0) {  // a new window; copies are less than one ahead
        w_id = ids;
        if (i > 0) {
          sc = sc1;
          sc1 = load_scales(ids1);
        }
        w_k = sc.k;
        w_inv = 1.f / sc.v;
        w_lg = (__float_as_uint(sc.v) & 0x7fffffu) == 0
                   ? static_cast<float>(static_cast<int>(__float_as_uint(sc.v) >> 23) - 127)
                   : __log2f(sc.v);
      }
      const bool two = U == 1 || i + 1 < ns;  // the second step exists
      uint32_t at_stage[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        at_stage[x] = ring + out_stage * C::kStage;
        if (x > 0 && !two) break;
        if (!dead && !sm103::mbar_wait_warp(&s_full[w][out_stage], out_phase)) {
          if (a.status) *a.status = ATTN_ERR_DEVICE_TIMEOUT;
          dead = true;
        }
        if (++out_stage == C::kStages) {
          out_stage = 0;
          out_phase ^= 1;
        }
      }
      __syncwarp();  // the stages filled next are read by every lane
#pragma unroll
      for (int x = 0; x < U; ++x) issue(i + C::kStages - U + x);

      // S^T
      float s[U][NT][4];
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[x][nt][j] = 0.f;
#pragma unroll
      for (int c = 0; c < C::kKch; ++c) {
#pragma unroll
        for (int x = 0; x < U; ++x) {
          // (a second step that does not exist multiplies what its stage held;
          // its scores are masked)
          constexpr int kBox = 16 * C::kKw;
          const uint32_t from =
              at_stage[x] + (C::kKw == 128 ? (c / 2) * kBox + k_at[c & 1] : c * kBox + k_at[0]);
          const uint4 x0 = lds128(from), x1 = lds128(from + 8 * C::kKw);
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
          constexpr int kPer = KIND == kCacheE4m3 ? 4 : 2;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int ks = c * kPer + j;
            uint32_t a0, a1, a2, a3;
            if constexpr (KIND == kCacheE4m3) {
              a0 = e4m3x2_f16x2(static_cast<uint16_t>(w0[j]));
              a2 = e4m3x2_f16x2(static_cast<uint16_t>(w0[j] >> 16));
              a1 = e4m3x2_f16x2(static_cast<uint16_t>(w1[j]));
              a3 = e4m3x2_f16x2(static_cast<uint16_t>(w1[j] >> 16));
            } else {
              a0 = w0[2 * j];
              a2 = w0[2 * j + 1];
              a1 = w1[2 * j];
              a3 = w1[2 * j + 1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (C::kQSmem) {
                const uint2 b = lds64(qs + (nt * C::kKs + ks) * 256 + lane * 8);
                mma16816<kBf>(s[x][nt], a0, a1, a2, a3, b.x, b.y);
              } else {
                mma16816<kBf>(s[x][nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
              }
            }
          }
        }
      }

      // softmax in base 2; with E4M3 pages the exponent carries log2 of the V
      // scale and the sum takes it out
      float ksc[U], lgv[U], inv_v[U];
      bool okp[U], whole[U];
      int key[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int from = (i + x) & 31;
        key[x] = (b_lo + wi + nw * (i + x)) << 4;
        okp[x] = (x == 0 || two) && __shfl_sync(0xffffffffu, w_id, from) >= 0;
        whole[x] = okp[x] && key[x] >= all_lo && key[x] + 16 <= all_hi;
        ksc[x] = inv_v[x] = 1.f;
        lgv[x] = 0.f;
        if (KIND == kCacheE4m3) {
          ksc[x] = __shfl_sync(0xffffffffu, w_k, from);
          lgv[x] = __shfl_sync(0xffffffffu, w_lg, from);
          inv_v[x] = __shfl_sync(0xffffffffu, w_inv, from);
        }
      }
      uint32_t pb[U][NT][2];
      bool moved = false;
      float al[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[U][4];
#pragma unroll
        for (int x = 0; x < U; ++x) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            p[x][j] = fmaf(s[x][nt][j], fac[nt][j & 1] * ksc[x], lgv[x]);
          if (!whole[x]) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!okp[x] || !kept(nt, j & 1, key[x] + g + 8 * (j >> 1))) p[x][j] = -INFINITY;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(p[0][c], p[0][2 + c]);
          if constexpr (U == 2) mx = sm103::fmax3(mx, p[U - 1][c], p[U - 1][2 + c]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(mx, m[nt][c]);
          const float mu = mx == -INFINITY ? 0.f : mx;
          al[nt][c] = ex2_approx(m[nt][c] - mu);
          moved |= mx != m[nt][c];
          m[nt][c] = mx;
          l[nt][c] *= al[nt][c];
#pragma unroll
          for (int x = 0; x < U; ++x) {
            p[x][c] = ex2_approx(p[x][c] - mu + kShift);
            p[x][2 + c] = ex2_approx(p[x][2 + c] - mu + kShift);
            l[nt][c] = fmaf(p[x][c] + p[x][2 + c], inv_v[x], l[nt][c]);
          }
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
          if constexpr (kBf) {
            pb[x][nt][0] = movmatrix(sm103::pack_bf16x2(p[x][0], p[x][1]));
            pb[x][nt][1] = movmatrix(sm103::pack_bf16x2(p[x][2], p[x][3]));
          } else {
            pb[x][nt][0] = movmatrix(sm103::pack_f16x2(p[x][0], p[x][1]));
            pb[x][nt][1] = movmatrix(sm103::pack_f16x2(p[x][2], p[x][3]));
          }
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][mt][j] *= al[nt][j & 1];
      }

#pragma unroll
      for (int x = 0; x < U; ++x) {
        if (x > 0 && !two) break;  // weights of 0 do not undo a NaN of an old stage
      // V: four keys, a dim pair per row tile
      constexpr int kW = C::kVb / 4;  // words per key
      uint32_t v[4][kW];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t src = at_stage[x] + v_at[j & 1] + (j >> 1) * 8 * C::kVw;
        if constexpr (C::kVb == 8) {
          const uint2 q = lds64(src);
          v[j][0] = q.x;
          v[j][1] = q.y;
        } else {
#pragma unroll
          for (int c = 0; c < C::kVb / 16; ++c) {
            const uint4 q = lds128(src + c * 16 * C::kVw);
            v[j][4 * c] = q.x;
            v[j][4 * c + 1] = q.y;
            v[j][4 * c + 2] = q.z;
            v[j][4 * c + 3] = q.w;
          }
        }
        if (!whole[x]) {  // what lies in slots that no row keeps, NaN included
          const int kk = key[x] + 2 * t + (j & 1) + 8 * (j >> 1);
          if (!okp[x] || kk < klo || kk >= khi) {
#pragma unroll
            for (int z = 0; z < kW; ++z) v[j][z] = 0;
          }
        }
      }
      // A step that some rows keep in part: values that are not finite may
      // not meet the zero weights of rows that mask them.  They are taken out
      // of the product and added to the rows that keep them.
      if (!whole[x] && tok_lo != tok_hi) {
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int z = 0; z < kW; ++z) bad |= not_finite<KIND>(v[j][z]);
        if (__any_sync(0xffffffffu, bad != 0)) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int z = 0; z < kW; ++z) v[j][z] = finite_only<KIND>(v[j][z]);
          for (int r = 0; r < 16; ++r) {
            if (!okp[x] || key[x] + r < klo || key[x] + r >= khi) continue;
            const uint32_t row = at_stage[x] + C::kStageK + r * C::kVw;
#pragma unroll
            for (int e = 0; e < 2 * C::kMt; ++e) {  // this lane's dims
              const int byte = e * C::kCb;
              const uint32_t src =
                  C::kVb == 8 ? row + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + 8 * (g & 1) + byte
                              : row + (byte / 16) * 16 * C::kVw + ((g ^ (r & 7)) << 4) + byte % 16;
              float y;
              if constexpr (KIND == kCacheE4m3) {
                uint32_t b;
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(src) : "memory");
                y = e4m3_value(static_cast<uint8_t>(b));
              } else {
                uint16_t b;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(src) : "memory");
                y = elem(b, KIND == kCacheF16);
              }
              if (!(fabsf(y) < INFINITY)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 2; ++c)
                    if (kept(nt, c, key[x] + r)) o[nt][e / 2][2 * (e & 1) + c] += y;
              }
            }
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < C::kMt; ++mt) {
        uint32_t a0, a1, a2, a3;
        if constexpr (KIND == kCacheE4m3) {
          const uint32_t sel = (mt & 1) ? 0x7362 : 0x5140;
          const uint32_t lo = __byte_perm(v[0][mt / 2], v[1][mt / 2], sel);
          const uint32_t hi = __byte_perm(v[2][mt / 2], v[3][mt / 2], sel);
          a0 = e4m3x2_f16x2(static_cast<uint16_t>(lo));
          a1 = e4m3x2_f16x2(static_cast<uint16_t>(lo >> 16));
          a2 = e4m3x2_f16x2(static_cast<uint16_t>(hi));
          a3 = e4m3x2_f16x2(static_cast<uint16_t>(hi >> 16));
        } else {
          a0 = __byte_perm(v[0][mt], v[1][mt], 0x5410);
          a1 = __byte_perm(v[0][mt], v[1][mt], 0x7632);
          a2 = __byte_perm(v[2][mt], v[3][mt], 0x5410);
          a3 = __byte_perm(v[2][mt], v[3][mt], 0x7632);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816<kBf>(o[nt][mt], a0, a1, a2, a3, pb[x][nt][0], pb[x][nt][1]);
      }
      }
    }

    // ---- join the warps' states.  A column's 16-byte groups are permuted in
    // shared memory so that the eight lanes of a store (two g, four t) meet
    // eight different bank groups.
    auto swz = [](int col) -> int {
      const int x = (col >> 1) & 3;
      return DV == 128 && KIND == kCacheE4m3 ? x : (x & 1) | ((x >> 1) << 2);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[nt][c] = x;
        if (g == 0) {
          s_m[w][nt * 8 + 2 * t + c] = m[nt][c];
          s_l[w][nt * 8 + 2 * t + c] = x;
        }
      }
    if (sh.solo) {
      // the warp's own state is the item's
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = r0 + nt * 8 + 2 * t + c;
          if (r >= rows) continue;
          const int tok = div_group(a, r), head = hk * a.group + r - tok * a.group;
          const bool none = no_key(m[nt][c], l[nt][c]);
          float mt = m[nt][c], lt = l[nt][c], keep = 1.f;
          if (a.sink) {
            const float s2 = a.sink[head] * kLog2e;
            mt = fmaxf(mt, s2);
            const float mu = mt == -INFINITY ? 0.f : mt;
            keep = ex2_approx(m[nt][c] - mu);
            lt = fmaf(lt, keep, ex2_approx(s2 - mu + kShift));
          }
          const float inv = none || lt == 0.f ? 0.f : keep / lt;
          uint16_t* const op = a.o + (static_cast<int64_t>(nd.q.row0 + tok) * a.Hq + head) * DV;
#pragma unroll
          for (int e = 0; e < 2 * C::kMt; e += 8) {  // eight dims a store
            const int d = KIND == kCacheE4m3 ? C::kVb * g + e : 64 * (e / 8) + 8 * g;
            auto at_dim = [&](int z) { return none ? 0.f : o[nt][z / 2][2 * (z & 1) + c] * inv; };
            *reinterpret_cast<uint4*>(op + d) =
                make_uint4(pack2(at_dim(e), at_dim(e + 1), a.f16),
                           pack2(at_dim(e + 2), at_dim(e + 3), a.f16),
                           pack2(at_dim(e + 4), at_dim(e + 5), a.f16),
                           pack2(at_dim(e + 6), at_dim(e + 7), a.f16));
          }
          if (a.lse && g == 0)
            a.lse[static_cast<int64_t>(head) * a.num_tokens + nd.q.row0 + tok] =
                none ? (a.sink ? a.sink[head] : -INFINITY) : (mt - kShift) * kLn2 + logf(lt);
        }
      __syncwarp();
      continue;
    }
    const bool complete = t0 == 0 && t1 == tiles;
    const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      __syncthreads();  // the ring, or the previous tile's sums, are read
#pragma unroll
      for (int i = 0; i < DV / 32; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int q4 = DV == 64               ? 2 * g + i
                         : KIND == kCacheE4m3 ? 4 * g + i
                                              : (i / 2) * 16 + 2 * g + (i & 1);
          const int col = 2 * t + c;
          *reinterpret_cast<float4*>(s_o + (w * 8 + col) * DV + (q4 ^ swz(col)) * 4) =
              make_float4(o[nt][2 * i][c], o[nt][2 * i][2 + c], o[nt][2 * i + 1][c],
                          o[nt][2 * i + 1][2 + c]);
        }
      __syncthreads();
      constexpr int kV = DV / 32;  // dims per lane; one warp a column at a time
      for (int cw = w; cw < 8; cw += kWarps) {
        const int r = r0 + nt * 8 + cw;
        if (r >= rows) break;
        float mt_ = -INFINITY;
        bool none = true;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float mx = s_m[x][nt * 8 + cw];
          mt_ = fmaxf(mt_, mx);
          none &= no_key(mx, s_l[x][nt * 8 + cw]);
        }
        const int tok = div_group(a, r), head = hk * a.group + r - tok * a.group;
        float snk = -INFINITY;
        if (complete && a.sink) {
          snk = a.sink[head] * kLog2e;
          mt_ = fmaxf(mt_, snk);
        }
        const float mu = mt_ == -INFINITY ? 0.f : mt_;
        float lt = complete && a.sink ? ex2_approx(snk - mu + kShift) : 0.f;
        float acc[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float mx = s_m[x][nt * 8 + cw];
          if (no_key(mx, s_l[x][nt * 8 + cw])) continue;  // nothing kept by this warp
          const float f = ex2_approx(mx - mu);
          lt = fmaf(s_l[x][nt * 8 + cw], f, lt);
          const float* so = s_o + (x * 8 + cw) * DV +
                            (kV == 4 ? (lane ^ swz(cw)) * 4
                                     : ((lane >> 1) ^ swz(cw)) * 4 + 2 * (lane & 1));
#pragma unroll
          for (int i = 0; i < kV; ++i) acc[i] = fmaf(so[i], f, acc[i]);
        }
        if (complete) {
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
          uint16_t* op = a.o + (static_cast<int64_t>(nd.q.row0 + tok) * a.Hq + head) * DV + lane * kV;
          if constexpr (kV == 4)
            *reinterpret_cast<uint2*>(op) = make_uint2(pack2(acc[0] * inv, acc[1] * inv, a.f16),
                                                       pack2(acc[2] * inv, acc[3] * inv, a.f16));
          else
            *reinterpret_cast<uint32_t*>(op) = pack2(acc[0] * inv, acc[1] * inv, a.f16);
          if (a.lse && lane == 0)
            a.lse[static_cast<int64_t>(head) * a.num_tokens + nd.q.row0 + tok] =
                none ? (a.sink ? a.sink[head] : -INFINITY) : (mu - kShift) * kLn2 + logf(lt);
        } else {
          float* pp = a.part + (static_cast<int64_t>(slot) * a.part_rows + nt * 8 + cw) * DV + lane * kV;
#pragma unroll
          for (int i = 0; i < kV; ++i) pp[i] = acc[i];
          if (lane == 0)
            a.part_ml[static_cast<int64_t>(slot) * a.part_rows + nt * 8 + cw] =
                make_float2(mt_, lt);
        }
      }
    }
    if (!complete && t0 == 0 && tid == 0) {
      // first of an item's pieces: blocks up to the one that holds its last tile
      const int64_t end = here + cost - u0;  // of the item's units
      a.split_desc[blockIdx.x] = make_int4(sh.of(end - 1) - blockIdx.x + 1, seq, hk, rb);
    }
    sm103::fence_proxy_async_smem();
    __syncthreads();  // the sums are read before the next piece's copies fill the ring
  }
  if (dead)  // copies in flight land before the block may leave
    for (int i = 0; i < C::kStages; ++i) sm103::mbar_wait(&s_full[w][i], out_phase, 100000000ull);
}

// Joins the pieces of each split item: block (i, y) rows 2y and 2y + 1 of the
// item whose first piece is block i's, four warps a row.
template <int DV>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a, float shift) {
  __shared__ float s_acc[2][4][DV], s_m[2][4], s_l[2][4];
  sm103::grid_dep_wait();
  const int4 d = a.split_desc[blockIdx.x];
  if (d.x == 0) return;
  const int w = threadIdx.x / 32, lane = threadIdx.x & 31, rr = w / 4, part = w & 3;
  const Seq q = load_seq(a, d.y);
  const int col = 2 * blockIdx.y + rr, r = d.w * a.part_rows + col, rows = q.n * a.group;
  constexpr int kV = DV / 32;
  float acc[kV], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
  if (r < rows) {
#pragma unroll 4
    for (int i = part; i < d.x; i += 4) {
      const int64_t slot = 2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0);
      const float2 ml = a.part_ml[slot * a.part_rows + col];
      const float* pp = a.part + (slot * a.part_rows + col) * DV + lane * kV;
      float x[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) x[j] = pp[j];
      const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2_approx(m - mu), f1 = ex2_approx(ml.x - mu);
      // a state without keys holds zeros
#pragma unroll
      for (int j = 0; j < kV; ++j) acc[j] = acc[j] * f0 + x[j] * f1;
      l = l * f0 + ml.y * f1;
      m = mn;
    }
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) s_acc[rr][part][lane * kV + j] = acc[j];
  if (lane == 0) {
    s_m[rr][part] = m;
    s_l[rr][part] = l;
  }
  __syncthreads();
  if (part != 0 || r >= rows) return;
  const int tok = div_group(a, r), head = d.z * a.group + r - tok * a.group;
  float mt = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) mt = fmaxf(mt, s_m[rr][i]);
  bool none = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) none &= no_key(s_m[rr][i], s_l[rr][i]);
  if (a.sink) mt = fmaxf(mt, a.sink[head] * kLog2e);
  const float mu = mt == -INFINITY ? 0.f : mt;
  float lt = a.sink ? ex2_approx(a.sink[head] * kLog2e - mu + shift) : 0.f;
#pragma unroll
  for (int j = 0; j < kV; ++j) acc[j] = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = ex2_approx(s_m[rr][i] - mu);
    lt = fmaf(s_l[rr][i], f, lt);
#pragma unroll
    for (int j = 0; j < kV; ++j) acc[j] = fmaf(s_acc[rr][i][lane * kV + j], f, acc[j]);
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  uint16_t* op = a.o + (static_cast<int64_t>(q.row0 + tok) * a.Hq + head) * DV + lane * kV;
  if constexpr (kV == 4)
    *reinterpret_cast<uint2*>(op) = make_uint2(pack2(acc[0] * inv, acc[1] * inv, a.f16),
                                               pack2(acc[2] * inv, acc[3] * inv, a.f16));
  else
    *reinterpret_cast<uint32_t*>(op) = pack2(acc[0] * inv, acc[1] * inv, a.f16);
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(head) * a.num_tokens + q.row0 + tok] =
        none ? (a.sink ? a.sink[head] : -INFINITY) : (mu - shift) * kLn2 + logf(lt);
}

template <int KIND, int DQK, int DV, int NT>
cudaError_t launch_one(const Args& a0, int sms, cudaStream_t st) {
  using C = Cfg<KIND, DQK, DV, NT>;
  Args a = a0;
  auto kern = decode_kernel<KIND, DQK, DV, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // as many blocks as can be resident, or as there can be tiles
  const int64_t most = (static_cast<int64_t>(a.max_pages) << a.page_shift) + C::kTileKeys - 1;
  const int64_t tiles = most / C::kTileKeys + 1;
  const int64_t items =
      (static_cast<int64_t>(a.num_tokens) * a.group / C::kRows + a.num_seqs) * a.Hkv;
  int64_t ctas = static_cast<int64_t>(sms) * C::kBlocks;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  if (tiles < ctas && items * tiles < ctas) ctas = items * tiles;
  a.part_rows = C::kRows;
  const bool split = (static_cast<int64_t>(a.max_pages) << a.page_shift) > C::kTileKeys;
  if (!split) a.split_desc = nullptr;
  CacheMaps maps;
  if (!cache_map(&maps.k, KIND, a.kc, DQK, a, a.k_tok, a.k_head, a.k_page, 16, C::kKw, C::kKw) ||
      !cache_map(&maps.v, KIND, a.vc, DV, a, a.v_tok, a.v_head, a.v_page, 16, C::kVw, C::kVw))
    return cudaErrorInvalidValue;
  e = launch_early(kern, dim3(static_cast<unsigned>(ctas)), dim3(C::kThreads), C::kSmem, st, a,
                   maps);
  if (e != cudaSuccess || !split) return e;
  return launch_early(join_kernel<DV>, dim3(static_cast<unsigned>(ctas), C::kRows / 2), dim3(256),
                      0, st, a, KIND == kCacheBf16 ? 0.f : 14.f);
}

template <int KIND, int DQK, int DV>
cudaError_t launch_rows(const Args& a, int rows, int sms, cudaStream_t st) {
  if (rows <= 8) return launch_one<KIND, DQK, DV, 1>(a, sms, st);
  if (rows <= 16) return launch_one<KIND, DQK, DV, 2>(a, sms, st);
  if (rows <= 24) return launch_one<KIND, DQK, DV, 3>(a, sms, st);
  return launch_one<KIND, DQK, DV, 4>(a, sms, st);
}

template <int KIND>
cudaError_t launch_dims(const Args& a, int rows, int sms, cudaStream_t st) {
  if (a.d_v == 64) {
    if (a.d_qk == 64) return launch_rows<KIND, 64, 64>(a, rows, sms, st);
    if (a.d_qk == 128) return launch_rows<KIND, 128, 64>(a, rows, sms, st);
    return launch_rows<KIND, 192, 64>(a, rows, sms, st);
  }
  if (a.d_qk == 64) return launch_rows<KIND, 64, 128>(a, rows, sms, st);
  if (a.d_qk == 128) return launch_rows<KIND, 128, 128>(a, rows, sms, st);
  return launch_rows<KIND, 192, 128>(a, rows, sms, st);
}

}  // namespace

}  // namespace paged
}  // namespace attn
