// Attention over the paged cache for many query rows per KV head: chunks of
// prompts behind a cached prefix.
//
// Mathematics and tiling.  The rows of one KV head (tokens x heads of its
// group) are packed, so both heads of a group and short chunks fill the MMA's
// 128 rows.  A block works on 256 rows in two halves A and B:
//   S_X = Q_X K^T (tcgen05.mma, both from shared memory), P_X = exp2(S_X - m)
//   by one thread per row, packed over S_X in tensor memory, O_X += P_X V.
// A key tile is 128 tokens, brought to shared memory once for both halves by
// TMA, a page (or 128 tokens of one) a box.  16-bit caches land in the
// 128-byte-swizzled layout the MMA reads; E4M3 codes land in a ring of their
// own, from which converter warps write them as fp16 (exact) into that layout.
// The converters also write zeros over value slots outside the mask.  The
// scales of 16-key groups (no page is smaller) are applied to the scores: one
// multiply-add per score as without them, since a group's maximum can be
// scaled after it is found.
//
// What bounds it (1024 tokens over 31744 cached ones, 64 query heads, E4M3:
// 790 us, 1.37 PFLOP/s, tensor pipe 58 % busy): S, P and O of two halves fill
// tensor memory, so a half's MMAs and its softmax take turns, with only the
// other half beside them; and shared memory, which the MMAs read at 192 KB a
// tile of 2048 MMA clocks while the conversion reads 32 and writes 64.
//
// Work split.  As for few rows: all tiles in order (sequence, head, row block,
// tile) cut into equal shares, one a block, one block an SM; causal row blocks
// count only the tiles they need.  Pieces of a row block meet in a second
// kernel.
//
// Roles: MMA issuer, TMA producer and scheduler (a warp each), four converter
// warps, four softmax warps a half.  The scheduler hands out pieces so that the
// walk's state stays out of the other roles' registers; loops that run once a
// piece are rolled, since the roles share instruction caches.
//
// Values that are not finite in a tile that some rows mask in part, or of which
// a page is masked for its id, are taken out of the product (their zero weight
// would make NaN of them) and added in the epilogue to the rows that keep them.
#pragma once
#include <cuda.h>

#include <climits>
#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

using namespace sm103;

constexpr int kHalf = 128;             // rows per half, keys per tile
constexpr int kChunkRows = 2 * kHalf;  // rows per block of rows
// the running maximum follows the true one within a factor of 2^8
constexpr float kLazy = 8.f;

// A piece of a block of rows, as the scheduler warp hands it to the others.
struct Piece {
  int n, key;        // key tiles (0: no row keeps a key, < 0: the end), first key
  int seq, head, rb; // sequence, KV head, block of rows
  int first, whole;  // begins with the block's first tile; holds all its tiles
  int pieces;        // of a split block, in its first piece: how many there are
  int row0, new_rows, pos0, hi;  // of the sequence: first row, tokens, first position, keys
  int2 any, all;     // keys some row, and every row, of the block keeps
  int2 half[2];      // keys every row of a half keeps
};

struct ChunkAux {
  uint64_t q_full[2], q_empty[2], kv_full[3], kv_empty[3];
  uint64_t raw_full[4], raw_empty[4];  // TMA: of the code ring, or of the K / V ring
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t piece_full[4], piece_empty[4];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  uint32_t bad[4];  // by piece: its number + 1 once a value was taken out of the product
  int ok_mask[8];   // by tile (the producer runs up to four tiles ahead of the
                    // softmax): 16-key groups whose page exists
  int64_t part[16];
  int64_t begin, total;  // the block's first unit, all units
  int ctas, unit0;
  int seq, head, rb;
  Piece piece[4];
  float4 scale[8][8];     // by tile and group: K scale, log2 V scale, 1 / V scale
  uint8_t q_exp[4][kChunkRows];  // by piece: biased exponent of the row's power of two
};

template <int KIND, int DQK, int DV>
struct ChunkCfg {
  static constexpr bool kCodes = KIND == kCacheE4m3;
  static constexpr bool kWide = DQK > 128;
  static constexpr int kQTile = kHalf * DQK * 2;  // one half's Q
  // K and V tiles take turns in the rings; with two stages K has the first
  static constexpr int kK = kHalf * DQK * 2, kV = kHalf * DV * 2;
  static constexpr int kKV = kK > kV ? kK : kV;
  static constexpr int kQStages = kWide || kCodes ? 1 : 2;
  static constexpr int kKVStages = kWide ? 2 : 3;
  static constexpr int kCodeStages = !kCodes ? 0 : kWide ? 2 : 4;
  static constexpr int kKVOff = kQStages * 2 * kQTile;
  static constexpr int kCodeOff = kKVOff + (kWide ? kK + kV : kKVStages * kKV);
  static constexpr int kAuxOff =
      kCodeOff + (!kCodes ? 0 : kWide ? (kK + kV) / 2 : kCodeStages * kKV / 2);
  static constexpr int kSmem = kAuxOff + (static_cast<int>(sizeof(ChunkAux)) + 127) / 128 * 128;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static __device__ __forceinline__ uint32_t kv(uint32_t e) {
    return kKVOff + (kWide ? (e & 1) * kK : (e % kKVStages) * kKV);
  }
  static __device__ __forceinline__ uint32_t code(uint32_t e) {
    return kCodeOff + (kWide ? (e & 1) * (kK / 2) : (e & 3) * (kKV / 2));
  }
};

struct SeqView {
  Seq q;
  int hi;  // keys it has in the cache
};
__device__ __forceinline__ SeqView view_of(const Args& a, int s) {
  SeqView v;
  v.q = load_seq(a, s);
  const int cap = a.max_pages << a.page_shift;
  v.hi = min(v.q.len, cap);
  return v;
}
__device__ __forceinline__ int rows_of(const Args& a, const SeqView& v) { return v.q.n * a.group; }
__device__ __forceinline__ int blocks_of(const Args& a, const SeqView& v) {
  return (v.q.n * a.group + kChunkRows - 1) / kChunkRows;
}
// Keys [x, y) that some (any) or every row of rows [r0, r1) keeps.
__device__ __forceinline__ int2 keys_any(const Args& a, const SeqView& v, int r0, int r1) {
  const int pos0 = v.q.len - v.q.n;
  const int lo = div_group(a, r0), hi = div_group(a, min(r1, rows_of(a, v)) - 1);
  return make_int2(a.window >= 0 ? max(0, pos0 + lo - a.window) : 0,
                   a.causal ? min(v.hi, pos0 + hi + 1) : v.hi);
}
__device__ __forceinline__ int2 keys_all(const Args& a, const SeqView& v, int r0, int r1) {
  const int pos0 = v.q.len - v.q.n;
  const int lo = div_group(a, r0), hi = div_group(a, min(r1, rows_of(a, v)) - 1);
  return make_int2(a.window >= 0 ? max(0, pos0 + hi - a.window) : 0,
                   a.causal ? min(v.hi, pos0 + lo + 1) : v.hi);
}
// A block of rows costs its tiles and about as much as this many more: queries
// to load, a pipeline to fill, O to write.  Shares are cut by that sum.
constexpr int kStart = 3;
// Tiles start at multiples of 128 keys, so that a tile is a whole number of
// pages or inside one.
__device__ __forceinline__ int tiles_of(const Args& a, const SeqView& v, int rb) {
  const int2 k = keys_any(a, v, rb * kChunkRows, (rb + 1) * kChunkRows);
  return max(1, (k.y - (k.x & ~(kHalf - 1)) + kHalf - 1) / kHalf);
}
__device__ __forceinline__ int64_t seq_units(const Args& a, const SeqView& v) {
  int64_t n = 0;
  const int nrb = blocks_of(a, v);
  for (int rb = 0; rb < nrb; ++rb) n += kStart + tiles_of(a, v, rb);
  return n;
}

// Walks the block's pieces (the scheduler warp does).  Units
// [0, kStart) of a block of rows are its start, the others its tiles.
struct Walk {
  int done, share;  // units behind the current piece's first, and in all
  int seq, head, rb, u0;
  SeqView v;
  // the current piece: tiles [t0, t1) of nt
  int u1, t0, t1, nt;
  int2 any;    // keys some row of the block of rows keeps
  int n, key;  // key tiles (0: no row keeps a key), first key of the first
};
__device__ __forceinline__ bool walk_piece(const Args& a, Walk& w) {
  w.nt = tiles_of(a, w.v, w.rb);
  w.u1 = min(w.nt + kStart, w.u0 + (w.share - w.done));
  w.t0 = max(0, w.u0 - kStart);
  w.t1 = max(0, w.u1 - kStart);
  w.any = keys_any(a, w.v, w.rb * kChunkRows, (w.rb + 1) * kChunkRows);
  w.key = (w.any.x & ~(kHalf - 1)) + w.t0 * kHalf;
  w.n = w.any.y > w.any.x ? w.t1 - w.t0 : 0;
  return w.t1 > w.t0;
}
// The next piece with tiles.
__device__ __forceinline__ bool walk_next(const Args& a, Walk& w) {
  do {
    w.done += w.u1 - w.u0;
    if (w.done >= w.share) return false;
    w.u0 = 0;
    if (++w.rb >= blocks_of(a, w.v)) {
      w.rb = 0;
      if (++w.head >= a.Hkv) {
        w.head = 0;
        do w.v = view_of(a, ++w.seq);
        while (w.v.q.n == 0);
      }
    }
  } while (!walk_piece(a, w));
  return true;
}

// This block's share, found by all 512 threads.
__device__ __forceinline__ void walk_init(const Args& a, ChunkAux* x, Walk& w) {
  constexpr int kN = 512;
  const int per = (a.num_seqs + kN - 1) / kN;
  const int first = threadIdx.x * per, last = min(a.num_seqs, first + per);
  int64_t mine = 0;
  for (int s = first; s < last; ++s) {
    const SeqView v = view_of(a, s);
    if (outside(a, v.q)) flag_bounds(a);
    mine += a.Hkv * seq_units(a, v);
  }
  int64_t sum = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, sum, i);
    if ((threadIdx.x & 31) >= i) sum += y;
  }
  if ((threadIdx.x & 31) == 31) x->part[threadIdx.x / 32] = sum;
  __syncthreads();
  int64_t total = 0, before = sum - mine;
  for (int i = 0; i < kN / 32; ++i) {
    if (i < static_cast<int>(threadIdx.x) / 32) before += x->part[i];
    total += x->part[i];
  }
  const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
  w.done = w.share = 0;
  if (static_cast<int>(blockIdx.x) < ctas) {
    const int64_t begin = blockIdx.x * total / ctas;
    w.share = static_cast<int>((blockIdx.x + 1) * total / ctas - begin);
    if (begin >= before && begin < before + mine) {
      int64_t off = begin - before;
      int s = first;
      for (;; ++s) {
        const SeqView v = view_of(a, s);
        const int64_t per_head = seq_units(a, v);
        if (off >= a.Hkv * per_head) {
          off -= a.Hkv * per_head;
          continue;
        }
        x->seq = s;
        x->head = static_cast<int>(off / per_head);
        off %= per_head;
        int rb = 0;
        for (int n; off >= (n = kStart + tiles_of(a, v, rb)); ++rb) off -= n;
        x->rb = rb;
        x->unit0 = static_cast<int>(off);
        x->begin = begin;
        x->total = total;
        x->ctas = ctas;
        break;
      }
    }
  }
  __syncthreads();
  if (w.share > 0) {
    w.seq = x->seq;
    w.head = x->head;
    w.rb = x->rb;
    w.u0 = x->unit0;
    w.v = view_of(a, w.seq);
    // a share that ends inside its only start has no piece
    if (!walk_piece(a, w) && !walk_next(a, w)) w.share = 0;
  }
}

// Eight E4M3 codes to fp16, stored as one 16-byte unit.
__device__ __forceinline__ void store_codes(uint32_t dst, uint32_t lo, uint32_t hi) {
  st_shared_v4(dst, e4m3x2_f16x2(static_cast<uint16_t>(lo)),
               e4m3x2_f16x2(static_cast<uint16_t>(lo >> 16)),
               e4m3x2_f16x2(static_cast<uint16_t>(hi)),
               e4m3x2_f16x2(static_cast<uint16_t>(hi >> 16)));
}

template <int KIND, int DQK, int DV>
__global__ void __launch_bounds__(512, 1) chunk_kernel(const __grid_constant__ Args a,
                                                       const __grid_constant__ CacheMaps maps) {
  using L = ChunkCfg<KIND, DQK, DV>;
  constexpr bool kBf = KIND == kCacheBf16;
  constexpr bool kCodes = KIND == kCacheE4m3;
  constexpr int NKV = L::kKVStages, NQ = L::kQStages;
  constexpr float kShift = kBf ? 0.f : 7.f;  // P <= 2^(7 + 8) in fp16
  constexpr uint32_t kColS = 0, kColO = 256;
  extern __shared__ __align__(1024) uint8_t sm[];
  ChunkAux* const x = reinterpret_cast<ChunkAux*>(sm + L::kAuxOff);
  volatile int* const abort = &x->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023u) return;  // the swizzle needs it; the window starts aligned

  auto timeout = [&]() {
    if (a.status) *a.status = ATTN_ERR_DEVICE_TIMEOUT;
    *abort = 1;
  };
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&x->q_full[s], 128);
      mbar_init(&x->q_empty[s], 1);
      mbar_init(&x->s_full[s], 1);
      mbar_init(&x->p_full[s], 128);
      mbar_init(&x->o_full[s], 1);
      mbar_init(&x->o_empty[s], 128);
    }
    for (int s = 0; s < 3; ++s) {
      mbar_init(&x->kv_full[s], 128);
      mbar_init(&x->kv_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&x->raw_full[s], 1);
      mbar_init(&x->raw_empty[s], 128);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&x->piece_full[s], 1);
      mbar_init(&x->piece_empty[s], 1 + 1 + 4 + 8);  // MMA, producer, converter, softmax warps
    }
    mbar_init(&x->drain, 1);
    x->abort = 0;
    for (uint32_t& b : x->bad) b = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&x->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  grid_dep_wait();
  if (tid == 0) a.split_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  Walk w;
  walk_init(a, x, w);  // two block barriers
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = x->tmem;

  // The i-th piece (in shared memory), and this warp's release of it.
  auto take = [&](uint32_t i, bool* ok) -> const Piece* {
    *ok = mbar_wait_warp(&x->piece_full[i & 3], (i >> 2) & 1);
    return &x->piece[i & 3];
  };
  auto release = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&x->piece_empty[i & 3]);
  };

  if (warp < 4) {
    if (warp == 2) {
      // ------------------------------------------------------------ scheduler
      // Keeps the walk's state and divisions out of the other roles' registers
      // and code.
      bool ok = true, live = w.share > 0;
      for (uint32_t i = 0; ok; ++i) {
        if (i >= 4 && !(ok = mbar_wait_warp(&x->piece_empty[i & 3], ((i >> 2) - 1) & 1))) break;
        if (lane == 0) {
          Piece& p = x->piece[i & 3];
          if (live) {
            const int r0 = w.rb * kChunkRows, rows = rows_of(a, w.v);
            p.n = w.n;
            p.key = w.key;
            p.seq = w.seq;
            p.head = w.head;
            p.rb = w.rb;
            p.first = w.t0 == 0;
            p.whole = w.t0 == 0 && w.t1 == w.nt;
            const int64_t end = x->begin + w.done + (w.nt + kStart - w.u0);  // of the block's units
            p.pieces = static_cast<int>((end * x->ctas + x->total - 1) / x->total) -
                       static_cast<int>(blockIdx.x);
            p.row0 = w.v.q.row0;
            p.new_rows = w.v.q.n;
            p.pos0 = w.v.q.len - w.v.q.n;
            p.hi = w.v.hi;
            p.any = w.any;
            p.all = keys_all(a, w.v, r0, r0 + kChunkRows);
            for (int h = 0; h < 2; ++h)  // a half without rows masks everything
              p.half[h] = r0 + h * kHalf < rows
                              ? keys_all(a, w.v, r0 + h * kHalf, r0 + (h + 1) * kHalf)
                              : make_int2(INT_MAX, INT_MIN);
          } else {
            p.n = -1;
          }
          mbar_arrive(&x->piece_full[i & 3]);
        }
        if (__any_sync(0xffffffffu, !live || *abort != 0)) break;
        live = walk_next(a, w);
      }
      if (!ok && lane == 0) timeout();
    }
    if (warp == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t id_s = idesc_f32acc(kBf ? 1 : 0, kHalf, kHalf, false, false);
      constexpr uint32_t id_o = idesc_f32acc(kBf ? 1 : 0, kHalf, DV, false, true);
      const uint32_t tm = warp_uniform(tmem);
      const uint64_t q_km = sdesc_sw128(smem_u32(sm), 16, 1024);
      const uint64_t kv_km = sdesc_sw128(smem_u32(sm + L::kKVOff), 16, 1024);
      const uint64_t kv_mn = sdesc_sw128(smem_u32(sm + L::kKVOff), 16384, 1024);
      auto stage = [&](uint32_t c) -> uint32_t { return (L::kv(c) - L::kKVOff) >> 4; };
      auto issue_s = [&](int h, uint32_t piece, uint32_t kc) {
        const uint64_t qd = q_km + ((((piece % NQ) * 2 + h) * L::kQTile) >> 4);
        mma_ss_warp<DQK / 16, 4, 2, 1018, 2, 1018>(tm + kColS + h * kHalf, qd, kv_km + stage(kc),
                                                   id_s, 0u);
        mma_commit_warp(&x->s_full[h]);
      };
      uint32_t it = 0, kvc = 0, st = 0, pi = 0;
      bool ok = true;
      // tiles of the next piece that has some, or -1 behind the last
      auto next = [&]() -> int {
        for (;;) {
          const Piece* p = take(pi, &ok);
          const int n = ok ? p->n : -1;
          release(pi++);
          if (n != 0) return n;
        }
      };
      int n = next();
      if (ok && n > 0) {
        if ((ok = mbar_wait_warp(&x->q_full[0], 0) && mbar_wait_warp(&x->kv_full[0], 0))) {
          tc_fence_after();
          issue_s(0, 0, 0);
          issue_s(1, 0, 0);
          mma_commit_warp(&x->kv_empty[0]);
          if (n == 1) mma_commit_warp(&x->q_empty[0]);
          kvc = 1;
        }
      }
      // Each step: P_X V, then over P_X's columns the S that comes next, of
      // this piece or the next one.  The pipe runs in order of issue.
      while (ok && n > 0) {
        int nx = -1;
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t k = st + j, vc = kvc;
          const bool more = j + 1 < n;
          if (!more) nx = next();
          if (!ok) break;
          const bool go_on = more || nx > 0;
          const uint32_t pc = more ? it : it + 1;
          if (!(ok = mbar_wait_warp(&x->kv_full[vc % NKV], (vc / NKV) & 1))) break;
          for (int h = 0; h < 2 && ok; ++h) {
            if (!(ok = mbar_wait_warp(&x->p_full[h], k & 1))) break;
            if (j == 0 && it > 0 && !(ok = mbar_wait_warp(&x->o_empty[h], (it - 1) & 1))) break;
            tc_fence_after();
            mma_ts_warp<kHalf / 16, 4, 8, 8, 128, 128>(tm + kColO + h * kHalf,
                                                       tm + kColS + h * kHalf, kv_mn + stage(vc),
                                                       id_o, j == 0 ? 0u : 1u);
            if (!more) mma_commit_warp(&x->o_full[h]);
            if (h == 1) mma_commit_warp(&x->kv_empty[vc % NKV]);
            if (!go_on) continue;
            if (h == 0) {
              if (!more && !(ok = mbar_wait_warp(&x->q_full[pc % NQ], (pc / NQ) & 1))) break;
              if (!(ok = mbar_wait_warp(&x->kv_full[(vc + 1) % NKV], ((vc + 1) / NKV) & 1))) break;
            }
            tc_fence_after();
            issue_s(h, pc, vc + 1);
          }
          if (!ok) break;
          if (go_on) {
            mma_commit_warp(&x->kv_empty[(vc + 1) % NKV]);
            // the last S of a piece: its Q may be replaced
            if (more ? j + 2 == n : nx == 1) mma_commit_warp(&x->q_empty[pc % NQ]);
          }
          kvc += go_on ? 2 : 1;
        }
        if (!ok) break;
        st += n;
        ++it;
        n = nx;
      }
      if (!ok && lane == 0) timeout();
      mma_commit_warp(&x->drain);
      mbar_wait(&x->drain, 0, 200000000ull);
    }
    if (warp == 1) {
      // ------------------------------------------------------------ TMA producer
      // Lane i looks after box i of a tile: a page, or 128 tokens of one.  The
      // table is read two tiles ahead and the scales one, so that no load of a
      // tile waits for another of the same tile.
      const int rows_log = min(a.page_shift, 7), boxes = kHalf >> rows_log;
      const int page_mask = (1 << a.page_shift) - 1;
      uint32_t st = 0, e = 0;  // tiles and ring entries so far
      bool ok = true;
      for (uint32_t pi = 0;; ++pi) {
        const Piece* const p = take(pi, &ok);
        if (!ok || p->n < 0) break;
        const int n = p->n, hk = p->head, key0 = p->key, last = p->any.y;
        const int32_t* const table = a.table + p->seq * a.table_stride;
        release(pi);
        auto key_of = [&](int j) -> int { return key0 + j * kHalf + (lane << rows_log); };
        auto load_entry = [&](int j) -> int {
          if (j >= n || lane >= boxes || key_of(j) >= last) return INT_MIN;
          const int col = key_of(j) >> a.page_shift;
          return col < a.max_pages ? table[col] : -1;
        };
        struct Ids {
          int id;
          float ks, vs;
        };
        auto load_ids = [&](int id) -> Ids {
          Ids r = {id, 1.f, 1.f};
          if (id < 0 || id >= a.num_pages) {
            if (id != INT_MIN) flag_bounds(a);
            r.id = -1;
          } else if (kCodes) {
            r.ks = a.k_scale[static_cast<int64_t>(id) * a.Hkv + hk];
            r.vs = a.v_scale[static_cast<int64_t>(id) * a.Hkv + hk];
          }
          return r;
        };
        int ahead = load_entry(1);
        Ids ids = load_ids(load_entry(0));
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t k = st + j;
          const Ids nxt = load_ids(ahead);
          ahead = load_entry(j + 2);
          const unsigned okm = __ballot_sync(0xffffffffu, ids.id >= 0);
          const uint32_t count = __popc(okm);
          const int slot = key_of(j) & page_mask;
          for (int m = 0; m < 2 && ok; ++m, ++e) {
            const int d = m == 0 ? DQK : DV;
            const uint32_t rs = kCodes ? e % (L::kCodeStages + !kCodes) : e % NKV;
            if (e >= (kCodes ? L::kCodeStages : NKV)) {
              const uint32_t ph = (e / (kCodes ? L::kCodeStages + !kCodes : NKV) - 1) & 1;
              if (!(ok = mbar_wait_warp(kCodes ? &x->raw_empty[rs] : &x->kv_empty[rs], ph))) break;
            }
            if (m == 0) {
              const int box = (16 * (lane & 7)) >> rows_log;
              const float ks = __shfl_sync(0xffffffffu, ids.ks, box);
              const float vs = fmaxf(__shfl_sync(0xffffffffu, ids.vs, box), kMinVScale);
              const unsigned groups = __ballot_sync(0xffffffffu, okm >> box & 1) & 0xffu;
              if (lane < 8) {
                const float lg = (__float_as_uint(vs) & 0x7fffffu) == 0
                                     ? static_cast<float>(
                                           static_cast<int>(__float_as_uint(vs) >> 23) - 127)
                                     : __log2f(vs);
                x->scale[k & 7][lane] = make_float4(ks, lg, 1.f / vs, 0.f);
                if (lane == 0) x->ok_mask[k & 7] = groups;
              }
            }
            // the arrival (release) publishes the scales; the loads follow it
            __syncwarp();
            if (lane == 0)
              mbar_arrive_expect_tx(&x->raw_full[rs],
                                    (count << rows_log) * d * (kCodes ? 1 : 2));
            __syncwarp();
            if (ids.id >= 0) {
              const void* map = m == 0 ? &maps.k : &maps.v;
              const uint32_t dst = smem_u32(sm);
              if constexpr (kCodes) {
                tma_load_4d(dst + L::code(e) + (lane << rows_log) * d, map, &x->raw_full[rs], 0,
                            slot, hk, ids.id);
              } else {
                for (int c = 0; c < d / 64; ++c)
                  tma_load_4d(dst + L::kv(e) + c * 16384 + (lane << rows_log) * 128, map,
                              &x->raw_full[rs], c * 64, slot, hk, ids.id);
              }
            }
            __syncwarp();
          }
          ids = nxt;
        }
        if (!ok) break;
        st += n;
      }
      if (!ok && lane == 0) timeout();
      // copies in flight land before the block may leave
      const uint32_t depth = kCodes ? L::kCodeStages : NKV;
      for (uint32_t i = e > depth ? e - depth : 0; i < e; ++i)
        mbar_wait(&x->raw_full[i % depth], (i / depth) & 1, 100000000ull);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ converters
    // They hold no global loads in flight at their proxy fences (a fence waits
    // for them): the codes come by TMA.
    const int ct = tid - 128;  // 0..127
    uint32_t it = 0, e = 0, st = 0;
    bool ok = true;
    for (uint32_t pi = 0;; ++pi) {
      const Piece* const p = take(pi, &ok);
      if (!ok || p->n < 0) break;
      const int n = p->n, r0 = p->rb * kChunkRows, head = p->head, key0 = p->key;
      const int row0 = p->row0, new_rows = p->new_rows;
      const int2 any = p->any, all = p->all;
      release(pi);
      if (n == 0) continue;
      // ---- queries: one row a thread and half, to fp16 where the cache is E4M3
      if (it >= NQ && !mbar_wait_warp(&x->q_empty[it % NQ], ((it / NQ) - 1) & 1)) {
        ok = false;
        break;
      }
      {
        // Lanes of a group copy one row together, 16 bytes each, to where the
        // MMA reads it; what a lane copied it turns to fp16 in place.  Small
        // rolled loops: this code runs once a piece and is fetched anew.
        constexpr int kL = DQK == 64 ? 8 : 16, kPer = 32 / kL;  // lanes a row, rows a load
        constexpr int kU = DQK == 192 ? 2 : 1;                  // units a lane (192: 16 + 8)
        constexpr int kSteps = 2 * 32 / kPer;                   // this warp's rows of both halves
        const int sub = lane % kL, first = (warp - 4) * 32 + lane / kL;
        const uint32_t qs = smem_u32(sm) + (it % NQ) * 2 * L::kQTile;
        auto place = [&](int b, int u) -> uint32_t {
          const int nr = b * kPer, rr = first + nr % 32, unit = sub + kL * u;
          return qs + (nr / 32) * L::kQTile + rr * 128 + (unit / 8) * 16384 +
                 (((unit & 7) ^ (rr & 7)) << 4);
        };
#pragma unroll 4
        for (int b = 0; b < kSteps; ++b) {
          const int nr = b * kPer, r = r0 + (nr / 32) * kHalf + first + nr % 32;
          const int tok = div_group(a, r);
          const bool real = tok < new_rows;
          const uint16_t* qp = a.q + (real ? (row0 + tok) * a.q_stride +
                                                 (head * a.group + r - tok * a.group) * DQK +
                                                 sub * 8
                                           : 0);
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (u == 0 || sub < 8)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(b, u)),
                           "l"(qp + (real ? kL * u * 8 : 0)), "r"(real ? 16 : 0)
                           : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (kCodes && !a.f16) {
#pragma unroll 4
          for (int b = 0; b < kSteps; ++b) {
            uint4 v[kU];
            uint32_t mx = 0;  // two 16-bit magnitudes
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              v[u] = u == 0 || sub < 8 ? lds128(place(b, u)) : make_uint4(0, 0, 0, 0);
              mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[u].x & 0x7fff7fffu, v[u].y & 0x7fff7fffu),
                                         __vmaxu2(v[u].z & 0x7fff7fffu, v[u].w & 0x7fff7fffu)));
            }
#pragma unroll
            for (int k = 1; k < kL; k <<= 1)
              mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            int ex = static_cast<int>(max(mx & 0xffffu, mx >> 16) >> 7);
            ex = ex == 255 ? 127 + 14 : max(ex, 27);
            const float to = __uint_as_float(static_cast<uint32_t>(254 + 14 - ex) << 23);
            const int nr = b * kPer;
            if (sub == 0)
              x->q_exp[it & 3][(nr / 32) * kHalf + first + nr % 32] = static_cast<uint8_t>(ex - 14);
            auto turn = [&](uint32_t e) -> uint32_t {
              return pack_f16x2(__uint_as_float(e << 16) * to,
                                __uint_as_float(e & 0xffff0000u) * to);
            };
#pragma unroll
            for (int u = 0; u < kU; ++u)
              if (u == 0 || sub < 8)
                st_shared_v4(place(b, u), turn(v[u].x), turn(v[u].y), turn(v[u].z), turn(v[u].w));
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&x->q_full[it % NQ]);

      // One ring entry: K (no row is ever masked by its content) or V, whose
      // slots outside the mask become zeros.
      auto convert = [&](auto dim, bool value, int key, uint32_t k) -> bool {
        constexpr int D = decltype(dim)::value;
        constexpr uint32_t kDepth = kCodes ? L::kCodeStages + !kCodes : NKV;
        if (!mbar_wait_warp(&x->raw_full[e % kDepth], (e / kDepth) & 1)) return false;
        const bool whole = key >= all.x && key + kHalf <= all.y && x->ok_mask[k & 7] == 0xff;
        const int okm = x->ok_mask[k & 7];
        auto in = [&](int r) -> bool {
          return (okm >> (r >> 4) & 1) && key + r >= any.x && key + r < any.y;
        };
        if constexpr (kCodes) {
          // D / 16 units of 16 codes a row, in the order of memory, four a
          // round.  (The stage's last reader is waited for first: the codes
          // are turned as they are read.)
          constexpr int kU = D / 16;
          if (e >= NKV && !mbar_wait_warp(&x->kv_empty[e % NKV], ((e / NKV) - 1) & 1)) return false;
          const uint32_t src = smem_u32(sm) + L::code(e) + ct * 16;
          const uint32_t dst = smem_u32(sm) + L::kv(e);
#pragma unroll 1
          for (int i0 = 0; i0 < kU; i0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lds128(src + (i0 + i) * 2048);
            if (value && !whole) {
              uint32_t bad = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (!in((ct + 128 * (i0 + i)) / kU)) v[i] = make_uint4(0, 0, 0, 0);
                bad |= not_finite<KIND>(v[i].x) | not_finite<KIND>(v[i].y) |
                       not_finite<KIND>(v[i].z) | not_finite<KIND>(v[i].w);
              }
              if (bad) {
                x->bad[it & 3] = it + 1;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  v[i] = make_uint4(finite_only<KIND>(v[i].x), finite_only<KIND>(v[i].y),
                                    finite_only<KIND>(v[i].z), finite_only<KIND>(v[i].w));
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int q = ct + 128 * (i0 + i), r = q / kU, u = q % kU;
              // lanes with u >= 4 (the second 64 dims) store their second half
              // first: eight lanes then meet eight bank groups
              const uint32_t row = dst + (u >> 2) * 16384 + r * 128;
              const int f = (u >> 2) & 1, u0 = 2 * (u & 3) + f, u1 = u0 ^ 1;
              store_codes(row + ((u0 ^ (r & 7)) << 4), f ? v[i].z : v[i].x, f ? v[i].w : v[i].y);
              store_codes(row + ((u1 ^ (r & 7)) << 4), f ? v[i].x : v[i].z, f ? v[i].y : v[i].w);
            }
          }
          mbar_arrive(&x->raw_empty[e % kDepth]);
        } else if (value && !whole) {
          const uint32_t at = smem_u32(sm) + L::kv(e);
          for (int i = 0; i < 8; ++i) {
            const int r = (ct >> 3) + 16 * i;
            for (int c = 0; c < D / 64; ++c) {
              const uint32_t p = at + c * 16384 + r * 128 + (ct & 7) * 16;
              if (!in(r)) {
                st_shared_v4(p, 0, 0, 0, 0);
                continue;
              }
              const uint4 v = lds128(p);
              if (not_finite<KIND>(v.x) | not_finite<KIND>(v.y) | not_finite<KIND>(v.z) |
                  not_finite<KIND>(v.w)) {
                x->bad[it & 3] = it + 1;
                st_shared_v4(p, finite_only<KIND>(v.x), finite_only<KIND>(v.y),
                             finite_only<KIND>(v.z), finite_only<KIND>(v.w));
              }
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&x->kv_full[e % NKV]);
        ++e;
        return true;
      };
      for (int j = 0; j < n && ok; ++j) {
        const int key = key0 + j * kHalf;
        if constexpr (DQK == DV) {
#pragma unroll 1
          for (int m = 0; m < 2 && ok; ++m)
            ok = convert(std::integral_constant<int, DV>{}, m == 1, key, st + j);
        } else {
          ok = convert(std::integral_constant<int, DQK>{}, false, key, st + j) &&
               convert(std::integral_constant<int, DV>{}, true, key, st + j);
        }
      }
      if (!ok) break;
      st += n;
      ++it;
    }
    if (!ok && lane == 0) timeout();
  } else {
    // ------------------------------------------------------------ softmax
    const int h = (warp - 8) >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lanes + kColS + h * kHalf;
    const uint32_t o_tm = tmem + lanes + kColO + h * kHalf;
    uint32_t st = 0, it = 0;
    bool ok = true;
    for (uint32_t pi = 0;; ++pi) {
      const Piece* const p = take(pi, &ok);
      if (!ok || p->n < 0 || __any_sync(0xffffffffu, *abort != 0)) break;
      const int n = p->n, key0 = p->key;
      const int2 all = p->half[h];
      int lo, hi;  // keys the row keeps
      {
        const int rr = p->rb * kChunkRows + h * kHalf + r, tok = div_group(a, rr);
        const int pos = p->pos0 + tok;
        lo = a.window >= 0 ? max(0, pos - a.window) : 0;
        hi = tok < p->new_rows ? (a.causal ? min(p->hi, pos + 1) : p->hi) : 0;
      }
      float m = -INFINITY, l = 0.f, fac = a.scale * kLog2e;
      for (int j = 0; j < n; ++j) {
        const uint32_t k = st + j;
        const int key = key0 + j * kHalf;
        if (!(ok = mbar_wait_warp(&x->s_full[h], k & 1))) break;
        tc_fence_after();
        if (j == 0 && kCodes && !a.f16)
          fac *= __uint_as_float(static_cast<uint32_t>(x->q_exp[it & 3][h * kHalf + r]) << 23);
        const int okm = x->ok_mask[k & 7];
        // The row's scores are read twice, 32 at a time and the next 32 while
        // these are worked on: held whole they would cost 128 registers, and
        // spills meet an L1 that shared memory has left small.  (1024 tokens
        // over 31744 cached ones, 64 query heads: 784 us when this was chosen,
        // 16 at a time 818, 64 at a time without reading ahead 880, rolled
        // loops 825-916.)
        const bool whole = key >= all.x && key + kHalf <= all.y && okm == 0xff;
        if (!whole) {
          // masked scores to -inf where they lie, so that one copy of the
          // passes serves every tile
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            uint32_t u[16];
            tmem_ld32x32b_x16(s_tm + g * 16, u);
            const int b = key + 16 * g;
            const int f = min(max(lo - b, 0), 16), e = min(max(hi - b, 0), 16);
            const uint32_t bits = (okm >> g & 1) && e > f ? (0xffffu >> (16 - (e - f))) << f : 0u;
            tmem_ld_wait(u);
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = (bits >> i & 1) ? u[i] : 0xff800000u;
            tmem_st32x32b_x16(s_tm + g * 16, u);
          }
          tmem_st_wait();
        }
        auto pass = [&](auto&& body) {
          uint32_t u[2][32];
          tmem_ld32x32b_x32(s_tm, u[0]);
#pragma unroll
          for (int g = 0; g < 8; g += 2) {
            tmem_ld_wait(u[(g >> 1) & 1]);
            if (g < 6) tmem_ld32x32b_x32(s_tm + g * 16 + 32, u[((g >> 1) + 1) & 1]);
            body(g, u[(g >> 1) & 1]);
          }
        };
        // A group's factor on the scores.  It may underflow (a query of zeros
        // over a page of zeros: 2^-117 * 2^-64) but not to 0, which would make
        // NaN of the -inf of masked scores.  A score that is not masked is below
        // 2^33, so that the bound moves its exponent by less than 2^-93.
        auto factor = [&](float ks) -> float { return max_nan(fac * ks, 0x1p-126f); };
        // the row's maximum: of each group, then scaled
        float mx = -INFINITY;
        auto largest = [&](int g, const uint32_t (&u)[32]) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t* e = u + 16 * q;
            float m0 = fmax3(__uint_as_float(e[0]), __uint_as_float(e[1]), __uint_as_float(e[2]));
            float m1 = fmax3(__uint_as_float(e[3]), __uint_as_float(e[4]), __uint_as_float(e[5]));
            m0 = fmax3(m0, __uint_as_float(e[6]), __uint_as_float(e[7]));
            m1 = fmax3(m1, __uint_as_float(e[8]), __uint_as_float(e[9]));
            m0 = fmax3(m0, __uint_as_float(e[10]), __uint_as_float(e[11]));
            m1 = fmax3(m1, __uint_as_float(e[12]), __uint_as_float(e[13]));
            m0 = fmax3(m0, __uint_as_float(e[14]), __uint_as_float(e[15]));
            if constexpr (kCodes) {
              const float4 sc = x->scale[k & 7][g + q];
              mx = fmaxf(mx, fmaf(fmaxf(m0, m1), factor(sc.x), sc.y));
            } else {
              mx = fmax3(mx, m0, m1);
            }
          }
        };
        pass(largest);
        if (!kCodes) mx *= fac;
        const float mn = fmaxf(m, mx);
        const bool grow = mn > m + kLazy || (m == -INFINITY && mn > m);
        const bool again = grow && j > 0 && m > -INFINITY;
        const float f = again ? ex2_approx(m - mn) : 1.f;
        if (grow) m = mn;
        const float base = kShift - (m == -INFINITY ? 0.f : m);
        float add = 0.f;
        // P over the columns of scores that have been read
        auto exps = [&](int g, const uint32_t (&u)[32]) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float A = fac, B = base, inv = 1.f;
            if constexpr (kCodes) {
              const float4 sc = x->scale[k & 7][g + q];
              A = factor(sc.x);
              B = base + sc.y;
              inv = sc.z;
            }
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 y = fma_f32x2(make_float2(__uint_as_float(u[16 * q + 2 * i]),
                                                     __uint_as_float(u[16 * q + 2 * i + 1])),
                                         make_float2(A, A), make_float2(B, B));
              const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
              sum = add_f32x2(sum, p);
              pk[8 * q + i] = kBf ? pack_bf16x2(p.x, p.y) : pack_f16x2(p.x, p.y);
            }
            add = fmaf(sum.x + sum.y, inv, add);
          }
          tmem_st32x32b_x16(s_tm + g * 8, pk);
        };
        pass(exps);
        l = fmaf(l, f, add);
        // S_X(j) was issued after P_X(j-1) V, which is therefore complete
        if (__any_sync(0xffffffffu, again)) {
#pragma unroll
          for (int q = 0; q < DV / 32; ++q) {
            uint32_t o[32];
            tmem_ld32x32b_x32(o_tm + q * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32x32b_x32(o_tm + q * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&x->p_full[h]);
      }
      if (!ok) break;
      // ---- epilogue: O or the piece's partial state
      const int rr = p->rb * kChunkRows + h * kHalf + r, tk = div_group(a, rr);
      const bool real = tk < p->new_rows;
      const int tok = real ? tk : 0, head = p->head * a.group + (real ? rr - tk * a.group : 0);
      const bool complete = p->whole;
      const int slot = 2 * blockIdx.x + p->first;
      if (n > 0) {
        if (!(ok = mbar_wait_warp(&x->o_full[h], it & 1))) break;
        tc_fence_after();
      }
      float lt = l, mt = m, keep = 1.f;
      const bool none = no_key(m, l);
      if (complete && a.sink) {
        const float s2 = a.sink[head] * kLog2e;
        mt = fmaxf(m, s2);
        const float mu = mt == -INFINITY ? 0.f : mt;
        keep = ex2_approx(m - mu);
        lt = l * keep + ex2_approx(s2 - mu + kShift);
      }
      const float inv = complete ? (lt == 0.f ? 0.f : keep / lt) : 1.f;
      // partial states lie [slot][16-byte column][row], so that a warp's
      // stores (a row a lane) are contiguous
      const int64_t prow = static_cast<int64_t>(slot) * kChunkRows + h * kHalf + r;
      float4* const pbase = reinterpret_cast<float4*>(a.part) +
                            static_cast<int64_t>(slot) * (DV / 4) * kChunkRows + h * kHalf + r;
      const bool bad = n > 0 && x->bad[it & 3] == it + 1;
      uint16_t* op = a.o + (static_cast<int64_t>(p->row0 + tok) * a.Hq + head) * DV;
#pragma unroll 1
      for (int q = 0; q < DV / 32; ++q) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32x32b_x32(o_tm + q * 32, o);
          tmem_ld_wait(o);
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = n > 0 && !none ? __uint_as_float(o[i]) * inv : 0.f;
        if (bad && real) {
          // values that are not finite, in the tiles they were taken out of:
          // those the block of rows masks in part, or of which a page is none
          const int2 blk = p->all;
          auto every_page = [&](int key) -> bool {
#pragma unroll 1
            for (int i = 0; i < kHalf; i += 16)
              if (page_of(a, p->seq, key + i) < 0) return false;
            return true;
          };
          for (int j = 0; j < n; ++j) {
            const int key = key0 + j * kHalf;
            if (key >= blk.x && key + kHalf <= blk.y && every_page(key)) continue;
            for (int kk = max(key, lo); kk < min(key + kHalf, hi); ++kk) {
              const int page = page_of(a, p->seq, kk);
              if (page < 0) continue;
              const char* vp = a.vc + page * a.v_page + p->head * a.v_head +
                               static_cast<int64_t>(kk & ((1 << a.page_shift) - 1)) * a.v_tok;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e =
                    kCodes ? e4m3_value(reinterpret_cast<const uint8_t*>(vp)[q * 32 + i])
                           : elem(reinterpret_cast<const uint16_t*>(vp)[q * 32 + i], !kBf);
                if (!(fabsf(e) < INFINITY)) v[i] += e;
              }
            }
          }
        }
        if (real && complete) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack2(v[2 * i], v[2 * i + 1], a.f16);
          if (a.o_st32) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              st_global_v8(op + q * 32 + 2 * i, pk[i], pk[i + 1], pk[i + 2], pk[i + 3], pk[i + 4],
                           pk[i + 5], pk[i + 6], pk[i + 7]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(op + q * 32 + 2 * i) =
                  make_uint4(pk[i], pk[i + 1], pk[i + 2], pk[i + 3]);
          }
        } else if (real) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            pbase[(q * 8 + i / 4) * kChunkRows] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&x->o_empty[h]);
      }
      if (real && complete && a.lse)
        a.lse[static_cast<int64_t>(head) * a.num_tokens + p->row0 + tok] =
            none ? (a.sink ? a.sink[head] : -INFINITY) : (mt - kShift) * kLn2 + logf(lt);
      if (real && !complete) a.part_ml[prow] = make_float2(m, l);
      if (!complete && p->first && h == 0 && r == 0)
        a.split_desc[blockIdx.x] = make_int4(p->pieces, p->seq, p->head, p->rb);
      release(pi);
      st += n;
      if (n > 0) ++it;
    }
    if (!ok && lane == 0) timeout();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of split blocks of rows: block (i, y) rows 32 y .. 32 y + 31
// of the block of rows whose first piece is block i's.  A lane reads a row's
// 16-byte columns (a warp's reads are contiguous), its eight warps share the
// columns; O goes through shared memory so that its rows are written whole.
template <int DV>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ Args a,
                                                         float shift) {
  __shared__ uint2 s_o[32][DV / 4 + 1];
  grid_dep_wait();
  const int4 d = a.split_desc[blockIdx.x];
  if (d.x == 0) return;
  const int lane = threadIdx.x & 31, wp = threadIdx.x / 32;
  const Seq q = load_seq(a, d.y);
  const int rows = q.n * a.group, r0 = d.w * kChunkRows + blockIdx.y * 32;
  if (r0 >= rows) return;
  constexpr int kC = DV / 4 / 8;  // 16-byte columns per warp
  const int col = blockIdx.y * 32 + lane, r = r0 + lane;
  const int rc = min(r, rows - 1), tok = div_group(a, rc);
  const int head = d.z * a.group + rc - tok * a.group;
  float4 acc[kC];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < kC; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < rows) {
#pragma unroll 2
    for (int p = 0; p < d.x; ++p) {
      const int64_t slot = 2 * (static_cast<int64_t>(blockIdx.x) + p) + (p == 0 ? 1 : 0);
      const float2 ml = a.part_ml[slot * kChunkRows + col];
      const float4* pp = reinterpret_cast<const float4*>(a.part) + slot * (DV / 4) * kChunkRows +
                         wp * kC * kChunkRows + col;
      float4 v[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) v[j] = pp[j * kChunkRows];
      const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2_approx(m - mu), f1 = ex2_approx(ml.x - mu);
#pragma unroll
      for (int j = 0; j < kC; ++j)
        acc[j] = make_float4(acc[j].x * f0 + v[j].x * f1, acc[j].y * f0 + v[j].y * f1,
                             acc[j].z * f0 + v[j].z * f1, acc[j].w * f0 + v[j].w * f1);
      l = l * f0 + ml.y * f1;
      m = mn;
    }
  }
  const bool none = no_key(m, l);
  float mt = m, lt = l, keep = 1.f;
  if (a.sink) {
    const float s2 = a.sink[head] * kLog2e;
    mt = fmaxf(m, s2);
    const float mu = mt == -INFINITY ? 0.f : mt;
    keep = ex2_approx(m - mu);
    lt = l * keep + ex2_approx(s2 - mu + shift);
  }
  const float inv = lt == 0.f ? 0.f : keep / lt;
#pragma unroll
  for (int j = 0; j < kC; ++j)
    s_o[lane][wp * kC + j] = make_uint2(pack2(acc[j].x * inv, acc[j].y * inv, a.f16),
                                        pack2(acc[j].z * inv, acc[j].w * inv, a.f16));
  if (a.lse && wp == 0 && r < rows)
    a.lse[static_cast<int64_t>(head) * a.num_tokens + q.row0 + tok] =
        none ? (a.sink ? a.sink[head] : -INFINITY) : (mt - shift) * kLn2 + logf(lt);
  __syncthreads();
  constexpr int kPer = 128 / DV;  // rows a warp writes at once
  for (int i = wp * kPer + lane / (DV / 4); i < 32; i += 8 * kPer) {
    const int rr = r0 + i;
    if (rr >= rows) break;
    const int tk = div_group(a, rr);
    uint16_t* op = a.o + (static_cast<int64_t>(q.row0 + tk) * a.Hq + d.z * a.group + rr -
                          tk * a.group) * DV;
    reinterpret_cast<uint2*>(op)[lane % (DV / 4)] = s_o[i][lane % (DV / 4)];
  }
}

template <int KIND, int DQK, int DV>
cudaError_t chunk_one(const Args& a, int sms, cudaStream_t st) {
  using L = ChunkCfg<KIND, DQK, DV>;
  auto kern = chunk_kernel<KIND, DQK, DV>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  CacheMaps maps;
  const int slots = a.page_shift < 7 ? 1 << a.page_shift : 128;
  const bool codes = KIND == kCacheE4m3;
  if (!cache_map(&maps.k, KIND, a.kc, DQK, a, a.k_tok, a.k_head, a.k_page, slots,
                 codes ? DQK : 128, codes ? 0 : 128) ||
      !cache_map(&maps.v, KIND, a.vc, DV, a, a.v_tok, a.v_head, a.v_page, slots, codes ? DV : 128,
                 codes ? 0 : 128))
    return cudaErrorInvalidValue;
  const unsigned ctas = sms < kMaxChunkCtas ? sms : kMaxChunkCtas;
  e = launch_early(kern, dim3(ctas), dim3(512), L::kSmem, st, a, maps);
  if (e != cudaSuccess) return e;
  return launch_early(chunk_join_kernel<DV>, dim3(ctas, kChunkRows / 32), dim3(256), 0, st, a,
                      KIND == kCacheBf16 ? 0.f : 7.f);
}

template <int KIND>
cudaError_t chunk_dims(const Args& a, int sms, cudaStream_t st) {
  if (a.d_v == 64) {
    if (a.d_qk == 64) return chunk_one<KIND, 64, 64>(a, sms, st);
    if (a.d_qk == 128) return chunk_one<KIND, 128, 64>(a, sms, st);
    return chunk_one<KIND, 192, 64>(a, sms, st);
  }
  if (a.d_qk == 64) return chunk_one<KIND, 64, 128>(a, sms, st);
  if (a.d_qk == 128) return chunk_one<KIND, 128, 128>(a, sms, st);
  return chunk_one<KIND, 192, 128>(a, sms, st);
}

}  // namespace
}  // namespace paged
}  // namespace attn
