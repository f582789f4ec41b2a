// Attention over the paged latent cache (tcgen05).
//
// Mathematics and tiling.  All heads of a token, and all new tokens of a sequence,
// attend to the same rows [c | k_r], and c is also the value.  The (token, head)
// rows are the columns of transposed products, so that 16 of them fill an MMA as
// well as 64 do:
//   S^T [64 keys x N] = [c | k_r] [q_lat | q_rot]^T,
//   O^T [d_c x N] += c^T P^T, in blocks of 128 coordinates,
// with the rows of a tile in shared memory once: the first product reads them as
// they lie (K-major), the second turned (MN-major).  N is 16, 32 or 64; O^T takes
// d_c / 128 * N columns of tensor memory and two tiles of scores 2 N.
//
// The softmax runs down the columns.  A thread holds two keys of N / 8 rows (the
// 16x256b shape).  The running maximum follows the true one within 2^8, so whether
// any row's has to move is one barrier's vote; only then (the first tile, and
// rarely after it) is the maximum joined across threads and O rescaled.  Sums stay
// in each thread's registers until the end.
//
// Work split.  As in the kernels of the paged cache: all tiles in order (sequence,
// row block, tile) cut into equal shares, one a block, one block an SM; pieces of
// a row block meet in a second kernel in a fixed order.  Where a token (or a few)
// has more rows than a block takes, two neighbouring blocks go through the same
// tiles, each for its 64 rows: the second finds them in the L2 cache.
//
// What bounds it.  One row read is 1152 bytes (d_c 512) for 2176 FLOP a (token, head):
//  - 16 rows: HBM (64 ragged contexts, 16 heads, 262 MB: 56 us, of which 39 at 6.7
//    TB/s; the rest are a block's start, 3 us, its state, 1.6, and the join);
//  - 64 rows: two tiles in shared memory, so that a tile's copies wait for the
//    products of the one before the last: 3570 clocks a tile where HBM allows 3390
//    (4 contexts of 100-131 k keys, 64 heads: 107 us, 4.9 TB/s);
//  - chunks of prompts, whose tiles come from the L2 cache: shared memory.  A tile of
//    64 rows moves 328 KB through it (147 for S, 98 for O, 82 written), 2560 clocks at
//    128 bytes each, and takes 2500-2700; its MMAs alone take 1960 (231 us for three
//    chunks over up to 16 k keys, 882 TFLOP/s, tensor pipe 58 % busy).  Pairs of blocks
//    are bound by it too (128 heads, 4 contexts: 148 us, one read of 527 MB, 54 % busy).
//
// Roles: an MMA issuer for each product, TMA producer, scheduler (a warp each), eight
// softmax warps (four read a tile's 64 lanes, for one half of the columns), four
// warps that copy queries.
//
// Values that are not finite in a tile that some rows mask in part are taken out of
// the product (their zero weight would make NaN of them); a row that keeps such a
// key gets NaN in that coordinate in the epilogue, which is what its score makes of
// it (0 * inf where the score is -inf, NaN throughout otherwise); O = 0 where no
// score of the row is above -inf.
#pragma once
#include <cfloat>
#include <climits>

#include "latent.cuh"

namespace attn {
namespace paged {
namespace {

using namespace sm103;

constexpr int kKeys = 64;      // keys a tile
constexpr int kThreads = 512;  // warps: S, TMA, scheduler, P c, 8 softmax, 4 queries
constexpr float kLazy = 8.f;
// Blocks in pairs bring tiles to the L2 cache this many ahead of their copies, which
// then take 740 clocks instead of 2000 or more: two tiles in shared memory do not
// cover that.  (4 contexts of 100-131 k keys, 128 heads: 150 us with 2 or 3, 157 with
// 5, 164 without.  Blocks that work alone are paced by HBM, where it only disturbs:
// 64 heads 108 us without, 111 with 2, 148 with 5.)
constexpr int kPrefetch = 2;

struct LatentMaps {
  CUtensorMap lat, rope;
};

// A piece of a block of rows, as the scheduler warp hands it to the others.
struct Piece {
  int n, key;   // key tiles (0: no row keeps a key, < 0: the end), first key
  int seq, rb;  // sequence, block of rows
  int first, whole;  // begins with the block's first tile; holds all its tiles
  int64_t end;       // in the first piece of a split block: of its units, of all
  int row0, new_rows, pos0, hi;  // of the sequence: first row, tokens, first position, keys
  int2 any, all;     // keys some row, and every row, of the block keeps
};

// a / b for a < 2^20: the approximate quotient (two units in the last of 24 bits)
// is off by one at most.
__device__ __forceinline__ uint32_t div_small(uint32_t a, uint32_t b) {
  const uint32_t q = __float2uint_rz(__fdividef(__uint2float_rz(a), __uint2float_rz(b)));
  const int32_t r = static_cast<int32_t>(a - q * b);
  return r < 0 ? q - 1 : r >= static_cast<int32_t>(b) ? q + 1 : q;
}
// Units in equal shares, block i from floor(i total / ctas) on.  (The divisions of
// 64 bits, and of 32, take a tenth of the time to a block's first copy, so the
// usual sizes go without.)
struct Shares {
  int64_t each;
  int rest, ctas;
  __device__ __forceinline__ int64_t begin(int i) const {
    return i * each + div_small(i * rest, ctas);
  }
  // The first block that does not begin before unit `end`.
  __device__ __forceinline__ int before(int64_t end) const {
    int i = max(0, static_cast<int>(__fdividef(static_cast<float>(end), static_cast<float>(each + 1))) - 2);
    while (i < ctas && begin(i) < end) ++i;
    return i;
  }
};
__device__ __forceinline__ Shares shares_of(int64_t total, int ctas) {
  Shares s;
  s.ctas = max(ctas, 1);
  s.each = total >> 20 ? total / s.ctas : div_small(static_cast<uint32_t>(total), s.ctas);
  s.rest = static_cast<int>(total - s.each * s.ctas);
  return s;
}

template <int N, int SLOTS, int RSLOTS>
struct LatentAux {
  uint64_t lat_full[SLOTS], lat_empty[SLOTS], rope_full[RSLOTS], rope_empty[RSLOTS];
  uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full, o_done, o_empty;
  uint64_t piece_full[4], piece_empty[4];
  uint64_t drain[2];
  uint32_t tmem;
  int abort;
  uint32_t bad;     // number + 1 of the last piece a value was taken out of
  int ok_mask[8];   // by tile: 16-key groups whose page exists
  int64_t begin;  // the block's first unit
  Shares shares;
  Piece piece[4];
  int row_lo[N], row_hi[N];
  float col[4][N];  // by softmax warp: maxima, or sums
  alignas(16) float fac[N];  // factors of the rows' O
  float top[N];              // the rows' maxima
};

template <int DC, int N>
struct LatentCfg {
  static constexpr int kNB = DC / 128;       // value blocks of a tile
  static constexpr int kSlot = kKeys * 256;  // one block: 128 coordinates of 64 keys
  static constexpr int kRope = kKeys * 128;
  static constexpr int kP = kKeys * 128;     // P^T [64 keys][64 rows], N of them used
  static constexpr int kQ = N * (DC + kLatentRope) * 2;
  static constexpr int kRSlots = DC == 512 ? 2 : 4;
  static constexpr int kAuxRoom = 3 * 1024;
  static constexpr int kFit = (227 * 1024 - kQ - kP - kRSlots * kRope - kAuxRoom) / kSlot;
  static constexpr int kSlots = kFit > 4 * kNB ? 4 * kNB : kFit;
  static_assert(kSlots >= 2 * kNB, "two tiles");
  static constexpr int kLatOff = kQ;
  static constexpr int kRopeOff = kLatOff + kSlots * kSlot;
  static constexpr int kPOff = kRopeOff + kRSlots * kRope;
  static constexpr int kAuxOff = kPOff + kP;
  using Aux = LatentAux<N, kSlots, kRSlots>;
  static constexpr int kSmem = kAuxOff + (static_cast<int>(sizeof(Aux)) + 127) / 128 * 128;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColO = 2 * N;
};

// One sequence and the keys it has in the cache.
struct SeqView {
  Seq q;
  int hi;
};
__device__ __forceinline__ SeqView view_of(const Args& a, int s) {
  SeqView v;
  v.q = load_seq(a, s);
  v.hi = min(v.q.len, a.max_pages << a.page_shift);
  return v;
}
// Row blocks of `rows` rows (a power of two).
__device__ __forceinline__ int blocks_of(const Args& a, const SeqView& v, int rows) {
  return (v.q.n * a.group + rows - 1) >> (31 - __clz(rows));
}
// Keys [x, y) that some (any) or every row of rows [r0, r1) keeps.
__device__ __forceinline__ int2 keys_any(const Args& a, const SeqView& v, int r0, int r1) {
  const int pos0 = v.q.len - v.q.n;
  const int lo = div_group(a, r0), hi = div_group(a, min(r1, v.q.n * a.group) - 1);
  return make_int2(a.window >= 0 ? max(0, pos0 + lo - a.window) : 0,
                   a.causal ? min(v.hi, pos0 + hi + 1) : v.hi);
}
__device__ __forceinline__ int2 keys_all(const Args& a, const SeqView& v, int r0, int r1) {
  const int pos0 = v.q.len - v.q.n;
  const int lo = div_group(a, r0), hi = div_group(a, min(r1, v.q.n * a.group) - 1);
  return make_int2(a.window >= 0 ? max(0, pos0 + hi - a.window) : 0,
                   a.causal ? min(v.hi, pos0 + lo + 1) : v.hi);
}
// A block of rows costs its tiles and about as much as this many more: queries to
// load, a pipeline to fill, O to write (131 KB of a partial state of 64 rows).  Shares
// are cut by that sum.  (6, 8, 10, 12, 15: three chunks over long prefixes, 64 rows,
// 243, 233, 237, 234, 236 us; 1, 2, 3, 4: 64 ragged contexts, 16 rows, 56.9, 55.6,
// 56.4, 56.9.)
template <int N>
constexpr int kStart = N == 64 ? 8 : 2;
__device__ __forceinline__ int tiles_of(const Args& a, const SeqView& v, int rows, int rb) {
  const int2 k = keys_any(a, v, rb * rows, (rb + 1) * rows);
  return max(1, (k.y - (k.x & ~(kKeys - 1)) + kKeys - 1) / kKeys);
}
// Units of a warp's sequences: `per` a lane, from `first` on.  The row blocks of a
// sequence that has many (a prompt's chunk) are summed by all lanes together.
template <int N>
__device__ __forceinline__ int64_t units_of(const Args& a, int rows, int first, int per) {
  const int lane = threadIdx.x & 31;
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    SeqView v = {{0, 0, 0}, 0};
    int nrb = 0;
    if (first + i < a.num_seqs) {
      v = view_of(a, first + i);
      if (outside(a, v.q)) flag_bounds(a);
      nrb = blocks_of(a, v, rows);
    }
    const bool many = nrb > 2;
    if (!many)
      for (int rb = 0; rb < nrb; ++rb) mine += kStart<N> + tiles_of(a, v, rows, rb);
    unsigned todo = __ballot_sync(0xffffffffu, many);
    while (todo) {
      const int o = __ffs(todo) - 1;
      todo &= todo - 1;
      SeqView u;
      u.q.len = __shfl_sync(0xffffffffu, v.q.len, o);
      u.q.n = __shfl_sync(0xffffffffu, v.q.n, o);
      u.hi = __shfl_sync(0xffffffffu, v.hi, o);
      const int n = __shfl_sync(0xffffffffu, nrb, o);
      int64_t sum = 0;
      for (int rb = lane; rb < n; rb += 32) sum += kStart<N> + tiles_of(a, u, rows, rb);
      const int lo = __reduce_add_sync(0xffffffffu, static_cast<int>(sum & 0xffffff));
      const int hi = __reduce_add_sync(0xffffffffu, static_cast<int>(sum >> 24));
      if (lane == o) mine += lo + (static_cast<int64_t>(hi) << 24);
    }
  }
  return mine;
}

// Walks the block's pieces (the scheduler warp does).  Units [0, kStart<N>) of a block
// of rows are its start, the others its tiles.
struct Walk {
  int64_t done, share;  // units behind the current piece's first, and in all
  int seq, rb, u0;
  int rows;  // of a block of rows
  SeqView v;
  // the current piece: tiles [t0, t1) of nt
  int u1, t0, t1, nt;
  int2 any;  // keys some row of the block of rows keeps
};
template <int N>
__device__ __forceinline__ bool walk_piece(const Args& a, Walk& w) {
  w.nt = tiles_of(a, w.v, w.rows, w.rb);
  w.u1 = static_cast<int>(min(static_cast<int64_t>(w.nt + kStart<N>), w.u0 + (w.share - w.done)));
  w.t0 = max(0, w.u0 - kStart<N>);
  w.t1 = max(0, w.u1 - kStart<N>);
  w.any = keys_any(a, w.v, w.rb * w.rows, (w.rb + 1) * w.rows);
  return w.t1 > w.t0;
}
// The first sequence from s on that has rows (or one behind the last): all lanes, a run
// of empty ones kSkip a lane at a time.  (Not inlined, as range_at below: what few calls
// reach would delay the start of all, by the instructions to be fetched.)
constexpr int kSkip = 4;
__device__ __noinline__ int next_rows(const Args& a, int s) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (; s < a.num_seqs; s += 32 * kSkip) {
    unsigned has[kSkip];
#pragma unroll
    for (int i = 0; i < kSkip; ++i) {
      const int x = s + 32 * i + lane;
      has[i] = __ballot_sync(0xffffffffu, x < a.num_seqs && load_seq(a, min(x, a.num_seqs - 1)).n > 0);
    }
#pragma unroll
    for (int i = 0; i < kSkip; ++i)
      if (has[i]) return s + 32 * i + __ffs(has[i]) - 1;
  }
  return a.num_seqs;
}
// The next piece with tiles.  (There is one while the share lasts, unless the offsets
// or lengths are changed under the call: then the walk ends with the sequences.)
template <int N>
__device__ __forceinline__ bool walk_next(const Args& a, Walk& w) {
  do {
    w.done += w.u1 - w.u0;
    if (w.done >= w.share) return false;
    w.u0 = 0;
    if (++w.rb >= blocks_of(a, w.v, w.rows)) {
      w.rb = 0;
      for (++w.seq;; w.seq = next_rows(a, w.seq + 1)) {
        if (w.seq >= a.num_seqs) return false;
        w.v = view_of(a, w.seq);
        if (w.v.q.n > 0) break;
      }
    }
  } while (!walk_piece<N>(a, w));
  return true;
}

// Where the sequences' units are summed.  Few sequences of few row blocks: by the
// scheduler warp, `per` a lane, without a barrier, so that the other roles start
// meanwhile.  Otherwise by all warps: 2 `ranges` lanes of each take `per` sequences
// and leave their units in shared memory (range r at 32 (r % ranges) + r / ranges),
// and a lane of the scheduler warp then stands for `ranges` of them.
struct Split {
  bool alone;
  int ranges, per;
};
__device__ __forceinline__ Split split_of(const Args& a, int rows) {
  Split s;
  s.alone = a.num_seqs <= 32 &&
            static_cast<int64_t>(a.num_tokens) * a.group <= 2ll * rows * a.num_seqs;
  s.ranges = s.alone ? 1 : min(kThreads / 32, (a.num_seqs + 31) / 32);
  s.per = (a.num_seqs + 32 * s.ranges - 1) / (32 * s.ranges);
  return s;
}

// The sequence of [s, last) that holds unit `off` of theirs, and the unit's number in it:
// 32 at a time, a lane each.
struct At {
  int64_t off;
  int seq;
};
template <int N>
__device__ __noinline__ At range_at(const Args& a, int rows, int s, int last, int64_t off) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (; s < last; s += 32) {
    const int64_t n = units_of<N>(a, rows, s + lane < last ? s + lane : a.num_seqs, 1);
    int64_t upto = n;
#pragma unroll 1
    for (int i = 1; i < 32; i <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, i);
      if (lane >= i) upto += y;
    }
    const unsigned in = __ballot_sync(0xffffffffu, upto > off);
    if (in) {
      const int f = __ffs(in) - 1;
      return {off - __shfl_sync(0xffffffffu, upto - n, f), s + f};
    }
    off -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return {off, last};
}

// This block's share, found by the scheduler warp.
template <int N, class Aux>
__device__ __forceinline__ void walk_init(const Args& a, Aux* x, const int64_t* scratch,
                                          const Split& sp, int block, int blocks, int rows,
                                          Walk& w) {
  const int lane = threadIdx.x & 31;
  int64_t mine = 0;
  if (sp.alone) {
    mine = units_of<N>(a, rows, lane * sp.per, sp.per);
  } else {
    for (int i = 0; i < sp.ranges; ++i) mine += scratch[32 * i + lane];
  }
  // sums up to each lane
  int64_t sum = mine;
  if (__any_sync(0xffffffffu, mine >> 25 != 0)) {
#pragma unroll 1
    for (int i = 1; i < 32; i <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, i);
      if (lane >= i) sum += y;
    }
  } else {
    int x32 = static_cast<int>(mine);
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x32, i);
      if (lane >= i) x32 += y;
    }
    sum = x32;
  }
  const int64_t total = __shfl_sync(0xffffffffu, sum, 31);
  const int ctas = static_cast<int>(min(static_cast<int64_t>(blocks), total));
  w.done = w.share = 0;
  w.rows = rows;
  if (block >= ctas) return;
  const Shares sh = shares_of(total, ctas);
  const int64_t begin = sh.begin(block);
  w.share = sh.begin(block + 1) - begin;
  // the lane, the range and the sequence that hold the first unit
  const unsigned at = __ballot_sync(0xffffffffu, sum > begin);
  const int o = __ffs(at) - 1;
  int64_t off = begin - __shfl_sync(0xffffffffu, sum - mine, o);
  int r = 0;
  if (!sp.alone) {
    if (off >> 24 == 0) {  // all of the lane's ranges at once
      int upto =
          lane < sp.ranges ? static_cast<int>(min(scratch[32 * lane + o], int64_t{1} << 24)) : 0;
      const int n = upto;
#pragma unroll
      for (int i = 1; i < kThreads / 32; i <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, i);
        if (lane >= i) upto += y;
      }
      r = __ffs(__ballot_sync(0xffffffffu, upto > off)) - 1;
      off -= __shfl_sync(0xffffffffu, upto - n, r);
    } else {
      while (off >= scratch[32 * r + o]) off -= scratch[32 * r++ + o];
    }
  }
  int s = (o * sp.ranges + r) * sp.per;
  if (sp.per > 1) {
    const At at = range_at<N>(a, rows, s, min(a.num_seqs, s + sp.per), off);
    s = at.seq;
    off = at.off;
  }
  SeqView v;
  int rb = 0;
  for (;; ++s) {  // row blocks of 32 at a time, all lanes
    if (s >= a.num_seqs) {
      w.share = 0;
      return;
    }
    v = view_of(a, s);
    const int nrb = blocks_of(a, v, rows);
    for (rb = 0; rb < nrb; rb += 32) {
      const int n = rb + lane < nrb ? kStart<N> + tiles_of(a, v, rows, rb + lane) : 0;
      int upto = n;  // (32 row blocks of at most 2^24 tiles)
      if (nrb > 1) {
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, i);
          if (lane >= i) upto += y;
        }
      }
      const unsigned in = __ballot_sync(0xffffffffu, upto > off);
      if (in) {
        const int f = __ffs(in) - 1;
        off -= __shfl_sync(0xffffffffu, upto - n, f);
        rb += f;
        break;
      }
      off -= __shfl_sync(0xffffffffu, upto, nrb > 1 ? 31 : 0);
    }
    if (rb < nrb) break;
  }
  if (lane == 0) {
    x->begin = begin;
    x->shares = sh;
  }
  __syncwarp();
  w.seq = s;
  w.rb = rb;
  w.u0 = static_cast<int>(off);
  w.v = v;
  // a share that ends inside its only start has no piece
  if (!walk_piece<N>(a, w) && !walk_next<N>(a, w)) w.share = 0;
}

// Brings a box into the L2 cache.
__device__ __forceinline__ void prefetch_4d(const void* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// A barrier of the softmax warps that also tells whether any thread's p holds.
__device__ __forceinline__ bool softmax_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// PAIR: two neighbouring blocks walk the same pieces of row blocks of twice the rows,
// each for one half of them.
template <bool F16, int DC, int N, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ LatentArgs l, const __grid_constant__ LatentMaps maps) {
  using L = LatentCfg<DC, N>;
  constexpr int NB = L::kNB, NS = L::kSlots, NR = L::kRSlots;
  constexpr int kC = N / 8;                       // columns a softmax thread holds
  constexpr float kShift = F16 ? 7.f : 0.f;       // P <= 2^(7 + 8) in fp16
  constexpr int kKind = F16 ? kCacheF16 : kCacheBf16;
  extern __shared__ __align__(1024) uint8_t sm[];
  typename L::Aux* const x = reinterpret_cast<typename L::Aux*>(sm + L::kAuxOff);
  const Args& a = l.a;
  volatile int* const abort = &x->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023u) return;  // the swizzle needs it; the window starts aligned

  auto timeout = [&]() {
    if (a.status) *a.status = ATTN_ERR_DEVICE_TIMEOUT;
    *abort = 1;
  };
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&x->lat_full[s], 1);
      mbar_init(&x->lat_empty[s], 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&x->rope_full[s], 1);
      mbar_init(&x->rope_empty[s], 1);
    }
    mbar_init(&x->q_full, 128);
    mbar_init(&x->q_empty, 1);
    mbar_init(&x->s_full[0], 1);
    mbar_init(&x->s_full[1], 1);
    mbar_init(&x->s_empty[0], 8);
    mbar_init(&x->s_empty[1], 8);
    mbar_init(&x->p_full, 256);
    mbar_init(&x->o_done, 1);
    mbar_init(&x->o_empty, 256);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&x->piece_full[s], 1);
      mbar_init(&x->piece_empty[s], 2 + 1 + 4 + 8);  // MMA, producer, query, softmax warps
    }
    mbar_init(&x->drain[0], 1);
    mbar_init(&x->drain[1], 1);
    x->abort = 0;
    x->bad = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&x->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    prefetch_tensormap(&maps.lat);
    prefetch_tensormap(&maps.rope);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  constexpr int pair = PAIR ? 1 : 0;
  int64_t* const scratch = reinterpret_cast<int64_t*>(sm);  // where queries will lie
  const Split split = split_of(a, N << pair);
  if (!split.alone) {
    const int r = warp * 2 * split.ranges + lane;
    const int64_t mine = units_of<N>(a, N << pair,
                                     lane < 2 * split.ranges ? r * split.per : a.num_seqs, split.per);
    if (lane < 2 * split.ranges) scratch[32 * (r % split.ranges) + r / split.ranges] = mine;
    __syncthreads();
  }
  grid_dep_launch();
  const uint32_t tmem = x->tmem;

  // The i-th piece (in shared memory), and this warp's release of it.
  auto take = [&](uint32_t i, bool* ok) -> const Piece* {
    *ok = mbar_wait_warp(&x->piece_full[i & 3], (i >> 2) & 1, l.wait_ns);
    return &x->piece[i & 3];
  };
  auto release = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&x->piece_empty[i & 3]);
  };

  if (warp == 2) {
    // -------------------------------------------------------------- scheduler
    if (lane == 0) a.split_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    Walk w;
    walk_init<N>(a, x, scratch, split, blockIdx.x >> pair, gridDim.x >> pair, N << pair, w);
    const int half = blockIdx.x & ((1 << pair) - 1);
    bool ok = true, live = w.share > 0;
    for (uint32_t i = 0; ok;) {
      const int rb = (w.rb << pair) + half;
      if (!live || rb * N < w.v.q.n * a.group) {  // (the last block may have one half)
        if (i >= 4 &&
            !(ok = mbar_wait_warp(&x->piece_empty[i & 3], ((i >> 2) - 1) & 1, l.wait_ns)))
          break;
        if (lane == 0) {
          Piece& p = x->piece[i & 3];
          if (live) {
            // of the walk's tiles those that some row of the half keeps
            const int2 any = keys_any(a, w.v, rb * N, (rb + 1) * N);
            const int base = w.any.x & ~(kKeys - 1);
            const int lo = max(base + w.t0 * kKeys, any.x & ~(kKeys - 1));
            const int hi = min(base + w.t1 * kKeys, any.y);
            p.n = any.y > any.x && hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;
            p.key = lo;
            p.seq = w.seq;
            p.rb = rb;
            p.first = w.t0 == 0;
            p.whole = w.t0 == 0 && w.t1 == w.nt;
            p.end = x->begin + w.done + (w.nt + kStart<N> - w.u0);
            p.row0 = w.v.q.row0;
            p.new_rows = w.v.q.n;
            p.pos0 = w.v.q.len - w.v.q.n;
            p.hi = w.v.hi;
            p.any = any;
            p.all = keys_all(a, w.v, rb * N, (rb + 1) * N);
          } else {
            p.n = -1;
          }
          mbar_arrive(&x->piece_full[i & 3]);
        }
        ++i;
      }
      if (__any_sync(0xffffffffu, !live || *abort != 0)) break;
      live = walk_next<N>(a, w);
    }
    if (!ok && lane == 0) timeout();
  } else if (warp == 0) {
    // -------------------------------------------------------------- scores' issuer
    // Up to two tiles ahead of the softmax; a tile's blocks join as they land.
    constexpr uint32_t id_s = idesc_f32acc(F16 ? 0 : 1, kKeys, N, false, false);
    const uint32_t tm = warp_uniform(tmem);
    const uint64_t q_km = sdesc_sw128(smem_u32(sm), 16, 1024);
    const uint64_t lat_km = sdesc_sw128(smem_u32(sm + L::kLatOff), 16, 1024);
    const uint64_t rope_km = sdesc_sw128(smem_u32(sm + L::kRopeOff), 16, 1024);
    uint32_t k = 0, it = 0;
    bool ok = true;
    for (uint32_t pi = 0;; ++pi) {
      const Piece* const p = take(pi, &ok);
      const int n = ok ? p->n : -1;
      release(pi);
      if (n < 0) break;
      if (n == 0) continue;
      if (!(ok = mbar_wait_warp(&x->q_full, it & 1))) break;
      for (int j = 0; j < n && ok; ++j, ++k) {
        // the softmax has read the scores these replace
        if (k >= 2 && !(ok = mbar_wait_warp(&x->s_empty[k & 1], ((k >> 1) - 1) & 1))) break;
        const uint32_t d = tm + (k & 1) * N;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t e = k * NB + b, s = e % NS;
          if (!(ok = mbar_wait_warp(&x->lat_full[s], (e / NS) & 1))) break;
          tc_fence_after();
          mma_ss_warp<8, 4, 2, 506, 2, 8 * N - 6>(d, lat_km + ((s * L::kSlot) >> 4),
                                                  q_km + ((b * 2 * N * 128) >> 4), id_s,
                                                  b == 0 ? 0u : 1u);
        }
        const uint32_t s = k % NR;
        if (!ok || !(ok = mbar_wait_warp(&x->rope_full[s], (k / NR) & 1))) break;
        tc_fence_after();
        mma_ss_warp<4, 4, 2, 2, 2, 2>(d, rope_km + ((s * L::kRope) >> 4),
                                      q_km + ((NB * 2 * N * 128) >> 4), id_s, 1u);
        mma_commit_warp(&x->s_full[k & 1]);
        mma_commit_warp(&x->rope_empty[s]);
      }
      if (!ok) break;
      mma_commit_warp(&x->q_empty);
      ++it;
    }
    if (!ok && lane == 0) timeout();
    mma_commit_warp(&x->drain[0]);
    mbar_wait(&x->drain[0], 0, 200000000ull);
  } else if (warp == 3) {
    // -------------------------------------------------------------- P c's issuer
    // A warp of its own: neither product waits for what the other waits for.
    constexpr uint32_t id_o = idesc_f32acc(F16 ? 0 : 1, 128, N, true, true);
    const uint32_t tm = warp_uniform(tmem);
    const uint64_t lat_mn = sdesc_sw128(smem_u32(sm + L::kLatOff), kKeys * 128, 1024);
    const uint64_t p_mn = sdesc_sw128(smem_u32(sm + L::kPOff), kKeys * 128, 1024);
    uint32_t k = 0, it = 0;
    bool ok = true;
    for (uint32_t pi = 0;; ++pi) {
      const Piece* const p = take(pi, &ok);
      const int n = ok ? p->n : -1;
      release(pi);
      if (n < 0) break;
      if (n == 0) continue;
      if (it > 0 && !(ok = mbar_wait_warp(&x->o_empty, (it - 1) & 1))) break;
      for (int j = 0; j < n; ++j, ++k) {
        if (!(ok = mbar_wait_warp(&x->p_full, k & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t s = (k * NB + b) % NS;
          mma_ss_warp<4, 4, 128, 128, 128, 128>(tm + L::kColO + b * N,
                                                lat_mn + ((s * L::kSlot) >> 4), p_mn, id_o,
                                                j == 0 ? 0u : 1u);
          mma_commit_warp(&x->lat_empty[s]);
        }
        mma_commit_warp(&x->o_done);
      }
      if (!ok) break;
      ++it;
    }
    if (!ok && lane == 0) timeout();
    mma_commit_warp(&x->drain[1]);
    mbar_wait(&x->drain[1], 0, 200000000ull);
  } else if (warp == 1) {
    // -------------------------------------------------------------- TMA producer
    // A tile's copies, by blocks of 128 coordinates and then the rotated part.  Where
    // a page holds a whole tile, lane 0 makes them alone (a copy every 100 clocks or
    // so; with the warp's votes and syncs around each it was 460, and the copies set
    // the pace of chunks over long prefixes).  Otherwise a lane looks after one page's
    // part of 64 coordinates.  The table is read a tile ahead.
    const int rows_log = min(a.page_shift, 6), boxes = kKeys >> rows_log;
    const int page_mask = (1 << a.page_shift) - 1;
    const int box = lane % boxes, chunk = lane / boxes;
    const uint32_t lat0 = smem_u32(sm + L::kLatOff), rope0 = smem_u32(sm + L::kRopeOff);
    uint32_t k = 0, slot = 0, phase = 0, rslot = 0, rphase = 0;  // tiles; places in the rings
    bool ok = true;
    for (uint32_t pi = 0;; ++pi) {
      const Piece* const p = take(pi, &ok);
      if (!ok || p->n < 0) break;
      const int n = p->n, key0 = p->key, end = p->any.y;
      const int32_t* const table = a.table + p->seq * a.table_stride;
      release(pi);
      auto key_of = [&](int j) -> int { return key0 + j * kKeys + (box << rows_log); };
      auto load_entry = [&](int j) -> int {
        if (j >= n || key_of(j) >= end) return INT_MIN;
        const int col = key_of(j) >> a.page_shift;
        return col < a.max_pages ? table[col] : -1;
      };
      auto checked = [&](int id) -> int {
        if (id >= 0 && id < a.num_pages) return id;
        if (id != INT_MIN) flag_bounds(a);
        return -1;
      };
      if (boxes == 1) {
        if (lane == 0) {
          int ids[kPrefetch + 1];  // of tiles j, j + 1, ...
#pragma unroll
          for (int i = 0; i <= kPrefetch; ++i) ids[i] = load_entry(i);
          for (int j = 0; j < n && ok; ++j, ++k) {
            const int id = checked(ids[0]), first = key_of(j) & page_mask, far = ids[kPrefetch];
#pragma unroll
            for (int i = 0; i < kPrefetch; ++i) ids[i] = ids[i + 1];
            ids[kPrefetch] = load_entry(j + kPrefetch + 1);
            if (pair && far >= 0 && far < a.num_pages) {
#pragma unroll
              for (int b = 0; b < NB; ++b)
                prefetch_4d(&maps.lat, 0, key_of(j + kPrefetch) & page_mask, 2 * b, far);
              prefetch_4d(&maps.rope, 0, key_of(j + kPrefetch) & page_mask, 2 * NB, far);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (!(ok = mbar_wait(&x->lat_empty[slot], phase ^ 1))) break;
              // the arrival (release) publishes the mask; the copy follows it
              if (b == 0) x->ok_mask[k & 7] = id >= 0 ? 0xf : 0;
              mbar_arrive_expect_tx(&x->lat_full[slot], id >= 0 ? L::kSlot : 0);
              if (id >= 0)
                tma_load_4d(lat0 + slot * L::kSlot, &maps.lat, &x->lat_full[slot], 0, first, 2 * b,
                            id);
              if (++slot == NS) slot = 0, phase ^= 1;
            }
            if (!ok || !(ok = mbar_wait(&x->rope_empty[rslot], rphase ^ 1))) break;
            mbar_arrive_expect_tx(&x->rope_full[rslot], id >= 0 ? L::kRope : 0);
            if (id >= 0)
              tma_load_4d(rope0 + rslot * L::kRope, &maps.rope, &x->rope_full[rslot], 0, first,
                          2 * NB, id);
            if (++rslot == NR) rslot = 0, rphase ^= 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      } else {
        int ahead = load_entry(0);
        for (int j = 0; j < n && ok; ++j, ++k) {
          const int id = checked(ahead);
          ahead = load_entry(j + 1);
          const unsigned okm = __ballot_sync(0xffffffffu, id >= 0);
          const uint32_t rows = __popc(okm & ((1u << boxes) - 1)) << rows_log;
          const int g = (16 * (lane & 3)) >> rows_log;  // 16-key groups whose page exists
          const unsigned groups = __ballot_sync(0xffffffffu, okm >> g & 1) & 0xfu;
          const uint32_t at = static_cast<uint32_t>(box << rows_log) * 128;
          const int first = key_of(j) & page_mask;
          // (a lane's copy may be under way before lane 0 has told the barrier of
          // its bytes: the barrier's phase ends with lane 0's arrival at the earliest)
#pragma unroll 1
          for (int b = 0; b < NB && ok; ++b) {
            ok = mbar_wait(&x->lat_empty[slot], phase ^ 1);
            if (!ok) break;
            if (lane == 0) {
              if (b == 0) x->ok_mask[k & 7] = groups;
              mbar_arrive_expect_tx(&x->lat_full[slot], rows * 256);
            }
            if (chunk < 2 && id >= 0)
              tma_load_4d(lat0 + slot * L::kSlot + chunk * (kKeys * 128) + at, &maps.lat,
                          &x->lat_full[slot], 0, first, 2 * b + chunk, id);
            if (++slot == NS) slot = 0, phase ^= 1;
          }
          ok = ok && mbar_wait(&x->rope_empty[rslot], rphase ^ 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&x->rope_full[rslot], rows * 128);
          if (chunk == 0 && id >= 0)
            tma_load_4d(rope0 + rslot * L::kRope + at, &maps.rope, &x->rope_full[rslot], 0, first,
                        2 * NB, id);
          if (++rslot == NR) rslot = 0, rphase ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) timeout();
    // copies in flight land before the block may leave
    k = __shfl_sync(0xffffffffu, k, 0);
    for (uint32_t e = k * NB > NS ? k * NB - NS : 0; e < k * NB; ++e)
      mbar_wait(&x->lat_full[e % NS], (e / NS) & 1, 100000000ull);
    for (uint32_t e = k > NR ? k - NR : 0; e < k; ++e)
      mbar_wait(&x->rope_full[e % NR], (e / NR) & 1, 100000000ull);
  } else if (warp >= 12) {
    // -------------------------------------------------------------- queries
    // A warp a row: 16 bytes a lane to where the MMA reads them.
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t pi = 0;; ++pi) {
      const Piece* const p = take(pi, &ok);
      if (!ok || p->n < 0) break;
      const int n = p->n, r0 = p->rb * N, row0 = p->row0, new_rows = p->new_rows;
      release(pi);
      if (n == 0) continue;
      if (it > 0 && !(ok = mbar_wait_warp(&x->q_empty, (it - 1) & 1, l.wait_ns))) break;
      // a lane finds a row's addresses (offsets in 16-byte units, < 0: no such row)
      constexpr int kRowsWarp = N / 4;
      int64_t lat_at = -1, rot_at = 0;
      if (lane < kRowsWarp) {
        const int rr = r0 + (warp - 12) * kRowsWarp + lane, tok = div_group(a, rr);
        if (tok < new_rows) {
          const int64_t t = row0 + tok, head = rr - tok * a.group;
          lat_at = (t * l.q_lat_tok + head * l.q_lat_head) >> 3;
          rot_at = (t * l.q_rot_tok + head * l.q_rot_head) >> 3;
        }
      }
      const uint4* const lat = reinterpret_cast<const uint4*>(l.q_lat);
      const uint4* const rot = reinterpret_cast<const uint4*>(l.q_rot);
#pragma unroll 4
      for (int i = 0; i < kRowsWarp; ++i) {
        const int r = (warp - 12) * kRowsWarp + i;
        const int64_t la = __shfl_sync(0xffffffffu, lat_at, i);
        const int64_t ra = __shfl_sync(0xffffffffu, rot_at, i);
        const int bytes = la >= 0 ? 16 : 0;
        const uint4* const src = lat + (la >= 0 ? la + lane : 0);
        const uint32_t dst = smem_u32(sm) + (lane >> 3) * (N * 128) + r * 128 +
                             (((lane & 7) ^ (r & 7)) << 4);
        auto copy = [&](uint32_t to, const uint4* from) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                       "r"(bytes)
                       : "memory");
        };
#pragma unroll
        for (int u = 0; u < DC / 256; ++u)
          copy(dst + u * 4 * (N * 128), src + (la >= 0 ? 32 * u : 0));
        if (lane < 8) copy(dst + (DC / 64) * (N * 128), rot + (la >= 0 ? ra + lane : 0));
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(&x->q_full);
      ++it;
    }
    if (!ok && lane == 0) timeout();
  } else if (warp >= 4) {
    // -------------------------------------------------------------- softmax
    // warp: 16 keys of the tile, one half of the rows
    const int sw = warp & 3, half = (warp - 4) >> 2, st = tid - 128;
    const int g = lane >> 2, c0 = half * (N / 2) + 2 * (lane & 3);
    const uint32_t lanes = static_cast<uint32_t>(sw * 32) << 16;
    const uint32_t o_half = tmem + lanes + L::kColO + half * (NB / 2) * N;
    const float fac = a.scale * kLog2e;
    uint32_t k = 0, it = 0;
    // A wait that ran out here is told to the other softmax warps at their next
    // vote, so that all eight leave together and none stays at their barrier.
    bool failed = false;
    for (uint32_t pi = 0;; ++pi) {
      bool ok;
      const Piece* const p = take(pi, &ok);
      failed |= !ok;
      const int n = ok ? p->n : -1, key0 = p->key;
      if (n >= 0 && st < N) {  // keys that row st keeps
        const int tok = div_group(a, p->rb * N + st), pos = p->pos0 + tok;
        x->row_lo[st] = a.window >= 0 ? max(0, pos - a.window) : 0;
        x->row_hi[st] = tok < p->new_rows ? (a.causal ? min(p->hi, pos + 1) : p->hi) : 0;
      }
      if (softmax_any(failed) || n < 0) break;
      // column c0 + 8 b + e is index 2 b + e
      float m[kC], sum[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        m[i] = -FLT_MAX;
        sum[i] = 0.f;
      }
      for (int j = 0; j < n; ++j, ++k) {
        const int key = key0 + j * kKeys;
        failed |= !mbar_wait_warp(&x->s_full[k & 1], (k >> 1) & 1);
        // (the tile has landed; this orders what the producer wrote for it)
        failed |= !mbar_wait_warp(&x->lat_full[(k * NB) % NS], (k * NB / NS) & 1);
        tc_fence_after();
        uint32_t u[2 * kC];
        tmem_ld16x256b(tmem + lanes + (k & 1) * N + half * (N / 2), u);
        const int okm = x->ok_mask[k & 7];
        const bool whole = key >= p->all.x && key + kKeys <= p->all.y && okm == 0xf;
        tmem_ld_wait(u);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x->s_empty[k & 1]);
        float s[2 * kC];
#pragma unroll
        for (int i = 0; i < 2 * kC; ++i) s[i] = __uint_as_float(u[i]);
        if (!whole) {
          const int k0 = key + 16 * sw + g;
          const bool page = okm >> sw & 1;
#pragma unroll
          for (int b = 0; b < N / 16; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int lo = x->row_lo[c0 + 8 * b + e], hi = x->row_hi[c0 + 8 * b + e];
              if (!(page && k0 >= lo && k0 < hi)) s[4 * b + e] = -INFINITY;
              if (!(page && k0 + 8 >= lo && k0 + 8 < hi)) s[4 * b + 2 + e] = -INFINITY;
            }
        }
        // exponents against the maximum so far
        bool grow = failed;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const float mx = fmaxf(s[4 * (i >> 1) + (i & 1)], s[4 * (i >> 1) + 2 + (i & 1)]);
          grow |= fmaf(mx, fac, -m[i]) > kLazy;
        }
        bool again = false;
        if (softmax_any(grow)) {
#pragma unroll
          for (int i = 0; i < kC; ++i) {
            float mx = fmaxf(s[4 * (i >> 1) + (i & 1)], s[4 * (i >> 1) + 2 + (i & 1)]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            if (g == 0) x->col[sw][c0 + 8 * (i >> 1) + (i & 1)] = mx;
          }
          if (softmax_any(failed)) {
            failed = true;
            break;
          }
#pragma unroll
          for (int i = 0; i < kC; ++i) {
            const int c = c0 + 8 * (i >> 1) + (i & 1);
            const float mx = fmax3(x->col[0][c], x->col[1][c], fmaxf(x->col[2][c], x->col[3][c])) * fac;
            const bool up = mx - m[i] > kLazy;
            const float f = up ? ex2_approx(m[i] - mx) : 1.f;
            if (up) m[i] = mx;
            sum[i] *= f;
            if (sw == 0 && g == 0) x->fac[c] = f;
          }
          again = softmax_any(j > 0);
        }
        // P, over its rounded pairs of columns
        uint32_t pk[kC];
#pragma unroll
        for (int b = 0; b < N / 16; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2_approx(fmaf(s[4 * b + 2 * h], fac, kShift - m[2 * b]));
            const float p1 = ex2_approx(fmaf(s[4 * b + 2 * h + 1], fac, kShift - m[2 * b + 1]));
            sum[2 * b] += p0;
            sum[2 * b + 1] += p1;
            pk[2 * b + h] = F16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
        // the tile before this one is done with P and O
        if (k > 0) failed |= !mbar_wait_warp(&x->o_done, (k - 1) & 1);
        tc_fence_after();
        if (again) {
#pragma unroll 1
          for (int q = 0; q < NB * N / 32; ++q) {  // this half of the blocks
            uint32_t o[16];
            tmem_ld32x32b_x16(o_half + q * 16, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&x->fac[(q * 16 + e) % N]);
              o[e] = __float_as_uint(__uint_as_float(o[e]) * f.x);
              o[e + 1] = __float_as_uint(__uint_as_float(o[e + 1]) * f.y);
              o[e + 2] = __float_as_uint(__uint_as_float(o[e + 2]) * f.z);
              o[e + 3] = __float_as_uint(__uint_as_float(o[e + 3]) * f.w);
            }
            tmem_st32x32b_x16(o_half + q * 16, o);
          }
          tmem_st_wait();
        }
        {
          const uint32_t row = smem_u32(sm + L::kPOff) + (16 * sw + g) * 128;
#pragma unroll
          for (int b = 0; b < N / 16; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + h * 1024 +
                                                                  (((half * (N / 16) + b) ^ g) << 4) +
                                                                  4 * (lane & 3)),
                           "r"(pk[2 * b + h])
                           : "memory");
        }
        if (!whole) {
          // keys no row keeps become zeros, and what is not finite of those that
          // some rows keep and some do not
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t e = k * NB + b;
            failed |= !mbar_wait_warp(&x->lat_full[e % NS], (e / NS) & 1);
          }
          const int2 any = p->any, all = p->all;
#pragma unroll 1
          for (int r = st >> 3; r < kKeys; r += 32) {
            const int kk = key + r;
            const bool in = (okm >> (r >> 4) & 1) && kk >= any.x && kk < any.y;
            if (in && kk >= all.x && kk < all.y) continue;
#pragma unroll 1
            for (int b = 0; b < 2 * NB; ++b) {
              const uint32_t q = smem_u32(sm + L::kLatOff) + ((k * NB + (b >> 1)) % NS) * L::kSlot +
                                 (b & 1) * (kKeys * 128) + r * 128 + ((st & 7) << 4);
              if (!in) {
                st_shared_v4(q, 0, 0, 0, 0);
                continue;
              }
              const uint4 v = lds128(q);
              if (not_finite<kKind>(v.x) | not_finite<kKind>(v.y) | not_finite<kKind>(v.z) |
                  not_finite<kKind>(v.w)) {
                x->bad = it + 1;
                st_shared_v4(q, finite_only<kKind>(v.x), finite_only<kKind>(v.y),
                             finite_only<kKind>(v.z), finite_only<kKind>(v.w));
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&x->p_full);
      }
      // ---- epilogue: O or the piece's partial state
      const bool complete = p->whole;
      const int slot = 2 * blockIdx.x + p->first;
      const int rows = min(N, p->new_rows * a.group - p->rb * N);
      const int64_t out0 = static_cast<int64_t>(p->row0) * a.group + p->rb * N;  // of [T * H]
#pragma unroll
      for (int i = 0; i < kC; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);
        if (g == 0) {
          const int c = c0 + 8 * (i >> 1) + (i & 1);
          x->col[sw][c] = sum[i];
          if (sw == 0) x->top[c] = m[i];
        }
      }
      if (softmax_any(failed)) break;
      float lt = 0.f, mt = 0.f;
      bool none = false;
      int head = 0, tok = 0;
      if (st < N) {
        lt = x->col[0][st] + x->col[1][st] + (x->col[2][st] + x->col[3][st]);
        const float mx = mt = x->top[st];
        none = mx == -FLT_MAX && lt == 0.f;
        const int rr = p->rb * N + st;
        tok = div_group(a, rr);
        head = rr - tok * a.group;
        float keep = 1.f, norm = 1.f;
        if (complete) {
          if (a.sink && st < rows) {
            const float s2 = a.sink[head] * kLog2e;
            mt = none ? s2 : fmaxf(mx, s2);
            const float mu = mt == -INFINITY ? 0.f : mt;
            keep = ex2_approx(mx - mu);
            lt = lt * keep + ex2_approx(s2 - mu + kShift);
          }
          norm = keep / lt;
        }
        // (below 0: no score of the row is above -inf, O = 0; a piece does not know of
        // the others, and hands on what its keys of weight 0 made of O)
        x->fac[st] = complete && none ? -1.f : norm;
        if (complete && none) x->row_hi[st] = 0;
      }
      softmax_any(false);
      // (behind the barrier: the other warps are at O already)
      if (st < N && !complete) {
        float* const ml = reinterpret_cast<float*>(a.part_ml + static_cast<int64_t>(slot) * N);
        ml[st] = none ? -INFINITY : mt;
        ml[N + st] = none ? 0.f : lt;
      } else if (st < rows && a.lse) {
        a.lse[static_cast<int64_t>(head) * a.num_tokens + p->row0 + tok] =
            none ? (a.sink ? a.sink[head] : -INFINITY) : (mt - kShift) * kLn2 + logf(lt);
      }
      const bool bad = n > 0 && x->bad == it + 1;
      if (n > 0) {
        failed |= !mbar_wait_warp(&x->o_done, (k - 1) & 1);
        tc_fence_after();
      }
      constexpr int kCols = N < 32 ? N : 32;  // columns at a time
#pragma unroll 1
      for (int q = 0; q < NB / 2 * N / kCols; ++q) {
        const int cc = q * kCols % N;
        const int d = (half * (NB / 2) + q * kCols / N) * 128 + sw * 32 + lane;  // coordinate
        if (cc >= rows) continue;
        uint32_t o[kCols];
        if (n > 0) {
          if constexpr (kCols == 32) tmem_ld32x32b_x32(o_half + q * kCols, o);
          else tmem_ld32x32b_x16(o_half + q * kCols, o);
          tmem_ld_wait(o);
        }
        float v[kCols];
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(&x->fac[cc + i]);
          const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[i + e] = n > 0 && !(f[e] < 0.f) ? __uint_as_float(o[i + e]) * f[e] : 0.f;
        }
        if (bad) {
          // (keys that every row keeps have stayed in the product: only those before and
          // behind them, no more than the block has tokens, are looked at)
          for (int kk = max(key0, p->any.x); kk < min(key0 + n * kKeys, p->any.y); ++kk) {
            if (kk >= p->all.x && kk < p->all.y) {
              kk = p->all.y - 1;
              continue;
            }
            const int page = page_of(a, p->seq, kk);
            if (page < 0) continue;
            const float e =
                elem(reinterpret_cast<const uint16_t*>(
                         a.kc + page * a.k_page +
                         static_cast<int64_t>(kk & ((1 << a.page_shift) - 1)) * a.k_tok)[d],
                     F16);
            if (fabsf(e) < INFINITY) continue;
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (kk >= x->row_lo[cc + i] && kk < x->row_hi[cc + i]) v[i] = NAN;
          }
        }
        if (complete) {
          // neighbours swap, so that a lane has two coordinates of one row
          const bool odd = lane & 1;
          uint16_t* dst = a.o + (out0 + cc + odd) * DC + (d & ~1);
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            const float y = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
            const uint32_t w2 = odd ? pack2(y, v[i + 1], F16) : pack2(v[i], y, F16);
            if (cc + i + odd < rows) *reinterpret_cast<uint32_t*>(dst + i * DC) = w2;
          }
        } else {
          float* dst = a.part + (static_cast<int64_t>(slot) * N + cc) * DC + d;
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (cc + i < rows) dst[i * DC] = v[i];
        }
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&x->o_empty);
      }
      if (!complete && p->first && st == 0)
        a.split_desc[blockIdx.x] =
            make_int4(x->shares.before(p->end) - static_cast<int>(blockIdx.x >> pair), p->seq, p->rb,
                      0);
      if (softmax_any(failed)) break;  // (row bounds, `fac` and the piece have been read)
      release(pi);
      if (n > 0) ++it;
    }
    if (failed && lane == 0) timeout();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of split blocks of rows.  A warp takes 128 coordinates of a row,
// four a lane, and works alone: it finds the row's statistics itself while the
// first values are on their way, of many pieces a piece a lane.  The grid fills the
// SMs; its blocks read all descriptors at once.
constexpr int kJoinThreads = 512;
constexpr int kJoinMost = (kLatentMaxCtas + 31) / 32;  // pieces a lane
constexpr int kAhead = 4;                              // pieces whose values are in flight

__device__ __forceinline__ void join_add(float4& acc, const float4& v, float w) {
  acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z),
                    fmaf(v.w, w, acc.w));
}
template <bool F16, int DC, int N>
__global__ void __launch_bounds__(kJoinThreads, 2)
    latent_join_kernel(const __grid_constant__ Args a, int blocks, int step) {
  constexpr float kShift = F16 ? 7.f : 0.f;
  constexpr int kParts = DC / 128, kUnits = N * kParts;
  constexpr int64_t kPiece = N * DC / 4;  // 16-byte units of a piece's O
  __shared__ int s_first[kLatentMaxCtas];
  __shared__ unsigned s_has[kJoinMost];
  __shared__ int4 s_desc[kLatentMaxCtas];
  const int tid = threadIdx.x, lane = tid & 31;
  grid_dep_wait();
  // the blocks that hold a first piece, in order
  if (tid < 32 * kJoinMost) {
    int4 desc = make_int4(0, 0, 0, 0);
    if (tid < blocks) s_desc[tid] = desc = a.split_desc[tid];
    const unsigned has = __ballot_sync(0xffffffffu, desc.x != 0);
    if (lane == 0) s_has[tid >> 5] = has;
  }
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int i = 0; i < kJoinMost; ++i) {
    const unsigned has = s_has[i];
    if (tid < 32 && (has >> lane & 1))
      s_first[count + __popc(has & ((1u << lane) - 1))] = 32 * i + lane;
    count += __popc(has);
  }
  __syncthreads();
  const int units = count * kUnits;
  for (int unit = (tid >> 5) * gridDim.x + blockIdx.x; unit < units;
       unit += gridDim.x * (kJoinThreads / 32)) {
    const int first = s_first[unit / kUnits];
    const int4 d = s_desc[first];
    const int pieces = d.x;
    const int row = unit % kUnits / kParts, col = unit % kParts * 32 + lane;  // (16-byte columns)
    auto slot_of = [&](int p) -> int64_t { return 2 * first + p * step + (p == 0 ? 1 : 0); };
    const float* const ml = reinterpret_cast<const float*>(a.part_ml) + row;
    const float4* const part = reinterpret_cast<const float4*>(a.part) + row * (DC / 4) + col;
    float4 v[kAhead];
    auto fetch = [&](int p0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (p0 + j < pieces) v[j] = part[slot_of(p0 + j) * kPiece];
    };
    fetch(0);
    const Seq q = load_seq(a, d.y);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, sum = 0.f;
    if (pieces <= kAhead) {
      float mx[kAhead], l[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        mx[j] = j < pieces ? ml[slot_of(j) * (2 * N)] : -INFINITY;
        l[j] = j < pieces ? ml[slot_of(j) * (2 * N) + N] : 0.f;
        m = fmaxf(m, mx[j]);
      }
      const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (j >= pieces) break;
        const float w = ex2_approx(mx[j] - mu);
        sum = fmaf(l[j], w, sum);
        join_add(acc, v[j], w);
      }
    } else {
      float wt[kJoinMost], l[kJoinMost];
#pragma unroll
      for (int i = 0; i < kJoinMost; ++i) {
        const int p = lane + 32 * i;
        wt[i] = p < pieces ? ml[slot_of(p) * (2 * N)] : -INFINITY;
        l[i] = p < pieces ? ml[slot_of(p) * (2 * N) + N] : 0.f;
        m = fmaxf(m, wt[i]);
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
      const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int i = 0; i < kJoinMost; ++i) {
        wt[i] = ex2_approx(wt[i] - mu);
        sum = fmaf(l[i], wt[i], sum);
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
#pragma unroll
      for (int i = 0; i < kJoinMost; ++i) {
#pragma unroll 1
        for (int p0 = 32 * i; p0 < min(pieces, 32 * (i + 1)); p0 += kAhead) {
          if (p0 > 0) fetch(p0);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const float w = __shfl_sync(0xffffffffu, wt[i], (p0 + j) & 31);
            if (p0 + j < pieces) join_add(acc, v[j], w);
          }
        }
      }
    }
    const int rr = d.z * N + row, tok = div_group(a, rr), head = rr - tok * a.group;
    if (tok >= q.n) continue;
    const bool none = no_key(m, sum);
    float mt = m, lt = sum, keep = 1.f;
    if (a.sink) {
      const float s2 = a.sink[head] * kLog2e;
      mt = fmaxf(m, s2);
      const float mx = mt == -INFINITY ? 0.f : mt;
      keep = ex2_approx(m - mx);
      lt = sum * keep + ex2_approx(s2 - mx + kShift);
    }
    const float f = keep / lt;
    if (none) acc = make_float4(0.f, 0.f, 0.f, 0.f);
    else acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    reinterpret_cast<uint2*>(a.o + (static_cast<int64_t>(q.row0) * a.group + rr) * DC)[col] =
        make_uint2(pack2(acc.x, acc.y, F16), pack2(acc.z, acc.w, F16));
    if (a.lse && col == 0)
      a.lse[static_cast<int64_t>(head) * a.num_tokens + q.row0 + tok] =
          none ? (a.sink ? a.sink[head] : -INFINITY) : (mt - kShift) * kLn2 + logf(lt);
  }
}

template <bool F16, int DC, int N, bool PAIR>
cudaError_t latent_one(const LatentArgs& l, int sms, cudaStream_t st) {
  using L = LatentCfg<DC, N>;
  auto kern = latent_kernel<F16, DC, N, PAIR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  LatentMaps maps;
  const int slots = l.a.page_shift < 6 ? 1 << l.a.page_shift : kKeys;
  if (!latent_map(&maps.lat, l, slots, slots == kKeys ? 2 : 1) ||
      !latent_map(&maps.rope, l, slots, 1))
    return cudaErrorInvalidValue;
  const unsigned ctas = sms < kLatentMaxCtas ? sms : kLatentMaxCtas;
  e = launch_early(kern, dim3(ctas), dim3(kThreads), L::kSmem, st, l, maps);
  if (e != cudaSuccess) return e;
  return launch_early(latent_join_kernel<F16, DC, N>, dim3(2 * ctas), dim3(kJoinThreads), 0, st, l.a,
                      static_cast<int>(ctas), PAIR ? 4 : 2);
}

template <bool F16, int DC>
cudaError_t latent_rows(const LatentArgs& l, int rows, int sms, cudaStream_t st) {
  return rows == 16   ? latent_one<F16, DC, 16, false>(l, sms, st)
         : rows == 32 ? latent_one<F16, DC, 32, false>(l, sms, st)
         : l.pair     ? latent_one<F16, DC, 64, true>(l, sms, st)
                      : latent_one<F16, DC, 64, false>(l, sms, st);
}
template <bool F16>
cudaError_t launch_latent(const LatentArgs& l, int rows, int sms, cudaStream_t st) {
  return l.d_c == 512 ? latent_rows<F16, 512>(l, rows, sms, st)
                      : latent_rows<F16, 256>(l, rows, sms, st);
}

}  // namespace
}  // namespace paged
}  // namespace attn
