// Latent (absorbed) attention over the paged cache on the 5th-generation
// tensor cores (sm_103a), DeepSeek-V3 head shape, bf16:
//   s_j = scale * q . c_j (576 columns), o = sum_j softmax(s)_j c_j[0:512), lse
// for every row (new token, head); the rows of a sequence share its cache rows.
//
// A key is 1152 bytes and costs a row 2 * (576 + 512) FLOP: with 128 rows that
// is 242 FLOP/byte, just under the GPU's bf16 : HBM ratio of 289, so both the
// tensor pipe and HBM have to be kept near their limits, and what limits the
// tensor pipe is how its operands fit on chip:
//   * O (rows x 512 float32) lives in tensor memory.  128 rows would take all
//     512 columns and leave none for S, so an SM holds 64 rows: 256 columns,
//     in the layout where lanes 0-63 have the rows with one half of D's
//     columns and lanes 64-127 the same rows with the other half.  Four softmax
//     threads share a row, each with a quarter of the keys.
//   * an MMA takes a clock per 128 bytes that it reads from shared memory, when
//     that is more than its products do (measured: M=64, N=64, K=16 of the
//     single form 32 clocks, N=256 80; pair M=128 N=64 25, N=256 64), so S,
//     with its small N, is bound by re-reading the queries.
// Two forms (template parameter):
//   single (rows of a unit: 64)  one CTA, weight-stationary MMAs of M=64; a
//          stage serves as K (K-major, 9 blocks of 64 columns) and as V (the
//          first 8 blocks, MN-major).
//   pair   (rows: 128)  a cluster of two CTAs, cta_group::2 MMAs of M=128 (64
//          rows in each).  An operand of such an MMA sits at the same offset
//          in both CTAs, so V (each CTA 256 columns of all keys) cannot share
//          the place of K (each CTA all columns of half of the keys).
//   Both take 64 keys at a time from two stages.  (128 keys a tile halve the
//   reads of the queries in the pair form, but leave room for one stage: S,
//   softmax and P V then follow each other, 4840 clocks per 128 keys.)
// Work split: the units (sequence, 64 or 128 rows) are laid end to end, each
// as long as its key tiles and a constant for its start and end, and dealt out
// in equal contiguous shares, one per cluster, by the kernel itself from the
// lengths on the device.  A unit that lies in one share is written directly;
// the pieces of a cut one go to scratch as normalised float32 with their
// log-sums, and latent_combine_kernel joins them.
// With a mask (template parameter TREE, mla_tree_attn) a token sees the keys
// before its sequence's new tokens, and of these the ones in its mask: where a
// tile has any, a softmax thread takes its 16 keys' bits from the mask row, which
// it asks for before it waits for the scores.
// Measured, 64 keys at 1.6-1.95 GHz: single 3380 clocks, of which HBM's rate
// takes 3200 (128 sequences of up to 8192 keys, 32 heads: 110 us, 83% of copy
// bandwidth); pair 1700 with pages of 64 and about 2000 with pages of 16 (24
// sequences x 4 tokens x 128 heads: 79 us, 52% of the bf16 rate).  The pair's MMAs
// alone take 1425 of that.  Counted a tile and CTA, in lines of 128 bytes of shared
// memory: 1193 by the tensor pipe, 306 by the softmax; the copies write 545 more,
// whether through the same port is not known.  HBM does not hold the pair form with
// one token a sequence either: 128 sequences of 4096 keys take 130 us, their bytes
// 94.  Where such work lasts, power does: 16 x 4096 keys with trees of
// 32 nodes, 128 heads, take 440-460 us, 1260-1310 TFLOP/s, at 1370 of 1400 W and
// 1.8 GHz (matrix products of the library keep up 1690 at 1.44 GHz).  Not faster:
// K in three column groups with barriers of their own (550 us for 437); S and P V
// with one commit each for all that waits for them; new tokens' rows looked at a
// tile later (463 for 445).  A launch has some 10000 clocks around its tiles:
// finding its share, the first loads, the last rows out, and the joining kernel.
// Warps: 0 K loads, 1 V loads (pair), 2 MMA issue, 3 query loads and prefetches
// to L2, 4-11 softmax and epilogue (two a quarter of tensor memory's lanes).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "row_join.h"
#include "sm103.cuh"
#include "unit_sum.h"

namespace mla {
namespace sm103 {
namespace {

constexpr int LAT = 512, WIDTH = 576, NBLK = 9;  // row: 9 blocks of 64 columns
constexpr int CROWS = 64;                        // rows of O in a CTA
constexpr int BLK_BYTES = 64 * 128;              // 64 rows x 64 columns, 128-byte swizzled
constexpr int Q_BYTES = NBLK * BLK_BYTES;
constexpr int SWARPS = 8, STHREADS = 32 * SWARPS;  // softmax
constexpr int THREADS = 128 + STHREADS;
constexpr int MAPS = 7;  // cache boxes of 1, 2, 4 .. 64 rows
constexpr uint32_t TMEM_COLS = 512, S_COL = 256;  // O: columns 0-255, S: from 256
constexpr float LN2 = 0.69314718055994531f;
// O is rescaled only when a row's maximum has grown by more than this (log2):
// until then p is at most 2^8, which float32 sums and bf16's exponent hold
// without loss.
constexpr float RESCALE = 8.f;

constexpr int TILE = 64;     // keys
constexpr int SC = TILE / 2; // S columns in tensor memory
constexpr int NC = SC / 2;   // of a softmax thread
template <bool PAIR>
struct Cfg {
  static constexpr int UROWS = PAIR ? 128 : 64;     // rows of a unit
  static constexpr int KROWS = PAIR ? 32 : 64;      // keys of a tile in a CTA's K
  static constexpr int K_STAGE = NBLK * KROWS * 128;
  static constexpr int V_STAGE = PAIR ? 4 * BLK_BYTES : 0;
  static constexpr int NP = PAIR ? 2 : 1;           // P buffers
  static constexpr int KV_BYTES = 2 * (K_STAGE + V_STAGE);
  static constexpr int P_BYTES = NP * BLK_BYTES;
  static constexpr int USED = Q_BYTES + KV_BYTES + P_BYTES + 2048 + 48 * 8;

  static constexpr int SMEM = 232448;  // all of it; the rest is room for alignment
};
// Work split, in positions of a tile.  UNIT_COST: what a unit costs beyond its
// tiles (queries in, first scores, rows out: 5000 to 8000 clocks, a tile taking
// 2000 to 3400).  31 short sequences beside one of 131072 keys took 55.3, 48.3,
// 47.4 and 47.6 us with 2, 3, 4 and 5 in the pair form.  One less or more in both
// forms moves long and ragged batches by 2% at most; 128 heads, 1 x 2048 keys
// 15.6 and 14.6 us (so 14.0), 100 x 500 36.5 and 33.9 (32.5), 200 x 400 38.5 and
// 45.1 (45.4).
// MIN_SHARE: the least that a share is worth; shorter ones cost more in scratch
// traffic and joining than they save (2 and 8: 128 heads, 4 x 2048 keys 25.9 and
// 19.1 us, so 16.7; 1 x 6000 16.7 and 19.8, so 16.9; 16 heads, 1 x 2048 10.6 and
// 17.7, so 13.0).
template <bool PAIR>
constexpr int UNIT_COST = PAIR ? 4 : 2;
constexpr int MIN_SHARE = 4;
// A cut costs another UNIT_COST and the joining, some 10 tiles' time of the
// whole GPU when it is the only one.  So: no cut nearer than SNAP to a unit's
// end; none at all through units of up to SHORT positions; and where there are
// no more units than clusters, one each, unless the longest is more than
// WHOLE_SLACK beyond an equal share.  Measured, 128 heads, us: SNAP 0 and 2,
// 16 x 4096 keys 31.0 and 31.5 (so 30.7), 200 x 400 49.0 and 45.4 (45.4).  SHORT 6
// and 16, 40 x 600 20.2 and 18.1 (20.2), 200 x 400 45.3 and 38.8 (45.4), 300 ragged
// of up to 700 56.1 and 53.1 (56.2).  WHOLE_SLACK 0 and 16, 40 x 600 27.6 and 20.2
// (20.2), 64 x 4096 76.5 and 69.3 (76.5), 64 heads 100 x 900 42.9 and 35.7 (35.6).
// Longer ragged batches and single long sequences move by less than 2%.
constexpr int SNAP = 1, SHORT = 10, WHOLE_SLACK = 8;

// Tiles between asking for keys in L2 and copying them to shared memory, whose
// two stages do not cover HBM's latency: 128 ragged sequences took 118 us so,
// 124 without, 126 with two tiles and 156 with four.
constexpr int AHEAD = 1;

struct Maps {
  CUtensorMap q;
  CUtensorMap v;  // pair: 16 rows x 4 column blocks
  CUtensorMap c[MAPS];
};

struct LatentArgs {
  const int32_t *qsl, *seq_lens, *block_table;
  const uint8_t *cache;
  __nv_bfloat16 *o;
  float *lse, *part_o, *part_lse;
  int4 *desc;
  int32_t *status;
  int T, R, H, bs, num_blocks, none, bt_stride, causal, box_log2;  // none: a row past the cache
  bool o_sectors;  // o is 32-byte aligned
  Divider by_bs, by_h;
  float scale_log2;
  TreeMask tree;
};

// ---- the work split ---------------------------------------------------------
struct Seq {
  int q0, nq, len, keys, nrt, tiles;  // keys: len, cut to the block table's row
};

template <bool PAIR>
__device__ __forceinline__ Seq load_seq(const LatentArgs &a, int r) {
  Seq s;
  s.q0 = min(max(__ldg(a.qsl + r), 0), a.T);
  s.nq = max(min(__ldg(a.qsl + r + 1), a.T) - s.q0, 0);
  s.len = max(__ldg(a.seq_lens + r), 0);
  s.keys = keys_of(s.len, a.bt_stride, a.bs);
  s.nrt = (s.nq * a.H + Cfg<PAIR>::UROWS - 1) / Cfg<PAIR>::UROWS;
  // a unit without keys still has its rows to write
  s.tiles = max(1, (s.keys + TILE - 1) / TILE);
  return s;
}

struct Share {  // of a cluster, in shared memory
  long long start, end;  // the positions [start, end)
  int share;             // of all clusters, before cuts were moved
  int r, rt, pos, snap;  // of the start; how far cuts were moved
  Seq seq;               // r's, so that nobody loads it again
};

// Piece of a unit: row tile rt of sequence r, key tiles [t0, t1).  Position v
// of a unit is its tile v - UNIT_COST: a share that ends (or starts) in the
// first UNIT_COST positions has none (or all) of the unit's tiles.
template <bool PAIR, bool TREE>
struct Walk {
  static constexpr int COST = UNIT_COST<PAIR>;
  const LatentArgs &a;
  Seq s;
  int r, rt, t0, t1, pos;
  long long left;
  __device__ __forceinline__ Walk(const LatentArgs &args, const Share &sh)
      : a(args), r(sh.r), rt(sh.rt), t0(0), t1(0), pos(sh.pos), left(sh.end - sh.start) {
    if (left > 0) {
      s = sh.seq;
      if (rt >= s.nrt) next_seq();  // the share starts behind the sequence
    }
  }
  __device__ __forceinline__ void next_seq() {
    rt = 0;
    do {
      if (++r >= a.R) {
        left = 0;
        return;
      }
      s = load_seq<PAIR>(a, r);
    } while (s.nrt == 0);
  }
  __device__ __forceinline__ bool next() {
    if (t1 > 0) {  // the previous piece ended its unit (or left is 0)
      pos = 0;
      if (left > 0 && ++rt == s.nrt) next_seq();
    }
    if (left <= 0) return false;
    const int take = int(min((long long)(s.tiles + COST - pos), left));
    t0 = max(0, pos - COST);
    pos += take;
    t1 = max(0, pos - COST);
    left -= take;
    return t1 > t0;
  }
  // token of the sequence that row `row` of the unit belongs to
  __device__ __forceinline__ int token(int row) const {
    return a.by_h.quotient(rt * Cfg<PAIR>::UROWS + row);
  }
  // keys that row `row` of the unit sees (tree: some of them, by its mask)
  __device__ __forceinline__ int seen(int row) const {
    if (TREE || !a.causal) return s.keys;
    return max(0, min(s.keys, s.len - s.nq + token(row) + 1));
  }
  // keys that all of the unit's rows see, and that any of them may see
  __device__ __forceinline__ int seen_by_all() const {
    return TREE ? max(0, min(s.keys, s.len - s.nq)) : seen(0);
  }
  __device__ __forceinline__ int seen_by_any() const {
    if (TREE) return s.keys;
    return seen(min(Cfg<PAIR>::UROWS, s.nq * a.H - rt * Cfg<PAIR>::UROWS) - 1);
  }
  // shares after this one that have a piece of this unit, which this one cuts
  __device__ __forceinline__ int others(const Share &sh) const {
    return 1 + int((s.tiles + COST - pos - sh.snap - 1) / sh.share);
  }
};

// All threads: this cluster's share of the positions of all units.  Cluster c
// of n starts at position c * share, moved to the end of a unit where one is
// near.  (Sequences' units and positions are summed in one 64-bit scan.)
template <bool PAIR>
__device__ __forceinline__ void find_share(const LatentArgs &a, int cluster, int clusters,
                                           Share *out, uint64_t *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int NW = THREADS / 32;
  int *most = reinterpret_cast<int *>(scratch + NW);  // [NW]
  int nrt, length;
  Seq s;
  auto look = [&](int r) -> uint64_t {
    nrt = 0;
    length = 1;
    if (r >= a.R) return 0;
    s = load_seq<PAIR>(a, r);
    nrt = s.nrt;
    length = s.tiles + UNIT_COST<PAIR>;
    return UnitSum::of(nrt, length);
  };
  // Gives a cluster whose share starts (or ends) in sequence r its part of it;
  // called by the thread that has the sequence, the positions up to its end
  // being sum.
  auto deal = [&](int r, uint64_t mine, uint64_t sum, uint64_t total, int longest) {
    if (nrt == 0) return;
    const long long positions = UnitSum::positions(total);
    const int units = UnitSum::units(total);
    // (64-bit divisions only where 32 bits do not hold the numbers)
    int share = positions <= 0x7fffffff
                    ? int((unsigned(positions) + clusters - 1) / unsigned(clusters))
                    : int(min((positions + clusters - 1) / clusters, 0x7fffffffLL));
    const long long lo = UnitSum::positions(sum - mine), hi = UnitSum::positions(sum);
    if (units <= clusters && longest <= share + WHOLE_SLACK) {
      const int u = cluster - UnitSum::units(sum - mine);  // of this sequence's
      if (u >= 0 && u < nrt) {
        out->end = out->share = length;
        out->seq = s;
        out->r = r;
        out->rt = u;
      }
      return;
    }
    if (share < MIN_SHARE) share = MIN_SHARE;
    const int snap = longest <= SHORT ? SHORT / 2 : SNAP;
    const long long start = (long long)share * cluster, end = start + share;
    // the cut nearest to position p of this sequence (from its start)
    int rt, pos;
    auto cut = [&](long long p) {
      rt = p <= 0x7fffffff ? int(unsigned(p) / unsigned(length)) : int(p / length);
      pos = int(p - (long long)rt * length);
      if (pos <= snap) {
        pos = 0;
      } else if (length - pos <= snap) {
        pos = 0;
        ++rt;
      }
      return lo + (long long)rt * length + pos;
    };
    if (start >= lo && start < hi) {
      out->start = cut(start - lo);
      out->share = share;
      out->snap = snap;
      out->seq = s;
      out->r = r;
      out->rt = rt;
      out->pos = pos;
      if (end >= positions) out->end = positions;
    }
    if (end < positions && end >= lo && end < hi) out->end = cut(end - lo);
  };
  auto warp_scan = [&](uint64_t v) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  if (threadIdx.x == 0) {  // no work, unless threads find some below
    out->start = out->end = 0;
    out->r = out->rt = out->pos = 0;
  }
  if (a.R <= 32) {  // one warp has them all: 0.3 us less than through shared memory
    if (warp == 0) {
      const uint64_t mine = look(lane), sum = warp_scan(mine);
      const int longest = __reduce_max_sync(0xffffffffu, nrt > 0 ? length : 0);
      __syncwarp();
      deal(lane, mine, sum, __shfl_sync(0xffffffffu, sum, 31), longest);
    }
    __syncthreads();
    return;
  }
  // inclusive scan over the block's threads, the total, and the longest unit
  int longest = 0;
  auto scan = [&](uint64_t v, int len, uint64_t &all) {
    v = warp_scan(v);
    len = __reduce_max_sync(0xffffffffu, len);
    if (lane == 31) {
      scratch[warp] = v;
      most[warp] = len;
    }
    __syncthreads();
    all = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (i == warp) v += all;
      all += scratch[i];
      longest = max(longest, most[i]);
    }
    return v;
  };
  // more sequences than threads: their totals first
  const bool many = a.R > THREADS;
  uint64_t total = 0;
  if (many) {
    uint64_t sum = 0;
    int len = 0;
    for (int r = threadIdx.x; r < a.R; r += THREADS) {
      sum += look(r);
      if (nrt > 0) len = max(len, length);
    }
    scan(sum, len, total);
    __syncthreads();
  }
  uint64_t base = 0;
  for (int r0 = 0; r0 < a.R; r0 += THREADS) {
    const uint64_t mine = look(r0 + threadIdx.x);
    uint64_t all;
    const uint64_t sum = base + scan(mine, nrt > 0 ? length : 0, all);
    if (!many) total = all;
    deal(r0 + threadIdx.x, mine, sum, total, longest);
    base += all;
    __syncthreads();
  }
}

// ---- cache loads --------------------------------------------------------------
// Cache row of position j of a sequence (block table row bt); a.none (which the
// loads fill with zeros) from position len on and for a bad block.
__device__ __forceinline__ int cache_row(const LatentArgs &a, const int32_t *bt, int len, int j) {
  if (j >= len) return a.none;
  const int b = a.by_bs.quotient(j);
  const int blk = __ldg(bt + b);
  if (blk < 0 || blk >= a.num_blocks) {
    if (a.status) atomicOr(a.status, MLA_STATUS_BAD_BLOCK);
    return a.none;
  }
  return blk * a.bs + (j - b * a.bs);
}

template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x,
                                         int y) {
  if (PAIR)
    tma_load_2d_pair(dst, m, bar, x, y);
  else
    tma_load_2d(dst, m, bar, x, y);
}

// V of the pair form lies in groups of 2^VB keys: [4 column blocks][2^VB keys][64
// columns].  Pages of 64 or 32 keys and their multiples make groups of that many,
// a copy for each column block; others groups of 16 (an MMA's K), which one copy
// of three dimensions brings whatever the page size (a multiple of 16).  Such a
// copy takes 330 clocks to issue, one of two dimensions with as many bytes 190
// (groups of 16 and as many as the page: pages of 64, 16 trees of 32 nodes on
// 2048 keys 265 and 240 us, 128 x 4096 keys 132 and 129.5; pages of 32, 265 and
// 243, 133 and 130); but 16 copies of 16 rows take longer than four of them (pages
// of 16, 24 ragged trees: 117, so 105).
template <int VB>
struct VLayout {
  static constexpr uint32_t BLOCK = 128u << VB;  // bytes to the next column block
  // of key j's row in the first column block
  __device__ __forceinline__ static uint32_t row(int j) {
    return (uint32_t(j >> VB) << (VB + 9)) + (uint32_t(j & ((1 << VB) - 1)) << 7);
  }
};

// A box of cache rows from `row`, the first `valid` of them real and the others
// zeros, to dst and, `count` times, on to the next column block `step` bytes
// further; called by one thread.  A whole box is one copy a block; a ragged
// one is put together from the smaller boxes (128-byte rows: any row is a
// legal destination, and the swizzle goes by the address).
template <bool PAIR>
__device__ __forceinline__ void load_rows(const Maps &m, int box_log2, uint32_t dst, uint32_t step,
                                          int count, int x, int row, int valid, int none,
                                          uint32_t bar) {
  const int rows = 1 << box_log2;
  if (valid <= 0 || valid >= rows) {
    const int y = valid <= 0 ? none : row;
    const CUtensorMap *map = &m.c[box_log2];
#pragma unroll 3
    for (int b = 0; b < count; ++b) load_box<PAIR>(dst + b * step, map, bar, x + b * 64, y);
    return;
  }
  int off = 0;
  for (int part = 0; part < 2; ++part)  // the real rows, then zeros
    for (int k = box_log2 - 1; k >= 0; --k)
      if ((part == 0 ? valid : rows - valid) & (1 << k)) {
        for (int b = 0; b < count; ++b)
          load_box<PAIR>(dst + b * step + off * 128, &m.c[k], bar, x + b * 64,
                         part == 0 ? row + off : none);
        off += 1 << k;
      }
}

// One MMA from the low words of its operands' descriptors; the high words are
// the same for all of them here (8-row groups 1024 bytes apart, 128-byte
// swizzle).  An MMA of these shapes takes 45-80 clocks, so the issuing thread
// can afford few instructions for each: descriptors differ by constants added
// to a low word (with 64-bit descriptors put together for every MMA it issued
// one in 129 clocks).
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t saddr) {
  return ((saddr >> 4) & 0x3FFF) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr, uint32_t mn_block_bytes) {
  return ((saddr >> 4) & 0x3FFF) | ((mn_block_bytes >> 4) << 16);
}
template <bool PAIR, int A = 0>
__device__ __forceinline__ void mma_lo(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                       uint32_t acc) {
  if (PAIR && A == 1)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n"
        " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::2.kind::f16.collector::a::fill [%0], x, y, %4, p;\n}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(DESC_HI), "r"(idesc), "r"(acc)
        : "memory");
  else if (PAIR && A == 2)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n"
        " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::2.kind::f16.collector::a::lastuse [%0], x, y, %4, p;\n}\n" ::"r"(
            d),
        "r"(alo), "r"(blo), "r"(DESC_HI), "r"(idesc), "r"(acc)
        : "memory");
  else if (PAIR)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n"
        " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(DESC_HI), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n"
        " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.ws.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(DESC_HI), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 bytes in one store where the address allows it, so that every sector is
// written at once.
__device__ __forceinline__ void st_global_32(void *p, const uint32_t (&v)[8], bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Any of 8 bf16 values infinite or NaN.
__device__ __forceinline__ bool not_finite(uint4 v) {
  auto bad = [](uint32_t x) {
    return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
  };
  return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
}

// Keys that some rows of a unit see and others do not: where a value row is not
// finite, zeros have to stand for it, as a weight of 0 would not hide it.  (The
// rows that see it are NaN by their scores, or, -inf, weigh it nothing.)  Which of a tile's keys [from, to)
// are not finite in the 256 columns from byte `col`; by a warp, whose lanes have
// the cache rows of groups of 2^bl keys in row0, row1.  (Not inlined, like the
// next: inlined, they cost every tile's loads a little, 1.5% of the whole.)
__device__ __noinline__ uint64_t hidden_rows(const LatentArgs &a, int row0, int row1, int bl,
                                             int from, int to, int col) {
  uint64_t hidden = 0;
  for (int j = from; j < to; ++j) {
    const int i = j >> bl;
    const int r = __shfl_sync(0xffffffffu, i < 32 ? row0 : row1, i & 31);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r != a.none)
      v = __ldg(reinterpret_cast<const uint4 *>(
              a.cache + int64_t(r + (j & ((1 << bl) - 1))) * (WIDTH * 2) + col) +
          (threadIdx.x & 31));
    if (__any_sync(0xffffffffu, not_finite(v))) hidden |= uint64_t(1) << j;
  }
  return hidden;
}

// A tile's V, row by row, without the hidden ones and those from `keys` on.
template <bool PAIR, int VB>
__device__ __noinline__ void load_unhidden(const Maps &m, int row0, int row1, int bl, int keys,
                                           uint64_t hidden, uint32_t dst, int x, int none,
                                           uint32_t bar) {
  for (int j = 0; j < TILE; ++j) {
    const int i = j >> bl;
    const int r = __shfl_sync(0xffffffffu, i < 32 ? row0 : row1, i & 31);
    const bool real = r != none && j < keys && !(hidden >> j & 1);
    if (elect_one())
      load_rows<PAIR>(m, 0, dst + VLayout<VB>::row(j), VLayout<VB>::BLOCK, 4, x,
                      r + (j & ((1 << bl) - 1)), real, none, bar);
    __syncwarp();
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void softmax_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(STHREADS) : "memory");
}

template <bool PAIR, bool TREE, int VB>
__global__ void __launch_bounds__(THREADS, 1)
    latent_attn_kernel(const __grid_constant__ Maps m, const LatentArgs a) {
  using C = Cfg<PAIR>;
  using Lay = VLayout<VB>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  static_assert(C::USED <= C::SMEM, "shared memory");
  if (smem + C::USED > smem_raw + C::SMEM) {  // (the base is 1024-byte aligned in practice)
    if (threadIdx.x == 0) atomicOr(&g_error_flags, kErrWaitTimeout);
    return;
  }
  const uint32_t sQ = smem_u32(smem), sK = sQ + Q_BYTES, sV = sK + 2 * C::K_STAGE,
                 sP = sK + C::KV_BYTES;
  float *xmax = reinterpret_cast<float *>(smem + Q_BYTES + C::KV_BYTES + C::P_BYTES);  // [2][256]
  uint64_t *bars = reinterpret_cast<uint64_t *>(xmax + 512);
  const uint32_t k_full = smem_u32(bars), k_empty = k_full + 16, v_full = k_full + 32,
                 v_empty = k_full + 48, s_full = k_full + 64,
                 p_full = k_full + 96, pv_done = k_full + 112, q_full = k_full + 128,
                 q_empty = k_full + 136, done = k_full + 144, v_own = k_full + 376;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 19);
  volatile int *progress = reinterpret_cast<volatile int *>(bars + 46);  // tiles K was loaded of
  Share *share = reinterpret_cast<Share *>(bars + 20);         // 64 bytes
  uint64_t *scan = bars + 28;  // [18]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const int cluster = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int clusters = PAIR ? gridDim.x >> 1 : gridDim.x;
  auto lead = [&](uint32_t bar) { return PAIR ? mapa_shared(bar, 0) : bar; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, TREE && PAIR ? 2 : 1);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, PAIR ? 2 * SWARPS : SWARPS);
      mbar_init(pv_done + 8 * i, 1);
    }
    *progress = 0;
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(done, 1);
    if (TREE && PAIR) mbar_init(v_own, 1);
    fence_mbar_init();
    prefetch_map(&m.q);
    prefetch_map(&m.c[a.box_log2]);
  }
  if (warp == 2) {
    if (PAIR)
      tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    else
      tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    chain_release();  // (not before: a later kernel's CTA could take the columns and wait for us)
  }
  tc_fence_before();
  if (PAIR) cluster_arrive();  // both CTAs' barriers exist before any load or arrive
  chain_wait();
  find_share<PAIR>(a, cluster, clusters, share, scan);  // (ends with a barrier)
  if (PAIR) cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int none = a.none;

  if (warp == 0 || (PAIR && warp == 1)) {
    // ---------------- K loads (single: which are V too) and V loads, one warp
    // each.  A lane finds the cache rows of row groups lane and lane + 32; one
    // thread issues the copies, from values that are the same in all lanes (a
    // copy issued by several lanes, each with its own operands, took 120-150
    // clocks, and the loads of a tile 2500 to 4000).
    const bool is_v = PAIR && warp == 1;
    const uint32_t full = is_v ? v_full : k_full, empty = is_v ? v_empty : k_empty;
    const uint32_t full_lead = lead(full);
    const uint32_t dst0 = is_v ? sV : sK, stage_bytes = is_v ? C::V_STAGE : C::K_STAGE;
    const int nrows = is_v ? 64 : C::KROWS, blocks = is_v ? 4 : NBLK;
    const int bl = min(a.box_log2, is_v ? VB : PAIR ? 5 : 6), bx = 1 << bl;  // rows at once
    const int skip = PAIR && !is_v ? int(rank) * C::KROWS : 0;  // first key of the tile here
    Walk<PAIR, TREE> w(a, *share);
    int g = 0, checked = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int32_t *bt = a.block_table + int64_t(w.r) * a.bt_stride;
      const int all = w.seen_by_all(), any = w.seen_by_any();
      for (int t = w.t0; t < w.t1; ++t, ++g) {
        const int key0 = t * TILE + skip, st = g & 1;
        const bool mixed = is_v && all < any && key0 + TILE > all;
        int row[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int off = (lane + 32 * i) << bl;
          row[i] = off < nrows ? cache_row(a, bt, any, key0 + off) : none;
        }
        uint64_t hidden = 0;
        if (!TREE && mixed)
          hidden = hidden_rows(a, row[0], row[1], bl, max(0, all - key0), min(TILE, any - key0),
                               int(rank) * 512);
        ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * st, ((g >> 1) & 1) ^ 1));
        if (!ok) break;
        // (a tree's mixed tile comes here on a barrier of this CTA's own)
        const bool own = TREE && mixed;
        if (lane == 0) {
          if (own)
            mbar_expect_tx(v_own, stage_bytes);
          else if (rank == 0)
            mbar_expect_tx(full + 8 * st, (PAIR ? 2 : 1) * stage_bytes);
          else if (TREE && is_v)
            mbar_arrive_remote(full_lead + 8 * st);
        }
        __syncwarp();
        if (hidden) {
          load_unhidden<PAIR, VB>(m, row[0], row[1], bl, any - key0, hidden,
                                  dst0 + st * stage_bytes, int(rank) * 256, none,
                                  full_lead + 8 * st);
          continue;
        }
        for (int i = 0; i < nrows >> bl; ++i) {
          const int r = __shfl_sync(0xffffffffu, i < 32 ? row[0] : row[1], i & 31);
          const int off = i << bl;
          // (a row past the length in K alone only makes scores that are masked)
          const int valid = r == none ? 0 : PAIR && !is_v ? bx : min(bx, any - key0 - off);
          if (elect_one()) {
            const uint32_t dst = dst0 + st * stage_bytes, bar = own ? v_own : full_lead + 8 * st;
            if (VB == 6 && !is_v) {  // one box of 32 keys: straight through
              const int y = valid > 0 ? r : none;
#pragma unroll
              for (int b = 0; b < NBLK; ++b)
                tma_load_2d_pair(dst + b * (C::KROWS * 128), &m.c[5], bar, b * 64, y);
            } else if (VB == 6 && valid == TILE) {  // one of 64
#pragma unroll
              for (int b = 0; b < 4; ++b)
                tma_load_2d_pair(dst + b * Lay::BLOCK, &m.c[6], bar, int(rank) * 256 + b * 64, r);
            } else if (!is_v)
              load_rows<PAIR>(m, bl, dst + off * 128, nrows * 128, blocks, 0, r, valid, none, bar);
            else if (VB == 4 && bl == 4 && (valid == 0 || valid == 16))
              tma_load_3d_pair(dst + Lay::row(off), &m.v, bar, 0, r, int(rank) * 4);
            else
              load_rows<PAIR>(m, bl, dst + Lay::row(off), Lay::BLOCK, 4, int(rank) * 256, r, valid,
                              none, bar);
          }
          __syncwarp();
        }
        if (own) {
          // A tree's rows differ in most of the new tokens that they see, so
          // these are looked at where they have landed: a row takes one load of
          // the warp.  (Read from memory beforehand, as where a few rows are
          // hidden, one takes some 600 clocks.)
          ok = __all_sync(0xffffffffu, mbar_wait(v_own, checked++ & 1));
          if (!ok) break;
          const uint32_t v = dst0 + st * stage_bytes + (lane >> 3) * Lay::BLOCK + (lane & 7) * 16;
          const int to = min(TILE, any - key0);
#pragma unroll 4
          for (int j = max(0, all - key0); j < to; ++j) {
            const uint32_t at = v + Lay::row(j);
            if (not_finite(ld_shared_v4(at))) st_shared_v4(at, make_uint4(0, 0, 0, 0));
          }
          fence_async_smem();
          __syncwarp();
          // As P is handed on: an arrive of CTA scope after the proxy fence, of which
          // it is taken, beyond what PTX states, that it suffices for the even CTA's
          // MMAs, as they read this CTA's rows through the async proxy.
          if (lane == 0) mbar_arrive_remote(full_lead + 8 * st);
        }
        if (!is_v && lane == 0) *progress = g + 1;
      }
    }
    // the loads issued here have landed before the CTA may exit
    for (int i = max(0, g - 2); i < g; ++i)
      mbar_wait((rank == 0 ? full : empty) + 8 * (i & 1), (i >> 1) & 1);
  } else if (warp == 3) {
    // ---------------- query loads, and this CTA's keys on their way to L2
    // AHEAD tiles before the K loads come to them, whose progress paces this
    // warp (nothing waits for it but the queries)
    const int bl = min(a.box_log2, PAIR ? 5 : 6);
    Walk<PAIR, TREE> w(a, *share);
    int g = 0, n = 0;
    bool ok = true;
    const uint32_t bar = lead(q_full);
    for (; ok && w.next(); ++n) {
      const int32_t *bt = a.block_table + int64_t(w.r) * a.bt_stride;
      const int any = w.seen_by_any();
      bool queries = false;
      auto load_queries = [&] {
        queries = true;
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(q_full, (PAIR ? 2 : 1) * Q_BYTES);
          const int row = w.s.q0 * a.H + w.rt * C::UROWS + int(rank) * CROWS;
          for (int kb = 0; kb < NBLK; ++kb)
            load_box<PAIR>(sQ + kb * BLK_BYTES, &m.q, bar, kb * 64, row);
        }
        __syncwarp();
      };
      for (int t = w.t0; ok && t < w.t1; ++t, ++g) {
        const long long c0 = clock64();
        int at;
        for (;;) {
          at = __shfl_sync(0xffffffffu, *progress, 0);
          if (!queries && __all_sync(0xffffffffu, mbar_test(q_empty, (n & 1) ^ 1))) load_queries();
          if (at >= g - AHEAD) break;
          ok = __all_sync(0xffffffffu, clock64() - c0 < kWaitCycles);
          if (!ok) break;
          __nanosleep(64);
        }
        if (at >= g) continue;  // already being loaded
        const int key0 = t * TILE + (PAIR ? int(rank) * C::KROWS : 0);
        for (int i = 0; i < C::KROWS >> bl; i += 32) {
          const int j = key0 + ((lane + i) << bl);
          int row = none;
          if (((lane + i) << bl) < C::KROWS) row = cache_row(a, bt, any, j);
          if (row != none)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             a.cache + int64_t(row) * (WIDTH * 2)),
                         "r"(min(1 << bl, any - j) * WIDTH * 2)
                         : "memory");
        }
        __syncwarp();
      }
      if (ok && !queries) {
        ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (n & 1) ^ 1));
        if (ok) load_queries();
      }
    }
    if (n > 0) mbar_wait(rank == 0 ? q_full : q_empty, (n - 1) & 1);
  } else if (warp == 2) {
    // ---------------- MMA issue (pair: the even CTA).
    if (rank == 0 && elect_one()) {
      constexpr uint32_t id_s = idesc_f16kind(PAIR ? 128 : 64, TILE, false, false, true);
      constexpr uint32_t id_o = idesc_f16kind(PAIR ? 128 : 64, 256, false, true, true);
      constexpr uint32_t BLK = BLK_BYTES >> 4;  // steps of descriptor addresses (16 bytes)
      auto commit = [](uint32_t bar) {
        if (PAIR)
          mma_commit_pair_mc(bar, uint16_t(3));
        else
          mma_commit(bar);
      };
      const uint32_t q_lo = desc_lo_k(sQ), k_lo = desc_lo_k(sK), p_lo = desc_lo_k(sP);
      // V, MN-major: blocks of 64 columns BLK_BYTES (pair: a group's rows) apart
      const uint32_t v_lo = desc_lo_mn(PAIR ? sV : sK, PAIR ? Lay::BLOCK : BLK_BYTES);
      // of 16 keys more (single: 64 rows in a block)
      auto v_ks = [](int ks) { return (PAIR ? Lay::row(16 * ks) : 2048u * ks) >> 4; };
      constexpr uint32_t V_J = PAIR ? 2 * Lay::BLOCK >> 4 : 4 * BLK;  // second MMA's columns
      constexpr uint32_t K_STEP = C::K_STAGE >> 4, V_STEP = (PAIR ? C::V_STAGE : C::K_STAGE) >> 4;
      constexpr uint32_t KBLK = C::KROWS * 128 >> 4;
      // O (+)= P V of tile g
      auto second = [&](int g, bool first) -> bool {
        const int st = g & 1;
        const uint32_t parity = (g >> 1) & 1;
        if (PAIR && !mbar_wait(v_full + 8 * st, parity)) return false;
        if (!mbar_wait(p_full + 8 * st, parity)) return false;
        tc_fence_after();
        const uint32_t acc0 = first ? 0 : 1;
        const uint32_t v = v_lo + st * V_STEP, p = p_lo + (PAIR ? st * BLK : 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          {
            const uint32_t vk = v + v_ks(ks), acc = ks == 0 ? acc0 : 1;
            // (P's rows are read for the first MMA and kept for the second)
            mma_lo<PAIR, 1>(tmem, p + ks * 2, vk, id_o, acc);
            mma_lo<PAIR, 2>(tmem + 128, p + ks * 2, vk + V_J, id_o, acc);
          }
        commit((PAIR ? v_empty : k_empty) + 8 * st);
        commit(pv_done + 8 * st);
        return true;
      };
      Walk<PAIR, TREE> w(a, *share);
      int g = 0, n = 0;
      bool ok = true, first = false;  // first: the pending P V starts a unit's O
      for (; ok && w.next(); ++n) {
        for (int t = w.t0; t < w.t1; ++t, ++g) {
          const int st = g & 1;
          const uint32_t parity = (g >> 1) & 1;
          // S of this tile goes ahead of P V of the one before, so that the
          // softmax has the tensor pipe's time, unless its keys (or queries)
          // have yet to land.  Then the single form waits for that P V, which
          // releases room for loads, its bottleneck (S always first took 1.6
          // times as long a tile); the pair form takes whichever is ready first
          // (that P V first: 1.1 times).
          auto ready = [&] {
            return mbar_test(k_full + 8 * st, parity) && (t > w.t0 || mbar_test(q_full, n & 1));
          };
          bool behind = g > 0, landed = ready();
          if (behind && !landed) {
            const long long c0 = clock64();
            while (PAIR && !mbar_test(p_full + 8 * (st ^ 1), ((g - 1) >> 1) & 1) && !landed &&
                   clock64() - c0 < kWaitCycles)
              landed = ready();
            if (!PAIR || !landed) {
              ok = second(g - 1, first);
              if (!ok) break;
              behind = false;
            }
          }
          // (a wait takes this thread some 100 clocks even where there is nothing
          // to wait for.  That the S of two tiles before has been read is known
          // from its P.)
          if (!landed) {
            ok = (t > w.t0 || mbar_wait(q_full, n & 1)) && mbar_wait(k_full + 8 * st, parity);
            if (!ok) break;
          }
          tc_fence_after();
          const uint32_t d = tmem + S_COL + st * SC, k = k_lo + st * K_STEP;
#pragma unroll
          for (int kb = 0; kb < NBLK; ++kb)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_lo<PAIR>(d, q_lo + kb * BLK + ks * 2, k + kb * KBLK + ks * 2, id_s,
                           (kb | ks) != 0);
          if (PAIR) commit(k_empty + 8 * st);
          commit(s_full + 8 * st);
          if (t + 1 == w.t1) commit(q_empty);
          if (behind) {
            ok = second(g - 1, first);
            if (!ok) break;
          }
          first = t == w.t0;
        }
      }
      if (ok && g > 0) second(g - 1, first);
      // every MMA has completed before tensor memory is released
      commit(done);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- softmax and epilogue: four threads a row, each a
    // quarter of the tile's keys (half: which half of D's columns its lanes
    // hold; part: which half of those is this warp's)
    const int tid = threadIdx.x - 128, tl = tid & 127;  // tl: tensor-memory lane
    const int part = tid >> 7, half = tl >> 6, rl = tl & 63;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t p_full_lead = lead(p_full);
    if (tid == 0 && rank == 0) a.desc[2 * cluster] = make_int4(0, 0, 0, 0);
    // the tiles' maxima and the pieces' sums, over the four threads of a row
    RowJoin<STHREADS> row_join(xmax, tid);
    auto barrier = [] { softmax_barrier(); };
    Walk<PAIR, TREE> w(a, *share);
    int g = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int rows = w.s.nq * a.H - w.rt * C::UROWS;  // of the unit (may exceed it)
      const int urow = int(rank) * CROWS + rl;
      const int vis = w.seen(min(urow, rows - 1));
      const uint64_t *tree = nullptr;  // this row's mask
      if (TREE)
        tree = a.tree.bits + int64_t(w.s.q0 + w.token(min(urow, rows - 1))) * a.tree.words;
      const int all = w.seen_by_all(), any = w.seen_by_any();
      if (w.s.keys < w.s.len && a.status && tid == 0) atomicOr(a.status, MLA_STATUS_BAD_BLOCK);
      float mref = neg_inf(), l = 0.f;
      for (int t = w.t0; t < w.t1; ++t, ++g) {
        const int sb = g & 1, key = t * TILE + half * SC + part * NC;  // this thread's first
        const int nvis = vis - key;
        const bool mixed = all < any && t * TILE + TILE > all;  // rows may differ in what they see
        uint32_t sees = nvis >= NC ? ~0u : nvis > 0 ? (1u << nvis) - 1 : 0;
        if (TREE && mixed) sees &= tree_bits(tree, a.tree.words, key - (w.s.len - w.s.nq));
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * sb, (g >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[NC];
        const uint32_t t_s = t_lane + S_COL + sb * SC + part * NC;
        tmem_ld16(t_s, s);
        tmem_wait_ld();
        tc_fence_before();
        if (TREE ? mixed || nvis < NC : nvis < NC) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (TREE ? !(sees >> c & 1) : c >= nvis) s[c] = __float_as_uint(neg_inf());
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < NC; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(s[c]));
        const float mt = row_join(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), barrier,
                                  [](float x, float y) { return fmaxf(x, y); }) *
                         a.scale_log2;
        // the threads of a row see the same maxima and decide alike
        float f = 1.f;
        if (mt > mref + RESCALE || (is_neg_inf(mref) && mt > mref)) {
          f = exp2_fast(mref - mt);  // 0 from -inf
          mref = mt;
          l *= f;
        }
        const float base = is_neg_inf(mref) ? 0.f : mref;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t p[NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float x = exp2_fast(fmaf(__uint_as_float(s[c]), a.scale_log2, -base));
          const float y = exp2_fast(fmaf(__uint_as_float(s[c + 1]), a.scale_log2, -base));
          sum[(c >> 1) & 3] += x + y;
          p[c / 2] = pack_bf16(x, y);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // O is rescaled once P V of the tile before is done; P's room is free
        // once that of NP tiles before is
        const bool rescale = t > w.t0 && __any_sync(0xffffffffu, f != 1.f);
        const int wait_for = rescale ? g - 1 : g - C::NP;
        if (wait_for >= 0) {
          ok = __all_sync(0xffffffffu,
                          mbar_wait(pv_done + 8 * (wait_for & 1), (wait_for >> 1) & 1));
          if (!ok) break;
        }
        if (rescale) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_lane + part * 128 + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(t_lane + part * 128 + c, o);
          }
          tmem_wait_st();
        }
        // P, K-major with 128-byte swizzle
        const uint32_t prow = sP + (PAIR ? sb * BLK_BYTES : 0) + rl * 128;
        const int c0 = half * 4 + part * 2;
#pragma unroll
        for (int c = 0; c < NC / 8; ++c)
          st_shared_v4(prow + (((c0 + c) ^ (rl & 7)) << 4),
                       make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]));
        // Value rows that are not finite and that only some rows see are
        // cleared: a weight of 0 would not hide them from the others.  The
        // scores of the rows that see them are not finite either, and make them
        // NaN (or, -inf, give a weight of 0; making NaN of those too costs every
        // tile some 30 clocks).  The pair form's V loads do this.
        if (!PAIR && mixed) {
          ok = __all_sync(0xffffffffu, mbar_wait(k_full + 8 * sb, (g >> 1) & 1));
          if (!ok) break;
          const int from = max(0, all - t * TILE), n = min(TILE, any - t * TILE) - from;
          for (int x = tid; x < n * 64; x += STHREADS) {  // row, column block, piece
            const uint32_t v = sK + sb * C::K_STAGE + (x >> 3 & 7) * BLK_BYTES +
                               (from + (x >> 6)) * 128 + (x & 7) * 16;
            if (not_finite(ld_shared_v4(v))) st_shared_v4(v, make_uint4(0, 0, 0, 0));
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote(p_full_lead + 8 * sb);
          else
            mbar_arrive(p_full + 8 * sb);
        }
      }
      if (!ok) break;
      // ---- the piece's rows
      l = row_join(l, barrier, [](float x, float y) { return x + y; });
      const bool whole = w.t0 == 0 && w.t1 == w.s.tiles;
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse2 = l > 0.f || l != l ? mref + log2f(l) : neg_inf();
      const int grow0 = w.s.q0 * a.H + w.rt * C::UROWS;  // the unit's first row
      const int slot = 2 * cluster + (w.t0 == 0 ? 1 : 0);
      const int64_t srow = int64_t(slot) * C::UROWS + int(rank) * CROWS;
      if (half == 0 && part == 0) {
        const int token = a.by_h.quotient(grow0 + urow);
        if (urow >= rows) {
        } else if (!whole)
          a.part_lse[srow + rl] = lse2;
        else if (a.lse)
          a.lse[int64_t(grow0 + urow - token * a.H) * a.T + token] = lse2 * LN2;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(pv_done + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      // D's columns: part 0 holds the first MMA's, part 1 the second's
      const int dim0 = PAIR ? half * 256 + part * 128 : part * 256 + half * 128;
      if (whole) {
        __nv_bfloat16 *dst = a.o + int64_t(grow0 + urow) * LAT + dim0;
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          uint32_t o[2][32];
          tmem_ld32(t_lane + part * 128 + c, o[0]);
          tmem_ld32(t_lane + part * 128 + c + 32, o[1]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // 16 columns: a whole sector of the row
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float x = __uint_as_float(o[e >> 1][(e & 1) * 16 + 2 * k]);
              const float y = __uint_as_float(o[e >> 1][(e & 1) * 16 + 2 * k + 1]);
              v[k] = inv == 0.f ? 0u : pack_bf16(x * inv, y * inv);
            }
            if (urow < rows) st_global_32(dst + c + e * 16, v, a.o_sectors);
          }
        }
      } else {
        // scratch of a slot and CTA: [512/4][64 rows][4], so that the lanes of
        // a warp write one contiguous piece
        float4 *dst = reinterpret_cast<float4 *>(a.part_o + srow * LAT) + rl;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t o[32];
          tmem_ld32(t_lane + part * 128 + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = inv == 0.f ? 0.f : __uint_as_float(o[e + k]) * inv;
            if (urow < rows)
              dst[((dim0 + c + e) / 4) * CROWS] = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        if (w.t0 == 0 && tid == 0 && rank == 0) {
          // the unit's first piece: its others are in the shares that follow
          // (never more than there are clusters, whatever the locations were)
          a.desc[2 * cluster] =
              make_int4(min(1 + w.others(*share), clusters - cluster), min(rows, C::UROWS), 0, 0);
          a.desc[2 * cluster + 1].x = grow0;
        }
      }
      tc_fence_before();  // the reads of O come before the next piece's P is handed over
    }
  }
  // Every MMA has completed; and in the pair neither CTA leaves while the other
  // may still arrive here.  (The odd CTA's warp 2 has issued nothing: its wait,
  // limited as all are, begins when the others' work ends, not the kernel.)
  if (rank != 0) __syncthreads();
  if (warp == 2) mbar_wait(done, 0);
  tc_fence_before();
  if (PAIR) {  // (a release would wait for the rows' way to L2)
    cluster_arrive_relaxed();
    cluster_wait();
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 2) {
    __syncwarp();
    if (PAIR)
      tmem_dealloc_pair(tmem, TMEM_COLS);
    else
      tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the pieces of cut units: o = sum_i w_i o_i / sum_i w_i with w_i =
// 2^(lse_i - max).  It lives on loads in flight: a thread has 16 of 16 bytes,
// U pieces of W float4 columns.  Units of at most FEW pieces: a warp takes 32
// rows x 4 W columns, W the widest that still takes all pieces at once (two
// columns of eight pieces for units of two or three cost 5-8 us more where
// there are a hundred of them).  Units of more (a long sequence spread over
// many clusters): a block takes 32 rows x 4 columns, its warps every eighth
// piece, and joins theirs in shared memory (a warp for all of 70 pieces: 3 us
// more).
constexpr int CT = 256, CW = CT / 32;  // threads, warps of a block; clusters <= CT
constexpr int FEW = 8, COMBINE_BLOCKS = 2;

__device__ __forceinline__ int few_columns(int pieces) {
  return pieces <= 2 ? 8 : pieces <= 4 ? 4 : 2;
}

template <int W>
struct Joined {
  float mx, sum;
  float4 acc[W];
};

template <int W>
__device__ __forceinline__ void join_more(Joined<W> &j, float ls, const float4 (&v)[W], float bs) {
  const float w = exp2_fast(ls - bs);
  j.sum += w;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    j.acc[k].x = fmaf(w, v[k].x, j.acc[k].x);
    j.acc[k].y = fmaf(w, v[k].y, j.acc[k].y);
    j.acc[k].z = fmaf(w, v[k].z, j.acc[k].z);
    j.acc[k].w = fmaf(w, v[k].w, j.acc[k].w);
  }
}

// pieces first, first + step, ... of n
template <int W, int U>
__device__ __forceinline__ Joined<W> join_pieces(const float *part_o, const float *part_lse, int c0,
                                                 int first, int step, int n, int urows, int row,
                                                 int col4) {
  Joined<W> j;
  j.mx = neg_inf();
  j.sum = 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) j.acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 < n; i0 += U * step) {
    float ls[U];
    float4 v[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * step;
      ls[u] = neg_inf();
#pragma unroll
      for (int k = 0; k < W; ++k) v[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const int64_t s = int64_t(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * urows + (row & ~63);
        ls[u] = part_lse[s + (row & 63)];
        const float4 *src = reinterpret_cast<const float4 *>(part_o + s * LAT) + (row & 63);
#pragma unroll
        for (int k = 0; k < W; ++k) v[u][k] = src[(col4 + k) * CROWS];
      }
    }
    float mn = j.mx;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = fmaxf(mn, ls[u]);
    const float bs = is_neg_inf(mn) ? 0.f : mn;
    const float f = exp2_fast(j.mx - bs);
    j.mx = mn;
    j.sum *= f;
#pragma unroll
    for (int k = 0; k < W; ++k)
      j.acc[k] = make_float4(j.acc[k].x * f, j.acc[k].y * f, j.acc[k].z * f, j.acc[k].w * f);
#pragma unroll
    for (int u = 0; u < U; ++u) join_more<W>(j, ls[u], v[u], bs);
  }
  return j;
}

template <int W>
__device__ __forceinline__ void join_store(const Joined<W> &j, int grow, int col4,
                                           __nv_bfloat16 *o, float *lse, int H, Divider by_h,
                                           int T) {
  const float inv = j.sum == 0.f ? 0.f : 1.f / j.sum;
  uint2 out[W];
#pragma unroll
  for (int k = 0; k < W; ++k)
    out[k] = make_uint2(pack_bf16(j.acc[k].x * inv, j.acc[k].y * inv),
                        pack_bf16(j.acc[k].z * inv, j.acc[k].w * inv));
  __nv_bfloat16 *dst = o + int64_t(grow) * LAT + col4 * 4;
  if constexpr (W > 1) {
#pragma unroll
    for (int k = 0; k < W; k += 2)
      *reinterpret_cast<uint4 *>(dst + 4 * k) =
          make_uint4(out[k].x, out[k].y, out[k + 1].x, out[k + 1].y);
  } else {
    *reinterpret_cast<uint2 *>(dst) = out[0];
  }
  if (lse && col4 == 0) {
    const int token = by_h.quotient(grow);
    lse[int64_t(grow - token * H) * T + token] =
        j.sum == 0.f ? neg_inf() : ((is_neg_inf(j.mx) ? 0.f : j.mx) + log2f(j.sum)) * LN2;
  }
}

__global__ void __launch_bounds__(CT) latent_combine_kernel(const int4 *desc, int clusters,
                                                            int urows, const float *part_o,
                                                            const float *part_lse,
                                                            __nv_bfloat16 *o, float *lse, int H,
                                                            Divider by_h, int T) {
  // cut units (cluster of the first piece) of many pieces, and of few with the
  // items before each
  __shared__ int few[CT], many[CT], first[CT], first_m[CT];
  __shared__ int warp_few[CW], warp_many[CW], warp_items[CW], warp_items_m[CW];
  __shared__ float4 sacc[CW][32];
  __shared__ float smax[CW][32], ssum[CW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  chain_release();
  chain_wait();
  int n_here = 0, groups = 0;  // pieces, groups of 32 rows
  if (int(threadIdx.x) < clusters) {
    const int4 d = desc[2 * threadIdx.x];
    n_here = d.x;
    groups = (d.y + 31) / 32;
  }
  const bool is_few = n_here > 0 && n_here <= FEW;
  const int items = is_few ? groups * (128 / few_columns(n_here)) : n_here > FEW ? groups * 128 : 0;
  int inc = is_few ? items : 0, inc_m = is_few ? 0 : items;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, d), u = __shfl_up_sync(0xffffffffu, inc_m, d);
    if (lane >= d) {
      inc += v;
      inc_m += u;
    }
  }
  const uint32_t bf = __ballot_sync(0xffffffffu, is_few);
  const uint32_t bm = __ballot_sync(0xffffffffu, n_here > FEW);
  if (lane == 31) {
    warp_few[warp] = __popc(bf);
    warp_many[warp] = __popc(bm);
    warp_items[warp] = inc;
    warp_items_m[warp] = inc_m;
  }
  __syncthreads();
  int base_f = 0, base_m = 0, base_i = 0, base_im = 0, num_f = 0, num_m = 0, num_i = 0, num_im = 0;
#pragma unroll
  for (int i = 0; i < CW; ++i) {
    if (i < warp) {
      base_f += warp_few[i];
      base_m += warp_many[i];
      base_i += warp_items[i];
      base_im += warp_items_m[i];
    }
    num_f += warp_few[i];
    num_m += warp_many[i];
    num_i += warp_items[i];
    num_im += warp_items_m[i];
  }
  const uint32_t below = (1u << lane) - 1;
  if (n_here > FEW) {
    const int u = base_m + __popc(bm & below);
    many[u] = threadIdx.x;
    first_m[u] = base_im + inc_m - items;
  } else if (is_few) {
    const int u = base_f + __popc(bf & below);
    few[u] = threadIdx.x;
    first[u] = base_i + inc - items;
  }
  __syncthreads();
  auto unit_of = [](const int *start, int n, int it) {  // the last that starts at or before it
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= it)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  };
  for (int it = blockIdx.x; it < num_im; it += gridDim.x) {
    const int u = unit_of(first_m, num_m, it), c0 = many[u], sub = it - first_m[u];
    const int row = (sub / 128) * 32 + lane, col4 = sub % 128;
    const int4 d = desc[2 * c0];
    const int grow0 = desc[2 * c0 + 1].x;
    Joined<1> j =
        join_pieces<1, 16>(part_o, part_lse, c0, warp, CW, row < d.y ? d.x : 0, urows, row, col4);
    sacc[warp][lane] = j.acc[0];
    smax[warp][lane] = j.mx;
    ssum[warp][lane] = j.sum;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 1; i < CW; ++i) j.mx = fmaxf(j.mx, smax[i][lane]);
      const float bs = is_neg_inf(j.mx) ? 0.f : j.mx;
      j.sum = 0.f;
      j.acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        const float f = exp2_fast(smax[i][lane] - bs);
        const float4 v = sacc[i][lane];
        j.sum = fmaf(f, ssum[i][lane], j.sum);
        j.acc[0].x = fmaf(f, v.x, j.acc[0].x);
        j.acc[0].y = fmaf(f, v.y, j.acc[0].y);
        j.acc[0].z = fmaf(f, v.z, j.acc[0].z);
        j.acc[0].w = fmaf(f, v.w, j.acc[0].w);
      }
      if (row < d.y) join_store<1>(j, grow0 + row, col4, o, lse, H, by_h, T);
    }
    __syncthreads();
  }
  // (from the block after the last that had an item above)
  const int turn = (blockIdx.x + gridDim.x - num_im % gridDim.x) % gridDim.x;
  for (int it = turn * CW + warp; it < num_i; it += gridDim.x * CW) {
    const int u = unit_of(first, num_f, it), c0 = few[u], sub = it - first[u];
    const int4 d = desc[2 * c0];
    const int grow0 = desc[2 * c0 + 1].x;
    const int w = few_columns(d.x), row = sub / (128 / w) * 32 + lane, col4 = sub % (128 / w) * w;
    auto one = [&](auto width, auto pieces) {
      constexpr int W = decltype(width)::value, U = decltype(pieces)::value;
      const Joined<W> j =
          join_pieces<W, U>(part_o, part_lse, c0, 0, 1, row < d.y ? d.x : 0, urows, row, col4);
      if (row < d.y) join_store<W>(j, grow0 + row, col4, o, lse, H, by_h, T);
    };
    if (w == 8)
      one(std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
    else if (w == 4)
      one(std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
    else
      one(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
  }
}

template <bool PAIR, bool TREE, int VB>
int launch_latent(const Maps &maps, const LatentArgs &a, int urows_limit, cudaStream_t s) {
  constexpr int MAX_DEV = 64;
  static std::atomic<int> grid_of[MAX_DEV];  // CTAs that fit the device, 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEV) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Cfg<PAIR>::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int grid = grid_of[dev].load(std::memory_order_acquire);
  if (grid == 0) {
    if (cudaFuncSetAttribute(latent_attn_kernel<PAIR, TREE, VB>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<PAIR>::SMEM) != cudaSuccess)
      return MLA_ERR_CUDA;
    const int cs = PAIR ? 2 : 1;
    cfg.gridDim = dim3(cs * (num_sms() / cs));
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, latent_attn_kernel<PAIR, TREE, VB>, &cfg) !=
            cudaSuccess ||
        n < 1)
      n = num_sms() / cs;
    grid = std::min(cs * n, urows_limit);
    grid_of[dev].store(grid, std::memory_order_release);
  }
  int rc = launch_chained(latent_attn_kernel<PAIR, TREE, VB>, grid, THREADS, Cfg<PAIR>::SMEM,
                          PAIR ? 2 : 1, s, TREE ? "tree_attn_kernel" : "latent_attn_kernel", maps,
                          a);
  if (rc) return rc;
  // sequences that the block table keeps short are never cut: nothing to join
  const int64_t most_tiles = (int64_t(a.bt_stride) * a.bs + TILE - 1) / TILE;
  if (most_tiles + UNIT_COST<PAIR> <= SHORT) return MLA_OK;
  return launch_chained(latent_combine_kernel, COMBINE_BLOCKS * num_sms(), CT, 0, 1, s,
                        "latent_combine_kernel", a.desc, PAIR ? grid / 2 : grid, Cfg<PAIR>::UROWS,
                        a.part_o, a.part_lse, a.o, a.lse, a.H, a.by_h, a.T);
}

}  // namespace
}  // namespace sm103

// part_o [2 * max_ctas * 64 * 512], part_lse [2 * max_ctas * 64], desc
// [2 * max_ctas] int4.
int launch_latent_attn_tc(const mla_dims_t &d, int causal, const TreeMask &tree, int R,
                          const int32_t *qsl, const int32_t *seq_lens, int T, const void *q,
                          const void *cache,
                          int num_blocks, const int32_t *block_table, int bt_stride, float *part_o,
                          float *part_lse, void *desc, int max_ctas, void *o, float *lse,
                          int32_t *status, cudaStream_t s) {
  using namespace sm103;
  // (a cache without blocks gets a map of one row, which nothing asks for)
  const int64_t cache_rows = std::max<int64_t>(1, int64_t(num_blocks) * d.block_size);
  if (cache_rows >= (int64_t(1) << 31) - 64) return MLA_ERR_UNSUPPORTED;
  Maps maps;
  if (!make_tmap_2d_16(&maps.q, false, q, WIDTH, uint64_t(T) * d.num_heads, WIDTH * 2, 64, CROWS,
                       true))
    return MLA_ERR_CUDA;
  if (!make_tmap_3d_16(&maps.v, false, cache, 64, uint64_t(cache_rows), NBLK,
                       WIDTH * 2, 128, 64, 16, true, 4))
    return MLA_ERR_CUDA;
  // the largest box (at most 64 rows) that never crosses a page
  int box_log2 = 0;
  while (box_log2 < MAPS - 1 && d.block_size % (2 << box_log2) == 0) ++box_log2;
  for (int i = 0; i <= box_log2; ++i)
    if (!make_tmap_2d_16(&maps.c[i], false, cache, WIDTH, uint64_t(cache_rows),
                         WIDTH * 2, 64, 1u << i, true))
      return MLA_ERR_CUDA;
  for (int i = box_log2 + 1; i < MAPS; ++i) maps.c[i] = maps.c[box_log2];
  LatentArgs a{qsl, seq_lens, block_table, static_cast<const uint8_t *>(cache),
               static_cast<__nv_bfloat16 *>(o), lse, part_o, part_lse,
               static_cast<int4 *>(desc), status, T, R, d.num_heads, d.block_size, num_blocks,
               int(cache_rows), bt_stride, causal, box_log2,
               reinterpret_cast<uintptr_t>(o) % 32 == 0, Divider(d.block_size),
               Divider(d.num_heads), d.softmax_scale * 1.4426950408889634f, tree};
  // Rows of an average sequence beyond one CTA's 64: pairs, which read the keys
  // once for 128 rows (16 x 4096 keys, 65 to 128 heads: 30 us, single 40; 64 x
  // 4096, 80 heads: 74.5, 115.7).  Up to 64 the single form streams better where
  // there are sequences enough for all SMs (128 x 4096, 32 heads: 109, pairs 119;
  // 128 x 512, 64 heads: 25.0, 35.7); of few long ones it makes more pieces to join
  // (16 x 4096, 64 heads: 52.5, 28.3).  The average is over the slots, of which
  // those without tokens count (their lengths are on the device): 8 of 32 slots x
  // 4096, 128 heads, run single in 51.6 us, pairs 34.8.
  auto launch = [&](auto tree_mask) {
    constexpr bool TREE = decltype(tree_mask)::value;
    if (int64_t(T) * d.num_heads <= int64_t(64) * R)
      return launch_latent<false, TREE, 4>(maps, a, max_ctas, s);
    if (box_log2 == 6) return launch_latent<true, TREE, 6>(maps, a, max_ctas, s);
    if (box_log2 == 5) return launch_latent<true, TREE, 5>(maps, a, max_ctas, s);
    return launch_latent<true, TREE, 4>(maps, a, max_ctas, s);
  };
  return tree.bits ? launch(std::true_type()) : launch(std::false_type());
}

int latent_take_errors() { return sm103::take_error_flags_here(); }

}  // namespace mla
