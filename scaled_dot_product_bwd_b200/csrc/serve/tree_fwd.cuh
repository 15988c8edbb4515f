// tree_fwd.cuh -- attention of drafted nodes (one: plain decoding) over a
// paged bf16 or e4m3 cache.
//
// Mathematics.  The nodes of a sequence times the query heads of a KV head's
// group are the rows of one score matrix against that head's keys, so every
// cached byte is read once for all of them.  Per row an online softmax in
// log2 units: a reference r near the running maximum, the sum l of 2^(s - r)
// and the accumulator O, rescaled when the maximum outgrows r.
//
// The tensor core takes the products transposed: S^T = K Q^T and
// O^T = V^T P^T, so that a tile's 128 keys, then the head's d, are the 128
// rows of a tcgen05 tile and the few query rows are its columns.  A thread of
// the softmax owns one key (one TMEM lane) with all query rows, which makes
// masks, key scales and value scales values of the thread.
//
// An e4m3 cache is multiplied as it lies in memory (kind::f8f6f4), never
// widened.  The other operand is split into two e4m3 parts x = x1 + x2 side
// by side in the columns of one product: 4 + 4 significant bits hold a bf16
// query exactly (down to 2^-21 of its row's largest element) and a weight to
// 2^-8 (small ones: to 2^-20 of the largest, without bias over the keys).  Over
// a bf16 cache a weight is rounded to bf16 (2^-8), as in the framework's forward.
// A key's scale multiplies its scores.  A value row's scale 2^e multiplies the
// weight that enters P V, and r is near the maximum of s + e (over keys whose
// value row is not all zeros), so that what enters stays in range whatever the
// scales are; l adds 2^(s - r).  Where e is beyond +-45, or r so large that e
// would be rounded away (every key under a bias of the type's lowest value), a
// row has a gain of its own for P V, renewed with every tile.
//
// Bound by DRAM: a cached byte takes 2 to 128 FLOPs (1 to 64 rows).  What
// costs is keeping enough loads in flight and every SM busy:
//  * work is cut into tiles of 128 keys of one KV head, laid out over all
//    sequences and heads in one line, and the CTAs (one per SM) take equal
//    pieces of the line, so ragged batches balance and one long sequence uses
//    the whole GPU; a (sequence, head) that spans CTAs leaves partial
//    (r, l, O) in the workspace and a second kernel joins them in order;
//  * roles run on across pieces: a producer warp (TMA, one box per page
//    piece, K and V in slots of their own so that K's is free as soon as S is
//    there), a query warp that lays the next piece's rows out as an operand,
//    an issuing thread each for S and for P V, and four softmax warpgroups
//    of 16 rows.  The softmax's chain of waits per tile (~700 cycles) is what
//    one warpgroup would pay again and again, so up to 16 rows the four take
//    turns by tile, each with an O of its own; at 32 two pairs do; at 64 they
//    share every tile by rows.  Up to 8 rows a thread does 8, not 16 (when it
//    came: e4m3 d = 64 49 -> 44 us, 1000 sequences of 500 bf16 keys 579 -> 484;
//    bf16 d = 64 53 -> 54).
// Measured (32 query, 8 KV heads; 6.56 TB/s is a copy's rate):
//   16 sequences of 8192 keys, one node: bf16 d = 128 88 us (6.1 TB/s, 93 %),
//     d = 64 51 us (80 %); e4m3 d = 128 54 us (77 %), d = 64 43 us (48 %:
//     bound by a tile's chain of steps, not by its bytes); 16 nodes: bf16 101 us
//     (81 %), e4m3 121 us (34 %: softmax instructions)
//   32 ragged sequences of up to 16 k keys, e4m3: 113 us (92 %)
//   16 ragged trees of 16 nodes over up to 8 k keys, bf16: 71 us (75 %; 64 rows,
//     2 to 3 pieces per CTA whose queries and results cost about 3 tiles each)
//   8 trees of 64 nodes over 2000 keys, 12 heads of 64, T5: 31 us (19 %: per
//     piece and softmax instructions)
//   1000 sequences of 500 keys, one node, bf16: 402 us (78 %)
//   one sequence of 4096 keys: 12.5 us (setup 1.2, queries 1.8, tiles, result 1.2,
//     joining kernel 3: a chain of latencies)
// The same with mma.sync and rows as tile rows: 150, 105, 50 us (32 sequences,
// 16 trees, 8 trees).
#pragma once

#include <cfloat>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "kv_cache.cuh"
#include "sm100.cuh"
#include "tmem_sync.cuh"

namespace sdpa {

constexpr uint64_t kTreeDrainNs = 1000000000ull;  // for what is in flight when a wait has run out
constexpr int kTreeMaxCtas = 148;   // one per SM; the workspace is sized for it
constexpr int kTreeMaxNodes = 64;
constexpr int kTreeMaxRows = 64;    // query rows of one product
constexpr int kTreeKeys = 128;      // keys per tile
constexpr int kTreeSoftWarps = 16;
constexpr int kTreeProducer = 16, kTreeIssueS = 17, kTreeIssueO = 18, kTreeQuery = 19;  // the other warps
constexpr int kTreeThreads = 20 * 32;
constexpr int kTreeRT = 16;         // rows of a softmax thread (8 where there are no more)
// Named barriers: 1 .. 4 a softmax warpgroup, 5 all four, 6 + turn those of one tile.
constexpr uint32_t kTreeBarAll = 5, kTreeBarTurn = 6;
// A (sequence, head, row block) costs its first CTA about three tiles more (its
// queries, first maximum, ragged end and result).  The line counts them, so
// that CTAs with many short ones get fewer tiles; where a CTA's share is a few
// tiles of one piece, every CTA pays once and they count as nothing.
__device__ __forceinline__ int tree_piece_cost(int tiles, int ctas) { return tiles >= 8 * ctas ? 3 : 0; }
// T5: buckets of the distances -kTreeNear .. 63 are tabulated per CTA, and the
// table's entries of a KV head's query heads per piece where they fit.
constexpr int kTreeNear = 960, kTreeBuckets = kTreeNear + 64, kTreeT5Slice = 1024;

struct TreeArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int64_t q_t, q_h, o_t, o_h;
  int B, T, max_nodes, Hq, Hkv, G;
  const int* cu;
  const int* ctx;
  const int* table;
  int64_t width, table_b;
  const int64_t* mask;
  int wl;                       // < 0: no window
  int page_size, page_shift, box_rows;
  int64_t num_pages;
  const uint8_t* ks;
  const uint8_t* vs;
  int64_t ss_page, ss_head;
  float scale_log2;
  // bias (BIAS instantiations): ALiBi slopes, or a T5 table when null
  const float* alibi_slopes;
  const float* t5_table;
  T5Spec t5;
  int t5_buckets;
  // workspace
  float2* part_ml;              // [ctas][2][rows] (r, l)
  float* part_o;                // [ctas][2][rows][D]
  uint64_t wait_limit_ns;
};

// What the softmax needs to know of a piece's query rows.
struct TreeRows {
  float scale[kTreeMaxRows];    // log2(e) * scale, and what undoes the operand's scaling (e4m3)
  float bias[kTreeMaxRows];     // ALiBi: its slope; T5: the bias of every distance <= one_lo_max
  uint32_t seen[kTreeMaxNodes][2];  // rows that see a node, 32 a word
  int64_t out[kTreeMaxRows];    // its element offset in o
  int64_t lse[kTreeMaxRows];    // its index in lse
  int pos[kTreeMaxRows];        // its position
  int head[kTreeMaxRows];       // its query head
  int depth[kTreeMaxNodes];     // of the sequence's nodes
};

template <int D, int FMT, int R, int BIAS>
struct TreeLayout {
  static constexpr bool kE4m3 = FMT == kCacheE4m3;
  static constexpr int kCell = kE4m3 ? 1 : 2;
  static constexpr int kRowBytes = D * kCell;               // 64, 128 or 256
  static constexpr int kHalves = kRowBytes == 256 ? 2 : 1;  // 128-byte columns
  static constexpr int kLine = kRowBytes / kHalves;         // bytes of a swizzled row
  static constexpr int kTile = kTreeKeys * kRowBytes;       // bytes of a slot: a tile of K or of V
  static constexpr int kParts = kE4m3 ? 2 : 1;              // of queries and weights
  static constexpr int kN = kParts * R < 16 ? 16 : kParts * R;  // columns of S and of O^T (16: the fewest)
  static constexpr int kQBytes = kN * kRowBytes;
  static constexpr int kPBytes = kN * kTreeKeys * kCell;
  static constexpr int kRT = R < kTreeRT ? R : kTreeRT;     // rows of a softmax thread
  static constexpr int kGroups = R / kRT;                   // softmax warpgroups that share a tile
  static constexpr int kTurns = 4 / kGroups;                // ... and how many such sets there are
  static constexpr int kBufs = kTurns > 2 ? kTurns : 2;     // of S and of the weights
  static constexpr int kRO = R / 4 > 8 ? R / 4 : 8;         // rows a warpgroup writes out
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + 2 * kQBytes;
  static constexpr int kRowsOff = kPOff + kBufs * kPBytes;
  static constexpr int kRowsBytes = (static_cast<int>(sizeof(TreeRows)) + 15) / 16 * 16;
  static constexpr int kMaxOff = kRowsOff + 2 * kRowsBytes;      // [4][kTreeRT][4] floats
  // what a piece leaves for its result, two pieces in turn (so that the
  // warpgroups that do not write it out go on to the next)
  static constexpr int kSumOff = kMaxOff + 4 * kTreeRT * 16;     // [2][4][kTreeRT][4] floats
  static constexpr int kRefOff = kSumOff + 2 * 4 * kTreeRT * 16; // [2][4][kTreeRT] floats
  static constexpr int kFacOff = kRefOff + 2 * 4 * kTreeRT * 4;  // [4][kTreeRT] floats, e4m3: three times
  static constexpr int kGainOff = kFacOff + (kE4m3 ? 3 : 1) * 4 * kTreeRT * 4;     // [2][4][kTreeRT] floats (e4m3)
  static constexpr int kBucketOff = kGainOff + (kE4m3 ? 2 * 4 * kTreeRT * 4 : 0);  // [kTreeBuckets] bytes
  static constexpr int kT5Off = kBucketOff + (BIAS ? kTreeBuckets : 0);  // [2][kTreeT5Slice] floats
  static constexpr int kMiscOff = kT5Off + (BIAS ? 2 * kTreeT5Slice * 4 : 0);
  static constexpr int kMaxSlots = 12;
  static constexpr int kNumBars = 2 * kMaxSlots + 4 * kBufs + 6;
  static constexpr int kMiscBytes = kNumBars * 8 + 160;
  static constexpr int kRingOff = (kMiscOff + kMiscBytes + 1023) / 1024 * 1024;
  // (2 KB of the SM's shared memory stay free: a CTA of the joining kernel
  // must find room beside this one to be ready when it ends)
  static constexpr int kBudget = 230400;
  static constexpr int kFit = (kBudget - kRingOff) / kTile / 2 * 2;
  static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;  // K and V in turn: even
  static constexpr int kSmem = kRingOff + kSlots * kTile;
  static constexpr int kOCol = kBufs * kN;                  // the O^T after the S buffers
  static constexpr int kCols = kOCol + 2 * kTurns * kN;     // ... of two pieces
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kSlots >= 4 && kSmem <= kBudget, "shared memory budget");
  static_assert(kCols <= 512, "tensor memory budget");
  static_assert(kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "operand alignment");
  static_assert(kMiscOff % 16 == 0, "barrier alignment");
  // byte offset of 16-byte piece c of row r in a block of `rows` swizzled rows
  static __device__ __forceinline__ uint32_t at(int r, int c, int rows) {
    if (kLine == 128)
      return static_cast<uint32_t>((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
};

// What one sequence needs of a kernel, from its entries in cu_nodes and ctx_lens.
struct TreeSeq {
  int row0, n, ctx, keys;  // first query row, nodes, context length, context + nodes
  int tile0, tiles, rb;    // first key tile any node sees, tiles, row blocks
  // length on the line: per (head, row block) the piece cost, then the tiles
  __device__ __forceinline__ int units(int Hkv, int cost) const { return Hkv * rb * (cost + tiles); }
};

template <int R>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b) {
  TreeSeq s;
  s.row0 = a.cu[b];
  s.n = a.cu[b + 1] - s.row0;
  s.ctx = a.ctx[b];
  const bool bad = s.row0 < 0 || s.n < 0 || s.n > a.max_nodes || s.row0 > a.T - s.n || s.ctx < 0 ||
                   (s.n > 0 && static_cast<int64_t>(s.ctx) + s.n > (a.width << a.page_shift));
  if (bad) {
    atomicOr(&g_device_status, kStatusBadSeqlens);
    s.row0 = s.n = s.ctx = 0;
  }
  s.keys = s.ctx + s.n;
  s.tile0 = a.wl >= 0 ? max(0, s.ctx - a.wl) / kTreeKeys : 0;
  s.tiles = (s.keys + kTreeKeys - 1) / kTreeKeys - s.tile0;
  s.rb = (s.n * a.G + R - 1) / R;
  if (s.n == 0) s.tiles = s.rb = 0;
  return s;
}

// One CTA's piece of the line of tiles; next() gives it (sequence, head, row
// block) by (sequence, head, row block).
template <int R>
struct TreeWalk {
  int left;           // of the CTA's part of the line, not walked yet
  int cost;           // of a piece
  int b, off, units;  // current sequence, how much of its part is walked, its length
  TreeSeq s;
  int hkv, block, t0, nt;  // this step: head, row block, first tile, tiles
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    while (left > 0) {
      while (off >= units) {
        off -= units;
        s = tree_seq<R>(a, ++b);
        units = s.units(a.Hkv, cost);
      }
      const int span = cost + s.tiles;
      const int seg = off / span;
      const int in = off - seg * span;
      const int n = min(span - in, left);
      left -= n;
      off += n;
      t0 = max(in - cost, 0);
      nt = in + n - cost - t0;
      hkv = seg / s.rb;
      block = seg - hkv * s.rb;
      if (nt > 0) return true;
    }
    return false;
  }
};

// A CTA's part of a line of `total` (which the host keeps below 2^31 - 2^16).
__device__ __forceinline__ int tree_share(int total, int ctas) { return (total + ctas - 1) / ctas; }

// Where the part of a CTA begins: `left` tiles and piece costs from `off` in
// sequence b on (nothing: left = 0).
struct TreeSpot {
  int left, per, cost;
  int b, off;
  TreeSeq s;
};

// The part of CTA `cta` of `ctas`, into shared memory, by one warp: up to 32
// sequences, a lane each.
template <int R>
__device__ __forceinline__ void tree_locate(const TreeArgs& a, int cta, int ctas, int lane, TreeSpot* out) {
  TreeSeq s{};
  if (lane < a.B) s = tree_seq<R>(a, lane);
  const int tiles = __reduce_add_sync(~0u, lane < a.B ? s.units(a.Hkv, 0) : 0);
  const int pieces = __reduce_add_sync(~0u, lane < a.B ? s.rb * a.Hkv : 0);
  const int cost = tree_piece_cost(tiles, ctas);
  const int total = tiles + cost * pieces;
  const int per = tree_share(total, ctas);
  const int from = static_cast<int>(min(static_cast<int64_t>(per) * cta, static_cast<int64_t>(total)));
  if (lane == 0) {
    out->left = min(total - from, per);
    out->per = per;
    out->cost = cost;
  }
  const int units = lane < a.B ? s.units(a.Hkv, cost) : 0;
  int upto = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += y;
  }
  if (upto - units <= from && from < upto) {
    out->b = lane;
    out->off = from - (upto - units);
    out->s = s;
  }
}

// The same for any number of sequences, by all NW warps of a block (`totals`:
// 2 * NW ints of shared memory; it may be read once all of the block are
// through a barrier).  Each warp adds up a range of its own, then each goes
// through the one range that holds the place.  Out of line: inlined it would
// hold up the setup of those that do not come here.
template <int R, int NW>
__device__ __noinline__ void tree_locate_many(const TreeArgs& a, int cta, int ctas, int warp, int lane, int* totals,
                                              TreeSpot* out) {
  const int range = ((a.B + NW - 1) / NW + 31) / 32 * 32;
  int tiles = 0, pieces = 0;
  for (int b = warp * range + lane; b < min(a.B, (warp + 1) * range); b += 32) {
    const TreeSeq s = tree_seq<R>(a, b);
    tiles += s.units(a.Hkv, 0);
    pieces += s.rb * a.Hkv;
  }
  tiles = __reduce_add_sync(~0u, tiles);
  pieces = __reduce_add_sync(~0u, pieces);
  if (lane == 0) {
    totals[2 * warp] = tiles;
    totals[2 * warp + 1] = pieces;
  }
  __syncthreads();
  const int mine_t = lane < NW ? totals[2 * lane] : 0, mine_p = lane < NW ? totals[2 * lane + 1] : 0;
  tiles = __reduce_add_sync(~0u, mine_t);
  pieces = __reduce_add_sync(~0u, mine_p);
  const int cost = tree_piece_cost(tiles, ctas);
  const int total = tiles + cost * pieces;
  const int per = tree_share(total, ctas);
  const int from = static_cast<int>(min(static_cast<int64_t>(per) * cta, static_cast<int64_t>(total)));
  if (threadIdx.x == 0) {
    out->left = min(total - from, per);
    out->per = per;
    out->cost = cost;
  }
  int upto = mine_t + cost * mine_p;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += y;
  }
  const uint32_t holds = __ballot_sync(~0u, lane < NW && from < upto);
  const int w = holds ? __ffs(holds) - 1 : NW;
  if (w != warp) return;  // one warp stays, or none: nothing left for this CTA
  int base = __shfl_sync(~0u, upto - (mine_t + cost * mine_p), w);
  for (int b0 = w * range; b0 < min(a.B, (w + 1) * range); b0 += 32) {
    const int b = b0 + lane;
    TreeSeq s{};
    if (b < a.B) s = tree_seq<R>(a, b);
    const int units = b < a.B ? s.units(a.Hkv, cost) : 0;
    int end = base + units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, end - base, o);
      if (lane >= o) end += y;
    }
    if (end - units <= from && from < end) {
      out->b = b;
      out->off = from - (end - units);
      out->s = s;
    }
    base = __shfl_sync(~0u, end, 31);
  }
}

// ------------------------------------------------- operands of the products
// Shared-memory matrix descriptor of a layout: 0 plain, 2 128-byte swizzle,
// 4 64-byte swizzle.  A K-major operand steps 8 rows by sbo; an MN-major one
// steps 8 rows of K by sbo and a swizzle width along M by lbo when swizzled,
// 8 rows of K by lbo and 16 bytes along N by sbo when plain.
__device__ __forceinline__ uint64_t tree_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo,
                                              uint32_t layout) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46 |
         static_cast<uint64_t>(layout) << 61;
}

template <int FMT>
__device__ __forceinline__ void tree_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  if (FMT == kCacheBf16) {
    mma_ss(d_tmem, adesc, bdesc, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// N fp32 columns of the warp's lanes, complete on return.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&x)[N]) {
  if constexpr (N == 8) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
  } else if constexpr (N == 16) {
    uint32_t r[16];
    tmem_ld16_sync(taddr, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
  } else {
    uint32_t r[32];
    tmem_ld32_sync(taddr, r);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
  }
}

// Twice 16 columns, with one wait for both.
__device__ __forceinline__ void tmem_ld_two(uint32_t at_x, uint32_t at_y, float (&x)[16], float (&y)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at_x), "r"(at_y)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = __uint_as_float(r[i]);
    y[i] = __uint_as_float(r[16 + i]);
  }
}

template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&x)[N]) {
  if constexpr (N == 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])),
        "r"(__float_as_uint(x[3])), "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])),
        "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
        : "memory");
  } else if constexpr (N == 16) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
    tmem_st16_sync(taddr, r);
  } else {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(x[i]);
    tmem_st32_sync(taddr, r);
  }
}

// y += x * f.
template <int N>
__device__ __forceinline__ void fma_rows(const float (&x)[N], float f, float* y) {
  const uint64_t f2 = f2_pack(f, f);
#pragma unroll
  for (int j = 0; j < N; j += 2)
    f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), f2, f2_pack(y[j], y[j + 1])), y[j], y[j + 1]);
}

// Row j's x[j] of all 32 lanes combined, for row lane / (32 / N): lanes trade
// halves of their rows, the upper ones keeping the upper half, until one row
// is left to each.
template <int N, typename Op>
__device__ __forceinline__ float by_halves(const float (&x)[N], int lane, Op op) {
  float y[N / 2];
  {
    const bool up = (lane & 16) != 0;
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      y[j] = op(up ? x[j + N / 2] : x[j], __shfl_xor_sync(~0u, up ? x[j] : x[j + N / 2], 16));
  }
#pragma unroll
  for (int n = N / 2, o = 8; n > 1; n >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int j = 0; j < n / 2; ++j)
      y[j] = op(up ? y[j + n / 2] : y[j], __shfl_xor_sync(~0u, up ? y[j] : y[j + n / 2], o));
  }
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) y[0] = op(y[0], __shfl_xor_sync(~0u, y[0], o));
  return y[0];
}

// Whether `x` holds for any thread of the named barrier's `count`.
__device__ __forceinline__ bool barrier_or(uint32_t id, uint32_t count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Two floats as e4m3 codes (x0 in the low byte), rounded to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

// What the second part of a split is multiplied by: with the first part
// rounded to 4 bits, |rest| <= 8 for queries below 256 and <= 16 for weights
// up to 416, so the products stay below 448 and far above 2^-9.
constexpr float kQueryRest = 16.f, kWeightRest = 16.f;
// Weights are 2^(s - r).  Over a bf16 cache r is a maximum that a later score
// may outgrow by 2^8 before O is rescaled; over e4m3, whose largest value is
// 448, r is set 7 below the maximum of s + e and outgrown at 2^8.7 = 416.  There
// e counts from kLeastE to kMostE: r then moves by at most 2^97 for the values'
// sake, and l, whose terms are 2^-e as large, loses nothing above 2^-29 of the
// largest when it does.  Where that leaves a row's weights small or large, or r
// has less than 3 bits below the point (from kManyDigits on), its weights are
// 2^(s - r) times 2^e times a gain 2^-t, t found as r is, from s - r + e.
constexpr float kTopBf16 = 0.f, kOverBf16 = 8.f, kTopE4m3 = 7.f, kOverE4m3 = 8.7f;
constexpr float kLeastE = -45.f, kMostE = 45.f, kManyDigits = 0x1p20f, kMostGain = 0x1p120f;
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// All bits of the codes / bf16 halves in w that are infinite or NaN.
template <int FMT>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  return FMT == kCacheBf16 ? __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u)
                           : __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// The codes of what the codes `w` leave of two weights, times kWeightRest, plus
// the key's share `d` of the last step, between -1/2 and 1/2 of it.  Weights below
// the last step (2^-20 of the largest) are many where a context is long: rounded
// to nearest, all of one size would be lost or doubled together; with shares
// spread evenly over the keys their sum is right.
__device__ __forceinline__ uint32_t e4m3x2_rest(float x0, float x1, uint32_t w, __half2 d) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  // at most 448 * 16 in fp16: exact (d is lost beside all but the smallest)
  const __half2 n = __hfma2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(-kWeightRest), d);
  const float2 nf = __half22float2(n);
  float r0, r1;
  f2_unpack(f2_fma(f2_pack(x0, x1), f2_pack(kWeightRest, kWeightRest), f2_pack(nf.x, nf.y)), r0, r1);
  return e4m3x2(r0, r1);
}

// b * log2(e) of a bias b, kept finite where b is: a bias of the type's lowest
// value then still orders below every other score instead of hiding its key.
// It stays above the reference -FLT_MAX of a row that has seen no key, so that
// the first such key is seen to outgrow it.
constexpr float kLowest = -0x1.fffffcp127f;
__device__ __forceinline__ float bias_to_log2(float b) {
  const float x = b * kLog2e;
  return isinf(b) ? x : fminf(fmaxf(x, kLowest), -kLowest);
}

// LSE of a row with reference r and sum l (0: it sees nothing).  A reference of
// kLowest is a bias of the lowest value.
__device__ __forceinline__ float tree_lse(float r, float l) {
  return r == kLowest ? -FLT_MAX : (r + log2f(l)) * kLn2;
}

__device__ __forceinline__ float t5_bias_log2(const TreeArgs& a, int rel, int h) {
  return bias_to_log2(a.t5_table[t5_bucket(rel, a.t5) * a.Hq + h]);
}

// ---------------------------------------------------------------- queries
// One piece's query rows as the K-major operand `dst` (kN rows; e4m3: first
// parts in rows 0 .. R - 1, second parts from row R on), by warp w of nw.
template <int D, int FMT, int R, int BIAS>
__device__ __forceinline__ void tree_load_queries(const TreeArgs& a, const TreeWalk<R>& wk, int w, int nw,
                                                  int lane, uint8_t* dst, TreeRows* info) {
  using L = TreeLayout<D, FMT, R, BIAS>;
  const TreeSeq& s = wk.s;
  const int n_rows = s.n * a.G - wk.block * R;  // of this block, may exceed R
  constexpr int kLanes = D / 8;        // lanes of a row, 8 elements each
  constexpr int kPass = 32 / kLanes;   // rows per pass
  constexpr int kFlight = 4;
  const int c = lane % kLanes, sub = lane / kLanes;
  for (int p0 = w; p0 * kPass < R; p0 += nw * kFlight) {
    uint4 x[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int r = (p0 + f * nw) * kPass + sub;
      x[f] = make_uint4(0, 0, 0, 0);
      if (r < min(R, n_rows)) {
        const int at = wk.block * R + r;
        const int n = at / a.G;
        x[f] = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(s.row0 + n) * a.q_t +
                                               (wk.hkv * a.G + at - n * a.G) * a.q_h + c * 8);
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int r = (p0 + f * nw) * kPass + sub;
      if ((p0 + f * nw) * kPass >= R) break;
      if (FMT == kCacheBf16) {
        *reinterpret_cast<uint4*>(dst + L::at(r, c, L::kN)) = x[f];
        continue;
      }
      // the row by a power of two that puts its largest element in [128, 256)
      const uint32_t v[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
      int e = static_cast<int>(m >> 7);          // biased exponent
      e = e == 255 ? 134 : min(max(e, 16), 250);
      // 2^(134 - e) in two factors, each a normal float
      const int e1 = (134 - e) / 2, e2 = 134 - e - e1;
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e1) << 23);
      const float f2 = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y0 = __uint_as_float(v[i] << 16) * f1 * f2;
        const float y1 = __uint_as_float(v[i] & 0xffff0000u) * f1 * f2;
        hi[i] = e4m3x2(y0, y1);
        const float2 h = e4m3x2_value(hi[i]);
        lo[i] = e4m3x2((y0 - h.x) * kQueryRest, (y1 - h.y) * kQueryRest);
      }
      // a row that is not finite gives what float32 gives: NaN
      if (m >= 0x7f80u) hi[0] = hi[1] = hi[2] = hi[3] = 0x7f7fu;
      *reinterpret_cast<uint2*>(dst + L::at(r, c >> 1, L::kN) + (c & 1) * 8) =
          make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(dst + L::at(R + r, c >> 1, L::kN) + (c & 1) * 8) =
          make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      // the other way round: 2^(e - 134)
      if (c == 0)
        info->scale[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e1) << 23) *
                         __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
    }
  }
}

// The rest of the piece's TreeRows.
template <int R, int BIAS>
__device__ __forceinline__ void tree_load_rows(const TreeArgs& a, const TreeWalk<R>& wk, int w, int nw,
                                               int lane, TreeRows* info, float* t5_slice) {
  const TreeSeq& s = wk.s;
  const int n_rows = s.n * a.G - wk.block * R;  // of this block, may exceed R
  const uint64_t node_bits = s.n >= 64 ? ~0ull : (1ull << s.n) - 1ull;
  auto sees_of = [&](int n) -> uint64_t {
    const uint64_t m = a.mask ? static_cast<uint64_t>(a.mask[s.row0 + n]) : ~0ull >> (63 - n);
    return m & node_bits;
  };
  for (int r0 = w * 32; r0 < R; r0 += nw * 32) {
    const int r = r0 + lane;
    uint64_t sees = 0;
    if (r < R) {
      float slope = 0.f;
      int pos = s.ctx, head = wk.hkv * a.G;
      int64_t out = 0, lse = 0;
      if (r < n_rows) {
        const int x = wk.block * R + r;
        const int n = x / a.G;
        sees = sees_of(n);
        pos += __popcll(sees & ~(1ull << n));
        head += x - n * a.G;
        out = static_cast<int64_t>(s.row0 + n) * a.o_t + static_cast<int64_t>(head) * a.o_h;
        lse = static_cast<int64_t>(head) * a.T + s.row0 + n;
        if constexpr (BIAS != 0) {
          if (a.alibi_slopes) slope = a.alibi_slopes[head];
          else if (a.t5.one_lo_max != INT_MIN) slope = t5_bias_log2(a, a.t5.one_lo_max, head);
        }
      } else {
        sees = node_bits;  // rows of padding count as seeing every node
      }
      info->bias[r] = slope;
      info->pos[r] = pos;
      info->head[r] = head;
      info->out[r] = out;
      info->lse[r] = lse;
    }
    for (int n = 0; n < s.n; ++n) {
      const uint32_t rows = __ballot_sync(~0u, (sees >> n) & 1ull);
      if (lane == (n & 31)) info->seen[n][r0 / 32] = rows;
    }
  }
  if (w == nw - 1)
    for (int n = lane; n < s.n; n += 32) info->depth[n] = __popcll(sees_of(n) & ~(1ull << n));
  if (BIAS != 0 && a.t5_table && a.t5_buckets * a.G <= kTreeT5Slice) {
#pragma unroll 4
    for (int i = w * 32 + lane; i < a.t5_buckets * a.G; i += nw * 32) {
      const int k = i / a.G;
      t5_slice[i] = bias_to_log2(a.t5_table[k * a.Hq + wk.hkv * a.G + (i - k * a.G)]);
    }
  }
}

// What follows runs for unusual values alone and is kept out of line: in line,
// its instructions would be fetched for every piece (256 sequences of 8 nodes
// over e4m3 301 us, so 282).

// Whether key `me` of a tile in the ring has e4m3 codes of zero alone.
template <typename L>
__device__ __noinline__ bool tree_row_of_zeros(const uint8_t* tile, int me) {
  uint32_t some = 0;
  for (int c = 0; c < L::kRowBytes / 16; ++c) {
    const uint4 w = *reinterpret_cast<const uint4*>(tile + L::at(me, c, kTreeKeys));
    some |= w.x | w.y | w.z | w.w;
  }
  return !(some & 0x7f7f7f7fu);
}

// New gains of a warpgroup's rows, from the scores `sc` of a thread's key under
// the new references with the exponent `e` of its value scale; whether any is
// not 1 (`had`: whether one was).  By all of the warpgroup.
template <int RT>
__device__ __noinline__ bool tree_renew_gains(const float* sc, float e, bool had, const float* refs, float* gains,
                                              const float* facs, float* facs_o, float* peaks, float* mine, int wg,
                                              int warp, int lane) {
  for (int j = 0; j < RT; ++j) {
    const float top = warp_max((sc[j] - refs[wg * RT + j]) + e);
    if (lane == 0) mine[j * 4 + (warp & 3)] = top;
  }
  named_barrier(1 + wg, 128);
  bool gained = false;
  if ((warp & 3) == 0 && lane < RT) {
    const int at = wg * RT + lane;
    const float4 w4 = *reinterpret_cast<const float4*>(mine + lane * 4);
    const float m = fmaxf(fmaxf(w4.x, w4.y), fmaxf(w4.z, w4.w)) - kTopE4m3;
    // the largest m that O holds weights of, under the new r: the gain lifts O
    // by 2^80 at most, so that it stays finite
    const float held = fmaxf((had ? peaks[at] : 0.f) + __log2f(facs[at]), m);
    const float old = gains[at];
    float gain = fabsf(refs[at]) >= kManyDigits || fabsf(m) > 1.f ? fast_exp2(-m) : 1.f;
    if (m == -INFINITY) gain = old;
    gain = fminf(fminf(gain, fast_exp2(80.f - held)), kMostGain);
    peaks[at] = held;
    gains[at] = gain;
    if (gain != old) facs_o[at] = facs[at] * gain * fast_rcp(old);
    gained = gain != 1.f;
  }
  return barrier_or(1 + wg, 128, gained);
}

// Takes infinite and NaN values of keys hidden from some row out of a tile of V
// (`odd`: this thread's key has some), and gives what the rows that see such a
// key then miss.  By all threads of the tile.
template <int D, int FMT, int R, int BIAS>
__device__ __noinline__ void tree_take_out(int wl, int ctx, int key0, const TreeRows* info, uint8_t* vrows,
                                           const uint8_t* weights, uint32_t* bits, uint32_t odd, uint32_t b_tile,
                                           int row0, int warp, int lane, float* missing) {
  using L = TreeLayout<D, FMT, R, BIAS>;
  constexpr bool E4 = L::kE4m3;
  constexpr uint32_t kTileThreads = 128 * L::kGroups;
  const int me = (warp & 3) * 32 + lane;
  const uint32_t some = __ballot_sync(~0u, odd != 0);
  if (lane == 0 && some) atomicOr(&bits[warp & 3], some);
  named_barrier(b_tile, kTileThreads);
  for (int j = 0; j < L::kRT; ++j) missing[j] = 0.f;
  for (int k4 = 0; k4 < 4; ++k4)
    for (uint32_t left = bits[k4]; left; left &= left - 1) {
      const int k = k4 * 32 + __ffs(left) - 1;
      float v = 0.f;
      if (me < D) {
        const int byte = me * L::kCell;
        const uint8_t* src = vrows + L::at(k, byte >> 4, kTreeKeys) + (byte & 15);
        if (E4) v = (*src & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : 0.f;
        else v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(src));
      }
      if (!isinf(v) && !isnan(v)) continue;
      // (a row that sees the key gets it whatever its weight, as in a tile that
      // all rows see)
      const int nd = key0 + k - ctx;
      const int pos = nd >= 0 ? ctx + info->depth[nd] : key0 + k;
      const uint32_t sees = nd >= 0 ? info->seen[nd][row0 / 32] >> (row0 % 32) : ~0u;
      const uint8_t* pk = weights + k * 16;
      for (int j = 0; j < L::kRT; ++j) {
        if (!((sees >> j) & 1u) || (wl >= 0 && info->pos[row0 + j] - pos > wl)) continue;
        const int byte = (row0 + j) * L::kCell;
        missing[j] += E4 ? v : v * __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                                       pk + (byte >> 4) * (kTreeKeys * 16) + (byte & 15)));
      }
    }
  named_barrier(b_tile, kTileThreads);
  if (row0 == 0 && me < 4) bits[me] = 0;
  if (odd != 0) {
    for (int c = 0; c < L::kRowBytes / 16; ++c) {
      uint4* p = reinterpret_cast<uint4*>(vrows + L::at(me, c, kTreeKeys));
      uint4 w = *p;
      w.x &= ~nonfinite_bits<FMT>(w.x);
      w.y &= ~nonfinite_bits<FMT>(w.y);
      w.z &= ~nonfinite_bits<FMT>(w.z);
      w.w &= ~nonfinite_bits<FMT>(w.w);
      *p = w;
    }
  }
}

// ---------------------------------------------------------------- kernel
template <int D, int FMT, int R, int BIAS>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_fwd_kernel(
    const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap mk,
    const __grid_constant__ CUtensorMap mv) {
  using L = TreeLayout<D, FMT, R, BIAS>;
  constexpr bool E4 = L::kE4m3;
  constexpr int NS = L::kSlots;
  constexpr int RT = L::kRT;
  constexpr int RO = L::kRO;
  constexpr int TN = L::kTurns, NB = L::kBufs, RG = L::kGroups;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!smem_base_ok(smem)) {
    if (threadIdx.x == 0) atomicOr(&g_device_status, kStatusMisaligned);
    return;
  }
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  auto bar = [&](int i) -> uint32_t { return sb + L::kMiscOff + 8 * i; };
  auto full = [&](int s) { return bar(s); };
  auto empty = [&](int s) { return bar(L::kMaxSlots + s); };
  constexpr int kB = 2 * L::kMaxSlots;
  auto s_full = [&](int x) { return bar(kB + x); };            // S of a tile is in tensor memory
  auto s_free = [&](int x) { return bar(kB + NB + x); };       // ... and in registers
  auto p_full = [&](int x) { return bar(kB + 2 * NB + x); };   // weights are in shared memory
  auto pv_done = [&](int x) { return bar(kB + 3 * NB + x); };  // ... and added to O
  constexpr int kQ = kB + 4 * NB;
  auto q_full = [&](int x) { return bar(kQ + x); };            // a piece's queries are laid out
  auto q_free = [&](int x) { return bar(kQ + 2 + x); };        // ... and the piece is done
  auto drain = [&](int x) { return bar(kQ + 4 + x); };
  // K of the CTA's tile `it` is item 2 it of the ring, its V item 2 it + 1
  auto slot_off = [&](uint32_t item) { return L::kRingOff + (item % NS) * L::kTile; };
  uint8_t* misc = smem + L::kMiscOff + L::kNumBars * 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  uint32_t* dirty = reinterpret_cast<uint32_t*>(misc + 80);   // [4 turns][4] bits of keys
  TreeSpot* spot = reinterpret_cast<TreeSpot*>(misc + 16);  // 48 bytes

  if (warp == kTreeIssueS) {
    if (lane == 0) {
      *abort_flag = 0;
      for (int x = 0; x < 16; ++x) dirty[x] = 0;
      for (int s = 0; s < NS; ++s) {
        mbar_init(full(s), 1);
        mbar_init(empty(s), 1);
      }
      for (int x = 0; x < NB; ++x) {
        mbar_init(s_full(x), 1);
        mbar_init(s_free(x), 4 * RG);
        mbar_init(p_full(x), 4 * RG);
        mbar_init(pv_done(x), 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(q_full(x), kTreeSoftWarps);
        mbar_init(q_free(x), kTreeSoftWarps);
        mbar_init(drain(x), 1);
      }
      fence_mbar_init();
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  } else if (warp == kTreeProducer) {
    if (a.B <= 32) tree_locate<R>(a, blockIdx.x, gridDim.x, lane, spot);
  } else if (BIAS != 0 && warp < kTreeSoftWarps && a.t5_table) {
    for (int i = tid; i < kTreeBuckets; i += kTreeSoftWarps * 32)
      smem[L::kBucketOff + i] = static_cast<uint8_t>(t5_bucket(i - kTreeNear, a.t5));
  }
  if (a.B > 32)
    tree_locate_many<R, kTreeThreads / 32>(a, blockIdx.x, gridDim.x, warp, lane,
                                           reinterpret_cast<int*>(smem + L::kRingOff), spot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, a.wait_limit_ns};
  TreeWalk<R> walk;
  walk.left = spot->left;
  walk.cost = spot->cost;
  walk.b = spot->b;
  walk.off = spot->off;
  walk.s = spot->s;
  walk.units = walk.s.units(a.Hkv, walk.cost);

  if (warp == kTreeProducer) {
    // ------------------------------------------------------------ producer
    const int boxes = kTreeKeys / a.box_rows;  // <= 8
    const uint32_t box_bytes = static_cast<uint32_t>(a.box_rows) * L::kRowBytes;
    uint32_t it = 0, item = 0;
    bool ok = true;
    while (ok && walk.next(a)) {
      const int* row = a.table + static_cast<int64_t>(walk.b) * a.table_b;
      // page ids, a lane per box: 32 boxes ahead, and the 32 after them on their way
      const int batch = 32 / boxes;  // tiles
      auto pages_of = [&](int t) {
        const int pos = (walk.s.tile0 + t) * kTreeKeys + lane * a.box_rows;
        int page = -1;
        if (pos < walk.s.keys) {
          page = row[pos >> a.page_shift];
          // past the cache: the copy fills zeros
          if (page < 0 || page >= a.num_pages) page = static_cast<int>(a.num_pages);
        }
        return page;
      };
      int pages = pages_of(walk.t0), next_pages = pages_of(walk.t0 + batch);
      for (int i = 0; ok && i < walk.nt; ++i, ++it) {
        const int t = walk.t0 + i;
        const int in = i & (batch - 1);
        if (in == 0 && i > 0) {
          pages = next_pages;
          next_pages = pages_of(t + batch);
        }
        const int page = __shfl_sync(~0u, pages, in * boxes + (lane & (boxes - 1)));
        const bool copy = lane < boxes && page >= 0;
        // (a page behind every node's window may be gone)
        if (copy && page == a.num_pages &&
            (a.wl < 0 || (walk.s.tile0 + t) * kTreeKeys + (lane + 1) * a.box_rows > walk.s.ctx - a.wl))
          atomicOr(&g_device_status, kStatusBadSeqlens);
        const int n_copy = __popc(__ballot_sync(~0u, copy));
        const int r = ((walk.s.tile0 + t) * kTreeKeys + lane * a.box_rows) & (a.page_size - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++item) {
          const uint32_t f = full(item % NS);
          if (item >= NS) ok = mbar_wait(empty(item % NS), ((item / NS) - 1) & 1, ctl);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(f, n_copy * box_bytes);
          __syncwarp();
          if (copy) {
            const uint32_t dst = sb + slot_off(item) + static_cast<uint32_t>(lane) * a.box_rows * L::kLine;
#pragma unroll
            for (int h = 0; h < L::kHalves; ++h)
              tma_load_4d(dst + h * kTreeKeys * 128, kv ? &mv : &mk, f, h * 64, r, walk.hkv, page);
          }
        }
      }
    }
    if (!ok) {
      // a wait that ran out ends the CTA: let the copies in flight land first
      volatile int never = 0;
      const WaitCtl ign{&never, max(a.wait_limit_ns, kTreeDrainNs)};
      for (uint32_t j = item > NS ? item - NS : 0; j < item; ++j) mbar_wait(full(j % NS), (j / NS) & 1, ign);
    }
  } else if (warp == kTreeQuery) {
    // ------------------------------------------------------------- queries
    // (the first piece's are laid out by the softmax warps, which have
    // nothing else to do yet)
    uint32_t u = 1;
    bool ok = walk.next(a);
    while (ok && walk.next(a)) {
      const int x = u & 1;
      if (u >= 2) ok = __all_sync(~0u, mbar_wait(q_free(x), ((u >> 1) - 1) & 1, ctl));
      if (!ok) break;
      TreeRows* info = reinterpret_cast<TreeRows*>(smem + L::kRowsOff + x * L::kRowsBytes);
      tree_load_queries<D, FMT, R, BIAS>(a, walk, 0, 1, lane, smem + L::kQOff + x * L::kQBytes, info);
      tree_load_rows<R, BIAS>(a, walk, 0, 1, lane, info,
                              reinterpret_cast<float*>(smem + L::kT5Off) + x * kTreeT5Slice);
      fence_async_shared();
      __syncwarp();
      if (lane < kTreeSoftWarps) mbar_arrive(q_full(x));
      ++u;
    }
  } else if (warp == kTreeIssueS || warp == kTreeIssueO) {
    // ----------------------------------------------------------- MMA issuers
    const bool is_s = warp == kTreeIssueS;
    if (lane == 0) {
      constexpr uint32_t kShape = (1u << 4) | (E4 ? 0u : (1u << 7) | (1u << 10)) |
                                  (static_cast<uint32_t>(L::kN >> 3) << 17) |
                                  (static_cast<uint32_t>(128 >> 4) << 24);  // f32, M = 128
      constexpr uint32_t kIdS = kShape, kIdO = kShape | (1u << 15) | (1u << 16);
      constexpr uint32_t kSwz = L::kLine == 128 ? 2u : 4u;
      constexpr int kStep = E4 ? 32 : 16;  // keys per instruction of P V
      const uint64_t dk = tree_desc(sb, 16, 8 * L::kLine, kSwz);  // K and Q, K-major
      // V, MN-major: 64-wide halves kTreeKeys rows apart; at d = 64 the
      // tile's rows 64 .. 127 repeat its first 64 and are not read back
      const uint64_t dv = tree_desc(sb, D == 128 && !E4 ? kTreeKeys * 128 : 0, 8 * L::kLine, kSwz);
      const uint64_t dp = tree_desc(sb, 128, kTreeKeys * 16, 0);  // weights, MN-major, plain
      uint32_t it = 0, u = 0;
      bool ok = true;
      while (ok && walk.next(a)) {
        if (is_s) ok = mbar_wait(q_full(u & 1), (u >> 1) & 1, ctl);
        const uint64_t qd = dk + ((L::kQOff + (u & 1) * L::kQBytes) >> 4);
        for (int i = 0; ok && i < walk.nt; ++i, ++it) {
          const uint32_t x = it % NB, item = 2 * it + (is_s ? 0 : 1);
          if (!(ok = mbar_wait(full(item % NS), (item / NS) & 1, ctl))) break;
          if (is_s) {  // S^T = K Q^T
            if (it >= NB && !(ok = mbar_wait(s_free(x), (it / NB - 1) & 1, ctl))) break;
            tc_fence_after();
            const uint64_t kd = dk + (slot_off(item) >> 4);
#pragma unroll
            for (int k = 0; k < L::kRowBytes / 32; ++k)
              tree_mma<FMT>(tmem + x * L::kN, kd + (kmajor_koff(k, kTreeKeys) >> 4),
                            qd + (kmajor_koff(k, L::kN) >> 4), kIdS, k > 0 ? 1u : 0u);
            mma_commit(s_full(x));
          } else {  // O^T += V^T P^T; a piece's first tile in an O overwrites it
            if (!(ok = mbar_wait(p_full(x), (it / NB) & 1, ctl))) break;
            tc_fence_after();
            const uint64_t vd = dv + (slot_off(item) >> 4);
            const uint64_t pd = dp + ((L::kPOff + x * L::kPBytes) >> 4);
            const uint32_t o = tmem + L::kOCol + ((u & 1) * TN + it % TN) * L::kN;
            const bool add = i >= TN;
#pragma unroll
            for (int k = 0; k < kTreeKeys / kStep; ++k)
              tree_mma<FMT>(o, vd + (k * kStep * L::kLine >> 4), pd + (k * kStep * 16 >> 4), kIdO,
                            add || k > 0 ? 1u : 0u);
            mma_commit(pv_done(x));
          }
          mma_commit(empty(item % NS));
        }
        ++u;
      }
      // every MMA issued is done before tensor memory is freed
      volatile int never = 0;
      const WaitCtl ign{&never, max(a.wait_limit_ns, kTreeDrainNs)};
      mma_commit(drain(is_s ? 0 : 1));
      mbar_wait(drain(is_s ? 0 : 1), 0, ign);
    }
    __syncwarp();
  } else {
    // ------------- softmax: thread = key of the tile, and row of O^T at the end
    const int wg = warp >> 2;
    const int me = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t turn = wg / RG;          // takes the tiles it = turn (mod TN)
    const int row0 = wg % RG * RT;          // first row of this thread's scores
    constexpr uint32_t kTileThreads = 128 * RG;  // that work on one tile
    const uint32_t b_tile = RG == 1 ? 1 + wg : kTreeBarTurn + turn;
    float* wmax = reinterpret_cast<float*>(smem + L::kMaxOff);    // [4][RT][4 warps]
    float* mine = wmax + wg * RT * 4;
    float* facs = reinterpret_cast<float*>(smem + L::kFacOff);    // [4][RT]: what the last rescaling took of l
    float* facs_o = facs + (E4 ? 4 * kTreeRT : 0);                // ... and of O
    float* peaks = facs_o + 4 * kTreeRT;                          // [4][RT] of rows with gains (e4m3)
    // After a wait that ran out the warps go on without waiting, through the
    // same barriers, so that no thread is left at one.
    bool ok = true;
    uint32_t it = 0, u = 0;
    auto wait = [&](uint32_t b, uint32_t phase) {
      if (ok) ok = mbar_wait(b, phase, ctl);
      ok = __all_sync(~0u, ok);
    };
    auto values_done = [&](uint32_t j) {  // P V of tile j has been added to O
      wait(pv_done(j % NB), (j / NB) & 1);
      tc_fence_after();
    };
    while (walk.next(a)) {
      const TreeSeq& s = walk.s;
      const uint32_t t_all = tmem + lanes + L::kOCol + (u & 1) * TN * L::kN;  // the piece's O
      const uint32_t t_o = t_all + turn * L::kN + row0;                       // this warpgroup's
      float* refs = reinterpret_cast<float*>(smem + L::kRefOff) + (u & 1) * 4 * RT;  // [4][RT]
      float* sums = reinterpret_cast<float*>(smem + L::kSumOff) + (u & 1) * 16 * RT; // [4][RT][4 warps]
      float* gains = reinterpret_cast<float*>(smem + L::kGainOff) + (u & 1) * 4 * RT; // [4][RT] (e4m3)
      if (u == 0) {
        TreeRows* first = reinterpret_cast<TreeRows*>(smem + L::kRowsOff);
        tree_load_queries<D, FMT, R, BIAS>(a, walk, warp, kTreeSoftWarps, lane, smem + L::kQOff, first);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(0));  // S can begin
        tree_load_rows<R, BIAS>(a, walk, warp, kTreeSoftWarps, lane, first,
                                reinterpret_cast<float*>(smem + L::kT5Off));
        named_barrier(kTreeBarAll, kTreeSoftWarps * 32);
      } else {
        wait(q_full(u & 1), (u >> 1) & 1);
      }
      // (after an abort: the first buffer, which has been filled and holds
      // addresses of this call)
      const TreeRows* info =
          reinterpret_cast<const TreeRows*>(smem + L::kRowsOff + (ok ? (u & 1) * L::kRowsBytes : 0));
      float ref[RT], l[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        ref[j] = -FLT_MAX;
        l[j] = 0.f;
      }
      bool fresh = true;  // no tile of the piece in this warpgroup's O yet
      bool gained = false;  // some row's gain is not 1 (e4m3)
      // e4m3: the scales of this thread's key, read one tile ahead: its page
      // at the tile's start, the bytes at its end
      uint32_t k_byte = 127, v_byte = 127;
      int page = -1;
      auto find_page = [&](int i) {
        const int pos = (s.tile0 + walk.t0 + i) * kTreeKeys + me;
        page = -1;
        if (i < walk.nt && pos < s.keys)
          page = a.table[static_cast<int64_t>(walk.b) * a.table_b + (pos >> a.page_shift)];
      };
      auto find_scales = [&](int i) {
        const int pos = (s.tile0 + walk.t0 + i) * kTreeKeys + me;
        if (page >= 0 && page < a.num_pages) {
          const int64_t at = page * a.ss_page + walk.hkv * a.ss_head + (pos & (a.page_size - 1));
          k_byte = a.ks[at];
          v_byte = a.vs[at];
        } else {
          k_byte = v_byte = 127;
        }
      };
      if constexpr (E4) {
        const int i = static_cast<int>((turn - it) & (TN - 1));  // its first tile
        find_page(i);
        find_scales(i);
      }
      for (int i = 0; i < walk.nt; ++i, ++it) {
        if (it % TN != turn) continue;
        const uint32_t x = it % NB;
        const int key0 = (s.tile0 + walk.t0 + i) * kTreeKeys;
        const int key = key0 + me;
        if constexpr (E4) find_page(i + TN);
        wait(s_full(x), (it / NB) & 1);
        tc_fence_after();
        float sc[RT];
        if constexpr (E4) {
          float rest[RT];
          if constexpr (RT == 8) {
            float both[16];
            tmem_ld_cols<16>(tmem + lanes + x * L::kN, both);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
              sc[j] = both[j];
              rest[j] = both[RT + j];
            }
          } else {
            tmem_ld_two(tmem + lanes + x * L::kN + row0, tmem + lanes + x * L::kN + R + row0, sc, rest);
          }
          fma_rows<RT>(rest, 1.f / kQueryRest, sc);
        } else {
          tmem_ld_cols<RT>(tmem + lanes + x * L::kN + row0, sc);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free(x));

        // scores in log2 units
        float e = 0.f;  // exponent of the key's value scale
        if constexpr (E4) {
          const float kf = e8m0_float(k_byte);
          e = fmaxf(static_cast<float>(static_cast<int>(v_byte) - 127), kLeastE);
          const uint64_t kf2 = f2_pack(kf, kf);
#pragma unroll
          for (int j = 0; j < RT; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(info->scale + row0 + j);
            // the row's factor and the key's first: either with the sum of codes could leave float32
            f2_unpack(f2_mul(f2_pack(sc[j], sc[j + 1]), f2_mul(f2_pack(f.x, f.y), kf2)), sc[j], sc[j + 1]);
            f2_unpack(f2_mul(f2_pack(sc[j + 2], sc[j + 3]), f2_mul(f2_pack(f.z, f.w), kf2)), sc[j + 2], sc[j + 3]);
          }
        } else {
          const uint64_t f2 = f2_pack(a.scale_log2, a.scale_log2);
#pragma unroll
          for (int j = 0; j < RT; j += 2) f2_unpack(f2_mul(f2_pack(sc[j], sc[j + 1]), f2), sc[j], sc[j + 1]);
        }
        // all keys of the tile seen by every row: context keys inside every
        // node's window (a node's position is below ctx + n)
        const bool masked = key0 + kTreeKeys > s.ctx || (a.wl >= 0 && key0 < s.ctx + s.n - 1 - a.wl);
        const int node = key - s.ctx;
        const int key_pos = node >= 0 ? s.ctx + (node < s.n ? info->depth[node] : 0) : key;
        bool hidden = false;  // from some row
        if constexpr (BIAS != 0) {
          if (a.alibi_slopes) {
#pragma unroll
            for (int j = 0; j < RT; ++j)
              sc[j] += bias_to_log2(-info->bias[row0 + j] *
                                    fabsf(static_cast<float>(key_pos - info->pos[row0 + j])));
          } else if (!ok) {
            // (after an abort the rows may be another piece's: no lookups by them)
          } else if (key0 + kTreeKeys - 1 - s.ctx <= a.t5.one_lo_max) {
            // every distance of the tile in the last bucket
#pragma unroll
            for (int j = 0; j < RT; ++j) sc[j] += info->bias[row0 + j];
          } else {
            const uint8_t* buckets = smem + L::kBucketOff;
            const float* slice = reinterpret_cast<const float*>(smem + L::kT5Off) + (u & 1) * kTreeT5Slice;
            const int head0 = walk.hkv * a.G;
            if (a.t5_buckets * a.G <= kTreeT5Slice && a.t5.one_lo_max >= -kTreeNear) {
              // eight lookups in flight, without a branch between them
#pragma unroll
              for (int j0 = 0; j0 < RT; j0 += 8) {
                int at[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  at[j] = buckets[min(max(key_pos - info->pos[row0 + j0 + j], -kTreeNear), 63) + kTreeNear];
#pragma unroll
                for (int j = 0; j < 8; ++j) sc[j0 + j] += slice[at[j] * a.G + info->head[row0 + j0 + j] - head0];
              }
            } else {
              // a table too large for the slice, or buckets beyond the tabulated distances
#pragma unroll
              for (int j = 0; j < RT; ++j) {
                const int rel = key_pos - info->pos[row0 + j];
                const int k = rel < -kTreeNear ? t5_bucket(rel, a.t5) : buckets[min(rel, 63) + kTreeNear];
                sc[j] += bias_to_log2(a.t5_table[k * a.Hq + info->head[row0 + j]]);
              }
            }
          }
        }
        if (masked) {
          uint32_t seen = node < 0 ? ~0u : node < s.n ? info->seen[node][row0 / 32] >> (row0 % 32) : 0u;
          if (a.wl >= 0) {
#pragma unroll
            for (int j = 0; j < RT; ++j)
              if (info->pos[row0 + j] - key_pos > a.wl) seen &= ~(1u << j);
          }
          constexpr uint32_t kRows = (1u << RT) - 1u;
          hidden = (seen & kRows) != kRows;
#pragma unroll
          for (int j = 0; j < RT; ++j)
            if (!((seen >> j) & 1u)) sc[j] = -INFINITY;
        }

        // the weight buffer is free, and with turns this warpgroup's O at rest
        if (it >= NB) values_done(it - NB);
        // a new reference where a score has outgrown the old one
        float over = -INFINITY;
#pragma unroll
        for (int j = 0; j < RT; j += 2) {
          float d0, d1;
          f2_unpack(f2_sub(f2_pack(sc[j], sc[j + 1]), f2_pack(ref[j], ref[j + 1])), d0, d1);
          over = fmax3(over, d0, d1);
        }
        if (barrier_or(1 + wg, 128, over + e > (E4 ? kOverE4m3 : kOverBf16) || fresh || gained ||
                                        (E4 && v_byte < 127 + static_cast<int>(kLeastE)))) {
          const bool scribe = (warp & 3) == 0 && lane < RT;  // keeps row `lane`'s reference
          const int at = wg * RT + lane;
          auto rows_top = [&](const float (&y)[RT]) {  // for the scribes: their row's largest, less kTop
            const float of_row = by_halves<RT>(y, lane, [](float x, float z) { return fmaxf(x, z); });
            if ((lane & (32 / RT - 1)) == 0) mine[(lane / (32 / RT)) * 4 + (warp & 3)] = of_row;
            named_barrier(1 + wg, 128);
            const float4 w4 = *reinterpret_cast<const float4*>(mine + lane % RT * 4);
            return fmaxf(fmaxf(w4.x, w4.y), fmaxf(w4.z, w4.w)) - (E4 ? kTopE4m3 : kTopBf16);
          };
          float in = fminf(e, kMostE), true_e = static_cast<float>(static_cast<int>(v_byte) - 127);
          if constexpr (E4) {
            // a value row of zeros raises r no more than l needs: its weight in
            // P V does not matter.  It is stored with a scale of 1 (byte 127);
            // rows are looked at where one could be far above its neighbours
            const bool there = key < s.keys;
            const uint32_t hi = __reduce_max_sync(~0u, there ? v_byte : 0u);
            const uint32_t lo = __reduce_min_sync(~0u, there ? v_byte : 255u);
            if (__builtin_expect(hi >= 127u || hi > lo + 4u, 0)) {
              const uint32_t item = 2 * it + 1;
              wait(full(item % NS), (item / NS) & 1);
              if (tree_row_of_zeros<L>(smem + slot_off(item), me)) {
                in = kLeastE;
                true_e = -INFINITY;
              }
            }
          }
          float top[RT];
#pragma unroll
          for (int j = 0; j < RT; j += 2) {
            if constexpr (E4) f2_unpack(f2_add(f2_pack(sc[j], sc[j + 1]), f2_pack(in, in)), top[j], top[j + 1]);
            else { top[j] = sc[j]; top[j + 1] = sc[j + 1]; }
          }
          const float m = rows_top(top);
          bool wide = E4 && (gained || (true_e < kLeastE && true_e > -INFINITY) || true_e > kMostE);  // gains have to be looked at
          if (scribe) {
            const float old = fresh ? -FLT_MAX : refs[at];
            const float r = fmaxf(m, old);
            refs[at] = r;
            facs[at] = fast_exp2(old - r);
            if constexpr (E4) {
              facs_o[at] = fast_exp2(old - r);
              if (fresh) gains[at] = 1.f;
              wide |= fabsf(r) >= kManyDigits && m > -INFINITY;
            }
          }
          if (TN < NB && !fresh) values_done(it - TN);
          if constexpr (E4) {
            if (barrier_or(1 + wg, 128, wide)) {
              float cold[RT];
#pragma unroll
              for (int j = 0; j < RT; ++j) cold[j] = sc[j];
              gained = tree_renew_gains<RT>(cold, true_e, gained, refs, gains, facs, facs_o, peaks, mine, wg, warp, lane);
            }
          } else {
            named_barrier(1 + wg, 128);
          }
#pragma unroll
          for (int j = 0; j < RT; j += 4) {
            const float4 r4 = *reinterpret_cast<const float4*>(refs + wg * RT + j);
            const float4 f4 = *reinterpret_cast<const float4*>(facs + wg * RT + j);
            ref[j] = r4.x;
            ref[j + 1] = r4.y;
            ref[j + 2] = r4.z;
            ref[j + 3] = r4.w;
            f2_unpack(f2_mul(f2_pack(l[j], l[j + 1]), f2_pack(f4.x, f4.y)), l[j], l[j + 1]);
            f2_unpack(f2_mul(f2_pack(l[j + 2], l[j + 3]), f2_pack(f4.z, f4.w)), l[j + 2], l[j + 3]);
          }
          if (!fresh) {
#pragma unroll 1
            for (int j0 = 0; j0 < RT * L::kParts; j0 += 8) {
              const uint32_t t = t_o + (j0 < RT ? j0 : R + j0 - RT);
              const float* f = facs_o + wg * RT + (j0 < RT ? j0 : j0 - RT);
              float o[8];
              tmem_ld_cols<8>(t, o);
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] *= f[j];
              tmem_st_cols<8>(t, o);
            }
          }
        }

        uint8_t* pbuf = smem + L::kPOff + x * L::kPBytes + me * 16;
        const float v_up = e8m0_float(min(v_byte, 254u));  // (finite, also of a hidden row that holds anything)
        const uint64_t up2 = f2_pack(v_up, v_up);
#pragma unroll
        for (int j = 0; j < RT; j += 2) {
          f2_unpack(f2_sub(f2_pack(sc[j], sc[j + 1]), f2_pack(ref[j], ref[j + 1])), sc[j], sc[j + 1]);
          sc[j] = fast_exp2(sc[j]);
          sc[j + 1] = fast_exp2(sc[j + 1]);
          const uint64_t p2 = f2_pack(sc[j], sc[j + 1]);
          f2_unpack(f2_add(p2, f2_pack(l[j], l[j + 1])), l[j], l[j + 1]);
          if constexpr (E4) f2_unpack(f2_mul(p2, up2), sc[j], sc[j + 1]);
        }
        if (E4 && __builtin_expect(gained, 0)) {
#pragma unroll
          for (int j = 0; j < RT; ++j) sc[j] *= gains[wg * RT + j];
        }
        // the weights: 16 bytes of one key's rows at a time
        if constexpr (E4) {
          uint32_t hi[RT / 4], lo[RT / 4];
          // van der Corput's sequence over the keys: 2^-9 is e4m3's last step
          const __half2 d = __float2half2_rn(static_cast<float>(static_cast<int>(__brev(key))) * 0x1p-41f);
#pragma unroll
          for (int j = 0; j < RT; j += 4) {
            const uint32_t h0 = e4m3x2(sc[j], sc[j + 1]), h1 = e4m3x2(sc[j + 2], sc[j + 3]);
            hi[j / 4] = h0 | h1 << 16;
            lo[j / 4] = e4m3x2_rest(sc[j], sc[j + 1], h0, d) | e4m3x2_rest(sc[j + 2], sc[j + 3], h1, d) << 16;
          }
          if constexpr (RT == 8) *reinterpret_cast<uint4*>(pbuf) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint32_t* w = part ? lo : hi;
#pragma unroll
            for (int j = 0; j + 4 <= RT / 4; j += 4)
              *reinterpret_cast<uint4*>(pbuf + ((part * R + row0) / 16 + j / 4) * (kTreeKeys * 16)) =
                  make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < RT; j += 8)
            *reinterpret_cast<uint4*>(pbuf + ((row0 + j) / 8) * (kTreeKeys * 16)) =
                make_uint4(pack_bf16x2(sc[j], sc[j + 1]), pack_bf16x2(sc[j + 2], sc[j + 3]),
                           pack_bf16x2(sc[j + 4], sc[j + 5]), pack_bf16x2(sc[j + 6], sc[j + 7]));
        }
        if constexpr (E4) find_scales(i + TN);
        bool mend = false;
        float missing[RT];  // what the rows of this thread miss in its column of O
        if (masked) {
          // 0 * NaN is NaN: rows behind the sequence's end are zeroed (they hold
          // anything), and an infinite or NaN value of a key hidden from some
          // row is taken out of the tile and added to the rows that do see it
          // once P V of the tile is in O
          constexpr int kPieces = L::kRowBytes / 16;
          const uint32_t item = 2 * it + 1;
          uint8_t* vrows = smem + slot_off(item);
          wait(full(item % NS), (item / NS) & 1);
          uint32_t odd = 0;
          if (key >= s.keys) {
            if (row0 == 0) {
#pragma unroll 4
              for (int c = 0; c < kPieces; ++c)
                *reinterpret_cast<uint4*>(vrows + L::at(me, c, kTreeKeys)) = make_uint4(0, 0, 0, 0);
            }
          } else if (hidden) {
#pragma unroll 4
            for (int c = 0; c < kPieces; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(vrows + L::at(me, c, kTreeKeys));
              odd |= nonfinite_bits<FMT>(w.x) | nonfinite_bits<FMT>(w.y) | nonfinite_bits<FMT>(w.z) |
                     nonfinite_bits<FMT>(w.w);
            }
          }
          mend = barrier_or(b_tile, kTileThreads, odd != 0);
          if (mend) {
            tree_take_out<D, FMT, R, BIAS>(a.wl, s.ctx, key0, info, vrows, smem + L::kPOff + x * L::kPBytes,
                                           dirty + turn * 4, odd, b_tile, row0, warp, lane, missing);
          }
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x));
        fresh = false;
        if (mend) {
          values_done(it);
#pragma unroll 1
          for (int j0 = 0; j0 < RT; j0 += 8) {
            float o[8];
            tmem_ld_cols<8>(t_o + j0, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += missing[j0 + j];
            tmem_st_cols<8>(t_o + j0, o);
          }
          tc_fence_before();
        }
      }

      // ---- the piece's result: row sums over the warpgroup's keys, then O
      const float total = by_halves<RT>(l, lane, [](float x, float y) { return x + y; });
      if ((lane & (32 / RT - 1)) == 0) sums[(wg * RT + lane / (32 / RT)) * 4 + (warp & 3)] = total;
      // the last P V of this warpgroup's O
      if (!fresh) values_done(it - 1 - ((it - 1 - turn) & (TN - 1)));
      constexpr uint32_t kMeet = TN == 1 ? 128 : kTreeSoftWarps * 32;  // threads whose results meet
      const uint32_t b_meet = TN == 1 ? 1 + wg : kTreeBarAll;
      tc_fence_before();
      named_barrier(b_meet, kMeet);
      tc_fence_after();

      const bool whole = walk.t0 == 0 && walk.nt == s.tiles;
      const int slot = walk.t0 == 0 ? 1 : 0;  // 0: began in an earlier CTA
      // first row that this thread writes; at 16 rows two warpgroups do, at 8
      // one does, in turn
      const int out0 = (R == 8 ? (wg + u) & 3 : R == 16 ? wg ^ ((u & 1) << 1) : wg) * RO;
      const int n_rows = min(R, s.n * a.G - walk.block * R) - out0;  // from there on, may exceed RO
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * R + out0;
      const int sets = min(walk.nt, TN);      // that had tiles, from the first tile's on
      // (rolled: straight-line code that runs once per piece would wait for
      // its instructions longer than it runs)
#pragma unroll 1
      for (int j0 = 0; ok && j0 < min(RO, n_rows); j0 += 8) {
        const int row = out0 + j0;
        float o[8], sum[8], rr[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = sum[j] = 0.f;
          rr[j] = -FLT_MAX;
        }
#pragma unroll 1
        for (int k = 0; k < sets; ++k) {
          const int t = (it - walk.nt + k) & (TN - 1);
          const int at = (t * RG + row / RT) * RT + row % RT;  // in the warpgroups' arrays
          float o2[8];
          tmem_ld_cols<8>(t_all + t * L::kN + row, o2);
          if constexpr (E4) {
            float rest[8];
            tmem_ld_cols<8>(t_all + t * L::kN + R + row, rest);
            fma_rows<8>(rest, 1.f / kWeightRest, o2);
#pragma unroll
            for (int j = 0; j < 8; ++j) o2[j] *= fast_rcp(gains[at + j]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 l4 = *reinterpret_cast<const float4*>(sums + (at + j) * 4);
            const float r2 = refs[at + j];
            const float top = fmaxf(rr[j], r2);
            const float f1 = fast_exp2(rr[j] - top), f2 = fast_exp2(r2 - top);
            o[j] = o[j] * f1 + o2[j] * f2;
            sum[j] = sum[j] * f1 + ((l4.x + l4.y) + (l4.z + l4.w)) * f2;
            rr[j] = top;
          }
        }
        // one logarithm a thread, of row + me (eight in line cost 1000 sequences a
        // fifth of their time in instruction fetches: 502 us, 402)
        float my_r = 0.f, my_sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (whole) o[j] *= sum[j] > 0.f || isnan(sum[j]) ? 1.f / sum[j] : 0.f;
          if (me == j) {
            my_r = rr[j];
            my_sum = sum[j];
          }
        }
        if (me < 8 && j0 + me < n_rows) {
          if (whole) a.lse[info->lse[row + me]] = tree_lse(my_r, my_sum);
          else a.part_ml[part + j0 + me] = make_float2(my_r, my_sum);
        }
        if (me < D) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            if (whole) {
              // lane pairs trade: the even lane stores two columns of row j,
              // the odd lane of row j + 1
              const bool up = lane & 1;
              const float got = __shfl_xor_sync(~0u, up ? o[j] : o[j + 1], 1);
              if (j0 + j + (up ? 1 : 0) < n_rows)
                *reinterpret_cast<uint32_t*>(a.o + info->out[row + j + (up ? 1 : 0)] + (me & ~1)) =
                    up ? pack_bf16x2(got, o[j + 1]) : pack_bf16x2(o[j], got);
            } else {
              if (j0 + j < n_rows) a.part_o[(part + j0 + j) * D + me] = o[j];
              if (j0 + j + 1 < n_rows) a.part_o[(part + j0 + j + 1) * D + me] = o[j + 1];
            }
          }
        }
      }
      // (the sums, references and O of this piece are written again two pieces
      // on, after the meeting at the next one's end)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_free(u & 1));
      ++u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTreeIssueS) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// One warp joins the pieces of query row `in` of a (sequence, head, row block)
// that CTAs c0 .. c1 have parts of, in their order.  The lanes first weigh up
// to 32 pieces at once, then add them, D / 32 columns each.
template <int D, int R, int U>
__device__ __forceinline__ void tree_join_row(const TreeArgs& a, int lane, int c0, int c1, int in, int row, int h) {
  constexpr int W = D / 32;
  float ref = -FLT_MAX, l = 0.f, acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.f;
  for (int base = c0; base <= c1; base += 32) {
    const int cta = base + lane;
    // the first CTA's piece began in it, every later one's before it
    float2 ml = make_float2(-FLT_MAX, 0.f);
    if (cta <= c1) ml = a.part_ml[(static_cast<int64_t>(cta) * 2 + (cta == c0 ? 1 : 0)) * R + in];
    const float top = fmaxf(warp_max(ml.x), ref);
    const float f_old = fast_exp2(ref - top);
    const float f = fast_exp2(ml.x - top);
    float add = ml.y * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(~0u, add, o);
    l = l * f_old + add;
    ref = top;
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] *= f_old;
    const int count = min(32, c1 - base + 1);
#pragma unroll U
    for (int j = 0; j < count; ++j) {
      const int cj = base + j;
      const float w = __shfl_sync(~0u, f, j);
      const float* src = a.part_o + ((static_cast<int64_t>(cj) * 2 + (cj == c0 ? 1 : 0)) * R + in) * D + lane * W;
      if constexpr (W == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] += w * v.x;
        acc[1] += w * v.y;
        acc[2] += w * v.z;
        acc[3] += w * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] += w * v.x;
        acc[1] += w * v.y;
      }
    }
  }
  const float inv = l > 0.f || isnan(l) ? 1.f / l : 0.f;
  __nv_bfloat16* dst = a.o + static_cast<int64_t>(row) * a.o_t + static_cast<int64_t>(h) * a.o_h + lane * W;
  if constexpr (W == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) a.lse[static_cast<int64_t>(h) * a.T + row] = tree_lse(ref, l);
}

// Up to 32 sequences: a warp per (node, head), which finds where its piece of
// the line lies.
constexpr int kTreeJoinWarps = 4;

template <int D, int R>
__global__ void __launch_bounds__(kTreeJoinWarps * 32) tree_join_kernel(const __grid_constant__ TreeArgs a,
                                                                       int ctas) {
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int x = blockIdx.x * kTreeJoinWarps + (threadIdx.x >> 5);  // node * Hq + head
  // all that the lengths decide, while the pieces are still being computed
  const TreeSeq s = tree_seq<R>(a, b);
  int tiles = 0, pieces = 0;
  if (lane < a.B) {
    const TreeSeq other = tree_seq<R>(a, lane);
    tiles = other.units(a.Hkv, 0);
    pieces = other.rb * a.Hkv;
  }
  const int tiles_before = __reduce_add_sync(~0u, lane < b ? tiles : 0);
  const int pieces_before = __reduce_add_sync(~0u, lane < b ? pieces : 0);
  tiles = __reduce_add_sync(~0u, tiles);
  pieces = __reduce_add_sync(~0u, pieces);
  const int n = x / a.Hq, h = x - n * a.Hq;
  const int hkv = h / a.G;
  const int r = n * a.G + (h - hkv * a.G);
  const int block = r / R, in = r - block * R;
  int c0 = 0, c1 = 0;
  if (n < s.n) {
    const int cost = tree_piece_cost(tiles, ctas);
    const int per = tree_share(tiles + cost * pieces, ctas);
    const int first = tiles_before + cost * pieces_before + (hkv * s.rb + block) * (cost + s.tiles) + cost;
    c0 = first / per;
    c1 = (first + s.tiles - 1) / per;
  }
  // (every thread waits, so that what follows this kernel follows the first too)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 != c1) tree_join_row<D, R, 16>(a, lane, c0, c1, in, s.row0 + n, h);
}

// More sequences: most of their pieces lie inside one CTA's part of the line,
// and each warp of the form above would go through all lengths for nothing.
// Here blockIdx.y + 1 names a CTA; if its part begins inside a piece that began
// in the CTA before, that piece is joined, a warp per query row.  The form above
// ends at the 32 sequences that one warp's lanes hold; a loop over more of them in
// each warp, with the search of the lengths in one warp, against this, when it
// came: 1000 sequences of 1 node over 500 keys 633 -> 578 us, 256 of 8 nodes over
// 1000 keys 255 -> 217, 256 of 1 node 193 -> 195, 64 of 1 node 64 -> 67: one form
// for all that are more, though up to some 256 single nodes it gains nothing.
// (32 registers and no more: a block has to find room beside the first
// kernel's, to be waiting when it ends.)
constexpr int kTreeCutWarps = 4;

template <int D, int R>
__global__ void __launch_bounds__(kTreeCutWarps * 32, 16) tree_join_cuts_kernel(const __grid_constant__ TreeArgs a,
                                                                           int ctas) {
  __shared__ int totals[2 * kTreeCutWarps];
  __shared__ TreeSpot spot;
  const int cut = blockIdx.y + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int in = blockIdx.x * kTreeCutWarps + warp;  // row of the block
  tree_locate_many<R, kTreeCutWarps>(a, cut, ctas, warp, lane, totals, &spot);
  __syncthreads();
  int c0 = 0, c1 = 0, row = 0, h = 0;
  if (spot.left > 0) {
    const TreeSeq& s = spot.s;
    const int span = spot.cost + s.tiles;
    const int seg = spot.off / span;
    const int done = spot.off - seg * span - spot.cost;  // its tiles before the cut
    const int hkv = seg / s.rb;
    const int r = (seg - hkv * s.rb) * R + in;
    if (done > 0 && done <= spot.per && r < s.n * a.G) {  // begun in CTA cut - 1
      c0 = cut - 1;
      c1 = cut + (s.tiles - done - 1) / spot.per;
      row = s.row0 + r / a.G;
      h = hkv * a.G + r % a.G;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 != c1) tree_join_row<D, R, 4>(a, lane, c0, c1, in, row, h);
}

}  // namespace sdpa
