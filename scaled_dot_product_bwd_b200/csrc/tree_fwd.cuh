// tree_fwd.cuh -- attention of drafted nodes (one: plain decoding) over a
// paged bf16 or e4m3 cache.
//
// Mathematics.  The nodes of a sequence times the query heads of a KV head's
// group are the rows of one score matrix against that head's keys, so every
// cached byte is read once for all of them.  Per row an online softmax in
// log2 units: running maximum m, sum l of 2^(s - m) and accumulator O.  An
// e4m3 key's scale multiplies its score column.  A value row's scale 2^e
// joins the exponent instead of the values: weights are 2^(s + e - m') with m'
// the maximum of s + e, so they lie in [0, 1] whatever the scales are and
// round to fp16 with 11 bits, and l adds weight * 2^-e.
//
// Bound by DRAM: at up to 16 rows per KV head a cached byte takes 8 to 32
// FLOPs.  What costs is keeping enough loads in flight and every SM busy:
//  * work is cut into tiles of one KV head's keys, laid out over all sequences
//    and heads in one line, and the CTAs (two per SM) take equal pieces of the
//    line, so ragged batches balance and one long sequence uses the whole GPU;
//    a (sequence, head) that spans CTAs leaves partial (m, l, O) in the
//    workspace and a second kernel joins them in order;
//  * a producer warp copies tiles by TMA (one box per page piece) into a ring
//    of 96 KB per CTA; four compute warps each take a quarter of a tile's keys
//    with all rows, so a stored value is read from shared memory and converted
//    by one warp only, and the warps meet only where a piece ends;
//  * the products are mma.sync m16n8k16: with 16 rows a 128-row tcgen05 tile
//    would be idle seven eighths of its rows.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "kv_cache.cuh"
#include "sm100.cuh"

namespace sdpa {

constexpr int kTreeMaxCtas = 296;   // two per SM; the workspace is sized for it
constexpr int kTreeMaxNodes = 64;
constexpr int kTreeKeyWarps = 4;
constexpr int kTreeThreads = (kTreeKeyWarps + 1) * 32;

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
  // workspace
  int64_t* prefix;              // [B + 1] tiles before each sequence
  float2* part_ml;              // [ctas][2][rows] (m, l)
  float* part_o;                // [ctas][2][rows][D]
  uint64_t wait_limit_ns;
};

// Shapes of a tile of keys in shared memory.
template <int D, int FMT>
struct TreeTile {
  static constexpr int kCell = FMT == kCacheBf16 ? 2 : 1;
  static constexpr int kRowBytes = D * kCell;                          // 64, 128 or 256
  static constexpr int kHalves = kRowBytes == 256 ? 2 : 1;             // 128-byte columns
  static constexpr int kLine = kRowBytes / kHalves;                    // bytes of a box row
  static constexpr int kKeys = kRowBytes == 256 ? 64 : 128;            // keys per tile
  static constexpr int kBytes = kKeys * kRowBytes;                     // of K, and of V
  static constexpr int kStage = 2 * kBytes + 1024;                     // + scales of 128 keys each
  static constexpr int kStages = kBytes == 16384 ? 3 : 6;
  static constexpr int kWarpKeys = kKeys / kTreeKeyWarps;              // 16 or 32
  // byte offset of 16-byte piece `c` of row `r`, as TMA's swizzle places it
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if (kLine == 128)
      return static_cast<uint32_t>((c >> 3) * kKeys * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
};

// What one sequence needs of a kernel, from its entries in cu_nodes and ctx_lens.
struct TreeSeq {
  int row0, n, ctx, keys;  // first query row, nodes, context length, context + nodes
  int tile0, tiles, rb;    // first key tile any node sees, tiles, row blocks
  __device__ __forceinline__ int units(int Hkv) const { return Hkv * rb * tiles; }
};

template <int KEYS, int ROWS>
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
  s.tile0 = a.wl >= 0 ? max(0, s.ctx - a.wl) / KEYS : 0;
  s.tiles = (s.keys + KEYS - 1) / KEYS - s.tile0;
  s.rb = (s.n * a.G + ROWS - 1) / ROWS;
  if (s.n == 0) s.tiles = s.rb = 0;
  return s;
}

// One CTA's piece [u, end) of the line of tiles; next() gives it (sequence,
// head, row block) by (sequence, head, row block).
template <int KEYS, int ROWS>
struct TreeWalk {
  int64_t u, end;
  int b, off, units;  // current sequence, tiles of it behind u, its tiles
  TreeSeq s;
  int hkv, block, t0, nt;  // this step: head, row block, first tile, tiles
  __device__ __forceinline__ void start(const TreeArgs& a, int64_t from, int64_t to, int b0,
                                        int off0) {
    u = from;
    end = to;
    b = b0;
    off = off0;
    if (u < end) {
      s = tree_seq<KEYS, ROWS>(a, b);
      units = s.units(a.Hkv);
    }
  }
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if (u >= end) return false;
    while (off >= units) {
      off -= units;
      s = tree_seq<KEYS, ROWS>(a, ++b);
      units = s.units(a.Hkv);
    }
    const int seg = off / s.tiles;
    t0 = off - seg * s.tiles;
    hkv = seg / s.rb;
    block = seg - hkv * s.rb;
    nt = static_cast<int>(min(static_cast<int64_t>(s.tiles - t0), end - u));
    u += nt;
    off += nt;
    return true;
  }
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d += a * b, 16 x 8 x 16, bf16 or fp16 operands.
template <int FMT>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if (FMT == kCacheBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes (low 16 bits) as an fp16 pair: exact.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// All bits of the codes / bf16 halves in w that are infinite or NaN.
template <int FMT>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  return FMT == kCacheBf16 ? __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u)
                           : __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// b * log2(e) of a bias b, kept finite where b is: a bias of the type's lowest
// value then still orders below every other score instead of hiding its key.
__device__ __forceinline__ float bias_to_log2(float b) {
  const float x = b * kLog2e;
  return isinf(x) && !isinf(b) ? copysignf(3.402823466e38f, b) : x;
}

__device__ __forceinline__ float t5_bias_log2(const TreeArgs& a, int rel, int h) {
  return bias_to_log2(a.t5_table[t5_bucket(rel, a.t5) * a.Hq + h]);
}

// The d index of accumulator element e (0, 1) of n-tile j for quad column c:
// with e4m3 the two n-tiles of a 16-wide group hold its even and odd columns
// (a transposed load moves pairs of codes).
template <int FMT>
__device__ __forceinline__ int acc_col(int j, int c, int e) {
  return FMT == kCacheBf16 ? j * 8 + 2 * c + e : (j >> 1) * 16 + 4 * c + 2 * e + (j & 1);
}

// Per-thread state of the two rows (lane / 4 and + 8) of a 16-row tile.
struct TreeRow {
  uint64_t sees;  // nodes it sees
  int pos;        // its position
  int head;       // its query head
  float bias;     // ALiBi: its slope; T5: the bias of every distance <= one_lo_max
};

template <int D, int FMT, int BIAS>
__global__ void __launch_bounds__(kTreeThreads, 2) tree_fwd_kernel(
    const TreeArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Tile = TreeTile<D, FMT>;
  constexpr int ROWS = 16;
  constexpr int KEYS = Tile::kKeys;
  constexpr int WK = Tile::kWarpKeys;
  constexpr int NT = WK / 8;    // score n-tiles per warp
  constexpr int DT = D / 8;     // output n-tiles
  constexpr int KS = D / 16;    // k-steps over d
  constexpr int kPad = D + 4;   // merge buffer row, floats
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * Tile::kStages];
  __shared__ int abort_flag;
  __shared__ int start_b, start_off;
  __shared__ int64_t total_sh;
  __shared__ int64_t scan_sh[kTreeThreads / 32];
  __shared__ float2 merge_ml[kTreeKeyWarps][ROWS];
  if (!smem_base_ok(smem)) {
    if (threadIdx.x == 0) atomicOr(&g_device_status, kStatusMisaligned);
    return;
  }
  float* merge_o = reinterpret_cast<float*>(smem + Tile::kStages * Tile::kStage);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (Tile::kStages + s); };
  if (tid == 0) {
    abort_flag = 0;
    start_b = -1;
    for (int s = 0; s < Tile::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kTreeKeyWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }

  // the line of tiles: its length, and where this CTA's piece begins
  int64_t mine = 0;
  for (int b = tid; b < a.B; b += kTreeThreads) mine += tree_seq<KEYS, ROWS>(a, b).units(a.Hkv);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) mine += __shfl_xor_sync(~0u, mine, s);
  if (lane == 0) scan_sh[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    int64_t total = 0;
    for (int w = 0; w < kTreeThreads / 32; ++w) total += scan_sh[w];
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    const int64_t from = per * blockIdx.x;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t units = b < a.B ? tree_seq<KEYS, ROWS>(a, b).units(a.Hkv) : 0;
      int64_t upto = units;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, upto, s);
        if (lane >= s) upto += y;
      }
      const int64_t before = base + upto - units;
      if (blockIdx.x == 0 && b < a.B) a.prefix[b] = before;
      if (b < a.B && before <= from && from < before + units) {
        start_b = b;
        start_off = static_cast<int>(from - before);
      }
      base += __shfl_sync(~0u, upto, 31);
    }
    if (lane == 0) {
      total_sh = total;
      if (blockIdx.x == 0) a.prefix[a.B] = total;
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t total = total_sh;
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  const int64_t from = per * blockIdx.x;
  const int64_t to = min(total, from + per);
  TreeWalk<KEYS, ROWS> walk;
  walk.start(a, from, start_b < 0 ? from : to, max(start_b, 0), start_b < 0 ? 0 : start_off);
  const WaitCtl ctl{&abort_flag, a.wait_limit_ns};

  if (warp == kTreeKeyWarps) {
    // ------------------------------------------------------------ producer
    const int boxes = KEYS / a.box_rows;   // <= 8
    const uint32_t box_bytes = static_cast<uint32_t>(a.box_rows) * Tile::kRowBytes;
    uint32_t it = 0;
    bool ok = true;
    while (ok && walk.next(a)) {
      const int* row = a.table + static_cast<int64_t>(walk.b) * a.table_b;
      auto page_of = [&](int t) {
        const int pos = (walk.s.tile0 + t) * KEYS + lane * a.box_rows;
        int page = -1;
        if (lane < boxes && pos < walk.s.keys) {
          page = row[pos >> a.page_shift];
          if (page < 0 || page >= a.num_pages) {
            atomicOr(&g_device_status, kStatusBadSeqlens);
            page = static_cast<int>(a.num_pages);  // past the cache: the copy fills zeros
          }
        }
        return page;
      };
      int page = page_of(walk.t0);
      for (int i = 0; i < walk.nt; ++i, ++it) {
        const int t = walk.t0 + i;
        const int next_page = i + 1 < walk.nt ? page_of(t + 1) : -1;
        const int st = it % Tile::kStages;
        if (it >= Tile::kStages) ok = mbar_wait(empty(st), ((it / Tile::kStages) - 1) & 1, ctl);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const bool copy = page >= 0;
        const bool scales = FMT == kCacheE4m3 && copy && page < a.num_pages;
        const int n_copy = __popc(__ballot_sync(~0u, copy));
        const int n_scale = __popc(__ballot_sync(~0u, scales));
        const uint32_t base = smem_u32(smem) + st * Tile::kStage;
        if (lane == 0)
          mbar_expect_tx(full(st), 2u * (n_copy * box_bytes + n_scale * a.box_rows));
        __syncwarp();
        if (copy) {
          const int pos = (walk.s.tile0 + t) * KEYS + lane * a.box_rows;
          const int r = pos & (a.page_size - 1);
          const uint32_t dst = base + static_cast<uint32_t>(lane) * a.box_rows * Tile::kLine;
#pragma unroll
          for (int h = 0; h < Tile::kHalves; ++h) {
            tma_load_4d(dst + h * KEYS * 128, &mk, full(st), h * 64, r, walk.hkv, page);
            tma_load_4d(dst + Tile::kBytes + h * KEYS * 128, &mv, full(st), h * 64, r, walk.hkv, page);
          }
          if (scales) {
            const int64_t off = page * a.ss_page + walk.hkv * a.ss_head + r;
            const uint32_t sdst = base + 2 * Tile::kBytes + lane * a.box_rows;
            bulk_load(sdst, a.ks + off, a.box_rows, full(st));
            bulk_load(sdst + 512, a.vs + off, a.box_rows, full(st));
          }
        }
        page = next_page;
      }
    }
    // a wait that ran out ends the CTA: let the copies in flight land first
    if (!ok) {
      const uint64_t t_end = globaltimer_ns() + a.wait_limit_ns;
      const uint32_t first = it > Tile::kStages ? it - Tile::kStages : 0;
      for (uint32_t j = first; j < it; ++j)
        while (!mbar_try_wait(full(j % Tile::kStages), (j / Tile::kStages) & 1) &&
               globaltimer_ns() < t_end) {
        }
    }
    return;
  }

  // -------------------------------------------------------------- compute
  const int quad = lane >> 2, c = lane & 3;
  const int lm = lane >> 3, lr = lane & 7;  // ldmatrix: matrix and row this lane addresses
  uint32_t it = 0;
  bool alive = true;
  // After a wait that ran out the warps go on through the rest of the walk
  // without tiles, so that they still meet at every barrier.
  while (walk.next(a)) {
    const TreeSeq& s = walk.s;
    const int n_rows = s.n * a.G;
    const uint64_t node_bits = s.n >= 64 ? ~0ull : (1ull << s.n) - 1ull;
    auto sees_of = [&](int n) -> uint64_t {
      const uint64_t w = a.mask ? static_cast<uint64_t>(a.mask[s.row0 + n]) : ~0ull >> (63 - n);
      return w & node_bits;
    };
    TreeRow row[2];
    float row_scale[2];
    uint32_t qa[KS][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = walk.block * ROWS + quad + 8 * i;
      row[i].sees = 0;
      row[i].pos = s.ctx;
      row[i].head = walk.hkv * a.G;
      row[i].bias = 0.f;
      row_scale[i] = a.scale_log2;
#pragma unroll
      for (int k = 0; k < KS; ++k) qa[k][i] = qa[k][2 + i] = 0u;
      if (r < n_rows) {
        const int n = r / a.G, h = walk.hkv * a.G + (r - n * a.G);
        row[i].sees = sees_of(n);
        row[i].pos = s.ctx + __popcll(row[i].sees & ~(1ull << n));
        row[i].head = h;
        if (BIAS && a.alibi_slopes)
          row[i].bias = a.alibi_slopes[h];
        else if (BIAS && a.t5.one_lo_max != INT_MIN)
          row[i].bias = t5_bias_log2(a, a.t5.one_lo_max, h);
        const __nv_bfloat16* src = a.q + static_cast<int64_t>(s.row0 + n) * a.q_t + h * a.q_h;
        if (FMT == kCacheBf16) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qa[k][i] = *reinterpret_cast<const uint32_t*>(src + k * 16 + 2 * c);
            qa[k][2 + i] = *reinterpret_cast<const uint32_t*>(src + k * 16 + 8 + 2 * c);
          }
        } else {
          // k-slots 2c, 2c + 1, 2c + 8, 2c + 9 hold d = 4c .. 4c + 3, the four
          // codes of one loaded word of K
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint2 w = *reinterpret_cast<const uint2*>(src + k * 16 + 4 * c);
            qa[k][i] = w.x;
            qa[k][2 + i] = w.y;
          }
        }
      }
      if (FMT == kCacheE4m3) {
        // fp16 operands: the row by a power of two that puts its largest
        // element in [2^14, 2^15), so that it neither overflows nor loses bits
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w = qa[k][2 * h + i];
            m = max(m, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
          }
        m = max(m, __shfl_xor_sync(~0u, m, 1));
        m = max(m, __shfl_xor_sync(~0u, m, 2));
        int e = static_cast<int>(m >> 7);  // biased exponent
        e = e == 255 ? 127 + 14 : min(max(e, 16), 250);
        // times 2^(141 - e), in two steps where the factor is beyond a float
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 + (141 - e) / 2) << 23);
        const float f2 = __uint_as_float(static_cast<uint32_t>(127 + (141 - e) - (141 - e) / 2) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w = qa[k][2 * h + i];
            qa[k][2 * h + i] = pack_half2(__uint_as_float(w << 16) * f1 * f2,
                                          __uint_as_float(w & 0xffff0000u) * f1 * f2);
          }
        row_scale[i] = a.scale_log2 / f1 / f2;
      }
    }
    // depths of nodes lane and lane + 32, for the tiles that hold nodes
    int depth_lo = 0, depth_hi = 0;
    if (lane < s.n) depth_lo = __popcll(sees_of(lane) & ~(1ull << lane));
    if (lane + 32 < s.n) depth_hi = __popcll(sees_of(lane + 32) & ~(1ull << (lane + 32)));

    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float acc[DT][4];
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

    for (int i = 0; alive && i < walk.nt; ++i, ++it) {
      const int st = it % Tile::kStages;
      alive = mbar_wait(full(st), (it / Tile::kStages) & 1, ctl);
      alive = __all_sync(~0u, alive);
      if (!alive) break;
      const int key_tile = (s.tile0 + walk.t0 + i) * KEYS;
      const int key0 = key_tile + warp * WK;      // this warp's first key
      const uint32_t kbase = smem_u32(smem) + st * Tile::kStage;
      const uint32_t vbase = kbase + Tile::kBytes;
      const uint8_t* ksc = smem + st * Tile::kStage + 2 * Tile::kBytes + warp * WK;

      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
      if (FMT == kCacheBf16) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < NT; j += 2) {
            uint32_t r[4];
            ldsm_x4(kbase + Tile::at(warp * WK + j * 8 + (lm >> 1) * 8 + lr, 2 * k + (lm & 1)), r);
            mma_16816<FMT>(sc[j], qa[k], r[0], r[1]);
            mma_16816<FMT>(sc[j + 1], qa[k], r[2], r[3]);
          }
      } else {
#pragma unroll
        for (int k = 0; k < KS; k += 4)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t r[4];
            ldsm_x4(kbase + Tile::at(warp * WK + j * 8 + lr, k + lm), r);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma_16816<FMT>(sc[j], qa[k + x], e4m3x2_half2(r[x] & 0xffffu),
                             e4m3x2_half2(r[x] >> 16));
          }
      }

      // all of this warp's keys seen by every row: context keys inside every
      // node's window (a node's position is below ctx + 64)
      const bool masked = key0 + WK > s.ctx || (a.wl >= 0 && key0 < s.ctx + s.n - 1 - a.wl);
      float vexp[NT][2];   // e4m3: exponent of the value scale, and 2^-it
      float vinv[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float kf[2] = {1.f, 1.f};
        if (FMT == kCacheE4m3) {
          const uint32_t ke = *reinterpret_cast<const uint16_t*>(ksc + j * 8 + 2 * c);
          const uint32_t ve = *reinterpret_cast<const uint16_t*>(ksc + 512 + j * 8 + 2 * c);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            kf[e] = e8m0_float((ke >> (8 * e)) & 0xffu);
            const int v = static_cast<int>((ve >> (8 * e)) & 0xffu);
            vexp[j][e] = static_cast<float>(v - 127);
            vinv[j][e] = e8m0_float(static_cast<uint32_t>(max(254 - v, 0)));
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[j][e] *= row_scale[e >> 1];
          if (FMT == kCacheE4m3) sc[j][e] *= kf[e & 1];
        }
      }
      if (BIAS) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            int pos = key0 + j * 8 + 2 * c + (e & 1);
            if (masked) {
              const int n = pos - s.ctx;
              const int lo = __shfl_sync(~0u, depth_lo, n & 31), hi = __shfl_sync(~0u, depth_hi, n & 31);
              if (n >= 0) pos = s.ctx + (n < 32 ? lo : hi);
            }
            const TreeRow& rw = row[e >> 1];
            const int rel = pos - rw.pos;
            if (a.alibi_slopes)
              sc[j][e] += bias_to_log2(-rw.bias * fabsf(static_cast<float>(rel)));
            else
              sc[j][e] += rel <= a.t5.one_lo_max ? rw.bias : t5_bias_log2(a, rel, rw.head);
          }
      }
      if (masked) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + j * 8 + 2 * c + (e & 1);
            const int n = key - s.ctx;
            const TreeRow& rw = row[e >> 1];
            int pos = key;
            if (a.wl >= 0) {
              const int lo = __shfl_sync(~0u, depth_lo, n & 31), hi = __shfl_sync(~0u, depth_hi, n & 31);
              if (n >= 0) pos = s.ctx + (n < 32 ? lo : hi);
            }
            bool seen = n < 0 || (n < 64 && ((rw.sees >> n) & 1ull));
            if (a.wl >= 0) seen = seen && rw.pos - pos <= a.wl;
            if (!seen) sc[j][e] = -INFINITY;
          }
      }
      if (FMT == kCacheE4m3) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[j][e] += vexp[j][e & 1];
      }

      float m_new[2];
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        float m = m_run[i2];
#pragma unroll
        for (int j = 0; j < NT; ++j) m = fmax3(m, sc[j][2 * i2], sc[j][2 * i2 + 1]);
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
        m_new[i2] = m;
      }
      if (__any_sync(~0u, m_new[0] != m_run[0] || m_new[1] != m_run[1])) {
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const float f = m_run[i2] == m_new[i2] ? 1.f : fast_exp2(m_run[i2] - m_new[i2]);
          l_run[i2] *= f;
#pragma unroll
          for (int j = 0; j < DT; ++j) {
            acc[j][2 * i2] *= f;
            acc[j][2 * i2 + 1] *= f;
          }
          m_run[i2] = m_new[i2];
        }
      }
      const float off0 = m_run[0] == -INFINITY ? 0.f : m_run[0];
      const float off1 = m_run[1] == -INFINITY ? 0.f : m_run[1];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = fast_exp2(sc[j][e] - (e < 2 ? off0 : off1));
          sc[j][e] = p;
          l_run[e >> 1] += FMT == kCacheE4m3 ? p * vinv[j][e & 1] : p;
        }

      // O += P V over 16 keys at a time
      auto values = [&](auto flag) {
        constexpr bool kClean = decltype(flag)::value;
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t pa[4];
          if (FMT == kCacheBf16) {
            pa[0] = pack_bf16x2(sc[j][0], sc[j][1]);
            pa[1] = pack_bf16x2(sc[j][2], sc[j][3]);
            pa[2] = pack_bf16x2(sc[j + 1][0], sc[j + 1][1]);
            pa[3] = pack_bf16x2(sc[j + 1][2], sc[j + 1][3]);
          } else {
            pa[0] = pack_half2(sc[j][0], sc[j][1]);
            pa[1] = pack_half2(sc[j][2], sc[j][3]);
            pa[2] = pack_half2(sc[j + 1][0], sc[j + 1][1]);
            pa[3] = pack_half2(sc[j + 1][2], sc[j + 1][3]);
          }
          uint32_t dirty = 0;
#pragma unroll
          for (int x = 0; x < Tile::kRowBytes / 16; x += 2) {
            uint32_t r[4];
            ldsm_x4_t(vbase + Tile::at(warp * WK + j * 8 + (lm & 1) * 8 + lr, x + (lm >> 1)), r);
            if (kClean) {
              // 0 * NaN is NaN: a value no row may see is taken out here, and
              // put back below for the rows that do see it
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t bits = nonfinite_bits<FMT>(r[y]);
                dirty |= bits;
                r[y] &= ~bits;
              }
            }
            if (FMT == kCacheBf16) {
              mma_16816<FMT>(acc[x], pa, r[0], r[1]);
              mma_16816<FMT>(acc[x + 1], pa, r[2], r[3]);
            } else {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t w0 = __byte_perm(r[2 * y], 0, 0x3120);
                const uint32_t w1 = __byte_perm(r[2 * y + 1], 0, 0x3120);
                mma_16816<FMT>(acc[2 * (x + y)], pa, e4m3x2_half2(w0 & 0xffffu),
                               e4m3x2_half2(w1 & 0xffffu));
                mma_16816<FMT>(acc[2 * (x + y) + 1], pa, e4m3x2_half2(w0 >> 16),
                               e4m3x2_half2(w1 >> 16));
              }
            }
          }
          if (kClean && __any_sync(~0u, dirty != 0)) {
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                  const float p0 = __shfl_sync(~0u, sc[j + jj][e], (lane & ~3) | cc);
                  const float p1 = __shfl_sync(~0u, sc[j + jj][2 + e], (lane & ~3) | cc);
                  const int r = warp * WK + (j + jj) * 8 + 2 * cc + e;
#pragma unroll
                  for (int n = 0; n < DT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                      const int byte = acc_col<FMT>(n, c, y) * Tile::kCell;
                      const uint8_t* src = smem + st * Tile::kStage + Tile::kBytes +
                                           Tile::at(r, byte >> 4) + (byte & 15);
                      float v;
                      bool odd;
                      if (FMT == kCacheBf16) {
                        v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(src));
                        odd = isinf(v) || isnan(v);
                      } else {
                        odd = (*src & 0x7fu) == 0x7fu;
                        v = __uint_as_float(0x7fc00000u);
                      }
                      if (odd && p0 > 0.f) acc[n][y] += p0 * v;
                      if (odd && p1 > 0.f) acc[n][2 + y] += p1 * v;
                    }
                }
          }
        }
      };
      if (masked) values(Flag<true>{});
      else values(Flag<false>{});
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
    }
    // join the four warps' (m, l, O) in order: everyone scales to the common
    // maximum, warp 0 adds the others' accumulators one after another
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      l_run[i2] += __shfl_xor_sync(~0u, l_run[i2], 1);
      l_run[i2] += __shfl_xor_sync(~0u, l_run[i2], 2);
      if (c == 0) merge_ml[warp][quad + 8 * i2] = make_float2(m_run[i2], l_run[i2]);
    }
    named_barrier(1, kTreeKeyWarps * 32);
    float m_all[2], l_all[2];
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kTreeKeyWarps; ++w) m = fmaxf(m, merge_ml[w][quad + 8 * i2].x);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kTreeKeyWarps; ++w) {
        const float2 ml = merge_ml[w][quad + 8 * i2];
        // a piece without a visible key has m = -inf, l = 0 (or NaN, which stays)
        l += ml.x == -INFINITY ? ml.y : ml.y * fast_exp2(ml.x - m);
      }
      m_all[i2] = m;
      l_all[i2] = l;
      const float f = m_run[i2] == -INFINITY ? 1.f : fast_exp2(m_run[i2] - m);
#pragma unroll
      for (int j = 0; j < DT; ++j) {
        acc[j][2 * i2] *= f;
        acc[j][2 * i2 + 1] *= f;
      }
    }
#pragma unroll 1
    for (int w = 1; w < kTreeKeyWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2)
            *reinterpret_cast<float2*>(merge_o + (quad + 8 * i2) * kPad + j * 8 + 2 * c) =
                make_float2(acc[j][2 * i2], acc[j][2 * i2 + 1]);
      }
      named_barrier(1, kTreeKeyWarps * 32);
      if (warp == 0) {
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            const float2 o = *reinterpret_cast<const float2*>(merge_o + (quad + 8 * i2) * kPad +
                                                              j * 8 + 2 * c);
            acc[j][2 * i2] += o.x;
            acc[j][2 * i2 + 1] += o.y;
          }
      }
      named_barrier(1, kTreeKeyWarps * 32);
    }
    if (warp != 0) continue;
    const bool whole = walk.t0 == 0 && walk.nt == s.tiles;
    const int slot = walk.t0 == 0 ? 1 : 0;  // 0: began in an earlier CTA
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      const int lr2 = quad + 8 * i2;
      const int r = walk.block * ROWS + lr2;
      if (r >= n_rows) continue;
      const int n = r / a.G;
      if (whole) {
        const float inv = l_all[i2] > 0.f || isnan(l_all[i2]) ? 1.f / l_all[i2] : 0.f;
        __nv_bfloat16* dst = a.o + static_cast<int64_t>(s.row0 + n) * a.o_t + row[i2].head * a.o_h;
        if (FMT == kCacheBf16) {
#pragma unroll
          for (int j = 0; j < DT; ++j)
            *reinterpret_cast<uint32_t*>(dst + j * 8 + 2 * c) =
                pack_bf16x2(acc[j][2 * i2] * inv, acc[j][2 * i2 + 1] * inv);
        } else {
#pragma unroll
          for (int j = 0; j < DT; j += 2)
            *reinterpret_cast<uint2*>(dst + j * 8 + 4 * c) =
                make_uint2(pack_bf16x2(acc[j][2 * i2] * inv, acc[j + 1][2 * i2] * inv),
                           pack_bf16x2(acc[j][2 * i2 + 1] * inv, acc[j + 1][2 * i2 + 1] * inv));
        }
        if (c == 0)
          a.lse[static_cast<int64_t>(row[i2].head) * a.T + s.row0 + n] =
              (m_all[i2] + log2f(l_all[i2])) * kLn2;
      } else {
        const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * ROWS + lr2;
        float* dst = a.part_o + at * D;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) dst[acc_col<FMT>(j, c, e)] = acc[j][2 * i2 + e];
        if (c == 0) a.part_ml[at] = make_float2(m_all[i2], l_all[i2]);
      }
    }
  }
}

// Joins the pieces of (row, head)s that span CTAs, in the CTAs' order.  One
// warp per query row and head; the lanes first weigh up to 32 pieces at once,
// then add them, D / 32 columns each.
constexpr int kTreeJoinWarps = 4;

template <int D, int FMT>
__global__ void __launch_bounds__(kTreeJoinWarps * 32) tree_join_kernel(const TreeArgs a, int ctas) {
  constexpr int ROWS = 16;
  constexpr int KEYS = TreeTile<D, FMT>::kKeys;
  constexpr int W = D / 32;
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int x = blockIdx.x * kTreeJoinWarps + (threadIdx.x >> 5);   // node * Hq + head
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeSeq s = tree_seq<KEYS, ROWS>(a, b);
  const int n = x / a.Hq, h = x - n * a.Hq;
  if (n >= s.n) return;
  const int hkv = h / a.G;
  const int r = n * a.G + (h - hkv * a.G);
  const int block = r / ROWS;
  const int64_t total = a.prefix[a.B];
  const int64_t per = (total + ctas - 1) / ctas;
  const int64_t first = a.prefix[b] + (static_cast<int64_t>(hkv) * s.rb + block) * s.tiles;
  const int c0 = static_cast<int>(first / per);
  const int c1 = static_cast<int>((first + s.tiles - 1) / per);
  if (c0 == c1) return;
  float m = -INFINITY, l = 0.f, acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.f;
  for (int base = c0; base <= c1; base += 32) {
    const int cta = base + lane;
    // the first CTA's piece began in it, every later one's before it
    const int64_t at = (static_cast<int64_t>(cta) * 2 + (cta == c0 ? 1 : 0)) * ROWS + (r & (ROWS - 1));
    float2 ml = make_float2(-INFINITY, 0.f);
    if (cta <= c1) ml = a.part_ml[at];
    float top = ml.x;
#pragma unroll
    for (int sft = 16; sft > 0; sft >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, sft));
    top = fmaxf(top, m);
    const float f_old = m == -INFINITY ? 1.f : fast_exp2(m - top);
    const float f = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - top);
    float add = ml.y * f;
#pragma unroll
    for (int sft = 16; sft > 0; sft >>= 1) add += __shfl_xor_sync(~0u, add, sft);
    l = l * f_old + add;
    m = top;
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] *= f_old;
    const int count = min(32, c1 - base + 1);
#pragma unroll 8
    for (int j = 0; j < count; ++j) {
      const int cj = base + j;
      const float w = __shfl_sync(~0u, f, j);
      const float* src = a.part_o + ((static_cast<int64_t>(cj) * 2 + (cj == c0 ? 1 : 0)) * ROWS +
                                     (r & (ROWS - 1))) * D + lane * W;
      if (W == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] += w * v.x;
        acc[1] += w * v.y;
        acc[2 % W] += w * v.z;
        acc[3 % W] += w * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] += w * v.x;
        acc[1] += w * v.y;
      }
    }
  }
  const float inv = l > 0.f || isnan(l) ? 1.f / l : 0.f;
  __nv_bfloat16* dst = a.o + static_cast<int64_t>(s.row0 + n) * a.o_t + h * a.o_h + lane * W;
  if (W == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2 % W] * inv, acc[3 % W] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0)
    a.lse[static_cast<int64_t>(h) * a.T + s.row0 + n] = (m + log2f(l)) * kLn2;
}

}  // namespace sdpa
