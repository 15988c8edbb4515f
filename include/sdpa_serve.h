/*
 * sdpa_serve.h -- C ABI of the serving side of the B200 attention library:
 * rotary positions, a paged key / value cache in bf16 or e4m3, attention of
 * drafted nodes over it, and the verification of drafted tokens.
 *
 * The conventions of sdpa.h hold (layout, heads, ownership, streams, errors,
 * status codes): the caller owns every buffer, no entry point allocates, frees
 * or synchronises (except sdpa_serve_read_device_status), arguments are checked
 * before anything is queued, and device pointers belong to the current device.
 * Every kernel takes its sums in a fixed order, so repeated calls give the same
 * bits.  The library (libsdpa_serve_b200.so) has a status word and a wait limit
 * of its own.
 */
#ifndef SDPA_B200_SDPA_SERVE_H
#define SDPA_B200_SDPA_SERVE_H

#include "sdpa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotary positions (RoFormer, Su et al. 2021): pair i of the first `rot`
 * elements of every head is turned by the angle position * freqs[i]:
 *     y1 = amplitude (x1 cos t - x2 sin t),  y2 = amplitude (x2 cos t + x1 sin t);
 * inverse = 1 turns by -t, which with the same amplitude is the gradient of
 * the rotation (dx from dy).  The pairs are (x[i], x[i + rot/2]), or
 * (x[2i], x[2i + 1]) when interleaved; elements from `rot` on are copied.
 * q [B, L, Hq, d] and k [B, L, Hkv, d] bf16, d contiguous, rotated in one
 * launch; Hkv = 0: q alone (k and k_out ignored).  Strides in elements,
 * multiples of 8, inputs and outputs each their own.  q_out may be q itself
 * with the same strides (and k_out k): in place; other overlap is not allowed.
 *   positions: device int32 [B, L] with row stride pos_b (L contiguous; 0: one
 *     row for all sequences), any sign; NULL: position offset + l.
 *   freqs: device float64 [rot / 2], radians per position
 *     (sdpa_rope_frequencies).  The angle is formed and reduced in float64, so
 *     positions of a long context lose nothing; the rest is float32 with one
 *     rounding to bf16.
 *   d in {64, 128}; rot even, 2 <= rot <= d; 1 <= B * L < 2^31.
 */
typedef struct sdpa_rope_desc {
  int64_t B, L, Hq, Hkv, d;
  int64_t q_b, q_l, q_h;    /* element strides of q */
  int64_t k_b, k_l, k_h;    /* element strides of k */
  int64_t qo_b, qo_l, qo_h; /* element strides of q_out */
  int64_t ko_b, ko_l, ko_h; /* element strides of k_out */
  const int32_t* positions;
  int64_t pos_b;
  int64_t offset;
  const double* freqs;
  int32_t rot, interleaved, inverse;
  float amplitude;
} sdpa_rope_desc;

sdpa_status_t sdpa_rope(const sdpa_rope_desc* rope, const void* q, const void* k, void* q_out,
                        void* k_out, void* stream);

/*
 * The frequencies of sdpa_rope, host arithmetic in float64, written to host
 * memory freqs[rot / 2], and the amplitude that goes with them (1 except for
 * YARN).  Unscaled: freqs[i] = base^(-2i / rot).
 *   LINEAR: divided by `factor` (position interpolation).
 *   NTK:    base replaced by base * factor^(rot / (rot - 2)); rot > 2.
 *   YARN:   (Peng et al. 2023) interpolated where a pair turns fewer than
 *           beta_slow times over original_length positions, kept where it
 *           turns more than beta_fast times, a linear blend over the pair
 *           index between; amplitude 0.1 ln(factor) + 1.
 * factor >= 1; base > 1; original_length >= 1 and beta_fast > beta_slow > 0
 * for YARN.
 */
typedef enum sdpa_rope_scaling {
  SDPA_ROPE_PLAIN = 0,
  SDPA_ROPE_LINEAR = 1,
  SDPA_ROPE_NTK = 2,
  SDPA_ROPE_YARN = 3
} sdpa_rope_scaling;

sdpa_status_t sdpa_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor,
                                    int64_t original_length, double beta_fast, double beta_slow,
                                    double* freqs, float* amplitude);

/*
 * A paged key / value cache.  Position p of a sequence lives in row
 * p % page_size of the page that the sequence's page table names at
 * p / page_size.  k and v are [num_pages][Hkv][page_size][d] with element
 * strides stride_page, stride_head, stride_row (the same for both, d
 * contiguous), 16-byte aligned, strides multiples of 16 bytes.
 *   SDPA_CACHE_BF16: bf16 rows; the scales are ignored.
 *   SDPA_CACHE_E4M3: 8-bit rows (e4m3, no infinities, largest value 448) with
 *     one power-of-two scale per row and head: value = code * 2^(e - 127), e
 *     a byte 0 .. 254 of k_scale / v_scale [num_pages][Hkv][page_size] (strides
 *     scale_stride_page, scale_stride_head, multiples of 16; rows contiguous;
 *     16-byte aligned).  A power of two costs an e4m3 code nothing (its
 *     relative step is the same in every binade) and makes scaling exact both
 *     ways.
 * page_size in {16, 32, 64, 128, 256}; d in {64, 128}; Hkv <= 65535;
 * num_pages < 2^31.
 */
typedef enum sdpa_cache_format { SDPA_CACHE_BF16 = 0, SDPA_CACHE_E4M3 = 1 } sdpa_cache_format;

typedef struct sdpa_kv_cache {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int32_t format; /* sdpa_cache_format */
  int64_t num_pages, page_size, Hkv, d;
  int64_t stride_page, stride_head, stride_row;
  int64_t scale_stride_page, scale_stride_head;
} sdpa_kv_cache;

/*
 * Writes T rows of bf16 K and V [T, Hkv, d] (element strides kv_t, kv_h,
 * multiples of 8, the same for both; d contiguous) into the cache, row t at
 * slots[t] = page * page_size + row in the page.  v NULL: K alone (and V alone,
 * with strides of its own, by a second call that gives the cache's v and
 * v_scale as its k and k_scale).  A negative slot skips its
 * row (padding); a slot past the cache is skipped and reported by
 * sdpa_serve_read_device_status as SDPA_ERR_UNSUPPORTED.  Two rows of one call must
 * not name the same slot (its contents would be unspecified).  e4m3: the scale
 * is the smallest power of two 2^(e - 127), 1 <= e <= 254, with the row's
 * largest finite magnitude at most 448 of it (e = 127 for a row of zeros);
 * codes round to nearest even; infinities become +-448, NaN stays NaN.
 * slots: device int64 [T].  T = 0 does nothing; T < 2^31.
 */
sdpa_status_t sdpa_cache_append(const sdpa_kv_cache* cache, const void* k, const void* v,
                                int64_t T, int64_t kv_t, int64_t kv_h, const int64_t* slots,
                                void* stream);

/*
 * Reads the first cu_seqlens[b + 1] - cu_seqlens[b] positions of every
 * sequence b back as packed bf16 K and V [total, Hkv, d] (element strides
 * kv_t, kv_h), the operands of sdpa_fwd_varlen.  A prompt chunk of more than 64
 * tokens attends to its cached prefix that way: with its own rows in the cache
 * too, and window_right = prefix length in place of the causal mask.  That mask
 * is the whole batch's, and sdpa_fwd_varlen counts the chunk's positions from 0:
 * so a call takes sequences of one prefix length, without a left window and
 * without T5, ALiBi or REL biases.  page_table: device int32 [B][table_width],
 * row stride table_b (0: one row for all).  Rows from cu_seqlens[B] to total are left as they
 * were, and so are rows whose page lies outside the table or the cache, which
 * sdpa_serve_read_device_status reports as SDPA_ERR_UNSUPPORTED.  An e4m3 value
 * times its scale is exact in bf16 (below bf16's smallest normal number, to
 * its rounding).  B <= 65535, total < 2^30.
 */
sdpa_status_t sdpa_cache_gather(const sdpa_kv_cache* cache, int64_t B, const int32_t* page_table,
                                int64_t table_width, int64_t table_b, const int32_t* cu_seqlens,
                                int64_t total, void* k, void* v, int64_t kv_t, int64_t kv_h,
                                void* stream);

/*
 * Attention of drafted nodes over a paged cache: the decoding form of
 * sdpa_fwd.  Sequence b owns query rows [cu_nodes[b], cu_nodes[b + 1]) of
 * q [T, Hq, d]: n <= max_nodes <= 64 nodes (1: plain decoding).  Its keys are
 * the cached positions 0 .. ctx_lens[b] - 1 (the context) and
 * ctx_lens[b] .. ctx_lens[b] + n - 1 (the nodes' own keys, in node order,
 * already in the cache).  Every node sees the context; node i sees node j iff
 * bit j of tree_mask[cu_nodes[b] + i] is set (bits from n on are ignored).
 * tree_mask NULL: a chain, node i sees nodes 0 .. i.
 *   Positions: a context key's is its own; node i's is ctx_lens[b] plus the
 *   number of other nodes with an index below n that i sees (its depth, when
 *   the mask holds its ancestors).
 *   window_left >= 0: keys with a position below the node's minus window_left
 *   are hidden too (the framework's inclusive window); < 0: no window.
 *   bias: NULL, NONE, T5 or ALIBI, at distance key position - node position;
 *   DENSE and REL -> SDPA_ERR_UNSUPPORTED.  For T5 a distance's magnitude is
 *   below 2^30.
 * Outputs: o bf16 [T, Hq, d] (strides o_t, o_h) and LSE float32 [Hq, T]
 * contiguous; a node that sees no key gets O = 0, LSE = -inf.  Rows of q
 * behind cu_nodes[B] are not computed and their outputs left as they were.
 * A key that every node of its sequence is kept from may hold anything, NaN
 * included; so may one that some nodes see: it reaches those alone.
 * Sequences whose cu_nodes, ctx_lens or pages do not fit (n outside
 * 0 .. max_nodes, rows outside T, ctx_lens[b] < 0, ctx_lens[b] + n positions
 * more than the table's width holds, a page outside the cache that holds a key
 * inside the window of a node at ctx_lens[b]) are reported by
 * sdpa_serve_read_device_status as SDPA_ERR_UNSUPPORTED; their outputs are
 * unspecified, and no memory outside the tensors is touched.
 * workspace: sdpa_tree_fwd_workspace_size() bytes, 256-byte aligned, contents
 * ignored on entry; calls that may overlap on the GPU need one each.
 * 1 <= B, Hq <= 65535; 1 <= T < 2^30 (a batch without rows is refused, as by
 * sdpa_fwd); table_width * page_size <= 2^30, and the batch's
 * tiles of 128 keys over KV heads and blocks of 16 query rows are counted in 32
 * bits: SDPA_ERR_UNSUPPORTED where they could pass that.
 * Deterministic: the split of the keys depends on the lengths and the GPU's
 * number of SMs alone, and sums are taken in a fixed order.
 * Accuracy: scores, maxima, sums and O are float32.  A weight enters the product
 * with V rounded to bf16 over a bf16 cache (half a step, 2^-9 of it), as in
 * sdpa_fwd, and as two e4m3 parts over an e4m3 cache: to 2^-8 of it, or to 2^-20
 * of the largest weight times value scale of its row, rounded without bias over
 * the keys, whichever is more.  What a key adds to LSE is not rounded.  A bf16
 * query's elements are exact over e4m3 down to 2^-21 of their row's largest (and
 * 2^-132).  A score's bias near the type's lowest value leaves no digits for the
 * score, as in float32.
 */
typedef struct sdpa_tree {
  int64_t B, T, max_nodes, Hq;
  int64_t q_t, q_h; /* element strides of q */
  int64_t o_t, o_h; /* element strides of o */
  const int32_t* cu_nodes;   /* device [B + 1] */
  const int32_t* ctx_lens;   /* device [B] */
  const int32_t* page_table; /* device [B][table_width], row stride table_b (0: one for all) */
  int64_t table_width, table_b;
  const int64_t* tree_mask;  /* device [T] or NULL */
  int64_t window_left;
} sdpa_tree;

size_t sdpa_tree_fwd_workspace_size(const sdpa_tree* tree, const sdpa_kv_cache* cache);
sdpa_status_t sdpa_tree_fwd(const sdpa_tree* tree, const sdpa_kv_cache* cache, const void* q,
                            const sdpa_bias_desc* bias, float scale, void* o, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Verification of drafted tokens by rejection sampling (Leviathan et al.
 * 2023; Chen et al. 2023), over a tree whose nodes' children are tried in
 * turn against what earlier ones left of the distribution (Miao et al. 2024).
 * Per sequence: node 0 is the last token already accepted; node n > 0 is a
 * token drafted as a child of parents[n] < n (a negative parent: no node).
 * target[n] is the target model's distribution after node n, draft[n] the one
 * that node n's children were drawn from.  From node `at` = 0, with
 * w = target[at]: for its children c in index order, x = tokens[c]:
 *     accept c if u_accept[c] * draft[at][x] < w[x]; then at = c, w = target[c];
 *     else w = max(w - draft[at], 0) divided by its sum (left at 0 if that is 0).
 * When no child is left, the next token is drawn from w (from target[at]
 * where w is all 0): the smallest x whose cumulative weight exceeds
 * u_sample * sum(w), and the last x with a weight where rounding leaves none.
 * Weights, sums and comparisons are float64, so a tie is a tie of the given
 * numbers.  Without children this samples from target[0].
 *   target, draft: device float32 [B, N, V], element strides *_b, *_n (V
 *     contiguous); N = 1: draft may be NULL.  1 <= N <= 64, 1 <= V < 2^30.
 *   tokens, parents: device int32 [B, N] contiguous; tokens[0], parents[0] and
 *     u_accept[0] are not read; parents NULL: a chain (parents[n] = n - 1).
 *     A token outside [0, V) is never accepted and removes draft[at] from w as
 *     any rejected one; a parent >= n makes n no node.  Both are reported by
 *     sdpa_serve_read_device_status as SDPA_ERR_UNSUPPORTED.  B >= 1.
 *   u_accept [B, N], u_sample [B]: device float32, in [0, 1).
 * Outputs: path int32 [B, N]: the accepted nodes from node 0 on, then -1;
 * accepted int32 [B]: how many after node 0; next_token int32 [B].  If all
 * weights are 0 or NaN the next token is 0.
 */
typedef struct sdpa_verify {
  int64_t B, N, V;
  int64_t target_b, target_n, draft_b, draft_n;
  const float* target;
  const float* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const float* u_accept;
  const float* u_sample;
} sdpa_verify;

sdpa_status_t sdpa_spec_verify(const sdpa_verify* verify, int32_t* path, int32_t* accepted,
                               int32_t* next_token, void* stream);

/*
 * Synchronises `stream`, then returns and clears the sticky status of this
 * library's kernels on the current device: SDPA_OK; SDPA_ERR_TIMEOUT if a
 * bounded wait ran out; SDPA_ERR_UNSUPPORTED if a kernel met a slot, page,
 * length, token or parent out of range (as each entry point says), or
 * misaligned shared memory; SDPA_ERR_CUDA if the reads fail.
 */
sdpa_status_t sdpa_serve_read_device_status(void* stream);

/* As sdpa_set_wait_limit_ns, for the waits of this library's kernels. */
void sdpa_serve_set_wait_limit_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_B200_SDPA_SERVE_H */
