// serve_api.cu -- host side of the serving entry points declared in
// include/sdpa_serve.h: argument validation, tensor maps, launches and the
// library's status word.  A library and translation unit of its own, so that
// the attention kernels are built from their own sources alone; the few host
// helpers that both need (tensor-map entry point, T5 thresholds) are repeated.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "sdpa_serve.h"
#include "kv_cache.cuh"
#include "rope.cuh"
#include "spec_verify.cuh"
#include "tree_fwd.cuh"

using namespace sdpa;

namespace {

uint64_t g_wait_limit_ns = 2000000000ull;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Integer thresholds of the T5 log buckets, evaluated in float64 exactly as
// the closed form reads: large(n) = max_exact + trunc(ln(n / max_exact) /
// ln(max_distance / max_exact) * (half - max_exact)).
bool fill_t5(T5Spec& t, int nb, int md, int bidir) {
  const int half = bidir ? nb / 2 : nb;
  const int me = half / 2;
  if (me < 1 || md <= me) return false;
  const int K = half - me;
  if (K > kMaxT5Thresholds) return false;
  t.half = half;
  t.max_exact = me;
  t.bidirectional = bidir ? 1 : 0;
  t.nthr = K;
  const double denom = std::log(static_cast<double>(md) / static_cast<double>(me));
  auto large = [&](int64_t n) -> int64_t {
    const double v = std::log(static_cast<double>(n) / static_cast<double>(me)) / denom *
                     static_cast<double>(half - me);
    return me + static_cast<int64_t>(v);
  };
  // thr[k]: the first n whose closed form reaches max_exact + k.  It is found
  // from its real-valued inverse (a decoding step makes one call, which must
  // not walk all distances up to max_distance).
  const int64_t limit = 4 * static_cast<int64_t>(md) + 1024;
  int64_t n = me;
  for (int k = 0; k < K; ++k) {
    const int64_t guess = static_cast<int64_t>(me * std::exp(denom * k / (half - me)));
    n = std::max(n, std::min(guess, limit));
    while (n > me && large(n - 1) >= me + k) --n;
    while (n < limit && large(n) < me + k) ++n;
    t.thr[k] = (n < limit) ? static_cast<int>(n) : INT_MAX;
  }
  for (int k = K; k < kMaxT5Thresholds; ++k) t.thr[k] = INT_MAX;
  // the capped bucket (half - 1) holds every n >= thr[K - 1]
  const int sat = t.thr[K - 1];
  t.one_lo_max = sat == INT_MAX ? INT_MIN : -sat;
  t.one_hi_min = bidir ? sat : 0;
  t.log_scale = static_cast<float>(static_cast<double>(half - me) / std::log2(static_cast<double>(md) / me));
  t.inv_max_exact = static_cast<float>(1.0 / me);
  return true;
}

int clamp_window(int64_t w, int64_t L) {
  if (w < 0) return -1;
  return static_cast<int>(w > L ? L : w);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

bool good_stride(int64_t v, int64_t multiple) {
  return v > 0 && v % multiple == 0 && v < (1ll << 38);
}

// Row stride of a matrix that is only read: rows side by side, or one for all.
bool row_step(int64_t v, int64_t width) { return v == 0 || v >= width; }

// ------------------------------------------------------------------ rotary
template <int D>
cudaError_t launch_rope(const RopeArgs& a, int mode, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((a.tokens + a.per_cta - 1) / a.per_cta);
  switch (mode) {
    case kRopeHalf: rope_kernel<D, kRopeHalf><<<grid, kRopeThreads, 0, st>>>(a); break;
    case kRopeInterleaved: rope_kernel<D, kRopeInterleaved><<<grid, kRopeThreads, 0, st>>>(a); break;
    default: rope_kernel<D, kRopeHalfAny><<<grid, kRopeThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------- cache
sdpa_status_t check_cache(const sdpa_kv_cache* c, CacheView& v) {
  if (!c || !c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return SDPA_ERR_INVALID_ARG;
  if (c->format != SDPA_CACHE_BF16 && c->format != SDPA_CACHE_E4M3) return SDPA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1) return SDPA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SDPA_ERR_UNSUPPORTED;
  const int64_t ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return SDPA_ERR_UNSUPPORTED;
  if (c->Hkv > 65535 || c->num_pages >= (1ll << 31) - 1) return SDPA_ERR_UNSUPPORTED;
  const bool e4m3 = c->format == SDPA_CACHE_E4M3;
  const int64_t mult = e4m3 ? 16 : 8;
  if (!good_stride(c->stride_page, mult) || !good_stride(c->stride_head, mult) ||
      !good_stride(c->stride_row, mult))
    return SDPA_ERR_INVALID_ARG;
  if (e4m3) {
    if (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale))
      return SDPA_ERR_INVALID_ARG;
    if (!good_stride(c->scale_stride_page, 16) || !good_stride(c->scale_stride_head, 16))
      return SDPA_ERR_INVALID_ARG;
  }
  v = CacheView{};
  v.k = c->k;
  v.v = c->v;
  v.ks = e4m3 ? c->k_scale : nullptr;
  v.vs = e4m3 ? c->v_scale : nullptr;
  v.num_pages = c->num_pages;
  v.page_size = static_cast<int>(ps);
  for (v.page_shift = 0; (1 << v.page_shift) < ps;) ++v.page_shift;
  v.Hkv = static_cast<int>(c->Hkv);
  v.s_page = c->stride_page;
  v.s_head = c->stride_head;
  v.s_row = c->stride_row;
  v.ss_page = c->scale_stride_page;
  v.ss_head = c->scale_stride_head;
  return SDPA_OK;
}

// Rows per CTA of the cache kernels, a power of two.  Up to 8 are loaded at
// once, so a short call takes as many as leave three CTAs per SM for each of K
// and V (gathers of 1500 rows: 3.5 us with 4, 4.6 with 2).  Beyond that, up to
// kCacheRows while four CTAs per SM stay (12000 rows: 17 us with 16, 20 with
// 28; 40000: 50 with 32, 54 with 64).
int cache_rows(int64_t total) {
  const int sms = sm_count();
  if (sms <= 0) return 0;
  int rows = 2;
  while (rows < 8 && total > 3ll * rows * sms) rows *= 2;
  while (rows >= 8 && rows < kCacheRows && total >= 2ll * rows * 4 * sms) rows *= 2;
  return rows;
}

// 4-D map of a cache tensor along (head_dim, row, head, page): boxes of
// box_rows rows of one head of one page, 128 bytes (or a whole 64-byte row)
// wide, swizzled as wide as they are.  A page past the last reads as zeros.
bool make_cache_map(CUtensorMap* m, const void* base, const sdpa_kv_cache* c, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const bool e4m3 = c->format == SDPA_CACHE_E4M3;
  const int64_t cell = e4m3 ? 1 : 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                        static_cast<cuuint64_t>(c->Hkv), static_cast<cuuint64_t>(c->num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c->stride_row * cell),
                           static_cast<cuuint64_t>(c->stride_head * cell),
                           static_cast<cuuint64_t>(c->stride_page * cell)};
  const int64_t line = c->d * cell < 128 ? c->d * cell : 128;
  cuuint32_t box[4] = {static_cast<cuuint32_t>(line / cell), static_cast<cuuint32_t>(box_rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// -------------------------------------------------------------------- tree
struct TreePlan {
  size_t ml, o, total;
};

sdpa_status_t check_tree(const sdpa_tree* t, const sdpa_kv_cache* c, CacheView& v, TreePlan& pl) {
  sdpa_status_t st = check_cache(c, v);
  if (st != SDPA_OK) return st;
  if (!t || t->B < 1 || t->T < 1 || t->max_nodes < 1 || t->Hq < 1) return SDPA_ERR_INVALID_ARG;
  if (t->Hq % c->Hkv != 0) return SDPA_ERR_INVALID_ARG;
  if (t->max_nodes > kTreeMaxNodes || t->B > 65535 || t->Hq > 65535 || t->T >= (1ll << 30))
    return SDPA_ERR_UNSUPPORTED;
  if (!t->cu_nodes || !t->ctx_lens || !t->page_table || t->table_width < 1 ||
      !row_step(t->table_b, t->table_width))
    return SDPA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(t->cu_nodes) & 3u) || (reinterpret_cast<uintptr_t>(t->ctx_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(t->page_table) & 3u) || (reinterpret_cast<uintptr_t>(t->tree_mask) & 7u))
    return SDPA_ERR_INVALID_ARG;
  // positions, and the tiles of the whole batch, are counted in 32 bits
  if (t->table_width > (1ll << 30) / c->page_size) return SDPA_ERR_UNSUPPORTED;
  const int64_t tiles = (t->table_width * c->page_size + kTreeKeys - 1) / kTreeKeys;
  const int64_t blocks = (t->max_nodes * (t->Hq / c->Hkv) + 15) / 16;
  if ((tiles + 3) * blocks >= ((1ll << 31) - (1ll << 16)) / (c->Hkv * t->B)) return SDPA_ERR_UNSUPPORTED;  // (3: a piece's cost)
  if (!good_stride(t->q_t, 8) || !good_stride(t->q_h, 8) || !good_stride(t->o_t, 8) ||
      !good_stride(t->o_h, 8))
    return SDPA_ERR_INVALID_ARG;
  pl.ml = 0;
  pl.o = round256(static_cast<size_t>(kTreeMaxCtas) * 2 * kTreeMaxRows * sizeof(float2));
  pl.total = pl.o + static_cast<size_t>(kTreeMaxCtas) * 2 * kTreeMaxRows * c->d * sizeof(float);
  return SDPA_OK;
}

template <int D, int FMT, int R, int BIAS>
cudaError_t launch_tree(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                        cudaStream_t st) {
  using L = TreeLayout<D, FMT, R, BIAS>;
  auto kern = tree_fwd_kernel<D, FMT, R, BIAS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int grid = std::min(sms, kTreeMaxCtas);
  kern<<<grid, kTreeThreads, L::kSmem, st>>>(a, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a (sequence, head) of one tile cannot span CTAs
  if (a.width * a.page_size <= kTreeKeys || grid == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (a.B <= 32) {
    cfg.gridDim = dim3((a.max_nodes * a.Hq + kTreeJoinWarps - 1) / kTreeJoinWarps, a.B);
    cfg.blockDim = dim3(kTreeJoinWarps * 32);
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, R>, a, grid);
  }
  const int rows = std::min(a.max_nodes * a.G, R);  // of a block at most
  cfg.gridDim = dim3((rows + kTreeCutWarps - 1) / kTreeCutWarps, grid - 1);
  cfg.blockDim = dim3(kTreeCutWarps * 32);
  return cudaLaunchKernelEx(&cfg, tree_join_cuts_kernel<D, R>, a, grid);
}

// Query rows of one product: the smallest of 8, 16, 32 and 64 that holds a
// sequence's, 64 (and several blocks) beyond.
template <int D, int FMT, int BIAS>
cudaError_t dispatch_tree_rows(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                               cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.max_nodes) * a.G;
  if (rows <= 8) return launch_tree<D, FMT, 8, BIAS>(a, mk, mv, st);
  if (rows <= 16) return launch_tree<D, FMT, 16, BIAS>(a, mk, mv, st);
  if (rows <= 32) return launch_tree<D, FMT, 32, BIAS>(a, mk, mv, st);
  return launch_tree<D, FMT, 64, BIAS>(a, mk, mv, st);
}

template <int D, int FMT>
cudaError_t dispatch_tree_bias(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                               cudaStream_t st) {
  return a.alibi_slopes || a.t5_table ? dispatch_tree_rows<D, FMT, 1>(a, mk, mv, st)
                                      : dispatch_tree_rows<D, FMT, 0>(a, mk, mv, st);
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_rope(const sdpa_rope_desc* r, const void* q, const void* k, void* q_out,
                        void* k_out, void* stream) {
  if (!r || r->B < 1 || r->L < 1 || r->Hq < 1 || r->Hkv < 0) return SDPA_ERR_INVALID_ARG;
  if (r->d != 64 && r->d != 128) return SDPA_ERR_UNSUPPORTED;
  if (r->rot < 2 || r->rot > r->d || r->rot % 2 != 0) return SDPA_ERR_INVALID_ARG;
  if (r->Hq > 65535 || r->Hkv > 65535 || r->B >= (1ll << 31) || r->L >= (1ll << 31) / r->B)
    return SDPA_ERR_UNSUPPORTED;
  if (!std::isfinite(r->amplitude)) return SDPA_ERR_INVALID_ARG;
  if (!r->freqs || (reinterpret_cast<uintptr_t>(r->freqs) & 7u) ||
      (reinterpret_cast<uintptr_t>(r->positions) & 3u) || (r->positions && r->B > 1 && !row_step(r->pos_b, r->L)))
    return SDPA_ERR_INVALID_ARG;
  if (!q || !q_out || !aligned16(q) || !aligned16(q_out)) return SDPA_ERR_INVALID_ARG;
  const int64_t sq[] = {r->q_b, r->q_l, r->q_h, r->qo_b, r->qo_l, r->qo_h};
  for (int64_t v : sq)
    if (!good_stride(v, 8)) return SDPA_ERR_INVALID_ARG;
  RopeArgs a{};
  if (r->Hkv > 0) {
    if (!k || !k_out || !aligned16(k) || !aligned16(k_out)) return SDPA_ERR_INVALID_ARG;
    const int64_t sk[] = {r->k_b, r->k_l, r->k_h, r->ko_b, r->ko_l, r->ko_h};
    for (int64_t v : sk)
      if (!good_stride(v, 8)) return SDPA_ERR_INVALID_ARG;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.ko = static_cast<__nv_bfloat16*>(k_out);
    a.k_b = r->k_b;
    a.k_l = r->k_l;
    a.k_h = r->k_h;
    a.ko_b = r->ko_b;
    a.ko_l = r->ko_l;
    a.ko_h = r->ko_h;
  }
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qo = static_cast<__nv_bfloat16*>(q_out);
  a.q_b = r->q_b;
  a.q_l = r->q_l;
  a.q_h = r->q_h;
  a.qo_b = r->qo_b;
  a.qo_l = r->qo_l;
  a.qo_h = r->qo_h;
  a.positions = r->positions;
  a.pos_b = r->pos_b;
  a.offset = r->offset;
  a.freqs = r->freqs;
  a.L = static_cast<int>(r->L);
  a.Hq = static_cast<int>(r->Hq);
  a.H = static_cast<int>(r->Hq + r->Hkv);
  a.tokens = r->B * r->L;
  a.half = r->rot / 2;
  a.amplitude = r->amplitude;
  a.sign = r->inverse ? -1.f : 1.f;
  const int sms = sm_count();
  if (sms <= 0) return SDPA_ERR_CUDA;
  // as many tokens per CTA as make one batch of loads, one where that would
  // leave SMs without work
  const int fill = kRopeFlight * kRopeThreads / (a.H * static_cast<int>(r->d) / 16);
  a.per_cta = a.tokens <= 8ll * sms ? 1 : std::max(1, std::min(kRopeTokens, fill));
  const int mode = r->interleaved ? kRopeInterleaved : (a.half % 8 == 0 ? kRopeHalf : kRopeHalfAny);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = r->d == 128 ? launch_rope<128>(a, mode, cs) : launch_rope<64>(a, mode, cs);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

sdpa_status_t sdpa_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor,
                                    int64_t original_length, double beta_fast, double beta_slow,
                                    double* freqs, float* amplitude) {
  if (rot < 2 || rot % 2 != 0 || !std::isfinite(base) || base <= 1.0 || !freqs || !amplitude)
    return SDPA_ERR_INVALID_ARG;
  if (scaling < SDPA_ROPE_PLAIN || scaling > SDPA_ROPE_YARN) return SDPA_ERR_INVALID_ARG;
  if (scaling != SDPA_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0))
    return SDPA_ERR_INVALID_ARG;
  if (scaling == SDPA_ROPE_NTK && rot < 4) return SDPA_ERR_INVALID_ARG;
  if (scaling == SDPA_ROPE_YARN &&
      (original_length < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) ||
       !(beta_fast > beta_slow)))
    return SDPA_ERR_INVALID_ARG;
  const double b = scaling == SDPA_ROPE_NTK ? base * std::pow(factor, rot / (rot - 2.0)) : base;
  *amplitude = 1.f;
  // YARN: the pair index at which `turns` turns fit into original_length positions
  double lo = 0.0, hi = 0.0;
  if (scaling == SDPA_ROPE_YARN) {
    auto index_of = [&](double turns) {
      return rot * std::log(static_cast<double>(original_length) / (turns * 2.0 * 3.14159265358979323846)) /
             (2.0 * std::log(base));
    };
    lo = std::max(std::floor(index_of(beta_fast)), 0.0);
    hi = std::min(std::ceil(index_of(beta_slow)), rot - 1.0);
    if (hi <= lo) hi = lo + 0.001;
    *amplitude = static_cast<float>(0.1 * std::log(factor) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(b, -2.0 * i / rot);
    double g = f;
    if (scaling == SDPA_ROPE_LINEAR) g = f / factor;
    if (scaling == SDPA_ROPE_YARN) {
      const double ramp = std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0);  // 1: interpolated
      g = f / factor * ramp + f * (1.0 - ramp);
    }
    freqs[i] = g;
  }
  return SDPA_OK;
}

sdpa_status_t sdpa_cache_append(const sdpa_kv_cache* cache, const void* k, const void* v,
                                int64_t T, int64_t kv_t, int64_t kv_h, const int64_t* slots,
                                void* stream) {
  AppendArgs a{};
  const sdpa_status_t st = check_cache(cache, a.c);
  if (st != SDPA_OK) return st;
  if (T < 0) return SDPA_ERR_INVALID_ARG;
  if (T == 0) return SDPA_OK;
  if (!k || !aligned16(k) || !aligned16(v) || !slots || (reinterpret_cast<uintptr_t>(slots) & 7u) ||
      !good_stride(kv_t, 8) || !good_stride(kv_h, 8))
    return SDPA_ERR_INVALID_ARG;
  if (T >= (1ll << 31)) return SDPA_ERR_UNSUPPORTED;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.T = T;
  a.kv_t = kv_t;
  a.kv_h = kv_h;
  a.slots = slots;
  a.rows = cache_rows(T);
  if (!a.rows) return SDPA_ERR_CUDA;
  const dim3 g(static_cast<unsigned>((T + a.rows - 1) / a.rows), v ? 2 : 1);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->format == SDPA_CACHE_E4M3;
  if (cache->d == 128) {
    if (e4m3) cache_append_kernel<128, kCacheE4m3><<<g, kCacheThreads, 0, cs>>>(a);
    else cache_append_kernel<128, kCacheBf16><<<g, kCacheThreads, 0, cs>>>(a);
  } else {
    if (e4m3) cache_append_kernel<64, kCacheE4m3><<<g, kCacheThreads, 0, cs>>>(a);
    else cache_append_kernel<64, kCacheBf16><<<g, kCacheThreads, 0, cs>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

sdpa_status_t sdpa_cache_gather(const sdpa_kv_cache* cache, int64_t B, const int32_t* page_table,
                                int64_t table_width, int64_t table_b, const int32_t* cu_seqlens,
                                int64_t total, void* k, void* v, int64_t kv_t, int64_t kv_h,
                                void* stream) {
  GatherArgs a{};
  const sdpa_status_t st = check_cache(cache, a.c);
  if (st != SDPA_OK) return st;
  if (B < 1 || total < 0 || !page_table || table_width < 1 || !row_step(table_b, table_width) || !cu_seqlens ||
      (reinterpret_cast<uintptr_t>(page_table) & 3u) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
    return SDPA_ERR_INVALID_ARG;
  if (B > 65535 || total >= (1ll << 30) || table_width >= (1ll << 31)) return SDPA_ERR_UNSUPPORTED;
  if (total == 0) return SDPA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !good_stride(kv_t, 8) || !good_stride(kv_h, 8))
    return SDPA_ERR_INVALID_ARG;
  a.B = static_cast<int>(B);
  a.table = page_table;
  a.width = table_width;
  a.table_b = table_b;
  a.cu = cu_seqlens;
  a.total = total;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.kv_t = kv_t;
  a.kv_h = kv_h;
  a.rows = cache_rows(total);
  if (!a.rows) return SDPA_ERR_CUDA;
  const dim3 g(static_cast<unsigned>((total + a.rows - 1) / a.rows), 2);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->format == SDPA_CACHE_E4M3;
  if (cache->d == 128) {
    if (e4m3) cache_gather_kernel<128, kCacheE4m3><<<g, kCacheThreads, 0, cs>>>(a);
    else cache_gather_kernel<128, kCacheBf16><<<g, kCacheThreads, 0, cs>>>(a);
  } else {
    if (e4m3) cache_gather_kernel<64, kCacheE4m3><<<g, kCacheThreads, 0, cs>>>(a);
    else cache_gather_kernel<64, kCacheBf16><<<g, kCacheThreads, 0, cs>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

size_t sdpa_tree_fwd_workspace_size(const sdpa_tree* tree, const sdpa_kv_cache* cache) {
  CacheView v;
  TreePlan pl;
  return check_tree(tree, cache, v, pl) == SDPA_OK ? pl.total : 0;
}

sdpa_status_t sdpa_tree_fwd(const sdpa_tree* t, const sdpa_kv_cache* cache, const void* q,
                            const sdpa_bias_desc* bias, float scale, void* o, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  CacheView v;
  TreePlan pl;
  const sdpa_status_t st = check_tree(t, cache, v, pl);
  if (st != SDPA_OK) return st;
  if (!std::isfinite(scale)) return SDPA_ERR_INVALID_ARG;
  if (!q || !o || !lse || !aligned16(q) || !aligned16(o) || !aligned16(lse))
    return SDPA_ERR_INVALID_ARG;
  TreeArgs a;
  std::memset(&a, 0, sizeof(a));
  if (bias && bias->kind != SDPA_BIAS_NONE) {
    if (bias->kind == SDPA_BIAS_ALIBI) {
      if (!bias->ptr) return SDPA_ERR_INVALID_ARG;
      a.alibi_slopes = bias->ptr;
    } else if (bias->kind == SDPA_BIAS_T5) {
      const int nb = bias->num_buckets;
      if (!bias->ptr || nb < 2 || nb > 128 || (bias->bidirectional && nb % 2 != 0) ||
          !fill_t5(a.t5, nb, bias->max_distance, bias->bidirectional))
        return SDPA_ERR_INVALID_ARG;
      a.t5_table = bias->ptr;
      a.t5_buckets = nb;
    } else {
      return bias->kind == SDPA_BIAS_DENSE || bias->kind == SDPA_BIAS_REL ? SDPA_ERR_UNSUPPORTED
                                                                         : SDPA_ERR_INVALID_ARG;
    }
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < pl.total)
    return SDPA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.q_t = t->q_t;
  a.q_h = t->q_h;
  a.o_t = t->o_t;
  a.o_h = t->o_h;
  a.B = static_cast<int>(t->B);
  a.T = static_cast<int>(t->T);
  a.max_nodes = static_cast<int>(t->max_nodes);
  a.Hq = static_cast<int>(t->Hq);
  a.Hkv = v.Hkv;
  a.G = a.Hq / a.Hkv;
  a.cu = t->cu_nodes;
  a.ctx = t->ctx_lens;
  a.table = t->page_table;
  a.width = t->table_width;
  a.table_b = t->table_b;
  a.mask = t->tree_mask;
  a.wl = clamp_window(t->window_left, 1ll << 30);
  a.page_size = v.page_size;
  a.page_shift = v.page_shift;
  a.num_pages = v.num_pages;
  a.ks = v.ks;
  a.vs = v.vs;
  a.ss_page = v.ss_page;
  a.ss_head = v.ss_head;
  a.scale_log2 = scale * kLog2e;
  a.part_ml = reinterpret_cast<float2*>(ws + pl.ml);
  a.part_o = reinterpret_cast<float*>(ws + pl.o);
  a.wait_limit_ns = g_wait_limit_ns;
  const bool e4m3 = cache->format == SDPA_CACHE_E4M3;
  a.box_rows = std::min(v.page_size, kTreeKeys);
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, cache->k, cache, a.box_rows) ||
      !make_cache_map(&mv, cache->v, cache, a.box_rows))
    return SDPA_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->d == 128)
    e = e4m3 ? dispatch_tree_bias<128, kCacheE4m3>(a, mk, mv, cs)
             : dispatch_tree_bias<128, kCacheBf16>(a, mk, mv, cs);
  else
    e = e4m3 ? dispatch_tree_bias<64, kCacheE4m3>(a, mk, mv, cs)
             : dispatch_tree_bias<64, kCacheBf16>(a, mk, mv, cs);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

sdpa_status_t sdpa_spec_verify(const sdpa_verify* s, int32_t* path, int32_t* accepted,
                               int32_t* next_token, void* stream) {
  if (!s || s->B < 1 || s->N < 1 || s->V < 1) return SDPA_ERR_INVALID_ARG;
  if (s->N > kVerifyMaxNodes || s->V >= (1ll << 30) || s->B > (1ll << 24)) return SDPA_ERR_UNSUPPORTED;
  if (!s->target || !s->u_sample || !path || !accepted || !next_token) return SDPA_ERR_INVALID_ARG;
  if (s->N > 1 && (!s->draft || !s->tokens || !s->u_accept)) return SDPA_ERR_INVALID_ARG;
  const void* ptrs[] = {s->target, s->draft, s->tokens, s->parents, s->u_accept, s->u_sample,
                        path, accepted, next_token};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return SDPA_ERR_INVALID_ARG;
  const int64_t st[] = {s->target_b, s->target_n, s->draft_b, s->draft_n};
  for (int64_t x : st)
    if (x < 0 || x >= (1ll << 38)) return SDPA_ERR_INVALID_ARG;
  VerifyArgs a{};
  a.B = static_cast<int>(s->B);
  a.N = static_cast<int>(s->N);
  a.V = static_cast<int>(s->V);
  a.t_b = s->target_b;
  a.t_n = s->target_n;
  a.d_b = s->draft_b;
  a.d_n = s->draft_n;
  a.target = s->target;
  a.draft = s->draft;
  a.tokens = s->tokens;
  a.parents = s->parents;
  a.u_accept = s->u_accept;
  a.u_sample = s->u_sample;
  a.path = path;
  a.accepted = accepted;
  a.next_token = next_token;
  a.wait_limit_ns = g_wait_limit_ns;
  // a CTA of the cluster per 4096 entries of the vocabulary, up to eight
  int cluster = 1;
  while (cluster < kVerifyMaxCluster && cluster * 4096ll < s->V) cluster *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * cluster);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool held = s->V <= static_cast<int64_t>(cluster) * kVerifyThreads * kVerifyHeld;
  const cudaError_t e = held ? cudaLaunchKernelEx(&cfg, spec_verify_kernel<true>, a)
                             : cudaLaunchKernelEx(&cfg, spec_verify_kernel<false>, a);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

sdpa_status_t sdpa_serve_read_device_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SDPA_ERR_CUDA;
  unsigned int h = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&h, g_device_status, sizeof(h)) != cudaSuccess) return SDPA_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(zero)) != cudaSuccess) return SDPA_ERR_CUDA;
  if (h & kStatusTimeout) return SDPA_ERR_TIMEOUT;
  if (h & (kStatusMisaligned | kStatusBadSeqlens)) return SDPA_ERR_UNSUPPORTED;
  return SDPA_OK;
}

void sdpa_serve_set_wait_limit_ns(uint64_t ns) { g_wait_limit_ns = ns < 1000 ? 1000 : ns; }

}  // extern "C"
