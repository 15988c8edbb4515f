// kv_cache.cuh -- a paged key / value cache in bf16 or e4m3: writing rows
// into it (quantising them on the way) and reading them back packed.
//
// An e4m3 row x is stored as codes x / 2^k rounded to nearest even and the
// byte k + 127, k the smallest integer with max |x| <= 448 * 2^k.  Scaling by
// a power of two is exact, so the only rounding is the one to e4m3 (at most
// 2^-4 of the value, half a step of its 3 mantissa bits; a value below 2^-6 of
// the scale by at most 2^-10 of it).
//
// Both kernels are bound by DRAM (append, e4m3: 2 bytes read and 1 written
// per element; gather the reverse).  Measured: append of 32 k rows of 8 heads of
// 128 as e4m3 42 us, 4.7 TB/s (71 % of a copy's rate; tried beside 41 us on
// another day: eight rows in flight per thread instead of four 43 us, CTAs that
// stay and walk the rows with the next rows' places read ahead 49 us); gather of 485 MB, two thirds of it written,
// 104 us, 4.7 TB/s (a plain fill of this GPU's memory reaches 3.8 TB/s, at which
// the written part alone takes 85 us); calls of a few rows 3 - 5 us, latency.
// A row is spread over the lanes of a part
// of a warp in 16-byte pieces, so its maximum is a few shuffles and every
// access is a full vector.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "sm100.cuh"

namespace sdpa {

constexpr int kCacheBf16 = 0, kCacheE4m3 = 1;

struct CacheView {
  void* k;
  void* v;
  uint8_t* ks;
  uint8_t* vs;
  int64_t num_pages;
  int page_size, page_shift;
  int Hkv;
  int64_t s_page, s_head, s_row;  // elements
  int64_t ss_page, ss_head;       // scales
};

// Byte e of the smallest power of two 2^(e - 127) with amax <= 448 of it, for
// finite amax >= 0: with amax = m 2^t, 1 <= m < 2, and 448 = 1.75 * 2^8 that
// is t - 8, or t - 7 when m > 1.75.
__device__ __forceinline__ uint32_t e4m3_scale_byte(float amax) {
  if (amax == 0.f) return 127u;
  const uint32_t u = __float_as_uint(amax);
  int t = static_cast<int>(u >> 23) - 127;
  uint32_t m = u & 0x7fffffu;
  if (t == -127) {  // bf16 subnormal
    const int z = __clz(m) - 8;
    t = -126 - z;
    m = (m << z) & 0x7fffffu;
  }
  const int k = t - 8 + (m > 0x600000u ? 1 : 0) + 127;
  return static_cast<uint32_t>(min(max(k, 1), 254));
}

// 2^(e - 127) of a scale byte 0 .. 254 as float32 (0: 2^-127, subnormal).
__device__ __forceinline__ float e8m0_float(uint32_t e) {
  return e ? __uint_as_float(e << 23) : __uint_as_float(0x400000u);
}

// 8 bf16 values (one uint4) times `inv` as 8 e4m3 codes.
__device__ __forceinline__ uint2 bf16x8_to_e4m3(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__uint_as_float(w[i] << 16) * inv,
                                 __uint_as_float(w[i] & 0xffff0000u) * inv);
    o[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

struct AppendArgs {
  CacheView c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t T, kv_t, kv_h;
  const int64_t* slots;
  int rows;  // per CTA, <= kCacheRows
};

// Both kernels: a CTA takes `rows` rows of K (blockIdx.y = 0) or V (1, where
// there is one) with all heads.  Its first threads find where each row lies in the cache; then a
// thread keeps one 16-byte piece of one head (several when the heads are
// many) and goes through the rows, four in flight.
constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 32;  // at most

struct CacheCells {
  int64_t off[kCacheRows];    // of the row in the cache, elements; < 0: none
  int64_t scale[kCacheRows];  // of its scales
};

__device__ __forceinline__ void cache_cell(CacheCells& s, int i, const CacheView& c, int64_t page, int row) {
  s.off[i] = page < 0 ? -1 : page * c.s_page + row * c.s_row;
  s.scale[i] = page * c.ss_page + row;
}

// One lane group (D / 8 lanes, 8 elements each) holds a row of one head.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kCacheThreads / kLanes;
  constexpr int kFlight = 4;
  __shared__ CacheCells cells;
  const bool is_v = blockIdx.y != 0;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.T - t0));
  if (threadIdx.x < rows) {
    const int64_t slot = a.slots[t0 + threadIdx.x];
    int64_t page = -1;
    if (slot >= a.c.num_pages << a.c.page_shift) atomicOr(&g_device_status, kStatusBadSeqlens);
    else if (slot >= 0) page = slot >> a.c.page_shift;
    cache_cell(cells, threadIdx.x, a.c, page, static_cast<int>(slot & (a.c.page_size - 1)));
  }
  __syncthreads();
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  // groups side by side over the heads, the rest over rows
  const int across = min(a.c.Hkv, kGroups);
  const int down = kGroups / across;
  const int sub = group / across;
  if (sub >= down) return;  // whole groups, after the last barrier
  const __nv_bfloat16* src0 = (is_v ? a.v : a.k) + t0 * a.kv_t + lane * 8;
  for (int h = group - sub * across; h < a.c.Hkv; h += across) {
    const __nv_bfloat16* src = src0 + h * a.kv_h;
    for (int r0 = sub; r0 < rows; r0 += down * kFlight) {
      uint4 x[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int r = r0 + f * down;
        x[f] = r < rows ? __ldcs(reinterpret_cast<const uint4*>(src + r * a.kv_t)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int r = r0 + f * down;
        const int64_t off = r < rows ? cells.off[r] : -1;
        if (FMT == kCacheBf16) {
          if (off >= 0)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? a.c.v : a.c.k) + off +
                                      h * a.c.s_head + lane * 8) = x[f];
        } else {
          // largest magnitude: bf16 magnitudes order as their bits
          const uint32_t w[4] = {x[f].x & 0x7fff7fffu, x[f].y & 0x7fff7fffu, x[f].z & 0x7fff7fffu,
                                 x[f].w & 0x7fff7fffu};
          constexpr uint32_t kGroup = kLanes == 16 ? 0xffffu : 0xffu;
          const uint32_t members = kGroup << (threadIdx.x & 31 & ~(kLanes - 1));
          uint32_t m2 = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
#pragma unroll
          for (int s = kLanes / 2; s > 0; s >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(members, m2, s));
          uint32_t m = max(m2 & 0xffffu, m2 >> 16);
          if (m >= 0x7f80u) {  // the largest finite one, then
            m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t lo = w[j] & 0xffffu, hi = w[j] >> 16;
              m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
#pragma unroll
            for (int s = kLanes / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(members, m, s));
          }
          const uint32_t e = e4m3_scale_byte(__uint_as_float(m << 16));
          if (off >= 0) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + off + h * a.c.s_head +
                                      lane * 8) = bf16x8_to_e4m3(x[f], e8m0_float(254u - e));
            if (lane == 0)
              (is_v ? a.c.vs : a.c.ks)[cells.scale[r] + h * a.c.ss_head] = static_cast<uint8_t>(e);
          }
        }
      }
    }
  }
}

// Two e4m3 codes as two floats.
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct GatherArgs {
  CacheView c;
  int B;
  const int32_t* table;
  int64_t width, table_b;
  const int32_t* cu;
  int64_t total;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int64_t kv_t, kv_h;
  int rows;
};

// The first threads find their row's sequence (binary search in cu_seqlens)
// and page.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_gather_kernel(const GatherArgs a) {
  constexpr int kLanes = FMT == kCacheBf16 ? D / 8 : D / 16;  // 16 stored bytes per lane
  constexpr int kGroups = kCacheThreads / kLanes;
  constexpr int kFlight = 4;
  __shared__ CacheCells cells;
  const bool is_v = blockIdx.y != 0;
  const int64_t r00 = static_cast<int64_t>(blockIdx.x) * a.rows;
  if (threadIdx.x < a.rows) {
    const int64_t r = r00 + threadIdx.x;
    int64_t page = -1, pos = 0;
    if (r < a.total && r < a.cu[a.B]) {
      int lo = 0, hi = a.B;  // cu[lo] <= r < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= r) lo = mid; else hi = mid;
      }
      pos = r - a.cu[lo];
      const int64_t col = pos >> a.c.page_shift;
      if (pos >= 0 && r < a.cu[lo + 1] && col < a.width) page = a.table[lo * a.table_b + col];
      if (page < 0 || page >= a.c.num_pages) {
        atomicOr(&g_device_status, kStatusBadSeqlens);
        page = -1;
      }
    }
    cache_cell(cells, threadIdx.x, a.c, page, static_cast<int>(pos & (a.c.page_size - 1)));
  }
  __syncthreads();
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int across = min(a.c.Hkv, kGroups);
  const int down = kGroups / across;
  const int sub = group / across;
  if (sub >= down) return;
  __nv_bfloat16* dst0 = (is_v ? a.v : a.k) + r00 * a.kv_t;
  for (int h = group - sub * across; h < a.c.Hkv; h += across) {
    for (int r0 = sub; r0 < a.rows; r0 += down * kFlight) {
      uint4 x[kFlight];
      uint32_t e[kFlight];
      bool has[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int r = r0 + f * down;
        const int64_t off = r < a.rows ? cells.off[r] : -1;
        has[f] = off >= 0;
        if (!has[f]) continue;
        if (FMT == kCacheBf16) {
          x[f] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_v ? a.c.v : a.c.k) +
                                                       off + h * a.c.s_head + lane * 8));
        } else {
          x[f] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(is_v ? a.c.v : a.c.k) + off +
                                                       h * a.c.s_head + lane * 16));
          e[f] = (is_v ? a.c.vs : a.c.ks)[cells.scale[r] + h * a.c.ss_head];
        }
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (!has[f]) continue;
        __nv_bfloat16* dst = dst0 + (r0 + f * down) * a.kv_t + h * a.kv_h;
        if (FMT == kCacheBf16) {
          __stcs(reinterpret_cast<uint4*>(dst + lane * 8), x[f]);
        } else {
          const float s = e8m0_float(e[f]);
          const uint64_t s2 = f2_pack(s, s);
          const uint32_t w[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 v = e4m3x2_floats(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
            float y0, y1;
            f2_unpack(f2_mul(f2_pack(v.x, v.y), s2), y0, y1);
            o[j] = pack_bf16x2(y0, y1);
          }
          __stcs(reinterpret_cast<uint4*>(dst + lane * 16), make_uint4(o[0], o[1], o[2], o[3]));
          __stcs(reinterpret_cast<uint4*>(dst + lane * 16 + 8), make_uint4(o[4], o[5], o[6], o[7]));
        }
      }
    }
  }
}

}  // namespace sdpa
