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
// per element; gather the reverse).  A row is spread over the lanes of a part
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
};

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;  // rows in flight per lane group

// One lane group (D / 8 lanes, 8 elements each) per (token, head) row of K or
// V; blockIdx.y picks K or V.
template <int D, int FMT>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kAppendThreads / kLanes;
  const bool is_v = blockIdx.y != 0;
  const __nv_bfloat16* src = is_v ? a.v : a.k;
  const int lane = threadIdx.x % kLanes;
  const int64_t n_rows = a.T * a.c.Hkv;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kGroups * kAppendRows) +
                     threadIdx.x / kLanes;
  const int64_t n_slots = a.c.num_pages << a.c.page_shift;
  uint4 x[kAppendRows];
  int64_t slot[kAppendRows];
  int head[kAppendRows];
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int64_t r = r0 + static_cast<int64_t>(i) * kGroups;
    slot[i] = -1;
    x[i] = make_uint4(0, 0, 0, 0);
    if (r < n_rows) {
      const int64_t t = r / a.c.Hkv;
      head[i] = static_cast<int>(r - t * a.c.Hkv);
      slot[i] = a.slots[t];
      x[i] = *reinterpret_cast<const uint4*>(src + t * a.kv_t + head[i] * a.kv_h + lane * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    if (slot[i] >= n_slots) {
      atomicOr(&g_device_status, kStatusBadSeqlens);
      slot[i] = -1;
    }
    const int64_t page = slot[i] >> a.c.page_shift;
    const int row = static_cast<int>(slot[i] & (a.c.page_size - 1));
    if (FMT == kCacheBf16) {
      if (slot[i] >= 0) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? a.c.v : a.c.k) +
                             page * a.c.s_page + head[i] * a.c.s_head + row * a.c.s_row;
        *reinterpret_cast<uint4*>(dst + lane * 8) = x[i];
      }
    } else {
      // largest finite magnitude: bf16 magnitudes order as their bits
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
        m = max(m, lo < 0x7f80u ? lo : 0u);
        m = max(m, hi < 0x7f80u ? hi : 0u);
      }
#pragma unroll
      for (int s = kLanes / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(~0u, m, s));
      const uint32_t e = e4m3_scale_byte(__uint_as_float(m << 16));
      // 2^(127 - e): e in 1 .. 254 keeps it a normal float except at 254
      const float inv = e8m0_float(254u - e);
      if (slot[i] >= 0) {
        uint8_t* dst = static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + page * a.c.s_page +
                       head[i] * a.c.s_head + row * a.c.s_row;
        *reinterpret_cast<uint2*>(dst + lane * 8) = bf16x8_to_e4m3(x[i], inv);
        if (lane == 0)
          (is_v ? a.c.vs : a.c.ks)[page * a.c.ss_page + head[i] * a.c.ss_head + row] =
              static_cast<uint8_t>(e);
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
};

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 16;  // packed rows per CTA

// kGatherRows packed rows of all heads, K (blockIdx.y = 0) or V per CTA.  The
// first kGatherRows threads find their row's sequence (binary search in
// cu_seqlens) and page; then lane groups copy (row, head) pieces.
template <int D, int FMT>
__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const GatherArgs a) {
  __shared__ int64_t cell[kGatherRows];   // page * page_size + row, or -1
  const bool is_v = blockIdx.y != 0;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGatherRows;
  if (threadIdx.x < kGatherRows) {
    const int64_t r = r0 + threadIdx.x;
    int64_t at = -1;
    if (r < a.total && r < a.cu[a.B]) {
      int lo = 0, hi = a.B;  // cu[lo] <= r < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= r) lo = mid; else hi = mid;
      }
      const int64_t pos = r - a.cu[lo];
      const int64_t col = pos >> a.c.page_shift;
      int64_t page = -1;
      if (pos >= 0 && r < a.cu[lo + 1] && col < a.width) page = a.table[lo * a.table_b + col];
      if (page >= 0 && page < a.c.num_pages)
        at = (page << a.c.page_shift) + (pos & (a.c.page_size - 1));
      else
        atomicOr(&g_device_status, kStatusBadSeqlens);
    }
    cell[threadIdx.x] = at;
  }
  __syncthreads();
  constexpr int kLanes = FMT == kCacheBf16 ? D / 8 : D / 16;  // 16 stored bytes per lane
  const int n = kGatherRows * a.c.Hkv * kLanes;
  constexpr int kFlight = 4;
  for (int base = threadIdx.x; base < n; base += kFlight * kGatherThreads) {
    uint4 x[kFlight];
    __nv_bfloat16* dst[kFlight];
    uint32_t e[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int it = base + f * kGatherThreads;
      dst[f] = nullptr;
      if (it >= n) continue;
      const int lane = it % kLanes;
      const int rh = it / kLanes;
      const int row = rh / a.c.Hkv, h = rh - row * a.c.Hkv;
      const int64_t at = cell[row];
      if (at < 0) continue;
      const int64_t page = at >> a.c.page_shift;
      const int in = static_cast<int>(at & (a.c.page_size - 1));
      const int64_t off = page * a.c.s_page + h * a.c.s_head + in * a.c.s_row;
      dst[f] = (is_v ? a.v : a.k) + (r0 + row) * a.kv_t + h * a.kv_h;
      if (FMT == kCacheBf16) {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? a.c.v : a.c.k) + off;
        x[f] = *reinterpret_cast<const uint4*>(src + lane * 8);
        dst[f] += lane * 8;
      } else {
        const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.c.v : a.c.k) + off;
        x[f] = *reinterpret_cast<const uint4*>(src + lane * 16);
        e[f] = (is_v ? a.c.vs : a.c.ks)[page * a.c.ss_page + h * a.c.ss_head + in];
        dst[f] += lane * 16;
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (!dst[f]) continue;
      if (FMT == kCacheBf16) {
        *reinterpret_cast<uint4*>(dst[f]) = x[f];
      } else {
        const float s = e8m0_float(e[f]);
        const uint32_t w[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = e4m3x2_floats(w[j] & 0xffffu), hi = e4m3x2_floats(w[j] >> 16);
          o[2 * j] = pack_bf16x2(lo.x * s, lo.y * s);
          o[2 * j + 1] = pack_bf16x2(hi.x * s, hi.y * s);
        }
        *reinterpret_cast<uint4*>(dst[f]) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst[f] + 8) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace sdpa
