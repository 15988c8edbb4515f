// rope.cuh -- rotary positions of Q and K in one launch, and (turning the
// other way) their gradient.
//
// A pair (x1, x2) of a head turns by t = position * freq_i:
//   y1 = a (x1 cos t - x2 sin t),  y2 = a (x2 cos t + x1 sin t).
// The map is a scaled rotation, so its transpose -- the gradient -- is the
// rotation by -t with the same amplitude a.
//
// Bound by DRAM: every element is read and written once (4 bytes), against
// about 3 fp32 operations.  The angles belong to (token, pair) and serve all
// heads of q and k, so a CTA forms the rot / 2 sines and cosines of its
// tokens once in shared memory and then streams the heads in 16-byte pieces.
// Measured: 4 x 4096 tokens of 32 + 8 heads of 128, 336 MB in 57 us, 5.9 TB/s
// (89 % of a copy's rate); a decoding step of 8 tokens 2.7 us, all of it latency.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sm100.cuh"

namespace sdpa {

struct RopeArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  __nv_bfloat16* qo;
  __nv_bfloat16* ko;
  int64_t q_b, q_l, q_h, k_b, k_l, k_h, qo_b, qo_l, qo_h, ko_b, ko_l, ko_h;
  const int32_t* positions;
  int64_t pos_b, offset;
  const double* freqs;
  int L, Hq, H;          // H = query + KV heads
  int64_t tokens;        // B * L
  int half;              // rot / 2
  int per_cta;           // tokens per CTA, <= kRopeTokens
  float amplitude, sign; // sign = -1 turns back
};

constexpr int kRopeTokens = 16;   // per CTA, at most
constexpr int kRopeThreads = 256;
constexpr int kRopeFlight = 4;    // items (16 elements) in flight per thread

// How the pairs of a head lie in its 16-byte pieces.
enum RopeMode : int {
  kRopeHalf = 0,         // (x[i], x[i + half]), half a multiple of 8: two whole pieces
  kRopeInterleaved = 1,  // (x[2i], x[2i + 1]): inside one piece
  kRopeHalfAny = 2       // (x[i], x[i + half]), any half: partners through shared memory
};

// cos and sin of one (token, pair).  The angle is formed in float64 and
// reduced to a fraction of a turn there: at position 10^6 a float32 angle of
// the fastest pair would be off by up to 0.03 rad.
__device__ __forceinline__ float2 rope_cos_sin(const RopeArgs& a, int b, int l, int i) {
  const int64_t pos = a.positions ? a.positions[b * a.pos_b + l] : a.offset + l;
  const double turns = static_cast<double>(pos) * (a.freqs[i] * 0.15915494309189533577);
  float s, c;
  sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
  return make_float2(c * a.amplitude, s * a.amplitude * a.sign);
}

__device__ __forceinline__ void rope_turn(float2 cs, float& x1, float& x2) {
  const float y1 = x1 * cs.x - x2 * cs.y;
  x2 = x2 * cs.x + x1 * cs.y;
  x1 = y1;
}

__device__ __forceinline__ float2 bf16x2_floats(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Head h's row of token (b, l) in the inputs and outputs.
__device__ __forceinline__ void rope_row(const RopeArgs& a, int b, int l, int h,
                                         const __nv_bfloat16*& src, __nv_bfloat16*& dst) {
  if (h < a.Hq) {
    src = a.q + b * a.q_b + l * a.q_l + h * a.q_h;
    dst = a.qo + b * a.qo_b + l * a.qo_l + h * a.qo_h;
  } else {
    h -= a.Hq;
    src = a.k + b * a.k_b + l * a.k_l + h * a.k_h;
    dst = a.ko + b * a.ko_b + l * a.ko_l + h * a.ko_h;
  }
}

// An item is 16 elements of one head, read whole before any is written (the
// call may be in place).  A CTA's tokens are chosen so that its items are one
// batch of four per thread: they are on their way while the angles are formed.
template <int D, int MODE>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeArgs a) {
  __shared__ __align__(16) float2 cs[kRopeTokens][D / 2];
  __shared__ __align__(16) __nv_bfloat16 rows[MODE == kRopeHalfAny ? kRopeThreads * 8 : 8];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.per_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.per_cta), a.tokens - t0));
  const int tid = threadIdx.x;
  __shared__ int row_b[kRopeTokens], row_l[kRopeTokens];
  if (tid < nt) {
    row_b[tid] = static_cast<int>((t0 + tid) / a.L);
    row_l[tid] = static_cast<int>((t0 + tid) - static_cast<int64_t>(row_b[tid]) * a.L);
  }
  __syncthreads();
  auto angles = [&] {
    for (int x = tid; x < nt * a.half; x += kRopeThreads) {
      const int t = x / a.half;
      const int i = x - t * a.half;
      // kRopeHalf: pairs i, i + 1 of item c (8 c + 2 e, + 1) at place e of the
      // items' rows, so that neighbouring items' threads read neighbouring words
      const int at = MODE == kRopeHalf ? ((i & 7) >> 1) * (D / 8) + (i >> 3) * 2 + (i & 1) : i;
      cs[t][at] = rope_cos_sin(a, row_b[t], row_l[t], i);
    }
    __syncthreads();
  };

  if constexpr (MODE == kRopeHalfAny) {
    // 8 elements per lane; a warp holds 256 / D heads' rows
    angles();
    constexpr int kLanes = D / 8;
    const int warp_rows = 32 / kLanes;
    __nv_bfloat16* mine = rows + (tid / 32) * 256;
    const int lane = tid & 31, c = lane % kLanes, sub = lane / kLanes;
    const int n_rows = nt * a.H;
    for (int r0 = (tid / 32) * warp_rows; r0 < n_rows; r0 += (kRopeThreads / 32) * warp_rows) {
      const int r = r0 + sub;
      const __nv_bfloat16* src = nullptr;
      __nv_bfloat16* dst = nullptr;
      int t = 0;
      if (r < n_rows) {
        t = r / a.H;
        rope_row(a, row_b[t], row_l[t], r - t * a.H, src, dst);
        *reinterpret_cast<uint4*>(mine + sub * D + c * 8) =
            *reinterpret_cast<const uint4*>(src + c * 8);
      }
      __syncwarp();
      uint4 out;
      if (r < n_rows) {
        __nv_bfloat16 y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = c * 8 + e;
          const __nv_bfloat16 raw = mine[sub * D + j];
          y[e] = raw;
          if (j < 2 * a.half) {
            const bool first = j < a.half;
            const int i = first ? j : j - a.half;
            float x1 = __bfloat162float(first ? raw : mine[sub * D + i]);
            float x2 = __bfloat162float(first ? mine[sub * D + j + a.half] : raw);
            rope_turn(cs[t][i], x1, x2);
            y[e] = __float2bfloat16(first ? x1 : x2);
          }
        }
        out = make_uint4(0, 0, 0, 0);
        memcpy(&out, y, 16);
        *reinterpret_cast<uint4*>(dst + c * 8) = out;
      }
      __syncwarp();
    }
  } else {
    constexpr int kItems = D / 16;  // per head
    const int per_token = a.H * kItems;
    const int n_items = nt * per_token;
    const int turned = a.half / 8;  // kRopeHalf: items of a head that turn
    for (int base = tid; base - tid < n_items; base += kRopeFlight * kRopeThreads) {
      uint4 xa[kRopeFlight], xb[kRopeFlight];
      __nv_bfloat16* pa[kRopeFlight];
      int tk[kRopeFlight], off_b[kRopeFlight], ci[kRopeFlight];
#pragma unroll
      for (int f = 0; f < kRopeFlight; ++f) {
        const int it = base + f * kRopeThreads;
        pa[f] = nullptr;
        if (it < n_items) {
          const int t = it / per_token;
          const int rem = it - t * per_token;
          const int h = rem / kItems, c = rem % kItems;
          int ea, eb;
          if (MODE == kRopeInterleaved) {
            ea = c * 16;
            eb = ea + 8;
          } else if (c < turned) {
            ea = c * 8;
            eb = ea + a.half;
          } else {
            ea = c * 16;
            eb = ea + 8;
          }
          const __nv_bfloat16* src;
          __nv_bfloat16* dst;
          rope_row(a, row_b[t], row_l[t], h, src, dst);
          xa[f] = __ldcs(reinterpret_cast<const uint4*>(src + ea));
          xb[f] = __ldcs(reinterpret_cast<const uint4*>(src + eb));
          pa[f] = dst + ea;
          off_b[f] = eb - ea;
          tk[f] = t;
          ci[f] = c;
        }
      }
      if (base == tid) angles();  // under the first batch's loads
#pragma unroll
      for (int f = 0; f < kRopeFlight; ++f) {
        if (!pa[f]) continue;
        uint32_t* wa = reinterpret_cast<uint32_t*>(&xa[f]);
        uint32_t* wb = reinterpret_cast<uint32_t*>(&xb[f]);
        const float2* row = cs[tk[f]];
        if (MODE == kRopeInterleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = ci[f] * 8 + e;
            uint32_t& w = e < 4 ? wa[e] : wb[e - 4];
            if (i < a.half) {
              float2 x = bf16x2_floats(w);
              rope_turn(row[i], x.x, x.y);
              w = pack_bf16x2(x.x, x.y);
            }
          }
        } else if (ci[f] < turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 x1 = bf16x2_floats(wa[e]), x2 = bf16x2_floats(wb[e]);
            const float4 t4 = *reinterpret_cast<const float4*>(row + e * (D / 8) + ci[f] * 2);
            rope_turn(make_float2(t4.x, t4.y), x1.x, x2.x);
            rope_turn(make_float2(t4.z, t4.w), x1.y, x2.y);
            wa[e] = pack_bf16x2(x1.x, x1.y);
            wb[e] = pack_bf16x2(x2.x, x2.y);
          }
        }
        __stcs(reinterpret_cast<uint4*>(pa[f]), xa[f]);
        __stcs(reinterpret_cast<uint4*>(pa[f] + off_b[f]), xb[f]);
      }
    }
  }
}

}  // namespace sdpa
