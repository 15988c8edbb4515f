// spec_verify.cuh -- verification of a tree of drafted tokens by rejection
// sampling with given random numbers.
//
// At node `at` with target distribution p and draft distribution q, child x
// is accepted when u q(x) < w(x); a rejected child leaves
//   w <- max(w - q, 0) / Z,  Z = sum max(w - q, 0),
// starting from w = p.  The next token is drawn from the w that remains where
// the walk ends, by inverting its cumulative sum.
//
// Everything a first child's test needs is two numbers per node, read for
// all nodes at once; only a rejection (and the final draw) takes a pass over
// the vocabulary, and it recomputes w from p, q and the earlier sums Z instead
// of storing it.  A typical sequence therefore reads one row pair, 8 V bytes,
// and the call is bound by latency: its chain of dependent loads, one cluster
// exchange per pass and the final search.  A cluster of CTAs shares a
// sequence's passes, so one sequence is not left to one SM's loads, and the
// partial sums travel through distributed shared memory inside one launch.
// All sums are float64 in a fixed order.
#pragma once

#include <cooperative_groups.h>
#include <stdint.h>

#include "sm100.cuh"

namespace sdpa {

struct VerifyArgs {
  int B, N, V;
  int64_t t_b, t_n, d_b, d_n;
  const float* target;
  const float* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const float* u_accept;
  const float* u_sample;
  int32_t* path;
  int32_t* accepted;
  int32_t* next_token;
};

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxNodes = 64;
constexpr int kVerifyMaxCluster = 8;

// What m rejections leave of x: t_m = max(w_{m-1} - q, 0), unnormalised, with
// w_j = t_j * inv[j]; m = 0: p itself.
__device__ __forceinline__ double verify_weight(float p, float q, int m, const double* inv) {
  double t = p;
  for (int j = 1; j <= m; ++j) {
    if (j > 1) t *= inv[j - 1];
    t = fmax(t - static_cast<double>(q), 0.0);
  }
  return t;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
  return x;
}

// The cluster's CTAs hold equal consecutive pieces of the vocabulary, a CTA's
// warps equal consecutive pieces of its own.
__global__ void __launch_bounds__(kVerifyThreads) spec_verify_kernel(const VerifyArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  __shared__ unsigned long long kids[kVerifyMaxNodes];  // bit n: node n is a child
  __shared__ unsigned int first_ok[2];                  // bit n: n passes against w = p
  __shared__ float px[kVerifyMaxNodes], qx[kVerifyMaxNodes], ux[kVerifyMaxNodes];
  __shared__ double inv[kVerifyMaxNodes + 1];
  __shared__ double warp_tot[kVerifyWarps];
  __shared__ double cta_tot[2][kVerifyMaxCluster];      // written by every CTA of the cluster

  if (tid < kVerifyMaxNodes) kids[tid] = 0;
  __syncthreads();
  if (tid < 64) {
    bool ok = false;
    if (tid > 0 && tid < a.N) {
      const int64_t at = static_cast<int64_t>(b) * a.N + tid;
      const int parent = a.parents ? a.parents[at] : tid - 1;
      if (parent >= tid) atomicOr(&g_device_status, kStatusBadSeqlens);
      if (parent >= 0 && parent < tid) {
        const int x = a.tokens[at];
        float p = 0.f, q = 0.f;
        if (x >= 0 && x < a.V) {
          p = a.target[b * a.t_b + parent * a.t_n + x];
          q = a.draft[b * a.d_b + parent * a.d_n + x];
        } else {
          atomicOr(&g_device_status, kStatusBadSeqlens);
        }
        const float u = a.u_accept[at];
        px[tid] = p;
        qx[tid] = q;
        ux[tid] = u;
        ok = static_cast<double>(u) * q < static_cast<double>(p);
        atomicOr(&kids[parent], 1ull << tid);
      }
    }
    const unsigned int w = __ballot_sync(~0u, ok);
    if (lane == 0) first_ok[warp] = w;
  }
  __syncthreads();
  const unsigned long long ok_first = first_ok[0] | (static_cast<unsigned long long>(first_ok[1]) << 32);

  const int chunk = (a.V + C - 1) / C;
  const int seg = (chunk + kVerifyWarps - 1) / kVerifyWarps;
  const int cta_hi = static_cast<int>(min(static_cast<int64_t>(a.V), static_cast<int64_t>(rank + 1) * chunk));
  const int lo = static_cast<int>(min(static_cast<int64_t>(cta_hi),
                                      static_cast<int64_t>(rank) * chunk + static_cast<int64_t>(warp) * seg));
  const int hi = min(cta_hi, lo + seg);
  int passes = 0;

  // Sum over the vocabulary of what m rejections leave of target[at]: the
  // total, with this CTA's warp sums in warp_tot and every CTA's in cta_tot.
  auto sum_pass = [&](int at, int m) -> double {
    const float* p = a.target + b * a.t_b + at * a.t_n;
    const float* q = m ? a.draft + b * a.d_b + at * a.d_n : p;
    double acc = 0.0;
    for (int x0 = lo + lane; x0 < hi; x0 += 32 * 8) {
      float pv[8], qv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = x0 + 32 * i;
        pv[i] = x < hi ? p[x] : 0.f;
        qv[i] = m && x < hi ? q[x] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += verify_weight(pv[i], qv[i], m, inv);
    }
    acc = warp_sum(acc);
    __syncthreads();  // earlier readers of warp_tot
    if (lane == 0) warp_tot[warp] = acc;
    __syncthreads();
    double (*tot)[kVerifyMaxCluster] = cta_tot;
    if (tid < C) {
      double mine = 0.0;
      for (int w = 0; w < kVerifyWarps; ++w) mine += warp_tot[w];
      double* there = cluster.map_shared_rank(&tot[passes & 1][rank], tid);
      *there = mine;
    }
    cluster.sync();
    double total = 0.0;
    for (int r = 0; r < C; ++r) total += tot[passes & 1][r];
    ++passes;
    return total;
  };

  // every thread of the cluster walks alike
  int at = 0, m = 0, n_acc = 0;
  unsigned long long left = a.N > 1 ? kids[0] : 0ull;
  if (rank == 0 && tid == 0) a.path[static_cast<int64_t>(b) * a.N] = 0;
  double total = 0.0;
  while (left) {
    const int n = __ffsll(static_cast<long long>(left)) - 1;
    left &= left - 1;
    bool ok;
    if (m == 0) {
      ok = (ok_first >> n) & 1ull;
    } else {
      const double w = verify_weight(px[n], qx[n], m, inv) * inv[m];
      ok = static_cast<double>(ux[n]) * qx[n] < w;
    }
    if (ok) {
      at = n;
      m = 0;
      left = kids[n];
      ++n_acc;
      if (rank == 0 && tid == 0) a.path[static_cast<int64_t>(b) * a.N + n_acc] = n;
    } else {
      total = sum_pass(at, m + 1);
      ++m;
      __syncthreads();
      if (tid == 0) inv[m] = total > 0.0 ? 1.0 / total : 0.0;
      __syncthreads();
    }
  }
  if (m > 0 && !(total > 0.0)) m = 0;  // nothing left: the target itself
  if (m == 0) total = sum_pass(at, 0);
  if (rank == 0) {
    for (int i = n_acc + 1 + tid; i < a.N; i += kVerifyThreads)
      a.path[static_cast<int64_t>(b) * a.N + i] = -1;
    if (tid == 0) a.accepted[b] = n_acc;
  }

  // the piece in which the cumulative weight first exceeds u * total; where
  // rounding (or u = 1) leaves none, the last piece with any weight
  const double aim = static_cast<double>(a.u_sample[b]) * total;
  const double* tot = cta_tot[(passes - 1) & 1];
  int pick = -1, last = -1;
  double base = 0.0, base_last = 0.0, run = 0.0;
  for (int r = 0; r < C; ++r) {
    if (tot[r] > 0.0) {
      last = r;
      base_last = run;
      if (pick < 0 && run + tot[r] > aim) {
        pick = r;
        base = run;
      }
    }
    run += tot[r];
  }
  if (pick < 0) {
    pick = last;
    base = base_last;
  }
  if (pick < 0) {
    if (rank == 0 && tid == 0) a.next_token[b] = 0;
    return;
  }
  if (rank != pick) return;
  int wpick = -1, wlast = -1;
  double wbase = base, wbase_last = base;
  run = base;
  for (int w = 0; w < kVerifyWarps; ++w) {
    if (warp_tot[w] > 0.0) {
      wlast = w;
      wbase_last = run;
      if (wpick < 0 && run + warp_tot[w] > aim) {
        wpick = w;
        wbase = run;
      }
    }
    run += warp_tot[w];
  }
  if (wpick < 0) {
    wpick = wlast;
    wbase = wbase_last;
  }
  if (warp != wpick) return;
  const float* p = a.target + b * a.t_b + at * a.t_n;
  const float* q = m ? a.draft + b * a.d_b + at * a.d_n : p;
  int token = -1, seen = 0;
  for (int x0 = lo; x0 < hi && token < 0; x0 += 32) {
    const int x = x0 + lane;
    const double w = x < hi ? verify_weight(p[x], m ? q[x] : 0.f, m, inv) : 0.0;
    double cum = w;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const double y = __shfl_up_sync(~0u, cum, s);
      if (lane >= s) cum += y;
    }
    const unsigned int some = __ballot_sync(~0u, w > 0.0);
    const unsigned int over = __ballot_sync(~0u, w > 0.0 && wbase + cum > aim);
    if (some) seen = x0 + 31 - __clz(some);
    if (over) token = x0 + __ffs(over) - 1;
    wbase += __shfl_sync(~0u, cum, 31);
  }
  if (lane == 0) a.next_token[b] = token >= 0 ? token : seen;
}

}  // namespace sdpa
