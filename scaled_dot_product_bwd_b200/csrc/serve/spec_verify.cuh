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
// the vocabulary.  A typical sequence therefore reads one row pair, 8 V bytes,
// and the call is bound by latency: its chain of dependent loads, one cluster
// exchange per pass and the final search.  A cluster of CTAs shares a
// sequence's passes, so one sequence is not left to one SM's loads, and the
// partial sums travel through distributed shared memory inside one launch.
// All sums are float64 in a fixed order.
// Measured at 32000 tokens: a chain of 5 nodes 6.1 us, 32 trees of 16 nodes
// 16.2 us (tried when they took 14.7: cluster barriers instead of counted stores
// 16.2, node 0's rows read ahead of the nodes' numbers the same); 8 trees of 16
// nodes at 128256 tokens, whose passes read the rows again, 53 us.
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
  uint64_t wait_limit_ns;
};

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxNodes = 64;
constexpr int kVerifyMaxCluster = 8;
constexpr int kVerifyHeld = 8;  // entries of a CTA's piece that a thread keeps in registers

// A sum Z of what a rejection left (1 for a sum of 0), and 1 / Z.
struct VerifySum {
  double z, inv;
};

// t / Z: the product with 1 / Z and one step by its residual t - w Z, which an
// fma gives exactly (Markstein, IBM J. Res. Dev. 34, 1990).  A quotient that is
// a float64 number comes out as itself, so ties stay ties; t * (1 / Z) alone,
// rounded twice, need not be it, and a division takes ten times as long (32 trees
// of 16 nodes 44 us).
__device__ __forceinline__ double verify_quotient(double t, const VerifySum& s) {
  const double w = t * s.inv;
  return fma(fma(-w, s.z, t), s.inv, w);
}

// max(w - q, 0) with w = t / Z (t itself for the first rejection, w = p)
__device__ __forceinline__ double verify_left(double w, float q) {
  return fmax(w - static_cast<double>(q), 0.0);
}

// What m rejections leave of x: t_m = max(w_{m-1} - q, 0), unnormalised, with
// w_j = t_j / Z_j; m = 0: p itself.
__device__ __forceinline__ double verify_weight(float p, float q, int m, const VerifySum* z) {
  double t = p;
  for (int j = 1; j <= m; ++j) t = verify_left(j > 1 ? verify_quotient(t, z[j - 1]) : t, q);
  return t;
}

// x to `sum` of CTA `to` of the cluster, counted by its barrier `bar`.
__device__ __forceinline__ void verify_send(uint32_t sum, uint32_t bar, int to, double x) {
  asm volatile(
      "{\n\t.reg .b32 s, b;\n\t"
      "mapa.shared::cluster.u32 s, %0, %2;\n\t"
      "mapa.shared::cluster.u32 b, %1, %2;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.f64 [s], %3, [b];\n\t}" ::"r"(sum),
      "r"(bar), "r"(to), "d"(x)
      : "memory");
}

// Waits for a phase of `bar` that other CTAs complete; false (and a status) at the limit.
__device__ __forceinline__ bool verify_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t k = 0;; ++k) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if ((k & 63u) == 0) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > limit_ns) {
        atomicOr(&g_device_status, kStatusTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
  return x;
}

// The cluster's CTAs hold equal consecutive pieces of the vocabulary, a CTA's
// warps equal consecutive pieces of its own.  HELD: a warp's piece fits its
// threads' registers (kVerifyHeld entries each), so a node's p and q are read
// once for all its rejections; else every pass reads them again and computes
// the weights from the earlier sums.
// Sums travel as stores that complete on the receiving CTA's mbarrier, one
// barrier per parity of the passes: a warp sends its sum of pass p + 1 once it
// has read those of pass p, so none of pass p + 2 arrives before all of pass p
// are read.
template <bool HELD>
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
  __shared__ VerifySum z[kVerifyMaxNodes + 1];          // by rejections of the current node
  // every warp's sum of the cluster, by two passes in turn
  __shared__ double sums[2][kVerifyMaxCluster * kVerifyWarps];
  __shared__ __align__(8) uint64_t bars[2];

  if (tid == 0) {
    mbar_init(smem_u32(bars), 1);
    mbar_init(smem_u32(bars + 1), 1);
    fence_mbar_init();
  }
  __syncwarp();
  // (a CTA's shared memory may be written to once it has started and its
  // barriers stand: arrived at here, waited for after the nodes' loads)
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  const float u_sample = a.u_sample[b];  // (early: nothing waits for it at the end)
  if (tid < kVerifyMaxNodes) kids[tid] = 0;
  __syncthreads();
  if (tid < 64) {
    bool ok = false;
    if (tid > 0 && tid < a.N) {
      const int64_t at = static_cast<int64_t>(b) * a.N + tid;
      const int parent = a.parents ? a.parents[at] : tid - 1;
      const int x = a.tokens[at];
      const float u = a.u_accept[at];
      if (parent >= tid) atomicOr(&g_device_status, kStatusBadSeqlens);
      if (parent >= 0 && parent < tid) {
        float p = 0.f, q = 0.f;
        if (x >= 0 && x < a.V) {
          p = a.target[b * a.t_b + parent * a.t_n + x];
          q = a.draft[b * a.d_b + parent * a.d_n + x];
        } else {
          atomicOr(&g_device_status, kStatusBadSeqlens);
        }
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
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  const unsigned long long ok_first = first_ok[0] | (static_cast<unsigned long long>(first_ok[1]) << 32);

  const int chunk = (a.V + C - 1) / C;
  const int seg = (chunk + kVerifyWarps - 1) / kVerifyWarps;
  const int cta_hi = static_cast<int>(min(static_cast<int64_t>(a.V), static_cast<int64_t>(rank + 1) * chunk));
  const int lo = static_cast<int>(min(static_cast<int64_t>(cta_hi),
                                      static_cast<int64_t>(rank) * chunk + static_cast<int64_t>(warp) * seg));
  const int hi = min(cta_hi, lo + seg);
  int passes = 0;
  bool ok = true;  // no wait has run out

  // HELD: entry lo + lane + 32 i of target[at] (then of what is left of it)
  // and of draft[at]
  double held[HELD ? kVerifyHeld : 1];
  float drawn[HELD ? kVerifyHeld : 1];

  // Sum over the vocabulary of what m rejections leave of target[at].
  auto sum_pass = [&](int at, int m) -> double {
    const float* p = a.target + b * a.t_b + at * a.t_n;
    const float* q = m ? a.draft + b * a.d_b + at * a.d_n : p;
    double acc = 0.0;
    if constexpr (HELD) {
      if (m <= 1) {
#pragma unroll
        for (int i = 0; i < kVerifyHeld; ++i) {
          const int x = lo + lane + 32 * i;
          drawn[i] = m && x < hi ? q[x] : 0.f;
          held[i] = x < hi ? static_cast<double>(p[x]) : 0.0;
        }
      }
      const VerifySum s = m > 1 ? z[m - 1] : VerifySum{1.0, 1.0};
#pragma unroll
      for (int i = 0; i < kVerifyHeld; ++i) {
        if (m > 0) held[i] = verify_left(m > 1 ? verify_quotient(held[i], s) : held[i], drawn[i]);
        acc += held[i];
      }
    } else {
      for (int x0 = lo + lane; x0 < hi; x0 += 32 * 8) {
        float pv[8], qv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int x = x0 + 32 * i;
          pv[i] = x < hi ? p[x] : 0.f;
          qv[i] = m && x < hi ? q[x] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc += verify_weight(pv[i], qv[i], m, z);
      }
    }
    acc = warp_sum(acc);
    const double* mine = sums[passes & 1];
    const uint32_t bar = smem_u32(bars + (passes & 1));
    if (tid == 0) mbar_expect_tx(bar, C * kVerifyWarps * 8);
    if (lane < C) verify_send(smem_u32(mine + rank * kVerifyWarps + warp), bar, lane, acc);
    if (ok) ok = __all_sync(~0u, verify_wait(bar, (passes >> 1) & 1, a.wait_limit_ns));
    // all warps of the cluster add the same numbers in the same order
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < kVerifyMaxCluster * kVerifyWarps / 32; ++i) {
      const int k = lane + 32 * i;
      if (k < C * kVerifyWarps) total += mine[k];
    }
    ++passes;
    return warp_sum(total);
  };

  // every thread of the cluster walks alike (until a wait runs out)
  int at = 0, m = 0, n_acc = 0;
  unsigned long long left = a.N > 1 ? kids[0] : 0ull;
  if (rank == 0 && tid == 0) a.path[static_cast<int64_t>(b) * a.N] = 0;
  double total = 0.0;
  while (left && ok) {
    const int n = __ffsll(static_cast<long long>(left)) - 1;
    left &= left - 1;
    bool taken;
    if (m == 0) {
      taken = (ok_first >> n) & 1ull;
    } else {
      const double w = verify_quotient(verify_weight(px[n], qx[n], m, z), z[m]);
      taken = static_cast<double>(ux[n]) * qx[n] < w;
    }
    if (taken) {
      at = n;
      m = 0;
      left = kids[n];
      ++n_acc;
      if (rank == 0 && tid == 0) a.path[static_cast<int64_t>(b) * a.N + n_acc] = n;
    } else {
      total = sum_pass(at, ++m);
      // (z[m] was last read before the pass's barrier)
      if (tid == 0) z[m] = total > 0.0 ? VerifySum{total, 1.0 / total} : VerifySum{1.0, 1.0};
      ok = __syncthreads_and(ok);
    }
  }
  if (m > 0 && !(total > 0.0)) m = 0;  // nothing left: the target itself
  if (m == 0 && ok) total = sum_pass(at, 0);
  if (!ok) {
    // stay until no other CTA can send here any more (one that has left counts
    // as arrived); one whose waits all ended has all that was sent to it
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
    return;
  }
  if (rank == 0) {
    for (int i = n_acc + 1 + tid; i < a.N; i += kVerifyThreads)
      a.path[static_cast<int64_t>(b) * a.N + i] = -1;
    if (tid == 0) a.accepted[b] = n_acc;
  }

  // the warp piece in which the cumulative weight first exceeds u * total;
  // where rounding (or u = 1) leaves none, the last piece with any weight.
  // Every warp scans all pieces' sums, four neighbours to a lane.
  const double aim = static_cast<double>(u_sample) * total;
  const double* last_sums = sums[(passes + 1) & 1];
  constexpr int kPer = kVerifyMaxCluster * kVerifyWarps / 32;
  double part[kPer], mine = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane * kPer + i;
    part[i] = k < C * kVerifyWarps ? last_sums[k] : 0.0;
    mine += part[i];
  }
  double before = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const double y = __shfl_up_sync(~0u, before, s);
    if (lane >= s) before += y;
  }
  before -= mine;
  int pick = -1, last = -1;       // pieces of this lane
  double base = 0.0, base_last = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (part[i] > 0.0) {
      last = lane * kPer + i;
      base_last = before;
      if (pick < 0 && before + part[i] > aim) {
        pick = last;
        base = before;
      }
    }
    before += part[i];
  }
  const unsigned int picks = __ballot_sync(~0u, pick >= 0), lasts = __ballot_sync(~0u, last >= 0);
  if (!lasts) {  // no weight anywhere
    if (rank == 0 && tid == 0) a.next_token[b] = 0;
    return;
  }
  const int from = picks ? __ffs(picks) - 1 : 31 - __clz(lasts);
  const int piece = __shfl_sync(~0u, picks ? pick : last, from);
  double run = __shfl_sync(~0u, picks ? base : base_last, from);
  if (piece != rank * kVerifyWarps + warp) return;
  const float* p = a.target + b * a.t_b + at * a.t_n;
  const float* q = m ? a.draft + b * a.d_b + at * a.d_n : p;
  int token = -1, seen = 0;
  auto search = [&](int x0, double w) {
    double cum = w;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const double y = __shfl_up_sync(~0u, cum, s);
      if (lane >= s) cum += y;
    }
    const unsigned int some = __ballot_sync(~0u, w > 0.0);
    const unsigned int over = __ballot_sync(~0u, w > 0.0 && run + cum > aim);
    if (some) seen = x0 + 31 - __clz(some);
    if (over) token = x0 + __ffs(over) - 1;
    run += __shfl_sync(~0u, cum, 31);
  };
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kVerifyHeld; ++i)
      if (token < 0) search(lo + 32 * i, held[i]);
  } else {
    for (int x0 = lo; x0 < hi && token < 0; x0 += 32) {
      const int x = x0 + lane;
      search(x0, x < hi ? verify_weight(p[x], m ? q[x] : 0.f, m, z) : 0.0);
    }
  }
  if (lane == 0) a.next_token[b] = token >= 0 ? token : seen;
}

}  // namespace sdpa
