// tree_verify.cu -- acceptance of drafted tokens against the target's
// probabilities (speculative sampling on a token tree).
//
// Method.  At a context with target distribution p and draft distribution q,
// the children are tried in index order.  What is still to be drawn is
// W = max(p - c q, 0) with mass a (at first c = 0, a = 1): child x is accepted
// when u q(x) a < W(x); a rejection takes a q away, W <- max(W - a q, 0).
// Since a, q >= 0 the nested maxima collapse, max(max(p - c q, 0) - a q, 0) =
// max(p - (c + a) q, 0), so W needs no storage: it is p, q and the scalar c,
// and one pass over the row gives the next a.  When no child is left the
// token is drawn from W: the least x whose cumulative W exceeds u sum(W).
// Without draft probabilities (q null: each draft is a point mass) a child is
// accepted when u a < W(x), and a rejection removes x and its mass.
//
// Rounding.  A decision sits on sums over the whole vocabulary, so they are
// held to about 2^-48: c is a pair of floats, each W(x) = p - c q is formed
// as an unevaluated pair hi + lo (the exact product by fma, the exact
// difference by Knuth's two-sum) and added into a pair accumulator.  That runs on the fp32 pipe;
// plain doubles would run at 1/64 of its rate here and bound the kernel.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "tree.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kStep = 128;  // elements of one warp step: 4 consecutive ones per lane

struct Pair {
  float hi, lo;
};

// acc + v in pair arithmetic (two-sum of the high parts).
__device__ __forceinline__ void add(Pair& acc, float hi, float lo) {
  const float s = acc.hi + hi;
  const float b = s - acc.hi;
  acc.lo += ((acc.hi - (s - b)) + (hi - b)) + lo;
  acc.hi = s;
}

__device__ __forceinline__ Pair warp_total(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, v.hi, o), lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
    // both partners form the same sum: two-sum is symmetric in its operands
    const float s = v.hi + hi, b = s - v.hi;
    const float e = (v.hi - (s - b)) + (hi - b);
    v.lo = (v.lo + lo) + e;
    v.hi = s;
  }
  return v;
}

__device__ __forceinline__ double value(const Pair& v) { return (double)v.hi + (double)v.lo; }

// max(p - (ch + cl) q, 0) as a pair.
__device__ __forceinline__ Pair left(float p, float q, float ch, float cl) {
  const float h = ch * q;
  const float e = fmaf(cl, q, fmaf(ch, q, -h));
  const float s = p - h, b = s - p;
  const float lo = ((p - (s - b)) - (h + b)) - e;
  const bool pos = s + lo > 0.f;
  // a NaN stays one, so that the total shows it
  return Pair{pos ? s : (s + lo != s + lo ? s : 0.f), pos ? lo : 0.f};
}

struct Shared {
  // node data, filled by rank 0 and copied by the others
  int parent[kMaxTree], token[kMaxTree];
  float u[kMaxTree + 1], pt[kMaxTree], qt[kMaxTree];
  double part[2][kCluster];  // slice totals of every CTA, alternating between passes
  double warp_sum[kWarps];
  int removed[kMaxTree];
};

// Row segment of one warp: elements [lo, hi) of the vocabulary.
struct Segment {
  const float* p;
  const float* q;  // null: point drafts, or no rejection yet
  int lo, hi;
  float ch, cl;
  const int* removed;
  int nremoved;  // removed tokens inside this segment are looked up when > 0
};

__device__ __forceinline__ Pair element(const Segment& g, int i, float p, float q) {
  if (g.q) return left(p, q, g.ch, g.cl);
  Pair v{p > 0.f || p != p ? p : 0.f, 0.f};
  for (int k = 0; k < g.nremoved; ++k)
    if (g.removed[k] == i) v.hi = 0.f;
  return v;
}

// Lane's 4 elements of the step that starts at i0 (zeros past the end).
__device__ __forceinline__ void load4(const Segment& g, int i0, int lane, float (&p)[4], float (&q)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = i0 + 4 * lane + k;
    p[k] = i < g.hi ? __ldg(g.p + i) : 0.f;
    q[k] = g.q && i < g.hi ? __ldg(g.q + i) : 0.f;
  }
}

__device__ __forceinline__ Pair segment_sum(const Segment& g, int lane) {
  Pair acc{0.f, 0.f};
#pragma unroll 2
  for (int i0 = g.lo; i0 < g.hi; i0 += kStep) {
    float p[4], q[4];
    load4(g, i0, lane, p, q);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Pair v = element(g, i0 + 4 * lane + k, p[k], q[k]);
      add(acc, v.hi, v.lo);
    }
  }
  return warp_total(acc);
}

// First index whose cumulative weight inside the segment exceeds t, else the last one of positive weight.
__device__ int segment_find(const Segment& g, double t, int lane) {
  double before = 0.0;
  int last = -1;
  for (int i0 = g.lo; i0 < g.hi; i0 += kStep) {
    float p[4], q[4];
    load4(g, i0, lane, p, q);
    double w[4], mine = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = value(element(g, i0 + 4 * lane + k, p[k], q[k]));
      mine += w[k];
    }
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned over = __ballot_sync(0xffffffffu, before + incl > t);
    const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0);
    const int pick = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
    if (pick >= 0) {
      int at = -1, lastpos = -1;
      double c = before + incl - mine;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c += w[k];
        if (w[k] > 0.0) lastpos = i0 + 4 * lane + k;
        if (at < 0 && c > t && w[k] > 0.0) at = i0 + 4 * lane + k;
      }
      // rounding may leave the lane's own sums at t: then its last positive one
      if (at < 0) at = lastpos;
      at = __shfl_sync(0xffffffffu, at, pick);
      if (over && at >= 0) return at;
      if (at >= 0) last = at;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return last;
}

// Index of the first of n totals at which the running sum exceeds *t (then *t
// is reduced by the sum before it), else of the last positive one; -1: none.
__device__ int pick_part(const double* part, int n, double* t) {
  double c = 0.0, at = 0.0;
  int last = -1;
  for (int i = 0; i < n; ++i) {
    if (part[i] > 0.0) {
      last = i;
      at = c;
    }
    c += part[i];
    if (part[i] > 0.0 && c > *t) break;
  }
  *t -= at;
  return last;
}

__global__ void __launch_bounds__(kThreads) tree_verify_kernel(const VerifyArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.x / kCluster, rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.S, V = a.V;
  const float* p0 = a.p + (long long)b * a.p_batch;
  const float* q0 = a.q ? a.q + (long long)b * a.q_batch : nullptr;

  // Rank 0 reads the nodes; the cluster's CTAs take them from its shared
  // memory, so that all of them walk the same tree whatever else happens.
  if (rank == 0 && tid <= S) {
    sh.u[tid] = a.u[(size_t)b * (S + 1) + tid];
    if (tid < S) {
      const TreeNode node = tree_node(a.parent + (size_t)b * S, tid);
      int up = node.state == kNodePresent ? a.parent[(size_t)b * S + tid] : -2;
      const int x = a.tokens[(size_t)b * S + tid];
      const bool bad = node.state == kNodeBad || (up >= -1 && (x < 0 || x >= V));
      if (bad) {
        raise_flag(a.flags, MLA_DEV_BAD_INDEX);
        up = -2;
      }
      sh.parent[tid] = up;
      sh.token[tid] = x;
      sh.pt[tid] = up >= -1 ? p0[(long long)(up + 1) * a.p_row + x] : 0.f;
      sh.qt[tid] = up >= -1 && q0 ? q0[(long long)(up + 1) * a.q_row + x] : 0.f;
    }
  }
  cluster.sync();
  if (rank != 0) {
    const Shared* first = cluster.map_shared_rank(&sh, 0);
    if (tid <= S) {
      sh.u[tid] = first->u[tid];
      if (tid < S) {
        sh.parent[tid] = first->parent[tid];
        sh.token[tid] = first->token[tid];
        sh.pt[tid] = first->pt[tid];
        sh.qt[tid] = first->qt[tid];
      }
    }
  }
  __syncthreads();

  // vocabulary slice of the CTA and segment of the warp, in whole warp steps
  const int steps = (V + kStep - 1) / kStep;
  const int per = (steps + kCluster * kWarps - 1) / (kCluster * kWarps);
  Segment seg{};
  seg.lo = min((rank * kWarps + warp) * per, steps) * kStep;
  seg.hi = min(min((rank * kWarps + warp + 1) * per, steps) * kStep, V);

  int pass = 0;
  // Sum of W at context `at`; every thread of the cluster gets the same value.
  // The warps' and CTAs' totals stay in sh for the draw.
  auto total = [&](int at, double c, int nremoved) -> double {
    seg.p = p0 + (long long)at * a.p_row;
    seg.q = q0 && c != 0.0 ? q0 + (long long)at * a.q_row : nullptr;  // W = p before any rejection
    seg.ch = (float)c;
    seg.cl = (float)(c - (double)seg.ch);
    seg.removed = sh.removed;
    int inside = 0;
    for (int k = 0; k < nremoved; ++k) inside |= sh.removed[k] >= seg.lo && sh.removed[k] < seg.hi;
    seg.nremoved = inside ? nremoved : 0;
    const Pair s = segment_sum(seg, lane);
    if (lane == 0) sh.warp_sum[warp] = value(s);
    __syncthreads();
    if (warp == 0) {
      double mine = 0.0;
      for (int w = 0; w < kWarps; ++w) mine += sh.warp_sum[w];
      if (lane < kCluster) cluster.map_shared_rank(&sh, lane)->part[pass & 1][rank] = mine;
    }
    cluster.sync();
    double z = 0.0;
    for (int r = 0; r < kCluster; ++r) z += sh.part[pass & 1][r];
    ++pass;
    return z;
  };

  int at = 0, n = 0, nremoved = 0;
  double c = 0.0, mass = 1.0;
  bool stale = false;  // mass not yet formed after a rejection
  for (int s = 0; s < S; ++s) {
    if (sh.parent[s] != at - 1) continue;
    const int x = sh.token[s];
    double w = sh.pt[s], chance = sh.u[s];
    if (q0) {
      if (stale) {
        mass = total(at, c, 0);
        stale = false;
      }
      w = w - c * (double)sh.qt[s];
      if (w < 0.0) w = 0.0;
      chance = chance * (double)sh.qt[s] * mass;
    } else {
      for (int k = 0; k < nremoved; ++k)
        if (sh.removed[k] == x) w = 0.0;
      chance = chance * mass;
    }
    if (chance < w) {
      if (rank == 0 && tid == 0) a.path[(size_t)b * S + n] = s;
      ++n;
      at = s + 1;
      c = 0.0;
      mass = 1.0;
      stale = false;
      nremoved = 0;
    } else if (q0) {
      c += mass;
      stale = true;
    } else {
      mass = mass > w ? mass - w : 0.0;
      __syncthreads();  // the list below is read by the passes and the tests above
      if (tid == 0) sh.removed[nremoved] = x;
      __syncthreads();
      ++nremoved;
    }
  }
  if (rank == 0) {
    for (int i = n + tid; i < S; i += kThreads) a.path[(size_t)b * S + i] = -1;
    if (tid == 0) a.n_acc[b] = n;
  }

  double z = total(at, c, nremoved);
  if (!(z > 0.0) && z == z) {  // nothing left: the target's own distribution
    c = 0.0;
    z = total(at, 0.0, 0);
  }
  if (!(z > 0.0) || !(z < 1e300)) {  // an empty or non-finite distribution
    if (rank == 0 && tid == 0) {
      raise_flag(a.flags, MLA_DEV_BAD_VALUE);
      a.token[b] = -1;
    }
    return;
  }
  double t = (double)sh.u[S] * z;
  if (pick_part(sh.part[(pass - 1) & 1], kCluster, &t) != rank) return;
  if (pick_part(sh.warp_sum, kWarps, &t) != warp) return;
  const int x = segment_find(seg, t, lane);
  if (lane == 0) a.token[b] = x;
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.B * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel, a);
}

}  // namespace mla
