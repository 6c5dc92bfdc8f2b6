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
// held to about 2^-48 without the fp64 pipe, which has 1/64 of the fp32 rate
// here and would bound the kernel: sum W = A - c B with A and B the sums of p and of q over
// the x where p > c q (an x misjudged by rounding has W(x) next to zero), and
// A and B are kept as unevaluated pairs hi + lo, added with Knuth's two-sum.
// The sums cost some 13 instructions an element (p and q added in packed
// pairs; 20 one by one; 30 with each W(x) formed as a pair).  Regrouped or
// small, such a sum can be zero or negative although a W(x) is positive, and the
// other way round.  So the draw takes CTA and warp by the rounded sums and,
// inside the warp's segment, sums the W(x) one by one; where these are all zero
// it looks through the whole vocabulary, so that a token is stored in any case.
//
// A sequence is a cluster of 8 CTAs, each with an eighth of the vocabulary: a
// row of p and of q of 131072 values, 1 MB, is 24 us of one SM's share of the
// memory bandwidth.  Every context on the way that rejects a child, and the last draw, is a
// pass over that context's rows that starts when the one before has decided,
// so the bound is the latency of the passes: load, block sum, cluster sum.
// Measured, vocabulary 131072, 32 trees of 24 nodes: 30 us, each byte of the
// rows that are looked at read from memory once (31.7 MB, 0.9 TB/s), barriers
// the first stall; a pass is about 6 us: loads and sums 3, totals and cluster
// barrier 1.8, decision 1.2.  5 drafts of one user over 32000: 9.4 us; 8 trees of
// 64 point drafts over 100003: 14 us, 4 of them the walk over the children.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;

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

// Two accumulators side by side: the packed instructions take one issue slot
// for both, and issue is what a pass waits for when two CTAs share an SM.
struct Pair2 {
  unsigned long long hi, lo;
};
__device__ __forceinline__ unsigned long long pack(float x, float y) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ void unpack(unsigned long long v, float* x, float* y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(v));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ unsigned long long sub2(unsigned long long a, unsigned long long b) {
  unsigned long long v;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ void add(Pair2& acc, float x, float y) {
  const unsigned long long v = pack(x, y);
  const unsigned long long s = add2(acc.hi, v), b = sub2(s, acc.hi);
  acc.lo = add2(acc.lo, add2(sub2(acc.hi, sub2(s, b)), sub2(v, b)));
  acc.hi = s;
}

// Total of the values of 2 * kFrom neighbouring lanes, the same in each of them.
template <int kFrom = 16>
__device__ __forceinline__ Pair warp_total(Pair v) {
#pragma unroll
  for (int o = kFrom; o > 0; o >>= 1) {
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

// a - (ch + cl) b as a pair.
__device__ __forceinline__ Pair minus_times(const Pair& a, const Pair& b, float ch, float cl) {
  const float h = ch * b.hi;
  const float e = fmaf(cl, b.hi, fmaf(ch, b.lo, fmaf(ch, b.hi, -h)));
  const float s = a.hi - h, t = s - a.hi;
  return Pair{s, ((a.hi - (s - t)) - (h + t)) + (a.lo - e)};
}

// max(p - (ch + cl) q, 0) as a pair whose high part is the rounded value, so
// that sums of such pairs are positive where one of them is.
__device__ __forceinline__ Pair left(float p, float q, float ch, float cl) {
  const float h = ch * q;
  const float e = fmaf(cl, q, fmaf(ch, q, -h));
  const float s = p - h, b = s - p;
  const float lo = ((p - (s - b)) - (h + b)) - e;
  const float w = s + lo, d = w - s;
  const bool pos = w > 0.f;
  // a NaN stays one, so that the total shows it
  return Pair{pos || w != w ? w : 0.f, pos ? (s - (w - d)) + (lo - d) : 0.f};
}

// What the warps do next: sum W at context `at`, or draw from it.
struct Command {
  int at;
  float ch, cl;                // c as a pair
  int draft;                   // q enters (a rejection has happened)
  unsigned long long removed;  // point drafts: rejected nodes of this context
  int done;
};

// The sums of p and of q over the x of a segment with p > c q (c = 0: of p).
struct Sums {
  Pair a, b;
};

struct Shared {
  // node data, filled by rank 0 and copied by the others
  int parent[kMaxTree], token[kMaxTree];
  float u[kMaxTree + 1], pt[kMaxTree], qt[kMaxTree];
  unsigned long long kids[kMaxTree + 1];  // children of every context
  Pair part[2][kCluster];                 // slice totals of every CTA, alternating between passes
  Sums warp_sums[kWarps];                 // of the warps' segments ...
  Pair warp_sum[kWarps];                  // ... and their W
  Command cmd;
  int bad[kMaxTree], up[kMaxTree];
  int warp_last[kWarps];  // last x of positive weight in the warps' segments
  int find_warp, find_last;
  double find_t;
};

// Shared::find_warp besides a warp's number: the draw is another CTA's, or no
// warp's rounded sum is positive.
constexpr int kNobody = -1, kSearch = -2;

// Segment of the vocabulary, in elements, and the weights there.
struct Segment {
  const float* p;
  const float* q;  // null: point drafts, or no rejection yet
  int lo, hi;
  float ch, cl;
  const int* token;            // of the nodes
  unsigned long long removed;  // nodes whose token is removed and lies inside the segment
};

__device__ __forceinline__ Pair element(const Segment& g, int i, float p, float q) {
  if (g.q) return left(p, q, g.ch, g.cl);
  Pair v{p > 0.f || p != p ? p : 0.f, 0.f};
  for (unsigned long long m = g.removed; m; m &= m - 1)
    if (g.token[__ffsll((long long)m) - 1] == i) v.hi = p != p ? p : 0.f;  // (a removed NaN stays one)
  return v;
}

// Nodes of `removed` whose token lies in [lo, hi) (the whole warp calls it).
__device__ __forceinline__ unsigned long long removed_inside(const Shared& sh, unsigned long long removed, int lo, int hi) {
  if (!removed) return 0;
  const int lane = threadIdx.x & 31;
  unsigned long long got = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int s = 32 * half + lane;
    const bool in = ((removed >> s) & 1ull) && sh.token[s] >= lo && sh.token[s] < hi;
    got |= (unsigned long long)__ballot_sync(0xffffffffu, in) << (32 * half);
  }
  return got;
}

// Sums over the segment, the same in every lane; the warp reads 32
// consecutive elements at a time, kAhead of them (of p and of q) in flight.
constexpr int kAhead = 8;
template <bool kDraft>
__device__ __forceinline__ Sums segment_sum(const Segment& g, int lane) {
  Pair2 sum{0, 0};  // of p and of q; without q, of every other element of p
  for (int i0 = g.lo; i0 < g.hi; i0 += 32 * kAhead) {
    float p[kAhead], q[kAhead];
    if (i0 + 32 * kAhead <= g.hi) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        p[k] = __ldg(g.p + i0 + 32 * k + lane);
        if (kDraft) q[k] = __ldg(g.q + i0 + 32 * k + lane);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + 32 * k + lane;
        p[k] = i < g.hi ? __ldg(g.p + i) : 0.f;
        q[k] = kDraft && i < g.hi ? __ldg(g.q + i) : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (kDraft) {
        const float w = fmaf(-g.cl, q[k], fmaf(-g.ch, q[k], p[k]));
        const bool in = !(w <= 0.f);  // (a NaN is in, so that the total shows it)
        add(sum, in ? p[k] : 0.f, in ? q[k] : 0.f);
      } else if (k % 2 == 0) {
        add(sum, element(g, i0 + 32 * k + lane, p[k], 0.f).hi, element(g, i0 + 32 * k + 32 + lane, p[k + 1], 0.f).hi);
      }
    }
  }
  Pair a, b;
  unpack(sum.hi, &a.hi, &b.hi);
  unpack(sum.lo, &a.lo, &b.lo);
  if (!kDraft) {
    add(a, b.hi, b.lo);
    b = Pair{0.f, 0.f};
  }
  return Sums{warp_total(a), kDraft ? warp_total(b) : b};
}
__device__ __forceinline__ Sums segment_sum(const Segment& g, int lane) {
  return g.q ? segment_sum<true>(g, lane) : segment_sum<false>(g, lane);
}

// Sum of the weights one by one, not as A - c B: it is positive exactly where a
// weight is.  *last: the last x of positive weight, or -1.
__device__ Pair weight_sum(const Segment& g, int lane, int* last) {
  Pair sum{0.f, 0.f};
  int at = -1;
#pragma unroll 2
  for (int i0 = g.lo; i0 < g.hi; i0 += 32) {
    const int i = i0 + lane;
    const float p = i < g.hi ? __ldg(g.p + i) : 0.f, q = g.q && i < g.hi ? __ldg(g.q + i) : 0.f;
    const Pair w = element(g, i, p, q);
    add(sum, w.hi, w.lo);
    if (w.hi > 0.f) at = i;
  }
  *last = __reduce_max_sync(0xffffffffu, at);
  return warp_total(sum);
}

// First index of the segment (at most 32 elements a step) whose cumulative
// weight exceeds t, else the last one of positive weight; -1: none.
__device__ int segment_find(const Segment& g, double t, int lane) {
  double before = 0.0;
  int last = -1;
  for (int i0 = g.lo; i0 < g.hi; i0 += 32) {
    const int i = i0 + lane;
    const float p = i < g.hi ? __ldg(g.p + i) : 0.f, q = g.q && i < g.hi ? __ldg(g.q + i) : 0.f;
    const double w = value(element(g, i, p, q));
    double incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned over = __ballot_sync(0xffffffffu, w > 0.0 && before + incl > t);
    const unsigned some = __ballot_sync(0xffffffffu, w > 0.0);
    if (over) return i0 + __ffs(over) - 1;
    if (some) last = i0 + 31 - __clz(some);
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return last;
}

// Index of the first of n <= 32 totals (one per lane, 0 beyond n) at which the
// running sum exceeds *t (then *t is reduced by the sum before it), else of
// the last positive one; -1: none.  The whole warp calls it.
__device__ __forceinline__ int pick_part(double mine, double* t) {
  const int lane = threadIdx.x & 31;
  double incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  const unsigned over = __ballot_sync(0xffffffffu, mine > 0.0 && incl > *t);
  const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0);
  const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
  if (at >= 0) *t -= __shfl_sync(0xffffffffu, incl - mine, at);
  return at;
}

// The warp of the CTA to whose segment g a draw of t falls (u >= 0: of u times
// the sum instead), sh.find_t then being what is left of t; -1: no weight is
// positive.  *last: the last x of positive weight in any of the segments, or -1.
// The whole CTA calls it.
__device__ int find_share(Shared& sh, Segment& g, unsigned long long removed, double t, float u, int* last) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  g.removed = removed_inside(sh, removed, g.lo, g.hi);
  const Pair mine = weight_sum(g, lane, last);
  if (lane == 0) {
    sh.warp_sum[warp] = mine;
    sh.warp_last[warp] = *last;
  }
  __syncthreads();
  if (warp == 0) {
    const double v = lane < kWarps ? value(sh.warp_sum[lane]) : 0.0;
    if (u >= 0.f) {
      t = v;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      t *= (double)u;
    }
    const int w = pick_part(v, &t);
    const int top = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.warp_last[lane] : -1);
    if (lane == 0) {
      sh.find_warp = w;
      sh.find_t = t;
      sh.find_last = top;
    }
  }
  __syncthreads();
  *last = sh.find_last;
  return sh.find_warp;
}

// The decisions (doubles: few, and made by one warp only, since all threads
// together would queue at the fp64 pipe) sit in warp 0 of every CTA; the other
// warps take its commands.  CTAs of a cluster reach the same decisions from
// the same numbers: rank 0's copy of the node data and the exchanged totals.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) tree_verify_kernel(const VerifyArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.x / kCluster, rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.S, V = a.V;
  const float* p0 = a.p + (long long)b * a.p_batch;
  const float* q0 = a.q ? a.q + (long long)b * a.q_batch : nullptr;

  if (rank == 0) {
    if (tid <= S) sh.u[tid] = a.u[(size_t)b * (S + 1) + tid];
    int up = -2, x = 0;
    bool bad = false;
    if (tid < S) {
      up = a.parent[(size_t)b * S + tid];
      x = a.tokens[(size_t)b * S + tid];
      bad = up < -2 || up >= tid || (up > -2 && (x < 0 || x >= V));
      const bool read = up > -2 && !bad;
      sh.token[tid] = x;
      sh.pt[tid] = read ? p0[(long long)(up + 1) * a.p_row + x] : 0.f;
      sh.qt[tid] = read && q0 ? q0[(long long)(up + 1) * a.q_row + x] : 0.f;
      sh.bad[tid] = bad;
      sh.up[tid] = bad ? -2 : up;
    }
    __syncthreads();
    // a node below an absent or bad one is bad: follow the parents by doubling
    if (tid < kMaxTree) {
      int far = tid < S && up >= 0 && !bad ? up : -1;
      for (int r = 0; r < 6; ++r) {
        const bool gone = far >= 0 && (sh.bad[far] || sh.up[far] == -2);
        const int next = far >= 0 ? sh.up[far] : -1;
        __syncwarp();
        asm volatile("bar.sync 1, 64;" ::: "memory");
        bad = bad || gone;
        if (tid < S) {
          sh.bad[tid] = bad;
          // (an absent ancestor is found before it is followed)
          sh.up[tid] = up == -2 || bad ? -2 : next;
        }
        far = next;
        __syncwarp();
        asm volatile("bar.sync 1, 64;" ::: "memory");
      }
      if (tid < S) {
        if (bad) raise_flag(a.flags, MLA_DEV_BAD_INDEX);
        sh.parent[tid] = bad ? -2 : up;
      }
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
  if (tid <= kMaxTree) sh.kids[tid] = 0;
  __syncthreads();
  if (tid < S && sh.parent[tid] >= -1) atomicOr(&sh.kids[sh.parent[tid] + 1], 1ull << tid);
  __syncthreads();

  // vocabulary segment of the warp, in whole groups of 32 elements
  const int groups = (V + 31) / 32;
  const int per = (groups + kCluster * kWarps - 1) / (kCluster * kWarps);
  Segment seg{};
  seg.token = sh.token;
  seg.lo = min((rank * kWarps + warp) * per, groups) * 32;
  seg.hi = min(min((rank * kWarps + warp + 1) * per, groups) * 32, V);

  int at = 0, n = 0, pass = 0;
  unsigned long long kids = sh.kids[0], removed = 0;
  double c = 0.0, mass = 1.0, z = 0.0;
  bool stale = false;  // mass not yet formed after a rejection
  bool drawing = false, fallback = false;
  for (;;) {
    if (warp == 0) {
      // walk until a sum is needed
      while (!drawing) {
        if (!kids) {
          drawing = true;
          break;
        }
        if (stale) break;  // another child of this context: its test needs the mass
        const int s = __ffsll((long long)kids) - 1;
        kids &= kids - 1;
        double w = sh.pt[s], chance = sh.u[s];
        if (q0) {
          w = w - c * (double)sh.qt[s];
          if (w < 0.0) w = 0.0;
          chance = chance * (double)sh.qt[s] * mass;
        } else {
          for (unsigned long long m = removed; m; m &= m - 1)
            if (sh.token[__ffsll((long long)m) - 1] == sh.token[s]) w = 0.0;
          chance = chance * mass;
        }
        if (chance < w) {
          if (rank == 0 && lane == 0) a.path[(size_t)b * S + n] = s;
          ++n;
          at = s + 1;
          kids = sh.kids[at];
          c = 0.0;
          mass = 1.0;
          removed = 0;
        } else if (q0) {
          c += mass;
          stale = true;
        } else {
          mass = mass <= w ? 0.0 : mass - w;  // (a NaN stays: no later child is accepted)
          removed |= 1ull << s;
        }
      }
      if (lane == 0) {
        const float ch = (float)c;
        sh.cmd = Command{at, ch, (float)(c - (double)ch), q0 && c != 0.0 ? 1 : 0, removed, 0};
      }
    }
    __syncthreads();
    const Command cmd = sh.cmd;
    if (cmd.done) break;
    seg.p = p0 + (long long)cmd.at * a.p_row;
    seg.q = cmd.draft ? q0 + (long long)cmd.at * a.q_row : nullptr;  // W = p before any rejection
    seg.ch = cmd.ch;
    seg.cl = cmd.cl;
    seg.removed = removed_inside(sh, cmd.removed, seg.lo, seg.hi);
    const Sums s = segment_sum(seg, lane);
    if (lane == 0) sh.warp_sums[warp] = s;
    __syncthreads();
    if (warp == 0) {  // in pairs: as doubles these totals took 1.1 us of a pass, now 0.3
      Pair mine{0.f, 0.f};
      if (lane < kWarps) {
        const Sums x = sh.warp_sums[lane];
        mine = minus_times(x.a, x.b, cmd.ch, cmd.cl);
        sh.warp_sum[lane] = mine;
      }
      mine = warp_total<kWarps / 2>(mine);
      if (lane < kCluster) cluster.map_shared_rank(&sh, lane)->part[pass & 1][rank] = mine;
    }
    cluster.sync();
    if (warp == 0) {
      Pair all = warp_total<kCluster / 2>(lane < kCluster ? sh.part[pass & 1][lane] : Pair{0.f, 0.f});
      all.hi = __shfl_sync(0xffffffffu, all.hi, 0);
      all.lo = __shfl_sync(0xffffffffu, all.lo, 0);
      z = value(all);
      if (!drawing) {
        mass = z < 0.0 ? 0.0 : z;  // (less than the sums' rounding is left; a NaN stays)
        stale = false;
      } else if (!(z > 0.0) && z == z && !fallback && (c != 0.0 || removed)) {
        fallback = true;  // nothing left: the target's own distribution
        c = 0.0;
        removed = 0;
      } else {
        if (lane == 0) sh.cmd.done = 1;
        // which CTA, then which warp, the draw falls to
        double t = (double)sh.u[S] * z;
        int hit = kNobody;
        if (z > 0.0 && z < 1e300) {
          const int owner = pick_part(lane < kCluster ? value(sh.part[pass & 1][lane]) : 0.0, &t);
          if (owner == rank) hit = pick_part(lane < kWarps ? value(sh.warp_sum[lane]) : 0.0, &t);
          if ((owner == rank && hit < 0) || (owner < 0 && rank == 0)) hit = kSearch;
        } else if (rank == 0 && lane == 0) {  // an empty or non-finite distribution
          raise_flag(a.flags, MLA_DEV_BAD_VALUE);
          a.token[b] = -1;
        }
        if (lane == 0) {
          sh.find_warp = hit;
          sh.find_t = t;
        }
        drawing = true;
      }
    }
    ++pass;
    __syncthreads();
    if (sh.cmd.done) break;
  }
  if (rank == 0 && warp == 0) {
    for (int i = n + lane; i < S; i += 32) a.path[(size_t)b * S + i] = -1;
    if (lane == 0) a.n_acc[b] = n;
  }
  // The warp's segment again, split over the CTA's warps, weight by weight.
  const int hit = sh.find_warp;
  if (hit == kNobody) return;
  const unsigned long long gone = sh.cmd.removed;
  if (hit != kSearch) {
    const int hlo = min((rank * kWarps + hit) * per, groups) * 32, hhi = min(min((rank * kWarps + hit + 1) * per, groups) * 32, V);
    const int sub = (per + kWarps - 1) / kWarps;  // groups of 32 per warp
    seg.lo = min(hlo + 32 * sub * warp, hhi);
    seg.hi = min(hlo + 32 * sub * (warp + 1), hhi);
    int last;
    const int w = find_share(sh, seg, gone, sh.find_t, -1.f, &last);
    if (w == warp) {
      const int x = segment_find(seg, sh.find_t, lane);
      if (lane == 0) a.token[b] = x;
    }
    if (w >= 0) return;
  }
  // The rounded sums pointed at weights that are all zero: what is left is at
  // most their rounding.  The last x of positive weight, or, where there is
  // none, a draw from p.  Never seen but on inputs made for it: 30 drafts
  // rejected one after the other at one context.
  const int stripe = (groups + kWarps - 1) / kWarps;
  seg.lo = min(32 * min(stripe * warp, groups), V);
  seg.hi = min(32 * min(stripe * (warp + 1), groups), V);
  int last;
  find_share(sh, seg, gone, 0.0, -1.f, &last);
  if (last >= 0) {
    if (tid == 0) a.token[b] = last;
    return;
  }
  seg.q = nullptr;
  const int w = find_share(sh, seg, 0, 0.0, sh.u[S], &last);
  if (w < 0) {
    if (tid == 0) {
      raise_flag(a.flags, MLA_DEV_BAD_VALUE);
      a.token[b] = -1;
    }
  } else if (w == warp) {
    const int x = segment_find(seg, sh.find_t, lane);
    if (lane == 0) a.token[b] = x;
  }
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyArgs& a, cudaStream_t st) {
  tree_verify_kernel<<<(unsigned)a.B * kCluster, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
