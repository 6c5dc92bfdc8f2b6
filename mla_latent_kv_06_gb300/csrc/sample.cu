// sample.cu -- tokens and filtered distributions from logits.
//
// Method.  The tokens of a row are ordered by (logit down, index up), and every
// filter keeps a prefix of that order, so the kept set is one threshold: a
// token's code, its ordered logit bits above its inverted index, is unique, and
// a token is kept when its code reaches the threshold's.  Nothing is sorted.
//   w(x)  = exp((x - max) / T)                      (T = 0: the first token alone)
//   min-p : w(x) >= min_p, a threshold on x itself
//   top-k : the code of the k-th token
//   top-p : the code of the token at which the running mass reaches top_p W
// The last two are found by select(): a histogram of counts or masses over
// kBins intervals of the order, which narrows the threshold down to one
// interval, until few enough candidates are left to rank them against each
// other.  The draw is the least index whose cumulative kept mass exceeds u W.
//
// Rounding.  A threshold and a draw compare sums over the vocabulary, so a
// weight is a 64-bit integer, w 2^44 rounded once: sums are then exact, in any
// order, and the kernel's atomics cannot change a result.  The exponential is
// taken in fp32 pairs without the fp64 pipe (1/64 of the fp32 rate): x - max
// by two-sum, times log2(e)/T as a pair, a table of 2^(-i/256) in 48 bits and
// a cubic for the rest, error below 2^-33 of the weight.
//
// A row is a cluster of up to 8 CTAs, each with a contiguous part of the
// vocabulary in shared memory as fp32, read once; a warp's part is contiguous
// too, and no other warp reads it.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCluster = 8;    // most CTAs of a row
constexpr int kList = 1024;    // candidates that are ranked against each other
constexpr int kOne = 44;       // a weight of 1 is 2^kOne; kMaxSampleVocab of them stay below 2^63
constexpr int kIndexBits = 20;
constexpr u64 kIndexMask = (1ull << kIndexBits) - 1;
constexpr float kNegligible = 256.f * (kOne + 2);  // 256 log2 of a weight that rounds to 0
static_assert(kMaxSampleVocab <= (1 << 19), "sums of weights stay below 2^63, indices below 2^kIndexBits");

// 2^(-i/256) as hi + lo, hi < 1 of 24 bits.
struct ExpTable {
  float hi[256], lo[256];
};
constexpr ExpTable make_table() {
  ExpTable t{};
  for (int i = 0; i < 256; ++i) {
    const double y = -0.69314718055994530942 * i / 256;
    double term = 1.0, sum = 1.0;  // Taylor series of exp(y)
    for (int n = 1; n < 30; ++n) {
      term *= y / n;
      sum += term;
    }
    const long long scaled = (long long)(sum * 16777216.0);
    const long long top = scaled < 16777216 ? scaled : 16777215;
    t.hi[i] = (float)((double)top / 16777216.0);
    t.lo[i] = (float)(sum - (double)top / 16777216.0);
  }
  return t;
}
__constant__ ExpTable kTable = make_table();

struct Bin {
  unsigned cnt, lo, hi;  // tokens; mass as two words
};

struct Shared {
  unsigned cnt[kBins], lo[kBins], hi[kBins];  // this CTA's histogram
  unsigned tot_cnt[kBins];                    // the cluster's, written by all CTAs
  u64 tot[kBins];
  u64 list_code[kList], list_w[kList];
  float2 table[256];
  float max[kCluster], min[kCluster];
  int bad[kCluster];
  u64 mass[kCluster];
  u64 warp_mass[kWarps];
  unsigned warp_cnt[kWarps];
  float warp_max[kWarps], warp_min[kWarps];
  int listed;
  int warp_bad;
  int bin;
  u64 before;
  u64 code, upto;
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan64(u64 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// log2(e) 256 / T as a pair.
struct Heat {
  float hi, lo;
};

// w = exp((x - max) / T) as (mant_hi + mant_lo) 2^-n; false where w < 2^(-limit / 256).
struct Parts {
  float hi, lo;
  int n;
};
__device__ __forceinline__ bool weight_parts(float x, float max, const Heat& h, const float2* table, float limit, Parts* p) {
  const float d = max - x, b = d - max, dl = (max - (d - b)) + (-x - b);
  const float y = d * h.hi;
  if (!(y < limit)) return false;
  const float e = fmaf(d, h.hi, -y) + fmaf(d, h.lo, dl * h.hi);
  const float m = y + 12582912.f;  // 1.5 2^23: the integer part in the low bits
  const int k = __float_as_int(m) - 0x4B400000;
  const float r = (y - (m - 12582912.f)) + e;
  const float z = r * -0.0027076061740622863f;  // ln(2) / 256
  const float q = fmaf(z * z, fmaf(z, 1.f / 6.f, 0.5f), z);  // exp(z) - 1
  const float2 t = table[k & 255];
  p->hi = t.x;
  p->lo = fmaf(t.x, q, t.y);
  p->n = k >> 8;
  return true;
}

__device__ __forceinline__ u64 weight(float x, float max, const Heat& h, const float2* table) {
  Parts p;
  if (!weight_parts(x, max, h, table, kNegligible, &p)) return 0;
  // hi < 1 has exponent -1: 24 bits with the hidden one
  const u64 a = (u64)((__float_as_uint(p.hi) & 0x7fffffu) | 0x800000u) << (kOne - 24);
  const long long c = (long long)__float2int_rn(p.lo * 1099511627776.f) << (kOne - 40);  // |lo| < 2^-9
  return (((a + (u64)c) << 1 >> p.n) + 1) >> 1;
}

__device__ __forceinline__ u64 code_of(float x, int index) {
  return ((u64)ordered_key(x) << kIndexBits) | (kIndexMask - (u64)index);
}

// floor(f m) for 0 <= f < 1; *inexact: whether anything was cut off.
__device__ __forceinline__ u64 fraction_of(float f, u64 m, bool* inexact) {
  const unsigned bits = __float_as_uint(f), e = bits >> 23;
  const u64 mant = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int s = 150 - (e ? (int)e : 1);  // f = mant 2^-s, s >= 24
  const u64 hi = __umul64hi(m, mant), lo = m * mant;
  if (s < 64) {
    *inexact = (lo & ((1ull << s) - 1)) != 0;
    return (hi << (64 - s)) | (lo >> s);
  }
  const int t = s - 64;  // below 86
  *inexact = lo != 0 || (t >= 64 ? hi != 0 : (hi & ((1ull << t) - 1)) != 0);
  return t >= 64 ? 0 : hi >> t;
}

// This CTA's part of a row, and what is known of the row.
struct Row {
  const float* x;  // shared memory
  int base, lo, hi;  // index of x[0]; the warp's elements
  float max;
  Heat heat;
  u64 floor;  // a token is kept when its code is at least this
};

// The code at which the running count (kMass: mass) of the kept tokens, in
// order, reaches a target: `target` for counts, the fraction `p` of the whole for masses.
// range: tokens further than this below the maximum share the last interval.
// Raises row.floor to that code (leaves it where the whole does not reach the
// target); with kMass returns the mass kept.
template <bool kMass>
__device__ u64 select(cg::cluster_group& cluster, Shared& sh, Row& row, float range, u64 target, float p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const float step = range > 0.f ? (float)kBins / range : 0.f;
  u64 lo = 0, hi = ~0ull, above = 0;  // the threshold lies in [lo, hi]; what the codes above it hold
  int b0 = -1, shift = 0;  // first level: intervals of x; later ones: of codes inside interval b0
  auto first_bin = [&](float x) -> int {
    const float f = (row.max - x) * step;
    return f < (float)(kBins - 1) ? (int)f : kBins - 1;
  };
  auto weigh = [&](float x) -> u64 { return kMass ? weight(x, row.max, row.heat, sh.table) : 1; };
  for (;;) {
    for (int i = tid; i < kBins; i += kThreads) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    u64 last_w = 0;  // of the last interval, which may hold most tokens
    unsigned last_n = 0;
    for (int i = row.lo + lane; i < row.hi; i += 32) {
      const float x = row.x[i];
      const u64 code = code_of(x, row.base + i);
      if (code < row.floor) continue;
      int bin = first_bin(x);
      if (b0 >= 0) {
        if (bin != b0 || code < lo || code > hi) continue;
        bin = (int)((hi - code) >> shift);
      }
      const u64 w = weigh(x);
      if (bin == kBins - 1) {
        last_w += w;
        ++last_n;
        continue;
      }
      atomicAdd(&sh.cnt[bin], 1u);
      if (kMass) {
        const unsigned wl = (unsigned)w, old = atomicAdd(&sh.lo[bin], wl);
        const unsigned wh = (unsigned)(w >> 32) + (old + wl < old ? 1u : 0u);
        if (wh) atomicAdd(&sh.hi[bin], wh);
      }
    }
    last_w = warp_sum64(last_w);
    last_n = __reduce_add_sync(0xffffffffu, last_n);
    if (lane == 0 && last_n) {
      atomicAdd(&sh.cnt[kBins - 1], last_n);
      if (kMass) {
        const unsigned wl = (unsigned)last_w, old = atomicAdd(&sh.lo[kBins - 1], wl);
        atomicAdd(&sh.hi[kBins - 1], (unsigned)(last_w >> 32) + (old + wl < old ? 1u : 0u));
      }
    }
    cluster.sync();
    // each CTA sums its share of the intervals over the cluster and hands the sums to all
    const int share = kBins / C;
    for (int i = tid; i < share; i += kThreads) {
      const int bin = rank * share + i;
      unsigned n = 0;
      u64 w = 0;
      for (int q = 0; q < C; ++q) {
        n += *cluster.map_shared_rank(&sh.cnt[bin], q);
        if (kMass) w += ((u64)*cluster.map_shared_rank(&sh.hi[bin], q) << 32) + *cluster.map_shared_rank(&sh.lo[bin], q);
      }
      if (!kMass) w = n;
      for (int q = 0; q < C; ++q) {
        *cluster.map_shared_rank(&sh.tot_cnt[bin], q) = n;
        *cluster.map_shared_rank(&sh.tot[bin], q) = w;
      }
    }
    cluster.sync();
    // the interval at which the running sum reaches the target
    constexpr int kPer = kBins / kThreads;
    u64 mine[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += mine[k] = sh.tot[tid * kPer + k];
    const u64 incl = warp_scan64(sum);
    if (lane == 31) sh.warp_mass[warp] = incl;
    __syncthreads();
    u64 run = above + incl - sum, whole = above;
    for (int q = 0; q < kWarps; ++q) {
      if (q < warp) run += sh.warp_mass[q];
      whole += sh.warp_mass[q];
    }
    if (b0 < 0) {
      if (kMass) {
        bool cut;
        target = fraction_of(p, whole, &cut);
        if (cut || target == 0) ++target;
      } else if (whole <= target) {
        return 0;
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (run < target && target <= run + mine[k]) {
        sh.bin = tid * kPer + k;
        sh.before = run;
      }
      run += mine[k];
    }
    __syncthreads();
    const int bin = sh.bin;
    const unsigned n = sh.tot_cnt[bin];
    above = sh.before;
    if (b0 < 0) {
      b0 = bin;
    } else {
      hi -= (u64)bin << shift;
      const u64 width = (1ull << shift) - 1;
      if (hi - lo > width) lo = hi - width;
    }
    if (n <= kList) break;
    // too many to rank: split the interval by codes
    if (b0 == bin && hi == ~0ull) {
      lo = 0;
      hi = (1ull << (32 + kIndexBits)) - 1;
    }
    shift = 64 - __clzll((long long)(hi - lo)) - 10;  // hi - lo < 2^(shift + 10), kBins intervals of 2^shift
    if (shift < 0) shift = 0;
    __syncthreads();
  }
  // the candidates, in every CTA's list
  for (int i = row.lo + lane; i < row.hi; i += 32) {
    const float x = row.x[i];
    const u64 code = code_of(x, row.base + i);
    if (code < row.floor || first_bin(x) != b0 || code < lo || code > hi) continue;
    const u64 w = weigh(x);
    for (int q = 0; q < C; ++q) {
      const int at = atomicAdd(cluster.map_shared_rank(&sh.listed, q), 1);
      if (at < kList) {
        *cluster.map_shared_rank(&sh.list_code[at], q) = code;
        *cluster.map_shared_rank(&sh.list_w[at], q) = w;
      }
    }
  }
  cluster.sync();
  const int n = min(sh.listed, kList);
  for (int i = tid; i < n; i += kThreads) {
    const u64 code = sh.list_code[i], w = sh.list_w[i];
    u64 before = above;
    for (int j = 0; j < n; ++j) before += sh.list_code[j] > code ? sh.list_w[j] : 0;
    if (before < target && target <= before + w) {
      sh.code = code;
      sh.upto = before + w;
    }
  }
  __syncthreads();
  row.floor = sh.code;
  const u64 kept = sh.upto;
  __syncthreads();
  return kept;
}

template <typename Tin>
__device__ __forceinline__ void load_part(const Tin* src, float* dst, int lo, int hi, int valid, int lane, float* mx, float* mn,
                                          bool* bad) {
  constexpr int kAhead = 8;
  for (int i0 = lo; i0 < hi; i0 += 32 * kAhead) {
    float v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + 32 * k + lane;
      v[k] = i < valid && i < hi ? to_f32(src[i]) : -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + 32 * k + lane;
      if (i < hi) dst[i] = v[k];
      *mx = fmaxf(*mx, v[k]);
      if (v[k] > -INFINITY) *mn = fminf(*mn, v[k]);
      *bad = *bad || !(v[k] < INFINITY);
    }
  }
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, int part) {
  extern __shared__ __align__(16) float x_sh[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / C, b = r / a.N, node = r % a.N;
  const int set = a.per_row ? r : b;  // the row's settings
  float heat = a.temperature ? a.temperature[set] : 1.f;
  int k = a.top_k ? a.top_k[set] : 0;
  const float p = a.top_p ? a.top_p[set] : 1.f, least = a.min_p ? a.min_p[set] : 0.f;

  Row row;
  row.x = x_sh;
  row.base = rank * part;
  row.lo = warp * (part / kWarps);
  row.hi = row.lo + part / kWarps;
  if (tid < 256) sh.table[tid] = make_float2(kTable.hi[tid], kTable.lo[tid]);
  if (tid == 0) sh.warp_bad = 0;
  __syncthreads();
  const Tin* src = static_cast<const Tin*>(a.logits) + (long long)b * a.l_batch + (long long)node * a.l_row + row.base;
  float mx = -INFINITY, mn = INFINITY;
  bool bad = false;
  load_part(src, x_sh, row.lo, row.hi, min(a.V - row.base, part), lane, &mx, &mn, &bad);
  mx = warp_max(mx);
  mn = -warp_max(-mn);
  if (__any_sync(0xffffffffu, bad) && lane == 0) sh.warp_bad = 1;
  if (lane == 0) {
    sh.warp_max[warp] = mx;
    sh.warp_min[warp] = mn;
  }
  __syncthreads();
  if (warp == 0) {
    mx = warp_max(lane < kWarps ? sh.warp_max[lane] : -INFINITY);
    mn = -warp_max(lane < kWarps ? -sh.warp_min[lane] : -INFINITY);
    if (lane < C) {
      *cluster.map_shared_rank(&sh.max[rank], lane) = mx;
      *cluster.map_shared_rank(&sh.min[rank], lane) = mn;
      *cluster.map_shared_rank(&sh.bad[rank], lane) = sh.warp_bad;
    }
  }
  cluster.sync();
  row.max = sh.max[0];
  mn = sh.min[0];
  bad = sh.bad[0] != 0;
  for (int q = 1; q < C; ++q) {
    row.max = fmaxf(row.max, sh.max[q]);
    mn = fminf(mn, sh.min[q]);
    bad = bad || sh.bad[q] != 0;
  }
  float* out = a.probs ? a.probs + (long long)b * a.p_batch + (long long)node * a.p_row + row.base : nullptr;
  const int valid = min(a.V - row.base, part);  // (below 1 for a CTA past the end)
  // no finite maximum, NaN or +inf among the logits, or settings that mean nothing
  if (bad || !(row.max > -INFINITY) || !(heat >= 0.f && heat < INFINITY) || p != p || least != least) {
    if (rank == 0 && tid == 0) {
      raise_flag(a.flags, MLA_DEV_BAD_VALUE);
      if (a.token) a.token[r] = -1;
    }
    if (out)
      for (int i = row.lo + lane; i < min(row.hi, valid); i += 32) out[i] = qnan();
    return;
  }
  if (heat == 0.f) {
    heat = 1.f;
    k = 1;
  }
  const double c = fmin(256.0 * 1.4426950408889634 / (double)heat, 1e36);  // (T below 4e-34 acts as that)
  row.heat.hi = (float)c;
  row.heat.lo = (float)(c - (double)row.heat.hi);
  row.floor = (u64)0x00800000u << kIndexBits;  // above -inf
  if (least > 0.f) {
    const double t = (double)row.max + (double)heat * log(fmin((double)least, 1.0));
    const u64 f = (u64)ordered_key(__double2float_ru(t)) << kIndexBits;
    if (f > row.floor) row.floor = f;
  }
  const float spread = row.max - mn;
  if (k > 0 && k < a.V) select<false>(cluster, sh, row, fminf(spread, 40.f * heat), (u64)k, 0.f);
  u64 total = 0;
  if (p < 1.f) {
    // tokens past this range hold less than 1 - p of the mass, whatever their number
    const float tail = logf((float)a.V) - logf(fmaxf(1.f - p, 1e-7f)) + 1.f;
    total = select<true>(cluster, sh, row, fminf(spread, tail * heat), 0, fmaxf(p, 0.f));
  }
  if (a.token || p >= 1.f) {
    u64 mine = 0;
    for (int i = row.lo + lane; i < row.hi; i += 32) {
      const float x = x_sh[i];
      if (code_of(x, row.base + i) >= row.floor) mine += weight(x, row.max, row.heat, sh.table);
    }
    mine = warp_sum64(mine);
    if (lane == 0) sh.warp_mass[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const u64 sum = warp_sum64(lane < kWarps ? sh.warp_mass[lane] : 0);
      if (lane < C) *cluster.map_shared_rank(&sh.mass[rank], lane) = sum;
    }
    cluster.sync();
    total = 0;
    for (int q = 0; q < C; ++q) total += sh.mass[q];
  }
  if (a.token) {
    // the CTA, the warp, the element at which the running mass exceeds t < total
    bool cut;
    const float u = a.u[r];
    u64 t = u >= 1.f ? total - 1 : u > 0.f ? fraction_of(u, total, &cut) : 0;
    for (int q = 0; q < rank; ++q) t -= sh.mass[q];  // (wraps where the draw is before this CTA)
    if (t < sh.mass[rank]) {
      int w = 0;
      while (t >= sh.warp_mass[w]) t -= sh.warp_mass[w++];
      if (w == warp) {
        for (int i0 = row.lo; i0 < row.hi; i0 += 32) {
          const float x = x_sh[i0 + lane];
          const u64 v = code_of(x, row.base + i0 + lane) >= row.floor ? weight(x, row.max, row.heat, sh.table) : 0;
          const u64 incl = warp_scan64(v);
          const unsigned over = __ballot_sync(0xffffffffu, incl > t);
          if (over) {
            if (lane == 0) a.token[r] = row.base + i0 + __ffs(over) - 1;
            break;
          }
          t -= __shfl_sync(0xffffffffu, incl, 31);
        }
      }
    }
  }
  if (out) {
    const float inv = (float)((double)(1ull << kOne) / (double)total);
    for (int i = row.lo + lane; i < min(row.hi, valid); i += 32) {
      const float x = x_sh[i];
      float v = 0.f;
      Parts w;
      if (code_of(x, row.base + i) >= row.floor && weight_parts(x, row.max, row.heat, sh.table, 256.f * 160.f, &w)) {
        const int n0 = w.n >> 1;  // two factors of 2: n may pass the exponent's range
        v = (w.hi + w.lo) * inv * __int_as_float((127 - n0) << 23) * __int_as_float((127 - (w.n - n0)) << 23);
      }
      out[i] = v;
    }
  }
}

template <typename Tin>
cudaError_t launch(const SampleArgs& a, cudaStream_t st) {
  static std::atomic<u64> done{0};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const u64 bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(sample_kernel<Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, 180 * 1024);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  const long long rows = (long long)a.B * a.N;
  int C = 1;
  while (C < kCluster && (a.V + C - 1) / C > 16384) C *= 2;
  while (C < kCluster && rows * C * 2 <= sms && a.V / C > 2048) C *= 2;
  const int part = ((a.V + C - 1) / C + kThreads - 1) / kThreads * kThreads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)part * sizeof(float);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<Tin>, a, part);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  return a.dtype == MLA_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace mla
