// sample.cu -- tokens and filtered distributions from logits.
//
// Method.  The tokens of a row are ordered by (logit down, index up), and every
// filter keeps a prefix of that order, so the kept set is one threshold: a
// token's code, its ordered logit bits above its inverted index, is unique, and
// a token is kept when its code reaches the threshold's.  No row is sorted.
//   w(x)  = exp((x - max) / T)                      (T = 0: the first token alone)
//   min-p : w(x) >= min_p, a threshold on x itself
//   top-k : the code of the k-th token
//   top-p : the code of the token at which the running mass reaches top_p W
// The last two come from a histogram that counts tokens in kBins intervals of x:
//   top-k: it names the k-th token's interval, whose tokens are then sorted.  A small k needs
// no histogram of the row: the k-th of the threads' largest tokens bounds the k-th token
// from below, and what reaches that bound, little more than k tokens, decides
// everything else, the other filters and the draw included.
//   top-p: a token's weight follows from its interval well enough to name the threshold's
// (nucleus()).  One pass with exact weights then gives W, the mass above that interval and
// the interval's tokens, or says that it is the next one.
//   An interval of more tokens than the list holds is split by the bits of x, on exact counts
// or masses, down to one value, and its tokens are counted out by index (refine()).
// The draw is the least index whose cumulative kept mass exceeds u W: the CTA and the warp
// by their sums, then that warp's elements by all threads.
//
// Rounding.  A threshold and a draw compare sums over the vocabulary, so a
// weight is an integer, w 2^44 rounded once: sums are then exact, in any order,
// and the kernel's atomics cannot change a result.  The exponential is taken
// without the fp64 pipe (1/64 of the fp32 rate) and without 64-bit shifts:
//   z = y c rounded to an integer, c = 256 log2(e) / T, t = y c - z by two fused
//   multiply-adds whose products are exact; relative to an integer `top` above max c,
//   w = 2^((z - top)/256) 2^(t/256);
//   a table of 2^(-i/256) as hi (1 + d) for the low 8 bits of top - z, the others moved into
//   hi's exponent by one addition (the table's entry holds i times that step, too);
//   a cubic for 2^(t/256) - 1 + d, whose product with hi is the weight's low part;
//   the two parts added to 3 and to 1.5 2^-21, whose last places are 2^-22 and 2^-44:
//   the integers are then in the sums' bits, and are added up as such.  (What the second
//   sum takes, up to 2^-23 and the low part's rounding, must stay inside its binade.)
// The error is below 2^-31 of the weight before the rounding.  Two elements go through
// packed fp32 instructions; 71 instructions an element with 64-bit integers, conversions
// and one element at a time.
//
// A row is a cluster of up to 8 CTAs, each with a contiguous part of the
// vocabulary in shared memory, read once, 16 bytes at a time from 16-byte
// boundaries; a warp's part is contiguous too, and mostly no other warp reads it.  (An early
// form with a CTA a row, streaming it from L2 in every pass, took 104 us where clusters then took
// 95: 256 rows of 131072 at a temperature alone.  It was not measured against the present passes.)
//
// Measured: 256 rows of 131072 bf16 logits of deviation 3 at a temperature of 0.8 53 us (1.3 TB/s),
// with top-p 0.9 97, with top-k 50 52, with min-p 0.05 38, of all kinds 69; 400 rows with their
// probabilities 128 (2.5 TB/s), with top-p 188.  No one unit is at its rate.  At a temperature alone
// issue slots are 55% used while an SM is busy and the shared-memory pipe 57%: the exponentials'
// table is read at random, 5.0 passes of the banks an instruction over all loads where 2 would do.  The
// stalls are not_selected 2.4, math pipes 2.3, barriers 1.8 and short scoreboard 1.2 warps an issue; with
// filters of all kinds barriers lead (3.0): a row goes through its passes with barriers of the CTA (500
// cycles each beside another CTA's work) and of the cluster (1500) between them.  Two CTAs fill an
// SM's registers, and 76 rows at a time are 3.4 rounds for 256.  Fetching the next round's rows
// into L2 ahead changed nothing.  CTAs of 1024 threads (one row of 131072 with top-p 29 us
// against 23) and clusters of twice the CTAs (79 against 55) cost more in barriers than they give; CTAs of
// twice the elements, one to an SM, 59 against 52.  One row of 32000 fp32 takes 6.6 us, with top-p 12.5.
#include <cooperative_groups.h>
#include <limits.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCluster = 8;  // most CTAs of a row
constexpr int kList = 1024;  // tokens that are ranked against each other: two a thread
constexpr int kAround = 128; // tokens around an estimated threshold that are looked at in any case
// top-k by the threads' largest tokens, whose list then serves top-p and the draw too, or by
// counts and a threshold.  64 rows of 131072 bf16 (256 of these; 8 of 32000 fp32), us: k = 200 21.0 and
// 23.9 (63.8 and 78.6; 13.7 and 12.3), k = 300 23.8 and 24.8 (72.0 and 82.4; 14.9 and 12.1), k = 500 33.3 and
// 26.7 (95.0 and 87.4; 21.1 and 12.3); with top-p after it k = 500 32.3 and 45.8 (93.2 and 148.5; 20.3 and 20.3).
constexpr int kSmallK = 256, kSmallKTopP = 512;
constexpr int kOne = 44;     // a weight of 1 is 2^kOne; kMaxSampleVocab of them stay below 2^63
constexpr int kIndexBits = 20;
constexpr u64 kIndexMask = (1ull << kIndexBits) - 1;
constexpr float kNegligible = 256.f * (kOne + 2);  // 256 log2 of a weight that rounds to 0
static_assert(kMaxSampleVocab < (1 << 18) + (1 << 17), "sums of weights stay below 2^63, indices below 2^kIndexBits");

// 2^(-i/256) = hi (1 + d), hi < 1 of 24 bits; hi's bits plus i 2^15 (the exponent's unit is 256 2^15).
struct ExpTable {
  int hi[256];
  float d[256];
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
    const long long scaled = (long long)(sum * 16777216.0);  // from 2^23 up
    const long long top = scaled < 16777216 ? scaled : 16777215;
    t.hi[i] = 0x3f000000 + (int)(top - 8388608) + (i << 15);
    t.d[i] = (float)(sum / ((double)top / 16777216.0) - 1.0);
  }
  return t;
}
__device__ const ExpTable kTable = make_table();

// An interval of more tokens than the list holds, in which the threshold lies, from xe up to xt
// or below.
struct Crowd {
  float xe, xt;
  u64 above, target;  // masses
};

struct Shared {
  Crowd crowd;
  unsigned cnt[kBins + 64];  // this CTA's histogram: tokens (the last interval and, from kBins + 32 on,
                             // what is no token have a place a lane) ...
  union {
    struct {
      unsigned lo[kBins], hi[kBins];  // ... or mass as two words
    };
    u64 own[kList];  // this CTA's share of the list
  };
  u64 tot[kBins];               // the cluster's
  u64 list[kList], sum[kList];  // codes; running mass once ranked
  int2 table[256];   // of i at -i mod 256: (hi, d's bits)
  double least;      // T log(min_p)
  float2 ends[kWarps], end;  // the warps' and the CTA's largest and smallest logits
  unsigned hidden[kWarps], all_hidden;  // the same, elements of -inf (padding too) where they are counted; then [0]: the row's
  int first[kCluster];
  u64 mass[kCluster], over[kCluster];
  u64 warp_mass[kWarps], warp_over[kWarps];
  float warp_part[kWarps];
  int warp_first[kWarps];
  int listed;  // entries of `own` (or what there would be)
  u64 part[2];  // this CTA's mass, and what of it is above an interval
  unsigned key_lo[kCluster], key_hi[kCluster], ties[kCluster];
  unsigned warp_lo[kWarps], warp_hi[kWarps];
  u64 span[kCluster];
  int tie;
  int bin, pick;
  u64 before;
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
// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// c = 256 log2(e) / T = hi + lo.  256 log2 of a weight is y c - top with y = x - shift: shift
// 0 and top an integer above max c (the common factor cancels wherever weights are
// used), or, where max c is 2^21 or more, shift max and top 0.  x - max is exact then for
// every x that weighs something: it is within 2% of max.
constexpr int kMagicBits = 0x4B400000;
constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, in the low bits
struct Heat {
  float hi, lo, max, shift;
  float magic;  // kMagic - top
  float least;  // x below it has no weight
  float none;   // a y without weight
};
__device__ __forceinline__ Heat make_heat(float max, float heat) {
  constexpr double kC = 256.0 * 1.4426950408889634;
  constexpr float kHi = (float)kC, kLo = (float)(kC - (double)kHi);
  Heat h;
  h.max = max;
  h.hi = kHi / heat;
  h.lo = (fmaf(-h.hi, heat, kHi) + kLo) / heat;
  const float m = max * h.hi;
  const bool far = !(fabsf(m) < 2097152.f);
  const float top = far ? 0.f : ceilf(m) + 1.f;
  h.shift = far ? max : 0.f;
  h.magic = kMagic - top;
  h.none = (top - kNegligible) / h.hi;
  h.least = h.shift + h.none;
  return h;
}

// Two floats in packed instructions.
struct Two {
  u64 v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void get(float* a, float* b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v)); }
};
__device__ __forceinline__ Two both(float a) { return Two(a, a); }
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two operator-(Two a, Two b) {
  Two r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Adding these rounds to multiples of 2^-22 and 2^-44, whatever is added: up to 1, and up to 2^-22.
constexpr float kHigh = 3.f, kLow = 1.5f / 2097152.f;
constexpr int kHighBits = 0x40400000, kLowBits = 0x35400000;
constexpr int kHighShift = kOne - 22;

// Weights of two y as w + l, |l| below 2^-9 w.  y from 2^-kTiny up, |y c| < 2^22.
constexpr int kTiny = 126;
__device__ __forceinline__ void weigh(Two y, const Heat& h, const int2* table, Two* w, Two* l) {
  const Two z = fma(y, both(h.hi), both(h.magic));
  const Two t = fma(y, both(h.lo), fma(y, both(h.hi), both(h.magic) - z));
  float z0, z1;
  z.get(&z0, &z1);
  const unsigned b0 = __float_as_uint(z0), b1 = __float_as_uint(z1);
  const int2 t0 = table[b0 & 255], t1 = table[b1 & 255];
  constexpr float kStep = 0.0027076061740622863f;  // ln(2) / 256
  const Two q = fma(t, fma(t, fma(t, both(kStep * kStep * kStep / 6.f), both(kStep * kStep / 2.f)), both(kStep)),
                    Two(__int_as_float(t0.y), __int_as_float(t1.y)));
  *w = Two(__uint_as_float((unsigned)t0.x + (b0 << 15)), __uint_as_float((unsigned)t1.x + (b1 << 15)));
  *l = *w * q;
}

// The integers of two weights, w 2^44 = (a - kHighBits) 2^22 + (b - kLowBits).
struct Units {
  int a[2], b[2];
};
__device__ __forceinline__ Units units(Two y, const Heat& h, const int2* table) {
  Two w, l;
  weigh(y, h, table, &w, &l);
  const Two z = (w + l) + both(kHigh), x = ((w - (z - both(kHigh))) + l) + both(kLow);  // (w - z exact)
  float a, b, c, d;
  z.get(&a, &b);
  x.get(&c, &d);
  return Units{{__float_as_int(a), __float_as_int(b)}, {__float_as_int(c), __float_as_int(d)}};
}
// Of two logits: 0 where not in, or (units_all) below least.
__device__ __forceinline__ Units units(float x0, float x1, bool in0, bool in1, const Heat& h, const int2* table) {
  float y0, y1;
  (Two(x0, x1) - both(h.shift)).get(&y0, &y1);
  return units(Two(in0 ? y0 : h.none, in1 ? y1 : h.none), h, table);
}
__device__ __forceinline__ Units units_all(float x0, float x1, const Heat& h, const int2* table) {
  float y0, y1;
  (Two(x0, x1) - both(h.shift)).get(&y0, &y1);
  return units(Two(fmaxf(y0, h.none), fmaxf(y1, h.none)), h, table);
}
__device__ __forceinline__ u64 weight_of(const Units& u, int j) {
  return ((u64)(unsigned)(u.a[j] - kHighBits) << kHighShift) + (u64)(long long)(u.b[j] - kLowBits);
}
__device__ __forceinline__ u64 weight(float x, const Heat& h, const int2* table) {  // x >= least
  return weight_of(units(x, x, true, true, h, table), 0);
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

// Of a mass W, what the running mass has to reach: the least integer >= p W, and at least 1.
__device__ __forceinline__ u64 wanted(float p, u64 whole) {
  bool cut;
  const u64 t = fraction_of(fmaxf(p, 0.f), whole, &cut);
  return t + (cut || t == 0 ? 1 : 0);
}

// floor(u W), below W.
__device__ __forceinline__ u64 drawn(float u, u64 whole) {
  bool cut;
  return u >= 1.f ? whole - 1 : u > 0.f ? fraction_of(u, whole, &cut) : 0;
}

// The float whose ordered_key() this is.
__device__ __forceinline__ float logit_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Ordered integers of the type's values.
template <typename Tin>
struct Keys;
template <>
struct Keys<float> {
  static __device__ __forceinline__ unsigned of(float x) { return ordered_key(x); }
  static __device__ __forceinline__ float value(unsigned k) { return logit_of(k); }
};
template <>
struct Keys<__nv_bfloat16> {
  static __device__ __forceinline__ unsigned of(float x) { return ordered_key(x) >> 16; }
  static __device__ __forceinline__ float value(unsigned k) {
    return __uint_as_float((k & 0x8000u ? k & 0x7fffu : ~k & 0xffffu) << 16);
  }
};

template <typename Tin>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float max(const uint4& v) {
    float x[4];
    get(v, x);
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  }
  // running largest (NaN if one is) and smallest value
  struct Extremes {
    float mx = -INFINITY, mn = INFINITY;
    __device__ __forceinline__ void add(const uint4& v) {
      float x[4];
      get(v, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mx = max_nan(mx, x[j]);
        mn = fminf(mn, x[j]);
      }
    }
    __device__ __forceinline__ float max() const { return mx; }
    __device__ __forceinline__ float min() const { return mn; }
  };
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float max(const uint4& v) {
    uint32_t m, n;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(n));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  struct Extremes {  // two values an instruction
    uint32_t mx = 0xff80ff80u, mn = 0x7f807f80u;
    __device__ __forceinline__ void add(const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(mx) : "r"(w[i]));
        asm("min.bf16x2 %0, %0, %1;" : "+r"(mn) : "r"(w[i]));
      }
    }
    __device__ __forceinline__ float max() const {
      return max_nan(__uint_as_float(mx << 16), __uint_as_float(mx & 0xffff0000u));
    }
    __device__ __forceinline__ float min() const {
      return fminf(__uint_as_float(mn << 16), __uint_as_float(mn & 0xffff0000u));
    }
  };
};

// This warp's part of a row, and what is kept of it.
struct Row {
  const unsigned char* part;  // the CTA's part in shared memory
  int base;                   // index of its first element (below 0 where that is padding)
  int lo, hi;                 // the warp's elements
  int from, to;               // the part's elements that are the row's
  Heat heat;
  float thr;                  // kept: x above thr, or equal to it with an index up to `last`
  int last;
  __device__ __forceinline__ bool kept(float x, int i) const { return x > thr || (x == thr && base + i <= last); }
  __device__ __forceinline__ void set(u64 code) {
    thr = logit_of((unsigned)(code >> kIndexBits));
    last = (int)(kIndexMask - (code & kIndexMask));
  }
  __device__ __forceinline__ float next() const {  // the float after thr
    const int bits = __float_as_int(thr);
    return thr == 0.f ? __int_as_float(1) : __int_as_float(bits + (bits < 0 ? -1 : 1));
  }
};

// The kept ones of a vector's elements by one bound each (weighed: those with a weight).
template <int kN>
struct Bounds {
  float thr, next, least;
  int last;  // in the part; -1: none of the equal ones
  __device__ __forceinline__ Bounds(const Row& row, bool weighed)
      : thr(row.thr), next(row.next()), least(weighed ? row.heat.least : -INFINITY) {
    const long long at = (long long)row.last - row.base;
    last = (int)(at < -1 ? -1 : at < (1 << 30) ? at : 1 << 30);
  }
  __device__ __forceinline__ void test(const float (&x)[kN], int i, bool (&in)[kN]) const {
    const float bound = fmaxf(i + kN - 1 <= last ? thr : next, least);
#pragma unroll
    for (int j = 0; j < kN; ++j) in[j] = x[j] >= bound;
    if (i <= last && last < i + kN - 1) {  // `last` lies inside
#pragma unroll
      for (int j = 0; j < kN; ++j) in[j] = in[j] || (x[j] == thr && i + j <= last && x[j] >= least);
    }
  }
};

// f(x, i) for the warp's elements, a vector x at the elements i, i + 1, .. per lane and step.
template <typename Tin, typename F>
__device__ __forceinline__ void for_each(const Row& row, F&& f) {
  constexpr int kN = Vec<Tin>::kN;
  for (int i = row.lo + kN * (int)(threadIdx.x & 31); i < row.hi; i += 32 * kN) {
    float x[kN];
    Vec<Tin>::get(*reinterpret_cast<const uint4*>(row.part + (size_t)i * sizeof(Tin)), x);
    f(x, i);
  }
}

// The same without the steps in which no lane's vector has an x from `bound` up.
template <typename Tin, typename F>
__device__ __forceinline__ void for_each_from(const Row& row, float bound, F&& f) {
  constexpr int kN = Vec<Tin>::kN;
  for (int i = row.lo + kN * (int)(threadIdx.x & 31); i < row.hi; i += 32 * kN) {
    const uint4 v = *reinterpret_cast<const uint4*>(row.part + (size_t)i * sizeof(Tin));
    if (!__any_sync(0xffffffffu, Vec<Tin>::max(v) >= bound)) continue;
    float x[kN];
    Vec<Tin>::get(v, x);
    f(x, i);
  }
}

// Sums of the cluster's histograms, in every CTA's tot: thread t's are intervals kPer t up.
// Tokens: one cluster barrier before, and one has to follow before cnt changes.  Mass: two.
constexpr int kPer = kBins / kThreads;
template <bool kMass>
__device__ __forceinline__ void sum_bins(cg::cluster_group& cluster, Shared& sh) {
  const int C = (int)cluster.num_blocks(), tid = threadIdx.x;
  cluster.sync();
  if (!kMass) {
    static_assert(kPer == 2, "two counters a load");
    uint2 n = make_uint2(0, 0);
    for (int q0 = 0; q0 < C; q0 += 4) {  // (four loads on their way before the first is used)
      uint2 m[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        m[q] = q0 + q < C ? *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&sh.cnt[2 * tid], q0 + q)) : make_uint2(0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        n.x += m[q].x;
        n.y += m[q].y;
      }
    }
    sh.tot[2 * tid] = n.x;
    sh.tot[2 * tid + 1] = n.y;
    return;
  }
  const int share = kBins / C, first = (int)cluster.block_rank() * share;
  for (int i = tid; i < share; i += kThreads) {
    const int bin = first + i;
    u64 w = 0;
    for (int q = 0; q < C; ++q) w += ((u64)*cluster.map_shared_rank(&sh.hi[bin], q) << 32) + *cluster.map_shared_rank(&sh.lo[bin], q);
    for (int q = 0; q < C; ++q) *cluster.map_shared_rank(&sh.tot[bin], q) = w;
  }
  cluster.sync();
}

__device__ __forceinline__ void add_mass(Shared& sh, int bin, u64 w) {
  const unsigned wl = (unsigned)w, old = atomicAdd(&sh.lo[bin], wl);
  const unsigned wh = (unsigned)(w >> 32) + (old + wl < old ? 1u : 0u);
  if (wh) atomicAdd(&sh.hi[bin], wh);
}

// The interval of tot in which the running sum, from `above` on, reaches the target, in
// sh.bin with the sum before it in sh.before; the last one where it never does.
// target(whole) gives the target for the sum of all.
template <typename F>
__device__ __forceinline__ u64 find_bin(Shared& sh, u64 above, F&& target) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const u64 want = target(whole);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if ((run < want && want <= run + mine[k]) || (tid * kPer + k == kBins - 1 && want > whole)) {
      sh.bin = tid * kPer + k;
      sh.before = run;
    }
    run += mine[k];
  }
  __syncthreads();
  return want;
}

__device__ __forceinline__ void list_own(Shared& sh, u64 code) {
  const int at = atomicAdd(&sh.listed, 1);
  if (at < kList) sh.own[at] = code;
}

// A barrier of the cluster in two halves: no thread is past the second before all have reached
// the first.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The CTAs' shares into this CTA's list, if it wants and they fit: how many there are.  A
// cluster barrier has to be passed before, and cluster_wait() before `own` changes or the CTA
// ends.  share: in lane q < C, CTA q's number.
__device__ __forceinline__ int gather_list(cg::cluster_group& cluster, Shared& sh, int share, bool want) {
  const int C = (int)cluster.num_blocks(), lane = threadIdx.x & 31;
  int end = lane < C ? min(share, kList + 1) : 0;
#pragma unroll
  for (int o = 1; o < kCluster; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += up;
  }
  const int n = __shfl_sync(0xffffffffu, end, C - 1);
  if (want && n <= kList)
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + (int)threadIdx.x;
      int q = 0, base = 0;
      for (int k = 0; k < C - 1; ++k) {
        const int e = __shfl_sync(0xffffffffu, end, k);
        if (i >= e) {
          q = k + 1;
          base = e;
        }
      }
      if (i < n) sh.list[i] = *cluster.map_shared_rank(&sh.own[i - base], q);
    }
  cluster_arrive();
  return n;
}

// A warp's 32 values in descending order.
__device__ __forceinline__ u64 sort32(u64 x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2) {
      const u64 y = __shfl_xor_sync(0xffffffffu, x, stride);
      const bool larger = ((lane & stride) == 0) == ((lane & size) == 0);  // keeps the larger one
      x = (x > y) == larger ? x : y;
    }
  return x;
}

// The first n entries, none 0 and all different, in descending order: 32 at a time in a warp's
// registers, then every entry's rank in the other lists of 32 by bisection.  (480 entries with
// their masses take 8000 to 13000 cycles beside another CTA's work; a bitonic network over all
// of them, 45 barriers, 14000 to 15700.)
__device__ __forceinline__ void sort_list(u64* v, int n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lists = (n + 31) / 32;
  u64 e[kList / kThreads];
  __syncthreads();  // (the entries are there)
#pragma unroll
  for (int q = 0; q < kList / kThreads; ++q) {
    const int l = warp + q * kWarps;
    if (l >= lists) break;
    e[q] = v[l * 32 + lane] = sort32(l * 32 + lane < n ? v[l * 32 + lane] : 0);
  }
  __syncthreads();
  int rank[kList / kThreads];
#pragma unroll
  for (int q = 0; q < kList / kThreads; ++q) {
    const int own = warp + q * kWarps;
    if (own >= lists) break;
    rank[q] = lane;
    for (int l = 0; l < lists; ++l) {
      if (l == own) continue;
      const u64* list = v + 32 * l;
      int at = 0;  // entries above e
#pragma unroll
      for (int step = 16; step > 0; step /= 2)
        if (list[at + step - 1] > e[q]) at += step;
      rank[q] += at + (list[at] > e[q] ? 1 : 0);
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kList / kThreads; ++q)
    if (warp + q * kWarps < lists && e[q]) v[rank[q]] = e[q];
  __syncthreads();
}

// The first n entries of the list in descending order, and their running masses; the logits
// are logit(entry).
template <typename F>
__device__ __forceinline__ void order_list(Shared& sh, const Heat& heat, int n, F&& logit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (n <= 32) {  // by warp 0: the barriers of all cost more than its work
    __syncthreads();
    if (warp == 0) {
      const u64 e = sort32(lane < n ? sh.list[lane] : 0);
      const float x = lane < n ? logit(e) : -INFINITY;
      sh.list[lane] = e;
      sh.sum[lane] = warp_scan64(weight_of(units(x, x, x >= heat.least, false, heat, sh.table), 0));
    }
    __syncthreads();
    return;
  }
  sort_list(sh.list, n);
  const int i = 2 * tid;
  const float x0 = i < n ? logit(sh.list[i]) : -INFINITY, x1 = i + 1 < n ? logit(sh.list[i + 1]) : -INFINITY;
  const Units w = units(x0, x1, x0 >= heat.least, x1 >= heat.least, heat, sh.table);
  const u64 w0 = weight_of(w, 0), w1 = weight_of(w, 1);
  const u64 incl = warp_scan64(w0 + w1);
  if (lane == 31) sh.warp_mass[warp] = incl;
  __syncthreads();
  u64 run = incl - w0 - w1;
  for (int q = 0; q < warp; ++q) run += sh.warp_mass[q];
  sh.sum[i] = run + w0;
  sh.sum[i + 1] = run + w0 + w1;
  __syncthreads();
}
__device__ __forceinline__ void rank_list(Shared& sh, const Heat& heat, int n) {
  order_list(sh, heat, n, [](u64 code) { return logit_of((unsigned)(code >> kIndexBits)); });
}

// The first of n entries whose running mass, from `above` on, reaches the target (there is one).
__device__ __forceinline__ int pick_entry(Shared& sh, u64 above, u64 target, int n) {
  if (threadIdx.x == 0) sh.pick = n - 1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (above + sh.sum[i] >= target && (i == 0 || above + sh.sum[i - 1] < target)) sh.pick = i;
  __syncthreads();
  return sh.pick;
}

// The codes of the kept tokens for which in(x, i) holds (none of them below `from`), in the list
// of every CTA that wants it.  Their number, above kList where the list does not hold them all.
// One cluster barrier, and cluster_wait() has to follow.
template <typename Tin, typename F>
__device__ __forceinline__ int collect(cg::cluster_group& cluster, Shared& sh, const Row& row, float from, bool want, F&& in) {
  constexpr int kN = Vec<Tin>::kN;
  const Bounds<kN> bounds(row, false);
  for_each_from<Tin>(row, fmaxf(from, row.thr), [&](const auto& x, int i) {
    bool take[kN], any = false;
    bounds.test(x, i, take);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      take[j] = take[j] && in(x[j], i + j);
      any = any || take[j];
    }
    if (!any) return;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      if (take[j]) list_own(sh, code_of(x[j], row.base + i + j));
    }
  });
  cluster.sync();
  const int lane = threadIdx.x & 31;
  return gather_list(cluster, sh, lane < (int)cluster.num_blocks() ? *cluster.map_shared_rank(&sh.listed, lane) : 0, want);
}

__device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
  if (threadIdx.x < 64) sh.cnt[kBins + threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();
}

// The least and the greatest key and the mass of the kept tokens for which in(x) holds (none of
// them below `from`); lo > hi: there is none.  One cluster barrier.
template <typename Tin, typename F>
__device__ __forceinline__ void extent(cg::cluster_group& cluster, Shared& sh, const Row& row, float from, unsigned* lo, unsigned* hi,
                                       u64* mass, F&& in) {
  constexpr int kN = Vec<Tin>::kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const Bounds<kN> bounds(row, false);
  unsigned l = ~0u, h = 0;
  u64 sum = 0;
  for_each_from<Tin>(row, fmaxf(from, row.thr), [&](const auto& x, int i) {
    bool take[kN];
    bounds.test(x, i, take);
#pragma unroll
    for (int j = 0; j < kN; j += 2) {
      take[j] = take[j] && in(x[j]);
      take[j + 1] = take[j + 1] && in(x[j + 1]);
      if (!__any_sync(0xffffffffu, take[j] || take[j + 1])) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (take[j + e]) {
          l = min(l, Keys<Tin>::of(x[j + e]));
          h = max(h, Keys<Tin>::of(x[j + e]));
        }
      const Units w = units(x[j], x[j + 1], take[j] && x[j] >= row.heat.least, take[j + 1] && x[j + 1] >= row.heat.least, row.heat, sh.table);
      sum += weight_of(w, 0) + weight_of(w, 1);
    }
  });
  l = __reduce_min_sync(0xffffffffu, l);
  h = __reduce_max_sync(0xffffffffu, h);
  sum = warp_sum64(sum);
  if (lane == 0) {
    sh.warp_lo[warp] = l;
    sh.warp_hi[warp] = h;
    sh.warp_mass[warp] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    l = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.warp_lo[lane] : ~0u);
    h = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.warp_hi[lane] : 0u);
    sum = warp_sum64(lane < kWarps ? sh.warp_mass[lane] : 0);
    if (lane < C) {
      *cluster.map_shared_rank(&sh.key_lo[rank], lane) = l;
      *cluster.map_shared_rank(&sh.key_hi[rank], lane) = h;
      *cluster.map_shared_rank(&sh.span[rank], lane) = sum;
    }
  }
  cluster.sync();
  *lo = ~0u;
  *hi = 0;
  *mass = 0;
  for (int q = 0; q < C; ++q) {
    *lo = min(*lo, sh.key_lo[q]);
    *hi = max(*hi, sh.key_hi[q]);
    *mass += sh.span[q];
  }
}

// Of the kept tokens equal to v, those up to the m-th by index stay, and nothing below v.
template <typename Tin>
__device__ __forceinline__ void pick_tie(cg::cluster_group& cluster, Shared& sh, Row& row, float v, unsigned m) {
  constexpr int kN = Vec<Tin>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const Bounds<kN> bounds(row, false);
  auto equal = [&](const float (&x)[kN], int i, bool (&in)[kN]) {
    unsigned n = 0;
    bounds.test(x, i, in);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      in[j] = in[j] && x[j] == v;
      n += in[j] ? 1u : 0u;
    }
    return n;
  };
  unsigned mine = 0;
  for_each_from<Tin>(row, v, [&](const auto& x, int i) {
    bool in[kN];
    mine += equal(x, i, in);
  });
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) sh.warp_lo[warp] = mine;
  if (tid == 0) sh.tie = INT_MAX;  // (all stay)
  __syncthreads();
  if (warp == 0) {
    const unsigned sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_lo[lane] : 0u);
    if (lane < C) *cluster.map_shared_rank(&sh.ties[rank], lane) = sum;
  }
  cluster.sync();
  unsigned left = m;
  for (int q = 0; q < rank; ++q) left -= min(left, sh.ties[q]);
  if (left > 0 && left <= sh.ties[rank]) {
    int w = 0;
    while (w < kWarps - 1 && left > sh.warp_lo[w]) left -= sh.warp_lo[w++];
    if (w == warp) {
      for (int i0 = row.lo; i0 < row.hi; i0 += 32 * kN) {
        const int i = i0 + kN * lane;
        float x[kN];
        Vec<Tin>::get(*reinterpret_cast<const uint4*>(row.part + (size_t)i * sizeof(Tin)), x);
        bool in[kN];
        const unsigned n = equal(x, i, in), before = (unsigned)warp_scan64(n) - n;
        if (before < left && left <= before + n) {  // (one lane)
          unsigned run = before;
          int at = 0;
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            run += in[j] ? 1u : 0u;
            if (in[j] && run == left) at = j;
          }
          for (int q = 0; q < C; ++q) *cluster.map_shared_rank(&sh.tie, q) = row.base + i + at;
        }
        const unsigned all = __shfl_sync(0xffffffffu, before + n, 31);
        if (left <= all) break;
        left -= all;
      }
    }
  }
  cluster.sync();
  row.thr = v;
  row.last = sh.tie;
}

// The threshold of the kept tokens with keys lo .. hi at which the running count (kMass: mass)
// from the greatest on, `above` at the start, reaches the target; where it does not, all
// stay.  Returns it there.
template <typename Tin, bool kMass>
__device__ __forceinline__ u64 refine(cg::cluster_group& cluster, Shared& sh, Row& row, unsigned lo, unsigned hi, u64 above,
                                      u64 target) {
  constexpr int kN = Vec<Tin>::kN;
  const int tid = threadIdx.x;
  for (;;) {
    if (lo > hi) return above;
    if (lo == hi) {
      const float v = Keys<Tin>::value(lo);
      const u64 w = kMass ? weight(v, row.heat, sh.table) : 1;
      const u64 m = (target - above + w - 1) / w;
      pick_tie<Tin>(cluster, sh, row, v, (unsigned)min(m, (u64)INT_MAX));
      return above + m * w;
    }
    const int shift = max(0, 32 - __clz((int)(hi - lo)) - 10);  // hi - lo < 2^(shift + 10), kBins intervals of 2^shift
    const bool mass = kMass && shift > 0;  // (else an interval is a value: its mass follows from its count)
    clear_bins(sh);
    const Bounds<kN> bounds(row, kMass);
    for_each_from<Tin>(row, fmaxf(Keys<Tin>::value(lo), row.thr), [&](const auto& x, int i) {
      bool in[kN];
      bounds.test(x, i, in);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const unsigned key = Keys<Tin>::of(x[j]);
        if (!in[j] || key < lo || key > hi) continue;
        const int bin = (int)((hi - key) >> shift);
        if (mass) add_mass(sh, bin, weight(x[j], row.heat, sh.table));
        else atomicAdd(&sh.cnt[bin], 1u);
      }
    });
    if (mass) {
      sum_bins<true>(cluster, sh);
    } else {
      sum_bins<false>(cluster, sh);
      if (kMass)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const unsigned off = (unsigned)(tid * kPer + k);
          if (off <= hi - lo) sh.tot[off] *= weight(Keys<Tin>::value(hi - off), row.heat, sh.table);
        }
    }
    find_bin(sh, above, [&](u64) { return target; });
    const unsigned off = (unsigned)sh.bin << shift;
    above = sh.before;
    if (off > hi - lo) {  // not reached
      cluster.sync();     // (all have read cnt)
      return above;
    }
    hi -= off;
    if (hi - lo >= (1u << shift)) lo = hi - ((1u << shift) - 1);
    if (shift > 0) {
      const unsigned l = lo, h = hi;
      u64 unused;
      extent<Tin>(cluster, sh, row, Keys<Tin>::value(l), &lo, &hi, &unused, [&](float x) {
        const unsigned key = Keys<Tin>::of(x);
        return (!kMass || x >= row.heat.least) && key >= l && key <= h;
      });
    }
  }
}

// Intervals of x from its maximum on, in one packed multiply-add and, for the place in cnt, one
// minimum, which gives what lies in the last interval or past it a place a lane.
struct Places {
  static constexpr float kLeast = 1e-34f;  // (step and width stay normal numbers: no place is NaN)
  float max, step, width;
  __device__ __forceinline__ Places(float max, float range)
      : max(max), step((float)kBins / fmaxf(range, kLeast)), width(fmaxf(range, kLeast) / (float)kBins) {}
  __device__ __forceinline__ void at(float x0, float x1, int (&place)[2]) const {
    const int last = kBins - 1 + (int)(threadIdx.x & 31);
    float f0, f1;
    fma(both(max) - Two(x0, x1), both(step), both(kMagic)).get(&f0, &f1);
    place[0] = min(__float_as_int(f0) - kMagicBits, last);
    place[1] = min(__float_as_int(f1) - kMagicBits, last);
  }
  __device__ __forceinline__ int bin(float x) const {
    return min(__float_as_int(__fmaf_rn(__fsub_rn(max, x), step, kMagic)) - kMagicBits, kBins - 1);
  }
  // a bound below every x of the intervals up to b
  __device__ __forceinline__ float from(int b) const {
    return b < kBins - 1 ? max - (float)(b + 1) * width - fabsf(max) * 0x1p-22f : -INFINITY;
  }
};

// The cluster's histogram of the kept tokens in tot.  Of an unfiltered row, what has no weight
// and what is outside the row counts as of the last interval.
template <typename Tin>
__device__ __forceinline__ void count_bins(cg::cluster_group& cluster, Shared& sh, const Row& row, const Places& places) {
  constexpr int kN = Vec<Tin>::kN;
  const int lane = threadIdx.x & 31;
  clear_bins(sh);
  if (row.thr == -INFINITY) {
    for_each<Tin>(row, [&](const auto& x, int) {
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        int at[2];
        places.at(x[j], x[j + 1], at);
        atomicAdd(&sh.cnt[at[0]], 1u);
        atomicAdd(&sh.cnt[at[1]], 1u);
      }
    });
  } else {
    const Bounds<kN> bounds(row, false);
    for_each_from<Tin>(row, bounds.thr, [&](const auto& x, int i) {
      bool in[kN];
      bounds.test(x, i, in);
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        int at[2];
        places.at(x[j], x[j + 1], at);
        atomicAdd(&sh.cnt[in[j] ? at[0] : kBins + 32 + lane], 1u);  // (no branch)
        atomicAdd(&sh.cnt[in[j + 1] ? at[1] : kBins + 32 + lane], 1u);
      }
    });
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const unsigned last = __reduce_add_sync(0xffffffffu, sh.cnt[kBins - 1 + lane]);
    if (lane == 0) sh.cnt[kBins - 1] = last;
  }
  sum_bins<false>(cluster, sh);
}

// top-k by counts: the row's threshold.
template <typename Tin>
__device__ __forceinline__ void top_count(cg::cluster_group& cluster, Shared& sh, Row& row, float range, int k) {
  const Places places(row.heat.max, range);
  count_bins<Tin>(cluster, sh, row, places);
  u64 whole = 0;
  find_bin(sh, 0, [&](u64 w) {
    whole = w;
    return (u64)k;
  });
  if (row.thr != -INFINITY && whole <= (u64)k) {  // all stay
    cluster.sync();  // (all have read cnt)
    return;
  }
  const int b = sh.bin, left = k - (int)sh.before;
  const int n = collect<Tin>(cluster, sh, row, places.from(b), true, [&](float x, int) { return places.bin(x) == b; });
  if (n <= kList) {
    sort_list(sh.list, n);
    if (left <= n) row.set(sh.list[left - 1]);  // (more than there are, with the last interval: all stay)
    __syncthreads();
    cluster_wait();
    return;
  }
  cluster_wait();
  unsigned lo, hi;
  u64 mass;
  extent<Tin>(cluster, sh, row, places.from(b), &lo, &hi, &mass, [&](float x) { return places.bin(x) == b; });
  refine<Tin, false>(cluster, sh, row, lo, hi, 0, (u64)left);
}

// The same for the mass and top_p = p, by an estimate of the interval.  *total: the mass kept.
// True: sh.over holds the CTAs' masses above the interval, sh.warp_over the warps'; the rest of
// what is kept is the list up to sh.pick.  False: the threshold is in sh.crowd.
template <typename Tin>
__device__ __forceinline__ bool nucleus(cg::cluster_group& cluster, Shared& sh, Row& row, float range, float heat, float p,
                                        u64* total) {
  constexpr int kN = Vec<Tin>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster.num_blocks();
  const Bounds<kN> bounds(row, true);
  const bool dense = row.thr == -INFINITY;
  const Places places(row.heat.max, range);
  count_bins<Tin>(cluster, sh, row, places);
  if (dense && tid == kThreads - 1) sh.tot[kBins - 1] -= sh.hidden[0];  // (its own entry: they are no tokens of the last interval)
  // the interval in which p of the mass is reached, a token taken to weigh what its interval's middle does
  const float fall = range > 0.f ? -1.4426950f * range / ((float)kBins * heat) : 0.f;
  float mine[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum += mine[k] = (float)sh.tot[tid * kPer + k] * exp2f(fall * (float)(tid * kPer + k));
  float run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) sh.warp_part[warp] = run;
  if (tid == 0) sh.bin = kBins - 1;
  __syncthreads();
  run -= sum;
  float whole = 0.f;
  for (int q = 0; q < kWarps; ++q) {
    if (q < warp) run += sh.warp_part[q];
    whole += sh.warp_part[q];
  }
  const float goal = p * whole;  // (not of the exact mass: the first tokens' errors are in both sides)
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    run += mine[k];
    if (run >= goal && mine[k] > 0.f) {
      atomicMin(&sh.bin, tid * kPer + k);
      break;
    }
  }
  __syncthreads();
  int bin = sh.bin;
  for (int tries = 0;; ++tries) {
    // its neighbours along with it while that is few tokens: where few tokens hold the mass
    // the estimate is rough
    int lo = bin, hi = bin;
    for (u64 n = sh.tot[bin]; lo > 0 && hi < kBins - 1 && hi - bin < 8; --lo, ++hi)
      if ((n += sh.tot[lo - 1] + sh.tot[hi + 1]) > kAround) break;
    // exact: the whole mass, the mass above these intervals, their tokens (from xe to xt)
    const float xt = lo > 0 ? fmaf(0.5f - (float)lo, places.width, row.heat.max) : INFINITY;
    const float xe = fmaxf(hi < kBins - 1 ? fmaf(-0.5f - (float)hi, places.width, row.heat.max) : -INFINITY, row.heat.least);
    unsigned high = 0, low = 0, high1 = 0, low1 = 0;
    auto step_of = [&](auto dense_t, const auto& x, int i) {
      constexpr bool kDense = decltype(dense_t)::value;
      bool in[kN], any = false;
      if (!kDense) bounds.test(x, i, in);
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        const Units w = kDense ? units_all(x[j], x[j + 1], row.heat, sh.table)
                               : units(x[j], x[j + 1], in[j], in[j + 1], row.heat, sh.table);
        high += (unsigned)(w.a[0] + w.a[1]);
        low += (unsigned)(w.b[0] + w.b[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool over = x[j + e] > xt;  // (what is not in weighs nothing)
          if (over) {
            high1 += (unsigned)(w.a[e] - kHighBits);
            low1 += (unsigned)(w.b[e] - kLowBits);
          }
          in[j + e] = (kDense || in[j + e]) && !over && x[j + e] >= xe;
          any = any || in[j + e];
        }
      }
      high -= (unsigned)kN * kHighBits;
      low -= (unsigned)kN * kLowBits;
      if (any)
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (in[j]) list_own(sh, code_of(x[j], row.base + i + j));
    };
    if (dense) for_each<Tin>(row, [&](const auto& x, int i) { step_of(std::true_type{}, x, i); });
    else for_each_from<Tin>(row, bounds.thr, [&](const auto& x, int i) { step_of(std::false_type{}, x, i); });
    const u64 all = warp_sum64(((u64)high << kHighShift) + (u64)(long long)(int)low);
    const u64 over = warp_sum64(((u64)high1 << kHighShift) + (u64)(long long)(int)low1);
    if (lane == 0) {
      sh.warp_mass[warp] = all;
      sh.warp_over[warp] = over;
    }
    __syncthreads();
    if (warp < 2) {
      const u64 v = warp_sum64(lane < kWarps ? (warp ? sh.warp_over[lane] : sh.warp_mass[lane]) : 0);
      if (lane == 0) sh.part[warp] = v;
    }
    cluster.sync();
    u64 mass = 0, above = 0;
    int share = 0;
    if (lane < C) {
      share = *cluster.map_shared_rank(&sh.listed, lane);
      const u64* part = cluster.map_shared_rank(&sh.part[0], lane);
      mass = part[0];
      above = part[1];
    }
    const int n = gather_list(cluster, sh, share, true);
    if (warp == 0 && lane < C) sh.over[lane] = above;
    mass = warp_sum64(mass);
    above = warp_sum64(above);
    const u64 target = wanted(p, mass);
    if (n <= kList) {
      if (n) rank_list(sh, row.heat, n);
      const u64 here = n ? sh.sum[n - 1] : 0;
      if (target > above && target <= above + here) {
        const int i = pick_entry(sh, above, target, n);
        row.set(sh.list[i]);
        *total = above + sh.sum[i];
        cluster_wait();
        return true;
      }
    }
    cluster_wait();
    bin = target <= above ? lo - 1 : hi + 1;
    const bool whole_row = tries == 2 || bin < 0 || bin >= kBins;  // (the estimate is of no use)
    if (whole_row || (n > kList && target > above)) {
      if (tid == 0) sh.crowd = whole_row ? Crowd{row.heat.least, INFINITY, 0, target} : Crowd{xe, xt, above, target};
      __syncthreads();
      return false;
    }
    __syncthreads();  // (sh.sum and sh.bin have been read)
    if (tid == 0) sh.listed = 0;
    __syncthreads();
  }
}

// The threshold in sh.crowd; returns the mass kept.
template <typename Tin>
__device__ __forceinline__ u64 settle(cg::cluster_group& cluster, Shared& sh, Row& row) {
  unsigned lo, hi;
  u64 here;
  const float xe = sh.crowd.xe, xt = sh.crowd.xt;
  extent<Tin>(cluster, sh, row, xe, &lo, &hi, &here, [&](float x) { return x >= xe && x <= xt; });
  u64 above = sh.crowd.above;
  if (sh.crowd.target > above + here) {  // below it
    above += here;
    lo = Keys<Tin>::of(row.heat.least);
    hi = Keys<Tin>::of(xe);
    if (Keys<Tin>::value(hi) >= xe) --hi;
  }
  return refine<Tin, true>(cluster, sh, row, lo, hi, above, sh.crowd.target);
}

// All filters and the draw among the n tokens of the list, which hold the first k of the row.
// Sets the row's threshold, returns the mass kept; *token, if wanted: the token drawn.
__device__ __forceinline__ u64 small_row(Shared& sh, Row& row, int n, int k, float p, float u, int32_t* token) {
  rank_list(sh, row.heat, n);
  int m = min(k, n);
  if (p < 1.f) m = pick_entry(sh, 0, wanted(p, sh.sum[m - 1]), m) + 1;
  const u64 whole = sh.sum[m - 1];
  row.set(sh.list[m - 1]);
  __syncthreads();
  if (token) {  // the kept ones by index
    for (int i = threadIdx.x; i < m; i += kThreads) {
      const u64 code = sh.list[i];
      sh.list[i] = (code & kIndexMask) << 32 | code >> kIndexBits;
    }
    order_list(sh, row.heat, m, [](u64 entry) { return logit_of((unsigned)entry); });
    const int i = pick_entry(sh, 0, drawn(u, whole) + 1, m);
    if (threadIdx.x == 0) *token = (int32_t)(kIndexMask - (sh.list[i] >> 32));
  }
  return whole;
}

// The part's elements into shared memory: whole 16-byte units by asynchronous copies, the
// units at the row's ends element by element, -inf outside the row.  Elements
// [head, head + V) of the padded row, whose element 0 lies at the 16-byte boundary `src`.
template <typename Tin>
__device__ __forceinline__ void load_part(const Tin* src, unsigned char* dst, int start, int lo, int hi, int head, int V) {
  constexpr int kN = Vec<Tin>::kN;
  for (int i = lo + kN * (int)(threadIdx.x & 31); i < hi; i += 32 * kN) {
    const int at = start + i;
    if (at >= head && at + kN <= head + V) {
      const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst + (size_t)i * sizeof(Tin)));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src + at) : "memory");
    } else {
      Tin* out = reinterpret_cast<Tin*>(dst) + i;
#pragma unroll
      for (int j = 0; j < kN; ++j)
        out[j] = at + j >= head && at + j < head + V ? src[at + j] : static_cast<Tin>(-INFINITY);
    }
  }
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  constexpr int kN = Vec<Tin>::kN;
  extern __shared__ __align__(16) unsigned char part_sh[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / C, b = r / a.N, node = r % a.N;
  const int set = a.per_row ? r : b;  // the row's settings

  Row row;
  row.part = part_sh;
  const Tin* src = static_cast<const Tin*>(a.logits) + (long long)b * a.l_batch + (long long)node * a.l_row;
  const int head = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(Tin));
  // the padded row in units of a warp's vectors: CTA q has those from first(q) on
  constexpr int kUnit = 32 * kN;
  const int n_units = (head + a.V + kUnit - 1) / kUnit;
  const int log_c = 31 - __clz(C);  // (a power of two)
  const auto first = [&](int q) { return n_units * q >> log_c; };
  const int u0 = first(rank), mine_units = first(rank + 1) - u0;
  row.lo = mine_units * warp / kWarps * kUnit;
  row.hi = mine_units * (warp + 1) / kWarps * kUnit;
  row.base = u0 * kUnit - head;
  row.from = max(0, -row.base);
  row.to = min(mine_units * kUnit, a.V - row.base);
  float heat = a.temperature ? a.temperature[set] : 1.f;
  int k = a.top_k ? a.top_k[set] : 0;
  const float p = a.top_p ? a.top_p[set] : 1.f, least = a.min_p ? a.min_p[set] : 0.f, u = a.u ? a.u[r] : 0.f;
  load_part<Tin>(src - head, part_sh, u0 * kUnit, row.lo, row.hi, head, a.V);
  if (tid < 256) sh.table[-tid & 255] = make_int2(kTable.hi[tid], __float_as_int(kTable.d[tid]));
  const bool valid = heat >= 0.f && heat < INFINITY && p == p && least == least;
  if (heat == 0.f) {
    heat = 1.f;
    k = 1;
  }
  // c stays a normal number.  Its low part is a denormal one from about 1e32 on, off by up to
  // 2^-150: times the |x - max| of a token that weighs something, at most 87 T, 2^-34 of its weight
  // at 3e35 (what all tokens have in common cancels).
  heat = fminf(fmaxf(heat, 4e-34f), 3e35f);
  // (in double by one thread: all 512 at the rate of that pipe take 5 us)
  if (tid == 32 && least > 0.f) sh.least = (double)heat * log(fmin((double)least, 1.0));
  asm volatile("cp.async.wait_all;" ::: "memory");
  // the thread's, the CTA's and the row's largest value (NaN if one is) and smallest
  typename Vec<Tin>::Extremes extremes;
  for (int i = row.lo + kN * lane; i < row.hi; i += 32 * kN)
    extremes.add(*reinterpret_cast<const uint4*>(part_sh + (size_t)i * sizeof(Tin)));
  float mx = extremes.max(), mn = extremes.min();
  const float own = mx;
  // The smallest logit bounds the intervals of top-k and top-p, so that what is never kept, masked
  // tokens and padding, must not count: with one of it in a flat row all tokens would lie in a few
  // of the intervals (256 rows of 50257 fp32, logits within 0.2: top-p 206 us instead of 73).
  unsigned hidden = 0;
  if (mn == -INFINITY && k != 1 && ((k > 0 && k < a.V) || p < 1.f)) {
    mn = INFINITY;
    for (int i = row.lo + kN * lane; i < row.hi; i += 32 * kN) {
      float x[kN];
      Vec<Tin>::get(*reinterpret_cast<const uint4*>(part_sh + (size_t)i * sizeof(Tin)), x);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const bool none = x[j] == -INFINITY;
        mn = fminf(mn, none ? INFINITY : x[j]);
        hidden += none ? 1u : 0u;
      }
    }
  }
  hidden = __reduce_add_sync(0xffffffffu, hidden);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  if (lane == 0) {
    sh.ends[warp] = make_float2(mx, mn);
    sh.hidden[warp] = hidden;
  }
  __syncthreads();
  if (warp == 0) {
    hidden = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.hidden[lane] : 0u);
    mx = sh.ends[lane % kWarps].x;
    mn = sh.ends[lane % kWarps].y;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (lane == 0) {
      sh.end = make_float2(mx, mn);
      sh.all_hidden = hidden;
    }
  }
  cluster.sync();
  {
    const float2 end = *cluster.map_shared_rank(&sh.end, lane & (C - 1));
    mx = end.x;
    mn = end.y;
  }
  if (warp == 0) {
    hidden = __reduce_add_sync(0xffffffffu, lane < C ? *cluster.map_shared_rank(&sh.all_hidden, lane) : 0u);
    if (lane == 0) sh.hidden[0] = hidden;
  }
#pragma unroll
  for (int o = kCluster / 2; o > 0; o >>= 1) {
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  float* out = a.probs ? a.probs + (long long)b * a.p_batch + (long long)node * a.p_row + row.base : nullptr;
  // no finite maximum, NaN or +inf among the logits, or settings that mean nothing
  if (!(mx > -INFINITY && mx < INFINITY) || !valid) {
    if (rank == 0 && tid == 0) {
      raise_flag(a.flags, MLA_DEV_BAD_VALUE);
      if (a.token) a.token[r] = -1;
    }
    if (out)
      for (int i = max(row.lo, row.from) + lane; i < min(row.hi, row.to); i += 32) out[i] = qnan();
    cluster.sync();  // (all have read ends)
    return;
  }
  row.heat = make_heat(mx, heat);
  row.thr = -INFINITY;
  row.last = INT_MIN;
  if (least > 0.f) {  // w >= least, as a bound of x
    row.thr = __double2float_ru((double)mx + sh.least);
    row.last = INT_MAX;
  }
  const float spread = mx - mn;
  u64 total = 0;
  bool done = false;  // token and total are known
  if (k == 1) {       // the first token of the order
    int first = INT_MAX;
    for_each_from<Tin>(row, mx, [&](const auto& x, int i) {
#pragma unroll
      for (int j = kN - 1; j >= 0; --j)
        if (x[j] == mx) first = min(first, row.base + i + j);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.warp_first[warp] = first;
    __syncthreads();
    if (warp == 0) {
      first = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.warp_first[lane] : INT_MAX);
      if (lane < C) *cluster.map_shared_rank(&sh.first[rank], lane) = first;
    }
    cluster.sync();
    first = sh.first[0];
    for (int q = 1; q < C; ++q) first = min(first, sh.first[q]);
    row.thr = mx;
    row.last = first;
    total = weight(mx, row.heat, sh.table);
    if (a.token && rank == 0 && tid == 0) a.token[r] = first;
    done = true;
  } else if (k > 0 && k < a.V) {
    const float range = fminf(spread, 64.f);
    int n = 0;  // tokens listed
    if (k <= (p < 1.f ? kSmallKTopP : kSmallK)) {
      // the k-th of the threads' largest tokens lies in interval b0: no token of the first k lies behind it
      const Places places(mx, range);
      clear_bins(sh);
      const int bin = places.bin(own);
      const bool there = own > row.thr || (own == row.thr && row.last == INT_MAX);
      const unsigned same = __ballot_sync(0xffffffffu, there && bin == kBins - 1);
      if (there && bin < kBins - 1) atomicAdd(&sh.cnt[bin], 1u);
      if (lane == 0 && same) atomicAdd(&sh.cnt[kBins - 1], (unsigned)__popc(same));
      sum_bins<false>(cluster, sh);
      find_bin(sh, 0, [&](u64) { return (u64)k; });
      const int b0 = sh.bin;
      n = collect<Tin>(cluster, sh, row, places.from(b0), rank == 0 || out, [&](float x, int) { return places.bin(x) <= b0; });
      if (n > kList) {
        n = 0;
        cluster_wait();
      }
    }
    if (n > 0) {
      if (rank != 0 && !out) {  // (one CTA is enough for the token)
        cluster_wait();
        return;
      }
      total = small_row(sh, row, n, k, p, u, a.token && rank == 0 ? a.token + r : nullptr);
      cluster_wait();
      done = true;
    } else {
      top_count<Tin>(cluster, sh, row, range, k);
    }
  }
  bool listed = false;  // the kept tokens: those above an interval, and some of the list
  if (!done && p < 1.f) {
    // tokens past the range hold less than (1 - p) / e^5 of the mass, whatever their number
    const float tail = logf((float)a.V) - logf(fmaxf(1.f - p, 1e-7f)) + 5.f;
    const float range = fminf(spread, tail * heat);
    listed = nucleus<Tin>(cluster, sh, row, range, heat, p, &total);
    if (!listed) total = settle<Tin>(cluster, sh, row);
  }
  if (listed && a.token) {
    // the CTAs' and this CTA's warps' kept masses: above the interval, and from the list
    u64 mine = 0, theirs = 0;
    for (int i = lane; i <= sh.pick; i += 32) {
      const int at = (int)(kIndexMask - (sh.list[i] & kIndexMask)) + head, own = at - u0 * kUnit;
      const u64 w = sh.sum[i] - (i ? sh.sum[i - 1] : 0);
      if (at >= first(warp) * kUnit && at < first(warp + 1) * kUnit) theirs += w;  // (of CTA `warp`)
      if (own >= row.lo && own < row.hi) mine += w;
    }
    mine = warp_sum64(mine);
    theirs = warp_sum64(theirs);
    if (lane == 0) {
      sh.warp_mass[warp] = sh.warp_over[warp] + mine;
      if (warp < C) sh.mass[warp] = sh.over[warp] + theirs;
    }
    __syncthreads();
  }
  if (!done && !listed && (a.token || p >= 1.f)) {
    const Bounds<kN> bounds(row, true);
    unsigned high = 0, low = 0;  // sums of the weights' integers: less than 2^8 of them
    auto add = [&](const Units& w) {
      high += (unsigned)(w.a[0] + w.a[1]) - 2u * kHighBits;
      low += (unsigned)(w.b[0] + w.b[1]) - 2u * kLowBits;
    };
    if (row.thr == -INFINITY) {  // straight through, so that the vector's chains overlap
      for_each<Tin>(row, [&](const auto& x, int) {
#pragma unroll
        for (int j = 0; j < kN; j += 2) add(units_all(x[j], x[j + 1], row.heat, sh.table));
      });
    } else {
      for_each_from<Tin>(row, bounds.thr, [&](const auto& x, int i) {
        bool in[kN];
        bounds.test(x, i, in);
#pragma unroll
        for (int j = 0; j < kN; j += 2)
          if (__any_sync(0xffffffffu, in[j] || in[j + 1])) add(units(x[j], x[j + 1], in[j], in[j + 1], row.heat, sh.table));
      });
    }
    u64 mine = ((u64)high << kHighShift) + (u64)(long long)(int)low;
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
  if (a.token && !done) {
    // the CTA, the warp, the element at which the running mass exceeds t < total
    const Bounds<kN> bounds(row, true);
    u64 t = drawn(u, total);
    for (int q = 0; q < rank; ++q) t -= sh.mass[q];  // (wraps where the draw is before this CTA)
    if (t < sh.mass[rank]) {
      int w = 0;
      while (w < kWarps - 1 && t >= sh.warp_mass[w]) t -= sh.warp_mass[w++];
      // that warp's elements by all warps (by itself, step after step, 7500 cycles)
      const int lo = mine_units * w / kWarps * kUnit, hi = mine_units * (w + 1) / kWarps * kUnit;
      for (int i0 = lo; i0 < hi; i0 += kThreads * kN) {
        const int i = i0 + kN * tid;
        u64 v[kN], sum = 0;
        if (i - kN * lane < hi) {
          float x[kN];
          Vec<Tin>::get(*reinterpret_cast<const uint4*>(part_sh + (size_t)i * sizeof(Tin)), x);
          bool in[kN];
          bounds.test(x, i, in);
#pragma unroll
          for (int j = 0; j < kN; j += 2) {
            const Units m = units(x[j], x[j + 1], in[j], in[j + 1], row.heat, sh.table);
            sum += v[j] = weight_of(m, 0);
            sum += v[j + 1] = weight_of(m, 1);
          }
        }
        const u64 incl = warp_scan64(sum);
        if (lane == 31) sh.warp_over[warp] = incl;
        __syncthreads();
        u64 run = incl - sum, all = 0;
        for (int q = 0; q < kWarps; ++q) {
          if (q < warp) run += sh.warp_over[q];
          all += sh.warp_over[q];
        }
        if (run <= t && t < run + sum) {  // (one thread)
          int at = -1;
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            run += v[j];
            if (at < 0 && run > t) at = j;
          }
          a.token[r] = row.base + i + at;
        }
        if (t < all) break;
        t -= all;
        __syncthreads();
      }
    }
  }
  if (out) {
    // 2^kOne / total as a pair: the quotient's own error would be in every probability
    const float t_hi = __ull2float_rn(total), t_lo = (float)(long long)(total - __float2ull_rn(t_hi));
    const float inv = (float)(1ull << kOne) / t_hi;
    const float inv_lo = fmaf(-t_lo, inv, fmaf(-t_hi, inv, (float)(1ull << kOne))) / t_hi;
    const float tiny = row.heat.none - (256.f * kTiny - kNegligible) / row.heat.hi;
    const bool dense = row.thr == -INFINITY;
    // probabilities of two logits, in0 and in1: whether they are kept
    auto probability = [&](float x0, float x1, bool in0, bool in1, float* v0, float* v1) {
      float y0, y1, a0, a1;
      (Two(x0, x1) - both(row.heat.shift)).get(&y0, &y1);
      Two w, l;
      weigh(Two(fmaxf(y0, tiny), fmaxf(y1, tiny)), row.heat, sh.table, &w, &l);
      const Two hi = w + l, lo = l - (hi - w);
      fma(hi, both(inv), fma(hi, both(inv_lo), lo * both(inv))).get(&a0, &a1);
      *v0 = in0 && y0 >= tiny ? a0 : 0.f;
      *v1 = in1 && y1 >= tiny ? a1 : 0.f;
    };
    if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {  // the vectors' places are 16-byte units
      const Bounds<kN> bounds(row, false);
      for (int i = row.lo + kN * lane; i < row.hi; i += 32 * kN) {
        const uint4 vec = *reinterpret_cast<const uint4*>(part_sh + (size_t)i * sizeof(Tin));
        float x[kN], v[kN];
        if (dense) {
          Vec<Tin>::get(vec, x);
#pragma unroll
          for (int j = 0; j < kN; j += 2) probability(x[j], x[j + 1], true, true, &v[j], &v[j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < kN; ++j) v[j] = 0.f;
          if (__any_sync(0xffffffffu, Vec<Tin>::max(vec) >= row.thr)) {
            Vec<Tin>::get(vec, x);
            bool in[kN];
            bounds.test(x, i, in);
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
              if (k == 1) {
                v[j] = in[j] ? 1.f : 0.f;
                v[j + 1] = in[j + 1] ? 1.f : 0.f;
              } else if (__any_sync(0xffffffffu, in[j] || in[j + 1])) {
                probability(x[j], x[j + 1], in[j], in[j + 1], &v[j], &v[j + 1]);
              }
            }
          }
        }
        if (i >= row.from && i + kN <= row.to) {
#pragma unroll
          for (int j = 0; j < kN; j += 4) *reinterpret_cast<float4*>(out + i + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (i + j >= row.from && i + j < row.to) out[i + j] = v[j];
        }
      }
    } else {  // an element per lane, so that a warp's stores are neighbours
      const Tin* xs = reinterpret_cast<const Tin*>(part_sh);
      const int end = min(row.hi, row.to);
      for (int i = max(row.lo, row.from) + lane; i - lane < end; i += 64) {
        const bool there0 = i < end, there1 = i + 32 < end;
        const float x0 = there0 ? to_f32(xs[i]) : -INFINITY, x1 = there1 ? to_f32(xs[i + 32]) : -INFINITY;
        const bool in0 = dense || row.kept(x0, i), in1 = dense || row.kept(x1, i + 32);
        float v0 = in0 ? 1.f : 0.f, v1 = in1 ? 1.f : 0.f;
        if (k != 1 && __any_sync(0xffffffffu, in0 || in1)) probability(x0, x1, in0, in1, &v0, &v1);
        if (there0) out[i] = v0;
        if (there1) out[i + 32] = v1;
      }
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
  // as few CTAs a row as leave room for two on an SM, more while the GPU is not full
  constexpr int kN = Vec<Tin>::kN, kUnit = 32 * kN, kHalf = 73728;
  const long long rows = (long long)a.B * a.N;
  const int units = (a.V + kN - 1 + kUnit - 1) / kUnit;  // (wherever the row begins in its first vector)
  const auto part = [&](int C) { return (size_t)((units + C - 1) / C) * kUnit * sizeof(Tin); };
  int C = 1;
  while (C < kCluster && part(C) > kHalf) C *= 2;
  while (C < kCluster && rows * C * 2 <= sms && a.V / C > 2048) C *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = part(C);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<Tin>, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  return a.dtype == MLA_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace mla
