// tree_simt.cu -- CUDA-core tree attention (fp32, and bf16 outside the
// tensor-core geometry), kv_lora up to 512.
//
// The absorbed path of the page "MLA 注意力与 KV 缓存", §2.3, for the nodes of
// a drafted tree.  A CTA takes 16 query rows (node, head) of one sequence and
// one split of its keys, which pass through shared memory 32 to 128 at a time: 16
// threads per row form 2 to 8 scores each, reduce the maximum and the sum among
// themselves and accumulate kv_lora / 16 latents each.  A key row is thus read once per
// 16 query rows.  The keys are split until the grid fills the GPU (a toy model
// on one sequence has one group of rows); a second kernel merges the splits
// and lifts with W_UV.  With one split the same CTA does both.
// Rows are ordered head-major, so that a CTA reads the W_UK of few heads.
// Bound: fp32 multiply-adds and shared-memory reads for long contexts, latency
// for the toy model (4 heads, 4 nodes, 64 keys: 11.3 us, of which the launch
// and the chain query - absorb - scores - softmax - lift is all).
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "tree.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;             // query rows per CTA, 16 threads each
constexpr int kMaxLat = 512;          // kv_lora

struct Params {
  DecodeArgs a;
  int splits;
  uint64_t turn[kMaxRopePairs];  // rope_turns(rope_base^(-2j/qk_rope)): angles without fp64
  float* part;  // [B][splits][S*H][kv_lora + 2]: latents, maximum, sum (splits > 1)
};

__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Elements c0, c0 + 8, .. below n of one row
// into shared memory.  fp32 rows go there by asynchronous 4-byte copies, so
// that a whole tile is in flight at once; bf16 rows are converted on the way.
__device__ __forceinline__ void copy_row(float* dst, const float* src, int c0, int n) {
  for (int c = c0; c < n; c += 8) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst + c));
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src + c) : "memory");
  }
}
__device__ __forceinline__ void copy_row(float* dst, const __nv_bfloat16* src, int c0, int n) {
  for (int c = c0; c < n; c += 8) dst[c] = to_f32(src[c]);
}
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void put(void* out, bool bf16, size_t i, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(out)[i] = v;
}

// out[row] = W_UV[head] clat[row] for rows0 .. rows0 + nrows - 1 of sequence b:
// a warp takes one output column at a time, its lanes the latents; `fill[r]`
// replaces a row by a constant (zero or NaN) where it is not one.
// kAcc: latents per thread of 16, kv_lora <= 16 kAcc (a toy model's 32 in
// loops of 2 instead of 32).
template <typename Tin, int kAcc>
__device__ __forceinline__ void lift(const DecodeArgs& a, int b, int row0, int nrows, const float* clat, int pitch,
                                     const float* fill) {
  const Geometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (kAcc <= 8) {  // short latents: a thread per output
    for (int e = threadIdx.x; e < nrows * g.Dv; e += blockDim.x) {
      const int r = e / g.Dv, v = e % g.Dv, h = (row0 + r) / a.S, s = (row0 + r) % a.S;
      const Tin* W = static_cast<const Tin*>(a.kv_b) + ((size_t)h * (g.Dn + g.Dv) + g.Dn + v) * g.Dl;
      float acc = 0.f;
#pragma unroll 16
      for (int l = 0; l < g.Dl; ++l) acc = fmaf(to_f32(W[l]), clat[r * pitch + l], acc);
      const float f = fill[r];
      put(a.out, a.out_bf16 != 0, (((size_t)b * a.S + s) * g.H + h) * g.Dv + v, f == 1.f ? acc : f);
    }
    return;
  }
  for (int r0 = 0; r0 < nrows;) {
    const int h = (row0 + r0) / a.S;
    int r1 = r0 + 1;
    while (r1 < nrows && (row0 + r1) / a.S == h) ++r1;
    const Tin* W = static_cast<const Tin*>(a.kv_b) + ((size_t)h * (g.Dn + g.Dv) + g.Dn) * g.Dl;
    for (int v = warp; v < g.Dv; v += nw) {
      float w[kAcc / 2];
#pragma unroll
      for (int j = 0; j < kAcc / 2; ++j) w[j] = lane + 32 * j < g.Dl ? to_f32(W[(size_t)v * g.Dl + lane + 32 * j]) : 0.f;
      for (int r = r0; r < r1; ++r) {
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < kAcc / 2; ++j)
          if (lane + 32 * j < g.Dl) acc = fmaf(w[j], clat[r * pitch + lane + 32 * j], acc);
        acc = warp_sum(acc);
        if (lane == 0) {
          const int s = (row0 + r) % a.S;
          const float f = fill[r];
          put(a.out, a.out_bf16 != 0, (((size_t)b * a.S + s) * g.H + h) * g.Dv + v, f == 1.f ? acc : f);
        }
      }
    }
    r0 = r1;
  }
}

// Keys per tile: short rows take more, for fewer round trips.
__host__ __device__ constexpr int keys_of(int acc) { return acc <= 2 ? 128 : acc <= 8 ? 64 : 32; }

template <typename Tin, int kAcc>
__global__ void __launch_bounds__(kThreads) tree_attend_kernel(const __grid_constant__ Params p) {
  const DecodeArgs& a = p.a;
  const Geometry& g = a.g;
  extern __shared__ float sm[];
  constexpr int kKeys = keys_of(kAcc), kPer = kKeys / 16;  // keys per tile, scores per thread
  const int D = g.Dl + g.Dr, kp = D | 1;           // odd pitch: the keys of a row of threads lie in different banks
  float* q = sm;                                    // [kRows][kp] absorbed latent query, rotated query
  float* kt = q + kRows * kp;                       // [kKeys][kp] key rows (first: the unrotated queries)
  float* ps = kt + kKeys * kp;                      // [kRows][kKeys]
  __shared__ unsigned long long mask_sh[kRows];
  __shared__ int depth_sh[kRows];
  __shared__ float fill[kRows];                     // 1, or the constant of an absent or bad row
  __shared__ int bad_page_sh;
  const int tid = threadIdx.x, rr = tid >> 4, tl = tid & 15;
  const int SH = a.S * g.H, row0 = blockIdx.x * kRows, split = blockIdx.y, b = blockIdx.z;
  const int nrows = min(kRows, SH - row0);
  const int Tb = a.T[b], base = Tb - a.S;
  const bool bad_len = Tb < a.S || Tb > a.T_cap;
  if (tid < kRows) {
    TreeNode node{0ull, 0, kNodeAbsent};
    if (tid < nrows) node = tree_node(a.parent + (size_t)b * a.S, (row0 + tid) % a.S);
    mask_sh[tid] = node.mask;
    depth_sh[tid] = node.depth;
    fill[tid] = bad_len || node.state == kNodeBad ? qnan() : node.state == kNodeAbsent ? 0.f : 1.f;
    if (tid < nrows && split == 0) {
      if (bad_len) raise_flag(a.flags, MLA_DEV_BAD_LENGTH);
      else if (node.state == kNodeBad) raise_flag(a.flags, MLA_DEV_BAD_INDEX);
    }
  }
  if (tid == 0) bad_page_sh = 0;
  // this split's keys
  const int n = bad_len ? 0 : Tb;
  const int k_lo = (int)((long long)n * split / p.splits), k_hi = (int)((long long)n * (split + 1) / p.splits);
  const Tin* qg = static_cast<const Tin*>(a.q);
  const int Dq = g.Dn + g.Dr;
  if (k_lo < k_hi) {
    // unrotated queries of the rows, W_UK folded into them a chunk of qk_nope at a time
    const int chunk = min(g.Dn, kKeys * kp / kRows);
    float qa[kAcc];
#pragma unroll
    for (int j = 0; j < kAcc; ++j) qa[j] = 0.f;
    const int my = row0 + min(rr, nrows - 1), h = my / a.S, s = my % a.S;
    const Tin* qrow = qg + (((size_t)b * a.S + s) * g.H + h) * Dq;
    const Tin* W = static_cast<const Tin*>(a.kv_b) + (size_t)h * (g.Dn + g.Dv) * g.Dl;
    for (int i0 = 0; i0 < g.Dn; i0 += chunk) {
      const int ni = min(chunk, g.Dn - i0);
      __syncthreads();
      for (int i = tl; i < ni; i += 16) kt[rr * chunk + i] = to_f32(qrow[i0 + i]);
      __syncthreads();
#pragma unroll 8
      for (int i = 0; i < ni; ++i) {
        const float x = kt[rr * chunk + i];
#pragma unroll
        for (int j = 0; j < kAcc; ++j)
          if (tl + 16 * j < g.Dl) qa[j] = fmaf(x, to_f32(W[(size_t)(i0 + i) * g.Dl + tl + 16 * j]), qa[j]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kAcc; ++j)
      if (tl + 16 * j < g.Dl) q[rr * kp + tl + 16 * j] = qa[j] * g.scale;
    for (int j = tl; j < g.Dr / 2; j += 16) {
      float c, sn;
      rope_cs_turns(base + depth_sh[rr], p.turn[j], &c, &sn);
      const float x0 = to_f32(qrow[g.Dn + 2 * j]), x1 = to_f32(qrow[g.Dn + 2 * j + 1]);
      q[rr * kp + g.Dl + j] = (x0 * c - x1 * sn) * g.scale;
      q[rr * kp + g.Dl + g.Dr / 2 + j] = (x1 * c + x0 * sn) * g.scale;
    }
  }
  __syncthreads();
  const unsigned long long mask = mask_sh[rr];
  float acc[kAcc];
#pragma unroll
  for (int j = 0; j < kAcc; ++j) acc[j] = 0.f;
  float m = kMaxFloor, l = 0.f;
  const Tin* Lc = static_cast<const Tin*>(a.Lc);
  const Tin* Rc = static_cast<const Tin*>(a.Rc);
  for (int k0 = k_lo; k0 < k_hi; k0 += kKeys) {
    const int nk = min(kKeys, k_hi - k0);
    // key rows: 8 threads per row
    for (int k = tid >> 3; k < nk; k += kThreads / 8) {
      bool bad = false;
      const long long row = cache_row(a.pages, b, a.T_cap, k0 + k, &bad);  // (row 0 where the page is bad)
      if (bad) bad_page_sh = 1;
      copy_row(kt + k * kp, Lc + (size_t)row * g.Dl, tid & 7, g.Dl);
      copy_row(kt + k * kp + g.Dl, Rc + (size_t)row * g.Dr, tid & 7, g.Dr);
    }
    copy_wait();
    __syncthreads();
    float sc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) sc[i] = 0.f;
    const float* qr = q + rr * kp;
    const float* ka = kt + tl * kp;
#pragma unroll 4
    for (int d = 0; d < D; ++d) {
      const float x = qr[d];
#pragma unroll
      for (int i = 0; i < kPer; ++i) sc[i] = fmaf(x, ka[16 * i * kp + d], sc[i]);
    }
    float top = -INFINITY;
    bool seen[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int k = tl + 16 * i, t = k0 + k;
      seen[i] = mask && k < nk && (t < base || ((mask >> (t - base)) & 1ull));
      sc[i] = seen[i] ? sc[i] : -INFINITY;
      top = fmaxf(top, sc[i]);
    }
    const float mn = fmaxf(m, half_max(top));
    const float al = expf(m - mn);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // a visible key with a score of -inf holds values that are not finite: NaN, not weight 0
      const float x = !seen[i] ? 0.f : sc[i] > -INFINITY ? expf(sc[i] - mn) : qnan();
      ps[rr * kKeys + tl + 16 * i] = x;
      sum += x;
    }
    l = l * al + half_sum(sum);
    m = mn;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kAcc; ++j) acc[j] *= al;
#pragma unroll 4
    for (int k = 0; k < nk; ++k) {
      const float x = ps[rr * kKeys + k];
#pragma unroll
      for (int j = 0; j < kAcc; ++j)
        if (tl + 16 * j < g.Dl) {
          const float y = fmaf(x, kt[k * kp + tl + 16 * j], acc[j]);
          acc[j] = x != 0.f ? y : acc[j];  // (a hidden row may hold anything)
        }
    }
    __syncthreads();
  }
  if (bad_page_sh && tid == 0) raise_flag(a.flags, MLA_DEV_BAD_INDEX);
  const float poison = bad_page_sh ? qnan() : 0.f;
  if (p.splits > 1) {
    grid_dep_launch();
    if (rr < nrows) {
      float* dst = p.part + (((size_t)b * p.splits + split) * SH + row0 + rr) * (g.Dl + 2);
#pragma unroll
      for (int j = 0; j < kAcc; ++j)
        if (tl + 16 * j < g.Dl) dst[tl + 16 * j] = acc[j];
      if (tl == 0) {
        dst[g.Dl] = m;
        dst[g.Dl + 1] = l + poison;
      }
    }
    return;
  }
  const float inv = 1.f / l + poison;
#pragma unroll
  for (int j = 0; j < kAcc; ++j)
    if (tl + 16 * j < g.Dl) kt[rr * kp + tl + 16 * j] = acc[j] * inv;
  __syncthreads();
  lift<Tin, kAcc>(a, b, row0, nrows, kt, kp, fill);
}

// Merge of the splits of up to 4 rows, then the lift.
constexpr int kMergeRows = 4;

template <typename Tin, int kAcc>
__global__ void __launch_bounds__(128) tree_merge_kernel(const __grid_constant__ Params p) {
  const DecodeArgs& a = p.a;
  const Geometry& g = a.g;
  __shared__ float clat[kMergeRows * kMaxLat];
  __shared__ float fill[kMergeRows];
  const int SH = a.S * g.H, row0 = blockIdx.x * kMergeRows, b = blockIdx.y;
  const int nrows = min(kMergeRows, SH - row0), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Tb = a.T[b];
  grid_dep_wait();
  if (warp < nrows) {
    const TreeNode node = tree_node(a.parent + (size_t)b * a.S, (row0 + warp) % a.S);
    const bool bad = Tb < a.S || Tb > a.T_cap || node.state == kNodeBad;
    if (lane == 0) fill[warp] = bad ? qnan() : node.state == kNodeAbsent ? 0.f : 1.f;
    const size_t step = (size_t)SH * (g.Dl + 2);
    const float* src = p.part + ((size_t)b * p.splits * SH + row0 + warp) * (g.Dl + 2);
    float M = kMaxFloor;
    for (int i = lane; i < p.splits; i += 32) M = fmaxf(M, src[i * step + g.Dl]);
    M = warp_max(M);
    float L = 0.f, acc[kAcc / 2];
#pragma unroll
    for (int j = 0; j < kAcc / 2; ++j) acc[j] = 0.f;
#pragma unroll 4
    for (int i = 0; i < p.splits; ++i) {
      const float w = expf(src[i * step + g.Dl] - M);
      L = fmaf(w, src[i * step + g.Dl + 1], L);
#pragma unroll
      for (int j = 0; j < kAcc / 2; ++j)
        if (lane + 32 * j < g.Dl) acc[j] = fmaf(w, src[i * step + lane + 32 * j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < kAcc / 2; ++j)
      if (lane + 32 * j < g.Dl) clat[warp * kMaxLat + lane + 32 * j] = acc[j] / L;
  }
  __syncthreads();
  lift<Tin, kAcc>(a, b, row0, nrows, clat, kMaxLat, fill);
}

int acc_of(const Geometry& g) { return g.Dl <= 32 ? 2 : g.Dl <= 128 ? 8 : 32; }

size_t smem_bytes(const Geometry& g) {
  const size_t kp = (g.Dl + g.Dr) | 1, keys = keys_of(acc_of(g));
  return ((kRows + keys) * kp + kRows * keys) * sizeof(float);
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n > 0 ? n : 148;
}

// Splits of the keys: enough CTAs for one per SM, at least a key tile each.
int split_count(const Geometry& g, int B, int S, int T_cap) {
  const long long groups = (long long)B * ((S * g.H + kRows - 1) / kRows);
  const int keys = keys_of(acc_of(g));
  const long long most = (T_cap + keys - 1) / keys;
  const long long want = (sm_count() + groups - 1) / groups;
  const long long s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s > 512 ? 512 : s);
}

template <typename Tin, int kAcc>
cudaError_t launch(const Params& p, cudaStream_t st) {
  const DecodeArgs& a = p.a;
  const int smem = (int)smem_bytes(a.g);
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(tree_attend_kernel<Tin, kAcc>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  const int SH = a.S * a.g.H;
  kernel_mark(st, "tree_attend");
  tree_attend_kernel<Tin, kAcc><<<dim3((SH + kRows - 1) / kRows, p.splits, a.B), kThreads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  kernel_mark(st, "tree_merge");
  return launch_pdl(tree_merge_kernel<Tin, kAcc>, dim3((SH + kMergeRows - 1) / kMergeRows, a.B), dim3(128), 0, st, p);
}

}  // namespace

bool tree_simt_ok(const Geometry& g, int B) {
  return g.Dl <= kMaxLat && g.Dr <= 2 * kMaxRopePairs && B <= 65535 && smem_bytes(g) <= 220 * 1024;
}

size_t tree_simt_workspace_bytes(const Geometry& g, int B, int S, int T_cap) {
  const int splits = split_count(g, B, S, T_cap);
  return splits > 1 ? (size_t)B * splits * S * g.H * (g.Dl + 2) * sizeof(float) : 0;
}

cudaError_t launch_tree_simt(const DecodeArgs& a, int dtype, void* ws, cudaStream_t st) {
  Params p{a, split_count(a.g, a.B, a.S, a.T_cap), {}, static_cast<float*>(ws)};
  for (int j = 0; j < a.g.Dr / 2; ++j) p.turn[j] = rope_turns(std::pow(a.g.rope_base, -2.0 * j / a.g.Dr));
  const bool f = dtype == MLA_F32;
  if (acc_of(a.g) == 2) return f ? launch<float, 2>(p, st) : launch<__nv_bfloat16, 2>(p, st);
  if (acc_of(a.g) == 8) return f ? launch<float, 8>(p, st) : launch<__nv_bfloat16, 8>(p, st);
  return f ? launch<float, 32>(p, st) : launch<__nv_bfloat16, 32>(p, st);
}

}  // namespace mla
