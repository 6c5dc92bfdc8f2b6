// tree_simt.cu -- CUDA-core tree attention (fp32, and bf16 outside the
// tensor-core geometry), kv_lora up to 512.
//
// The absorbed path of the page "MLA 注意力与 KV 缓存", §2.3, for the nodes of
// a drafted tree.  A CTA takes 16 query rows (node, head) of one sequence and
// one split of its keys, which pass through shared memory 32 at a time: 16
// threads per row form two scores each, reduce the maximum and the sum among
// themselves and accumulate kv_lora / 16 latents each.  A key row is thus read once per
// 16 query rows.  The keys are split until the grid fills the GPU (a toy model
// on one sequence has one group of rows); a second kernel merges the splits
// and lifts with W_UV.  With one split the same CTA does both.
// Rows are ordered head-major, so that a CTA reads the W_UK of few heads.
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "tree.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;             // query rows per CTA, 16 threads each
constexpr int kKeys = 32;             // keys per tile
constexpr int kMaxLat = 512;          // kv_lora; 32 accumulators per thread
constexpr int kAcc = kMaxLat / 16;

struct Params {
  DecodeArgs a;
  int splits;
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

__device__ __forceinline__ void put(void* out, bool bf16, size_t i, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(out)[i] = v;
}

// out[row] = W_UV[head] clat[row] for rows0 .. rows0 + nrows - 1 of sequence b:
// a warp takes one output column at a time, its lanes the latents; `fill[r]`
// replaces a row by a constant (zero or NaN) where it is not one.
template <typename Tin>
__device__ __forceinline__ void lift(const DecodeArgs& a, int b, int row0, int nrows, const float* clat, int pitch,
                                     const float* fill) {
  const Geometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int r0 = 0; r0 < nrows;) {
    const int h = (row0 + r0) / a.S;
    int r1 = r0 + 1;
    while (r1 < nrows && (row0 + r1) / a.S == h) ++r1;
    const Tin* W = static_cast<const Tin*>(a.kv_b) + ((size_t)h * (g.Dn + g.Dv) + g.Dn) * g.Dl;
    for (int v = warp; v < g.Dv; v += nw) {
      float w[kMaxLat / 32];
#pragma unroll
      for (int j = 0; j < kMaxLat / 32; ++j) w[j] = lane + 32 * j < g.Dl ? to_f32(W[(size_t)v * g.Dl + lane + 32 * j]) : 0.f;
      for (int r = r0; r < r1; ++r) {
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxLat / 32; ++j)
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

template <typename Tin>
__global__ void __launch_bounds__(kThreads) tree_attend_kernel(const __grid_constant__ Params p) {
  const DecodeArgs& a = p.a;
  const Geometry& g = a.g;
  extern __shared__ float sm[];
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
      rope_cos_sin(base + depth_sh[rr], j, g.Dr, g.rope_base, &c, &sn);
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
  float m = -1e30f, l = 0.f;
  const Tin* Lc = static_cast<const Tin*>(a.Lc);
  const Tin* Rc = static_cast<const Tin*>(a.Rc);
  for (int k0 = k_lo; k0 < k_hi; k0 += kKeys) {
    const int nk = min(kKeys, k_hi - k0);
    // key rows: 8 threads per row
    {
      const int k = tid >> 3, c0 = tid & 7;
      if (k < nk) {
        bool bad = false;
        const long long row = cache_row(a.pages, b, a.T_cap, k0 + k, &bad);
        if (bad) bad_page_sh = 1;
        const Tin* L = Lc + (size_t)row * g.Dl;
        const Tin* R = Rc + (size_t)row * g.Dr;
        for (int c = c0; c < g.Dl; c += 8) kt[k * kp + c] = bad ? 0.f : to_f32(L[c]);
        for (int c = c0; c < g.Dr; c += 8) kt[k * kp + g.Dl + c] = bad ? 0.f : to_f32(R[c]);
      }
    }
    __syncthreads();
    float s0 = 0.f, s1 = 0.f;
    const float* qr = q + rr * kp;
    const float* ka = kt + tl * kp;
    const float* kb = ka + 16 * kp;
    for (int d = 0; d < D; ++d) {
      const float x = qr[d];
      s0 = fmaf(x, ka[d], s0);
      s1 = fmaf(x, kb[d], s1);
    }
    const int t0 = k0 + tl, t1 = t0 + 16;
    const bool v0 = mask && tl < nk && (t0 < base || ((mask >> (t0 - base)) & 1ull));
    const bool v1 = mask && tl + 16 < nk && (t1 < base || ((mask >> (t1 - base)) & 1ull));
    s0 = v0 ? s0 : -INFINITY;
    s1 = v1 ? s1 : -INFINITY;
    const float mn = fmaxf(m, half_max(fmaxf(s0, s1)));
    const float al = expf(m - mn);
    const float p0 = v0 ? expf(s0 - mn) : 0.f, p1 = v1 ? expf(s1 - mn) : 0.f;
    l = l * al + half_sum(p0 + p1);
    m = mn;
    ps[rr * kKeys + tl] = p0;
    ps[rr * kKeys + tl + 16] = p1;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kAcc; ++j) acc[j] *= al;
    for (int k = 0; k < nk; ++k) {
      const float x = ps[rr * kKeys + k];
      if (x != 0.f) {  // (a hidden row may hold anything)
#pragma unroll
        for (int j = 0; j < kAcc; ++j)
          if (tl + 16 * j < g.Dl) acc[j] = fmaf(x, kt[k * kp + tl + 16 * j], acc[j]);
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
  lift<Tin>(a, b, row0, nrows, kt, kp, fill);
}

// Merge of the splits of up to 4 rows, then the lift.
constexpr int kMergeRows = 4;

template <typename Tin>
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
    float M = -1e30f;
    for (int i = lane; i < p.splits; i += 32) M = fmaxf(M, src[i * step + g.Dl]);
    M = warp_max(M);
    float L = 0.f, acc[kMaxLat / 32];
#pragma unroll
    for (int j = 0; j < kMaxLat / 32; ++j) acc[j] = 0.f;
    for (int i = 0; i < p.splits; ++i) {
      const float w = expf(src[i * step + g.Dl] - M);
      L = fmaf(w, src[i * step + g.Dl + 1], L);
#pragma unroll
      for (int j = 0; j < kMaxLat / 32; ++j)
        if (lane + 32 * j < g.Dl) acc[j] = fmaf(w, src[i * step + lane + 32 * j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < kMaxLat / 32; ++j)
      if (lane + 32 * j < g.Dl) clat[warp * kMaxLat + lane + 32 * j] = acc[j] / L;
  }
  __syncthreads();
  lift<Tin>(a, b, row0, nrows, clat, kMaxLat, fill);
}

size_t smem_bytes(const Geometry& g) {
  const size_t kp = (g.Dl + g.Dr) | 1;
  return ((kRows + kKeys) * kp + kRows * kKeys) * sizeof(float);
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n > 0 ? n : 148;
}

// Splits of the keys: enough CTAs for two per SM, at least two key tiles each.
int split_count(const Geometry& g, int B, int S, int T_cap) {
  const long long groups = (long long)B * ((S * g.H + kRows - 1) / kRows);
  const long long most = (T_cap + 2 * kKeys - 1) / (2 * kKeys);
  const long long want = (2LL * sm_count() + groups - 1) / groups;
  const long long s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s > 512 ? 512 : s);
}

template <typename Tin>
cudaError_t launch(const Params& p, cudaStream_t st) {
  const DecodeArgs& a = p.a;
  const int smem = (int)smem_bytes(a.g);
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(tree_attend_kernel<Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  const int SH = a.S * a.g.H;
  kernel_mark(st, "tree_attend");
  tree_attend_kernel<Tin><<<dim3((SH + kRows - 1) / kRows, p.splits, a.B), kThreads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  kernel_mark(st, "tree_merge");
  return launch_pdl(tree_merge_kernel<Tin>, dim3((SH + kMergeRows - 1) / kMergeRows, a.B), dim3(128), 0, st, p);
}

}  // namespace

bool tree_simt_ok(const Geometry& g, int B) {
  return g.Dl <= kMaxLat && B <= 65535 && smem_bytes(g) <= 220 * 1024;
}

size_t tree_simt_workspace_bytes(const Geometry& g, int B, int S, int T_cap) {
  const int splits = split_count(g, B, S, T_cap);
  return splits > 1 ? (size_t)B * splits * S * g.H * (g.Dl + 2) * sizeof(float) : 0;
}

cudaError_t launch_tree_simt(const DecodeArgs& a, int dtype, void* ws, cudaStream_t st) {
  Params p{a, split_count(a.g, a.B, a.S, a.T_cap), static_cast<float*>(ws)};
  return dtype == MLA_F32 ? launch<float>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace mla
