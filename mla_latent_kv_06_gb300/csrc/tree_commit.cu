// tree_commit.cu -- moves the cache rows of the accepted tree nodes together.
//
// Row T - S + i of each cache receives row T - S + path[i] for i < n, after
// which the sequence has T - S + n cached tokens.  path is increasing, so
// path[i] >= i: a row is never written before the moves that read it have
// read it as long as each thread keeps the order of i within its own column
// of the rows.  Columns are independent, so the kernel needs no barrier: a
// thread owns one 16-byte column, loads it for eight rows at a time and then
// stores it (later sources lie at or above the next destination).
//
// All caches of a call (every layer's latent and rotary rows, say) go through
// one launch; the bound is the latency of three dependent reads (length and
// path, page, row), not the few KB per sequence: 2.1 us for 2 caches and one
// sequence, 4.8 us for 96 caches and 16 sequences (1.9 TB/s).
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kThreads = 64;
constexpr int kBatch = 8;

template <typename Vec>
__device__ __forceinline__ void move_rows(unsigned char* cache, int row_bytes, int n, int p_lo, int p_hi,
                                          const long long (&row)[2]) {
  const int cols = row_bytes / (int)sizeof(Vec);
  for (int col0 = 0; col0 < cols; col0 += kThreads) {
    const int col = col0 + threadIdx.x;
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      Vec v[kBatch];
      long long dst[kBatch];
      bool move[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k;
        // every lane takes part in the shuffles
        const int src = __shfl_sync(0xffffffffu, i < 32 ? p_lo : p_hi, i & 31);
        const long long src_row = __shfl_sync(0xffffffffu, src < 32 ? row[0] : row[1], src & 31);
        dst[k] = __shfl_sync(0xffffffffu, i < 32 ? row[0] : row[1], i & 31);
        move[k] = i < n && src != i && col < cols;
        if (move[k]) v[k] = *reinterpret_cast<const Vec*>(cache + src_row * row_bytes + (size_t)col * sizeof(Vec));
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (move[k]) *reinterpret_cast<Vec*>(cache + dst[k] * row_bytes + (size_t)col * sizeof(Vec)) = v[k];
    }
  }
}

// Few caches take a launch with a short parameter block (1.6 KB of it costs the host time).
template <int kCaches>
struct CommitLaunch {
  CommitArgs a;
  void* cache[kCaches];
  int row_bytes[kCaches];
};

template <int kCaches>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ CommitLaunch<kCaches> c) {
  const CommitArgs& a = c.a;
  const int cache = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31;
  const int S = a.S, Tb = __ldg(a.T + b), n = __ldg(a.n_acc + b);
  // lane holds path[lane] and path[32 + lane], and the pool rows of tree rows lane and 32 + lane
  const int32_t* path = a.path + (size_t)b * S;
  const int p_lo = lane < S ? __ldg(path + lane) : 0, p_hi = 32 + lane < S ? __ldg(path + 32 + lane) : 0;
  const bool bad_len = Tb < S || Tb > a.T_cap;
  const int base = Tb - S;
  bool bad_page = false;
  long long row[2] = {0, 0};
  if (!bad_len) {
    if (lane < S) row[0] = cache_row(a.pages, b, a.T_cap, base + lane, &bad_page);
    if (32 + lane < S) row[1] = cache_row(a.pages, b, a.T_cap, base + 32 + lane, &bad_page);
  }
  // n in [0, S] and path[0..n) increasing within [0, S)
  const int prev_lo = __shfl_up_sync(0xffffffffu, p_lo, 1), top_lo = __shfl_sync(0xffffffffu, p_lo, 31);
  const int prev_hi = __shfl_up_sync(0xffffffffu, p_hi, 1);
  bool bad = n < 0 || n > S || bad_page;
  if (lane < n) bad = bad || p_lo >= S || p_lo <= (lane ? prev_lo : -1);
  if (32 + lane < n) bad = bad || p_hi >= S || p_hi <= (lane ? prev_hi : top_lo);
  bad = __any_sync(0xffffffffu, bad);
  if (cache == 0 && threadIdx.x == 0) {
    if (bad_len) raise_flag(a.flags, MLA_DEV_BAD_LENGTH);
    else if (bad) raise_flag(a.flags, MLA_DEV_BAD_INDEX);
    if (a.T_out) a.T_out[b] = bad_len ? Tb : bad ? base : base + n;
  }
  if (bad_len || bad) return;
  unsigned char* rows = static_cast<unsigned char*>(c.cache[cache]);
  const int rb = c.row_bytes[cache];
  const unsigned odd = (unsigned)(reinterpret_cast<uintptr_t>(rows) | (unsigned)rb);
  if ((odd & 15u) == 0) move_rows<uint4>(rows, rb, n, p_lo, p_hi, row);
  else if ((odd & 3u) == 0) move_rows<uint32_t>(rows, rb, n, p_lo, p_hi, row);
  else move_rows<unsigned char>(rows, rb, n, p_lo, p_hi, row);
}

template <int kCaches>
cudaError_t launch(const CommitArgs& a, void* const* cache, const int* row_bytes, cudaStream_t st) {
  CommitLaunch<kCaches> c;
  c.a = a;
  for (int i = 0; i < a.n; ++i) {
    c.cache[i] = cache[i];
    c.row_bytes[i] = row_bytes[i];
  }
  tree_commit_kernel<kCaches><<<dim3(a.n, a.B), kThreads, 0, st>>>(c);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_commit(const CommitArgs& a, void* const* cache, const int* row_bytes, cudaStream_t st) {
  return a.n <= 8 ? launch<8>(a, cache, row_bytes, st) : launch<kCommitCaches>(a, cache, row_bytes, st);
}

}  // namespace mla
