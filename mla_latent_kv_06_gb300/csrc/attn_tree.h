// attn_tree.h -- prefix-and-tree attention over CTA pairs (see attn_tree.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace mla {

constexpr int kPairTile = 256;   // keys per tile
constexpr int kPairStage = 128;  // rows of one sequence in the staging buffer (80 are used)

// Length of the prefix part that is read from the cache in whole 16-key
// steps; the rest of the sequence (up to 15 prefix rows and the tree's) is the
// tail tile, staged.  t0: where the sequence's own tiles start behind a shared
// prefix (a multiple of kPairTile, at most T - S), else 0.
__host__ __device__ __forceinline__ int pair_base16(int T, int S) { return (T - S) & ~15; }
__host__ __device__ __forceinline__ int pair_tiles(int T, int S, int t0 = 0) {
  return (pair_base16(T, S) - t0 + kPairTile - 1) / kPairTile + 1;
}

struct PairParams {
  CUtensorMap mQ;   // qcat [R*64, 576], box 64 x 64
  CUtensorMap mQl;  // remainders of the rotated queries [R*64, 64], box 64 x 64
  CUtensorMap mK;   // latent rows, box 128 x 64
  CUtensorMap mKr;  // rotary key rows, box 128 x 64
  CUtensorMap mV;   // latents as (column in atom, row, 64-column atom), box 64 x 64 x 2
  CUtensorMap mT;   // staging [B*128, 576], box 128 x 64
  CUtensorMap mTv;  // staged latents likewise
  const int32_t* T;
  const int32_t* parent;
  const int32_t* tile_start;  // [B + 1] prefix of pair_tiles, then the first sequence of a good length (-1: none)
  int B, S, T_cap, G, NP;     // G chunks of the tile list, NP = ceil(S / 2) node pairs
  int shared, tiles, t0;      // shared prefix: pairs of query rows (0 without tiles), whole tiles, tokens in them
  float c;                    // softmax scale * log2(e)
  float* o_part;              // [(g + b) * S + s][64][512]
  float* ml_part;             // [(g + b) * S + s][64][2]
  unsigned int* flags;
  long long wait_ns;
  PageTable pages;
};

// Chunks of the tile list, at most kPairChunks (the few-row combine lists a row's splits).
constexpr int kPairChunks = 256;
int pair_chunks(int B, int S, int T_cap, int sms);

cudaError_t launch_attn_pair(const PairParams& p, cudaStream_t st);

// The pass of a batch that shares a prefix.  Its list holds items: first, for every pair
// of the batch's query rows, the prefix's tiles, then, for every
// sequence and pair of its nodes, the sequence's own tiles.  The prefix is read through the first
// sequence of a good length: what the table holds for one of a bad length, which is skipped,
// may name any page or none.  An item is kItemCost units
// for its query load, pipeline fill and partial, then one per tile; the clusters split the
// units evenly.  Chunk g's partials of item i are slots 2 (g + i) and 2 (g + i) + 1.
// kItemCost 1, 2 and 4, attention in us: 32 x 6 nodes on 32k shared tokens and none, 575,
// 543, 540; and up to 1k of their own, 554, 563, 588; 64 rows on 16k and up to 2k, 131,
// 126, 135.  (Weighing own tiles 4:3 against the prefix's: 559 and 133 for the last two.)
constexpr int kItemCost = 2;
struct SharedItems {
  int B, NP, shared, tiles;
  const int32_t* ts;
  __host__ __device__ __forceinline__ int count() const { return shared + B * NP; }
  __device__ __forceinline__ long long prefix_units() const { return (long long)shared * (kItemCost + tiles); }
  // units of one item of sequence b, and where the sequence's items begin
  __device__ __forceinline__ int each(int b) const { return kItemCost + ts[b + 1] - ts[b]; }
  __device__ __forceinline__ long long own(int b) const {
    return prefix_units() + (long long)NP * (ts[b] + (long long)kItemCost * b);
  }
  __device__ __forceinline__ long long total() const { return own(B); }
  struct Item {
    long long at;  // unit of the first tile
    int tiles;
    // the tiles of a chunk of units [c0, c1): from lo up to hi
    __device__ __forceinline__ void range(long long c0, long long c1, int* lo, int* hi) const {
      const long long l = c0 - at, h = c1 - at;
      *lo = (int)(l < 0 ? 0 : l < tiles ? l : tiles);
      *hi = (int)(h < 0 ? 0 : h < tiles ? h : tiles);
    }
  };
  __device__ __forceinline__ Item item(int i) const {
    if (i < shared) return Item{(long long)i * (kItemCost + tiles) + kItemCost, tiles};
    const int b = (i - shared) / NP, k = (i - shared) - b * NP;
    return Item{own(b) + (long long)k * each(b) + kItemCost, ts[b + 1] - ts[b]};
  }
};

// a / d for a >= 0, d > 0: in 32 bits wherever a fits.
__device__ __forceinline__ long long over_chunks(long long a, int d) {
  return ((unsigned long long)a >> 32) == 0 ? (long long)((unsigned)a / (unsigned)d) : a / d;
}

// The partials of one query row: at most kSharedSplits chunks of its two items.
constexpr int kSharedChunks = 128, kSharedSplits = 2 * kSharedChunks;
struct SharedSplits {
  SharedItems::Item item[2];
  int at[2], from[2], odd[2], n0, n;
  // row r of the batch, node s of sequence b, whose length is good
  __device__ __forceinline__ void start(const SharedItems& it, long long N, int G, int r, int b, int s) {
    at[0] = r >> 1;
    at[1] = it.shared + b * it.NP + (s >> 1);
    odd[0] = r & 1;
    odd[1] = s & 1;
    n = n0 = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      n0 = n;
      if (k == 0 && !it.shared) continue;
      item[k] = it.item(at[k]);
      from[k] = chunk(item[k].at, N, G);
      n += chunk(item[k].at + item[k].tiles - 1, N, G) - from[k] + 1;
    }
  }
  // slot of the i-th split, -1: none (a chunk that holds no tile of the item)
  __device__ __forceinline__ long long slot(int i, long long N, int G) const {
    if (i >= n) return -1;
    const bool own = i >= n0;
    const int g = own ? from[1] + i - n0 : from[0] + i;
    int lo, hi;
    (own ? item[1] : item[0]).range(over_chunks(N * g, G), over_chunks(N * (g + 1), G), &lo, &hi);
    return lo < hi ? (long long)(g + (own ? at[1] : at[0])) * 2 + (own ? odd[1] : odd[0]) : -1;
  }
  // the chunk that holds unit x: the largest g with N g / G <= x
  static __device__ __forceinline__ int chunk(long long x, long long N, int G) {
    int g = ((unsigned long long)(N * G) >> 32) == 0 ? (int)((unsigned)(x * G) / (unsigned)N) : (int)(x * G / N);
    if (g > G - 1) g = G - 1;
    while (g + 1 < G && over_chunks(N * (g + 1), G) <= x) ++g;
    return g;
  }
};
cudaError_t launch_attn_shared(const PairParams& p, cudaStream_t st);

}  // namespace mla
