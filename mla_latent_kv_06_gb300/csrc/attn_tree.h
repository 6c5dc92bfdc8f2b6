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
// tail tile, staged.
__host__ __device__ __forceinline__ int pair_base16(int T, int S) { return (T - S) & ~15; }
__host__ __device__ __forceinline__ int pair_tiles(int T, int S) {
  return (pair_base16(T, S) + kPairTile - 1) / kPairTile + 1;
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
  const int32_t* tile_start;  // [B + 1] prefix of pair_tiles
  int B, S, T_cap, G, NP;     // G chunks of the tile list, NP = ceil(S / 2) node pairs
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

}  // namespace mla
