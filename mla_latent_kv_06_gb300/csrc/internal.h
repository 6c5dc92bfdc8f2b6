// internal.h -- launchers shared between the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

struct Geometry {
  int H, Dn, Dr, Dl, Dv;  // heads, qk_nope, qk_rope, kv_lora, v_head
  float scale;            // resolved softmax scale
  double rope_base;       // resolved RoPE base
};

// Paged cache layout.  Token t of sequence b sits at row
// table[b * max_pages + t / page_size] * page_size + t % page_size of the page
// pool; table == nullptr means the contiguous layout (row b * T_cap + t).
struct PageTable {
  const int32_t* table;
  int max_pages, page_size, num_pages;
};

// Pool row of token t of sequence b.  A page index outside [0, num_pages)
// sets *bad and yields row 0, so that no access leaves the pool.
__host__ __device__ __forceinline__ long long cache_row(const PageTable& pt, int b, int T_cap, int t, bool* bad) {
  if (!pt.table) return (long long)b * T_cap + t;
  const int pg = pt.table[(size_t)b * pt.max_pages + t / pt.page_size];
  if (pg < 0 || pg >= pt.num_pages) {
    *bad = true;
    return 0;
  }
  return (long long)pg * pt.page_size + t % pt.page_size;
}

// Arguments common to the decode kernels (dense and sparse).
struct DecodeArgs {
  Geometry g;
  int B, S, T_cap;
  const void* q;
  const void* Lc;
  const void* Rc;
  const int32_t* T;
  const void* kv_b;
  void* out;            // float, or bf16 where out_bf16
  const int32_t* sel;   // sparse only: [B,S,topk]
  const int32_t* nsel;  // sparse only: [B,S]
  int topk;
  unsigned int* flags;
  long long wait_limit_ns;
  PageTable pages;  // table == nullptr: contiguous [B, T_cap] caches
  int lat_fp8;      // Lc holds E4M3 codes (the FP8 cache); latent = lat_scale * code
  float lat_scale;
  // Sparse decode inside a multi-layer call: staging buffer 0 or 1, and
  // whether the gather may launch as a programmatic dependent of the
  // previous kernel (true only when that buffer was last read two layers back)
  int stage_parity;
  int gather_pdl;
  // Tree attention (dense only): parents of the S drafted nodes [B, S], else null
  const int32_t* parent;
  int out_bf16;
  // Shared prefix: tokens below `lead` lie in the same rows for all sequences, and
  // every length is at least S + lead
  int lead;
  int shared;  // a shared-prefix call (lead may be 0), whose arithmetic is the tree attention's
};

cudaError_t launch_decode_simt(const DecodeArgs& a, int dtype, bool sparse, cudaStream_t st);

struct PrefillArgs {
  Geometry g;
  int B, S, pos_base;
  const void* q;
  const void* Lc;
  const void* Rc;
  const void* kv_b;
  void* kv;  // rebuilt [B, Tk, H, Dn+Dv], input dtype
  float* out;
};

cudaError_t launch_prefill_simt(const PrefillArgs& a, int dtype, cudaStream_t st);

struct IndexArgs {
  int B, S, n_ih, hd, T_cap;
  const float* q_idx;
  const float* w;
  const float* Ic;
  const int32_t* T;
  float* scores;
  unsigned int* flags;
  long long wait_ns;  // bound of every wait inside a kernel
  // Optional [B*S, parts, 2048] histograms of the top 11 bits of the ordered
  // score keys of the candidates t <= pos, one per indexer CTA of a row (the
  // first radix pass of the top-k); only the tensor-core indexer writes them.
  uint32_t* hpart;
};

cudaError_t launch_index_scores(const IndexArgs& a, cudaStream_t st);
// Tensor-core indexer (32 index heads x 128, fp32 through three tf32 products);
// returns cudaErrorNotSupported when the request does not fit it.
cudaError_t launch_index_scores_tc(const IndexArgs& a, cudaStream_t st);
// CTAs per (b, s) row of the tensor-core indexer, 0 when it does not take the shape.
int index_tc_parts(int B, int S, int n_ih, int hd, int T_cap);

struct TopkArgs {
  int B, S, T_cap, topk;
  const float* scores;
  const int32_t* T;
  int32_t* sel;
  int32_t* nsel;
  unsigned int* flags;
  const uint32_t* hpart;  // optional first-pass histograms from the indexer (IndexArgs::hpart)
  int hparts;
};

cudaError_t launch_topk_select(const TopkArgs& a, cudaStream_t st);

// Output projection y[r, n] = sum_k W_O[n, k] x[r, k] (W_O [hidden, in_dim] in dtype, x and y fp32).
struct OprojArgs {
  int R, in_dim, hidden, dtype;
  const void* w_o;
  const float* x;
  float* y;
  void* x_bf16;  // [R, in_dim] scratch for the tensor-core path (R > 8, bf16 weights), else unused
};
// Rows per GEMV launch; more rows take the tensor-core GEMM (bf16 weights).
constexpr int kOprojGemvRows = 8;
size_t oproj_workspace_bytes(int R, int in_dim, int hidden, int dtype);
cudaError_t launch_oproj(const OprojArgs& a, bool pdl, unsigned int* flags, long long wait_ns, cudaStream_t st);

// RoPE frequencies base^(-2j/d) travel in the launch parameters: rope widths up to 2 * kMaxRopePairs.
constexpr int kMaxRopePairs = 128;
// The append kernels hold a row in registers: at most kMaxAppendPer values per thread of 128.
constexpr int kMaxAppendPer = 32;
constexpr int kMaxAppendWidth = 128 * kMaxAppendPer;

struct AppendArgs {
  int B, S, T_cap, kv_lora, qk_rope;
  const void* comp;     // [B, S, kv_lora + qk_rope]
  const void* kv_a_ln;  // [kv_lora]
  float eps;
  const int32_t* T;
  void* Lc;  // [B, T_cap, kv_lora] or the page pool
  void* Rc;  // [B, T_cap, qk_rope] or the page pool
  unsigned int* flags;
  PageTable pages;
  const int32_t* parent;  // [B, S] parents of a drafted tree, else null
  uint64_t turn[kMaxRopePairs];  // rope_turns(rope_base^(-2j/qk_rope))
  int lat_fp8;          // Lc receives E4M3 codes of the normalised row * lat_inv_scale
  float lat_inv_scale;
};
cudaError_t launch_cache_append(const AppendArgs& a, int dtype, cudaStream_t st);

struct KeyAppendArgs {
  int B, S, T_cap, hd, rope_dim;
  const float* k;     // [B, S, hd]
  const float* ln_w;  // [hd]
  const float* ln_b;  // [hd] or null
  float eps;
  const int32_t* T;
  float* Ic;  // [B, T_cap, hd]
  unsigned int* flags;
  uint64_t turn[kMaxRopePairs];  // rope_turns(rope_base^(-2j/rope_dim))
};
cudaError_t launch_index_key_append(const KeyAppendArgs& a, cudaStream_t st);

// CUDA-core tree attention, chains where a.parent is null (kv_lora up to 512; other shapes take launch_decode_simt).
bool tree_simt_ok(const Geometry& g, int B);
size_t tree_simt_workspace_bytes(const Geometry& g, int B, int S, int T_cap);
cudaError_t launch_tree_simt(const DecodeArgs& a, int dtype, void* ws, cudaStream_t st);

// Largest drafted tree: its ancestor masks are 64-bit words.
constexpr int kMaxTree = 64;

// Largest capacity of a sequence in tree and shared-prefix attention: the kernels' key indices
// step past a length by up to a tile (256), and stay within int.
constexpr int kMaxTreeCap = 0x7fffffff - 1023;

// Query rows B * S of a shared-prefix call.
constexpr int kMaxSharedRows = 8192;
// Its sequences' own capacities together: their tiles are counted in 32 bits.
constexpr long long kMaxSharedOwn = 1ll << 38;

struct VerifyArgs {
  int B, S, V;
  const float* p;  // row r of sequence b at p + b * p_batch + r * p_row, r = 0 .. S
  const float* q;  // likewise, or null: point drafts
  long long p_row, p_batch, q_row, q_batch;
  const int32_t* tokens;  // [B, S]
  const int32_t* parent;  // [B, S]
  const float* u;         // [B, S + 1]
  int32_t* path;          // [B, S]
  int32_t* n_acc;         // [B]
  int32_t* token;         // [B]
  unsigned int* flags;
};
cudaError_t launch_tree_verify(const VerifyArgs& a, cudaStream_t st);

// Largest vocabulary of mla_sample: a row lies in the shared memory of 8 CTAs.
constexpr int kMaxSampleVocab = 8 * 40960;

struct SampleArgs {
  int B, N, V, dtype;
  const void* logits;  // row n of sequence b at element b * l_batch + n * l_row
  long long l_row, l_batch;
  const float* temperature;  // settings of row b * N + n: entry b * N + n where per_row, else b; null: off
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int per_row;
  const float* u;  // [B, N], with token
  int32_t* token;  // [B, N], or null
  float* probs;    // as logits, or null
  long long p_row, p_batch;
  unsigned int* flags;
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st);

// Caches of one commit launch: pointers travel in the launch parameters.
constexpr int kCommitCaches = 128;

struct CommitArgs {
  int n, B, S, T_cap;
  const int32_t* T;
  const int32_t* path;   // [B, S]
  const int32_t* n_acc;  // [B]
  int32_t* T_out;        // [B], or null: a later launch of the same call
  unsigned int* flags;
  PageTable pages;
};
// The n caches and their row sizes (host arrays, n <= kCommitCaches).
cudaError_t launch_tree_commit(const CommitArgs& a, void* const* cache, const int* row_bytes, cudaStream_t st);

// Sets the thread-local message returned by mla_last_error().
void set_last_error(const char* msg);

// Device address of the library's status word on the current device (null
// when it cannot be resolved), and the bound of every wait inside a kernel
// (mla_set_wait_limit_ns).
unsigned int* device_flags();
long long wait_limit_ns();

// Per-call launch bookkeeping behind mla_set_kernel_events / mla_last_launch_names:
// call_begin() at the start of each API call, kernel_mark() right before each
// kernel launch, call_end() after the last one.
void call_begin();
void kernel_mark(cudaStream_t st, const char* name);
void call_end(cudaStream_t st);

}  // namespace mla
