// attn_tree.cu -- tree attention for many query rows on CTA pairs.
//
// Scores qabs . Lc + q_rot . Rc, softmax and latent context sum p Lc of the
// page "MLA 注意力与 KV 缓存", §2.3, for the nodes of a drafted tree.
//
// A key row is 1152 bytes and one node's 64 heads do 64 * 1088 multiply-adds
// with it, so with several nodes the tensor pipe is the bound, and the work
// per SM is limited by TMEM: the fp32 latent context of 64 query rows takes
// 256 of its 512 columns.  One node per SM at M = 64 would run the pipe at half
// rate and a transposed product (keys as M, heads as N = 64) reads shared
// memory for every 64 columns.  So two SMs form a pair and run M = 128
// products of cta_group::2: CTA r holds the query rows, probabilities, scores
// and context of its own node (tree node 2i + r), and each supplies half of
// the B operand, which the pair's tensor cores share:
//   S[64 rows x 256 keys] = Q [K-major] . K^T    (K = 576 + 64; CTA r loads keys 128r ..)
//   O[64 rows x 512]     += P [K-major] . V      (two N = 256 blocks; CTA r loads
//                                                 latents 256n + 128r .. of all keys)
// All products have N = 256: measured 64.6 cycles each, the full rate, against
// 52.8 for N = 128 (62%).  Softmax, running maximum and rescale are local to a
// CTA: only barriers cross the pair.
//
// Operands stream through one ring of 16 KB stages in the order of use, K(0),
// K(1), V(0), K(2), V(1), ...: the score product of tile j + 1 runs while the
// softmax works on tile j.  TMEM: two S buffers of 128 columns, O of 256.  A
// row of S sits in two lanes (l: keys 0-127, 64 + l: keys 128-255), a row of O
// likewise (halves of each 256-column block).
//
// Masks cost the main loop nothing.  Prefix keys come from the cache in whole
// 16-key steps and are visible to every node.  The up to 15 prefix rows past
// the last step and the tree's rows form one tail tile, copied beforehand into
// a staging buffer (stage_tail): a row with a value that is not finite is staged as zero
// latents with a NaN rotary part, so that it turns the nodes that see it into
// NaN through their scores and the others, whose probability is zero, stay
// untouched although the pair shares the value operand.  A visible score of
// -inf (an infinite rotary key under a finite latent) has weight zero and would
// hide its row: the pass for the maximum takes the minimum along, and the row
// sum becomes NaN (32 x 6 nodes 0.3% longer, other cases within the noise).
//
// Rounding.  The absorbed query and the probabilities are rounded to bf16,
// because the products take both operands in one 16-bit type and the cache is
// bf16.  The rotated query is taken in two bf16 terms, 4 more products a tile:
// its 64 values carry half of the scores' error, and the output's goes from 1.50
// to 1.43 times that of its own rounding (emulated on 200 and 1000 keys) for 2%
// of the time of a long context (a second term of the 512 latents would be 32 products more, one of the
// probabilities 32).  The row sums add the rounded probabilities, so that both
// sides of the quotient use the same weights.  Scores, running maximum, sums and context are fp32.
//
// Measured: 8 trees of 64 nodes on 16k to 32k keys 1.03 ms, 1.70 PFLOP/s of the
// formula's (1.80 issued), the sustained rate of the tensor pipe under the
// power limit.  32 trees of 6 nodes on 1k to 32k keys 372 us, 1.22 PFLOP/s:
// with 3 pairs on a tile, 3.7 us a tile against 3.1 with 32 pairs, although
// DRAM runs at a quarter of its rate and L2 below a fifth of its sectors'
// (4 x 6 x 4096); fetching the tiles into L2 ahead of time changed nothing (315
// against 313 us on 32 x 6 x 16384).
#include "attn_tree.h"

#include <atomic>

#include "common.cuh"
#include "sm100.cuh"
#include "tree.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 320;  // warp 0: TMA, warp 1: MMA (leader CTA), warps 2-9: softmax
constexpr int kSoft = 256, kSoftWarps = 8;
constexpr int kRows = 64, kDl = 512, kDc = 576;
constexpr int kStages = 7;
constexpr int kFree = 4;  // barriers that free stages, two at a time (see issue)
constexpr uint32_t kStageBytes = 16384, kQAtom = 8192;
constexpr uint32_t kQBytes = 10 * kQAtom, kPBytes = 4 * 8192;
constexpr uint32_t kRingOff = kQBytes + kPBytes;
constexpr uint32_t kSmem = kRingOff + kStages * kStageBytes + 1024;
constexpr uint32_t kColS = 0, kColO = 256, kCols = 512;
constexpr float kTau = 8.f;  // lazy rescale threshold (log2 units)
constexpr long long kDrainNs = 1000000000LL;

struct Shared {
  uint64_t full[kStages];  // the leader's, for both CTAs' bytes
  uint64_t free2[kFree];   // stages 2m and 2m + 1 have been consumed: barrier m % kFree
  uint64_t q_full, q_empty, s_full[2], p_full, pv_done, mma_done;
  uint32_t tmem;
  int abort;
  int issued[2], q_issued[2];  // stages and query blocks each CTA has issued (leader's copy, at the end)
  float red[4][kRows];
  float m[kRows], alpha[kRows];
};

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared-cluster address of `p`'s counterpart in CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

// One arrival per warp on the leader's barrier.
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}

// A condition that is the same in every lane, as a vote: the compiler then
// knows the branch on it does not diverge.
__device__ __forceinline__ bool uni(bool c) { return __any_sync(0xffffffffu, c); }

// Tile loads into this CTA's shared memory, completing on a barrier of either
// CTA of the pair; issued by the lane with lead != 0 of a converged warp.
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                        uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 st;\n\tsetp.ne.b32 e, %2, 0;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(lead)
      : "memory");
}

// MMA and commit of the lane with lead != 0, called by the whole warp.  The
// code around them stays free of divergence, so that the compiler keeps the
// descriptors in uniform registers: the same loop run by one lane issues an
// MMA every 84 cycles or slower (more instructions between MMAs, more idle
// pipe), run by the warp every 64, the pipe's own rate.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// Arrive on both CTAs' `bar` once the MMAs issued so far have retired.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3), "r"(lead)
      : "memory");
}

// The pieces (sequence, tile range) of one chunk of the tile list.
struct Pieces {
  const int32_t* ts;
  int B, b, lo, hi;
  long long c0, c1;
  __device__ __forceinline__ void start(const PairParams& p, int g) {
    ts = p.tile_start;
    B = p.B;
    const long long N = ts[B];
    c0 = N * g / p.G;
    c1 = N * (g + 1) / p.G;
    int l = 0, h = B;  // first sequence whose tiles reach past c0
    while (l < h) {
      const int mid = (l + h) >> 1;
      if (ts[mid + 1] > c0) h = mid;
      else l = mid + 1;
    }
    b = l - 1;
  }
  __device__ __forceinline__ bool next() {
    for (++b; b < B; ++b) {
      const long long a = ts[b], e = ts[b + 1];
      if (a >= c1) return false;
      lo = (int)((a > c0 ? a : c0) - a);
      hi = (int)((e < c1 ? e : c1) - a);
      if (lo < hi) return true;
    }
    return false;
  }
};

struct Tile {
  bool tail;
  int row0, keys;  // prefix: first key and number of keys (a multiple of 16); tail: staged rows
};

__device__ __forceinline__ Tile tile_at(int Tb, int S, int k) {
  const int b16 = pair_base16(Tb, S);
  Tile t;
  t.row0 = k * kPairTile;
  t.tail = t.row0 >= b16;
  t.keys = t.tail ? Tb - b16 : min(kPairTile, b16 - t.row0);
  return t;
}

// mbar_wait out of line, for the MMA loop: its iterations then hold a test and
// a call per barrier.  Inlined waits and unrolled stage loops lengthen the code
// between MMAs and cost 20% of the kernel.
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* flags,
                                       long long limit_ns) {
  return mbar_wait(bar, parity, abort, flags, limit_ns);
}

// ------------------------------------------------------------ TMA producer (warp 0 of each CTA, converged)
__device__ __forceinline__ void produce(const PairParams& p, Shared& sh, unsigned char* smem, uint32_t rank, int g, int pair,
                                        int* issued, int* q_issued) {
  volatile int* abort = &sh.abort;
  const uint32_t lead = elect_lane(), arm = rank == 0 ? lead : 0;  // the leader's lane arms the barriers
  int n = 0, s = 0, freed = 0;  // stages issued, the next one's slot, freed pairs waited for
  bool ok = true;
  const uint32_t full0 = in_cta(&sh.full[0], 0), own0 = smem_u32(&sh.full[0]), ring0 = smem_u32(smem + kRingOff);
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, p.flags, p.wait_ns));
  };
  // Waits until the next stage is free: the one seven back, once its pair is.
  auto acquire = [&]() -> bool {
    if (n >= kStages && (n - kStages) / 2 >= freed) {
      if (!wait(&sh.free2[freed % kFree], (freed / kFree) & 1)) return ok = false;
      ++freed;
    }
    expect_bytes(own0 + 8 * s, 2 * kStageBytes, arm);
    return true;
  };
  auto advance = [&]() {
    ++n;
    s = s + 1 == kStages ? 0 : s + 1;
  };
  // Source rows of the two 128-key halves of tile k (a half lies in one page).
  // Looked up a tile ahead: a page table read in the way of the loads would
  // hold up the ring.
  struct Rows {
    int y[2];
  };
  auto rows_of = [&](int b, int Tb, int k) -> Rows {
    const Tile t = tile_at(Tb, p.S, k);
    if (t.tail) return Rows{{b * kPairStage, b * kPairStage}};
    bool bad = false;
    Rows r;
    r.y[0] = (int)cache_row(p.pages, b, p.T_cap, t.row0, &bad);
    // no key in the second half: its rows are not looked up (any do)
    r.y[1] = t.row0 + 128 < Tb ? (int)cache_row(p.pages, b, p.T_cap, t.row0 + 128, &bad) : r.y[0];
    if (bad) raise_flag(p.flags, MLA_DEV_BAD_INDEX);
    return r;
  };
  auto load_k = [&](const Tile& t, const Rows& r) {
    const int y = r.y[rank];
    const CUtensorMap* lat = t.tail ? &p.mT : &p.mK;
#pragma unroll 1
    for (int d = 0; d < 9; ++d) {
      if (!acquire()) return;
      const bool rope = d == 8 && !t.tail;
      load_2d(ring0 + s * kStageBytes, rope ? &p.mKr : lat, rope ? 0 : 64 * d, y, full0 + 8 * s, lead);
      advance();
    }
  };
  auto load_v = [&](const Tile& t, const Rows& r) {
    const CUtensorMap* map = t.tail ? &p.mTv : &p.mV;
#pragma unroll 1
    for (int kc = 0; uni(kc < (t.keys + 63) / 64); ++kc) {
      const int y = (t.tail || kc < 2 ? r.y[0] : r.y[1] - 128) + 64 * kc;
      for (int nb = 0; nb < 2; ++nb) {  // two 64-latent atoms of 64 keys each
        if (!acquire()) return;
        load_3d(ring0 + s * kStageBytes, map, 0, y, 4 * nb + 2 * (int)rank, full0 + 8 * s, lead);
        advance();
      }
    }
  };
  Pieces pc;
  int np = 0;
  for (pc.start(p, g); ok && uni(pc.next()); ++np) {
    const int Tb = p.T[pc.b];
    ok = wait(&sh.q_empty, (np & 1) ^ 1);
    if (!ok) break;
    expect_bytes(smem_u32(&sh.q_full), 2 * kQBytes, arm);
    const uint32_t qbar = in_cta(&sh.q_full, 0);
    const int qrow = (pc.b * p.S + 2 * pair + (int)rank) * kRows;  // past the last node: another row or zeros
    for (int d = 0; d < 9; ++d) load_2d(smem_u32(smem + d * kQAtom), &p.mQ, 64 * d, qrow, qbar, lead);
    load_2d(smem_u32(smem + 9 * kQAtom), &p.mQl, 0, qrow, qbar, lead);
    ++*q_issued;
    Rows r0 = rows_of(pc.b, Tb, pc.lo), r1 = pc.lo + 1 < pc.hi ? rows_of(pc.b, Tb, pc.lo + 1) : r0;
    load_k(tile_at(Tb, p.S, pc.lo), r0);
    for (int k = pc.lo; uni(k < pc.hi) && ok; ++k) {
      const Rows r2 = k + 2 < pc.hi ? rows_of(pc.b, Tb, k + 2) : r1;
      if (uni(k + 1 < pc.hi)) load_k(tile_at(Tb, p.S, k + 1), r1);
      if (ok) load_v(tile_at(Tb, p.S, k), r0);
      r0 = r1;
      r1 = r2;
    }
  }
  *issued = n;
  __syncwarp();
}

// ------------------------------------------------------------ MMA issuer (warp 1 of the leader CTA, converged)
__device__ __forceinline__ void issue(const PairParams& p, Shared& sh, unsigned char* smem, uint32_t tmem_any, int g) {
  volatile int* abort = &sh.abort;
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0), lead = elect_lane();
  const uint32_t idS = idesc_bf16_f32(128, 256, 0, 0), idO = idesc_bf16_f32(128, 256, 0, 1);
  const uint64_t dQ = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t dP = smem_desc_sw128(smem_u32(smem + kQBytes), 16, 1024);
  const uint64_t dK = smem_desc_sw128(smem_u32(smem + kRingOff), 16, 1024);
  const uint64_t dV = smem_desc_sw128(smem_u32(smem + kRingOff), 8192, 1024);
  int n = 0, it = 0, s = 0;
  uint32_t par = 0;  // parity of the slot's phase
  bool ok = true, ready = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, slow_wait(bar, parity, abort, p.flags, p.wait_ns));
  };
  // Waits for stage n.  The test of the stage after it is issued here, ahead
  // of this stage's MMAs, and its answer used one stage later: a barrier test
  // takes some 190 cycles, and four MMAs run for 258.
  auto acquire = [&]() -> bool {
    if (!__all_sync(0xffffffffu, ready) && !wait(&sh.full[s], par)) return ok = false;
    const int s1 = s + 1 == kStages ? 0 : s + 1;
    ready = mbar_test_wait(&sh.full[s1], s1 ? par : par ^ 1);
    return true;
  };
  // A commit after four MMAs costs the issuing warp 58 cycles that the pipe
  // idles, after eight none: stages are freed in pairs.
  auto release = [&]() {
    if (n & 1) commit_pair(&sh.free2[(n >> 1) % kFree], lead);
    ++n;
    if (++s == kStages) {
      s = 0;
      par ^= 1;
    }
  };
  auto scores = [&](int j) {  // S of tile number j
    const uint32_t d = tmem + kColS + 128 * (j & 1);
#pragma unroll 1
    for (int a = 0; a < 9; ++a) {
      if (!acquire()) return;
      const uint64_t db = dK + (uint64_t)(s * (kStageBytes >> 4)), da = dQ + (uint64_t)(a * (kQAtom >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_pair(d, da + 2 * kk, db + 2 * kk, idS, (a | kk) != 0 ? 1u : 0u, lead);
      if (a == 8) {  // the rotary keys again, with what rounding the rotated query left
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_pair(d, da + (kQAtom >> 4) + 2 * kk, db + 2 * kk, idS, 1u, lead);
      }
      release();
    }
    commit_pair(&sh.s_full[j & 1], lead);
  };
  Pieces pc;
  int np = 0;
  for (pc.start(p, g); ok && uni(pc.next()); ++np) {
    const int Tb = p.T[pc.b];
    ok = wait(&sh.q_full, np & 1);
    if (!ok) break;
    tc_fence_after();
    scores(it);
    if (ok && uni(pc.lo + 1 == pc.hi)) commit_pair(&sh.q_empty, lead);
    for (int k = pc.lo; uni(k < pc.hi) && ok; ++k, ++it) {
      if (uni(k + 1 < pc.hi)) {
        scores(it + 1);
        if (ok && uni(k + 2 == pc.hi)) commit_pair(&sh.q_empty, lead);  // the piece's last score product
      }
      ok = ok && wait(&sh.p_full, it & 1);
      if (!ok) break;
      tc_fence_after();
      const Tile t = tile_at(Tb, p.S, k);
      const uint32_t keep = uni(k > pc.lo) ? 1u : 0u;
      if (uni(t.keys == kPairTile)) {
#pragma unroll 1
        for (int kc = 0; kc < 4; ++kc) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            if (!ok || !acquire()) break;
            const uint64_t db = dV + (uint64_t)(s * (kStageBytes >> 4)), da = dP + (uint64_t)(kc * (8192 >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair(tmem + kColO + 128 * nb, da + 2 * kk, db + 128 * kk, idO, (kc | kk) != 0 ? 1u : keep, lead);
            release();
          }
        }
      } else {  // a piece's last tiles: whole 16-key steps
        for (int kc = 0; uni(kc < (t.keys + 63) / 64) && ok; ++kc) {
          const int steps = min(4, (t.keys - 64 * kc + 15) / 16);
          for (int nb = 0; nb < 2; ++nb) {
            if (!acquire()) break;
            const uint64_t db = dV + (uint64_t)(s * (kStageBytes >> 4)), da = dP + (uint64_t)(kc * (8192 >> 4));
            for (int kk = 0; uni(kk < steps); ++kk)
              mma_pair(tmem + kColO + 128 * nb, da + 2 * kk, db + 128 * kk, idO, (kc | kk) != 0 ? 1u : keep, lead);
            release();
          }
        }
      }
      if (ok) commit_pair(&sh.pv_done, lead);
    }
  }
  __syncwarp();
  commit_pair(&sh.mma_done, lead);
}

// ------------------------------------------------------------ softmax warps
// 32 lanes x 32 bits, 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The low n bits (none for n <= 0, all for n >= 64).
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

__device__ __forceinline__ void soften(const PairParams& p, Shared& sh, unsigned char* smem, uint32_t tmem, uint32_t rank,
                                       int g, int pair) {
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tsm = threadIdx.x - 64;
  const int q = warp & 3, ch = (warp - 2) >> 2;      // TMEM lane quadrant, half of its columns
  const int row = 32 * (q & 1) + lane;               // head
  const int key0 = 128 * (q >> 1) + 64 * ch;         // first key of the thread's 64 within the tile
  const uint32_t t_lane = tmem + ((uint32_t)(32 * q) << 16);
  const uint32_t p_bar = in_cta(&sh.p_full, 0);
  unsigned char* prow = smem + kQBytes + (key0 >> 6) * 8192 + row * 128;
  const int s = 2 * pair + (int)rank;
  const float c = p.c;
  int it = 0;
  Pieces pc;
  for (pc.start(p, g); pc.next();) {
    const int b = pc.b, Tb = p.T[b], b16 = pair_base16(Tb, p.S);
    unsigned long long mask = 0;
    if (s < p.S) {
      const TreeNode node = tree_node(p.parent + (size_t)b * p.S, s);
      mask = node.mask;
      if (node.state == kNodeBad && tsm == 0) raise_flag(p.flags, MLA_DEV_BAD_INDEX);
    }
    const int rem = Tb - p.S - b16;  // prefix rows at the start of the tail
    float lsum = 0.f;
    for (int k = pc.lo; k < pc.hi; ++k, ++it) {
      const bool first = k == pc.lo;
      const Tile t = tile_at(Tb, p.S, k);
      bool fail = !mbar_wait(&sh.s_full[it & 1], (it >> 1) & 1, abort, p.flags, p.wait_ns);
      if (bar_red_or(1, kSoft, fail)) return;
      tc_fence_after();
      // Scores are read from TMEM sixteen columns at a time, once for the maximum
      // and once for the probabilities, in loops that are not unrolled: the
      // eight warps' code then stays within the instruction cache next to the
      // issuing warp's, whose fetches otherwise stall the tensor pipe.
      const uint32_t sc = t_lane + kColS + 128 * (it & 1) + 64 * ch;
      unsigned long long vis = ~0ull;  // bit i: key key0 + i is visible
      const bool masked = t.tail || t.keys < kPairTile || mask == 0;
      if (masked) {
        vis = low_bits(t.keys - key0);
        if (t.tail) {  // the prefix remainder, then the tree's rows through the node's mask
          const int sh0 = rem - key0;  // the tree's first row
          vis &= low_bits(sh0) | (sh0 >= 64 ? 0 : sh0 >= 0 ? mask << sh0 : sh0 > -64 ? mask >> -sh0 : 0);
        }
        if (mask == 0) vis = 0;
      }
      float mx = -INFINITY, least = INFINITY;  // over the visible keys
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 16) {
        float v[16];
        tmem_ld16(sc + c0, v);
        tmem_wait_ld();
        const uint32_t bits = (uint32_t)(vis >> c0);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            least = (bits >> i) & 1u ? fminf(least, v[i]) : least;
            mx = (bits >> i) & 1u ? fmaxf(mx, v[i]) : mx;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) least = fminf(least, v[i]);
#pragma unroll
          for (int i = 0; i < 16; ++i) mx = fmaxf(mx, v[i]);
        }
      }
      // running maximum, moved only when a score exceeds it by more than kTau
      bool slow = first;
      float mrow = 0.f;
      if (!first) {
        mrow = sh.m[row];
        slow = bar_red_or(2, kSoft, mx * c > mrow + kTau);
      }
      bool rescale = false;
      if (slow) {
        sh.red[2 * (q >> 1) + ch][row] = mx;
        named_barrier(1, kSoft);
        bool need = false;
        if (tsm < kRows) {
          const float tmax = fmaxf(fmaxf(sh.red[0][tsm], sh.red[1][tsm]), fmaxf(sh.red[2][tsm], sh.red[3][tsm])) * c;
          const float mo = first ? kMaxFloor : sh.m[tsm];
          float mn = mo, al = 1.f;
          if (tmax > mo + kTau) {
            mn = tmax;
            al = exp2f(mo - mn);
          }
          sh.m[tsm] = mn;
          sh.alpha[tsm] = al;
          need = !first && al != 1.f;
        }
        rescale = bar_red_or(2, kSoft, need);
        mrow = sh.m[row];
      }
      if (it > 0) {  // the previous value product has read P and written O
        fail = !mbar_wait(&sh.pv_done, (it - 1) & 1, abort, p.flags, p.wait_ns);
        if (bar_red_or(1, kSoft, fail)) return;
        tc_fence_after();
      }
      // probabilities: bf16 is the value product's operand; the row sum adds the rounded values
      if (rescale) lsum *= sh.alpha[row];
      // a score of -inf stands for values that are not finite: its weight of 0 would hide them
      if (least == -INFINITY) lsum = qnan();
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 16) {
        float v[16];
        tmem_ld16(sc + c0, v);
        tmem_wait_ld();
        const uint32_t bits = (uint32_t)(vis >> c0);
        uint32_t pk[8];
        float add0 = 0.f, add1 = 0.f;
        if (masked) {  // (a branch around the loop: one inside it would cost more than the exponentials)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = (bits >> i) & 1u ? v[i] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = ex2(fmaf(v[i], c, -mrow));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pk[i] = pack2(v[2 * i], v[2 * i + 1]);
          const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&pk[i]));
          add0 += f.x;
          add1 += f.y;
        }
        lsum += add0 + add1;
        const int ck = c0 >> 3;  // 16-byte chunks ck and ck + 1 of the row, swizzled
        *reinterpret_cast<uint4*>(prow + ((ck ^ (row & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<uint4*>(prow + (((ck + 1) ^ (row & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      }
      if (rescale) {
        const float al = sh.alpha[row];
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float w[32];
          tmem_ld32(t_lane + kColO + 128 * ch + c0, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] *= al;
          tmem_st32(t_lane + kColO + 128 * ch + c0, w);
        }
        tmem_wait_st();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive_leader(p_bar);
    }
    // the piece's partial: O, running maximum and row sum
    const bool fail = !mbar_wait(&sh.pv_done, (it - 1) & 1, abort, p.flags, p.wait_ns);
    if (bar_red_or(1, kSoft, fail)) return;
    tc_fence_after();
    sh.red[2 * (q >> 1) + ch][row] = lsum;
    named_barrier(1, kSoft);
    const size_t slot = (size_t)(g + b) * p.S + s;
    if (s < p.S) {
      if (tsm < kRows) {
        float* ml = p.ml_part + (slot * kRows + tsm) * 2;
        ml[0] = sh.m[tsm];
        ml[1] = sh.red[0][tsm] + sh.red[1][tsm] + sh.red[2][tsm] + sh.red[3][tsm];
      }
      // Through the warp's 4 KB of the P buffer, so that eight lanes store 128 bytes of a
      // row: with a row per lane every store was 32 partial sectors (8 nodes on 4096 keys,
      // 19 MB of partials: the call 36.6 us against 33.8; 8 x 64 nodes 1122 against 1111).
      float* op = p.o_part + (slot * kRows + 32 * (q & 1) + (lane >> 3)) * kDl + 256 * ch + 128 * (q >> 1) + 4 * (lane & 7);
      float4* st = reinterpret_cast<float4*>(smem + kQBytes + (warp - 2) * 4096);
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float w[32];
        tmem_ld32(t_lane + kColO + 128 * ch + c0, w);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st[8 * lane + (i ^ (lane & 7))] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3);
          *reinterpret_cast<float4*>(op + (size_t)(4 * i) * kDl + c0) = st[8 * r + ((lane & 7) ^ (r & 7))];
        }
        __syncwarp();
      }
    }
    tc_fence_before();
    named_barrier(1, kSoft);  // sh.red and sh.m are reused
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) attn_pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cta_rank();
  const int cluster = blockIdx.x >> 1, pair = cluster % p.NP, g = cluster / p.NP;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1);
    for (int i = 0; i < kFree; ++i) mbar_init(&sh.free2[i], 1);
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.s_full[0], 1);
    mbar_init(&sh.s_full[1], 1);
    mbar_init(&sh.p_full, 2 * kSoftWarps);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.mma_done, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(kCols)
                 : "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  grid_dep_wait();  // queries, tile list and staged rows come from the previous kernels
  grid_dep_launch();

  int issued = 0, q_issued = 0;
  if (warp == 0) {
    produce(p, sh, smem, rank, g, pair, &issued, &q_issued);
  } else if (warp == 1) {
    if (rank == 0) issue(p, sh, smem, tmem, g);
    // both CTAs: every MMA and every arrival of its commits has happened
    volatile int no_abort = 0;
    mbar_wait(&sh.mma_done, 0, &no_abort, p.flags, p.wait_ns > kDrainNs ? p.wait_ns : kDrainNs);
    __syncwarp();
  } else {
    soften(p, sh, smem, tmem, rank, g, pair);
    __syncwarp();
  }
  // Never leave with copies in flight.  A stage's barrier expects the leader's
  // arrival and both CTAs' bytes; after an abort one of the two may have
  // issued a stage that the other has not, and the leader makes up for the
  // missing part before it waits.
  if (threadIdx.x == 0) {
    const uint32_t a = in_cta(&sh.issued[rank], 0), qa = in_cta(&sh.q_issued[rank], 0);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(issued) : "memory");
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(qa), "r"(q_issued) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    volatile int no_abort = 0;
    const long long drain = p.wait_ns > kDrainNs ? p.wait_ns : kDrainNs;
    auto settle = [&](uint64_t* bar, int i, int own, int peer, uint32_t bytes) {
      if (i >= own) mbar_arrive_expect_tx(bar, bytes);  // only the peer's bytes come
      else if (i >= peer)                               // only this CTA's do
        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                     : "memory");
    };
    const int own = sh.issued[0], peer = sh.issued[1], top = max(own, peer);
    for (int i = max(0, top - kStages); i < top; ++i) {
      settle(&sh.full[i % kStages], i, own, peer, kStageBytes);
      mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, &no_abort, p.flags, drain);
    }
    const int qo = sh.q_issued[0], qp = sh.q_issued[1], qt = max(qo, qp);
    if (qt > 0) {
      settle(&sh.q_full, qt - 1, qo, qp, kQBytes);
      mbar_wait(&sh.q_full, (qt - 1) & 1, &no_abort, p.flags, drain);
    }
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

}  // namespace

// Chunks of the tile list: G chunks times the node pairs are the items that the
// clusters take in turn, so the candidates fill one to four rounds.  More
// rounds leave fewer clusters idle, and cost a query load, a pipeline fill and
// a partial each (an item as much as about 2 tiles of 3.1 us, a node's partial
// 0.05 us to write and merge; 8 trees of 64 nodes, 32 pairs: 1130 us in two
// items per cluster, one idle in six, 1012 us in three).
int pair_chunks(int B, int S, int T_cap, int sms) {
  const int np = (S + 1) / 2, clusters = sms / 2 > 0 ? sms / 2 : 1;
  const long long tiles = (long long)B * pair_tiles(T_cap, S);
  int best = 1;
  double least = 1e30;
  for (int rounds = 1; rounds <= 4; ++rounds) {
    long long g = (long long)rounds * clusters / np;
    if (g < 1) g = 1;
    if (g > tiles) g = tiles;
    if (g > kPairChunks) break;
    const long long turns = (g * np + clusters - 1) / clusters;
    const double us = turns * 3.1 * ((double)tiles / g + 2.0) + 0.05 * (double)(g + B - 1) * S;
    if (us < least) {
      least = us;
      best = (int)g;
    }
  }
  return best;
}

cudaError_t launch_attn_pair(const PairParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(attn_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  return launch_pdl(attn_pair_kernel, dim3((unsigned)(2 * p.G * p.NP)), dim3(kThreads), kSmem, st, p);
}

}  // namespace mla
