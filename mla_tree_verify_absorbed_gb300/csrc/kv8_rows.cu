// The paged 8-bit latent cache's attention for many query rows (mla_kv8_attn), on
// tcgen05 tensor cores: 128 rows ((node, head) pairs) against tiles of 64 tokens.
//
// S = Q [128 x 576] . K^T, online softmax, O += P [128 x 64] . V [64 x 512], V the
// latent part of K.  As in the 4-bit cache's kernel an fp32 O of 128 x 512 fills one
// SM's Tensor Memory, so a cluster of two CTAs shares a work item:
//   rank 0, scores: queries in Tensor Memory (the A operand), three S tiles; softmax
//           in registers, one thread per row and tile;
//   rank 1, values: O (512 columns).
// Weights and rescale factors go from rank 0 to rank 1 by bulk copies.
//
// Both products take the cache's e4m3 codes as they are, as their B operand, so the
// tiles come by tensor copies and nothing converts them.  The A operands are sums of
// 8-bit terms that accumulate in the same columns:
//   queries  q 2^t = hi + lo, both e4m3, t per row (see kv8_attn.cu);
//   weights  three e5m2 terms.  An e5m2 number is the upper byte of an f16 one, so the
//            terms are cut off an f16 weight byte by byte: w = t1 + t2 + t3, t1 and t2
//            the upper bytes of w and of what is left, t3 what is left then, rounded:
//            3 + 3 + 3 significant bits, off by at most 2^-9, as bf16, or by 2^-17
//            where that is more.
// The rope product (bf16) accumulates in the same columns too.
//
// Blocks' scales: see kv8_attn.cu.  A row's score is s_j = c_r 2^k_j S_rj, and m follows
// the largest s_j + k_j, up and down: it falls where a tile's largest weight T of a row is
// not above 2^F, F = log2 n + d - 8 for n tokens whose k_j differ by d at most.  Beside
// their 9 bits, they are then off by 2^-17 each, as softmax weights by n 2^-17 2^d / T <=
// 2^-9 of the tile's largest together.  Where a tile's tokens share one k, c_r 2^k is one
// factor; else the scores are replaced by s_j + k_j in Tensor Memory first, as masked ones
// are by -infinity, so that the softmax's loops know of neither.
//
// What bounds it: the value CTA's products.  Per tile they are 12 MMAs of 128 cycles,
// 1,536, and their operands, the weights' arrival and the latents' loads pass 200 KB
// through shared memory, 1,590 cycles; measured 1,690 where no m moves.  The score CTA has
// 36 MMAs of 32 cycles (the bf16 rate: two terms at twice the rate) and a softmax of 1,700
// for two tiles in turn.  A tree of 64 nodes x 64 heads over 200,000 tokens, 1.78e12
// operations: 1,340 us (1,260 at the best clocks), 1.33 PFLOP/s of the 1.93 measured for
// bf16; 1,490 with queries four times as large, where some m moves at most tiles.  Short
// work adds a cluster's start, 6 us per piece for the queries' way into Tensor Memory, 4 us
// for its output, and the merge: 30 sequences of 4,096 to 8,192 tokens x 128 heads 69 us.
//
// Work split as in split.cuh; pieces of a row group are merged by a second kernel.  Every
// wait is bounded (2 s, less in the self-test); on timeout both CTAs stop issuing, drain
// what they issued, free their Tensor Memory and report MLA_DEVERR_TIMEOUT.
#include <cuda.h>
#include <cuda_fp8.h>

#include <cstddef>
#include <mutex>

#include "kv8.cuh"
#include "sm100.cuh"
#include "split.cuh"
#include "tensor_map.cuh"

namespace mlav {
namespace kv8 {
namespace rows {
using namespace sm100;
using kvq::for_pieces;
using kvq::kErrFirst;
using kvq::kPieces;
using kvq::NodeView;
using kvq::Piece;
using kvq::Start;

constexpr int kRG = kvq::kRows128;
constexpr int kTK = 64;  // tokens per tile
// Warps 0-7 hold rows, in two groups that take the tiles of one parity; 8 and 9 fetch
// 32 tokens each.
constexpr int kRowWarps = 8, kProducerWarps = 2;
constexpr int kWarpProd = kRowWarps;
constexpr int kWarpAux = 10;    // TMEM allocation; rank 0: weight copies
constexpr int kWarpMma = 11;
constexpr int kWarpSched = 12;  // the pieces of work
constexpr int kThreads = 32 * (kWarpSched + 1);
constexpr uint32_t kTmemCols = 512;

// A piece costs kFixed tiles beside its own: the queries' way into Tensor Memory, the
// output, its merging.  Single sizes jump by 6% with where the cuts fall; the mean of 14
// (decode of 7 to 60 sequences x 128 heads, trees of 8 and 32 nodes x 64 heads, windows
// of 4,096) took, against kFixed 4: 6 1.8% less, 7 1.9%, 8 2.2%, 10 0.8%.
constexpr int kFixed = 8, kMinTiles = 4;
using Work = kvq::Split<kTK, kFixed, kMinTiles, kThreads, true>;

constexpr int kChunk = kTK * 128;             // 128 bytes of each token: 128 latents, or the rope key
constexpr int kChunksS = 5, kChunksV = 4;     // score CTA: with the rope keys
constexpr int kStageS = kChunksS * kChunk;    // 40 KB
constexpr int kStageV = kChunksV * kChunk;    // 32 KB
constexpr int kStages = 4;
constexpr int kTerm = kRG * kTK;              // a term of a tile's weights, e5m2: rows of 64 bytes
constexpr int kPBytes = 3 * kTerm;
constexpr int kPBufs = 3;                     // value CTA: weights landed
constexpr int kPStages = 2;                   // score CTA: weights staged
constexpr int kOffPS = kStages * kStageS, kOffPV = kStages * kStageV;
constexpr int kOffCtl = kOffPS + kPStages * kPBytes > kOffPV + kPBufs * kPBytes ? kOffPS + kPStages * kPBytes
                                                                                : kOffPV + kPBufs * kPBytes;
// Tiles whose tokens' scales are kept: a place is written again when S of the tile 12
// behind is complete, for which every row warp has passed the tile 8 behind.
constexpr int kInv = 16;
// A row group with few rows leaves whole lane quadrants of 32 rows unused: their
// softmax, weights and outputs are left out.
__device__ __forceinline__ int live_quads(int rows, int g) { return min(4, (rows - g * kRG + 31) >> 5); }

// Tensor Memory columns: score CTA, three S tiles and the queries (hi, lo: four e4m3
// elements a column; rope: bf16 pairs); value CTA, O from column 0
constexpr int kSBufs = 3;
constexpr uint32_t kColS = 0, kColHi = kSBufs * kTK, kColLo = kColHi + kDl / 4, kColPe = kColLo + kDl / 4;
static_assert(kColPe + kDr / 2 <= kTmemCols, "Tensor Memory columns");

// halves of the operand descriptors (smem_desc): only the start address, in the
// lower half, differs from MMA to MMA
constexpr uint32_t kDescHi128 = (1024u >> 4) | (1u << 14) | (kLayoutSw128 << 29);  // keys, values
constexpr uint32_t kDescHi64 = (512u >> 4) | (1u << 14) | (kLayoutSw64 << 29);     // weights: rows of 64 bytes
constexpr uint32_t kDescLoK = (16u >> 4) << 16;               // K-major
constexpr uint32_t kDescLoV = ((uint32_t)kChunk >> 4) << 16;  // MN-major: chunks of 128 latents
__device__ __forceinline__ uint32_t desc_addr(const uint8_t* smem, uint32_t off) {
  return ((smem_u32(smem) & 0x3FFFFu) + off) >> 4;
}
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
constexpr uint32_t kIdescS = idesc_e4m3_f32(kRG, kTK, 0, 0), kIdescPe = idesc_bf16_f32(kRG, kTK, 0, 0);
constexpr uint32_t kIdescPV = idesc_e5m2_e4m3_f32(kRG, 256, 0, 1);

constexpr uint64_t kDrainLimitNs = 20000000ull;

// Weights are 2^(s + k - m + kWeightShift), at most 2^kTop, below e5m2's 57,344.  m moves
// rarely, since O's products wait meanwhile: the largest weight of a piece's first tile is
// put at 2^kWeightShift, one that is too large, and thus rare, at 2^kRisen, a tile whose
// weights are too small 2^kFallen above the least.
constexpr float kTop = 15.f, kWeightShift = 7.f, kRisen = 14.f, kFallen = 3.f;
constexpr int kLossLog2 = 8;
// m stays within 2^kDeepest of the largest so far: O and the sums stay far from fp32's
// limits, and what is lost is below 2^-64 of the largest weight.
constexpr float kDeepest = 40.f;

// Barriers that two groups of warps pass at different tiles have one instance
// per buffer they guard: a wait must never be able to pass on the parity of an
// older phase.
struct alignas(16) Ctl {
  uint64_t full[kStages];      // tile landed (each producer warp's copies)
  uint64_t empty[kStages];     // the MMAs reading it are complete
  uint64_t s_full[kSBufs];     // score: S tile in TMEM, and the MMA warp's word that the tile's scales are there
  uint64_t s_free[kSBufs];     // score: softmax has loaded S (4 row warps)
  uint64_t q_ready[kPieces];   // score: a piece's queries in TMEM, stages free again (8 row warps)
  uint64_t q_in[3];            // score: three chunks of the queries copied (copy bytes)
  uint64_t q_max;              // score: halves' largest queries written (8 row warps)
  uint64_t m_ready[2][4];      // score: m_run, best after a tile written (per lane quadrant, 1 warp)
  uint64_t p_free[kPBufs];     // score: the PV MMAs that read rank 1's buffer are complete (its commit)
  uint64_t ps_free[kPStages];  // score: the staged weights have landed in rank 1 (its first row warp)
  uint64_t fin_free;           // score: rank 1 consumed lfin / mfin (256 arrivals)
  uint64_t p_staged[kPStages]; // score: weights and factors staged (4 row warps)
  uint64_t p_full[kPBufs];     // value: weights and factors landed (copy bytes)
  uint64_t pv_done[2][kPBufs];  // value: a tile's MMAs into half of O's columns complete
  uint64_t o_ready[2][kPBufs];  // value: that half rescaled, weights in (4 row warps)
  uint64_t fin_full;           // value: lfin / mfin written (256 remote arrivals)
  uint64_t drain;
  uint64_t piece_full[kPieces];   // piece written (scheduler warp)
  uint64_t piece_empty[kPieces];  // read by every warp of this CTA that follows the pieces
  Piece piece[kPieces];
  alignas(16) float alpha[kPBufs][kRG];  // rescale factors: staged in rank 0 ([kPStages]), landed in rank 1
  alignas(16) float inv[kInv][kTK];      // score: 2^-k of the tokens' blocks
  uint32_t q_big[2][kRG];      // score: largest magnitude of half a query, as bits
  float m_run[2][kRG];         // score: m after the last tile of each parity,
  float best[2][kRG];          // and the largest score + k so far
  float lfin[2][kRG];          // value: each group's row sums of the weights
  float mfin[kRG];             // value: rows' m, base-2 units
  int64_t scan[kThreads / 32];
  int64_t left;                // units of this cluster's interval
  int64_t start_x;             // this cluster's first unit within sequence start_b
  int start_b, start_T;        // that sequence, its tiles,
  int start_P;                 // its prefix length
  int64_t start_entry;         // and its first table entry
  uint64_t wait_ns;            // Params::wait_ns
  uint32_t tmem_base;
  int abort;
  uint32_t err;
};
constexpr int kSmemBytes = kOffCtl + (int)sizeof(Ctl);
constexpr int kSmemAlloc = (kSmemBytes + 1023) & ~1023;
static_assert(kSmemAlloc <= 232448, "shared memory budget");
static_assert(offsetof(Ctl, alpha) % 16 == 0 && kOffCtl % 16 == 0, "bulk-copy alignment");
static_assert(kOffPS % 1024 == 0 && kOffPV % 1024 == 0 && kPBytes % 1024 == 0, "swizzle atoms");
static_assert(9 * kRG * 128 <= kStages * kStageS, "queries fit the stages");

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Ctl* c) {
  if (mbar_wait(bar, parity, &c->abort, c->wait_ns, true)) return true;
  for (uint32_t rk = 0; rk < 2; ++rk) st_cluster_u32(mapa_shared(smem_u32(&c->abort), rk), 1u);
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* c) {
  return mbar_try_wait_cluster(bar, parity) || wait_slow(bar, parity, c);
}
// Every lane waits; the result is warp-uniform and the warp converged.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctl* c) {
  return __all_sync(0xffffffffu, wait(bar, parity, c));
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t sub_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

constexpr int kFollowers = kRowWarps + kProducerWarps + 1;  // and, in the score CTA, the copier

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
// As in kv8_attn.cu: tensor copies of a page's rows where pages allow it, else cp.async,
// which takes the score CTA 3,500 cycles per tile where the products take 1,690.  (Four
// warps in place of two: 17% slower; tiles in flight one or two in place of four: the same.)
template <bool kScore>
__device__ __forceinline__ void producer(const Params& p, const CUtensorMap& map, uint8_t* smem, Ctl* c, int pw) {
  constexpr int kChunks = kScore ? kChunksS : kChunksV;
  const int lane = threadIdx.x & 31;
  uint32_t err = 0, j = 0, seg = 0;
  for_pieces(c, [&](const Piece& pc) {
    const int32_t* idx = (p.page_size == 1 ? p.kv_indices : p.block_table) + pc.entry;
    auto pos_of = [&](int v) { return (uint32_t)pc.tile(v) * kTK + 32 * pw + lane; };
    auto seen = [&](int v, uint32_t pos) {
      return v < pc.t1 && pos < (uint32_t)pc.N && (pos >= (uint32_t)pc.lo || pos < (uint32_t)p.sinks);
    };
    auto entry_of = [&](int v) -> int32_t {
      const uint32_t pos = pos_of(v);
      return seen(v, pos) ? __ldg(idx + kvq::page_of(p, pos)) : -1;
    };
    // -1: not read, zeros in its place
    auto slot_of = [&](int32_t e, int v) -> int32_t {
      const uint32_t pos = pos_of(v);
      const int64_t s = (int64_t)e * p.page_size + (pos - kvq::page_of(p, pos) * (uint32_t)p.page_size);
      if (e >= 0 && s < p.slots) return (int32_t)s;
      if (seen(v, pos)) err |= MLA_DEVERR_SLOT;
      return -1;
    };
    auto word_of = [&](int32_t slot) {
      return kScore && slot >= 0 ? (uint32_t)__ldg(p.scales + p.block((uint32_t)slot)) : 0u;
    };
    int32_t slot = slot_of(entry_of(pc.t0), pc.t0), ent = entry_of(pc.t0 + 1);
    uint32_t word = word_of(slot);
    // the queries pass through the stages first
    if (kScore && !wait_warp(&c->q_ready[seg % kPieces], (seg / kPieces) & 1u, c)) return false;
    ++seg;
#pragma unroll 1
    for (int v = pc.t0; v < pc.t1; ++v, ++j) {
      const int32_t next = slot_of(ent, v + 1);
      const uint32_t next_word = word_of(next);
      ent = entry_of(v + 2);
      const uint32_t st = j % kStages;
      uint8_t* to = smem + st * (kScore ? kStageS : kStageV) + 32 * pw * 128;
      const uint32_t dst = smem_u32(to);
      const bool boxes = p.box > 0 && __all_sync(0xffffffffu, seen(v, pos_of(v)));
      uint64_t* full = &c->full[st];
      if (!wait_warp(&c->empty[st], ((j / kStages) & 1u) ^ 1u, c)) return false;
      if (kScore) {
        c->inv[j % kInv][32 * pw + lane] = pow2(-scale_of(word));
        __syncwarp();
      }
      if (boxes) {
        if (lane == 0) mbar_arrive_expect_tx(full, kChunks * 32 * 128);
        __syncwarp();
        const bool leader = elect_one();
#pragma unroll 1
        for (int i = 0; i < 32; i += p.box) {
          const int32_t s = __shfl_sync(0xffffffffu, slot, i);
          if (leader) {
#pragma unroll
            for (int ck = 0; ck < kChunks; ++ck) tensor_copy_2d(to + ck * kChunk + i * 128, &map, 128 * ck, s, full);
          }
          __syncwarp();
        }
      } else {
        const int r7 = lane & 7, ch = lane >> 3;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int token = 4 * i + ch;
          const int32_t s = __shfl_sync(0xffffffffu, slot, token);
          const uint8_t* src = p.cache + (uint64_t)(uint32_t)max(s, 0) * (uint32_t)p.row_stride + 16 * r7;
          const uint32_t at = dst + token * 128 + ((r7 ^ (token & 7)) << 4), bytes = s >= 0 ? 16u : 0u;
#pragma unroll
          for (int ck = 0; ck < kChunks; ++ck) cp_async_16_zfill(at + ck * kChunk, src + 128 * ck, bytes);
        }
        cp_async_mbar_hold(full);  // until they have landed
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      slot = next;
      word = next_word;
    }
    return true;
  });
  cp_async_wait_all();
  if (err) atomicOr(&c->err, err);
}

// On abort, outstanding MMAs must finish before Tensor Memory is released.
__device__ void drain_mmas(Ctl* c, bool leader) {
  __syncwarp();
  if (!__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&c->abort) != 0)) return;
  if (leader) {
    mma_cta_commit(&c->drain);
    mbar_wait_drain(&c->drain, 0, kDrainLimitNs);
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// score CTA
// ---------------------------------------------------------------------------
__device__ void score_mma(uint8_t* smem, Ctl* c) {
  const bool leader = elect_one();
  uint32_t j = 0, seg = 0;
  for_pieces(c, [&](const Piece& pc) {
    if (!wait_warp(&c->q_ready[seg % kPieces], (seg / kPieces) & 1u, c)) return false;
#pragma unroll 1
    for (int t = pc.t0; t < pc.t1; ++t, ++j) {
      const uint32_t st = j % kStages, sb = j % kSBufs;
      if (!wait_warp(&c->s_free[sb], ((j / kSBufs) & 1u) ^ 1u, c)) return false;
      if (!wait_warp(&c->full[st], (j / kStages) & 1u, c)) return false;
      fence_proxy_async_smem();  // the tile may have come by cp.async, without a fence of its writers
      tc_fence_after();
      if (leader) {
        const uint32_t lo = desc_addr(smem, st * kStageS) | kDescLoK, d = kColS + sb * kTK;
#pragma unroll
        for (uint32_t term = 0; term < 2; ++term) {
#pragma unroll
          for (uint32_t k = 0; k < 16; ++k)
            mma_cta_ts_f8(d, (term ? kColLo : kColHi) + 8 * k,
                          desc_at(lo + (((k >> 2) * kChunk + (k & 3) * 32) >> 4), kDescHi128), kIdescS, term | k);
        }
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          mma_cta_ts(d, kColPe + 8 * k, desc_at(lo + ((4 * kChunk + k * 32) >> 4), kDescHi128), kIdescPe, 1);
        mma_cta_commit(&c->s_full[sb]);
        mma_cta_commit(&c->empty[st]);
        mbar_arrive(&c->s_full[sb]);  // passes on that the tile's scales are visible
      }
      __syncwarp();
    }
    ++seg;
    return true;
  });
  drain_mmas(c, leader);
}

// Brings a piece's query rows into Tensor Memory as e4m3 terms, all row warps together:
// nine tensor copies of 64 elements of the rows fill the stages, which are free between
// pieces (the producers wait for q_ready before they fill them); a thread then takes
// half a row.  Returns the row's score factor.
__device__ bool stage_queries(const Params& p, const QueryMaps& maps, uint8_t* smem, Ctl* c, const Piece& pc, int warp,
                              uint32_t seg, float* unit) {
  const int lane = threadIdx.x & 31;
  const int wq = warp & 3, wg = warp >> 2;
  const int r = wq * 32 + lane;
  const int rows = min(kRG, p.rows - pc.g * kRG);
  const uint32_t chunk = (uint32_t)p.box_rows * 128;
  if (warp == 0 && elect_one()) {
    fence_proxy_async_smem();  // parts of the stages may have been read or written through the generic proxy
    const int y = pc.b * p.rows + pc.g * kRG;
#pragma unroll 1
    for (int ck = 0; ck < 9; ++ck) {
      if (ck % 3 == 0) mbar_arrive_expect_tx(&c->q_in[ck / 3], 3u * chunk);
      tensor_copy_2d(smem + ck * kRG * 128, ck < 8 ? &maps.lat : &maps.pe, ck < 8 ? 64 * ck : 0, y, &c->q_in[ck / 3]);
    }
  }
  __syncwarp();
  const bool live = r < rows;  // else another sequence's rows, or none
  auto half_chunk = [&](int ck, uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0;
    if (!live) return;
    const uint32_t src = smem_u32(smem) + ck * kRG * 128 + r * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ld_shared_v4(src + (((4 * wg + i) ^ (r & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  };
  uint32_t big2 = 0;  // magnitudes compare as their bits
#pragma unroll 1
  for (int ck = 0; ck < 9; ++ck) {
    if (ck % 3 == 0 && !wait_warp(&c->q_in[ck / 3], seg & 1u, c)) return false;
    uint32_t w[16];
    half_chunk(ck, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) big2 = __vmaxu2(big2, w[i] & 0x7fff7fffu);
  }
  uint32_t big = max(big2 & 0xffffu, big2 >> 16);
  c->q_big[wg][r] = big;
  __syncwarp();
  if (lane == 0) mbar_arrive(&c->q_max);
  if (!wait_warp(&c->q_max, seg & 1u, c)) return false;
  big = max(big, c->q_big[wg ^ 1][r]);
  const int t = query_unit(big);
  const float mul = pow2(t);
  *unit = query_factor(p.scale_log2, t);
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
#pragma unroll 1
  for (int ck = 0; ck < 9; ++ck) {
    uint32_t w[16];
    half_chunk(ck, w);
    if (ck < 8) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) query_terms(w[2 * i], w[2 * i + 1], mul, big < 0x7f80u, hi[i], lo[i]);
      __syncwarp();
      tmem_st_32x32b_x8(lanes + kColHi + 16 * ck + 8 * wg, hi);
      tmem_st_32x32b_x8(lanes + kColLo + 16 * ck + 8 * wg, lo);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16(__uint_as_float(w[i] << 16) * mul, __uint_as_float(w[i] & 0xffff0000u) * mul);
      __syncwarp();
      tmem_st_32x32b_x16(lanes + kColPe + 16 * wg, w);
    }
  }
  tmem_wait_st();
  return true;
}

// The low n bits, n clamped to [0, 64].
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : ~0ull >> (64 - n); }

// Online softmax: a thread per row and group of row warps; group `wg` takes
// the tiles of its parity, all 64 columns of a row in one thread.  m passes
// from group to group, warp to warp of the same rows, before the
// exponentials; each group sums its own weights.
__device__ void score_softmax(const Params& p, const QueryMaps& maps, uint8_t* smem, Ctl* c, int warp) {
  const int lane = threadIdx.x & 31;
  const int wq = warp & 3, wg = warp >> 2;
  const int r = wq * 32 + lane;
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const int nq = p.Q;
  uint32_t j = 0, seg = 0;
  bool bad = false;
  for_pieces(c, [&](const Piece& pc) {
    const int t0 = pc.t0, t1 = pc.t1;
    const int row = pc.g * kRG + r;
    const bool live = row < p.rows;
    const bool idle = wq >= live_quads(p.rows, pc.g);  // none of the warp's rows exists
    const int P = pc.P;
    float unit = 0.f;
    if (!stage_queries(p, maps, smem, c, pc, warp, seg, &unit)) return false;
    tc_fence_before();
    fence_proxy_async_smem();  // the stages have been read; tensor copies fill them next
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->q_ready[seg % kPieces]);
    // rows past the last take the last one's mask: their results are dropped
    const NodeView nv = kvq::node_view_warp(p, pc.b, (live ? row : p.rows - 1) / p.H, P, &bad);
    // Prefix positions up to this one are outside the window (unless sinks).
    // Lengths fit 32 bits with the nodes counted, so these do too, and so do
    // their differences from a position as long as they are not below -1.
    const int past = p.window > 0 ? max(P - p.window + nv.depth, -1) : -1;
    const int past_any = p.window > 0 ? max(P - p.window + nq - 1, -1) : -1;

    // m: as of this group's last tile, base-2 units;
    // l: its sum of the shifted weights before rounding, times 2^-k
    float m = -INFINITY, l = 0.f;
    const uint32_t jl = j + (uint32_t)(t1 - t0) - 1;  // the piece's last tile
    uint32_t i = j + ((wg ^ j) & 1u);
#pragma unroll 1
    for (int t = t0 + (int)(i - j); t < t1; t += 2, i += 2) {
      const uint32_t sb = i % kSBufs;
      if (!wait_warp(&c->s_full[sb], (i / kSBufs) & 1u, c)) return false;
      const uint32_t ps = i % kPStages;
      if (idle) {
        // every barrier's phases count on: the next piece may use the rows
        if (lane == 0) {
          mbar_arrive(&c->m_ready[wg][wq]);
          mbar_arrive(&c->s_free[sb]);
        }
        if (!wait_warp(&c->ps_free[ps], ((i / kPStages) & 1u) ^ 1u, c)) return false;
        if (lane == 0) mbar_arrive(&c->p_staged[ps]);
        continue;
      }
      tc_fence_after();
      const float* inv = c->inv[i % kInv];
      const uint32_t i0 = __float_as_uint(inv[lane]), i1 = __float_as_uint(inv[lane + 32]);
      const uint32_t small = __reduce_min_sync(0xffffffffu, min(i0, i1)), large = __reduce_max_sync(0xffffffffu, max(i0, i1));
      const bool one = small == large;  // one scale for all tokens
      const int k0 = one ? 127 - (int)(small >> 23) : 0;
      const float factor = one ? unit * pow2(k0) : 1.f, kf = (float)k0;
      // which of the tile's 64 tokens the row sees, where not all of them
      const int pos0 = pc.tile(t) * kTK;
      const int d = (int)(large >> 23) - (int)(small >> 23);
      const float least = (float)(32 - __clz(min(pc.N - pos0, kTK) - 1) + d - kLossLog2);  // F
      const uint32_t tS = lane_off + kColS + sb * kTK;
      const bool masked = pos0 > P - kTK || pos0 <= past_any;
      if (masked || !one) {
        uint64_t vis = ~0ull;
        if (masked) {
          const int rel0 = pos0 - P;
          vis = low_bits(-rel0) & ~(low_bits(past - pos0 + 1) & ~low_bits(p.sinks - pos0));
          if (rel0 < 64 && rel0 > -64) vis |= rel0 >= 0 ? nv.mask >> rel0 : nv.mask << -rel0;
        }
        // the scores go back, and the loops below know of no mask and of one scale
#pragma unroll 1
        for (int hc = 0; hc < 2; ++hc) {
          uint32_t u[32];
          tmem_ld32_sync(tS + 32 * hc, u);
          if (!one) {
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const uint32_t b = __float_as_uint(inv[32 * hc + q]);  // of 2^-k: 2^k and k from its exponent
              u[q] = __float_as_uint(fmaf(__uint_as_float(u[q]) * __uint_as_float((254u << 23) - b), unit,
                                          (float)(127 - (int)(b >> 23))));
            }
          }
          const uint32_t v32 = (uint32_t)(vis >> (32 * hc));
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (!((v32 >> q) & 1u)) u[q] = 0xff800000u;
          tmem_st_32x32b_x32(tS + 32 * hc, u);
        }
        tmem_wait_st();
      }
      // Two passes of 32 columns, for the maximum and for the weights: the
      // scores stay in Tensor Memory in between, which halves the registers
      // and the code.  The maximum comes with the load.  A NaN score makes the
      // row's sum NaN whichever way the maximum takes it.
      float tmax = -INFINITY;
#pragma unroll 1
      for (int hc = 0; hc < 2; ++hc) tmax = fmaxf(tmax, tmem_max32(tS + 32 * hc));
      // the factor is positive: the scaled maximum is the maximum of the scaled scores
      tmax = fmaf(tmax, factor, kf);
      // m after the tile before, from the other group (in the first tile of a
      // piece the wait only keeps the groups in step)
      float mp = -INFINITY, best = -INFINITY;
      if (i > 0) {
        if (!wait_warp(&c->m_ready[wg ^ 1][wq], ((i - 1) >> 1) & 1u, c)) return false;
        if (t > t0) {
          mp = c->m_run[wg ^ 1][r];
          best = c->best[wg ^ 1][r];
        }
      }
      // It rises only when this tile's weights are too large in some row of the warp, and
      // then in all rows where they are large: O's rows are rescaled together, which holds
      // up its products for 1,300 cycles, and so less often.  It falls row by row, by whole
      // numbers, which move O and the sums exactly.
      best = fmaxf(best, tmax);
      float mn = mp;
      if (__any_sync(0xffffffffu, tmax > mp + (kTop - kWeightShift)))
        mn = mp == -INFINITY ? tmax : fmaxf(mp, tmax - (kRisen - kWeightShift));
      const float largest = tmax - mn + kWeightShift;
      if (tmax > -INFINITY && largest <= least)
        mn -= floorf(fminf(fminf(least + kFallen, kTop) - largest, mn - best + kDeepest));
      c->m_run[wg][r] = mn;
      c->best[wg][r] = best;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->m_ready[wg][wq]);
      const float alpha = mn == mp ? 1.f : exp2f(mp - mn);  // 0 when mp is -infinity
      if (mn != m) {
        l *= exp2f(m - mn);
        m = mn;
      }
      const float nmu = (m == -INFINITY ? 0.f : kWeightShift - m) + kf;

      if (!wait_warp(&c->ps_free[ps], ((i / kPStages) & 1u) ^ 1u, c)) return false;
      const uint32_t pst = smem_u32(smem) + kOffPS + ps * kPBytes + r * 64;
      const uint64_t factor2 = pair(factor, factor), nmu2 = pair(nmu, nmu);
      uint64_t ls = 0;  // two fp32 sums
#pragma unroll 1
      for (int hc = 0; hc < 2; ++hc) {
        uint32_t u[32];
        tmem_ld32_sync(tS + 32 * hc, u);
        if (hc) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->s_free[sb]);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {  // 16 tokens
          uint32_t a[4], b[4], d[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const ulonglong2 iv = reinterpret_cast<const ulonglong2*>(inv + 32 * hc + 16 * g)[q];
            uint32_t w[2], r1[2], r2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int n = 16 * g + 4 * q + 2 * h;
              const uint64_t x = fma_f32x2(pair(u[n], u[n + 1]), factor2, nmu2);
              const float e0 = ex2_approx(lo_f32(x)), e1 = ex2_approx(hi_f32(x));
              ls = fma_f32x2(pair(e0, e1), h ? iv.y : iv.x, ls);
              w[h] = pack_f16(e0, e1);
              r1[h] = sub_f16(w[h], w[h] & 0xff00ff00u);            // exact
              r2[h] = sub_f16(r1[h], r1[h] & 0xff00ff00u) + 0x00800080u;  // exact, then rounded at the upper byte
            }
            a[q] = __byte_perm(w[0], w[1], 0x7531);
            b[q] = __byte_perm(r1[0], r1[1], 0x7531);
            d[q] = __byte_perm(r2[0], r2[1], 0x7531);
          }
          const uint32_t at = pst + (((2 * hc + g) ^ ((r >> 1) & 3)) << 4);
          st_shared_v4(at, a);
          st_shared_v4(at + kTerm, b);
          st_shared_v4(at + 2 * kTerm, d);
        }
      }
      l += lo_f32(ls) + hi_f32(ls);
      c->alpha[ps][r] = alpha;
      fence_proxy_async_smem();  // read by the copy engine
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->p_staged[ps]);
    }

    // both groups' sums go to the value CTA relative to the last m, which the
    // group of the last tile has
    if ((jl & 1u) != (uint32_t)wg && !idle) {
      if (!wait_warp(&c->m_ready[wg ^ 1][wq], (jl >> 1) & 1u, c)) return false;
      const float mn = c->m_run[wg ^ 1][r];
      if (mn != m) l *= exp2f(m - mn);
    }
    if (!wait_warp(&c->fin_free, (seg & 1u) ^ 1u, c)) return false;
    st_cluster_f32(mapa_shared(smem_u32(&c->lfin[wg][r]), 1), l);
    if ((jl & 1u) == (uint32_t)wg) st_cluster_f32(mapa_shared(smem_u32(&c->mfin[r]), 1), m);
    mbar_arrive_cluster(&c->fin_full, 1);
    j = jl + 1;
    ++seg;
    return true;
  });
  if (bad) atomicOr(&c->err, MLA_DEVERR_PARENT);
}

// One warp of the score CTA, one thread of it copying: ships each tile's weights and
// factors to the value CTA, where their bytes complete p_full.
__device__ __forceinline__ uint32_t term_bytes(int quads) { return (uint32_t)quads * 32u * kTK; }
__device__ void weight_copier(const Params& p, uint8_t* smem, Ctl* c) {
  const bool leader = elect_one();
  uint32_t j = 0;
  for_pieces(c, [&](const Piece& pc) {
    const uint32_t bytes = term_bytes(live_quads(p.rows, pc.g));
    for (int t = pc.t0; t < pc.t1; ++t, ++j) {
      const uint32_t ps = j % kPStages, pb = j % kPBufs;
      if (!wait_warp(&c->p_staged[ps], (j / kPStages) & 1u, c)) return false;
      if (!wait_warp(&c->p_free[pb], ((j / kPBufs) & 1u) ^ 1u, c)) return false;
      if (leader) {
        const uint32_t bar = mapa_shared(smem_u32(&c->p_full[pb]), 1);
        const uint32_t to = mapa_shared(smem_u32(smem + kOffPV + pb * kPBytes), 1);
        const uint8_t* from = smem + kOffPS + ps * kPBytes;
        if (bytes == kTerm) {
          bulk_copy_s2c(to, from, kPBytes, bar);
        } else {
#pragma unroll 1
          for (int k = 0; k < 3; ++k) bulk_copy_s2c(to + k * kTerm, from + k * kTerm, bytes, bar);
        }
        bulk_copy_s2c(mapa_shared(smem_u32(&c->alpha[pb][0]), 1), &c->alpha[ps][0], kRG * 4, bar);
      }
      __syncwarp();
    }
    return true;
  });
}

// ---------------------------------------------------------------------------
// value CTA
// ---------------------------------------------------------------------------
__device__ void value_mma(const Params& p, uint8_t* smem, Ctl* c) {
  const bool leader = elect_one();
  uint32_t j = 0;
  // the self-test: nothing completes this barrier, so the roles before this one
  // fill every buffer and wait, each on its own barrier
  if (p.hold && !wait_warp(&c->drain, 0u, c)) return;
  for_pieces(c, [&](const Piece& pc) {
#pragma unroll 1
    for (int t = pc.t0; t < pc.t1; ++t, ++j) {
      const uint32_t st = j % kStages, pb = j % kPBufs;
      if (!wait_warp(&c->full[st], (j / kStages) & 1u, c)) return false;
      // Half of the columns after the other: while the products of one are running, the
      // other can be rescaled.
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        if (!wait_warp(&c->o_ready[h][pb], (j / kPBufs) & 1u, c)) return false;
        fence_proxy_async_smem();  // the tile may have come by cp.async, without a fence of its writers
        tc_fence_after();
        if (leader) {
          const uint32_t da = desc_addr(smem, kOffPV + pb * kPBytes) | kDescLoK;
          const uint32_t dv = desc_addr(smem, st * kStageV + h * 2 * kChunk) | kDescLoV;
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k) {  // 32 tokens
#pragma unroll
            for (uint32_t term = 0; term < 3; ++term)
              mma_cta_ss_f8(h * 256, desc_at(da + ((term * kTerm + k * 32) >> 4), kDescHi64),
                            desc_at(dv + ((k * 32 * 128) >> 4), kDescHi128), kIdescPV,
                            k | term | (uint32_t)(t - pc.t0));
          }
          mma_cta_commit(&c->pv_done[h][pb]);
          if (h == 1) {
            mma_cta_commit(&c->empty[st]);
            mma_cta_commit(&c->p_free[pb], 0x1);
          }
        }
        __syncwarp();
      }
    }
    return true;
  });
  drain_mmas(c, leader);
}

// Row warps of the value CTA (warpgroup h: columns [256 h, 256 h + 256)):
// rescale O where a factor is not 1, and per piece normalise and store it.
__device__ void value_rows(const Params& p, Ctl* c) {
  const int lane = threadIdx.x & 31;
  const int w = threadIdx.x >> 5;
  const int wq = w & 3, h = w >> 2;
  const int r = wq * 32 + lane;
  const int col0 = 256 * h;
  const uint32_t tO = ((uint32_t)(wq * 32) << 16) + (uint32_t)col0;
  int j = 0, seg = 0;
  for_pieces(c, [&](const Piece& pc) {
    const int slot = pc.slot, b = pc.b, g = pc.g, t0 = pc.t0;
    const int quads = live_quads(p.rows, g);
    for (int t = t0; t < pc.t1; ++t, ++j) {
      const int pb = j % kPBufs;
      if (w == 0 && lane == 0) mbar_arrive_expect_tx(&c->p_full[pb], 3 * term_bytes(quads) + kRG * 4);
      if (!wait_warp(&c->p_full[pb], (uint32_t)(j / kPBufs) & 1u, c)) return false;
      if (w == 0 && lane == 0) mbar_arrive_cluster_relaxed(&c->ps_free[j % kPStages], 0);
      if (t != t0 && wq < quads) {
        const float a = c->alpha[pb][r];
        if (__any_sync(0xffffffffu, a != 1.f)) {
          if (!wait_warp(&c->pv_done[h][(j - 1) % kPBufs], (uint32_t)((j - 1) / kPBufs) & 1u, c)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 256; c0 += 64) {
            uint32_t u[64];
            tmem_ld64_sync(tO + c0, u);
#pragma unroll
            for (int q = 0; q < 64; ++q) u[q] = __float_as_uint(__uint_as_float(u[q]) * a);
            tmem_st64(tO + c0, u);
          }
          tmem_wait_st();
        }
      }
      fence_proxy_async_smem();  // the weights feed the MMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->o_ready[h][pb]);
    }

    if (!wait_warp(&c->pv_done[h][(j - 1) % kPBufs], (uint32_t)((j - 1) / kPBufs) & 1u, c)) return false;
    if (!wait_warp(&c->fin_full, (uint32_t)seg & 1u, c)) return false;
    tc_fence_after();
    const float l = c->lfin[0][r] + c->lfin[1][r], m = c->mfin[r];
    // The sums are read before the score CTA may write the next piece's: a release at
    // cluster scope orders its remote stores behind these loads.  A piece that is known
    // to be the cluster's last goes without: nothing waits for it.
    const uint32_t nq = (uint32_t)(seg + 1) % kPieces;
    const bool last =
        mbar_test_wait_cluster(&c->piece_full[nq], ((uint32_t)(seg + 1) / kPieces) & 1u) && c->piece[nq].b < 0;
    if (!last) mbar_arrive_cluster(&c->fin_free, 0);
    ++seg;
    if (wq >= quads) return true;
    const int row = g * kRG + r;
    const bool live = row < p.rows;
    // a row that sees nothing of this piece has l = 0 and O = 0
    const float inv = l > 0.f ? p.out_mul / l : l;
    const float lse = l > 0.f ? (m + log2f(l) - kWeightShift) * 0.69314718055994530942f : l == 0.f ? -INFINITY : l;
    const int64_t orow = (int64_t)b * p.rows + row;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
#pragma unroll 1
    for (int c0 = 0; c0 < 256; c0 += 32) {
      uint32_t u[32];
      __syncwarp();
      tmem_ld32_sync(tO + c0, u);
      if (!live) continue;
      if (slot < 0) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * kDl + col0);
        uint32_t o[16];
#pragma unroll
        for (int v = 0; v < 16; ++v)
          o[v] = pack_bf16(__uint_as_float(u[2 * v]) * inv, __uint_as_float(u[2 * v + 1]) * inv);
        if (wide) {
          st_global_v8(dst + c0 / 2, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
          st_global_v8(dst + c0 / 2 + 8, o[8], o[9], o[10], o[11], o[12], o[13], o[14], o[15]);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            reinterpret_cast<uint4*>(dst + c0 / 2)[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        }
      } else {
        float* dst = p.part_o + kvq::part_index(slot, (col0 + c0) / 8, r);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          st_global_v8(dst + v * kRG * 8, __uint_as_float(u[8 * v + 0]) * inv, __uint_as_float(u[8 * v + 1]) * inv,
                       __uint_as_float(u[8 * v + 2]) * inv, __uint_as_float(u[8 * v + 3]) * inv,
                       __uint_as_float(u[8 * v + 4]) * inv, __uint_as_float(u[8 * v + 5]) * inv,
                       __uint_as_float(u[8 * v + 6]) * inv, __uint_as_float(u[8 * v + 7]) * inv);
      }
    }
    if (live && h == 0) {
      if (slot >= 0) p.part_lse[(int64_t)slot * kRG + r] = lse;
      else if (p.lse) p.lse[orow] = lse;
    }
    tc_fence_before();
    return true;
  });
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    kv8_rows_kernel(const Params p, const __grid_constant__ CUtensorMap cache, const __grid_constant__ QueryMaps queries) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5;
  const int cluster = blockIdx.x / 2;
  Ctl* c = reinterpret_cast<Ctl*>(smem + kOffCtl);
  grid_dep_wait();  // launched before the stream's last kernel has ended
  // Barriers, a few per warp.
  if ((threadIdx.x & 31) == 0) {
    if (warp < 4) {
      mbar_init(&c->full[warp], kProducerWarps);
      mbar_init(&c->empty[warp], 1);
      mbar_init(&c->m_ready[0][warp], 1);
      mbar_init(&c->m_ready[1][warp], 1);
      mbar_init(&c->q_ready[warp], kRowWarps);
      mbar_init(&c->piece_full[warp], 1);
      mbar_init(&c->piece_empty[warp], kFollowers + (rank == 0 ? 1 : 0));
    } else if (warp < 4 + kSBufs) {
      const int q = warp - 4;
      mbar_init(&c->s_full[q], 2);
      mbar_init(&c->s_free[q], kRowWarps / 2);
      mbar_init(&c->p_free[q], 1);
      mbar_init(&c->p_full[q], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&c->pv_done[h][q], 1);
        mbar_init(&c->o_ready[h][q], kRowWarps / 2);
      }
    } else if (warp < 4 + kSBufs + kPStages) {
      const int q = warp - 4 - kSBufs;
      mbar_init(&c->p_staged[q], kRowWarps / 2);
      mbar_init(&c->ps_free[q], 1);
    } else if (warp == 9) {
      for (int k = 0; k < 3; ++k) mbar_init(&c->q_in[k], 1);
      mbar_init(&c->q_max, kRowWarps);
      mbar_init(&c->fin_free, 32 * kRowWarps);
      mbar_init(&c->fin_full, 32 * kRowWarps);
      mbar_init(&c->drain, 1);
    } else if (warp == 11) {
      c->abort = 0;
      c->start_b = p.B;
      c->start_x = 0;
      c->start_T = 0;
      c->left = 0;
      c->wait_ns = p.wait_ns;
      c->err = (smem_u32(smem) & 1023u) ? MLA_DEVERR_LAYOUT : 0u;
    }
    fence_mbar_init();
  }
  static_assert(kStages == 4 && kPieces == 4 && kPBufs == kSBufs && 4 + kSBufs + kPStages <= 9, "barriers per warp");
  if (warp == kWarpAux) {
    tmem_alloc_cta(&c->tmem_base, kTmemCols);
    tmem_relinquish_cta();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // barriers initialised; the peer's are waited for after the split
  const int n = Work::make_split(p, c, cluster);  // the same n in every CTA
  const bool work = cluster < n;
  if (threadIdx.x == 0) {
    if (rank == 0) {
      Start* st = static_cast<Start*>(p.starts) + cluster;
      *st = Start{c->start_x, c->start_b, c->start_T, n > 0 ? n : 0, {0, 0, 0}};
    }
    if (blockIdx.x == 0) p.err[0] = gridDim.x;
  }
  cluster_wait();
  tc_fence_after();
  if (!work) {
    // both CTAs of the cluster leave here
    grid_dep_launch();
    if (threadIdx.x == 0) p.err[kErrFirst + blockIdx.x] = c->err;
    if (warp == kWarpAux) tmem_dealloc_cta(c->tmem_base, kTmemCols);
    return;
  }

  const bool base0 = c->tmem_base == 0;  // all columns are allocated
  if (!base0 && threadIdx.x == 0) c->err = MLA_DEVERR_LAYOUT;
  if (base0) {
    if (warp < kRowWarps) {
      if (rank == 0) score_softmax(p, queries, smem, c, warp);
      else value_rows(p, c);
    } else if (warp < kWarpProd + kProducerWarps) {
      if (rank == 0) producer<true>(p, cache, smem, c, warp - kWarpProd);
      else producer<false>(p, cache, smem, c, warp - kWarpProd);
    } else if (warp == kWarpMma) {
      if (rank == 0) score_mma(smem, c);
      else value_mma(p, smem, c);
    } else if (warp == kWarpAux) {
      if (rank == 0) weight_copier(p, smem, c);
    } else {
      Work::schedule(p, c, cluster);
    }
  }

  __syncwarp();
  grid_dep_launch();  // the merging kernel may start launching; it waits for this grid
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.err[kErrFirst + blockIdx.x] = c->err | (c->abort ? MLA_DEVERR_TIMEOUT : 0u);
  // after an abort nobody has waited for the last copies into shared memory: give
  // them far longer than they take
  if (c->abort) __nanosleep(100000);
  tc_fence_after();
  cluster_sync();  // no CTA leaves while its peer may still touch its shared memory
  if (warp == kWarpAux) tmem_dealloc_cta(c->tmem_base, kTmemCols);
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// As the few-rows kernel's: the pieces of a row group that several clusters shared,
//   lse = ln sum_k exp(lse_k),  out = sum_k exp(lse_k - lse) out_k.
// Partial results lie 8 columns of all rows after each other, so a warp takes 8 rows x
// 32 columns, a row and 8 columns per lane, and needs nothing of other warps; with few
// rows in many pieces four warps share that, every fourth piece each.  The partial
// results come from the second level cache; of the 9 us that it adds to 30 sequences of
// 4,096 to 8,192 tokens x 128 heads 2 are for the launch and 2.5 for the data.
constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32, kMergeParts = 4, kMergeRows = 8;
__global__ void __launch_bounds__(kMergeThreads, 2) kv8_rows_merge_kernel(const Params p) {
  __shared__ kvq::Cuts<kvq::kMaxClusters> c;
  __shared__ float sums[kMergeWarps][9][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int cuts = Work::list_cuts<kRG>(p, &c);
  const int octets = (min(p.rows, kRG) + kMergeRows - 1) / kMergeRows;
  const int tasks = cuts * octets * (kDl / 32);
  const bool split = tasks * kMergeParts <= (int)gridDim.x * kMergeWarps;
  const int at_once = split ? kMergeWarps / kMergeParts : kMergeWarps;
  const int part = split ? warp % kMergeParts : 0, step = split ? kMergeParts : 1;
  for (int t0 = blockIdx.x * at_once; t0 < tasks; t0 += gridDim.x * at_once) {
    const int task = t0 + (split ? warp / kMergeParts : warp);
    const int block8 = (task % (kDl / 32)) * 4 + (lane >> 3);
    const int oct = task / (kDl / 32);
    float acc[8], total = 0.f, m = -INFINITY;
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
    int64_t orow = -1;
    if (task < tasks) {
      const auto g = c.group[oct / octets];
      const int n = g.n, r = oct % octets * kMergeRows + (lane & 7);
      const bool live = r < g.rows;
      if (live) orow = g.row + r;
      constexpr int kDeep = 3;
      uint32_t v[kDeep][8];
      float e[kDeep];
      auto lse_of = [&](int i) {
        const int at = live && i < n ? c.slot_of(g, i) : -1;
        return at >= 0 ? __ldcg(p.part_lse + (int64_t)at * kRG + r) : -INFINITY;
      };
      auto load = [&](int i0) {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
          const int i = i0 + d * step, at = live && i < n ? c.slot_of(g, i) : -1;
#pragma unroll
          for (int q = 0; q < 8; ++q) v[d][q] = 0u;
          if (at >= 0) ld_global_v8(p.part_o + kvq::part_index(at, block8, r), v[d]);
          e[d] = lse_of(i);
        }
      };
      load(part);
      for (int i = lane >> 3; i < n; i += 4) m = fmaxf(m, lse_of(i));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if (m == -INFINITY) m = 0.f;  // no piece has any weight
      for (int i0 = part;;) {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
          const float f = __expf(e[d] - m);  // 0 for an empty piece
          total += f;
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] = fmaf(f, __uint_as_float(v[d][q]), acc[q]);
        }
        i0 += kDeep * step;
        if (i0 >= n) break;
        load(i0);
      }
    }
    if (split) {  // the same in every block
#pragma unroll
      for (int q = 0; q < 8; ++q) sums[warp][q][lane] = acc[q];
      sums[warp][8][lane] = total;
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int o = 1; o < kMergeParts; ++o) {
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] += sums[warp + o][q][lane];
          total += sums[warp + o][8][lane];
        }
      }
      __syncthreads();
    }
    if (orow >= 0 && part == 0) {
      const float inv = 1.f / (total == 0.f ? 1.f : total);  // then a row of zeros, as from one piece
      uint4 o;
      o.x = pack_bf16(acc[0] * inv, acc[1] * inv);
      o.y = pack_bf16(acc[2] * inv, acc[3] * inv);
      o.z = pack_bf16(acc[4] * inv, acc[5] * inv);
      o.w = pack_bf16(acc[6] * inv, acc[7] * inv);
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * kDl + 8 * block8) = o;
      if (p.lse && block8 == 0) p.lse[orow] = m + logf(total);
    }
  }
}

namespace {

bool query_map(CUtensorMap* m, const void* base, int64_t rows, int width, int box_rows) {
  const kvq::EncodeTiledFn f = kvq::encode_tiled();
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int clusters_per_gpu() {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static int cached[kMaxDevices] = {};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev] > 0) return cached[dev];
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaFuncSetAttribute(kv8_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemAlloc;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kv8_rows_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = sms / 2;
  }
  if (n > kvq::kMaxClusters) n = kvq::kMaxClusters;
  cached[dev] = n;
  return n;
}

mla_status launch(Params p, const CUtensorMap& cache, cudaStream_t s) {
  p.groups = (p.rows + kRG - 1) / kRG;
  p.box_rows = p.rows < kRG ? p.rows : kRG;
  // per call: the attribute belongs to the context, which may be a new one
  if (cudaFuncSetAttribute(kv8_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc) != cudaSuccess)
    return MLA_ERR_CUDA;
  QueryMaps maps;
  const int64_t rows = (int64_t)p.B * p.rows;
  if (!query_map(&maps.lat, p.q_lat, rows, kDl, p.box_rows) || !query_map(&maps.pe, p.q_pe, rows, kDr, p.box_rows))
    return MLA_ERR_CUDA;
  if (launch_kernel(kv8_rows_kernel, dim3(2 * p.clusters), dim3(kThreads), kSmemAlloc, s, true, p, cache, maps) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  if (p.clusters > 1 && launch_kernel(kv8_rows_merge_kernel, dim3(4 * p.clusters), dim3(kMergeThreads), 0, s, true,
                                      static_cast<const Params&>(p)) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

}  // namespace rows
}  // namespace kv8
}  // namespace mlav
