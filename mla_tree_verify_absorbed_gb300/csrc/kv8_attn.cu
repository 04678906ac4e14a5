// Verify attention and decoding over the paged 8-bit latent cache (mla_kv8_attn)
// on tcgen05 tensor cores.
//
// The work.  32 query rows ((node, head) pairs) against tiles of 128 tokens:
// S^T = K Q^T, online softmax, O^T += V^T P^T, V the latent part of K.  Tokens are
// the 128 lanes of the first product and latents those of the second, so that the
// cache's e4m3 codes, as they lie in shared memory, are the A operand of both: rows
// of tokens in the first (K-major), columns of latents in the second (MN-major).
// Nothing is converted, every byte is fetched once, and one CTA does all of it.
//
// The other operands are made of several 8-bit terms, each in columns of its own, whose
// products are added in fp32: queries' as the scores are read, weights' when O is.
//   queries  q 2^t = hi + lo, both e4m3, t per row.  bf16 has 8 significant bits and a
//            term 4, so the sum is exact down to 2^-9 of the row's largest element;
//   weights  w = t1 + 2^-3 t2 + 2^-6 t3 of w rounded to f16, all e5m2.  An e5m2 number
//            is the upper byte of an f16 one: t1 and t2 are the upper bytes of w and of 2^3
//            times what is left, t3 2^3 times what is left then, rounded.  3 + 3 + 3
//            significant bits, off by at most 2^-9, as bf16, or by 2^-23 where that is more.
// The rope product (bf16) is accumulated on the queries' terms, half on each.
//
// Blocks' scales.  A token's score is s_j = c_r 2^k_j S_jr (c_r: scale, row unit),
// and its value 2^k_j times its codes, so O takes the weights 2^(s_j + k_j - m): m
// follows the largest s_j + k_j, a weight's size says what the token can add to the
// output, and the sum for the normaliser takes 2^-k_j off again.
//
// m follows the tiles, up and down.  Weights end at 2^-23, so behind a token that towers
// over all others a running maximum would leave nothing of theirs, though the sum counts
// them: O, in fp32, has room for both.  So m falls where a tile's largest weight T of a
// row is below 2^F, F = log2 n + d - 14 for n tokens whose k_j differ by d at most.  Beside
// their 9 bits, they are then off by 2^-23 each (and 2^-25 from f16), as softmax weights by
// n 2^-22.6 2^d / T <= 2^-8.6 of the tile's largest together.  It falls by whole numbers, so
// that O and the sums move exactly, and rises to the largest itself, whose weight is then a
// power of two and exact: with whole numbers there too, rows of which one token has the
// most were off twice as much.
//
// What bounds it.  HBM where at most 32 rows share a token: 128 ragged sequences of up
// to 16,384 tokens x 16 heads read their 280 MB in 69.0 us, 4.1 TB/s; the CTAs' loops run at
// about 90% of the measured copy rate, the rest is their start (7 us: the split, the queries,
// the first tiles), the output (2 us) and the merge (5 us).  With two row groups to a
// sequence (16 sequences of 100,000 in windows of 4,096 x 64 heads: 34.6 us) that fixed
// part, and shared memory: a tile's S takes 1,260 cycles and its O 1,200, not the 640 and
// 768 of the tensor pipe, since both read their A operand, the 64 or 80 KB of the tile.
//
// Shared memory: two stages of 80 KB (128 tokens x 640 bytes; a tile's weights take
// the place of its rope keys) and 40 KB of queries.  Tensor Memory: O 4 x 96 columns
// (latent block; row half, term, row), two S tiles of 64 columns (row half, term, row).
//
// Work split as in split.cuh; pieces of a row group are merged by a second kernel.
//
// Masks are applied to scores by selection.  Positions that no node sees are
// filled with zeros in place of being read, so that whatever lies in the pool under
// a weight of zero is finite.
//
// Every wait is bounded (2 s, less in the self-test); on timeout the roles stop,
// drain what they issued, free their Tensor Memory and report MLA_DEVERR_TIMEOUT.
#include <cuda.h>
#include <cuda_fp8.h>

#include <cmath>
#include <cstddef>
#include <mutex>

#include "kv8.cuh"
#include "sm100.cuh"
#include "split.cuh"
#include "tensor_map.cuh"

namespace mlav {
namespace kv8 {
using namespace sm100;
using kvq::for_pieces;
using kvq::kErrFirst;
using kvq::kErrMax;
using kvq::kPieces;
using kvq::NodeView;
using kvq::Piece;
using kvq::Start;

constexpr int kRG = 32;        // query rows per work item
constexpr int kHalfRows = 16;  // rows of a group of row warps
constexpr int kTK = 128;       // tokens per tile
// Warps 0-7 hold scores (warp w: tokens 32 (w % 4) .., rows 16 (w / 4) ..), 8-11
// fetch, 12 issues the products, 13 hands out the pieces of work.
constexpr int kRowWarps = 8, kProducerWarps = 4;
constexpr int kWarpProd = kRowWarps, kWarpMma = kWarpProd + kProducerWarps, kWarpSched = kWarpMma + 1;
constexpr int kThreads = 32 * (kWarpSched + 1);
constexpr uint32_t kTmemCols = 512;

// A piece costs kFixed tiles beside its own.  The mean of 11 sizes (decode of 40 to 200
// ragged sequences x 16 to 64 heads, windows) took, against 3: 2 2.1% more, 4 1.4%, 5 3.5%.
constexpr int kFixed = 3;
constexpr int kMinTiles = 2;
using Work = kvq::Split<kTK, kFixed, kMinTiles, kThreads, true>;

constexpr int kChunk = kTK * 128;              // 128 bytes of each token: 128 latents, or the rope key
constexpr int kChunks = MLA_KV8_ROW_BYTES / 128;
constexpr int kStage = kChunks * kChunk;       // 80 KB
constexpr int kStages = 2;
constexpr int kQRows = 2 * kRG;                // (row half, term, row)
constexpr int kQChunk = kQRows * 128;          // 8 KB
constexpr int kOffQ = kStages * kStage;
constexpr int kOffCtl = kOffQ + kChunks * kQChunk;
// A tile's weights, a row of 128 bytes per token of which 96 are used, take the
// place of its rope keys, which only its S product reads.
constexpr int kOffP = 4 * kChunk;

// Tensor Memory columns
constexpr uint32_t kColO = 0, kBlockO = 3 * kRG;  // a block of 128 latents
constexpr uint32_t kColS = 4 * kBlockO;
static_assert(kColS + 2 * kQRows <= kTmemCols, "Tensor Memory columns");

// operand descriptors (smem_desc): all have 128-byte rows in groups of 8, 1 KB apart
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (kLayoutSw128 << 29);
constexpr uint32_t kDescLo = ((uint32_t)kChunk >> 4) << 16;  // no operand reaches beyond one row of 128 bytes
__device__ __forceinline__ uint64_t desc_at(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
  return d;
}
__device__ __forceinline__ uint32_t desc_lo(const uint8_t* smem, uint32_t off) {
  return (((smem_u32(smem) & 0x3FFFFu) + off) >> 4) | kDescLo;
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 20000000ull;

// Weights are 2^(s + k - m + kWeightShift), at most 2^kTop, below e5m2's 57,344.  Moving m
// costs a pass over a row of O (with 2^2 in place of 2^8 to go, every second tile of 64
// nodes x 64 heads x 20,000 tokens moved one of its 16), so it is lazy: the largest weight
// of a piece's first tile is put at 2^kWeightShift, one that is too large, and thus rare,
// at 2^kRisen, a tile whose weights are too small 2^kFallen above the least.
constexpr float kTop = 15.f, kWeightShift = 7.f, kRisen = 14.f, kFallen = 8.f;
constexpr int kLossLog2 = 14;
// m stays within 2^kDeepest of the largest so far: O and the sums stay far from fp32's
// limits, and what is lost is below 2^-70 of the largest weight.
constexpr float kDeepest = 40.f;
constexpr uint32_t kTermMul = 0x48004800u;  // 2^3 in f16, twice
constexpr float kTermInv = 0.125f;

struct alignas(16) Ctl {
  uint64_t full[kStages];      // tile landed (each producer warp's copies)
  uint64_t empty[kStages];     // the products that read it are complete
  uint64_t s_full[2];          // S tile in Tensor Memory
  uint64_t q_ready;            // a piece's queries, row constants and masks written (8 row warps)
  uint64_t m_ready[2];         // a tile's votes or partial maxima written (4 row warps of a half)
  uint64_t l_ready[2];         // a piece's partial sums written (the same)
  uint64_t p_ready[2];         // weights in, O rescaled (8 row warps)
  uint64_t pv_done[2];         // a tile's O product complete
  uint64_t drain;
  uint64_t piece_full[kPieces];   // piece written (scheduler warp)
  uint64_t piece_empty[kPieces];  // read by every warp that follows the pieces
  Piece piece[kPieces];
  alignas(16) uint32_t vote[2][2][4];    // parity of the exchange, half, token quadrant
  alignas(16) uint32_t k_range[kStages][kProducerWarps];  // of 32 tokens: largest k, and 15 - the least above it
  float part_max[2][2][4][kHalfRows];    // the same, and row
  float part_sum[2][4][kHalfRows];
  alignas(16) float unit[kRG]; // c_r: score factor of a row
  uint64_t mask[kRG];          // what the row's node sees of the tree,
  int depth[kRG];              // and its depth
  float shift[kRowWarps][kHalfRows];  // each row warp's copy of Rows::shift, a row to a lane
  int tok_k[kStages][kTK];     // k of the tokens' blocks
  int64_t scan[kThreads / 32];
  int64_t left;                // units of this CTA's interval
  int64_t start_x;             // its first unit within sequence start_b
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
constexpr int kFollowers = kRowWarps + kProducerWarps + 1;

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Ctl* c) {
  if (mbar_wait(bar, parity, &c->abort, c->wait_ns)) return true;
  c->abort = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* c) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, c);
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
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t sub_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t push_sign(uint32_t bits, float x) {  // into the lowest bit
  return __funnelshift_l(__float_as_uint(x), bits, 1);
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
// Warp pw fetches tokens 32 pw .. of every tile: each lane looks up a token, a tile
// ahead.  Where pages hold a multiple of 16 tokens and the tile is seen whole, the rows
// of 16 or 32 tokens come by one tensor copy per chunk (128 bytes of a row), else row by
// row by cp.async, eight lanes to 128 bytes, zeros for positions that no node sees.
// Small copies cost the copy engine more than their bytes: 8 ragged sequences x 32 nodes
// x 64 heads in the kernel for many rows take 173 us in pages of 64, 181 of 16, and of 8
// 206 by cp.async and 222 by copies of 8 rows; here, where HBM bounds both, 128 ragged
// sequences x 16 heads in pages of 8 take 69 us either way.  (Gathers of four rows take
// the engine 30 cycles each, 17 bytes per cycle: with them for two of the five chunks
// the same took a quarter longer.)
__device__ void producer(const Params& p, const CUtensorMap& map, uint8_t* smem, Ctl* c, int pw) {
  const int lane = threadIdx.x & 31;
  uint32_t err = 0, j = 0;
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
    auto word_of = [&](int32_t slot) { return slot >= 0 ? (uint32_t)__ldg(p.scales + p.block((uint32_t)slot)) : 0u; };
    int32_t slot = slot_of(entry_of(pc.t0), pc.t0), ent = entry_of(pc.t0 + 1);
    uint32_t word = word_of(slot);
#pragma unroll 1
    for (int v = pc.t0; v < pc.t1; ++v, ++j) {
      const int32_t next = slot_of(ent, v + 1);
      const uint32_t next_word = word_of(next);
      ent = entry_of(v + 2);
      const uint32_t st = j % kStages, par = ((j / kStages) & 1u) ^ 1u;
      uint8_t* to = smem + st * kStage + 32 * pw * 128;
      const uint32_t dst = smem_u32(to);
      const bool boxes = p.box > 0 && __all_sync(0xffffffffu, seen(v, pos_of(v)));
      if (!wait_warp(&c->empty[st], par, c)) return false;
      uint64_t* full = &c->full[st];
      const int k = scale_of(word);
      const uint32_t range = __reduce_max_sync(0xffffffffu, slot >= 0 ? k : 0) |
                             __reduce_max_sync(0xffffffffu, slot >= 0 ? kMaxK - k : 0) << 16;
      c->tok_k[st][32 * pw + lane] = k;
      if (lane == 0) c->k_range[st][pw] = range;
      __syncwarp();
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

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// One warp, which issues what can be issued next: the O product of a tile when its
// weights are there, else the next S product when its tile is.  (S chunk by chunk as
// they land, and O freeing them one by one, took longer: each test and each branch
// into the issuing lane costs some 300 cycles.)
__device__ void products(const Params& p, uint8_t* smem, Ctl* c) {
  const bool leader = elect_one();
  if (p.hold && !wait_warp(&c->drain, 0u, c)) return;
  uint32_t j = 0, seg = 0;
  const uint32_t q_lo = desc_lo(smem, kOffQ);
  for_pieces(c, [&](const Piece& pc) {
    if (!wait_warp(&c->q_ready, seg & 1u, c)) return false;
    ++seg;
    const int halves = p.rows - pc.g * kRG > kHalfRows ? 2 : 1;
    const uint32_t is8 = idesc_e4m3_f32(kTK, 32 * halves, 0, 0), is16 = idesc_bf16_f32(kTK, 32 * halves, 0, 0);
    const uint32_t io = idesc_e4m3_e5m2_f32(128, 48 * halves, 1, 1);
    const uint32_t end = j + (uint32_t)(pc.t1 - pc.t0), first = j;
    uint32_t s = j;  // the next S product
    auto test = [&](uint64_t* bar, uint32_t n) {  // tile n's phase of a barrier that every second tile uses
      return __all_sync(0xffffffffu, mbar_test_wait(bar, (n >> 1) & 1u));
    };
    uint64_t t0 = 0;
    uint32_t polls = 0;
    while (j < end) {
      if (s > j && test(&c->p_ready[j & 1u], j)) {
        const uint32_t st = j % kStages;
        tc_fence_after();
        if (leader) {
          const uint32_t a = desc_lo(smem, st * kStage);
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk) {  // 32 tokens
#pragma unroll
            for (uint32_t m = 0; m < 4; ++m)
              mma_cta_ss_f8(kColO + m * kBlockO, desc_at(a + ((m * kChunk + kk * 32 * 128) >> 4)),
                            desc_at(a + ((kOffP + kk * 32 * 128) >> 4)), io, (j - first) | kk);
          }
          mma_cta_commit(&c->empty[st]);
          mma_cta_commit(&c->pv_done[st]);
        }
        __syncwarp();
        ++j;
        polls = 0;
        continue;
      }
      // The S tile before the last has been read when its weights are there.
      if (s < end && s <= j + 1 && test(&c->full[s % kStages], s)) {
        tc_fence_after();
        fence_proxy_async_smem();  // the tile may have come by cp.async, without a fence of its writers
        if (leader) {
          const uint32_t d = kColS + (s & 1u) * kQRows, a = desc_lo(smem, (s % kStages) * kStage);
#pragma unroll
          for (uint32_t ck = 0; ck < 4; ++ck) {
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
              mma_cta_ss_f8(d, desc_at(a + ((ck * kChunk + kk * 32) >> 4)), desc_at(q_lo + ((ck * kQChunk + kk * 32) >> 4)),
                            is8, ck | kk);
          }
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk)
            mma_cta_ss(d, desc_at(a + ((4 * kChunk + kk * 32) >> 4)), desc_at(q_lo + ((4 * kQChunk + kk * 32) >> 4)),
                       is16, 1);
          mma_cta_commit(&c->s_full[s & 1u]);
        }
        __syncwarp();
        ++s;
        polls = 0;
        continue;
      }
      if (++polls & 63u) continue;
      const uint64_t now = globaltimer_ns();
      if (polls == 64u) t0 = now;
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&c->abort) || now - t0 > c->wait_ns)) {
        c->abort = 1;
        return false;
      }
    }
    return true;
  });
  __syncwarp();
  // on abort, outstanding MMAs must finish before Tensor Memory is released
  if (!__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&c->abort) != 0)) return;
  if (leader && !p.hold) {
    mma_cta_commit(&c->drain);
    mbar_wait_drain(&c->drain, 0, kDrainLimitNs);
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// softmax and output
// ---------------------------------------------------------------------------
// Brings a piece's queries into shared memory as two e4m3 terms, a row to a warp, two
// of a warp's rows in flight.  Rows that do not exist, up to the end of a half, are zeros.
__device__ __forceinline__ void stage_queries(const Params& p, uint8_t* smem, Ctl* c, const Piece& pc, int warp) {
  const int lane = threadIdx.x & 31;
  const int rows = min(kRG, p.rows - pc.g * kRG), padded = rows > kHalfRows ? kRG : kHalfRows;
#pragma unroll 1
  for (int r0 = warp; r0 < padded; r0 += 2 * kRowWarps) {
    uint4 all[2][2] = {};
    uint32_t rope_all[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + kRowWarps * i;
      if (r < rows) {
        const int64_t row = (int64_t)pc.b * p.rows + pc.g * kRG + r;
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q_lat) + row * (2 * kDl)) + 2 * lane;
        all[i][0] = __ldg(q);
        all[i][1] = __ldg(q + 1);
        rope_all[i] = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.q_pe) + row * (2 * kDr)) + lane);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + kRowWarps * i;
      const uint4 a = all[i][0], b = all[i][1];
      const uint32_t pe = rope_all[i], w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t big = max(pe & 0x7fffu, (pe >> 16) & 0x7fffu);  // magnitudes compare as their bits
#pragma unroll
      for (int q = 0; q < 8; ++q) big = max(big, max(w[q] & 0x7fffu, (w[q] >> 16) & 0x7fffu));
      big = __reduce_max_sync(0xffffffffu, big);
      const bool finite = big < 0x7f80u;
      const int t = query_unit(big);
      const float mul = pow2(t);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) query_terms(w[2 * q], w[2 * q + 1], mul, finite, hi[q], lo[q]);
      // the rope query by halves on both terms: zeros on one of them would make NaN of infinite rope keys
      const float half = 0.5f * mul;
      const __nv_bfloat162 pm =
          __floats2bfloat162_rn(__uint_as_float(pe << 16) * half, __uint_as_float(pe & 0xffff0000u) * half);
      const int n = 32 * (r >> 4) + (r & 15);
      const uint32_t q0 = smem_u32(smem) + kOffQ;
      const uint32_t at = q0 + (lane >> 3) * kQChunk + n * 128 + (((lane & 7) ^ (n & 7)) << 4);
      st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(at + 16 * 128, lo[0], lo[1], lo[2], lo[3]);  // 16 rows on: the same swizzle
      const uint32_t rope = 4 * kQChunk + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) + 4 * (lane & 3);
      *reinterpret_cast<uint32_t*>(smem + kOffQ + rope) = *reinterpret_cast<const uint32_t*>(&pm);
      *reinterpret_cast<uint32_t*>(smem + kOffQ + rope + 16 * 128) = *reinterpret_cast<const uint32_t*>(&pm);
      if (lane == 0) c->unit[r] = query_factor(p.scale_log2, t);
    }
  }
}

// Multiplies a row's columns of O, in the warp's lanes, by a factor.
__device__ __forceinline__ void rescale_row(uint32_t tO, float a) {
  uint32_t u[12];
#pragma unroll
  for (int q = 0; q < 12; ++q)  // block, term
    tmem_ld1(tO + (q / 3) * kBlockO + (q % 3) * kHalfRows, u[q]);
  tmem_wait_ld(u);
#pragma unroll
  for (int q = 0; q < 12; ++q)
    tmem_st1(tO + (q / 3) * kBlockO + (q % 3) * kHalfRows, __float_as_uint(__uint_as_float(u[q]) * a));
  tmem_wait_st();
}

// One piece's state of a row warp: per row, two by two, 2^(score + k) is weighted
// by 2^shift, shift = kWeightShift - m; sum of the weights.
struct Rows {
  uint64_t shift[kHalfRows / 2], sum[kHalfRows / 2];
};
constexpr float kNone = 3.402823466e38f;  // shift before the first score: any score beats that m

__device__ void softmax(const Params& p, uint8_t* smem, Ctl* c, int warp) {
  const int lane = threadIdx.x & 31;
  const int quad = warp & 3, half = warp >> 2;
  const int token = 32 * quad + lane;
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  const uint32_t tO = lane_off + kColO + half * 3 * kHalfRows;
  const uint32_t tP = smem_u32(smem) + kOffP + token * 128;
  uint32_t j = 0, seg = 0;
  uint32_t i = 0;  // exchanges among the half's warps
  bool bad = false;
  auto exchange = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->m_ready[half]);
  };
  for_pieces(c, [&](const Piece& pc) {
    const int rows = min(kRG, p.rows - pc.g * kRG);
    const int P = pc.P;
    // This warp has seen the end of every S product of the piece before, and with
    // the end of its last O product that no warp needs its masks any more.
    stage_queries(p, smem, c, pc, warp);
    if (warp == 0) {
      const NodeView nv = kvq::node_view_warp(p, pc.b, (pc.g * kRG + min(lane, rows - 1)) / p.H, P, &bad);
      c->mask[lane] = nv.mask;
      c->depth[lane] = nv.depth;
    }
    fence_proxy_async_smem();  // read by the MMA
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->q_ready);
    if (!wait_warp(&c->q_ready, seg & 1u, c)) return false;
    const bool idle = kHalfRows * half >= rows;
    // positions up to this one are outside some node's window
    const int past_any = p.window > 0 ? max(P - p.window + p.Q - 1, -1) : -1;
    Rows R;
#pragma unroll
    for (int r = 0; r < kHalfRows / 2; ++r) {
      R.shift[r] = pair(kNone, kNone);
      R.sum[r] = 0;
    }
    if (lane < kHalfRows) c->shift[warp][lane] = kNone;
    float best = -INFINITY;  // a row to a lane, twice: its largest score + k when m last moved
#pragma unroll 1
    for (int t = pc.t0; t < pc.t1; ++t, ++j) {
      const uint32_t st = j % kStages, par = (j >> 1) & 1u;
      if (!wait_warp(&c->s_full[j & 1u], par, c)) return false;
      if (idle) {
        // every barrier's phases count on
        if (lane == 0) mbar_arrive(&c->p_ready[j & 1u]);
        continue;
      }
      if (!wait_warp(&c->full[st], par, c)) return false;  // has passed: the producers' scales are visible
      tc_fence_after();
      const int k = c->tok_k[st][token];
      const uint64_t k2 = pair((float)k, (float)k), mul2 = pair(pow2(k), pow2(k)), inv2 = pair(pow2(-k), pow2(-k));
      uint64_t y[kHalfRows / 2];  // score + k, base 2
      {
        uint32_t u[32];
        tmem_ld32_sync(lane_off + kColS + (j & 1u) * kQRows + 32 * half, u);
        const ulonglong2* unit = reinterpret_cast<const ulonglong2*>(c->unit + kHalfRows * half);
#pragma unroll
        for (int q = 0; q < kHalfRows / 4; ++q) {
          const ulonglong2 f = unit[q];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 2 * q + h;
            const uint64_t v = add_f32x2(pair(u[2 * r], u[2 * r + 1]), pair(u[16 + 2 * r], u[17 + 2 * r]));
            y[r] = fma_f32x2(mul_f32x2(v, mul2), h ? f.y : f.x, k2);
          }
        }
      }
      const int pos0 = pc.tile(t) * kTK;
      if (pos0 > P - kTK || pos0 <= past_any) {
        const int pos = pos0 + token, rel = pos - P;
#pragma unroll
        for (int r = 0; r < kHalfRows / 2; ++r) {
          bool see[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int rr = kHalfRows * half + 2 * r + h;
            if (rel >= 0) see[h] = rel < 64 && ((c->mask[rr] >> rel) & 1u);
            else see[h] = p.window == 0 || pos < p.sinks || pos > P - p.window + c->depth[rr];
          }
          y[r] = pair(see[0] ? lo_f32(y[r]) : -INFINITY, see[1] ? hi_f32(y[r]) : -INFINITY);
        }
      }
      // m moves only when the tile's weights are too large or too small, for the four
      // warps of the half together; until they have all voted the weights are taken with
      // m as it is.  A vote: bit 16, no weight is too large; bits 0-15, a row whose weights
      // are all too small (or that sees none of the tile).
      uint32_t hi[4] = {}, lo[4] = {}, third[4] = {};
      uint64_t x[kHalfRows / 2] = {}, sum[kHalfRows / 2];
      auto weigh = [&](int q) {  // two rows' weights, and their three terms
        const float e0 = ex2_approx(lo_f32(x[q])), e1 = ex2_approx(hi_f32(x[q]));
        sum[q] = fma_f32x2(pair(e0, e1), inv2, R.sum[q]);
        const uint32_t w = pack_f16(e0, e1);
        const uint32_t r1 = kvq::hmul2_f16(sub_f16(w, w & 0xff00ff00u), kTermMul);  // exact
        const uint32_t r2 = kvq::hmul2_f16(sub_f16(r1, r1 & 0xff00ff00u), kTermMul) + 0x00800080u;  // exact, then rounded at the upper byte
        const uint32_t place = q & 1 ? 0x7510u : 0x3275u;  // upper bytes into the pair's half of the word
        hi[q >> 1] = __byte_perm(hi[q >> 1], w, place);
        lo[q >> 1] = __byte_perm(lo[q >> 1], r1, place);
        third[q >> 1] = __byte_perm(third[q >> 1], r2, place);
      };
      const uint4 ranges = *reinterpret_cast<const uint4*>(c->k_range[st]);
      const uint32_t range = __vmaxu2(__vmaxu2(ranges.x, ranges.y), __vmaxu2(ranges.z, ranges.w));
      const int d = max((int)(range & 0xffffu) + (int)(range >> 16) - kMaxK, 0);
      const float least = (float)(32 - __clz(min(pc.N - pos0, kTK) - 1) + d - kLossLog2);  // F
      uint32_t moved = 0xffffffffu;  // rows; in a piece's first tile all, from no m at all
      bool move = t == pc.t0;
      if (!move) {
        const uint64_t least2 = pair(-least, -least);
        float top = -INFINITY;
        uint32_t small = 0;
#pragma unroll
        for (int r = 0; r < kHalfRows / 2; ++r) {
          x[r] = add_f32x2(y[r], R.shift[r]);
          top = fmaxf(top, fmaxf(lo_f32(x[r]), hi_f32(x[r])));
          const uint64_t above = add_f32x2(x[r], least2);
          small = push_sign(push_sign(small, lo_f32(above)), hi_f32(above));
        }
        const uint32_t mine = __reduce_and_sync(0xffffffffu, small | (top > kTop ? 0u : 1u << kHalfRows));
        if (lane == 0) c->vote[i & 1u][half][quad] = mine;
        exchange();
#pragma unroll
        for (int q = 0; q < kHalfRows / 2; ++q) weigh(q);
        if (!wait_warp(&c->m_ready[half], i & 1u, c)) return false;
        const uint4 vote = *reinterpret_cast<const uint4*>(c->vote[i & 1u][half]);
        ++i;
        move = (vote.x & vote.y & vote.z & vote.w) != 1u << kHalfRows;
      }
      if (move) {
        // the tile's maxima: of the warp's tokens, then of the half's four warps; a row to a lane
        float2* pm = reinterpret_cast<float2*>(c->part_max[i & 1u][half][quad]);
#pragma unroll
        for (int r = 0; r < kHalfRows / 2; ++r) {
          const float2 v = make_float2(warp_max(lo_f32(y[r])), warp_max(hi_f32(y[r])));
          if (lane == 0) pm[r] = v;
        }
        exchange();
        if (!wait_warp(&c->m_ready[half], i & 1u, c)) return false;
        const int r = lane % kHalfRows;
        const float (&m4)[4][kHalfRows] = c->part_max[i & 1u][half];
        const float m = fmaxf(fmaxf(m4[0][r], m4[1][r]), fmaxf(m4[2][r], m4[3][r])), was = c->shift[warp][r];
        ++i;
        best = fmaxf(best, m);
        const float largest = m + was;
        float now = was;
        if (largest > kTop)
          now = (was == kNone ? kWeightShift : kRisen) - m;
        else if (m > -INFINITY && largest <= least)
          now += floorf(fminf(fminf(least + kFallen, kTop) - largest, kWeightShift + kDeepest - best - was));
        const bool moves = now != was;
        const float a = moves ? (was == kNone ? 0.f : exp2f(now - was)) : 1.f;
        __syncwarp();
        c->shift[warp][r] = now;
        moved = __ballot_sync(0xffffffffu, moves) & ((1u << kHalfRows) - 1u);
        if (t > pc.t0) {
          if (!wait_warp(&c->pv_done[(j - 1) & 1u], ((j - 1) >> 1) & 1u, c)) return false;
          tc_fence_after();
          for (uint32_t left = moved; left; left &= left - 1) {
            const int q = __ffs(left) - 1;
            rescale_row(tO + q, __shfl_sync(0xffffffffu, a, q));
          }
        } else {
          moved = (1u << kHalfRows) - 1u;  // no weights yet
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kHalfRows / 2; ++q) {
          if (!((moved >> (2 * q)) & 3u)) continue;
          R.shift[q] = reinterpret_cast<const uint64_t*>(c->shift[warp])[q];
          R.sum[q] = mul_f32x2(R.sum[q], pair(__shfl_sync(0xffffffffu, a, 2 * q), __shfl_sync(0xffffffffu, a, 2 * q + 1)));
          x[q] = add_f32x2(y[q], R.shift[q]);
          weigh(q);
        }
      }
#pragma unroll
      for (int r = 0; r < kHalfRows / 2; ++r) R.sum[r] = sum[r];
      const uint32_t at = tP + st * kStage;
      st_shared_v4(at + (((3 * half) ^ (token & 7)) << 4), hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(at + (((3 * half + 1) ^ (token & 7)) << 4), lo[0], lo[1], lo[2], lo[3]);
      st_shared_v4(at + (((3 * half + 2) ^ (token & 7)) << 4), third[0], third[1], third[2], third[3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->p_ready[j & 1u]);
    }

    // The piece's sums over all tokens, then O: the warp's lanes hold latents
    // 32 quad + lane of each block of 128.
    const uint32_t phase = seg & 1u;
    ++seg;
    float l[kHalfRows];
#pragma unroll
    for (int r = 0; r < kHalfRows; ++r) l[r] = r & 1 ? hi_f32(R.sum[r >> 1]) : lo_f32(R.sum[r >> 1]);
    if (!idle) {
#pragma unroll
      for (int r = 0; r < kHalfRows; ++r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        if (lane == 0) c->part_sum[half][quad][r] = l[r];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->l_ready[half]);
      if (!wait_warp(&c->l_ready[half], phase, c)) return false;
    } else if (lane == 0) {
      mbar_arrive(&c->l_ready[half]);
    }
    if (!wait_warp(&c->pv_done[(j - 1) & 1u], ((j - 1) >> 1) & 1u, c)) return false;
    if (idle) return true;
    tc_fence_after();
    float inv[kHalfRows];
#pragma unroll
    for (int r = 0; r < kHalfRows; ++r) {
      const float (&s)[4][kHalfRows] = c->part_sum[half];
      l[r] = (s[0][r] + s[1][r]) + (s[2][r] + s[3][r]);
      inv[r] = l[r] > 0.f ? p.out_mul / l[r] : l[r];  // a row that sees nothing of this piece has l = 0 and O = 0
    }
    const int row0 = pc.g * kRG + kHalfRows * half, live = min(kHalfRows, p.rows - row0);
    const int64_t orow = (int64_t)pc.b * p.rows + row0;
    const int latent = 32 * quad + lane;
#pragma unroll 1
    for (int mb = 0; mb < 4; ++mb) {
      uint32_t u[16], v[16], w[16];
      __syncwarp();
      tmem_ld16_sync(tO + mb * kBlockO, u);
      tmem_ld16_sync(tO + mb * kBlockO + kHalfRows, v);
      tmem_ld16_sync(tO + mb * kBlockO + 2 * kHalfRows, w);
#pragma unroll
      for (int r = 0; r < kHalfRows; ++r) {
        const float lo = fmaf(__uint_as_float(w[r]), kTermInv, __uint_as_float(v[r]));
        const float o = fmaf(lo, kTermInv, __uint_as_float(u[r])) * inv[r];
        if (r < live) {
          if (pc.slot < 0)
            static_cast<__nv_bfloat16*>(p.out)[(orow + r) * kDl + 128 * mb + latent] = __float2bfloat16_rn(o);
          else
            p.part_o[((int64_t)pc.slot * kRG + kHalfRows * half + r) * kDl + 128 * mb + latent] = o;
        }
      }
    }
    if (quad == 0 && lane < live) {
      float ml = 0.f, ll = 0.f;
#pragma unroll
      for (int r = 0; r < kHalfRows; ++r)
        if (lane == r) {
          ml = kWeightShift - (r & 1 ? hi_f32(R.shift[r >> 1]) : lo_f32(R.shift[r >> 1]));
          ll = l[r];
        }
      const float lse =
          ll > 0.f ? (ml + log2f(ll) - kWeightShift) * 0.69314718055994530942f : ll == 0.f ? -INFINITY : ll;
      if (pc.slot >= 0) p.part_lse[(int64_t)pc.slot * kRG + kHalfRows * half + lane] = lse;
      else if (p.lse) p.lse[orow + lane] = lse;
    }
    tc_fence_before();
    return true;
  });
  if (bad) atomicOr(&c->err, MLA_DEVERR_PARENT);
}

__global__ void __launch_bounds__(kThreads, 1) kv8_attn_kernel(const Params p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  Ctl* c = reinterpret_cast<Ctl*>(smem + kOffCtl);
  grid_dep_wait();  // launched before the stream's last kernel has ended
  if (threadIdx.x == 0) {
    for (int q = 0; q < kStages; ++q) {
      mbar_init(&c->full[q], kProducerWarps);
      mbar_init(&c->empty[q], 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&c->s_full[q], 1);
      mbar_init(&c->p_ready[q], kRowWarps);
      mbar_init(&c->pv_done[q], 1);
      mbar_init(&c->m_ready[q], 4);
      mbar_init(&c->l_ready[q], 4);
    }
    mbar_init(&c->q_ready, kRowWarps);
    mbar_init(&c->drain, 1);
    for (int q = 0; q < kPieces; ++q) {
      mbar_init(&c->piece_full[q], 1);
      mbar_init(&c->piece_empty[q], kFollowers);
    }
    c->abort = 0;
    c->start_b = p.B;
    c->start_x = 0;
    c->start_T = 0;
    c->left = 0;
    c->wait_ns = p.wait_ns;
    c->err = (smem_u32(smem) & 1023u) ? MLA_DEVERR_LAYOUT : 0u;
    fence_mbar_init();
  }
  if (warp == kWarpSched) {
    tmem_alloc_cta(&c->tmem_base, kTmemCols);
    tmem_relinquish_cta();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int worker = blockIdx.x;
  const int n = Work::make_split(p, c, worker);  // the same n in every CTA
  if (threadIdx.x == 0) {
    static_cast<Start*>(p.starts)[worker] = Start{c->start_x, c->start_b, c->start_T, n > 0 ? n : 0, {0, 0, 0}};
    if (worker == 0) p.err[0] = gridDim.x;
    if (c->tmem_base != 0) c->err = MLA_DEVERR_LAYOUT;  // all columns are allocated
  }
  if (worker < n && c->tmem_base == 0) {
    if (warp < kRowWarps) softmax(p, smem, c, warp);
    else if (warp < kWarpMma) producer(p, map, smem, c, warp - kWarpProd);
    else if (warp == kWarpMma) products(p, smem, c);
    else Work::schedule(p, c, worker);
  }
  __syncwarp();
  grid_dep_launch();  // the merging kernel may start launching; it waits for this grid
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.err[kErrFirst + worker] = c->err | (c->abort ? MLA_DEVERR_TIMEOUT : 0u);
  // after an abort nobody has waited for the last copies into shared memory: give
  // them far longer than they take
  if (c->abort) __nanosleep(100000);
  tc_fence_after();
  if (warp == kWarpSched) tmem_dealloc_cta(c->tmem_base, kTmemCols);
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// The pieces of a row group that several CTAs shared:
//   lse = ln sum_k exp(lse_k),  out = sum_k exp(lse_k - lse) out_k.
// Every block reads where the CTAs' intervals begin and lists the row groups that a
// boundary cuts.  A warp takes a quarter of the columns of a row; with few rows in many
// pieces four warps share that, every fourth piece each.
constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32, kMergeParts = 4;
constexpr int kMaxWorkers = 256;
static_assert(kMaxWorkers <= kErrMax && kMaxWorkers <= kMergeThreads, "an error word per CTA");
__global__ void __launch_bounds__(kMergeThreads, 2) kv8_merge_kernel(const Params p) {
  __shared__ kvq::Cuts<kMaxWorkers> c;
  __shared__ float weight[kMergeWarps][kMaxWorkers];
  __shared__ float4 sums[kMergeWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int cuts = Work::list_cuts<kRG>(p, &c);
  // A task is a quarter of a row's columns, or every fourth piece of it; a block takes
  // 16 or 4 of them at a time.
  const int rows_max = min(p.rows, kRG);
  const bool split = cuts * rows_max <= (int)gridDim.x * 2;
  const int at_once = split ? kMergeWarps / kMergeParts : kMergeWarps;
  const int part = split ? warp % kMergeParts : 0, step = split ? kMergeParts : 1;
  const int tasks = cuts * rows_max * 4;
  for (int t0 = blockIdx.x * at_once; t0 < tasks; t0 += gridDim.x * at_once) {
    const int task = t0 + (split ? warp / kMergeParts : warp);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    int64_t orow = -1;
    const int quarter = task & 3, r = (task >> 2) % rows_max;
    if (task < tasks) {
      const auto g = c.group[(task >> 2) / rows_max];
      const int n = g.n;
      float* wt = weight[warp];
      float m = -INFINITY;
      for (int i = lane; i < n; i += 32) {
        const int at = c.slot_of(g, i);
        wt[i] = at >= 0 ? p.part_lse[(int64_t)at * kRG + r] : -INFINITY;
        m = fmaxf(m, wt[i]);
      }
      if (r < g.rows) {
        orow = g.row + r;
        // the first pieces' results are on their way while the weights are computed
        constexpr int kDeep = 4;
        float4 v[kDeep];
        const float4* src = reinterpret_cast<const float4*>(p.part_o + (int64_t)r * kDl + 128 * quarter) + lane;
        auto load = [&](int i0) {
#pragma unroll
          for (int d = 0; d < kDeep; ++d) {
            const int i = i0 + d * step, at = i < n ? c.slot_of(g, i) : -1;
            v[d] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at >= 0) v[d] = __ldcg(src + (int64_t)at * (kRG * kDl / 4));
          }
        };
        load(part);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -INFINITY) m = 0.f;  // no piece has any weight
        float sum = 0.f;
        for (int i = lane; i < n; i += 32) {
          wt[i] = __expf(wt[i] - m);
          sum += wt[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        total = sum == 0.f ? 1.f : sum;  // then a row of zeros, as from one piece
        if (p.lse && quarter == 0 && part == 0 && lane == 0) p.lse[orow] = m + logf(sum);
        __syncwarp();
        for (int i0 = part;;) {
#pragma unroll
          for (int d = 0; d < kDeep; ++d) {
            const int i = i0 + d * step;
            const float f = i < n ? wt[i] : 0.f;  // 0 for an empty piece
            acc.x = fmaf(f, v[d].x, acc.x);
            acc.y = fmaf(f, v[d].y, acc.y);
            acc.z = fmaf(f, v[d].z, acc.z);
            acc.w = fmaf(f, v[d].w, acc.w);
          }
          i0 += kDeep * step;
          if (i0 >= n) break;
          load(i0);
        }
      }
      __syncwarp();  // weight is reused
    }
    if (split) {  // the same in every block
      sums[warp][lane] = acc;
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int o = 1; o < kMergeParts; ++o) {
          const float4 a = sums[warp + o][lane];
          acc.x += a.x;
          acc.y += a.y;
          acc.z += a.z;
          acc.w += a.w;
        }
      }
      __syncthreads();
    }
    if (orow >= 0 && part == 0) {
      const float inv = 1.f / total;
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                           b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * kDl + 128 * quarter)[lane] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

float score_factor(const mla_kv8_attn_args& a) {
  return (float)std::ldexp((double)a.scale * 1.4426950408889634, a.cache.exponent);
}

mla_status validate_shape(const mla_kv8_attn_args* a) {
  if (!a) return MLA_ERR_INVALID_ARG;
  if (a->B < 0 || a->Q < 0 || a->H < 1) return MLA_ERR_INVALID_ARG;
  if (a->Q > MLA_MAX_Q) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)a->H * a->Q > (int64_t)1 << 24 || (int64_t)a->H * a->Q * a->B > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

mla_status validate_call(const mla_kv8_attn_args* a) {
  mla_status st = validate_cache(&a->cache);
  if (st != MLA_OK) return st;
  if (!a->q_lat || !a->q_pe || !a->prefix_lens || !a->out) return MLA_ERR_INVALID_ARG;
  if (!aligned(a->q_lat, 16) || !aligned(a->q_pe, 16) || !aligned(a->out, 16)) return MLA_ERR_INVALID_ARG;
  if (!aligned(a->prefix_lens, 4) || !aligned(a->tree_parent, 4) || !aligned(a->lse, 4)) return MLA_ERR_INVALID_ARG;
  if (a->page_size < 1) return MLA_ERR_INVALID_ARG;
  if (a->page_size == 1) {
    if (!a->kv_indptr || !a->kv_indices || !aligned(a->kv_indptr, 4) || !aligned(a->kv_indices, 4))
      return MLA_ERR_INVALID_ARG;
  } else {
    if (!a->block_table || a->max_pages < 1 || !aligned(a->block_table, 4)) return MLA_ERR_INVALID_ARG;
    if ((int64_t)a->max_pages * a->page_size > INT32_MAX) return MLA_ERR_INVALID_ARG;
  }
  if (a->window < 0 || a->sinks < 0 || (a->window == 0 && a->sinks != 0)) return MLA_ERR_INVALID_ARG;
  // rounded to zero or infinity, the factor would turn scores of -inf or 0 into NaN
  if (!std::isfinite(a->scale) || !(a->scale > 0.f) || !std::isnormal(score_factor(*a))) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

// CTAs of a launch, one per SM of the current device; 0 when it cannot be had.
int workers_per_gpu() {
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
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cached[dev] = sms < kMaxWorkers ? sms : kMaxWorkers;
  return cached[dev];
}

// The pool's rows as a tensor of bytes, a chunk of `rows` rows to a box.
bool cache_map(CUtensorMap* m, const mla_kv8_cache& cache, int rows) {
  const kvq::EncodeTiledFn f = kvq::encode_tiled();
  const cuuint64_t dims[2] = {MLA_KV8_ROW_BYTES, (cuuint64_t)cache.slots}, strides[1] = {(cuuint64_t)cache.row_stride};
  const cuuint32_t box[2] = {128, (cuuint32_t)rows}, step[2] = {1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, cache.rows, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which kernel a call takes, by the query rows of a sequence, its workers (CTAs, or
// clusters of two), and the rows that a worker takes at once.  Two groups of 32 rows cost
// less than one of 128 that is half empty, three do not; us, few rows' kernel and many
// rows', 30 sequences of 4,096 to 8,192 tokens: 40 rows 58.0 and 59.5, 64 61.4 and 61.1,
// 96 78.9 and 64.8, 128 95.7 and 69.1; 16 windows of 4,096: 64 rows 33.9 and 37.2, 128
// 51.6 and 41.2.
constexpr int kFewRows = 64;
struct Plan {
  bool many;
  int workers, group;
};
Plan plan(int rows) {
  Plan pl;
  pl.many = rows > kFewRows;
  pl.workers = pl.many ? rows::clusters_per_gpu() : workers_per_gpu();
  pl.group = pl.many ? kvq::kRows128 : kRG;
  return pl;
}

struct Layout {
  size_t starts, part_lse, part_o, total;
};
Layout layout(const Plan& pl) {
  const int workers = pl.workers, kRG = pl.group;
  Layout l;
  size_t o = MLA_KV8_WORKSPACE_BYTES;
  l.starts = o;    o = align256(o + sizeof(Start) * (size_t)workers);
  l.part_lse = o;  o = align256(o + sizeof(float) * 2 * (size_t)workers * kRG);
  l.part_o = o;    o = align256(o + sizeof(float) * 2 * (size_t)workers * kRG * kDl);
  l.total = o;
  return l;
}

Params make_params(const mla_kv8_attn_args* a, void* ws, const Plan& pl) {
  Params p = {};
  p.B = a->B;
  p.Q = a->Q;
  p.H = a->H;
  p.rows = a->H * a->Q;
  p.cache = static_cast<const uint8_t*>(a->cache.rows);
  p.row_stride = a->cache.row_stride;
  p.slots = a->cache.slots;
  p.q_lat = a->q_lat;
  p.q_pe = a->q_pe;
  p.page_size = a->page_size;
  Divider d;
  d.set(a->page_size);
  p.page_shift = d.shift;
  p.page_mul = d.mul;
  p.kv_indptr = a->kv_indptr;
  p.kv_indices = a->kv_indices;
  p.block_table = a->block_table;
  p.max_pages = a->max_pages;
  p.prefix_lens = a->prefix_lens;
  p.tree_parent = a->tree_parent;
  p.window = a->window;
  p.sinks = a->sinks;
  p.scale_log2 = score_factor(*a);
  p.out_mul = (float)std::ldexp(1.0, a->cache.exponent);
  p.out = a->out;
  p.lse = a->lse;
  p.groups = (p.rows + kRG - 1) / kRG;
  p.clusters = pl.workers;
  p.scales = a->cache.scales;
  p.block.set(a->cache.block);
  p.box = a->page_size & -a->page_size;  // the largest power of two that divides the page size; see producer()
  if (p.box > 32) p.box = 32;
  if (p.box < 16) p.box = 0;
  const Layout l = layout(pl);
  char* base = static_cast<char*>(ws);
  p.err = reinterpret_cast<uint32_t*>(base);
  p.starts = base + l.starts;
  p.part_lse = reinterpret_cast<float*>(base + l.part_lse);
  p.part_o = reinterpret_cast<float*>(base + l.part_o);
  return p;
}

mla_status run_attn(const mla_kv8_attn_args* a, void* workspace, size_t ws_bytes, mla_stream_t stream,
                    uint64_t hold_ns) {
  mla_status st = validate_shape(a);
  if (st != MLA_OK) return st;
  if (a->B == 0 || a->Q == 0) return hold_ns ? MLA_ERR_INVALID_ARG : MLA_OK;  // the self-test needs a launch
  st = validate_call(a);
  if (st != MLA_OK) return st;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < MLA_KV8_WORKSPACE_BYTES) return MLA_ERR_WORKSPACE;
  const Plan pl = plan(a->H * a->Q);
  if (pl.workers < 1) return MLA_ERR_CUDA;
  if (ws_bytes < layout(pl).total) return MLA_ERR_WORKSPACE;
  Params p = make_params(a, workspace, pl);
  p.hold = hold_ns != 0;
  p.wait_ns = p.hold ? hold_ns : kWaitLimitNs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap map;
  if (!cache_map(&map, a->cache, p.box > 0 ? p.box : 1)) return MLA_ERR_CUDA;
  if (pl.many) return rows::launch(p, map, s);
  const int n = pl.workers;
  // per call: the attribute belongs to the context, which may be a new one
  if (cudaFuncSetAttribute(kv8_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (launch_kernel(kv8_attn_kernel, dim3(n), dim3(kThreads), kSmemAlloc, s, true, p, map) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (n > 1 && launch_kernel(kv8_merge_kernel, dim3(2 * n), dim3(kMergeThreads), 0, s, true, p) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

}  // namespace
}  // namespace kv8
}  // namespace mlav

using namespace mlav;

extern "C" size_t mla_kv8_attn_workspace_size(const mla_kv8_attn_args* a) {
  if (kv8::validate_shape(a) != MLA_OK) return 0;
  const kv8::Plan pl = kv8::plan(a->H * a->Q);
  return pl.workers > 0 ? kv8::layout(pl).total : 0;
}

extern "C" mla_status mla_kv8_attn(const mla_kv8_attn_args* a, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  return kv8::run_attn(a, workspace, ws_bytes, stream, 0);
}

extern "C" mla_status mla_kv8_selftest_timeout(const mla_kv8_attn_args* a, void* workspace, size_t ws_bytes,
                                               uint64_t hold_ns, mla_stream_t stream) {
  if (hold_ns == 0 || hold_ns > 1000000000ull) return MLA_ERR_INVALID_ARG;
  return kv8::run_attn(a, workspace, ws_bytes, stream, hold_ns);
}
