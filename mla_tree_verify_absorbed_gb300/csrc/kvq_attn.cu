// Verify attention and decoding over the 4-bit latent cache (mla_kvq_attn) on
// tcgen05 tensor cores.
//
// The work.  128 query rows ((node, head) pairs) against tiles of 64 tokens:
// S = Q [128 x 576] . K^T, online softmax, O += P [128 x 64] . V [64 x 512],
// V the latent part of K.  The latents arrive as 4-bit codes and are converted
// to operands on the way into shared memory: to bf16 for S (whose other operand
// is the caller's bf16 queries), to f16 for O, where the weights then keep 11
// bits instead of 8; both conversions are exact (kvq.cuh).
//
// Two CTAs per work item.  An fp32 accumulator for 128 x 512 fills one SM's
// Tensor Memory, so S and O live in different SMs of a cluster:
//   rank 0, scores: queries in Tensor Memory (288 columns, the A operand), three
//           S tiles (192 columns); converts the whole tile (64 tokens x 576) to
//           bf16; softmax in registers, one thread per row and tile;
//   rank 1, values: O (512 columns); converts the same tile's latents to f16.
// The weights and the rows' rescale factors go from rank 0 to rank 1 by bulk
// shared -> shared::cluster copies.  Both CTAs read the packed rows themselves:
// 416 + 288 bytes per token and cluster, where a pair that shares converted
// operands would exchange halves of 1152.
//
// What bounds it.  With many rows per token, the score CTA's shared memory and
// the warps that feed it: per tile it takes in 26 KB of packed rows, hands them
// to the producers, takes back 72 KB of operand, gives that to the MMAs, and
// passes 16 KB of weights on, about 1,700 cycles of its 128 bytes per cycle
// with 1,152 cycles of MMA beneath.  A half tile takes a producer warp 650
// cycles to convert in the value CTA, where nothing else uses the schedulers,
// and 1,100 to 1,400 beside the softmax.  Measured on 64 nodes x 64 heads x
// 200,000 tokens: 1.58 ms, 1.13 PFLOP/s.  With few rows the same conversion
// serves fewer products: 128 ragged sequences x 16 heads (429,667 tokens) take
// 109 us, 1.7 TB/s.  A call of 257 tokens takes 16 us: launch and split 2.2, the
// first piece 1.1, its queries 1.6, first scores 2.5, first weights 1.6, 1.0 a
// tile, output 1.5, exit 0.8.
//
// Conversion.  8 producer warps per CTA, in each a lane per (token, 64-element
// chunk): 32 bytes of codes and 4 scales make the 128 bytes of one operand row
// in one chunk.  The 8 lanes of a quarter warp hold 8 different tokens, so
// their 16-byte stores fall into 8 different bank groups of the 128-byte
// swizzle.
//
// Work split.  Row group g of sequence b costs T_b + kFixed units (T_b tiles).
// The units of all row groups, in order, are cut into equal intervals, one per
// cluster; a row group that falls into several clusters is merged from their
// partial results by a second kernel.  Every CTA computes the cut itself from
// prefix_lens, so there is no planning kernel, and equal arguments give equal
// cuts.
//
// Masks.  Tiles that hold no visible position are never visited (a window
// leaves the tiles of the first `sinks` tokens and those from the oldest
// visible position on); inside a tile the mask is applied to the scores of
// tiles that need one.  Masked scores are -inf by selection, and any bytes in
// the cache stand for finite latents, so 0 * V is 0 whatever V holds.
//
// Every wait is bounded (2 s, less in the self-test); on timeout both CTAs stop
// issuing, drain what they issued, free their Tensor Memory and report
// MLA_DEVERR_TIMEOUT.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "kvq.cuh"
#include "sm100.cuh"

namespace mlav {
namespace kvq {
using namespace sm100;

mla_status validate_cache(const mla_kvq_cache* c);

// Tensor maps of the queries, [B Q H] rows of 512 and of 64, in boxes of 64
// elements x Params::box_rows rows.
struct QueryMaps {
  CUtensorMap lat, pe;
};

constexpr int kRG = 128;       // query rows per work item
constexpr int kTK = 64;        // tokens per tile
constexpr int kThreads = 640;  // 20 warps: 96 registers a thread
constexpr uint32_t kTmemCols = 512;
// Warps 0-7 convert, warps 8-15 hold rows; each in two groups that take the
// tiles of one parity, so a group has two tile periods for its chain of loads,
// conversion and barriers.  The roles' loops are kept short: together they have
// to stay in the SM's instruction cache (unrolled twice as far they ran at half
// the speed).
constexpr int kProducerWarps = 8, kGroupWarps = 4;
constexpr int kWarpRows = 8, kRowWarps = 8;
constexpr int kWarpSched = 16;  // the pieces of work
constexpr int kWarpAux = 17;    // TMEM allocation; rank 0: weight copies
// Warps w, w + 4, .. share a scheduler, and issuing a tile's MMAs is work for it:
// away from the one that has the row warps of few rows (beside them, 128 ragged
// sequences x 16 heads took 4% longer).
constexpr int kWarpMma = 19;

// A tile is staged as two halves, each with its own full / empty barriers:
// half h holds latent columns [256 h, 256 h + 256) as 4 chunks of 64 columns
// (64 token rows of 128 bytes each); in the score CTA half 1 ends with the
// rope chunk.  Tile j uses stage j % 2.
constexpr int kChunk = kTK * 128;             // 8 KB
constexpr int kStageS = 9 * kChunk;           // score CTA: 72 KB per tile
constexpr int kStageV = 8 * kChunk;           // value CTA: 64 KB
constexpr int kHalf = 4 * kChunk;
constexpr int kPBytes = kRG * 128;            // weights of a tile, f16
constexpr int kPBufs = 3;                     // value CTA: weights landed
constexpr int kPStages = 2;                   // score CTA: weights staged
constexpr int kRawRow = 336;                  // 256 bytes of codes, two buffers of 32 bytes of scales
constexpr int kTok = kTK / kGroupWarps;       // tokens of a producer warp
constexpr int kRawWarp = kTok * kRawRow;
// Offsets: stages first in both CTAs, then the score CTA's staged weights or
// the value CTA's landed ones, then the raw rows.
constexpr int kOffPS = 2 * kStageS, kOffPV = 2 * kStageV;
constexpr int kOffRaw = kOffPS + kPStages * kPBytes > kOffPV + kPBufs * kPBytes ? kOffPS + kPStages * kPBytes
                                                                                : kOffPV + kPBufs * kPBytes;
constexpr int kOffCtl = kOffRaw + kProducerWarps * kRawWarp;
// A row group with few rows (decoding with few heads) leaves whole lane
// quadrants of 32 rows unused: their softmax, weights and outputs are left out.
__device__ __forceinline__ int live_quads(int rows, int g) { return min(4, (rows - g * kRG + 31) >> 5); }
__device__ __forceinline__ uint32_t weight_bytes(int quads) { return (uint32_t)quads * 32u * 128u; }

// Tensor Memory columns: score CTA, three S tiles and the queries (bf16 pairs);
// value CTA, O from column 0
constexpr int kSBufs = 3;
constexpr uint32_t kColS = 0, kColQ = kSBufs * kTK;
static_assert(kColQ + kDk / 2 <= kTmemCols, "Tensor Memory columns");
// upper halves of the operand descriptors (smem_desc): only the start address,
// in the lower half, differs from MMA to MMA
constexpr uint32_t kDescHiK = (1024u >> 4) | (1u << 14) | (kLayoutSw128 << 29);
constexpr uint32_t kDescLoK = (16u >> 4) << 16;        // K-major: queries' and weights' operands
constexpr uint32_t kDescLoV = ((uint32_t)kChunk >> 4) << 16;  // MN-major: 64-column chunks 8 KB apart
// start-address field of offset `off` (the window's address of a cluster CTA
// has bits above the field)
__device__ __forceinline__ uint32_t desc_addr(const uint8_t* smem, uint32_t off) {
  return ((smem_u32(smem) & 0x3FFFFu) + off) >> 4;
}
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}

constexpr uint32_t kIdescS = idesc_bf16_f32(kRG, kTK, 0, 0);   // queries (TMEM), keys K-major
constexpr uint32_t kIdescPV = idesc_f16_f32(kRG, 256, 0, 1);   // weights K-major, values MN-major

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 20000000ull;

// Weights are 2^(score - max + kWeightShift) in f16: a lazy maximum lets them
// reach 2^8 above 1, which the shift puts at 2^15, below f16's 65504, so that
// weights down to 2^-21 of the maximum keep 11 bits and down to 2^-31 some.
constexpr float kLazy = 8.f;
constexpr float kWeightShift = 7.f;

// What the split counts for a row group or a piece of one, in tiles, beside its
// own, and the fewest tiles worth a cluster of its own.  Chosen by the times of
// whole calls: a piece of 128 rows spends longer (queries 5 to 6 us, fp32 output
// 4.4, at 1.0 to 1.2 a tile), but the even cut makes two pieces of an interval
// wherever it crosses a border, and a larger count moves the cuts without saving
// any.  Single sizes jump by 10% with where the cuts fall, so these are means, us:
// 64 nodes x 64 heads in windows of 1,000 .. 1,256; 16 sequences x 64 heads in
// windows of 4,096 .. 4,352; 128 ragged sequences x 16 heads, three sets of
// lengths.  kFixed 3: 43.4, 41.9, 101.7; 4: 44.5, 40.8, 99.7; 5: 45.3, 39.9, 101.9;
// 6: 46.5, 40.3, 103.3; 8: 48.9, 43.2, 106.5; kMinTiles 6 in place of 4: 45.3, 40.8,
// 100.4.  Row groups in long pieces (32 sequences x 128 heads, trees) move by 1%.
constexpr int kFixed = 4;
constexpr int kMinTiles = 4;

// One cluster's share of a row group, as the roles need it.
struct alignas(16) Piece {
  int32_t b, g, slot, t0;      // slot: partial-result slot, -1 for a whole row group
  int32_t t1, ns, tw, N;       // tiles [t0, t1), numbered over [0, ns) and from tw on; b < 0: no more pieces
  int32_t lo, P, pad0, pad1;
  int64_t entry;               // first table entry of the sequence
  int64_t pad2;
  __device__ __forceinline__ int tile(int v) const { return v < ns ? v : v - ns + tw; }
};
constexpr int kPieces = 4;

// Barriers that two groups of warps pass at different tiles have one instance
// per buffer they guard: a wait must never be able to pass on the parity of an
// older phase.
struct alignas(16) Ctl {
  uint64_t full[4];            // half tile converted (8 producer warps); index 2 (j % 2) + half
  uint64_t empty[4];           // the MMAs reading it are complete
  uint64_t s_full[kSBufs];     // score: S tile in TMEM
  uint64_t s_free[kSBufs];         // score: softmax has loaded S (4 row warps)
  uint64_t q_ready[kPieces];   // score: a piece's queries in TMEM, stages free again (8 row warps)
  uint64_t q_in;               // score: queries copied (copy bytes)
  uint64_t m_ready[2][4];      // score: running maxima after a tile written (per lane quadrant, 1 warp)
  uint64_t p_free[kPBufs];     // score: the PV MMAs that read rank 1's buffer are complete (its commit)
  uint64_t ps_free[kPStages];  // score: the staged weights have landed in rank 1 (its first row warp)
  uint64_t fin_free;           // score: rank 1 consumed lfin / mfin (256 arrivals)
  uint64_t p_staged[kPStages]; // score: weights and factors staged (4 row warps)
  uint64_t p_full[kPBufs];     // value: weights and factors landed (copy bytes)
  uint64_t pv_done[kPBufs];    // value: PV MMAs of a tile complete
  uint64_t o_ready[kPBufs];    // value: O rescaled, weights in (8 row warps)
  uint64_t fin_full;           // value: lfin / mfin written (256 remote arrivals)
  uint64_t drain;
  uint64_t piece_full[kPieces];   // piece written (scheduler warp)
  uint64_t piece_empty[kPieces];  // read by every warp of this CTA that follows the pieces
  Piece piece[kPieces];
  alignas(16) float alpha[kPBufs][kRG];  // rescale factors: staged in rank 0 ([kPStages]), landed in rank 1
  float m_run[2][kRG];         // score: running maxima after the last tile of each parity
  float lfin[2][kRG];          // value: each group's row sums of the shifted weights
  float mfin[kRG];             // value: row maxima, base-2 units
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
static_assert(kOffPS % 1024 == 0 && kOffPV % 1024 == 0 && kStageS % 1024 == 0, "swizzle atoms");

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Ctl* c) {
  if (mbar_wait(bar, parity, &c->abort, c->wait_ns, true)) return true;
  for (uint32_t rk = 0; rk < 2; ++rk) st_cluster_u32(mapa_shared(smem_u32(&c->abort), rk), 1u);
  return false;
}
// The first try is inline, everything after it one shared copy: the roles'
// loops have to fit the instruction cache together.
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
// ---------------------------------------------------------------------------
// work split
// ---------------------------------------------------------------------------
// The tiles of a sequence that any of its nodes sees: [0, ns) and [tw, te).
struct Tiles {
  int ns, tw;
  int T;  // ns + te - tw; 0 for an unused sequence
  int64_t lo;  // positions in [sinks, lo) are seen by no node
};
__device__ __forceinline__ Tiles tiles_of(const Params& p, int64_t P) {
  Tiles t;
  t.lo = 0;
  t.ns = t.tw = t.T = 0;
  if (P < 0) return t;
  if (p.window > 0 && P - p.window + 1 > 0) {
    t.lo = P - p.window + 1;
    t.tw = (int)(t.lo / kTK);
    const int64_t ns = ((int64_t)p.sinks + kTK - 1) / kTK;
    t.ns = (int)(ns < t.tw ? ns : t.tw);
  }
  t.T = t.ns + (int)((P + p.Q + kTK - 1) / kTK) - t.tw;
  return t;
}

// First tile of what a cut at unit z of a row group (kFixed + T units) leaves
// to the right: the fixed cost comes first.
__device__ __forceinline__ int cut_tile(int64_t z, int T) {
  return z <= kFixed ? 0 : z >= kFixed + T ? T : (int)(z - kFixed);
}

// a / b for a >= 0, b > 0: a 32-bit division wherever it will do.
__device__ __noinline__ int64_t div_long(int64_t a, int b) { return a / b; }
__device__ __forceinline__ int64_t div_fast(int64_t a, int b) {
  return a >> 32 ? div_long(a, b) : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Clusters that share `total` units.
__device__ __forceinline__ int active_clusters(const Params& p, int64_t total) {
  const int64_t n = div_fast(total, kFixed + kMinTiles);
  return (int)(n < 1 ? 1 : n > p.clusters ? p.clusters : n);
}
__device__ __forceinline__ int64_t first_unit(int64_t total, int n, int k) { return div_fast(total * k, n); }

// Where a cluster's interval begins: unit x of the groups * (kFixed + T) units
// of sequence b, for the merging kernel.
struct alignas(16) Start {
  int64_t x;
  int32_t b, T;
  int32_t n;  // clusters that share the call (0: nothing to merge)
  int32_t pad[3];
};

// The last unused sequence from b on before a used one.  Unused ones are passed
// 128 at a time: one after the other they took 0.18 us each, 204 us for 1,024
// between two short sequences, and the roles' waits ran out behind ten million.
// Not inlined: the smallest calls pay for cold code between the hot (15.6 -> 15.8).
__device__ __noinline__ int last_unused(const int32_t* prefix_lens, int B, int b) {
  const int lane = threadIdx.x & 31;
  for (; b < B; b += 128) {
    bool used[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = b + 32 * q + lane;
      used[q] = i < B && prefix_lens[i] >= 0;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t mask = __ballot_sync(0xffffffffu, used[q]);
      if (mask) return b + 32 * q + __ffs(mask) - 2;
    }
  }
  return B;
}

// Scheduler warp of each CTA: writes this cluster's pieces in order, then an
// end mark, into the ring that the other roles follow.  A piece that does not
// begin its row group is the cluster's first, one that does not end it the
// last, so two partial slots are enough.
__device__ void schedule(const Params& p, Ctl* c, int cluster) {
  const int lane = threadIdx.x & 31;
  int64_t left = c->left;
  int64_t x = c->start_x;
  uint32_t seg = 0;
  auto put = [&](const Piece& pc) {
    const uint32_t q = seg % kPieces;
    if (!wait_warp(&c->piece_empty[q], ((seg / kPieces) & 1u) ^ 1u, c)) return false;
    if (lane == 0) {
      c->piece[q] = pc;
      mbar_arrive(&c->piece_full[q]);
    }
    __syncwarp();
    ++seg;
    return true;
  };
  Sequence sq{c->start_P, c->start_entry, 0u};
  for (int b = c->start_b; left > 0 && b < p.B; ++b, x = 0) {
    if (b != c->start_b) sq = read_sequence(p, b);
    const Tiles tl = tiles_of(p, sq.P);
    if (tl.T == 0) {
      b = last_unused(p.prefix_lens, p.B, b);
      continue;
    }
    const int L = kFixed + tl.T;
    Piece pc;
    pc.b = b;
    pc.ns = tl.ns;
    pc.tw = tl.tw;
    pc.lo = (int32_t)tl.lo;
    pc.P = sq.P;
    pc.N = (int32_t)((int64_t)pc.P + p.Q);
    pc.entry = sq.entry;
    for (int g = (int)div_fast(x, L); g < p.groups && left > 0; ++g) {
      const int64_t z = x - (int64_t)g * L;
      const int64_t take = L - z < left ? L - z : left;
      pc.g = g;
      pc.t0 = cut_tile(z, tl.T);
      pc.t1 = cut_tile(z + take, tl.T);
      pc.slot = pc.t0 == 0 && pc.t1 == tl.T ? -1 : 2 * cluster + (pc.t0 == 0);
      x += take;
      left -= take;
      if (pc.t1 > pc.t0 && !put(pc)) return;
    }
  }
  Piece end = {};
  end.b = -1;
  put(end);
}

// Calls f(piece) for the pieces of the ring in order; f's piece stays valid
// only as far as f copied it.  Every lane of the warp takes part.
template <class F>
__device__ __forceinline__ void for_pieces(Ctl* c, F&& f) {
#pragma unroll 1
  for (uint32_t seg = 0;; ++seg) {
    const uint32_t q = seg % kPieces;
    if (!wait_warp(&c->piece_full[q], (seg / kPieces) & 1u, c)) return;
    const Piece pc = c->piece[q];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&c->piece_empty[q]);
    if (pc.b < 0) return;
    if (!f(pc)) return;
  }
}
// Warps that follow the pieces: producers, row warps, the MMA warp and, in the
// score CTA, the copier.
constexpr int kFollowers = kProducerWarps + kRowWarps + 1;

// Block-wide: validates every sequence, sums the units and finds where this
// cluster's interval begins.  Returns the clusters that share the call, 0 when
// a table is bad, -1 when every sequence is unused.  Threads take consecutive
// sequences.
__device__ int make_split(const Params& p, Ctl* c, int cluster) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = tid * per, b1 = min(b0 + per, p.B);
  uint32_t e = 0;
  int64_t sum = 0;
  Sequence q;
  int T = 0;
  auto units = [&](int b) -> int64_t {  // and q, T
    q = read_sequence(p, b);
    T = q.err ? 0 : tiles_of(p, q.P).T;
    return T ? (int64_t)p.groups * (kFixed + T) : 0;
  };
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    sum += units(b);
    e |= q.err;
  }
  auto warp_scan = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  const int64_t inc = warp_scan(sum);
  if (lane == 31) c->scan[warp] = inc;
  if (e) atomicOr(&c->err, e);
  __syncthreads();
  const int64_t warps = warp_scan(lane < kThreads / 32 ? c->scan[lane] : 0);
  const int64_t total = __shfl_sync(0xffffffffu, warps, 31);
  int64_t at = __shfl_sync(0xffffffffu, warps, max(warp - 1, 0));  // units before this thread's sequences
  at = (warp > 0 ? at : 0) + inc - sum;
  if (c->err) return 0;  // the same in every CTA: each has read every sequence
  const int n = active_clusters(p, total);
  if (cluster < n && total > 0) {
    const int64_t w0 = first_unit(total, n, cluster);
    if (w0 >= at && w0 < at + sum) {
      c->left = first_unit(total, n, cluster + 1) - w0;
      int b = b0;
      if (per > 1) {  // q and T are those of the thread's last sequence
#pragma unroll 1
        for (;; ++b) {
          const int64_t u = units(b);
          if (w0 < at + u) break;
          at += u;
        }
      }
      c->start_b = b;
      c->start_x = w0 - at;
      c->start_T = T;
      c->start_P = q.P;
      c->start_entry = q.entry;
    }
  }
  __syncthreads();
  return total > 0 ? n : -1;
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
// Converts 64 codes with their 4 scales into the 8 pieces of an operand row;
// piece q goes to dst ^ 16 q (dst: the row's address plus 16 times the row's
// place in its swizzle group).
template <class To>
__device__ __forceinline__ void convert_chunk(const uint32_t (&code)[8], uint32_t scale, uint32_t dst, int r7) {
#pragma unroll
  for (int pr = 0; pr < 2; ++pr) {
    const uint32_t s = To::scales(__byte_perm(scale, 0, pr ? 0x4342 : 0x4140));
    const uint32_t o = To::offsets(s);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t sk = k ? hi2(s) : lo2(s), ok = k ? hi2(o) : lo2(o);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int q = 4 * pr + 2 * k + w;
        uint32_t v[4];
        To::word(code[q], sk, ok, v);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((q ^ r7) << 4)), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3])
                     : "memory");
      }
    }
  }
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// pos / page_size by a multiplication that the host prepares: for page_size in
// (2^(L-1), 2^L], ceil(2^(31+L) / page_size) fits 32 bits and is off by less than
// 2^L over 2^(31+L), too little to matter for pos < 2^31.  Page size 1 needs no
// branch, and the producers' loops stay short.
__device__ __forceinline__ uint32_t page_of(const Params& p, uint32_t pos) {
  return (uint32_t)(((uint64_t)pos * p.page_mul) >> p.page_shift);
}

// Queries of up to 64 rows pass through one stage, that of the piece's second
// tile, so that its first is converted meanwhile.
__device__ __forceinline__ bool one_stage(const Params& p) { return p.box_rows <= 64; }

// One warp of producer group `grp`: tokens kTok pw .. of the tiles of that
// parity.  The packed rows (codes and scales, 288 bytes) come by cp.async into
// rows of shared memory that the warp has to itself; a half tile's codes are
// fetched as soon as the tile before has been converted that far, so they have
// about two tile periods to arrive.  (Loads into registers pass through the
// small L1 that this much shared memory leaves, and its lines, not the latency,
// then limited the bytes in flight.)  The rope keys need no conversion and go
// straight to their place in the stage.  Rows 336 bytes apart put the 8 tokens
// that a quarter warp reads at once into different banks.
template <bool kScore>
__device__ __forceinline__ void producer(const Params& p, uint8_t* smem, Ctl* c, int warp) {
  using To = typename std::conditional<kScore, ToBf16, ToF16>::type;
  const int lane = threadIdx.x & 31;
  const int grp = warp / kGroupWarps, pw = warp % kGroupWarps;
  const int r7 = lane & 7, ch = lane >> 3;
  const int r = kTok * pw + r7;  // token row of the first set of 8 within the tile
  const uint32_t stage = smem_u32(smem) + grp * (kScore ? kStageS : kStageV);
  const uint32_t raw = smem_u32(smem) + kOffRaw + warp * kRawWarp;
  uint32_t err = 0;
  uint32_t j = 0, seg = 0;
  for_pieces(c, [&](const Piece& pc) {
    int t = pc.t0 + (int)((grp ^ j) & 1u);
    const bool ahead = kScore && one_stage(p) && t == pc.t0;  // the queries use the other stage
    j += (uint32_t)(pc.t1 - pc.t0);
    const uint32_t q_bar = seg % kPieces, q_phase = (seg / kPieces) & 1u;
    ++seg;
    // Every warp waits for every piece's queries: a phase left out could be
    // taken for the next one.  A group whose tiles do not need the wait may come
    // to it late, but of the two pieces after this one, one at least has a tile
    // of the group, so the queries of the fourth, which use the same barrier,
    // cannot overtake it.
    if (t >= pc.t1) return !kScore || wait_warp(&c->q_ready[q_bar], q_phase, c);
    uint32_t turn = (j - (uint32_t)(pc.t1 - t)) >> 1;  // tiles this group has taken before
    const int32_t* idx = (p.page_size == 1 ? p.kv_indices : p.block_table) + pc.entry;
    // Pool row of token kTok pw + lane % kTok of tile v, in two steps: the table
    // entry (a slot, or a page), and, a tile later, the slot.  Positions that no
    // node sees have the entry -1 and read slot 0, under a weight of zero; a
    // table's own entries may be any number, so a bad one is told from those by
    // its position.
    auto pos_of = [&](int v) { return (uint32_t)pc.tile(v) * kTK + kTok * pw + lane % kTok; };
    auto seen = [&](int v, uint32_t pos) {
      return v < pc.t1 && pos < (uint32_t)pc.N && (pos >= (uint32_t)pc.lo || pos < (uint32_t)p.sinks);
    };
    auto entry_of = [&](int v) -> int32_t {
      const uint32_t pos = pos_of(v);
      return seen(v, pos) ? __ldg(idx + page_of(p, pos)) : -1;
    };
    auto slot_of = [&](int32_t e, int v) -> uint32_t {
      const uint32_t pos = pos_of(v);
      int64_t s = (int64_t)e * p.page_size + (pos - page_of(p, pos) * (uint32_t)p.page_size);
      if (e < 0 || s >= p.slots) {
        if (seen(v, pos)) err |= MLA_DEVERR_SLOT;
        s = 0;
      }
      return (uint32_t)s;
    };
    auto row_of = [&](uint32_t slot, int token) {
      return p.cache + (uint64_t)__shfl_sync(0xffffffffu, slot, token) * (uint32_t)p.row_stride;
    };
    // 16-byte piece lane & 7 of tokens lane >> 3, + 4, .. of half h, and
    // with the first half all scales, into the buffer of this turn's parity.
    // Past the piece's last tile nothing is fetched: what the next piece
    // fetches first must not race with it.
    const uint8_t* rows[kTok / 4];  // of the tile fetched last: piece r7 of tokens ch, ch + 4, ..
    auto fetch = [&](uint32_t slot, int h, uint32_t turn, bool more) {
#pragma unroll
      for (int i = 0; i < kTok / 4; ++i) {
        const int token = 4 * i + ch;
        if (h == 0) rows[i] = row_of(slot, token) + 16 * r7;
        if (more) cp_async_16(raw + token * kRawRow + 128 * h + 16 * r7, rows[i] + 128 * h);
      }
      const int token = lane >> 1;
      const uint8_t* row = row_of(slot, token % kTok);
      if (more && h == 0 && token < kTok)
        cp_async_16(raw + token * kRawRow + kScaleOff + 32 * (turn & 1u) + 16 * (lane & 1),
                    row + kScaleOff + 16 * (lane & 1));
      cp_async_commit();
    };
    uint32_t slot = slot_of(entry_of(t), t), slot_next = 0;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) fetch(slot, h, turn, true);
    int32_t ent = entry_of(t + 2);
    // until then the queries pass through the stages
    if (kScore && !ahead && !wait_warp(&c->q_ready[q_bar], q_phase, c)) return false;
#pragma unroll 1
    for (int h = 0; t < pc.t1; h ^= 1) {
      cp_async_wait_group<1>();  // this half's pieces, of this lane
      __syncwarp();              // of every lane
      const uint32_t full = 2 * grp + h;
      if (!wait_warp(&c->empty[full], (turn & 1u) ^ 1u, c)) return false;
      if (kScore && h) {
#pragma unroll
        for (int i = 0; i < kTok / 4; ++i) {
          const int token = 4 * i + ch, row = kTok * pw + token;
          cp_async_16(stage + 8 * kChunk + row * 128 + ((r7 ^ (row & 7)) << 4),
                      row_of(slot, token) + kRopeOff + 16 * r7);
        }
        cp_async_mbar_arrive(&c->full[full]);  // when they have landed
      }
      uint32_t src = raw + r7 * kRawRow, dst = stage + h * kHalf + ch * kChunk + r * 128;
#pragma unroll 1
      for (int s = 0; s < kTok / 8; ++s) {
        uint32_t code[8];
        ld_shared_v4(src + 128 * h + 32 * ch, code[0], code[1], code[2], code[3]);
        ld_shared_v4(src + 128 * h + 32 * ch + 16, code[4], code[5], code[6], code[7]);
        convert_chunk<To>(code, ld_shared(src + kScaleOff + 32 * (turn & 1u) + 16 * h + 4 * ch), dst, r7);
        src += 8 * kRawRow;
        dst += 8 * 128;
      }
      fence_proxy_async_smem();  // generic stores, read by the MMA
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->full[full]);
      // the next tile's half into the place of this one
      if (h == 0) {
        slot_next = slot_of(ent, t + 2);
        ent = entry_of(t + 4);
        fetch(slot_next, 0, turn + 1, t + 2 < pc.t1);
      } else {
        t += 2;
        ++turn;
        slot = slot_next;
        fetch(slot, 1, turn, t < pc.t1);
      }
    }
    return !ahead || wait_warp(&c->q_ready[q_bar], q_phase, c);
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
// Tensor Memory addresses are constants here (all 512 columns are allocated, so
// the base is 0).  A tile's 36 MMAs of 32 cycles are issued straight: in a loop
// of four per iteration the one issuing thread took 75 cycles for each.
__device__ void score_mma(uint8_t* smem, Ctl* c) {
  const bool leader = elect_one();
  uint32_t j = 0, seg = 0;
  for_pieces(c, [&](const Piece& pc) {
    if (!wait_warp(&c->q_ready[seg % kPieces], (seg / kPieces) & 1u, c)) return false;
#pragma unroll 1
    for (int t = pc.t0; t < pc.t1; ++t, ++j) {
      const uint32_t par = j & 1u, turn = j >> 1, sb = j % kSBufs;
      if (!wait_warp(&c->s_free[sb], ((j / kSBufs) & 1u) ^ 1u, c)) return false;
      const uint32_t lo = desc_addr(smem, par * kStageS) | kDescLoK;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait_warp(&c->full[2 * par + h], turn & 1u, c)) return false;
        if (h) fence_proxy_async_smem();  // the rope keys came by cp.async, without a fence of their writers
        tc_fence_after();
        if (leader) {
#pragma unroll 2
          for (int kc = 4 * h; kc < (h ? 9 : 4); ++kc) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_cta_ts(kColS + sb * kTK, kColQ + kc * 32 + kk * 8,
                         desc_at(lo + ((kc * kChunk + kk * 32) >> 4), kDescHiK), kIdescS, (kc | kk) != 0);
          }
          if (h) mma_cta_commit(&c->s_full[sb]);
          mma_cta_commit(&c->empty[2 * par + h]);
        }
        __syncwarp();
      }
    }
    ++seg;
    return true;
  });
  drain_mmas(c, leader);
}

// Brings a piece's query rows into Tensor Memory (column c holds elements 2c,
// 2c + 1 of 512 latent and 64 rope ones), all row warps together.  Nine tensor
// copies, 64 elements of the rows each, fill the two stages, or with up to 64
// rows that of the second tile (a call of 257 tokens: 17.1 -> 16.6 us); they are
// free between pieces (the producers wait for q_ready before they fill them).
// The copies' 128-byte swizzle puts the 8 rows that a quarter warp reads at once
// into different banks.  (For 128 rows, a thread loading its own row took 14 us,
// cp.async of 16 bytes a lane 9, a bulk copy per row 9.)
static_assert(9 * kRG * 128 <= 2 * kStageS && 9 * 64 * 128 <= kStageS, "queries fit the stages");
__device__ bool stage_queries(const Params& p, const QueryMaps& maps, uint8_t* smem, Ctl* c, const Piece& pc, int warp,
                              uint32_t seg, uint32_t j) {
  const int lane = threadIdx.x & 31;
  const int wq = warp & 3, wg = (warp - kWarpRows) >> 2;
  const int r = wq * 32 + lane;
  const int rows = min(kRG, p.rows - pc.g * kRG);
  const uint32_t mul = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(p.qpe_mul)) * 0x10001u;  // a power of two
  uint8_t* stage = smem + (one_stage(p) && !(j & 1u) ? kStageS : 0);
  const uint32_t chunk = one_stage(p) ? 64 * 128 : kRG * 128;
  if (warp == kWarpRows && elect_one()) {
    fence_proxy_async_smem();  // the stages were written through the generic proxy
    mbar_arrive_expect_tx(&c->q_in, 9u * 128u * (uint32_t)p.box_rows);
    const int y = pc.b * p.rows + pc.g * kRG;
#pragma unroll 1
    for (int ck = 0; ck < 9; ++ck)
      tensor_copy_2d(stage + ck * chunk, ck < 8 ? &maps.lat : &maps.pe, ck < 8 ? 64 * ck : 0, y, &c->q_in);
  }
  __syncwarp();
  if (!wait_warp(&c->q_in, seg & 1u, c)) return false;
#pragma unroll 3
  for (int ck = 0; ck < 9; ++ck) {
    const uint32_t src = smem_u32(stage) + ck * chunk + r * 128;
    uint32_t w[16] = {};
    if (r < rows) {  // else another sequence's rows, or none
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ld_shared_v4(src + (((4 * wg + i) ^ (r & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (ck == 8) w[i] = hmul2_bf16(w[i], mul);
    __syncwarp();
    tmem_st_32x32b_x16(((uint32_t)(wq * 32) << 16) + kColQ + 32 * ck + 16 * wg, w);
  }
  tmem_wait_st();
  return true;
}

// The low n bits, n clamped to [0, 64].
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : ~0ull >> (64 - n); }
// Scores of the tokens whose bit is 0 become -inf, whatever they were.
__device__ __forceinline__ void mask32(uint32_t (&u)[32], uint32_t vis) {
#pragma unroll
  for (int q = 0; q < 32; ++q)
    if (!((vis >> q) & 1u)) u[q] = 0xff800000u;
}

// Online softmax: a thread per row and group of row warps; group `wg` takes
// the tiles of its parity, all 64 columns of a row in one thread.  The running
// maximum passes from group to group, warp to warp of the same rows, before
// the exponentials; each group sums its own weights.
__device__ void score_softmax(const Params& p, const QueryMaps& maps, uint8_t* smem, Ctl* c, int warp) {
  const int lane = threadIdx.x & 31;
  const int wq = warp & 3, wg = (warp - kWarpRows) >> 2;
  const int r = wq * 32 + lane;
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const float sl2 = p.scale_log2;
  const uint64_t sl2x2 = pair(sl2, sl2);
  const int nq = p.Q;
  uint32_t j = 0, seg = 0;
  bool bad = false;
  for_pieces(c, [&](const Piece& pc) {
    const int t0 = pc.t0, t1 = pc.t1;
    const int row = pc.g * kRG + r;
    const bool live = row < p.rows;
    const bool idle = wq >= live_quads(p.rows, pc.g);  // none of the warp's rows exists
    const int P = pc.P;
    if (!stage_queries(p, maps, smem, c, pc, warp, seg, j)) return false;
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->q_ready[seg % kPieces]);
    // rows past the last take the last one's mask: their results are dropped
    const NodeView nv = node_view_warp(p, pc.b, (live ? row : p.rows - 1) / p.H, P, &bad);
    // Prefix positions up to this one are outside the window (unless sinks).
    // Lengths fit 32 bits with the nodes counted, so these do too, and so do
    // their differences from a position as long as they are not below -1.
    const int past = p.window > 0 ? max(P - p.window + nv.depth, -1) : -1;
    const int past_any = p.window > 0 ? max(P - p.window + nq - 1, -1) : -1;

    // m: running maximum of the scaled scores (base-2 units) as of this
    // group's last tile; l: its sum of the shifted weights before rounding
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
      // which of the tile's 64 tokens the row sees, where not all of them
      const int pos0 = pc.tile(t) * kTK;
      const uint32_t tS = lane_off + kColS + sb * kTK;
      if (pos0 > P - kTK || pos0 <= past_any) {
        const int rel0 = pos0 - P;
        uint64_t vis = low_bits(-rel0) & ~(low_bits(past - pos0 + 1) & ~low_bits(p.sinks - pos0));
        if (rel0 < 64 && rel0 > -64) vis |= rel0 >= 0 ? nv.mask >> rel0 : nv.mask << -rel0;
        // few tiles need it: the masked scores go back, and the loops below know of no mask
#pragma unroll 1
        for (int hc = 0; hc < 2; ++hc) {
          uint32_t u[32];
          tmem_ld32_sync(tS + 32 * hc, u);
          mask32(u, (uint32_t)(vis >> (32 * hc)));
          tmem_st_32x32b_x32(tS + 32 * hc, u);
        }
        tmem_wait_st();
      }
      // Two passes of 32 columns, for the maximum and for the weights: the
      // scores stay in Tensor Memory in between, which halves the registers
      // and the code.  The maximum comes with the load (by instructions of its
      // own, 64 nodes x 64 heads x 200,000 tokens took 1,624 us, not 1,603).  A
      // NaN score makes the row's sum NaN whichever way the maximum takes it.
      float tmax = -INFINITY;
#pragma unroll 1
      for (int hc = 0; hc < 2; ++hc) tmax = fmaxf(tmax, tmem_max32(tS + 32 * hc));
      // the scale is positive: the scaled maximum is the maximum of the scaled scores
      tmax *= sl2;
      // the maximum after the tile before, from the other group (in the first
      // tile of a piece the wait only keeps the groups in step)
      float mp = -INFINITY;
      if (i > 0) {
        if (!wait_warp(&c->m_ready[wg ^ 1][wq], ((i - 1) >> 1) & 1u, c)) return false;
        if (t > t0) mp = c->m_run[wg ^ 1][r];
      }
      // it moves only when this tile beats it by 2^kLazy
      const float mn = tmax > mp + kLazy ? tmax : mp;
      c->m_run[wg][r] = mn;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->m_ready[wg][wq]);
      const float alpha = mn == mp ? 1.f : exp2f(mp - mn);  // 0 when mp is -inf
      if (mn != m) {
        l *= exp2f(m - mn);
        m = mn;
      }
      const float nmu = m == -INFINITY ? 0.f : kWeightShift - m;

      if (!wait_warp(&c->ps_free[ps], ((i / kPStages) & 1u) ^ 1u, c)) return false;
      const uint32_t pst = smem_u32(smem) + kOffPS + ps * kPBytes + r * 128;
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
        for (int q8 = 0; q8 < 4; ++q8) {
          uint32_t wv[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint64_t x = fma_f32x2(pair(u[8 * q8 + 2 * v], u[8 * q8 + 2 * v + 1]), sl2x2, pair(nmu, nmu));
            const float e0 = ex2_approx(lo_f32(x)), e1 = ex2_approx(hi_f32(x));
            ls = add_f32x2(ls, pair(e0, e1));
            wv[v] = pack_f16(e0, e1);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(pst + (((4 * hc + q8) ^ (r & 7)) << 4)),
                       "r"(wv[0]), "r"(wv[1]), "r"(wv[2]), "r"(wv[3])
                       : "memory");
        }
      }
      l += lo_f32(ls) + hi_f32(ls);
      c->alpha[ps][r] = alpha;
      fence_proxy_async_smem();  // read by the copy engine
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->p_staged[ps]);
    }

    // both groups' sums go to the value CTA relative to the final maximum,
    // which the group of the last tile has
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

// One warp of the score CTA, one thread of it copying: ships each tile's weights and factors to the
// value CTA, where their bytes complete p_full.
__device__ void weight_copier(const Params& p, uint8_t* smem, Ctl* c) {
  const bool leader = elect_one();
  uint32_t j = 0;
  for_pieces(c, [&](const Piece& pc) {
    for (int t = pc.t0; t < pc.t1; ++t, ++j) {
      const uint32_t ps = j % kPStages, pb = j % kPBufs;
      if (!wait_warp(&c->p_staged[ps], (j / kPStages) & 1u, c)) return false;
      if (!wait_warp(&c->p_free[pb], ((j / kPBufs) & 1u) ^ 1u, c)) return false;
      if (leader) {
        const uint32_t bar = mapa_shared(smem_u32(&c->p_full[pb]), 1);
        bulk_copy_s2c(mapa_shared(smem_u32(smem + kOffPV + pb * kPBytes), 1), smem + kOffPS + ps * kPBytes,
                      weight_bytes(live_quads(p.rows, pc.g)), bar);
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
      const uint32_t par = j & 1u, pb = j % kPBufs;
      if (!wait_warp(&c->o_ready[pb], (j / kPBufs) & 1u, c)) return false;
      const uint32_t da = desc_addr(smem, kOffPV + pb * kPBytes) | kDescLoK;
      const uint32_t dv = desc_addr(smem, par * kStageV) | kDescLoV;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!wait_warp(&c->full[2 * par + h], (j >> 1) & 1u, c)) return false;
        tc_fence_after();
        if (leader) {
          // 8-token groups 1 KB apart along K
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_cta_ss(h * 256, desc_at(da + ((kk * 32) >> 4), kDescHiK),
                       desc_at(dv + ((h * kHalf + kk * 16 * 128) >> 4), kDescHiK), kIdescPV,
                       (uint32_t)(kk | (t - pc.t0)));
          mma_cta_commit(&c->empty[2 * par + h]);
          if (h) {
            mma_cta_commit(&c->p_free[pb], 0x1);
            mma_cta_commit(&c->pv_done[pb]);
          }
        }
        __syncwarp();
      }
    }
    return true;
  });
  drain_mmas(c, leader);
}

// Partial results: 8 columns of all rows after each other, so that the rows of
// a warp, one to a lane, fill whole lines (row after row, a warp's store touches
// 32 lines; 32 sequences x 128 heads x 8,192 tokens then took 76.7 us, not 74.3).
__device__ __forceinline__ int64_t part_index(int slot, int block8, int r) {
  return (((int64_t)slot * (kDl / 8) + block8) * kRG + r) * 8;
}

// Row warps of the value CTA (warpgroup h: columns [256 h, 256 h + 256)):
// rescale O where a factor is not 1, and per piece normalise and store it.
__device__ void value_rows(const Params& p, Ctl* c) {
  const int lane = threadIdx.x & 31;
  const int w = (threadIdx.x >> 5) - kWarpRows;
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
      if (w == 0 && lane == 0) mbar_arrive_expect_tx(&c->p_full[pb], weight_bytes(quads) + kRG * 4);
      if (!wait_warp(&c->p_full[pb], (uint32_t)(j / kPBufs) & 1u, c)) return false;
      if (w == 0 && lane == 0) mbar_arrive_cluster_relaxed(&c->ps_free[j % kPStages], 0);
      if (t != t0 && wq < quads) {
        const float a = c->alpha[pb][r];
        if (__any_sync(0xffffffffu, a != 1.f)) {
          if (!wait_warp(&c->pv_done[(j - 1) % kPBufs], (uint32_t)((j - 1) / kPBufs) & 1u, c)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 256; c0 += 32) {
            uint32_t u[32];
            tmem_ld32_sync(tO + c0, u);
#pragma unroll
            for (int q = 0; q < 32; ++q) u[q] = __float_as_uint(__uint_as_float(u[q]) * a);
            tmem_st_32x32b_x32(tO + c0, u);
          }
          tmem_wait_st();
        }
      }
      fence_proxy_async_smem();  // the weights feed the MMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->o_ready[pb]);
    }

    if (!wait_warp(&c->pv_done[(j - 1) % kPBufs], (uint32_t)((j - 1) / kPBufs) & 1u, c)) return false;
    if (!wait_warp(&c->fin_full, (uint32_t)seg & 1u, c)) return false;
    tc_fence_after();
    const float l = c->lfin[0][r] + c->lfin[1][r], m = c->mfin[r];
    // The sums are read before the score CTA may write the next piece's.  Its
    // remote stores are ordered behind these loads by a release at cluster scope
    // only: behind a relaxed arrive, a load held up by a miss of the instruction
    // cache has read the next piece's zero.  The release takes 0.4 us, so a piece
    // that is known to be the cluster's last goes without: nothing waits for it.
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
    if (slot < 0) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * kDl + col0);
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 32) {
        uint32_t u[32];
        __syncwarp();
        tmem_ld32_sync(tO + c0, u);
        if (live) {
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
        }
      }
      if (live && p.lse && h == 0) p.lse[orow] = lse;
    } else {
      float* dst = p.part_o + part_index(slot, col0 / 8, r);
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 32) {
        uint32_t u[32];
        __syncwarp();
        tmem_ld32_sync(tO + c0, u);
        if (live) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            st_global_v8(dst + (c0 / 8 + v) * kRG * 8, __uint_as_float(u[8 * v + 0]) * inv, __uint_as_float(u[8 * v + 1]) * inv,
                         __uint_as_float(u[8 * v + 2]) * inv, __uint_as_float(u[8 * v + 3]) * inv,
                         __uint_as_float(u[8 * v + 4]) * inv, __uint_as_float(u[8 * v + 5]) * inv,
                         __uint_as_float(u[8 * v + 6]) * inv, __uint_as_float(u[8 * v + 7]) * inv);
        }
      }
      if (live && h == 0) p.part_lse[(int64_t)slot * kRG + r] = lse;
    }
    tc_fence_before();
    return true;
  });
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) kvq_attn_kernel(const Params p,
                                                                                              const __grid_constant__ QueryMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5;
  const int cluster = blockIdx.x / 2;
  Ctl* c = reinterpret_cast<Ctl*>(smem + kOffCtl);
  grid_dep_wait();  // launched before the stream's last kernel has ended
  // Barriers, a few per warp.
  if ((threadIdx.x & 31) == 0) {
    if (warp < 4) {
      // the score CTA's second halves wait for every lane's rope copies too
      mbar_init(&c->full[warp], kGroupWarps + (rank == 0 && (warp & 1) ? 32 * kGroupWarps : 0));
      mbar_init(&c->empty[warp], 1);
      mbar_init(&c->m_ready[0][warp], 1);
      mbar_init(&c->m_ready[1][warp], 1);
    } else if (warp < 4 + kSBufs) {
      mbar_init(&c->s_full[warp - 4], 1);
      mbar_init(&c->s_free[warp - 4], kRowWarps / 2);
    } else if (warp < 4 + kSBufs + kPBufs) {
      const int q = warp - 4 - kSBufs;
      mbar_init(&c->p_free[q], 1);
      mbar_init(&c->p_full[q], 1);
      mbar_init(&c->pv_done[q], 1);
      mbar_init(&c->o_ready[q], kRowWarps);
    } else if (warp < 4 + kSBufs + kPBufs + kPStages) {
      const int q = warp - 4 - kSBufs - kPBufs;
      mbar_init(&c->p_staged[q], kRowWarps / 2);
      mbar_init(&c->ps_free[q], 1);
    } else if (warp == 12) {
      mbar_init(&c->q_in, 1);
      mbar_init(&c->fin_free, 32 * kRowWarps);
      mbar_init(&c->fin_full, 32 * kRowWarps);
      mbar_init(&c->drain, 1);
    } else if (warp == 13) {
      for (int q = 0; q < kPieces; ++q) {
        mbar_init(&c->q_ready[q], kRowWarps);
        mbar_init(&c->piece_full[q], 1);
        mbar_init(&c->piece_empty[q], kFollowers + (rank == 0 ? 1 : 0));
      }
    } else if (warp == 14) {
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
  static_assert(4 + kSBufs + kPBufs + kPStages <= 12 && kPStages == 2, "barriers per warp");
  if (warp == kWarpAux) {
    tmem_alloc_cta(&c->tmem_base, kTmemCols);
    tmem_relinquish_cta();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // barriers initialised; the peer's are waited for after the split
  const int n = make_split(p, c, cluster);  // the same n in every CTA
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
  if (warp < kProducerWarps) {
    if (!base0) {
    } else if (rank == 0) {
      producer<true>(p, smem, c, warp);
    } else {
      producer<false>(p, smem, c, warp);
    }
  } else if (warp < kWarpRows + kRowWarps) {
    if (!base0) {
    } else if (rank == 0) {
      score_softmax(p, maps, smem, c, warp);
    } else {
      value_rows(p, c);
    }
  } else {
    if (!base0) {
    } else if (warp == kWarpMma) {
      if (rank == 0) score_mma(smem, c);
      else value_mma(p, smem, c);
    } else if (warp == kWarpAux) {
      if (rank == 0) weight_copier(p, smem, c);
    } else if (warp == kWarpSched) {
      schedule(p, c, cluster);
    }
  }

  __syncwarp();
  grid_dep_launch();  // the merging kernel may start launching; it waits for this grid
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.err[kErrFirst + blockIdx.x] = c->err | (c->abort ? MLA_DEVERR_TIMEOUT : 0u);
  // after an abort nobody has waited for the last copies into the value CTA:
  // give them far longer than they take
  if (c->abort) __nanosleep(100000);
  tc_fence_after();
  cluster_sync();  // no CTA leaves while its peer may still touch its shared memory
  if (warp == kWarpAux) tmem_dealloc_cta(c->tmem_base, kTmemCols);
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// The pieces of a row group that several clusters shared:
//   lse = ln sum_k exp(lse_k),  out = sum_k exp(lse_k - lse) out_k.
// Every block reads where the clusters' intervals begin and lists the row
// groups that a boundary cuts; the blocks then take these eight rows at a time.
// For eight rows a block gathers every piece's slot and lse, a warp per row
// turns them into weights, and each thread sums 8 columns of a row with four
// pieces' loads in flight.  Where that makes at most a quarter as many tasks as
// blocks (few row groups, in many pieces each), a task is a quarter of the
// columns instead, and a quarter of the threads each takes every fourth piece:
// two row groups of 38 pieces took 11 us less, but 32 row groups of two or three
// pieces 10 us more.  (A block for every eight rows behind every boundary, most
// of which find nothing to do, took 6 us longer: several waves of blocks that
// wait for one load each.)
constexpr int kMergeThreads = 512, kMergeRows = 8, kMergeParts = 4;
static_assert(kMergeThreads == kMergeRows * (kDl / 8), "a thread per row and 8 columns");
constexpr int kMaxClusters = 128;
static_assert(2 * kMaxClusters <= kErrMax, "an error word per CTA");
__global__ void __launch_bounds__(kMergeThreads, 2) kvq_merge_kernel(const Params p, int chunks) {
  __shared__ Start start[kMaxClusters];
  __shared__ int cut[kMaxClusters];                    // boundaries that are the first inside a row group
  __shared__ uint32_t cut_mask[kMaxClusters / 32];
  __shared__ int slot[kMaxClusters];                   // -1: an empty piece
  __shared__ float weight[kMergeRows][kMaxClusters];   // each piece's lse, then its weight
  __shared__ float total[kMergeRows];                  // sum of the weights
  __shared__ float4 sums[kMergeParts - 1][2][kMergeThreads / kMergeParts];
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (tid < p.clusters) start[tid] = static_cast<const Start*>(p.starts)[tid];
  __syncthreads();
  const int clusters = start[0].n;
  bool first = false;
  if (tid > 0 && tid < clusters) {
    const Start s0 = start[tid - 1], s = start[tid];
    const int64_t base = div_fast(s.x, kFixed + s.T) * (kFixed + s.T);
    first = s.x > base && (s0.b != s.b || s0.x <= base);
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, first);
  if (lane == 0 && warp < kMaxClusters / 32) cut_mask[warp] = mask;
  __syncthreads();
  // every block lists them in the same order: they share the list
  int cuts = 0;
#pragma unroll
  for (int w = 0; w < kMaxClusters / 32; ++w) {
    if (w == warp && first) cut[cuts + __popc(mask & ((1u << lane) - 1u))] = tid;
    cuts += __popc(cut_mask[w]);
  }
  __syncthreads();
  const int parts = cuts * chunks * kMergeParts <= (int)gridDim.x ? kMergeParts : 1;
  const int items = kMergeThreads / parts, item = tid & (items - 1), part = tid / items;
  for (int task = blockIdx.x; task < cuts * chunks * parts; task += gridDim.x) {
    const int k = cut[task / parts / chunks], r0 = (task / parts % chunks) * kMergeRows;
    const int cb = task % parts;
    const Start s = start[k];
    const int T = s.T, L = kFixed + T;
    const int64_t g = div_fast(s.x, L), base = g * L;
    const int rows = (int)min((int64_t)kRG, p.rows - g * kRG) - r0;
    // pieces: cluster k - 1 has units [0, x_k) of the row group, cluster i >= k [x_i, x_{i+1})
    auto unit = [&](int i) -> int64_t {
      return i < k ? 0 : i >= clusters || start[i].b != s.b || start[i].x - base > L ? L : start[i].x - base;
    };
    bool mine = false, whole = false;
    const int c = k - 1 + tid;
    if (c < clusters) {
      const int64_t z0 = unit(c), z1 = unit(c + 1);
      mine = z0 < L;
      if (mine) {
        const int t0 = cut_tile(z0, T), t1 = cut_tile(z1, T);
        whole = t0 == 0 && t1 == T;
        slot[tid] = t1 > t0 ? 2 * c + (t0 == 0) : -1;
      }
    }
    const int n = __syncthreads_count(mine);
    // when one cluster has it all it stored the results
    if (__syncthreads_or(whole) || rows <= 0) continue;
    // the first pieces' results are on their way while the weights are computed
    constexpr int kDeep = 4;
    const int r = item & 7, block8 = (cb * items + item) >> 3;
    uint32_t v[kDeep][8];
    auto load = [&](int i0) {
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const int i = i0 + d * parts, sl = i < n && r < rows ? slot[i] : -1;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[d][q] = 0u;
        if (sl >= 0) ld_global_v8(p.part_o + part_index(sl, block8, r0 + r), v[d]);
      }
    };
    load(part);
    for (int i = tid; i < n * kMergeRows; i += kMergeThreads) {
      const int pc = i / kMergeRows, r = i % kMergeRows;
      weight[r][pc] = slot[pc] >= 0 && r < rows ? p.part_lse[(int64_t)slot[pc] * kRG + r0 + r] : -INFINITY;
    }
    __syncthreads();
    if (warp < min(rows, kMergeRows)) {
      float* w = weight[warp];
      float m = -INFINITY, sum = 0.f;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, w[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (m == -INFINITY) m = 0.f;  // no piece has any weight
      for (int i = lane; i < n; i += 32) {
        w[i] = __expf(w[i] - m);
        sum += w[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        total[warp] = sum == 0.f ? 1.f : sum;  // then a row of zeros, as from one piece
        if (p.lse && cb == 0) p.lse[(int64_t)s.b * p.rows + g * kRG + r0 + warp] = m + logf(sum);
      }
    }
    __syncthreads();
    uint64_t acc[4] = {0, 0, 0, 0};  // 8 columns, two by two
    for (int i0 = part;;) {
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const int i = i0 + d * parts;
        const float w = i < n ? weight[r][i] : 0.f;  // 0 for an empty piece
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = fma_f32x2(pair(w, w), pair(v[d][2 * q], v[d][2 * q + 1]), acc[q]);
      }
      i0 += kDeep * parts;
      if (i0 >= n) break;
      load(i0);
    }
    if (parts > 1) {
      if (part > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sums[part - 1][h][item] =
              make_float4(lo_f32(acc[2 * h]), hi_f32(acc[2 * h]), lo_f32(acc[2 * h + 1]), hi_f32(acc[2 * h + 1]));
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int o = 0; o < kMergeParts - 1; ++o) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 a = sums[o][h][item];
            acc[2 * h] = add_f32x2(acc[2 * h], pair(a.x, a.y));
            acc[2 * h + 1] = add_f32x2(acc[2 * h + 1], pair(a.z, a.w));
          }
        }
      }
    }
    if (part == 0 && r < rows) {
      const float inv = 1.f / total[r];
      const int64_t orow = (int64_t)s.b * p.rows + g * kRG + r0 + r;
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack_bf16(lo_f32(acc[q]) * inv, hi_f32(acc[q]) * inv);
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * kDl + 8 * block8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncthreads();  // slot, weight and sums are reused
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

float score_factor(const mla_kvq_attn_args& a) {
  return (float)std::ldexp((double)a.scale * 1.4426950408889634, a.cache.exponent);
}

mla_status validate_shape(const mla_kvq_attn_args* a) {
  if (!a) return MLA_ERR_INVALID_ARG;
  if (a->B < 0 || a->Q < 0 || a->H < 1) return MLA_ERR_INVALID_ARG;
  if (a->Q > MLA_MAX_Q) return MLA_ERR_UNSUPPORTED;
  // row numbers of the whole batch are 32-bit coordinates of the query copies
  if ((int64_t)a->H * a->Q > (int64_t)1 << 24 || (int64_t)a->H * a->Q * a->B > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

mla_status validate_call(const mla_kvq_attn_args* a) {
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
  // the factor of the scores in base-2 units: rounded to zero or infinity it
  // would turn masked scores of -inf, or scores of 0, into NaN
  if (!std::isfinite(a->scale) || !(a->scale > 0.f) || !std::isnormal(score_factor(*a))) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

// Two-CTA clusters that can be resident at once on the current device, looked
// up once per device under a lock; 0 when it cannot be had.
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
      cudaFuncSetAttribute(kvq_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemAlloc;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kvq_attn_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = sms / 2;
  }
  if (n > kMaxClusters) n = kMaxClusters;
  cached[dev] = n;
  return n;
}

// The driver's encoder of tensor maps, looked up once.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static std::mutex mu;
  static EncodeTiledFn fn = nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
    else
      cudaGetLastError();
  }
  return fn;
}
bool query_map(CUtensorMap* m, const void* base, int64_t rows, int width, int box_rows) {
  const EncodeTiledFn f = encode_tiled();
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
  size_t starts, part_lse, part_o, total;
};
Layout layout(int clusters) {
  Layout l;
  size_t o = MLA_KVQ_WORKSPACE_BYTES;
  l.starts = o;    o = align256(o + sizeof(Start) * (size_t)clusters);
  l.part_lse = o;  o = align256(o + sizeof(float) * 2 * (size_t)clusters * kRG);
  l.part_o = o;    o = align256(o + sizeof(float) * 2 * (size_t)clusters * kRG * kDl);
  l.total = o;
  return l;
}

Params make_params(const mla_kvq_attn_args* a, void* ws, int clusters) {
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
  int L = 0;
  while (((int64_t)1 << L) < a->page_size) ++L;
  p.page_shift = 31 + L;
  p.page_mul = (uint32_t)((((uint64_t)1 << (31 + L)) + (uint64_t)a->page_size - 1) / (uint64_t)a->page_size);
  p.kv_indptr = a->kv_indptr;
  p.kv_indices = a->kv_indices;
  p.block_table = a->block_table;
  p.max_pages = a->max_pages;
  p.prefix_lens = a->prefix_lens;
  p.tree_parent = a->tree_parent;
  p.window = a->window;
  p.sinks = a->sinks;
  const int e = a->cache.exponent;
  p.qpe_mul = (float)std::ldexp(1.0, -e);
  p.scale_log2 = score_factor(*a);
  p.out_mul = (float)std::ldexp(1.0, e + kF16Shift);
  p.out = a->out;
  p.lse = a->lse;
  p.groups = (p.rows + kRG - 1) / kRG;
  p.box_rows = p.rows < kRG ? p.rows : kRG;
  p.clusters = clusters;
  const Layout l = layout(clusters);
  char* base = static_cast<char*>(ws);
  p.err = reinterpret_cast<uint32_t*>(base);
  p.starts = base + l.starts;
  p.part_lse = reinterpret_cast<float*>(base + l.part_lse);
  p.part_o = reinterpret_cast<float*>(base + l.part_o);
  return p;
}

}  // namespace
}  // namespace kvq
}  // namespace mlav

using namespace mlav;
using namespace mlav::kvq;

extern "C" size_t mla_kvq_attn_workspace_size(const mla_kvq_attn_args* a) {
  if (validate_shape(a) != MLA_OK) return 0;
  const int n = clusters_per_gpu();
  return n > 0 ? layout(n).total : 0;
}

namespace {
mla_status run_attn(const mla_kvq_attn_args* a, void* workspace, size_t ws_bytes, mla_stream_t stream,
                    uint64_t hold_ns) {
  mla_status st = validate_shape(a);
  if (st != MLA_OK) return st;
  if (a->B == 0 || a->Q == 0) return hold_ns ? MLA_ERR_INVALID_ARG : MLA_OK;  // the self-test needs a launch
  st = validate_call(a);
  if (st != MLA_OK) return st;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < MLA_KVQ_WORKSPACE_BYTES) return MLA_ERR_WORKSPACE;
  const int n = clusters_per_gpu();
  if (n < 1) return MLA_ERR_CUDA;
  if (ws_bytes < layout(n).total) return MLA_ERR_WORKSPACE;
  kvq::Params p = make_params(a, workspace, n);
  p.hold = hold_ns != 0;
  p.wait_ns = p.hold ? hold_ns : kWaitLimitNs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // per call: the attribute belongs to the context, which may be a new one
  if (cudaFuncSetAttribute(kvq_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc) != cudaSuccess)
    return MLA_ERR_CUDA;
  QueryMaps maps;
  const int64_t rows = (int64_t)p.B * p.rows;
  if (!query_map(&maps.lat, p.q_lat, rows, kDl, p.box_rows) || !query_map(&maps.pe, p.q_pe, rows, kDr, p.box_rows))
    return MLA_ERR_CUDA;
  if (launch_kernel(kvq_attn_kernel, dim3(2 * n), dim3(kThreads), kSmemAlloc, s, true, p, maps) != cudaSuccess)
    return MLA_ERR_CUDA;
  // two blocks per SM of the clusters, fewer when even n - 1 cut row groups make fewer tasks
  const int chunks = ((p.rows < kRG ? p.rows : kRG) + kMergeRows - 1) / kMergeRows;
  const int tasks = (n - 1) * chunks * kMergeParts;
  const int blocks = tasks < 4 * n ? tasks : 4 * n;
  if (n > 1 && launch_kernel(kvq_merge_kernel, dim3(blocks), dim3(kMergeThreads), 0, s, true, p, chunks) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}
}  // namespace

extern "C" mla_status mla_kvq_attn(const mla_kvq_attn_args* a, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  return run_attn(a, workspace, ws_bytes, stream, 0);
}

extern "C" mla_status mla_kvq_selftest_timeout(const mla_kvq_attn_args* a, void* workspace, size_t ws_bytes,
                                               uint64_t hold_ns, mla_stream_t stream) {
  if (hold_ns == 0 || hold_ns > 1000000000ull) return MLA_ERR_INVALID_ARG;
  return run_attn(a, workspace, ws_bytes, stream, hold_ns);
}
