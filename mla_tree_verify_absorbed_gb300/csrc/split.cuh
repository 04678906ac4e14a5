// How the quantised caches' attention kernels share out their work: the tiles of
// a sequence, the cut of all row groups' tiles into one interval per worker (a
// cluster of the 4-bit kernel, a CTA of the 8-bit one; "cluster" below), and the
// ring of pieces that the roles of a worker follow.
//
// Row group g of sequence b costs T_b + kFixed units (T_b tiles).  The units of
// all row groups, in order, are cut into equal intervals, one per cluster.  Every
// CTA computes the cut itself from prefix_lens, so there is no planning kernel,
// and equal arguments give equal cuts.
//
// Ctl is a kernel's control block in shared memory; its namespace has
// wait_warp(barrier, parity, Ctl*).
#pragma once

#include "kvq.cuh"
#include "sm100.cuh"

namespace mlav {
namespace kvq {
using namespace sm100;

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

// The tiles of a sequence that any of its nodes sees: [0, ns) and [tw, te).
struct Tiles {
  int ns, tw;
  int T;  // ns + te - tw; 0 for an unused sequence
  int64_t lo;  // positions in [sinks, lo) are seen by no node
};

// a / b for a >= 0, b > 0: a 32-bit division wherever it will do.
static __device__ __noinline__ int64_t div_long(int64_t a, int b) { return a / b; }
__device__ __forceinline__ int64_t div_fast(int64_t a, int b) {
  return a >> 32 ? div_long(a, b) : (int64_t)((uint32_t)a / (uint32_t)b);
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

// What the 8-bit cache's merging kernels share among a block's threads: the row groups
// that several workers have pieces of.  A group's pieces are worker k - 1's, which ends
// there, and those of workers k, k + 1, ..., which begin in it.
template <int kMax>
struct Cuts {
  struct Group {
    int64_t row;         // first output row
    int32_t rows;
    int32_t k, n, head;  // n pieces; the first one's slot (-1: no tiles)
  };
  Start start[kMax];
  Group group[kMax];
  int16_t slot[kMax];    // of the piece that a worker begins with (-1: no tiles)
  uint32_t masks[3][kMax / 32];
  __device__ __forceinline__ int slot_of(const Group& g, int i) const { return i == 0 ? g.head : slot[g.k - 1 + i]; }
};

// The last unused sequence from b on before a used one.  Unused ones are passed
// 128 at a time: one after the other they took 0.18 us each, 204 us for 1,024
// between two short sequences, and the roles' waits ran out behind ten million.
// Not inlined: the smallest calls pay for cold code between the hot (15.6 -> 15.8).
static __device__ __noinline__ int last_unused(const int32_t* prefix_lens, int B, int b) {
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

// pos / page_size by a multiplication that the host prepares: for page_size in
// (2^(L-1), 2^L], ceil(2^(31+L) / page_size) fits 32 bits and is off by less than
// 2^L over 2^(31+L), too little to matter for pos < 2^31.  Page size 1 needs no
// branch, and the producers' loops stay short.
__device__ __forceinline__ uint32_t page_of(const Params& p, uint32_t pos) {
  return (uint32_t)(((uint64_t)pos * p.page_mul) >> p.page_shift);
}

// Calls f(piece) for the pieces of the ring in order; f's piece stays valid
// only as far as f copied it.  Every lane of the warp takes part.
template <class Ctl, class F>
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

// Kernels that give a cluster of two CTAs 128 query rows: the most clusters, and where
// partial results lie: 8 columns of all rows after each other, so that the rows of a
// warp, one to a lane, fill whole lines (row after row, a warp's store touches 32 lines;
// 32 sequences x 128 heads x 8,192 tokens then took 76.7 us, not 74.3).
constexpr int kRows128 = 128, kMaxClusters = 128;
__device__ __forceinline__ int64_t part_index(int slot, int block8, int r) {
  return (((int64_t)slot * (kDl / 8) + block8) * kRows128 + r) * 8;
}

// kTK tokens per tile, kThreads threads per CTA; kFixed units for a row group or a
// piece of one beside its tiles, and kMinTiles tiles at least for a cluster.
template <int kTK, int kFixed, int kMinTiles, int kThreads, bool kHeadFirst>
struct Split {
  __device__ __forceinline__ static Tiles tiles_of(const Params& p, int64_t P) {
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
  __device__ __forceinline__ static int cut_tile(int64_t z, int T) {
    return z <= kFixed ? 0 : z >= kFixed + T ? T : (int)(z - kFixed);
  }

  // Clusters that share `total` units.
  __device__ __forceinline__ static int active_clusters(const Params& p, int64_t total) {
    const int64_t n = div_fast(total, kFixed + kMinTiles);
    return (int)(n < 1 ? 1 : n > p.clusters ? p.clusters : n);
  }

  // Scheduler warp of each CTA: writes this cluster's pieces in order, then an
  // end mark, into the ring that the other roles follow.  A piece that does not
  // begin its row group is the cluster's first, one that does not end it the
  // last, so two partial slots are enough.  kHeadFirst puts that first piece at the
  // end: the clusters then begin near the beginning of a row group each, and read
  // the tokens that several row groups share at about the same time.
  template <class Ctl>
  __device__ static void schedule(const Params& p, Ctl* c, int cluster) {
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
    Piece tail = {};  // without tiles: none
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
        if (kHeadFirst && pc.t0 > 0) {
          tail = pc;
          continue;
        }
        if (pc.t1 > pc.t0 && !put(pc)) return;
      }
    }
    if (kHeadFirst && tail.t1 > tail.t0 && !put(tail)) return;
    Piece end = {};
    end.b = -1;
    put(end);
  }

  // Block-wide: validates every sequence, sums the units and finds where this
  // cluster's interval begins.  Returns the clusters that share the call, 0 when
  // a table is bad, -1 when every sequence is unused.  Threads take consecutive
  // sequences.
  template <class Ctl>
  __device__ static int make_split(const Params& p, Ctl* c, int cluster) {
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

  // Lists in every block, in the same order, the row groups of kRG rows that no worker has
  // all tiles of (the others' results are stored); returns how many.  All threads call it,
  // at least kMax of them.
  template <int kRG, int kMax>
  __device__ __forceinline__ static int list_cuts(const Params& p, Cuts<kMax>* c) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < p.clusters) c->start[tid] = static_cast<const Start*>(p.starts)[tid];
    __syncthreads();
    const int workers = c->start[0].n;
    bool first = false, more = false, whole = false;
    int head = -1;
    int64_t g = 0;
    Start s = {};
    if (tid > 0 && tid < workers) {
      const Start s0 = c->start[tid - 1], s1 = c->start[min(tid + 1, workers - 1)];
      s = c->start[tid];
      const int L = kFixed + s.T;
      g = div_fast(s.x, L);
      const int64_t base = g * L;
      first = s.x > base && (s0.b != s.b || s0.x <= base);  // the group's first boundary
      more = s.x > base && !first;
      const bool ends = tid + 1 < workers && s1.b == s.b && s1.x - base <= L;
      const int u0 = cut_tile(s.x - base, s.T), u1 = cut_tile(ends ? s1.x - base : L, s.T);
      c->slot[tid] = (int16_t)(u1 > u0 ? 2 * tid + (u0 == 0) : -1);
      whole = (u0 == 0 && u1 == s.T) || (first && u0 == s.T);
      head = u0 > 0 ? 2 * tid - 1 : -1;
    }
    const uint32_t more_mask = __ballot_sync(0xffffffffu, more), whole_mask = __ballot_sync(0xffffffffu, whole);
    if (lane == 0 && warp < kMax / 32) {
      c->masks[0][warp] = more_mask;
      c->masks[1][warp] = whole_mask;
    }
    __syncthreads();
    int end = tid + 1;
    if (first) {
      while (end < workers && (c->masks[0][end >> 5] >> (end & 31)) & 1u) {
        whole |= (c->masks[1][end >> 5] >> (end & 31)) & 1u;
        ++end;
      }
    }
    first = first && !whole;
    const uint32_t mask = __ballot_sync(0xffffffffu, first);
    if (lane == 0 && warp < kMax / 32) c->masks[2][warp] = mask;
    __syncthreads();
    int cuts = 0;
#pragma unroll
    for (int w = 0; w < kMax / 32; ++w) {
      if (w == warp && first)
        c->group[cuts + __popc(mask & ((1u << lane) - 1u))] = {
            (int64_t)s.b * p.rows + g * kRG, (int32_t)min((int64_t)kRG, p.rows - g * kRG), tid, end - tid + 1, head};
      cuts += __popc(c->masks[2][w]);
    }
    __syncthreads();
    return cuts;
  }
};

}  // namespace kvq
}  // namespace mlav
