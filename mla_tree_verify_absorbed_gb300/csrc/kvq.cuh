// Shared definitions of the 4-bit latent cache: the packed row, the codes'
// conversion to the two operand types, the launch parameter block of the
// attention, and the per-call error words.
//
// A row (include/mla_kvq.h) stands for latents (code - 8) * scale * 2^exponent.
// code - 8 has at most 4 significant bits and an e4m3 scale 4, so the product
// fits the 8 bits of bf16 and the 11 of f16 (magnitudes 2^-9 .. 3840): both
// conversions are exact, and the exponent is applied outside the products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mla_kvq.h"
#include "common.cuh"

namespace mlav {
namespace kvq {

constexpr int kCodeBytes = 256;                // 512 codes
constexpr int kScaleOff = kCodeBytes;          // 32 scales
constexpr int kRopeOff = kCodeBytes + 32;      // 64 bf16
static_assert(kRopeOff + 2 * kDr == MLA_KVQ_ROW_BYTES, "row layout");

// ---------------------------------------------------------------------------
// Error words.  Word 0 of a workspace holds the number of words that the call
// uses from kErrFirst on; every block (or cluster) stores its own, so nothing
// needs clearing before a call and no atomics are involved.
// ---------------------------------------------------------------------------
constexpr int kErrFirst = 16;  // first error word
constexpr int kErrMax = (int)(MLA_KVQ_WORKSPACE_BYTES / 4) - kErrFirst;

// ---------------------------------------------------------------------------
// Codes to values.  Nibble pair t of a code word (bits 4t.. of both halves) is
// put into the mantissa of a number whose exponent is fixed, so that each
// half reads base + code exactly; one fused multiply-add then gives
// (base + code) * s - (base + 8) * s = (code - 8) * s, exact because the
// product is formed without rounding and the constant (base + 8) * s is exact
// too: bf16, base 128, 136 s has 5 + 4 bits less one, 8 of 8; f16, bases 1024
// and 64, 1032 s has 8 + 4 bits less one, 11 of 11, and 72 s 8.  Lowest bits
// first, a code needs no shift (bf16: one of four; f16, whose mantissa holds two
// codes: two of four, the others share one).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(m), "r"(o));  // (a & m) | o
  return d;
}
__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hfma2_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// bf16 operand values.
struct ToBf16 {
  // two scale bytes (bits 0-7 and 16-23 of b) as bf16 pair: the e4m3 field
  // shifted to the bottom of the bf16 exponent is the magnitude times 2^-120
  __device__ __forceinline__ static uint32_t scales(uint32_t b) {
    return hmul2_bf16((b << 4) & 0x07F007F0u, 0x7B807B80u);  // * 2^120
  }
  __device__ __forceinline__ static uint32_t offsets(uint32_t s) { return hmul2_bf16(s, 0xC308C308u); }  // -136 s
  // the eight values of a code word, in element order; s one scale twice
  __device__ __forceinline__ static void word(uint32_t w, uint32_t s, uint32_t o, uint32_t (&v)[4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = hfma2_bf16(and_or(w >> (4 * t), 0x000F000Fu, 0x43004300u), s, o);
  }
};

// f16 operand values, times 2^-kF16Shift: 1032 s has to stay below 65504.  The
// smallest, 2^-13, is still a normal number.
constexpr int kF16Shift = 4;
struct ToF16 {
  // the e4m3 field in the f16 exponent and mantissa is the magnitude times 2^-8
  __device__ __forceinline__ static uint32_t scales(uint32_t b) {
    return hmul2_f16((b << 7) & 0x3F803F80u, 0x4C004C00u);  // * 2^(8 - kF16Shift)
  }
  __device__ __forceinline__ static uint32_t offsets(uint32_t s) { return hmul2_f16(s, 0xE408E408u); }   // -1032 s
  __device__ __forceinline__ static uint32_t offsets2(uint32_t s) { return hmul2_f16(s, 0xD480D480u); }  // -72 s
  __device__ __forceinline__ static void word(uint32_t w, uint32_t s, uint32_t o, uint32_t (&v)[4]) {
    const uint32_t u = w >> 8, o2 = offsets2(s);
    v[0] = hfma2_f16(and_or(w, 0x000F000Fu, 0x64006400u), s, o);
    v[1] = hfma2_f16(and_or(w, 0x00F000F0u, 0x54005400u), s, o2);
    v[2] = hfma2_f16(and_or(u, 0x000F000Fu, 0x64006400u), s, o);
    v[3] = hfma2_f16(and_or(u, 0x00F000F0u, 0x54005400u), s, o2);
  }
};

// One half of a pair in both halves.
__device__ __forceinline__ uint32_t lo2(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t hi2(uint32_t x) { return __byte_perm(x, x, 0x3232); }

// ---------------------------------------------------------------------------
// The attention's launch parameters
// ---------------------------------------------------------------------------
struct Params {
  int B, Q, H;
  int rows;  // H * Q rows per sequence; row r = node (r / H), head (r % H)
  const uint8_t* cache;
  int64_t row_stride, slots;
  const void* q_lat;
  const void* q_pe;
  int page_size;
  uint32_t page_mul;  // pos / page_size = pos * page_mul >> page_shift
  int page_shift;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* block_table;
  int max_pages;
  const int32_t* prefix_lens;
  const int32_t* tree_parent;  // NULL: chain
  int window, sinks;           // window 0: none
  float qpe_mul;               // 2^-exponent, on the rope queries
  float scale_log2;            // scale * 2^exponent * log2(e): scores in base-2 units
  float out_mul;               // 2^(exponent + kF16Shift)
  void* out;
  float* lse;
  int groups;                  // row groups per sequence
  int box_rows;                // rows of a query copy: those of a row group, or of a sequence that has fewer
  int clusters;                // clusters launched
  uint64_t wait_ns;            // how long a device wait may take
  bool hold;                   // failure-detection self-test only: the value product never starts
  // workspace
  uint32_t* err;               // word 0, and the error words from kErrFirst on
  void* starts;                // [clusters]: see Start
  float* part_lse;             // [2 clusters][rows of a group], natural log
  float* part_o;               // [2 clusters][512 / 8][rows of a group][8], normalised
};

// What a call needs of sequence b's tables before anything else, and the
// MLA_DEVERR_* bits they deserve.  With kv_indptr[0] == 0 and every span equal
// to its sequence's length, all reads stay in kv_indices[0 .. kv_indptr[B]).
struct Sequence {
  int32_t P;      // prefix length; -1: unused
  int64_t entry;  // its first table entry
  uint32_t err;
};
__device__ __forceinline__ Sequence read_sequence(const Params& p, int b) {
  Sequence s;
  s.P = p.prefix_lens[b];
  int64_t lo = 0, hi = 0;
  if (p.page_size == 1) {
    lo = p.kv_indptr[b];
    hi = p.kv_indptr[b + 1];
  }
  s.err = s.P < -1 ? MLA_DEVERR_PREFIX : 0u;
  const int64_t N = s.P < 0 ? 0 : (int64_t)s.P + p.Q;
  if (p.page_size == 1) {
    s.entry = lo;
    if ((b == 0 && lo != 0) || lo < 0 || hi - lo != N) s.err |= MLA_DEVERR_INDPTR;
  } else {
    s.entry = (int64_t)b * p.max_pages;
    if (N > (int64_t)p.max_pages * p.page_size) s.err |= MLA_DEVERR_PAGES;
  }
  return s;
}

// What one node sees of the tree: the mask of its visible nodes and its depth.
struct NodeView {
  uint64_t mask;  // bit t: node t is the node itself or a visible ancestor
  int depth;      // 0 for a node without parent
};

// Node i of sequence b, for every lane of a warp at once (lanes may name
// different nodes, or the same).  The warp holds the sequence's parents two to
// a lane, so a step up is a shuffle rather than a load that waits for the one
// before.  A link outside [-1, t-1] sets *bad and ends the walk.
// A window drops ancestors at least `window` places back unless their place
// P + depth is among the first `sinks`: ancestors have smaller indices than
// their descendants, so the k-th highest bit is the ancestor k places back, at
// depth n - k.
__device__ __forceinline__ NodeView node_view_warp(const Params& p, int b, int i, int64_t P, bool* bad) {
  NodeView v;
  if (!p.tree_parent) {
    v.mask = ~0ull >> (63 - i);
    v.depth = i;
  } else {
    const int lane = threadIdx.x & 31;
    const int32_t* par = p.tree_parent + (int64_t)b * p.Q;
    const int lo = lane < p.Q ? par[lane] : -1, hi = lane + 32 < p.Q ? par[lane + 32] : -1;
    v.mask = 1ull << i;
    v.depth = 0;
    int cur = i;
    bool more = true;
    while (__any_sync(0xffffffffu, more)) {
      const int a = __shfl_sync(0xffffffffu, lo, cur & 31), c = __shfl_sync(0xffffffffu, hi, cur & 31);
      const int up = cur < 32 ? a : c;
      if (more && (up < -1 || up >= cur)) *bad = true;
      more = more && up >= 0 && up < cur;
      if (more) {
        v.mask |= 1ull << up;
        cur = up;
        ++v.depth;
      }
    }
  }
  if (p.window > 0 && v.depth >= p.window) {
    uint64_t left = v.mask, keep = 0;
    for (int k = 0; left; ++k) {
      const int t = 63 - __clzll((long long)left);
      left &= ~(1ull << t);
      if (k < p.window || P + (v.depth - k) < p.sinks) keep |= 1ull << t;
    }
    v.mask = keep;
  }
  return v;
}

}  // namespace kvq
}  // namespace mlav
