// Shared definitions of the paged 8-bit latent cache: the row, the blocks'
// scale words and the attention's launch parameters.
//
// A row (include/mla_kv8.h) holds 512 e4m3 codes and 64 bf16 rope values, both in
// units of 2^(exponent + k); k belongs to the row's block of pool slots.  The unit
// is a power of two, so a block's rows move to a larger unit exactly (but for what
// falls below the smallest code), and e4m3's relative precision does not depend on
// where in a power of two the largest value lies, as that of evenly spaced codes
// would.
#pragma once

#include "../../include/mla_kv8.h"
#include "kvq.cuh"

namespace mlav {
namespace kv8 {

constexpr int kRopeOff = kDl;  // bytes of codes
static_assert(kRopeOff + 2 * kDr == MLA_KV8_ROW_BYTES, "row layout");
constexpr int kMaxK = MLA_KV8_MAX_SCALE;

// A block's scale word: k + 1 once it holds rows, 0 before.  During a write the
// bits from kPendingShift on hold what the new rows need, in the same form.
constexpr int kPendingShift = 8;
constexpr uint32_t kScaleMask = (1u << kPendingShift) - 1u;

// k of a scale word, whatever is in it.
__device__ __forceinline__ int scale_of(uint32_t word) { return min(max((int)(word & kScaleMask) - 1, 0), kMaxK); }
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// x / d for 0 <= x < 2^31 by a multiplication: for d in (2^(L-1), 2^L],
// ceil(2^(31+L) / d) fits 32 bits and is off by less than 2^L over 2^(31+L).
struct Divider {
  uint32_t mul;
  int shift;
  __host__ void set(int64_t d) {
    int L = 0;
    while (((int64_t)1 << L) < d) ++L;
    shift = 31 + L;
    mul = (uint32_t)((((uint64_t)1 << shift) + (uint64_t)d - 1) / (uint64_t)d);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (uint32_t)(((uint64_t)x * mul) >> shift); }
};

// The attention's launch parameters: those of the 4-bit cache's, of which
// qpe_mul and box_rows are not used, and the blocks.
struct Params : kvq::Params {
  const int32_t* scales;
  Divider block;  // slot -> block
  int box;        // tokens that lie in a row within a page, at most 32; 0: fewer than 8
};

mla_status validate_cache(const mla_kv8_cache* c);

}  // namespace kv8
}  // namespace mlav
