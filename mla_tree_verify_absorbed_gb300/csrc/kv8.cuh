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

#include <cuda.h>
#include <cuda_fp8.h>

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

// The attention's launch parameters: those of the 4-bit cache's, of which qpe_mul is
// not used, and the blocks.
struct Params : kvq::Params {
  const int32_t* scales;
  Divider block;  // slot -> block
  int box;        // tokens that lie in a row within a page, 16 or 32; 0: fewer
};

// Tensor maps of the queries, [B Q H] rows of 512 and of 64, in boxes of 64 elements
// x Params::box_rows rows.
struct QueryMaps {
  CUtensorMap lat, pe;
};

// Two e4m3 codes as f16 numbers.
__device__ __forceinline__ uint32_t from_e4m3(uint32_t codes) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)codes));
  return d;
}

// A query row of largest magnitude `big` (bf16 bits without sign) times 2^t lies
// within e4m3's 448, its largest element at [2^7, 2^8) or, where its fraction allows
// it, at [2^8, 448].
__device__ __forceinline__ int query_unit(uint32_t big) {
  return max(min(((big & 0x7fu) <= 0x60u ? 135 : 134) - (int)(big >> 7), 120), -120);
}
// The factor of that row's scores, kept a normal number: 0 or infinity would turn
// masked scores of -infinity, or scores of 0, into NaN.
__device__ __forceinline__ float query_factor(float scale_log2, int t) {
  return fminf(fmaxf(scale_log2 * pow2(-t), 1.17549435e-38f), 3.402823466e38f);
}
// Four bf16 elements x 2^t as two e4m3 terms: hi the sign, exponent and three bits
// behind the first of each, lo the other four; hi is NaN in a row that is not finite.
__device__ __forceinline__ void query_terms(uint32_t x0, uint32_t x1, float mul, bool finite, uint32_t& hi,
                                            uint32_t& lo) {
  hi = lo = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t x = k ? x1 : x0, a = x << 16, b = x & 0xffff0000u;
    const float h0 = __uint_as_float(a & 0xfff00000u), h1 = __uint_as_float(b & 0xfff00000u);
    const float l0 = __uint_as_float(a) - h0, l1 = __uint_as_float(b) - h1;
    const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(h0 * mul, h1 * mul), __NV_SATFINITE, __NV_E4M3);
    hi |= (finite ? h : 0x7f7fu) << (16 * k);
    lo |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(l0 * mul, l1 * mul), __NV_SATFINITE, __NV_E4M3) << (16 * k);
  }
}

// The kernel for many query rows (kv8_rows.cu): clusters that a launch can have on the
// current device (0 when it cannot be had), and the launch.
namespace rows {
int clusters_per_gpu();
mla_status launch(Params p, const CUtensorMap& cache, cudaStream_t stream);
}  // namespace rows

mla_status validate_cache(const mla_kv8_cache* c);

}  // namespace kv8
}  // namespace mlav
