// Writing rows of the 4-bit latent cache and reading them back
// (mla_kvq_write, mla_kvq_read, mla_kvq_check).
//
// Write.  Per block of 16 latents x:  s = e4m3(max|x| / 7),  q = rint(x / s).
// Both roundings are decided as if nothing had been rounded before:
//   * the tie points of q are t s with t = k + 1/2, at most 4 + 4 significant
//     bits, so on the grid of fp32 numbers around x; a quotient x / s that is
//     not t differs from it by more than 2^-24 relative, and the correctly
//     rounded fp32 quotient lies on the same side;
//   * the quotient is x * (1/s) corrected by one residual step
//     q1 = q0 + (x - q0 s) * (1/s), correctly rounded when 1/s is (Markstein,
//     "Computation of elementary functions on the IBM RISC System/6000
//     processor", 1990): three multiply-adds per element in place of a division;
//   * max|x| / 7 is one fp32 division per block; the same argument holds for
//     the e4m3 tie points (5 bits, times 7: 8 bits).
// Read is the exact conversion of kvq.cuh.
//
// Bound: HBM.  A bf16 row is 1152 bytes on one side and 416 on the other; one
// warp takes a row, lane l its scale block l.  Measured on 200,000 rows in
// random slots (us; GB/s of both sides): bf16 write 60 (5,270), fp32 write 82
// (6,660), bf16 read 52 (6,100), fp32 read 86 (6,350).  The bf16 write is held
// by its instructions rather than by HBM.
#include <cuda_fp8.h>

#include "io.cuh"
#include "kvq.cuh"
#include "sm100.cuh"

namespace mlav {
namespace kvq {

struct IoParams {
  uint8_t* cache;
  int64_t row_stride, slots;
  float mul, inv_mul;  // 2^exponent, 2^-exponent
  int64_t n;
  const int32_t* slot;
  void* kv_c;
  void* k_pe;
  int64_t kv_c_stride, k_pe_stride;  // elements
  bool wide;                         // kv_c rows are 32-byte aligned
  uint32_t* err;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The 16 latents of one scale block: as fp32, two by two, and the largest
// magnitude (NaN when there is one).
template <class T>
struct Block16;
template <>
struct Block16<__nv_bfloat16> {
  uint32_t v[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool wide) { ld_words(p, wide, v); }
  __device__ __forceinline__ uint64_t two(int i) const { return sm100::pair(v[i] << 16, v[i] & 0xffff0000u); }
  __device__ __forceinline__ float largest() const {
    uint32_t m = v[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan_bf16x2(m, v[i] & 0x7fff7fffu);
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
template <>
struct Block16<float> {
  uint32_t v[2][8];
  __device__ __forceinline__ void load(const float* p, bool wide) {
    ld_words(p, wide, v[0]);
    ld_words(p + 8, wide, v[1]);
  }
  __device__ __forceinline__ uint64_t two(int i) const {
    return sm100::pair(v[i >> 2][2 * (i & 3)], v[i >> 2][2 * (i & 3) + 1]);
  }
  __device__ __forceinline__ float largest() const {
    float m = fabsf(__uint_as_float(v[0][0]));
#pragma unroll
    for (int i = 1; i < 16; ++i) m = max_nan(m, fabsf(__uint_as_float(v[i >> 3][i & 7])));
    return m;
  }
};

// The number whose fp32 bits end in the 4-bit code of q = x / s: adding
// 1.5 * 2^23 + 8 rounds q to an integer, ties to even, in the low bits.
constexpr float kRound = 12582912.f + 8.f;
constexpr uint32_t kRoundBits = 0x4B400000u;  // bits of 1.5 * 2^23
// nibble position of element i of a word, and the sum of what the bits above
// the codes add when eight shifted numbers are summed (mod 2^32)
__host__ __device__ constexpr int nib_shift(int i) { return 4 * (i >> 1) + 16 * (i & 1); }
constexpr uint32_t kRoundSum = kRoundBits * 0x11111111u;

// Quantises one block: two code words and the scale byte; false in *finite
// when a value was infinite or NaN.
template <class T>
__device__ __forceinline__ void quantise(const Block16<T>& x, float mul, float inv_mul, uint32_t (&w)[2],
                                         uint32_t& byte, bool* finite) {
  const float a = x.largest();
  const float as = a * inv_mul;
  byte = (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(fminf(as, 4096.f), 7.f), __NV_SATFINITE, __NV_E4M3);
  w[0] = w[1] = 0u - kRoundSum;
  if (byte >= 8u && as <= 3248.f) {
    // a normal scale is within 1/16 of max|x| / 7, so |q| < 7.5 without a clamp
    const float s = __uint_as_float((byte << 20) + (120u << 23)) * mul;  // e4m3 normal as fp32
    const float inv = __frcp_rn(s);
    const uint64_t s2 = sm100::pair(-s, -s), inv2 = sm100::pair(inv, inv), round2 = sm100::pair(kRound, kRound);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t v = x.two(i);
      const uint64_t q0 = sm100::mul_f32x2(v, inv2);
      const uint64_t q1 = sm100::fma_f32x2(sm100::fma_f32x2(q0, s2, v), inv2, q0);
      const uint64_t c = sm100::add_f32x2(q1, round2);
      w[i >> 2] += (uint32_t)c << nib_shift(2 * (i & 3));
      w[i >> 2] += (uint32_t)(c >> 32) << nib_shift(2 * (i & 3) + 1);
    }
    return;
  }
  // scale 0, subnormal or at its largest, infinities, NaN
  if (!(a <= 3.402823466e38f)) {
    *finite = false;
    float m = 0.f;  // the block's maximum without NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(sm100::lo_f32(x.two(i))), fabsf(sm100::hi_f32(x.two(i)))));
    byte = (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(fminf(m * inv_mul, 4096.f), 7.f), __NV_SATFINITE, __NV_E4M3);
  }
  const float s = byte >= 8u ? __uint_as_float((byte << 20) + (120u << 23)) : (float)byte * 0.001953125f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = ((i & 1) ? sm100::hi_f32(x.two(i >> 1)) : sm100::lo_f32(x.two(i >> 1))) * inv_mul;
    v = v == v ? fminf(fmaxf(v, -4096.f), 4096.f) : 0.f;
    const float q = byte ? fminf(fmaxf(__fdiv_rn(v, s), -7.f), 7.f) : 0.f;
    w[i >> 3] += __float_as_uint(q + kRound) << nib_shift(i & 7);
  }
}

template <class T>
__device__ __forceinline__ uint32_t rope_pair(const T* p);
template <>
__device__ __forceinline__ uint32_t rope_pair(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}
template <>
__device__ __forceinline__ uint32_t rope_pair(const float* p) {
  const float2 f = *reinterpret_cast<const float2*>(p);
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One warp per row, kDeep rows in flight per warp: for 200,000 rows 1, 2 and 4
// took 63, 60 and 72 us from bf16, 82, 85 and 123 from fp32, whose rows are
// twice as long and at 4 leave too few warps.
template <class T, int kDeep>
__global__ void __launch_bounds__(kIoThreads) kvq_write_kernel(const IoParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kIoWarps + (threadIdx.x >> 5);
  const int64_t nwarps = (int64_t)gridDim.x * kIoWarps;
  grid_dep_wait();  // launched before the stream's last kernel has ended
  grid_dep_launch();
  uint32_t e = 0;
  for (int64_t i0 = warp; i0 < p.n; i0 += kDeep * nwarps) {
    int64_t slot[kDeep];
    Block16<T> x[kDeep];
    uint32_t rope[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t i = i0 + d * nwarps;
      slot[d] = i < p.n ? p.slot[i] : -1;
      if (slot[d] < -1 || slot[d] >= p.slots) {
        e |= MLA_DEVERR_SLOT;
        slot[d] = -1;
      }
      if (slot[d] >= 0) {
        x[d].load(static_cast<const T*>(p.kv_c) + i * p.kv_c_stride + 16 * lane, p.wide);
        rope[d] = rope_pair(static_cast<const T*>(p.k_pe) + i * p.k_pe_stride + 2 * lane);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (slot[d] < 0) continue;
      uint32_t w[2], byte;
      bool finite = true;
      quantise(x[d], p.mul, p.inv_mul, w, byte, &finite);
      if (!finite) e |= MLA_DEVERR_NONFINITE;
      uint8_t* row = p.cache + slot[d] * p.row_stride;
      reinterpret_cast<uint2*>(row)[lane] = make_uint2(w[0], w[1]);
      row[kScaleOff + lane] = (uint8_t)byte;
      reinterpret_cast<uint32_t*>(row + kRopeOff)[lane] = rope[d];
    }
  }
  put_block_err(p.err, e);
}

__device__ __forceinline__ void put_latents(__nv_bfloat16* dst, const uint32_t (&v)[8], float, bool wide) {
  st_words(dst, wide, v);
}
__device__ __forceinline__ void put_latents(float* dst, const uint32_t (&v)[8], float mul, bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __float_as_uint(__uint_as_float(v[4 * h + i] << 16) * mul);
      f[2 * i + 1] = __float_as_uint(__uint_as_float(v[4 * h + i] & 0xffff0000u) * mul);
    }
    st_words(dst + 8 * h, wide, f);
  }
}
__device__ __forceinline__ void put_rope(__nv_bfloat16* dst, uint32_t v) { *reinterpret_cast<uint32_t*>(dst) = v; }
__device__ __forceinline__ void put_rope(float* dst, uint32_t v) {
  *reinterpret_cast<float2*>(dst) = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Two rows in flight per warp: for 200,000 rows 1, 2 and 4 took 63, 52 and 53 us
// to bf16, 86 each to fp32.
template <class T, int kDeep>
__global__ void __launch_bounds__(kIoThreads) kvq_read_kernel(const IoParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kIoWarps + (threadIdx.x >> 5);
  const int64_t nwarps = (int64_t)gridDim.x * kIoWarps;
  // the exponent in bf16: a power of two, exact
  const __nv_bfloat16 mb = __float2bfloat16_rn(p.mul);
  const uint32_t mul2 = (uint32_t)__bfloat16_as_ushort(mb) * 0x10001u;
  grid_dep_wait();  // launched before the stream's last kernel has ended
  grid_dep_launch();
  uint32_t e = 0;
  for (int64_t i0 = warp; i0 < p.n; i0 += kDeep * nwarps) {
    int64_t slot[kDeep];
    uint2 w[kDeep];
    uint32_t byte[kDeep], rope[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t i = i0 + d * nwarps;
      slot[d] = i < p.n ? p.slot[i] : -1;
      if (slot[d] < -1 || slot[d] >= p.slots) {
        e |= MLA_DEVERR_SLOT;
        slot[d] = -1;
      }
      if (slot[d] >= 0) {
        const uint8_t* row = p.cache + slot[d] * p.row_stride;
        w[d] = reinterpret_cast<const uint2*>(row)[lane];
        byte[d] = row[kScaleOff + lane];
        rope[d] = reinterpret_cast<const uint32_t*>(row + kRopeOff)[lane];
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (slot[d] < 0) continue;
      const int64_t i = i0 + d * nwarps;
      const uint32_t s = ToBf16::scales(byte[d] | byte[d] << 16);
      const uint32_t o = ToBf16::offsets(s);
      uint32_t a[4], b[4];
      ToBf16::word(w[d].x, s, o, a);
      ToBf16::word(w[d].y, s, o, b);
      uint32_t v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      if (sizeof(T) == 2) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = hmul2_bf16(v[q], mul2);
      }
      put_latents(static_cast<T*>(p.kv_c) + i * p.kv_c_stride + 16 * lane, v, p.mul, p.wide);
      put_rope(static_cast<T*>(p.k_pe) + i * p.k_pe_stride + 2 * lane, rope[d]);
    }
  }
  put_block_err(p.err, e);
}

mla_status validate_cache(const mla_kvq_cache* c) {
  if (!c || !c->rows || (reinterpret_cast<uintptr_t>(c->rows) & 31u)) return MLA_ERR_INVALID_ARG;
  if (c->row_stride < MLA_KVQ_ROW_BYTES || (c->row_stride & 31) || c->row_stride > INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  if (c->slots < 1 || c->slots > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (c->exponent < -MLA_KVQ_MAX_EXPONENT || c->exponent > MLA_KVQ_MAX_EXPONENT) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

namespace {

float pow2(int e) {
  float f = 1.f;
  for (; e > 0; --e) f *= 2.f;
  for (; e < 0; ++e) f *= 0.5f;
  return f;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks shared by both directions; *noop when there is nothing to launch.
mla_status make_io(const mla_kvq_cache* c, const mla_kvq_rows* r, void* ws, size_t ws_bytes, IoParams* p, bool* noop) {
  mla_status st = validate_cache(c);
  if (st != MLA_OK) return st;
  if (!r || r->n < 0 || r->n > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (r->dtype != MLA_BF16 && r->dtype != MLA_FP32) return MLA_ERR_INVALID_ARG;
  *noop = r->n == 0;
  if (*noop) return MLA_OK;
  const int64_t el = r->dtype == MLA_BF16 ? 2 : 4;
  if (!r->kv_c || !r->k_pe || !r->slots) return MLA_ERR_INVALID_ARG;
  if (!aligned(r->kv_c, 16) || !aligned(r->k_pe, 16) || !aligned(r->slots, 4)) return MLA_ERR_INVALID_ARG;
  // row strides beyond 2^31 elements would let row offsets pass 64 bits
  if (r->kv_c_stride < kDl || r->k_pe_stride < kDr || r->kv_c_stride > INT32_MAX || r->k_pe_stride > INT32_MAX ||
      (r->kv_c_stride * el) % 16 || (r->k_pe_stride * el) % 16)
    return MLA_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || ws_bytes < MLA_KVQ_WORKSPACE_BYTES) return MLA_ERR_WORKSPACE;
  p->cache = static_cast<uint8_t*>(c->rows);
  p->row_stride = c->row_stride;
  p->slots = c->slots;
  p->mul = pow2(c->exponent);
  p->inv_mul = pow2(-c->exponent);
  p->n = r->n;
  p->slot = r->slots;
  p->kv_c = r->kv_c;
  p->k_pe = r->k_pe;
  p->kv_c_stride = r->kv_c_stride;
  p->k_pe_stride = r->k_pe_stride;
  p->wide = aligned(r->kv_c, 32) && (r->kv_c_stride * el) % 32 == 0;
  p->err = static_cast<uint32_t*>(ws);
  return MLA_OK;
}

}  // namespace
}  // namespace kvq
}  // namespace mlav

using namespace mlav;
using namespace mlav::kvq;

extern "C" mla_status mla_kvq_write(const mla_kvq_cache* cache, const mla_kvq_rows* src, void* workspace,
                                    size_t ws_bytes, mla_stream_t stream) {
  IoParams p;
  bool noop = false;
  mla_status st = make_io(cache, src, workspace, ws_bytes, &p, &noop);
  if (st != MLA_OK || noop) return st;
  int grid = 0;
  st = io_grid(p.n, 8, &grid);
  if (st != MLA_OK) return st;
  const auto kernel = src->dtype == MLA_BF16 ? kvq_write_kernel<__nv_bfloat16, 2> : kvq_write_kernel<float, 1>;
  const cudaError_t e = launch_kernel(kernel, dim3(grid), dim3(kIoThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                                      true, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_kvq_read(const mla_kvq_cache* cache, const mla_kvq_rows* dst, void* workspace,
                                   size_t ws_bytes, mla_stream_t stream) {
  IoParams p;
  bool noop = false;
  mla_status st = make_io(cache, dst, workspace, ws_bytes, &p, &noop);
  if (st != MLA_OK || noop) return st;
  int grid = 0;
  st = io_grid(p.n, 16, &grid);
  if (st != MLA_OK) return st;
  const auto kernel = dst->dtype == MLA_BF16 ? kvq_read_kernel<__nv_bfloat16, 2> : kvq_read_kernel<float, 2>;
  const cudaError_t e = launch_kernel(kernel, dim3(grid), dim3(kIoThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                                      true, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_kvq_check(const void* workspace, mla_stream_t stream, uint32_t* bits) {
  if (!workspace) return MLA_ERR_WORKSPACE;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_CUDA;
  uint32_t n = 0, v = 0;
  if (cudaMemcpy(&n, workspace, sizeof(n), cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
  if (n > (uint32_t)kErrMax) return MLA_ERR_WORKSPACE;  // no call of this header has used it
  uint32_t words[kErrMax];
  if (n > 0 && cudaMemcpy(words, static_cast<const uint32_t*>(workspace) + kErrFirst, n * sizeof(uint32_t),
                          cudaMemcpyDeviceToHost) != cudaSuccess)
    return MLA_ERR_CUDA;
  for (uint32_t i = 0; i < n; ++i) v |= words[i];
  if (bits) *bits = v;
  return v ? MLA_ERR_DEVICE_CHECK : MLA_OK;
}
