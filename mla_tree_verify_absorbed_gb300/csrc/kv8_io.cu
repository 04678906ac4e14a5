// Writing rows of the paged 8-bit latent cache and reading them back
// (mla_kv8_write, mla_kv8_read, mla_kv8_check).
//
// Write.  A block's unit depends on all rows that go to it, so a write is three
// kernels: the first gathers what every block's new rows need (an integer maximum
// per block, the same in any order), the second moves the rows that grown blocks
// held to their new unit, and the third quantises the new rows.  Where no block
// grows, the usual case of decoding, the second finds nothing to do.
//
// The need of a row of largest magnitude a = f 2^E (1 <= f < 2):
//   a <= 448 2^(e+k) = 1.75 2^(e+k+8)   <=>   k >= E - e - 8 + (f > 1.75),
// so it comes from the exponent bits and one comparison.  x 2^-(e+k) is exact in
// fp32, and the conversion to e4m3 rounds once.
//
// Bound: HBM, and the launches for few rows.  200,000 rows read back to bf16 take 57.5 us
// (359 MB: 6.3 TB/s, 92% of the measured copy rate), to fp32 90.7 (590 MB, 96%).  40,011
// fp32 rows of a prompt are written in 27.6 us, bf16 ones in 23, where their blocks have the
// scales that they need; the source is read by the first kernel and the third, whose order
// finds the last of it in the second level cache (17.4 us, fp32, if each byte came once).
// Into empty blocks they take 92 and 82 us: rows that follow each other raise the same word
// at the same time (in blocks of 16 slots 49, fp32, of 1 30, 64-slot blocks in random order
// 43).  A block that held rows and grows is moved by one thread block: 64 rows written in
// blocks of 16 slots that grow take 8 us, of 64 18, of 1,024 215, and where the pool is one
// block of 262,144 7,800.

#include <cuda_fp8.h>

#include "io.cuh"
#include "kv8.cuh"
#include "sm100.cuh"

namespace mlav {
namespace kv8 {
using kvq::io_grid;
using kvq::kErrMax;
using kvq::kIoThreads;
using kvq::kIoWarps;
using kvq::put_block_err;

struct IoParams {
  uint8_t* cache;
  int64_t row_stride, slots;
  uint32_t* scales;
  Divider div;
  int block, exponent;
  int64_t n;
  const int32_t* slot;
  void* kv_c;
  void* k_pe;
  int64_t kv_c_stride, k_pe_stride;  // elements
  bool wide;                         // kv_c rows are 32-byte aligned
  int per;                           // growing: rows per block of threads
  uint32_t* err;
};

// Sixteen latents of a row as bits of fp32 (the lane's part).
template <class T>
struct Part;
template <>
struct Part<__nv_bfloat16> {
  uint32_t v[8];
  __device__ __forceinline__ void load(const void* row, int lane, bool wide) {
    kvq::ld_words(static_cast<const __nv_bfloat16*>(row) + 16 * lane, wide, v);
  }
  __device__ __forceinline__ uint32_t bits(int i) const { return (i & 1) ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16; }
};
template <>
struct Part<float> {
  uint32_t v[2][8];
  __device__ __forceinline__ void load(const void* row, int lane, bool wide) {
    const float* p = static_cast<const float*>(row) + 16 * lane;
    kvq::ld_words(p, wide, v[0]);
    kvq::ld_words(p + 8, wide, v[1]);
  }
  __device__ __forceinline__ uint32_t bits(int i) const { return v[i >> 3][i & 7]; }
};

__device__ __forceinline__ int64_t slot_at(const IoParams& p, int64_t i, uint32_t* e) {
  const int64_t s = i < p.n ? p.slot[i] : -1;
  if (s >= -1 && s < p.slots) return s;
  *e |= MLA_DEVERR_SLOT;
  return -1;
}

// What a row needs of its block, in the form of a scale word; the same in every lane.
template <class T>
__device__ __forceinline__ uint32_t need_of(const IoParams& p, const Part<T>& x, uint32_t* e) {
  uint32_t big = 0;  // magnitudes compare as their bits
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = x.bits(i) & 0x7fffffffu;
    if (a >= 0x7f800000u) *e |= MLA_DEVERR_NONFINITE;
    else big = max(big, a);
  }
  big = __reduce_max_sync(0xffffffffu, big);
  const int k = (int)(big >> 23) - 127 - p.exponent - 8 + ((big & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)min(max(k, 0), kMaxK) + 1u;
}
// Into the pending bits of the block's word.
__device__ __forceinline__ void put_need(const IoParams& p, int64_t slot, uint32_t need) {
  uint32_t* word = p.scales + p.div((uint32_t)slot);
  const uint32_t w = *reinterpret_cast<volatile uint32_t*>(word), had = w & kScaleMask;
  if (need > had && (need << kPendingShift | had) > w) atomicMax(word, need << kPendingShift | had);
}

// What the new rows need.
template <class T, int kDeep>
__global__ void __launch_bounds__(kIoThreads) kv8_need_kernel(const IoParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kIoWarps + (threadIdx.x >> 5);
  const int64_t nwarps = (int64_t)gridDim.x * kIoWarps;
  grid_dep_wait();  // launched before the stream's last kernel has ended
  grid_dep_launch();
  uint32_t e = 0;
  for (int64_t i0 = warp; i0 < p.n; i0 += kDeep * nwarps) {
    int64_t slot[kDeep];
    Part<T> x[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      slot[d] = slot_at(p, i0 + d * nwarps, &e);
      if (slot[d] >= 0)
        x[d].load(static_cast<const T*>(p.kv_c) + (i0 + d * nwarps) * p.kv_c_stride, lane, p.wide);
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (slot[d] < 0) continue;
      const uint32_t need = need_of(p, x[d], &e);
      if (lane == 0) put_need(p, slot[d], need);
    }
  }
  put_block_err(p.err, e);
}

// k of a word between the kernels of a write.
__device__ __forceinline__ int grown_scale(uint32_t w) {
  return scale_of(max(w & kScaleMask, (w >> kPendingShift) & kScaleMask));
}

constexpr uint32_t kClaimed = 1u << (2 * kPendingShift);

// Claims slot s's block if it held rows, has grown and nobody has claimed it; *w
// receives its word.
__device__ __forceinline__ bool claim(const IoParams& p, int64_t s, uint32_t* w) {
  uint32_t* word = p.scales + p.div((uint32_t)s);
  *w = *reinterpret_cast<volatile uint32_t*>(word);
  return (*w & kScaleMask) && ((*w >> kPendingShift) & kScaleMask) > (*w & kScaleMask) && !(*w & kClaimed) &&
         !(atomicOr(word, kClaimed) & kClaimed);
}

// Moves all rows of `count` claimed blocks to their new units, also those that are
// overwritten next; a block of kWarps warps.
template <int kWarps>
__device__ __forceinline__ void grow(const IoParams& p, const uint32_t* claimed, const uint32_t* word, int count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = (int64_t)count * p.block;
  constexpr int kDeep = 4;
  for (int64_t r0 = warp; r0 < rows; r0 += kDeep * kWarps) {
    uint8_t* row[kDeep];
    int down[kDeep];
    uint4 c[kDeep];
    uint32_t rope[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t r = r0 + d * kWarps;
      row[d] = nullptr;
      if (r >= rows) continue;
      const int at = (int)(r / p.block);
      const int64_t slot = (int64_t)claimed[at] * p.block + r % p.block;
      if (slot >= p.slots) continue;
      row[d] = p.cache + slot * p.row_stride;
      down[d] = grown_scale(word[at]) - scale_of(word[at]);
      c[d] = reinterpret_cast<const uint4*>(row[d])[lane];
      rope[d] = reinterpret_cast<const uint32_t*>(row[d] + kRopeOff)[lane];
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (!row[d]) continue;
      const float mul = pow2(-down[d]);
      uint32_t v[4] = {c[d].x, c[d].y, c[d].z, c[d].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t o = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v[q] >> (16 * h)), __NV_E4M3);
          const float2 g = __half22float2(__half2(f));
          o |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(g.x * mul, g.y * mul), __NV_SATFINITE, __NV_E4M3)
               << (16 * h);
        }
        v[q] = o;
      }
      reinterpret_cast<uint4*>(row[d])[lane] = make_uint4(v[0], v[1], v[2], v[3]);
      const __nv_bfloat162 k = __floats2bfloat162_rn(__uint_as_float(rope[d] << 16) * mul,
                                                     __uint_as_float(rope[d] & 0xffff0000u) * mul);
      reinterpret_cast<uint32_t*>(row[d] + kRopeOff)[lane] = *reinterpret_cast<const uint32_t*>(&k);
    }
  }
}

// The rows of blocks that held some and have grown: a thread block looks at `per` of
// the new rows.
__global__ void __launch_bounds__(kIoThreads) kv8_grow_kernel(const IoParams p) {
  __shared__ uint32_t claimed[kIoThreads], word[kIoThreads];
  __shared__ int count;
  if (threadIdx.x == 0) count = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  uint32_t e = 0, w;
  const int64_t i = (int64_t)blockIdx.x * p.per + threadIdx.x;
  const int64_t s = (int)threadIdx.x < p.per ? slot_at(p, i, &e) : -1;
  if (s >= 0 && claim(p, s, &w)) {
    const int at = atomicAdd(&count, 1);
    claimed[at] = p.div((uint32_t)s);
    word[at] = w;
  }
  __syncthreads();
  grow<kIoWarps>(p, claimed, word, count);
}

__device__ __forceinline__ float2 rope_pair(const __nv_bfloat16* p) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 rope_pair(const float* p) { return *reinterpret_cast<const float2*>(p); }

// A new row in its block's unit, by the block's word.  The row's warp also puts the
// word into its final form (all of a block's rows store the same word, and whichever
// form another row reads says the same).
template <class T>
__device__ __forceinline__ void put_row(const IoParams& p, int64_t slot, uint32_t word, const Part<T>& x, float2 rope) {
  const int lane = threadIdx.x & 31;
  const int k = grown_scale(word);
  const float mul = pow2(-(p.exponent + k));
  uint32_t v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float f[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      f[h] = __uint_as_float(x.bits(4 * q + h)) * mul;
      f[h] = f[h] == f[h] ? f[h] : 0.f;
    }
    v[q] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3) << 16;
  }
  uint8_t* row = p.cache + slot * p.row_stride;
  reinterpret_cast<uint4*>(row)[lane] = make_uint4(v[0], v[1], v[2], v[3]);
  const __nv_bfloat162 r = __floats2bfloat162_rn(rope.x * mul, rope.y * mul);
  reinterpret_cast<uint32_t*>(row + kRopeOff)[lane] = *reinterpret_cast<const uint32_t*>(&r);
  if (lane == 0 && word != (uint32_t)k + 1u)
    *reinterpret_cast<volatile uint32_t*>(p.scales + p.div((uint32_t)slot)) = (uint32_t)k + 1u;
}

// The new rows, last ones first: the second level cache still holds what the first
// kernel has read last.
template <class T, int kDeep>
__global__ void __launch_bounds__(kIoThreads) kv8_write_kernel(const IoParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kIoWarps + (threadIdx.x >> 5);
  const int64_t nwarps = (int64_t)gridDim.x * kIoWarps;
  grid_dep_wait();
  grid_dep_launch();
  uint32_t e = 0;
  for (int64_t i0 = warp; i0 < p.n; i0 += kDeep * nwarps) {
    int64_t slot[kDeep];
    uint32_t word[kDeep];
    Part<T> x[kDeep];
    float2 rope[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t i = p.n - 1 - (i0 + d * nwarps);
      slot[d] = i >= 0 ? slot_at(p, i, &e) : -1;
      if (slot[d] < 0) continue;
      word[d] = *reinterpret_cast<volatile uint32_t*>(p.scales + p.div((uint32_t)slot[d]));
      x[d].load(static_cast<const T*>(p.kv_c) + i * p.kv_c_stride, lane, p.wide);
      rope[d] = rope_pair(static_cast<const T*>(p.k_pe) + i * p.k_pe_stride + 2 * lane);
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
      if (slot[d] >= 0) put_row(p, slot[d], word[d], x[d], rope[d]);
  }
}

// All three steps for few rows: one cluster, a warp per row, whose barrier stands between
// the steps where the larger calls have a launch.  One launch and three, us: 16 rows 3.1
// and 4.0, 64 3.4 and 4.2, 128 3.7 and 4.4; with two rows to a warp 256 rows 5.0 and 4.4.
constexpr int kSmallBlocks = 8, kSmallWarps = 16, kSmallRows = kSmallBlocks * kSmallWarps;
template <class T>
__global__ void __cluster_dims__(kSmallBlocks, 1, 1) __launch_bounds__(32 * kSmallWarps)
    kv8_write_small_kernel(const IoParams p) {
  __shared__ uint32_t claimed[kSmallWarps], word[kSmallWarps];
  __shared__ uint32_t found[kSmallWarps];
  __shared__ int count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) count = 0;
  grid_dep_wait();  // launched before the stream's last kernel has ended
  grid_dep_launch();
  uint32_t e = 0;
  Part<T> x;
  float2 rope;
  const int64_t i = blockIdx.x + kSmallBlocks * warp;
  const int64_t slot = slot_at(p, i, &e);
  if (slot >= 0) {
    x.load(static_cast<const T*>(p.kv_c) + i * p.kv_c_stride, lane, p.wide);
    rope = rope_pair(static_cast<const T*>(p.k_pe) + i * p.k_pe_stride + 2 * lane);
    const uint32_t need = need_of(p, x, &e);
    if (lane == 0) put_need(p, slot, need);
  }
  const uint32_t any = __reduce_or_sync(0xffffffffu, e);
  if (lane == 0) found[warp] = any;
  sm100::cluster_sync();
  if (threadIdx.x == 0) {
    uint32_t f = 0;
    for (int w = 0; w < kSmallWarps; ++w) f |= found[w];
    p.err[kvq::kErrFirst + blockIdx.x] = f;
    if (blockIdx.x == 0) p.err[0] = gridDim.x;
  }
  uint32_t mine;
  if (lane == 0 && slot >= 0 && claim(p, slot, &mine)) {
    const int at = atomicAdd(&count, 1);
    claimed[at] = p.div((uint32_t)slot);
    word[at] = mine;
  }
  __syncthreads();
  grow<kSmallWarps>(p, claimed, word, count);
  sm100::cluster_sync();
  if (slot >= 0)
    put_row(p, slot, *reinterpret_cast<volatile uint32_t*>(p.scales + p.div((uint32_t)slot)), x, rope);
}

__device__ __forceinline__ void put_latents(__nv_bfloat16* dst, const float (&f)[16], bool wide) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  kvq::st_words(dst, wide, v);
}
__device__ __forceinline__ void put_latents(float* dst, const float (&f)[16], bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(f[8 * h + i]);
    kvq::st_words(dst + 8 * h, wide, v);
  }
}
__device__ __forceinline__ void put_rope(__nv_bfloat16* dst, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void put_rope(float* dst, float a, float b) {
  *reinterpret_cast<float2*>(dst) = make_float2(a, b);
}

template <class T, int kDeep>
__global__ void __launch_bounds__(kIoThreads) kv8_read_kernel(const IoParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kIoWarps + (threadIdx.x >> 5);
  const int64_t nwarps = (int64_t)gridDim.x * kIoWarps;
  grid_dep_wait();  // launched before the stream's last kernel has ended
  grid_dep_launch();
  uint32_t e = 0;
  for (int64_t i0 = warp; i0 < p.n; i0 += kDeep * nwarps) {
    int64_t slot[kDeep];
    uint4 c[kDeep];
    uint32_t rope[kDeep], word[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      slot[d] = slot_at(p, i0 + d * nwarps, &e);
      if (slot[d] < 0) continue;
      const uint8_t* row = p.cache + slot[d] * p.row_stride;
      c[d] = reinterpret_cast<const uint4*>(row)[lane];
      rope[d] = reinterpret_cast<const uint32_t*>(row + kRopeOff)[lane];
      word[d] = p.scales[p.div((uint32_t)slot[d])];
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (slot[d] < 0) continue;
      const int64_t i = i0 + d * nwarps;
      const float mul = pow2(p.exponent + scale_of(word[d]));
      const uint32_t v[4] = {c[d].x, c[d].y, c[d].z, c[d].w};
      float f[16];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v[q >> 1] >> (16 * (q & 1))), __NV_E4M3);
        const float2 g = __half22float2(__half2(h));
        f[2 * q] = g.x * mul;
        f[2 * q + 1] = g.y * mul;
      }
      put_latents(static_cast<T*>(p.kv_c) + i * p.kv_c_stride + 16 * lane, f, p.wide);
      put_rope(static_cast<T*>(p.k_pe) + i * p.k_pe_stride + 2 * lane, __uint_as_float(rope[d] << 16) * mul,
               __uint_as_float(rope[d] & 0xffff0000u) * mul);
    }
  }
  put_block_err(p.err, e);
}

mla_status validate_cache(const mla_kv8_cache* c) {
  if (!c || !c->rows || (reinterpret_cast<uintptr_t>(c->rows) & 31u)) return MLA_ERR_INVALID_ARG;
  if (c->row_stride < MLA_KV8_ROW_BYTES || (c->row_stride & 31) || c->row_stride > INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  if (c->slots < 1 || c->slots > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (!c->scales || (reinterpret_cast<uintptr_t>(c->scales) & 3u) || c->block < 1) return MLA_ERR_INVALID_ARG;
  if (c->exponent < -MLA_KV8_MAX_EXPONENT || c->exponent > MLA_KV8_MAX_EXPONENT) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks shared by both directions; *noop when there is nothing to launch.
mla_status make_io(const mla_kv8_cache* c, const mla_kvq_rows* r, void* ws, size_t ws_bytes, IoParams* p, bool* noop) {
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
  if (!ws || !aligned(ws, 256) || ws_bytes < MLA_KV8_WORKSPACE_BYTES) return MLA_ERR_WORKSPACE;
  p->cache = static_cast<uint8_t*>(c->rows);
  p->row_stride = c->row_stride;
  p->slots = c->slots;
  p->scales = reinterpret_cast<uint32_t*>(c->scales);
  p->div.set(c->block);
  p->block = c->block;
  p->exponent = c->exponent;
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
}  // namespace kv8
}  // namespace mlav

using namespace mlav;
using namespace mlav::kv8;

extern "C" mla_status mla_kv8_write(const mla_kv8_cache* cache, const mla_kvq_rows* src, void* workspace,
                                    size_t ws_bytes, mla_stream_t stream) {
  kv8::IoParams p;
  bool noop = false;
  mla_status st = make_io(cache, src, workspace, ws_bytes, &p, &noop);
  if (st != MLA_OK || noop) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = src->dtype == MLA_BF16;
  if (p.n <= kSmallRows) {
    const auto small = bf16 ? kv8_write_small_kernel<__nv_bfloat16> : kv8_write_small_kernel<float>;
    const cudaError_t e = launch_kernel(small, dim3(kSmallBlocks), dim3(32 * kSmallWarps), 0, s, true, p);
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
  }
  int grid = 0;
  st = io_grid(p.n, 8, &grid);
  if (st != MLA_OK) return st;
  const auto need = bf16 ? kv8_need_kernel<__nv_bfloat16, 2> : kv8_need_kernel<float, 1>;
  const auto write = bf16 ? kv8_write_kernel<__nv_bfloat16, 2> : kv8_write_kernel<float, 1>;
  // rows per block of the growing kernel: a few blocks of threads per SM
  p.per = (int)((p.n + 1023) / 1024);
  if (p.per < kIoWarps) p.per = kIoWarps;
  if (p.per > kIoThreads) p.per = kIoThreads;
  const int64_t growers = (p.n + p.per - 1) / p.per;
  if (launch_kernel(need, dim3(grid), dim3(kIoThreads), 0, s, true, p) != cudaSuccess ||
      launch_kernel(kv8_grow_kernel, dim3((unsigned)growers), dim3(kIoThreads), 0, s, true, p) != cudaSuccess ||
      launch_kernel(write, dim3(grid), dim3(kIoThreads), 0, s, true, p) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

extern "C" mla_status mla_kv8_read(const mla_kv8_cache* cache, const mla_kvq_rows* dst, void* workspace,
                                   size_t ws_bytes, mla_stream_t stream) {
  kv8::IoParams p;
  bool noop = false;
  mla_status st = make_io(cache, dst, workspace, ws_bytes, &p, &noop);
  if (st != MLA_OK || noop) return st;
  int grid = 0;
  st = io_grid(p.n, 16, &grid);
  if (st != MLA_OK) return st;
  const auto kernel = dst->dtype == MLA_BF16 ? kv8_read_kernel<__nv_bfloat16, 2> : kv8_read_kernel<float, 2>;
  const cudaError_t e = launch_kernel(kernel, dim3(grid), dim3(kIoThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                                      true, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_kv8_check(const void* workspace, mla_stream_t stream, uint32_t* bits) {
  return mla_kvq_check(workspace, stream, bits);  // the same error words
}
