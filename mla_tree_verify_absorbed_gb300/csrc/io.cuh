// What the quantised caches' writes and reads share: wide loads and stores of rows
// that pass once, the blocks' error words, and the number of blocks.
#pragma once

#include <atomic>

#include "kvq.cuh"
#include "sm100.cuh"

namespace mlav {
namespace kvq {

constexpr int kIoThreads = 256;
constexpr int kIoWarps = kIoThreads / 32;

// Stores this block's error bits (and, block 0, the number of words).
__device__ __forceinline__ void put_block_err(uint32_t* err, uint32_t e) {
  const uint32_t any = __reduce_or_sync(0xffffffffu, e);
  __shared__ uint32_t sh[kIoWarps];
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = any;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t b = 0;
#pragma unroll
    for (int w = 0; w < kIoWarps; ++w) b |= sh[w];
    err[kErrFirst + blockIdx.x] = b;
    if (blockIdx.x == 0) err[0] = gridDim.x;
  }
}

// Eight 32-bit words at once, a whole sector when the caller's rows are 32-byte
// aligned (`wide`, the same for the whole call), else as two halves, which for
// 200,000 rows takes 63 us in place of 60 for a bf16 write, 86 for 82 for an fp32
// write, 64 for 52 for a bf16 read and 168 for 86 for an fp32 read, whose stores
// then fill half sectors.  Rows pass once, so they are kept out of L1.
__device__ __forceinline__ void ld_words(const void* p, bool wide, uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldcs(static_cast<const uint4*>(p)), b = __ldcs(static_cast<const uint4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
__device__ __forceinline__ void st_words(void* p, bool wide, const uint32_t (&v)[8]) {
  if (wide) {
    sm100::st_global_v8(static_cast<uint32_t*>(p), v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
  } else {
    __stcs(static_cast<uint4*>(p), make_uint4(v[0], v[1], v[2], v[3]));
    __stcs(static_cast<uint4*>(p) + 1, make_uint4(v[4], v[5], v[6], v[7]));
  }
}

// Blocks for n rows: one row per warp while they fit the GPU, then a
// persistent grid of per_sm blocks per SM (for 200,000 rows 4, 8 and 16 took 59,
// 60 and 61 us for a bf16 write, 82 each for an fp32 one, 54, 55 and 52 for a bf16
// read, 103, 90 and 86 for an fp32 one: 8 for writes, 16 for reads).
inline mla_status io_grid(int64_t n, int per_sm, int* grid) {
  // looked up once per device: the two queries took as long as the launch
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_CUDA;
  sms = cached[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MLA_ERR_CUDA;
    cached[dev].store(sms, std::memory_order_relaxed);
  }
  int64_t g = (n + kIoWarps - 1) / kIoWarps;
  if (g > (int64_t)sms * per_sm) g = (int64_t)sms * per_sm;
  if (g > kErrMax) g = kErrMax;
  *grid = (int)g;
  return MLA_OK;
}

}  // namespace kvq
}  // namespace mlav
