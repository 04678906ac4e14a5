// A step's page tables from the requests' lengths (mla_kv_tables).
//
// One launch.  Every block sums what the requests need (four prefix sums over at
// most 4096 requests, kept in shared memory), so the blocks need not wait for one
// another: each then takes its share of the pages that change hands and of the
// slots to list, looking up an entry's request in the sums.  What other blocks read
// at the start, the held counts and the ring's ends, is changed by the block that
// finishes last.  Pages that change hands are read from the ring and never from an
// entry that this call writes: the ring gives from its head and takes at its tail.
//
// Bound: for short lists the chain launch, lengths, sums, entry (8 requests of one new
// token: 5.4 us; 256 with ragged prefixes and a listing of 1.3 million slots: 9.8 us, and
// 10.4 where 15,937 pages change hands);
// for long ones the stores, 4 bytes per position.
#include "kv8.cuh"

namespace mlav {
namespace tables {

using kvq::kErrFirst;
using kvq::kErrMax;
constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Params {
  mla_kv_tables_args a;
  kv8::Divider page;
  uint32_t* err;
};

// exclusive sums over the requests, one more entry than requests, and the held counts
struct Sums {
  int32_t *length, *fresh, *take, *drop, *held;
};

struct Request {
  int32_t length, fresh;  // positions, new tokens
  int need, held;
  uint32_t err;
};
__device__ __forceinline__ Request read_request(const Params& p, int b) {
  Request r;
  const int32_t prefix = p.a.prefix_lens[b];
  const int32_t held = p.a.pages_held[b];
  const int32_t fresh = prefix >= 0 ? p.a.new_lens ? p.a.new_lens[b] : p.a.Q : 0;
  r.err = prefix < -1 || fresh < 0 ? MLA_DEVERR_PREFIX : 0u;
  if (held < 0 || held > p.a.max_pages) r.err |= MLA_DEVERR_PAGES;
  r.fresh = max(fresh, 0);
  const int64_t length = (int64_t)max(prefix, 0) + r.fresh;
  r.length = (int32_t)length;
  if (length > (int64_t)p.a.max_pages * p.a.page_size) {
    r.err |= MLA_DEVERR_PAGES;
    r.length = r.fresh = 0;
  }
  r.need = r.length > 0 ? (int)p.page((uint32_t)r.length - 1u) + 1 : 0;
  r.held = held;
  return r;
}

// a % b for a >= 0, b > 0: a 32-bit division wherever it will do.
__device__ __forceinline__ uint32_t mod_fast(int64_t a, int b) {
  return a >> 32 ? (uint32_t)(a % b) : (uint32_t)a % (uint32_t)b;
}

// The request that entry i of a sum belongs to: the last one that begins at or
// before i, which is not empty.
__device__ __forceinline__ int request_of(const int32_t* sum, int B, int32_t i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sum[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// N holds the sums: 32 bits where B requests of max_pages pages cannot pass them
// (every block sums for itself, and in 64 bits that takes twice as long).
// kList positions are listed by a thread, which looks up a page once for those of
// them that lie in it: 16 in long lists with pages of at least 8 slots, else 4 (256
// requests, 1.35 million positions in pages of 16: 13.9 us with 4, 9.7 with 16; 8
// requests, 20,000 positions: 5.5 and 6.4).
template <class N, int kList>
__global__ void __launch_bounds__(kThreads) kv_tables_kernel(const Params p) {
  extern __shared__ int32_t dynamic[];
  __shared__ N part[4][kWarps];
  __shared__ uint32_t bad;
  __shared__ bool last;
  const mla_kv_tables_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.B;
  const Sums s{dynamic, dynamic + (B + 1), dynamic + 2 * (B + 1), dynamic + 3 * (B + 1), dynamic + 4 * (B + 1)};
  if (tid == 0) bad = 0;
  grid_dep_wait();  // launched before the stream's last kernel has ended
  grid_dep_launch();
  const int64_t head = a.free_state[0], tail = a.free_state[1];
  __syncthreads();
  // sums: threads take consecutive requests
  const int per = (B + kThreads - 1) / kThreads, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  const int warps = (B + 32 * per - 1) / (32 * per);  // that have requests
  N at[4] = {0, 0, 0, 0};
  uint32_t e = 0;
  Request r = {};
  if (warp < warps) {
    N sum[4] = {0, 0, 0, 0};
    for (int b = b0; b < b1; ++b) {
      r = read_request(p, b);
      e |= r.err;
      sum[0] += r.length;
      sum[1] += r.fresh;
      sum[2] += max(r.need - r.held, 0);
      sum[3] += max(r.held - r.need, 0);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      N v = sum[q];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const N u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      at[q] = v - sum[q];
      if (lane == 31) part[q][warp] = v;
    }
    if (e) atomicOr(&bad, e);
  }
  __syncthreads();
  N total[4] = {0, 0, 0, 0};
#pragma unroll 1
  for (int w = 0; w < warps; ++w) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (w == warp) at[q] += total[q];
      total[q] += part[q][w];
    }
  }
  const int64_t takes = total[2], drops = total[3];
  uint32_t err = bad;
  if (head < 0 || tail < head || tail - head > a.ring) err |= MLA_DEVERR_PAGES;
  // with a bad request the sums mean nothing
  if (!err && (takes > tail - head || tail - head + drops > a.ring || total[0] > (N)INT32_MAX ||
               total[1] > (N)INT32_MAX || takes > INT32_MAX || drops > INT32_MAX ||
               (a.kv_indices && total[0] > a.indices_len) || (a.slots && a.new_lens && total[1] > a.slots_len)))
    err = MLA_DEVERR_CAPACITY;
  // length + page_size - 1 may pass 32 bits
  auto pages_of = [&](int32_t length) { return length > 0 ? (int)p.page((uint32_t)length - 1u) + 1 : 0; };
  uint32_t late = 0;
  if (!err) {  // the same in every block
    for (int b = b0; b < b1; ++b) {
      if (per > 1) r = read_request(p, b);
      s.length[b] = (int32_t)at[0];
      s.fresh[b] = (int32_t)at[1];
      s.take[b] = (int32_t)at[2];
      s.drop[b] = (int32_t)at[3];
      s.held[b] = r.held;
      at[0] += r.length;
      at[1] += r.fresh;
      at[2] += max(r.need - r.held, 0);
      at[3] += max(r.held - r.need, 0);
    }
    if (tid < 4) dynamic[tid * (B + 1) + B] = (int32_t)total[tid];
    __syncthreads();
    const uint32_t ring0 = mod_fast(head, a.ring), ring1 = mod_fast(tail, a.ring);
    auto entry = [&](uint32_t from, int32_t i) {  // i < ring
      const uint32_t at = from + (uint32_t)i;
      return at < (uint32_t)a.ring ? at : at - (uint32_t)a.ring;
    };
    auto valid = [&](int32_t page) {
      if (page >= 0 && page < a.num_pages) return true;
      late |= MLA_DEVERR_SLOT;
      return false;
    };
    const bool wide = (reinterpret_cast<uintptr_t>(a.kv_indices) & 15u) == 0;
    // first slot of page j of request b, -1 where its id is none
    auto page_of = [&](int b, int j) -> int32_t {
      const int held = s.held[b];
      const int32_t page = j < held ? a.block_table[(int64_t)b * a.max_pages + j]
                                    : a.free_ring[entry(ring0, s.take[b] + j - held)];
      return valid(page) ? page * a.page_size : -1;
    };
    // All that is to be done, one kind after the other, so that no thread has much of
    // it: pages that are taken, pages that come back, offsets, the new tokens' slots,
    // and the positions' slots, kList to a thread.
    const int64_t slots = a.slots ? a.slots_len : 0, listed = a.kv_indices ? ((int64_t)total[0] + kList - 1) / kList : 0;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < takes + drops + (B + 1) + slots + listed; i += step) {
      int64_t n = i;
      if (n < takes) {
        const int b = request_of(s.take, B, (int32_t)n);
        const int32_t page = a.free_ring[entry(ring0, (int32_t)n)];
        a.block_table[(int64_t)b * a.max_pages + s.held[b] + ((int32_t)n - s.take[b])] = page;
        if (valid(page) && a.scales) {
          const int64_t lo = (int64_t)page * a.page_size, hi = lo + a.page_size;
          for (int64_t k = (lo + a.block - 1) / a.block; k < hi / a.block; ++k) a.scales[k] = 0;
        }
        continue;
      }
      n -= takes;
      if (n < drops) {
        const int b = request_of(s.drop, B, (int32_t)n);
        int32_t* at = a.block_table + (int64_t)b * a.max_pages + pages_of(s.length[b + 1] - s.length[b]) +
                      ((int32_t)n - s.drop[b]);
        a.free_ring[entry(ring1, (int32_t)n)] = *at;
        valid(*at);
        *at = -1;
        continue;
      }
      n -= drops;
      if (n <= B) {
        if (a.kv_indptr) a.kv_indptr[n] = s.length[n];
        continue;
      }
      n -= B + 1;
      if (n < slots) {
        int32_t v = -1;
        if (!a.new_lens || n < total[1]) {
          const int b = a.new_lens ? request_of(s.fresh, B, (int32_t)n) : (int)((uint32_t)n / (uint32_t)a.Q);
          const int32_t k = (int32_t)n - (a.new_lens ? s.fresh[b] : b * a.Q);
          const int32_t length = s.length[b + 1] - s.length[b], fresh = s.fresh[b + 1] - s.fresh[b];
          if (k < fresh) {
            const uint32_t pos = (uint32_t)(length - fresh + k);
            const int j = (int)p.page(pos);
            const int32_t first = page_of(b, j);
            v = first >= 0 ? first + (int32_t)(pos - (uint32_t)j * (uint32_t)a.page_size) : -1;
          }
        }
        a.slots[n] = v;
        continue;
      }
      n = kList * (n - slots);
      int b = request_of(s.length, B, (int32_t)n);
      int32_t v[kList], first = -1;
      int64_t from = n, end = n;  // the positions of one page that the loop is in
#pragma unroll
      for (int q = 0; q < kList; ++q) {
        if (n + q >= total[0]) continue;
        if (n + q >= end) {
          while (n + q >= s.length[b + 1]) ++b;
          const uint32_t pos = (uint32_t)(n + q - s.length[b]);
          const int j = (int)p.page(pos);
          first = page_of(b, j);
          from = s.length[b] + (int64_t)j * a.page_size;
          end = min(from + a.page_size, (int64_t)s.length[b + 1]);
        }
        v[q] = first >= 0 ? first + (int32_t)(n + q - from) : -1;
      }
      if (wide && n + kList <= total[0]) {
#pragma unroll
        for (int q = 0; q < kList; q += 4)
          *reinterpret_cast<int4*>(a.kv_indices + n + q) = make_int4(v[q], v[q + 1], v[q + 2], v[q + 3]);
      } else {
#pragma unroll
        for (int q = 0; q < kList; ++q)
          if (n + q < total[0]) a.kv_indices[n + q] = v[q];
      }
    }
  }
  __shared__ uint32_t found[kWarps];
  const uint32_t any = __reduce_or_sync(0xffffffffu, late);
  if (lane == 0) found[warp] = any;
  __syncthreads();
  if (tid == 0) {
    __threadfence();  // the block's reads of the state come before the count that says so
    uint32_t f = err;
    for (int w = 0; w < kWarps; ++w) f |= found[w];
    p.err[kErrFirst + blockIdx.x] = f;
    if (blockIdx.x == 0) p.err[0] = gridDim.x;
    // counts up to the number of blocks and then starts again from 0
    last = atomicInc(reinterpret_cast<unsigned int*>(a.free_state + 2), gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last || err) return;
  __threadfence();
  for (int b = tid; b < B; b += kThreads) a.pages_held[b] = pages_of(s.length[b + 1] - s.length[b]);
  if (tid == 0) {
    a.free_state[0] = head + takes;
    a.free_state[1] = tail + drops;
  }
}

namespace {
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status validate(const mla_kv_tables_args* a) {
  if (!a || a->B < 0 || a->Q < 0 || a->page_size < 1 || a->max_pages < 1 || a->num_pages < 1 || a->ring < 1)
    return MLA_ERR_INVALID_ARG;
  if (a->B > MLA_KV_TABLES_MAX_B) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)a->max_pages * a->page_size > INT32_MAX || (int64_t)a->num_pages * a->page_size > INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  if (a->B == 0) return MLA_OK;
  if (!a->prefix_lens || !a->block_table || !a->pages_held || !a->free_ring || !a->free_state)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(a->prefix_lens, 4) || !aligned(a->new_lens, 4) || !aligned(a->block_table, 4) ||
      !aligned(a->pages_held, 4) || !aligned(a->free_ring, 4) || !aligned(a->free_state, 8) || !aligned(a->slots, 4) ||
      !aligned(a->kv_indptr, 4) || !aligned(a->kv_indices, 4) || !aligned(a->scales, 4))
    return MLA_ERR_INVALID_ARG;
  if (a->slots && (a->slots_len < 0 || a->slots_len > INT32_MAX ||
                   (!a->new_lens && a->slots_len != (int64_t)a->B * a->Q)))
    return MLA_ERR_INVALID_ARG;
  if (a->kv_indices && (a->indices_len < 0 || a->indices_len > INT32_MAX)) return MLA_ERR_INVALID_ARG;
  if (a->scales && a->block < 1) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}
}  // namespace
}  // namespace tables
}  // namespace mlav

using namespace mlav;

extern "C" mla_status mla_kv_tables(const mla_kv_tables_args* a, void* workspace, size_t ws_bytes,
                                    mla_stream_t stream) {
  mla_status st = tables::validate(a);
  if (st != MLA_OK) return st;
  if (a->B == 0) return MLA_OK;
  if (!workspace || !tables::aligned(workspace, 256) || ws_bytes < MLA_KV_TABLES_WORKSPACE_BYTES)
    return MLA_ERR_WORKSPACE;
  tables::Params p;
  p.a = *a;
  p.page.set(a->page_size);
  p.err = static_cast<uint32_t*>(workspace);
  // a block for every 512 things that a thread does, as far as the host can tell; at most 128
  const int list = a->page_size >= 8 && a->kv_indices && a->indices_len > 65536 ? 16 : 4;
  const int64_t n = (a->kv_indices ? a->indices_len / list : 0) + (a->slots ? a->slots_len : 0);
  int64_t blocks = (n + tables::kThreads - 1) / tables::kThreads;
  blocks = blocks < 1 ? 1 : blocks > 128 ? 128 : blocks;
  const size_t smem = 5 * sizeof(int32_t) * ((size_t)a->B + 1);
  const bool narrow = (int64_t)a->B * a->max_pages * a->page_size <= INT32_MAX;
  const auto kernel = list == 16 ? narrow ? tables::kv_tables_kernel<int32_t, 16> : tables::kv_tables_kernel<int64_t, 16>
                      : narrow   ? tables::kv_tables_kernel<int32_t, 4>
                                 : tables::kv_tables_kernel<int64_t, 4>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MLA_ERR_CUDA;
  const cudaError_t e = launch_kernel(kernel, dim3((unsigned)blocks), dim3(tables::kThreads), smem,
                                      reinterpret_cast<cudaStream_t>(stream), true, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
