// Verify attention over the 4-bit latent cache (mla_kvq_attn): one warp per
// query row, online softmax in registers.  Lane l holds elements 16 l .. + 15
// of the query and of the output, and rope elements 2 l, 2 l + 1.
#include <cmath>

#include "kvq.cuh"

namespace mlav {
namespace kvq {

mla_status validate_cache(const mla_kvq_cache* c);

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads) kvq_attn_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  uint32_t e = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) e |= check_sequence(p, b);
  const int stop = __syncthreads_or((int)e);
  const int64_t total = (int64_t)p.B * p.rows;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); !stop && w < total;
       w += (int64_t)gridDim.x * kWarps) {
    const int b = (int)(w / p.rows), i = (int)(w % p.rows) / p.H;
    const int64_t P = p.prefix_lens[b];
    if (P < 0) continue;
    bool bad = false;
    const NodeView nv = node_view(i, P, p.window, p.sinks, &bad, [&](int t) {
      return p.tree_parent ? p.tree_parent[(int64_t)b * p.Q + t] : t - 1;
    });
    if (bad) e |= MLA_DEVERR_PARENT;
    float q[16], o[16];
    const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(p.q_lat) + w * kDl + 16 * lane;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q_pe) + w * kDr + 2 * lane;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      q[k] = __bfloat162float(ql[k]);
      o[k] = 0.f;
    }
    const float q0 = __bfloat162float(qp[0]) * p.qpe_mul, q1 = __bfloat162float(qp[1]) * p.qpe_mul;
    const int64_t idx0 = p.page_size == 1 ? p.kv_indptr[b] : 0;
    float m = -INFINITY, l = 0.f;
    for (int64_t pos = 0; pos < P + p.Q; ++pos) {
      if (pos < P) {
        if (p.window && pos >= p.sinks && P + nv.depth - pos >= p.window) {
          pos = P + nv.depth - p.window;  // the first position inside the window is next
          if (pos >= P) pos = P - 1;
          continue;
        }
      } else if (!((nv.mask >> (pos - P)) & 1ull)) {
        continue;
      }
      int64_t s = slot_at(p, b, idx0, pos);
      if (s < 0) {
        e |= MLA_DEVERR_SLOT;
        s = 0;
      }
      const uint8_t* row = p.cache + s * p.row_stride;
      const uint2 cw = reinterpret_cast<const uint2*>(row)[lane];
      const uint32_t sc = ToBf16::scales((uint32_t)row[kScaleOff + lane] * 0x10001u);
      const uint32_t of = ToBf16::offsets(sc);
      const uint32_t kr = reinterpret_cast<const uint32_t*>(row + kRopeOff)[lane];
      uint32_t a[4], c[4];
      ToBf16::word(cw.x, sc, of, a);
      ToBf16::word(cw.y, sc, of, c);
      float v[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(a[k] << 16);
        v[2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u);
        v[8 + 2 * k] = __uint_as_float(c[k] << 16);
        v[8 + 2 * k + 1] = __uint_as_float(c[k] & 0xffff0000u);
      }
      float d = q0 * __uint_as_float(kr << 16) + q1 * __uint_as_float(kr & 0xffff0000u);
#pragma unroll
      for (int k = 0; k < 16; ++k) d = fmaf(q[k], v[k], d);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
      d *= p.scale_log2;
      const float mn = fmaxf(m, d), alpha = exp2f(m - mn), pw = exp2f(d - mn);
      m = mn;
      l = l * alpha + pw;
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = fmaf(pw, v[k], o[k] * alpha);
    }
    const float inv = p.out_mul / l;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + w * kDl + 16 * lane;
#pragma unroll
    for (int k = 0; k < 16; ++k) out[k] = __float2bfloat16_rn(o[k] * inv);
    if (lane == 0 && p.lse) p.lse[w] = (m + log2f(l)) * 0.69314718055994530942f;
  }
  const int any = __syncthreads_or((int)e);
  // the words of all threads of a block, bit by bit
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < 10; ++k) bits |= __syncthreads_or((int)((e >> k) & 1u)) ? 1u << k : 0u;
  if (threadIdx.x == 0) {
    p.err[kErrFirst + blockIdx.x] = any ? bits : 0u;
    if (blockIdx.x == 0) p.err[0] = gridDim.x;
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status validate_shape(const mla_kvq_attn_args* a) {
  if (!a) return MLA_ERR_INVALID_ARG;
  if (a->B < 0 || a->Q < 0 || a->H < 1) return MLA_ERR_INVALID_ARG;
  if (a->Q > MLA_MAX_Q) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)a->H * a->Q > (int64_t)1 << 24) return MLA_ERR_UNSUPPORTED;
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
  // a zero scale would turn masked scores of -inf into NaN
  if (!std::isfinite(a->scale) || !(a->scale > 0.f)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

Params make_params(const mla_kvq_attn_args* a, void* ws) {
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
  p.scale_log2 = (float)std::ldexp((double)a->scale * 1.4426950408889634, e);
  p.out_mul = (float)std::ldexp(1.0, e);
  p.out = a->out;
  p.lse = a->lse;
  p.err = static_cast<uint32_t*>(ws);
  return p;
}

}  // namespace
}  // namespace kvq
}  // namespace mlav

using namespace mlav::kvq;

extern "C" size_t mla_kvq_attn_workspace_size(const mla_kvq_attn_args* a) {
  if (validate_shape(a) != MLA_OK) return 0;
  return MLA_KVQ_WORKSPACE_BYTES;
}

extern "C" mla_status mla_kvq_attn(const mla_kvq_attn_args* a, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  mla_status st = validate_shape(a);
  if (st != MLA_OK) return st;
  if (a->B == 0 || a->Q == 0) return MLA_OK;
  st = validate_call(a);
  if (st != MLA_OK) return st;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < MLA_KVQ_WORKSPACE_BYTES) return MLA_ERR_WORKSPACE;
  const Params p = make_params(a, workspace);
  int64_t grid = ((int64_t)p.B * p.rows + kWarps - 1) / kWarps;
  if (grid > kErrMax) grid = kErrMax;
  kvq_attn_kernel<<<(int)grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
