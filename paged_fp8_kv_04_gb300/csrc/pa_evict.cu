// pa_evict.cu -- eviction from the paged cache: pa_evict_select chooses the tokens that stay,
// pa_kv_compact moves them to the front of their pages.  See include/pa.h for the contract.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa.h"
#include "pa_host.cuh"

namespace {

using pa_host::aligned;

constexpr int kD = pa_host::kD;
constexpr int kMaxSeqs = 65535;

// --------------------------------------------------------------------------- selection

struct SelectParams {
  const float *mass;
  const int32_t *L;
  int32_t *keep, *new_lens;
  uint32_t *status;
  int32_t Hkv, stride, budget, first, recent;
};

// Unsigned keys in the order of the masses: NaN lowest, -0 = +0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;

// Sum of v over the CTA, known to every thread.
__device__ int block_sum(int v, int *buf) {
  const int s = __reduce_add_sync(~0u, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  return __reduce_add_sync(~0u, buf[threadIdx.x & 31]);
}

// Exclusive prefix sum of v over the CTA's threads; total in *total.
__device__ int block_scan(int v, int *buf, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int w = buf[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(~0u, w, 31);
  const int before = warp == 0 ? 0 : __shfl_sync(~0u, w, warp == 0 ? 0 : warp - 1);
  return before + x - v;
}

// A CTA per (request, KV head).  The key of the last token taken from the middle is found bit by
// bit: the largest key T with at least `want` middle keys >= T.  Then the positions are written in
// order: those above T, and the first ones equal to it.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
  __shared__ int buf[32];
  const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int L = p.L[r];
  int32_t *keep = p.keep + ((int64_t)r * p.Hkv + h) * p.budget;
  const bool bad = L < 0 || L > p.stride;
  const int n = bad ? 0 : min(L, p.budget);
  if (h == 0 && tid == 0) {
    p.new_lens[r] = n;
    if (bad && p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_CONTEXT);
  }
  for (int64_t i = n + tid; i < p.budget; i += kSelThreads) keep[i] = -1;
  if (n == L || bad) {
    for (int i = tid; i < n; i += kSelThreads) keep[i] = i;
    return;
  }
  const float *m = p.mass + ((int64_t)r * p.Hkv + h) * p.stride;
  const int lo = p.first, hi = L - p.recent, want = p.budget - p.first - p.recent;
  uint32_t T = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = T | (1u << bit);
    int c = 0;
    for (int64_t i = (int64_t)lo + tid; i < hi; i += kSelThreads) c += mass_key(m[i]) >= cand;
    if (block_sum(c, buf) >= want && want > 0) T = cand;
  }
  int above = 0;
  for (int64_t i = (int64_t)lo + tid; i < hi; i += kSelThreads) above += mass_key(m[i]) > T;
  int ties = want - block_sum(above, buf);  // equal keys that stay
  int at = 0;
  for (int64_t base = 0; base < L; base += kSelThreads) {
    const int64_t i = base + tid;
    const bool mid = i >= lo && i < hi && want > 0;
    const uint32_t k = mid ? mass_key(m[i]) : 0u;
    const bool eq = mid && k == T;
    int total;
    const int e = block_scan(eq, buf, &total);
    const bool stays = (i < L && (i < lo || i >= hi)) || (mid && (k > T || (eq && e < ties)));
    ties -= min(ties, total);
    const int x = block_scan(stays, buf, &total);
    if (stays) keep[at + x] = (int32_t)i;
    at += total;
  }
}

// -------------------------------------------------------------------------- compaction

struct CompactParams {
  const int32_t *keep, *new_lens, *bt, *dt;
  uint8_t *k, *v;
  float *ks, *vs;
  const float *mass;
  float *mass_out;
  uint32_t *status;
  int64_t num_pages;
  int32_t Hkv, ps, ps_shift, row_chunks, keep_stride, bt_stride, dt_stride, m_stride, mo_stride;
  int32_t in_place;
};

constexpr int kMoveThreads = 512;

// A CTA per (request, KV head), in rounds of kMoveThreads / row_chunks tokens: the round's rows are
// read into registers, then written.  Kept positions ascend, so keep[i] >= i: a round's
// destinations are sources of this round or an earlier one only, whose reads are done.
__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const CompactParams p) {
  const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int32_t *keep = p.keep + ((int64_t)r * p.Hkv + h) * p.keep_stride;
  int n = p.new_lens[r];
  if (n < 0 || n > p.keep_stride || ((int64_t)n + p.ps - 1) >> p.ps_shift > p.dt_stride ||
      (p.mass != nullptr && n > p.mo_stride)) {
    if (h == 0 && tid == 0 && p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_KEEP);
    n = 0;
  }
  const int per = kMoveThreads / p.row_chunks, c = tid % p.row_chunks, row_bytes = 16 * p.row_chunks;
  for (int64_t base = 0; base < n; base += per) {
    const int64_t i = base + tid / p.row_chunks;
    uint4 kx, vx;
    float ksx = 0.f, vsx = 0.f, mx = 0.f;
    int64_t to = -1;
    if (i < n) {
      const int s = keep[i], prev = i > 0 ? keep[i - 1] : -1;
      uint32_t fl = 0;
      if (s <= prev || s < i || s >> p.ps_shift >= p.bt_stride || (p.mass != nullptr && s >= p.m_stride))
        fl = PA_DEV_BAD_KEEP;
      int sp = -1, dp = -1;
      if (!fl) {
        sp = p.bt[(int64_t)r * p.bt_stride + (s >> p.ps_shift)];
        dp = p.dt[(int64_t)r * p.dt_stride + (i >> p.ps_shift)];
        if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) fl = PA_DEV_BAD_PAGE;
      }
      if (fl) {
        if (c == 0 && p.status != nullptr) atomicOr(p.status, fl);
      } else if (!p.in_place || s != i) {
        const int64_t from = (((int64_t)sp * p.Hkv + h) << p.ps_shift) + (s & (p.ps - 1));
        to = (((int64_t)dp * p.Hkv + h) << p.ps_shift) + (i & (p.ps - 1));
        kx = *reinterpret_cast<const uint4 *>(p.k + from * row_bytes + 16 * c);
        vx = *reinterpret_cast<const uint4 *>(p.v + from * row_bytes + 16 * c);
        if (c == 0) {
          if (p.ks != nullptr) {
            ksx = p.ks[from];
            vsx = p.vs[from];
          }
          if (p.mass != nullptr) mx = p.mass[((int64_t)r * p.Hkv + h) * p.m_stride + s];
        }
      }
    }
    __syncthreads();
    if (to >= 0) {
      *reinterpret_cast<uint4 *>(p.k + to * row_bytes + 16 * c) = kx;
      *reinterpret_cast<uint4 *>(p.v + to * row_bytes + 16 * c) = vx;
      if (c == 0) {
        if (p.ks != nullptr) {
          p.ks[to] = ksx;
          p.vs[to] = vsx;
        }
        if (p.mass != nullptr) p.mass_out[((int64_t)r * p.Hkv + h) * p.mo_stride + i] = mx;
      }
    }
    __syncthreads();
  }
}

}  // namespace

extern "C" pa_status_t pa_evict_select(const pa_evict_select_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_kv_heads < 1 || a->mass_stride < 1 || a->budget < 1 || a->keep_first < 0 ||
      a->keep_recent < 0 || (int64_t)a->keep_first + a->keep_recent > a->budget || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (a->num_kv_heads > pa_host::kMaxHeads || a->num_seqs > kMaxSeqs) return PA_ERR_UNSUPPORTED;
  if (a->mass == nullptr || a->context_lens == nullptr || a->keep == nullptr || a->new_lens == nullptr ||
      (const int32_t *)a->new_lens == a->context_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(a->mass, 4) || !aligned(a->context_lens, 4) || !aligned(a->keep, 4) ||
      !aligned(a->new_lens, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  if (a->num_seqs == 0) return PA_OK;
  SelectParams p;
  p.mass = a->mass;
  p.L = a->context_lens;
  p.keep = a->keep;
  p.new_lens = a->new_lens;
  p.status = a->status;
  p.Hkv = a->num_kv_heads;
  p.stride = a->mass_stride;
  p.budget = a->budget;
  p.first = a->keep_first;
  p.recent = a->keep_recent;
  (void)cudaGetLastError();  // drop an earlier, unrelated launch error
  evict_select_kernel<<<dim3(a->num_kv_heads, a->num_seqs), kSelThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status_t pa_kv_compact(const pa_kv_compact_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  const bool in_place = a->dst_block_table == nullptr;
  if (a->num_seqs < 0 || a->keep_stride < 1 || a->block_table_stride < 1 ||
      (!in_place && a->dst_block_table_stride < 1) || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  const pa_status_t st = pa_host::check_cache(a->num_pages, a->num_kv_heads, a->head_dim, a->page_size,
                                              a->kv_dtype, a->scale_mode);
  if (st != PA_OK) return st;
  if (a->num_seqs > kMaxSeqs) return PA_ERR_UNSUPPORTED;
  const bool per_token = a->scale_mode == PA_SCALE_PER_TOKEN;
  if (a->keep == nullptr || a->new_lens == nullptr || a->block_table == nullptr || a->k_cache == nullptr ||
      a->v_cache == nullptr || (per_token && (a->k_scale == nullptr || a->v_scale == nullptr)))
    return PA_ERR_INVALID_ARG;
  if (a->mass != nullptr) {
    if (a->mass_out == nullptr || a->mass_stride < 1 || a->mass_out_stride < 1) return PA_ERR_INVALID_ARG;
    const uint64_t rows = (uint64_t)a->num_seqs * a->num_kv_heads * sizeof(float);
    if (in_place ? (a->mass_out != a->mass || a->mass_out_stride != a->mass_stride)
                 : pa_host::overlap(a->mass, rows * a->mass_stride, a->mass_out, rows * a->mass_out_stride))
      return PA_ERR_INVALID_ARG;
  }
  if (!aligned(a->keep, 4) || !aligned(a->new_lens, 4) || !aligned(a->block_table, 4) ||
      !aligned(a->dst_block_table, 4) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) ||
      (per_token && (!aligned(a->k_scale, 4) || !aligned(a->v_scale, 4))) || !aligned(a->mass, 4) ||
      !aligned(a->mass_out, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  if (a->num_seqs == 0) return PA_OK;
  CompactParams p;
  p.keep = a->keep;
  p.new_lens = a->new_lens;
  p.bt = a->block_table;
  p.dt = in_place ? a->block_table : a->dst_block_table;
  p.k = static_cast<uint8_t *>(a->k_cache);
  p.v = static_cast<uint8_t *>(a->v_cache);
  p.ks = per_token ? a->k_scale : nullptr;
  p.vs = per_token ? a->v_scale : nullptr;
  p.mass = a->mass;
  p.mass_out = a->mass_out;
  p.status = a->status;
  p.num_pages = a->num_pages;
  p.Hkv = a->num_kv_heads;
  p.ps = a->page_size;
  p.ps_shift = pa_host::log2_page(a->page_size);
  p.row_chunks = a->kv_dtype == PA_KV_BF16 ? 16 : 8;
  p.keep_stride = a->keep_stride;
  p.bt_stride = a->block_table_stride;
  p.dt_stride = in_place ? a->block_table_stride : a->dst_block_table_stride;
  p.m_stride = a->mass_stride;
  p.mo_stride = a->mass_out_stride;
  p.in_place = in_place;
  (void)cudaGetLastError();  // drop an earlier, unrelated launch error
  kv_compact_kernel<<<dim3(a->num_kv_heads, a->num_seqs), kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
