// pa_beam.cu -- beam search over the paged cache: pa_beam_select picks the beams that go on,
// pa_beam_reorder lets their block tables, last pages and states follow.  See include/pa.h for
// the contract.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kD = pa_host::kD;
constexpr int kMaxBeams = 32;
constexpr int kMaxVocab = 1 << 24;
constexpr int kMaxReqs = 65535;

// --------------------------------------------------------------------------- selection

struct BeamParams {
  const void *logits;
  const float *scores;
  const uint8_t *finished;
  const int32_t *lengths;
  int32_t *tokens, *parents;
  float *scores_out;
  uint8_t *finished_out;
  int32_t *lengths_out;
  int64_t stride;
  int32_t W, V, f32, eos;
  float penalty;
};

__device__ __forceinline__ float logit(const BeamParams &p, int64_t row, int v) {
  const int64_t i = row * p.stride + v;
  if (p.f32) return static_cast<const float *>(p.logits)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p.logits)[i] << 16);
}

// Keys that order (value, index) pairs: larger value first, then lower index; NaN is -inf.  The
// largest key is the best pair.
__device__ __forceinline__ unsigned long long pair_key(float x, int v) {
  const float y = x != x ? -INFINITY : x + 0.f;  // -0 = +0
  const uint32_t u = __float_as_uint(y);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)o << 32) | (0xFFFFFFFFu - (uint32_t)v);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return (int)(0xFFFFFFFFu - (uint32_t)(k & 0xFFFFFFFFull));
}
// Ordered bits of a double that is not NaN; greater than 0 for every such double.
__device__ __forceinline__ unsigned long long rank_key(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

constexpr int kBeamThreads = 1024;

__device__ unsigned long long block_max(unsigned long long k, unsigned long long *buf) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(~0u, k, o);
    k = k > y ? k : y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = k;
  __syncthreads();
  k = buf[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(~0u, k, o);
    k = k > y ? k : y;
  }
  return k;
}

// A CTA per request.  For every beam: the row's log-sum-exp, then its W best tokens, one
// reduction over the row each; then one warp merges the beams' lists, a lane per beam.
__global__ void __launch_bounds__(kBeamThreads) beam_select_kernel(const BeamParams p) {
  __shared__ unsigned long long buf[32];
  __shared__ double dbuf[32];
  __shared__ unsigned long long list[kMaxBeams][kMaxBeams];  // [beam][k]: the k-th best (logit, token)
  __shared__ double lse[kMaxBeams];
  const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = 0; b < p.W; ++b) {
    const int64_t row = (int64_t)n * p.W + b;
    unsigned long long best = 0;
    for (int v = tid; v < p.V; v += kBeamThreads) {
      const unsigned long long k = pair_key(logit(p, row, v), v);
      best = k > best ? k : best;
    }
    best = block_max(best, buf);
    const float m = key_value(best);
    double s = 0.0;
    for (int v = tid; v < p.V; v += kBeamThreads)
      s += pa::fast_exp2((logit(p, row, v) - m) * 1.4426950408889634f);  // NaN for NaN, and for +-inf - itself
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    __syncthreads();
    if (lane == 0) dbuf[warp] = s;
    __syncthreads();
    s = dbuf[lane];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (tid == 0) lse[b] = (double)m + log(s);
    for (int k = 0; k < p.W; ++k) {
      if (tid == 0) list[b][k] = best;
      if (k + 1 == p.W) break;
      unsigned long long next = 0;
      for (int v = tid; v < p.V; v += kBeamThreads) {
        const unsigned long long key = pair_key(logit(p, row, v), v);
        if (key < best && key > next) next = key;
      }
      best = block_max(next, buf);  // 0 once the vocabulary is used up
    }
  }
  __syncthreads();
  if (warp != 0) return;
  // Lane b walks beam b's candidates in order: `at` counts those taken.
  const bool mine = lane < p.W;
  const int64_t me = (int64_t)n * p.W + lane;
  const float cum = mine ? p.scores[me] : -INFINITY;
  const bool done = mine && p.finished != nullptr && p.finished[me] != 0;
  const int len = mine && p.lengths != nullptr ? p.lengths[me] : 0;
  const int newlen = done ? len : (len == INT_MAX ? len : len + 1);
  const double norm = p.penalty == 0.f ? 1.0 : pow((double)max(newlen, 1), (double)p.penalty);
  // no continuation at a number: every candidate counts as -inf
  const bool dead = mine && (cum != cum || cum == -INFINITY || (!done && !(fabs(lse[mine ? lane : 0]) < INFINITY)));
  int at = 0;
  for (int j = 0; j < p.W; ++j) {
    unsigned long long key = 0;
    int tok = -1;
    double total = -INFINITY;
    if (mine && at < p.V) {
      if (dead) {
        tok = at;
      } else if (done) {
        tok = at == 0 ? p.eos : (at <= p.eos ? at - 1 : at);
        if (at == 0) total = (double)cum;
      } else {
        tok = key_index(list[lane][at]);
        total = (double)cum + ((double)key_value(list[lane][at]) - lse[lane]);
        if (total != total) total = -INFINITY;
      }
      key = rank_key(total / norm);
    }
    unsigned long long top = key;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(~0u, top, o);
      top = top > y ? top : y;
    }
    const int win = __ffs(__ballot_sync(~0u, key == top)) - 1;  // equal ranks: the lower beam
    if (lane == win) {
      const int64_t o = (int64_t)n * p.W + j;
      p.tokens[o] = tok;
      p.parents[o] = lane;
      p.scores_out[o] = (float)total;
      if (p.finished_out != nullptr) p.finished_out[o] = done || (p.eos >= 0 && tok == p.eos);
      if (p.lengths_out != nullptr) p.lengths_out[o] = newlen;
      ++at;
    }
  }
}

// -------------------------------------------------------------------------- reordering

struct ReorderParams {
  const int32_t *parents, *L, *bt;
  int32_t *bt_out;
  uint8_t *k, *v;
  float *ks, *vs;
  uint32_t *status;
  const uint8_t *sin[PA_MAX_BEAM_STATES];
  uint8_t *sout[PA_MAX_BEAM_STATES];
  int64_t sbytes[PA_MAX_BEAM_STATES];
  int32_t sunit[PA_MAX_BEAM_STATES];  // bytes per access: 16, 4 or 1
  int64_t num_pages;
  int32_t W, Hkv, ps, ps_shift, row_chunks, stride, num_states;
};

constexpr int kReorderThreads = 256;

template <typename T>
__device__ void copy_row(const uint8_t *src, uint8_t *dst, int64_t n, int64_t i, int64_t step) {
  for (; i < n; i += step) reinterpret_cast<T *>(dst)[i] = reinterpret_cast<const T *>(src)[i];
}

// Row j = blockIdx.y of a request: its table row (CTA x = 0), its share of the copy of the partial
// page, its share of the states.  Every CTA works the request's parents out by itself, a lane per beam.
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const ReorderParams p) {
  const int n = blockIdx.y / p.W, j = blockIdx.y % p.W, tid = threadIdx.x, lane = tid & 31;
  const int64_t base = (int64_t)n * p.W, row = base + j;
  const unsigned beams = p.W == 32 ? ~0u : (1u << p.W) - 1u;
  int par = lane < p.W ? p.parents[base + lane] : 0;
  const int L = p.L[base];
  uint32_t fl = 0;
  if (__any_sync(~0u, lane < p.W && (par < 0 || par >= p.W || p.L[base + lane] != L))) fl |= PA_DEV_BAD_BEAM;
  if (L < 0 || ((int64_t)L + p.ps - 1) >> p.ps_shift > p.stride) fl |= PA_DEV_BAD_CONTEXT;
  if (fl) {
    par = lane < p.W ? lane : 0;
    if (blockIdx.x == 0 && j == 0 && tid == 0 && p.status != nullptr) atomicOr(p.status, fl);
  }
  // first child of its parent; beams without children
  bool first = lane < p.W;
  unsigned alive = 0;
  for (int b = 0; b < p.W; ++b) {
    const int pb = __shfl_sync(~0u, par, b);
    if (b < lane && pb == par) first = false;
    alive |= 1u << pb;
  }
  const unsigned extra = __ballot_sync(~0u, lane < p.W && !first);
  const int parent = __shfl_sync(~0u, par, j);
  int giver = parent;  // whose partial page row j takes
  const bool copies = (extra >> j) & 1u;
  if (copies) {
    unsigned dead = beams & ~alive;
    for (int k = __popc(extra & ((1u << j) - 1u)); k > 0; --k) dead &= dead - 1u;
    giver = __ffs(dead) - 1;
  }
  const int full = fl ? 0 : L >> p.ps_shift, part = fl ? 0 : L & (p.ps - 1);
  const int64_t prow = base + parent, grow = base + giver;
  if (blockIdx.x == 0)
    for (int i = tid; i < p.stride; i += kReorderThreads)
      p.bt_out[row * p.stride + i] = p.bt[(i < full ? prow : (i == full && part > 0 ? grow : row)) * p.stride + i];
  const int64_t gid = (int64_t)blockIdx.x * kReorderThreads + tid, step = (int64_t)gridDim.x * kReorderThreads;
  if (copies && part > 0) {
    const int from = p.bt[prow * p.stride + full], to = p.bt[grow * p.stride + full];
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
      if (gid == 0 && p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_PAGE);
    } else {
      const int row_bytes = 16 * p.row_chunks;
      const int64_t units = (int64_t)p.Hkv * part * p.row_chunks;
      for (int64_t u = gid; u < units; u += step) {
        const int c = (int)(u % p.row_chunks);
        const int64_t t = u / p.row_chunks;
        const int h = (int)(t / part), s = (int)(t % part);
        const int64_t a = (((int64_t)from * p.Hkv + h) << p.ps_shift) + s;
        const int64_t b = (((int64_t)to * p.Hkv + h) << p.ps_shift) + s;
        *reinterpret_cast<uint4 *>(p.k + b * row_bytes + 16 * c) =
            *reinterpret_cast<const uint4 *>(p.k + a * row_bytes + 16 * c);
        *reinterpret_cast<uint4 *>(p.v + b * row_bytes + 16 * c) =
            *reinterpret_cast<const uint4 *>(p.v + a * row_bytes + 16 * c);
        if (c == 0 && p.ks != nullptr) {
          p.ks[b] = p.ks[a];
          p.vs[b] = p.vs[a];
        }
      }
    }
  }
  for (int k = 0; k < p.num_states; ++k) {
    const uint8_t *src = p.sin[k] + prow * p.sbytes[k];
    uint8_t *dst = p.sout[k] + row * p.sbytes[k];
    if (p.sunit[k] == 16)
      copy_row<uint4>(src, dst, p.sbytes[k] / 16, gid, step);
    else if (p.sunit[k] == 4)
      copy_row<uint32_t>(src, dst, p.sbytes[k] / 4, gid, step);
    else
      copy_row<uint8_t>(src, dst, p.sbytes[k], gid, step);
  }
}

}  // namespace

extern "C" pa_status_t pa_beam_select(const pa_beam_select_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_reqs < 0 || a->num_beams < 1 || a->vocab < 1 || a->logits_stride < a->vocab || a->reserved != 0 ||
      (a->logits_dtype != PA_LOGITS_BF16 && a->logits_dtype != PA_LOGITS_F32) || a->eos_token < -1 ||
      a->eos_token >= a->vocab || !(a->length_penalty >= 0.f) || !std::isfinite(a->length_penalty))
    return PA_ERR_INVALID_ARG;
  if (a->num_beams > kMaxBeams || a->vocab > kMaxVocab || a->num_reqs > kMaxReqs) return PA_ERR_UNSUPPORTED;
  if (a->logits == nullptr || a->scores == nullptr || a->tokens == nullptr || a->parents == nullptr ||
      a->scores_out == nullptr || (a->finished != nullptr && a->eos_token < 0) ||
      (a->lengths == nullptr && (a->length_penalty != 0.f || a->lengths_out != nullptr)))
    return PA_ERR_INVALID_ARG;
  if (!aligned(a->logits, a->logits_dtype == PA_LOGITS_F32 ? 4 : 2) || !aligned(a->scores, 4) ||
      !aligned(a->lengths, 4) || !aligned(a->tokens, 4) || !aligned(a->parents, 4) || !aligned(a->scores_out, 4) ||
      !aligned(a->lengths_out, 4))
    return PA_ERR_ALIGN;
  if (a->num_reqs == 0) return PA_OK;
  BeamParams p;
  p.logits = a->logits;
  p.scores = a->scores;
  p.finished = a->finished;
  p.lengths = a->lengths;
  p.tokens = a->tokens;
  p.parents = a->parents;
  p.scores_out = a->scores_out;
  p.finished_out = a->finished_out;
  p.lengths_out = a->lengths_out;
  p.stride = a->logits_stride;
  p.W = a->num_beams;
  p.V = a->vocab;
  p.f32 = a->logits_dtype == PA_LOGITS_F32;
  p.eos = a->eos_token;
  p.penalty = a->length_penalty;
  (void)cudaGetLastError();  // drop an earlier, unrelated launch error
  beam_select_kernel<<<a->num_reqs, kBeamThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status_t pa_beam_reorder(const pa_beam_reorder_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_reqs < 0 || a->num_beams < 1 || a->block_table_stride < 1 || a->num_states < 0 ||
      a->num_states > PA_MAX_BEAM_STATES || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  const pa_status_t st = pa_host::check_cache(a->num_pages, a->num_kv_heads, a->head_dim, a->page_size,
                                              a->kv_dtype, a->scale_mode);
  if (st != PA_OK) return st;
  if (a->num_beams > kMaxBeams || (int64_t)a->num_reqs * a->num_beams > kMaxReqs) return PA_ERR_UNSUPPORTED;
  const bool per_token = a->scale_mode == PA_SCALE_PER_TOKEN;
  if (a->parents == nullptr || a->context_lens == nullptr || a->block_table == nullptr ||
      a->block_table_out == nullptr || a->k_cache == nullptr || a->v_cache == nullptr ||
      (per_token && (a->k_scale == nullptr || a->v_scale == nullptr)))
    return PA_ERR_INVALID_ARG;
  const uint64_t rows = (uint64_t)a->num_reqs * a->num_beams;
  const uint64_t tbytes = rows * a->block_table_stride * sizeof(int32_t);
  if (pa_host::overlap(a->block_table, tbytes, a->block_table_out, tbytes)) return PA_ERR_INVALID_ARG;
  int64_t widest = 0;
  for (int k = 0; k < a->num_states; ++k) {
    if (a->state_in[k] == nullptr || a->state_out[k] == nullptr || a->state_bytes[k] < 1 ||
        a->state_bytes[k] > (INT64_MAX >> 17))
      return PA_ERR_INVALID_ARG;
    const uint64_t n = rows * (uint64_t)a->state_bytes[k];
    for (int i = 0; i <= k; ++i) {
      const uint64_t ni = rows * (uint64_t)a->state_bytes[i];
      if (pa_host::overlap(a->state_in[i], ni, a->state_out[k], n) ||
          pa_host::overlap(a->state_in[k], n, a->state_out[i], ni) ||
          (i != k && pa_host::overlap(a->state_out[i], ni, a->state_out[k], n)))
        return PA_ERR_INVALID_ARG;
    }
    widest = a->state_bytes[k] > widest ? a->state_bytes[k] : widest;
  }
  if (!aligned(a->parents, 4) || !aligned(a->context_lens, 4) || !aligned(a->block_table, 4) ||
      !aligned(a->block_table_out, 4) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) ||
      (per_token && (!aligned(a->k_scale, 4) || !aligned(a->v_scale, 4))) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  if (a->num_reqs == 0) return PA_OK;
  ReorderParams p;
  p.parents = a->parents;
  p.L = a->context_lens;
  p.bt = a->block_table;
  p.bt_out = a->block_table_out;
  p.k = static_cast<uint8_t *>(a->k_cache);
  p.v = static_cast<uint8_t *>(a->v_cache);
  p.ks = per_token ? a->k_scale : nullptr;
  p.vs = per_token ? a->v_scale : nullptr;
  p.status = a->status;
  p.num_pages = a->num_pages;
  p.W = a->num_beams;
  p.Hkv = a->num_kv_heads;
  p.ps = a->page_size;
  p.ps_shift = pa_host::log2_page(a->page_size);
  p.row_chunks = a->kv_dtype == PA_KV_BF16 ? 16 : 8;
  p.stride = a->block_table_stride;
  p.num_states = a->num_states;
  for (int k = 0; k < a->num_states; ++k) {
    p.sin[k] = static_cast<const uint8_t *>(a->state_in[k]);
    p.sout[k] = static_cast<uint8_t *>(a->state_out[k]);
    p.sbytes[k] = a->state_bytes[k];
    const uintptr_t all = reinterpret_cast<uintptr_t>(p.sin[k]) | reinterpret_cast<uintptr_t>(p.sout[k]) |
                          static_cast<uintptr_t>(p.sbytes[k]);
    p.sunit[k] = all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : 1);
  }
  // a CTA for each 16 KB of the row's widest part
  const int64_t page_bytes = (int64_t)a->num_kv_heads * a->page_size * 16 * p.row_chunks;
  int64_t gx = ((page_bytes > widest ? page_bytes : widest) + 16383) / 16384;
  gx = gx < 1 ? 1 : (gx > 64 ? 64 : gx);
  (void)cudaGetLastError();  // drop an earlier, unrelated launch error
  beam_reorder_kernel<<<dim3((unsigned)gx, a->num_reqs * a->num_beams), kReorderThreads, 0,
                        static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
