// pa_mass.cu -- attention mass: pa_attn_mass adds one decode step's attention weights to the
// mass of the cached tokens.  See include/pa.h for the contract.
//
//   w[p] = sum over rows t, heads g of exp(sm_scale q[t][g] . k[p] k_scale[p] - lse[t][g])
//
// A thread per cached token: it reads the token's K row once per query row and keeps the 16
// heads' products in registers; the query rows sit in shared memory as fp32.  With the
// log-sum-exp known beforehand the weights need no running maximum and no second pass.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kG = 16;          // query heads per KV head
constexpr int kD = pa_host::kD;
constexpr int kTile = 128;      // tokens per CTA
constexpr int kMaxSeqs = 4096;
constexpr int kMaxQ = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct MassParams {
  const uint16_t *q;
  const uint8_t *k;
  const float *ks;
  const int32_t *bt, *L, *cu;
  const float *lse, *mass;
  float *out;
  uint32_t *status;
  int64_t num_pages;
  int32_t B, R, Hkv, ps, ps_shift, bt_stride, mass_stride, maxq, bf16;
  float kfold, decay;  // kfold = sm_scale * log2 e (* k_scale_scalar)
};

__global__ void __launch_bounds__(kTile) attn_mass_kernel(const MassParams p) {
  __shared__ float qs[kG][kD];
  __shared__ float l2[kG];
  const int h = blockIdx.y, r = blockIdx.z, tid = threadIdx.x;
  const int L = p.L[r], row0 = p.cu[r], ql = p.cu[r + 1] - row0;
  uint32_t fl = 0;
  if (L < 0 || L > p.mass_stride || ((int64_t)L + p.ps - 1) >> p.ps_shift > p.bt_stride)
    fl |= PA_DEV_BAD_CONTEXT;
  if (ql < 0 || ql > p.maxq || L < ql || row0 < 0 || row0 > p.R - ql) fl |= PA_DEV_BAD_QLEN;
  if (fl) {
    if (blockIdx.x == 0 && h == 0 && tid == 0 && p.status != nullptr) atomicOr(p.status, fl);
    return;
  }
  const int64_t base = (int64_t)blockIdx.x * kTile;
  if (ql == 0 || base >= L) return;
  const int pos = (int)base + tid;
  const bool live = pos < L;
  int64_t krow = -1;
  if (live) {
    const int page = p.bt[(int64_t)r * p.bt_stride + (pos >> p.ps_shift)];
    if (page < 0 || page >= p.num_pages) {
      if (p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_PAGE);
    } else {
      krow = (((int64_t)page * p.Hkv + h) << p.ps_shift) + (pos & (p.ps - 1));
    }
  }
  const float c = krow < 0 ? 0.f : (p.ks != nullptr ? p.kfold * p.ks[krow] : p.kfold);
  const int64_t Hq = (int64_t)p.Hkv * kG;
  float w = 0.f;
  for (int t = 0; t < ql; ++t) {
    const int64_t qrow = (int64_t)(row0 + t) * Hq + h * kG;
    __syncthreads();
    for (int i = tid; i < kG * kD; i += kTile)
      qs[i / kD][i % kD] = __uint_as_float((uint32_t)p.q[qrow * kD + i] << 16);
    if (tid < kG) l2[tid] = p.lse[qrow + tid] * kLog2e;
    __syncthreads();
    if (krow < 0 || pos >= L - ql + t + 1) continue;
    float acc[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) acc[g] = 0.f;
    for (int d0 = 0; d0 < kD; d0 += 8) {
      float x[8];
      if (p.bf16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p.k + krow * (2 * kD) + 2 * d0);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[2 * j] = pa::bf16lo(u[j]);
          x[2 * j + 1] = pa::bf16hi(u[j]);
        }
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p.k + krow * kD + d0);
        pa::e4m3x2_to_f32x2(v.x & 0xFFFFu, x[0], x[1]);
        pa::e4m3x2_to_f32x2(v.x >> 16, x[2], x[3]);
        pa::e4m3x2_to_f32x2(v.y & 0xFFFFu, x[4], x[5]);
        pa::e4m3x2_to_f32x2(v.y >> 16, x[6], x[7]);
      }
#pragma unroll
      for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[g] = fmaf(qs[g][d0 + j], x[j], acc[g]);
    }
#pragma unroll
    for (int g = 0; g < kG; ++g)
      if (l2[g] != -INFINITY) w += pa::fast_exp2(fmaf(acc[g], c, -l2[g]));
  }
  if (live) {
    const int64_t o = ((int64_t)r * p.Hkv + h) * p.mass_stride + pos;
    const float old = pos < L - ql && p.decay != 0.f ? p.decay * p.mass[o] : 0.f;
    p.out[o] = old + w;
  }
}

}  // namespace

extern "C" pa_status_t pa_attn_mass(const pa_attn_mass_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_rows < 0 || a->max_q_len < 1 || a->block_table_stride < 1 ||
      a->mass_stride < 1 || a->reserved != 0 || !(a->sm_scale > 0.f) ||
      !std::isfinite(a->sm_scale) || !(a->decay >= 0.f && a->decay <= 1.f))
    return PA_ERR_INVALID_ARG;
  const pa_status_t st = pa_host::check_cache(a->num_pages, a->num_kv_heads, a->head_dim, a->page_size,
                                              a->kv_dtype, a->scale_mode);
  if (st != PA_OK) return st;
  if (a->group_size != kG || a->max_q_len > kMaxQ || a->num_seqs > kMaxSeqs) return PA_ERR_UNSUPPORTED;
  if (a->scale_mode == PA_SCALE_SCALAR && (!std::isfinite(a->k_scale_scalar) || a->k_scale_scalar < 0.f))
    return PA_ERR_INVALID_ARG;
  const bool per_token = a->scale_mode == PA_SCALE_PER_TOKEN;
  if (a->q == nullptr || a->k_cache == nullptr || a->block_table == nullptr || a->context_lens == nullptr ||
      a->cu_seqlens_q == nullptr || a->lse == nullptr || a->mass_out == nullptr ||
      (a->mass == nullptr && a->decay != 0.f) || (per_token && a->k_scale == nullptr))
    return PA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->k_cache, 16) || (per_token && !aligned(a->k_scale, 16)) ||
      !aligned(a->block_table, 4) || !aligned(a->context_lens, 4) || !aligned(a->cu_seqlens_q, 4) ||
      !aligned(a->lse, 4) || !aligned(a->mass, 4) || !aligned(a->mass_out, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  const uint64_t bytes = (uint64_t)a->num_seqs * a->num_kv_heads * a->mass_stride * sizeof(float);
  if (a->mass != nullptr && a->mass != a->mass_out && pa_host::overlap(a->mass, bytes, a->mass_out, bytes))
    return PA_ERR_INVALID_ARG;
  if (a->num_seqs == 0 || a->num_rows == 0) return PA_OK;

  MassParams p;
  p.q = static_cast<const uint16_t *>(a->q);
  p.k = static_cast<const uint8_t *>(a->k_cache);
  p.ks = per_token ? a->k_scale : nullptr;
  p.bt = a->block_table;
  p.L = a->context_lens;
  p.cu = a->cu_seqlens_q;
  p.lse = a->lse;
  p.mass = a->mass;
  p.out = a->mass_out;
  p.status = a->status;
  p.num_pages = a->num_pages;
  p.B = a->num_seqs;
  p.R = a->num_rows;
  p.Hkv = a->num_kv_heads;
  p.ps = a->page_size;
  p.ps_shift = pa_host::log2_page(a->page_size);
  p.bt_stride = a->block_table_stride;
  p.mass_stride = a->mass_stride;
  p.maxq = a->max_q_len;
  p.bf16 = a->kv_dtype == PA_KV_BF16;
  p.kfold = (float)((double)a->sm_scale * 1.4426950408889634 *
                    (a->scale_mode == PA_SCALE_SCALAR ? (double)a->k_scale_scalar : 1.0));
  p.decay = a->decay;
  (void)cudaGetLastError();  // drop an earlier, unrelated launch error
  const dim3 grid((unsigned)(((int64_t)a->mass_stride + kTile - 1) / kTile), a->num_kv_heads, a->num_seqs);
  attn_mass_kernel<<<grid, kTile, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
