// pa_rope.cu -- rotary positions of queries and keys: pa_rope.  See include/pa.h for the contract.
//
// Bound by HBM: every element is read and written once.  16384 tokens x 17 heads, bf16, 143 MB: 25.5 us, 5.6 TB/s (0.83 of a
// copy's); 32 tokens 1.6 us.  A thread's first elements asked for before the angles are worked out: no faster (registers, so fewer
// threads).  A CTA takes kTokens tokens (one where there
// are few): first a thread per (token, pair) works out cosine and sine into shared memory, then a
// thread per two accesses of a head turns them, of 16 bytes where alignment and the number of turning pairs allow
// it and of 8, 4 or 2 where not (half layout: 8 elements at a time need a multiple of 16 turning ones).  A token's cosines serve all its heads.
//
// The angle of pair i at position p is p * freqs[i] / 2^64 turns: the 64-bit product modulo 2^64 is the
// fraction of a turn without any rounding.  The nearest quarter turn is taken off it as an integer, and what is
// left, at most an eighth either way, becomes a float with 24 bits of its own.
#include <cuda_bf16.h>
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
constexpr int kThreads = 192;  // (256: 8.9 us, not 7.7, for 4096 tokens x 17 heads, bf16)
constexpr int kTokens = 4;    // per CTA (2 and 8: 30 and 27 us, not 26, for 16384 x 17)

struct RopeParams {
  const void *q, *k;
  const int32_t *pos;
  const int64_t *freqs;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int32_t T, hq, heads, rot;  // heads: hq and the keys'
  float scale, sign;
};

// E consecutive elements as floats: 16, 8, 4 or 2 bytes in one access.
template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
  using type = uint4;
};
template <>
struct Raw<8> {
  using type = uint2;
};
template <>
struct Raw<4> {
  using type = uint32_t;
};
template <>
struct Raw<2> {
  using type = uint16_t;
};

template <typename T, int E>
struct Vec {
  using R = typename Raw<E * sizeof(T)>::type;
  float x[E];
  __device__ __forceinline__ void load(const T *p) {
    const R w = *reinterpret_cast<const R *>(p);
    if constexpr (sizeof(R) == 2) {
      x[0] = __uint_as_float((uint32_t)w << 16);
    } else {
      alignas(16) uint32_t v[sizeof(R) / 4];
      *reinterpret_cast<R *>(v) = w;
#pragma unroll
      for (int i = 0; i < (int)sizeof(R) / 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          x[2 * i] = pa::bf16lo(v[i]);
          x[2 * i + 1] = pa::bf16hi(v[i]);
        } else {
          x[i] = __uint_as_float(v[i]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (sizeof(R) == 2) {
      *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(x[0]);
    } else {
      alignas(16) uint32_t v[sizeof(R) / 4];
#pragma unroll
      for (int i = 0; i < (int)sizeof(R) / 4; ++i) {
        if constexpr (sizeof(T) == 2)
          v[i] = pa::pack_bf16x2(x[2 * i], x[2 * i + 1]);
        else
          v[i] = __float_as_uint(x[i]);
      }
      *reinterpret_cast<R *>(p) = *reinterpret_cast<const R *>(v);
    }
  }
};

// Cosine and sine of the CTA's tokens, a thread to a pair.
template <int TOK>
__device__ __forceinline__ void angles(const RopeParams &p, int t0, float (*cs)[kD / 2], float (*sn)[kD / 2]) {
  const int tid = threadIdx.x, half = p.rot >> 1;
  for (int u = tid; u < TOK * (kD / 2); u += kThreads) {
    const int t = u / (kD / 2), i = u % (kD / 2);
    if (t0 + t >= p.T || i >= half) continue;
    const uint64_t turn = (uint64_t)(int64_t)p.pos[t0 + t] * (uint64_t)p.freqs[i];
    const uint64_t quarter = (turn + (1ull << 61)) >> 62;  // the nearest one, 0 .. 3
    float s, c;
    sincospif(__ll2float_rn((int64_t)(turn - (quarter << 62))) * 0x1p-63f, &s, &c);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;  // |cos|, |sin| of the whole angle
    cs[t][i] = (quarter == 1 || quarter == 2 ? -a : a) * p.scale;
    sn[t][i] = (quarter >= 2 ? -b : b) * p.scale * p.sign;
  }
}

// T: uint16_t (bf16) or float; E: elements per access; HALF: the layout; TOK: tokens per CTA.
template <typename T, int E, bool HALF, int TOK>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float cs[TOK][kD / 2], sn[TOK][kD / 2];
  const int tid = threadIdx.x, t0 = blockIdx.x * TOK, half = p.rot >> 1;
  pa::pdl_wait();
  pa::pdl_launch_dependents();
  angles<TOK>(p, t0, cs, sn);
  __syncthreads();
  // units of two accesses, of all heads of all the CTA's tokens
  constexpr int kUnits = kD / E / 2;
  const int per_token = p.heads * kUnits, left = min(TOK, p.T - t0) * per_token;
  for (int u = tid; u < left; u += kThreads) {
    const int t = TOK == 1 ? 0 : u / per_token, v = u - t * per_token, h = v / kUnits, i = v % kUnits;
    const bool is_q = h < p.hq;
    const int64_t token = t0 + t;
    const T *src = is_q ? static_cast<const T *>(p.q) + token * p.q_stride + h * kD
                        : static_cast<const T *>(p.k) + token * p.k_stride + (h - p.hq) * kD;
    T *dst = is_q ? static_cast<T *>(p.q_out) + token * p.q_out_stride + h * kD
                  : static_cast<T *>(p.k_out) + token * p.k_out_stride + (h - p.hq) * kD;
    if constexpr (HALF) {
      const bool turns = i * E < half;
      const int a = turns ? i * E : i * E + half, b = turns ? half + i * E : i * E + kD / 2;  // what does not turn: in halves too
      if (!turns && src == dst) continue;
      Vec<T, E> x, y;
      x.load(src + a);
      y.load(src + b);
      if (turns) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float c = cs[t][i * E + e], s = sn[t][i * E + e], xa = x.x[e], xb = y.x[e];
          x.x[e] = fmaf(xa, c, -(xb * s));
          y.x[e] = fmaf(xb, c, xa * s);
        }
      }
      x.store(dst + a);
      y.store(dst + b);
    } else if constexpr (E == 1) {
      const bool turns = i < half;
      if (!turns && src == dst) continue;
      Vec<T, 1> x, y;
      x.load(src + 2 * i);
      y.load(src + 2 * i + 1);
      if (turns) {
        const float c = cs[t][i], s = sn[t][i], xa = x.x[0], xb = y.x[0];
        x.x[0] = fmaf(xa, c, -(xb * s));
        y.x[0] = fmaf(xb, c, xa * s);
      }
      x.store(dst + 2 * i);
      y.store(dst + 2 * i + 1);
    } else {
      // half a head apart, so that neighbours read neighbouring accesses (next to each other: 15.4 us, not 10.2, for 4096 tokens x 17
      // heads, fp32)
      Vec<T, E> x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) x[j].load(src + j * (kD / 2) + i * E);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int a = j * (kD / 2) + i * E;
        if (a < p.rot) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            if (a + e >= p.rot) break;
            const float c = cs[t][(a + e) >> 1], s = sn[t][(a + e) >> 1], xa = x[j].x[e], xb = x[j].x[e + 1];
            x[j].x[e] = fmaf(xa, c, -(xb * s));
            x[j].x[e + 1] = fmaf(xb, c, xa * s);
          }
        }
        x[j].store(dst + a);
      }
    }
  }
}

// Half layout with an odd number of turning pairs, not in place: the sides of a pair lie in accesses of their own.  A thread
// takes 16 bytes of a head and reads the elements' other sides one by one, from L1 (8192 tokens x 17 heads, 34 elements turning,
// bf16: 21 us; element by element throughout 33).
template <typename T, int TOK>
__global__ void __launch_bounds__(kThreads) rope_odd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int E = 16 / sizeof(T), kUnits = kD / E;
  __shared__ __align__(16) float cs[TOK][kD / 2], sn[TOK][kD / 2];
  const int tid = threadIdx.x, t0 = blockIdx.x * TOK, half = p.rot >> 1;
  pa::pdl_wait();
  pa::pdl_launch_dependents();
  angles<TOK>(p, t0, cs, sn);
  __syncthreads();
  const int per_token = p.heads * kUnits, left = min(TOK, p.T - t0) * per_token;
  for (int u = tid; u < left; u += kThreads) {
    const int t = TOK == 1 ? 0 : u / per_token, v = u - t * per_token, h = v / kUnits, a = v % kUnits * E;
    const bool is_q = h < p.hq;
    const int64_t token = t0 + t;
    const T *src = is_q ? static_cast<const T *>(p.q) + token * p.q_stride + h * kD
                        : static_cast<const T *>(p.k) + token * p.k_stride + (h - p.hq) * kD;
    T *dst = is_q ? static_cast<T *>(p.q_out) + token * p.q_out_stride + h * kD
                  : static_cast<T *>(p.k_out) + token * p.k_out_stride + (h - p.hq) * kD;
    Vec<T, E> x;
    x.load(src + a);
    if (a < p.rot) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int j = a + e;
        if (j < p.rot) {
          const bool first = j < half;
          const int i = first ? j : j - half;
          Vec<T, 1> other;
          other.load(src + (first ? j + half : i));
          const float c = cs[t][i], s = sn[t][i];
          x.x[e] = fmaf(x.x[e], c, first ? -(other.x[0] * s) : other.x[0] * s);
        }
      }
    }
    x.store(dst + a);
  }
}

template <typename T, int E, bool HALF>
cudaError_t launch(const RopeParams &p, bool few, void *stream) {
  const int tokens = few ? 1 : kTokens;
  const pa_host::Launch run(dim3((unsigned)((p.T + tokens - 1) / tokens)), dim3(kThreads), 0, stream);
  return few ? cudaLaunchKernelEx(run.cfg(), rope_kernel<T, E, HALF, 1>, p)
             : cudaLaunchKernelEx(run.cfg(), rope_kernel<T, E, HALF, kTokens>, p);
}

// `bytes`: what every row is aligned to, at most 16.
template <typename T>
cudaError_t launch(const RopeParams &p, bool half, int bytes, bool few, bool in_place, void *stream) {
  constexpr int kWide = 16 / sizeof(T);
  int e = bytes / (int)sizeof(T);
  if (!half) return e == kWide ? launch<T, kWide, false>(p, few, stream) : launch<T, 1, false>(p, few, stream);
  if (e == kWide && p.rot % 4 != 0 && !in_place) {
    const pa_host::Launch run(dim3((unsigned)((p.T + (few ? 1 : kTokens) - 1) / (few ? 1 : kTokens))), dim3(kThreads), 0, stream);
    return few ? cudaLaunchKernelEx(run.cfg(), rope_odd_kernel<T, 1>, p) : cudaLaunchKernelEx(run.cfg(), rope_odd_kernel<T, kTokens>, p);
  }
  while (e > 1 && (p.rot / 2) % e != 0) e /= 2;  // whole accesses on either side of the pairs
  if constexpr (sizeof(T) == 2)
    if (e == 8) return launch<T, 8, true>(p, few, stream);
  return e == 4   ? launch<T, 4, true>(p, few, stream)
         : e == 2 ? launch<T, 2, true>(p, few, stream)
                  : launch<T, 1, true>(p, few, stream);
}

}  // namespace

extern "C" pa_status_t pa_rope(const pa_rope_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  const bool keys = a->num_kv_heads > 0;
  if (a->num_tokens < 0 || a->num_q_heads < 1 || a->num_kv_heads < 0 || a->rot_dim < 2 || a->rot_dim > kD || a->rot_dim % 2 != 0 ||
      (a->dtype != PA_ROPE_BF16 && a->dtype != PA_ROPE_F32) || (a->layout != PA_ROPE_HALF && a->layout != PA_ROPE_PAIRS) ||
      (a->inverse != 0 && a->inverse != 1) || !std::isfinite(a->scale) || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (a->head_dim != kD) return PA_ERR_UNSUPPORTED;
  if ((int64_t)a->num_q_heads + a->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  const int64_t q_row = (int64_t)a->num_q_heads * kD, k_row = (int64_t)a->num_kv_heads * kD;
  constexpr int64_t kMost = 1ll << 40;  // elements between tokens
  if (a->q_stride < q_row || a->q_out_stride < q_row || a->q_stride > kMost || a->q_out_stride > kMost ||
      (keys && (a->k_stride < k_row || a->k_out_stride < k_row || a->k_stride > kMost || a->k_out_stride > kMost)))
    return PA_ERR_INVALID_ARG;
  if (a->q == nullptr || a->q_out == nullptr || a->positions == nullptr || a->freqs == nullptr ||
      (keys ? a->k == nullptr || a->k_out == nullptr : a->k != nullptr || a->k_out != nullptr))
    return PA_ERR_INVALID_ARG;
  const int size = a->dtype == PA_ROPE_BF16 ? 2 : 4;
  if (!aligned(a->q, size) || !aligned(a->k, size) || !aligned(a->q_out, size) || !aligned(a->k_out, size) || !aligned(a->positions, 4) ||
      !aligned(a->freqs, 8))
    return PA_ERR_ALIGN;
  if (a->num_tokens == 0) return PA_OK;
  using pa_host::Rows;
  const int64_t n = a->num_tokens;
  const Rows q{a->q, n, q_row * size, a->q_stride * size}, qo{a->q_out, n, q_row * size, a->q_out_stride * size},
      k{a->k, n, k_row * size, a->k_stride * size}, ko{a->k_out, n, k_row * size, a->k_out_stride * size},
      pos{a->positions, 1, n * 4, n * 4}, freqs{a->freqs, 1, a->rot_dim * 4, a->rot_dim * 4};
  const bool q_in_place = a->q_out == a->q && a->q_out_stride == a->q_stride;
  const bool k_in_place = a->k_out == a->k && a->k_out_stride == a->k_stride;
  if ((!q_in_place && pa_host::rows_overlap(qo, q)) || pa_host::rows_overlap(qo, pos) || pa_host::rows_overlap(qo, freqs) ||
      (keys && (pa_host::rows_overlap(qo, k) || pa_host::rows_overlap(qo, ko) || (!k_in_place && pa_host::rows_overlap(ko, k)) ||
                pa_host::rows_overlap(ko, q) || pa_host::rows_overlap(ko, pos) || pa_host::rows_overlap(ko, freqs))))
    return PA_ERR_INVALID_ARG;

  RopeParams p;
  p.q = a->q;
  p.k = a->k;
  p.pos = a->positions;
  p.freqs = a->freqs;
  p.q_out = a->q_out;
  p.k_out = a->k_out;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.q_out_stride = a->q_out_stride;
  p.k_out_stride = a->k_out_stride;
  p.T = a->num_tokens;
  p.hq = a->num_q_heads;
  p.heads = a->num_q_heads + a->num_kv_heads;
  p.rot = a->rot_dim;
  p.scale = a->scale;
  p.sign = a->inverse ? -1.f : 1.f;
  const bool half = a->layout == PA_ROPE_HALF;
  // the widest accesses that every row's place allows
  int bytes = 16;
  for (const Rows &r : {q, qo, k, ko})
    if (r.p != nullptr && r.bytes > 0)
      while (!aligned(r.p, bytes) || r.stride % bytes != 0) bytes /= 2;
  // a CTA for every token while they would not fill the GPU otherwise (32 tokens: 1.6 us, 2.7 in fours; 16384: 38 us, 26 in fours)
  const bool few = n <= 2048;
  const bool in_place = a->q_out == a->q || (keys && a->k_out == a->k);
  const cudaError_t st = size == 2 ? launch<uint16_t>(p, half, bytes, few, in_place, stream) : launch<float>(p, half, bytes, few, in_place, stream);
  return st == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
