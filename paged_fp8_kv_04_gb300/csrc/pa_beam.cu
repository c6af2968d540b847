// pa_beam.cu -- beam search over the paged cache: pa_beam_select picks the beams that go on,
// pa_beam_reorder lets their block tables, last pages and states follow.  See include/pa.h for
// the contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kMaxBeams = 32;
constexpr int kMaxVocab = 1 << 24;
constexpr int kMaxReqs = 65535;

// --------------------------------------------------------------------------- selection

// The beams of one request are handled by a cluster of C CTAs: rows are dealt out, and a row is cut
// into parts where there are more CTAs than beams.  Each part is read once: a thread keeps the
// running maximum and sum of exponentials of its elements, and the vector its maximum came from.
//   lse = m + log sum exp(x - m),  total = score + (x - lse).
// Within a row the order of the totals is the order of the logits but for their rounding, so the W best of a
// part are found without its lse: of the best elements of every 16 (or 8) threads the W-th, tau, bounds them
// from below, and elements at or above tau lie with the few threads whose best does.  Only those threads'
// elements are looked at again (from L2), whatever the values: keys are (value, index) pairs,
// all different.  Every CTA leaves its list, maximum and sum in the shared memory of the
// cluster's first CTA, one cluster barrier follows, and a warp there joins parts and beams.
//
// Bound by HBM while the logits stream, then by the chain of joins.  Measured: 32 requests x 8 beams x
// 131072 bf16, 67 MB (9.9 us at a copy's rate), 21.9 us: 11 to 13 us of streaming (5.5 TB/s), 2 to tau, 2 to
// the part's list, 2 for the barrier, 2 in the first CTA, 2 of launch; 1 x 4 x 32001 fp32 8.8 us (0.2 of it the checks whether
// equal ranks are in order; where one fails the launch takes some 12 us more).  One CTA per
// request and one pass per candidate took 1644 and 152 us.  Lists sent as asynchronous stores that an mbarrier
// counts, in place of stores and a cluster barrier, cost 0.5 us more: some hundred 8-byte transactions.
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
  int32_t W, V, eos, parts;
  float penalty;
};

typedef unsigned long long u64;

// Keys that order (value, index) pairs: larger value first, then lower index; NaN is -inf.  The
// largest key is the best pair; no pair has key 0.
__device__ __forceinline__ u64 pair_key(float x, int v) {
  const float y = x != x ? -INFINITY : x + 0.f;  // -0 = +0
  const uint32_t u = __float_as_uint(y);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((u64)o << 32) | (0xFFFFFFFFu - (uint32_t)v);
}
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(u64 k) { return (int)(0xFFFFFFFFu - (uint32_t)(k & 0xFFFFFFFFull)); }
// Ordered bits of a double that is not NaN, -0 = +0; greater than 0 for every such double.  (These tests go by the bits: a
// comparison in fp64 takes as long as any of its operations.)
__device__ __forceinline__ u64 rank_key(double x) {
  const u64 u = (u64)__double_as_longlong(x);
  return u > (1ull << 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ bool is_finite(double x) { return (__double2hiint(x) & 0x7FF00000) != 0x7FF00000; }
__device__ __forceinline__ bool is_nan(double x) { return (__double2hiint(x) & 0x7FF80000) == 0x7FF80000; }  // a quiet one, as results are

// 32 keys, one per lane, in descending order over the lanes: bitonic networks on shuffles.
__device__ __forceinline__ u64 exchange(u64 k, int lane, int j, bool up) {
  const u64 y = __shfl_xor_sync(~0u, k, j);
  const bool larger = ((lane & j) == 0) == up;
  return larger ? (k > y ? k : y) : (k < y ? k : y);
}
__device__ __forceinline__ u64 sort32(u64 k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int j = n >> 1; j >= 1; j >>= 1) k = exchange(k, lane, j, (lane & n) == 0);
  return k;
}
// The 32 best of two descending lists, the other's given from its end.
__device__ __forceinline__ u64 merge32(u64 k, u64 other_reversed, int lane) {
  k = k > other_reversed ? k : other_reversed;
#pragma unroll
  for (int j = 16; j >= 1; j >>= 1) k = exchange(k, lane, j, true);
  return k;
}

// The 32 best of a descending list and 32 keys in any order.  (They take as many instructions as one inserted at its
// place.)
__device__ __forceinline__ u64 take32(u64 list, u64 k) {
  const int lane = threadIdx.x & 31;
  return merge32(list, __shfl_sync(~0u, sort32(k, lane), 31 - lane), lane);
}

constexpr int kBeamThreads = 512;
constexpr int kBeamWarps = kBeamThreads / 32;
// Vectors cut from two: 1 x 4 x 32001 8.8 us with 3 at a time, 9.3 with 4; 32 x 8 x 131071 fp32 33.7 with 3, 34.2
// with 4, 36.8 with 2 (30.9 where rows of other alignment were other vectors).
constexpr int kCutUnroll = 3;
constexpr int kUnroll = 4;  // 16-byte loads in flight per thread: 32 KB per CTA, two CTAs per SM

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int E = 8;
  static __device__ __forceinline__ float get(const uint4 &v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return (e & 1) ? pa::bf16hi(w) : pa::bf16lo(w);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // the largest element (NaN only if all are)
  static __device__ __forceinline__ float max(const uint4 &v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(pa::bf16lo(m), pa::bf16hi(m));
  }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ float get(const uint4 &v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float max(const uint4 &v) {
    return fmaxf(fmaxf(get(v, 0), get(v, 1)), fmaxf(get(v, 2), get(v, 3)));
  }
};

// A row seen as vectors of 16 bytes: vector j holds the elements E j .. E j + E - 1, of which the last may
// have fewer.  Also where the row does not begin on a 16-byte boundary: rows of the same values give the
// same sums in the same order, wherever they lie, so that equal totals are equal.  Such a vector
// is cut from the two it lies in (the second is in L1, it is the next thread's first).
template <typename T>
struct RowView {
  static constexpr int E = Vec<T>::E;
  const T *x;
  int V, nv;
  int mis;          // bytes that the row begins behind a boundary
  int begin, whole;  // vectors [begin, whole) lie, with what is fetched around them, within the row
  __device__ RowView(const T *row, int vocab) : x(row), V(vocab) {
    mis = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
    nv = (V + E - 1) / E;
    begin = mis != 0;
    whole = mis == 0 ? V / E : (V * (int)sizeof(T) + mis) / 16 - 1;
  }
  __device__ __forceinline__ int first(int j) const { return E * j; }
  __device__ __forceinline__ const uint4 *aligned() const {
    return reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(x) - mis);
  }
  // The 16 bytes from byte `mis` of a and b on.
  __device__ __forceinline__ uint4 cut(const uint4 &a, const uint4 &b) const {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (mis & 8)
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (mis & 4)
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (sizeof(T) == 2 && (mis & 2))
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 load(int j) const {
    if (j >= begin && j < whole) {
      const uint4 *at = aligned() + j;
      return mis == 0 ? __ldg(at) : cut(__ldg(at), __ldg(at + 1));
    }
    const int f = first(j);
    uint32_t w[4];  // a ragged end: what is missing is -inf
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 4) {
        w[i] = f + i < V ? ((const uint32_t *)x)[f + i] : 0xFF800000u;
      } else {
        const int a = f + 2 * i;
        const uint32_t lo = a < V ? ((const uint16_t *)x)[a] : 0xFF80u;
        const uint32_t hi = a + 1 < V ? ((const uint16_t *)x)[a + 1] : 0xFF80u;
        w[i] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxLists = kMaxBeams;  // rows * parts <= 32

constexpr int kMaxCands = 256;        // elements at or above tau that are put in order at once

struct BeamShared {
  u64 buf[kBeamWarps][32];
  u64 best[kBeamThreads / 8];       // the best element of every 16 or 8 threads
  u64 cand[kMaxCands];              // the part's elements at or above tau, in any order
  int owners, cands;
  long long wsum[kBeamWarps];
  // the first CTA's
  u64 list[kMaxLists][kMaxBeams];   // each (row, part)'s best, descending; then each row's
  long long sum[kMaxLists];         // sum of exp(x - m) in units of 2^-36, or -1: NaN
  float max[kMaxLists];
  double part[kMaxLists];           // that sum relative to the row's maximum
  double lse[kMaxBeams], inv[kMaxBeams];  // inv: max(new length, 1) ^ -length_penalty; then that power itself
  u64 rank[kMaxBeams][kMaxBeams];   // of each beam's candidates, descending; 0: none
  float total[kMaxBeams][kMaxBeams];
  int token[kMaxBeams][kMaxBeams];
  int used[kMaxBeams];              // of each beam: how many of its candidates are chosen,
  int open[kMaxBeams];              // and the first place from which their order may not be that of the logits
  bool unsure;                      // candidates of two lengths too close for the tables
};

// The few logarithms and powers of a step.  This GPU computes in fp64 slowly (some 70 cycles for each
// dependent operation; the general pow took 7 us here, and Taylor polynomials in fp64 2 to 3), so
// they are taken by tables with the small terms in fp32, after P. T. P. Tang's table-driven logarithm
// and exponential: within 1e-10, a hundredth of what the sums of exponentials carry.
constexpr double kLn2 = 0.69314718055994530942;
__constant__ float kInverse[16] = {  // 1 / (1 + (k + 1/2) / 16), to fp32
    0.969696999f, 0.914285719f, 0.864864886f, 0.820512831f, 0.780487776f, 0.744186044f, 0.711111128f, 0.680851042f,
    0.653061211f, 0.627451003f, 0.603773594f, 0.581818163f, 0.561403513f, 0.542372882f, 0.524590135f, 0.507936537f};
__constant__ double kMinusLnInverse[16] = {  // of those very numbers
    0.030771628864431744, 0.089612153101751704, 0.14518198563011125, 0.19782573029140393,
    0.24783620115748495,  0.2954642166191262,   0.34092656275620659, 0.38441173057530009,
    0.4260844157999969,   0.46608969453434201,  0.50455599585123423, 0.54159731409771239,
    0.57731535758424302,  0.61180153924334779,  0.64513801725294073, 0.67739876584980818};
__constant__ double kExp2Sixteenths[16] = {  // 2^(j / 16)
    1.0,                1.0442737824274138, 1.0905077326652577, 1.1387886347566916, 1.189207115002721,  1.241857812073484,
    1.2968395546510096, 1.3542555469368927, 1.4142135623730951, 1.4768261459394993, 1.5422108254079407, 1.6104903319492543,
    1.681792830507429,  1.7562521603732995, 1.8340080864093424, 1.9152065613971474};
// e^x: x = k ln 2 / 16 + t, |t| <= ln 2 / 32, e^t - 1 - t by Taylor; 0 below -700 and +inf above 700.
__device__ __forceinline__ double exp64(double x) {
  if (!(x > -700.0)) return 0.0;
  if (x > 700.0) return INFINITY;
  const int k = __float2int_rn((float)x * (16.f * kLog2e));
  const double t = fma(-(double)k, kLn2 / 16, x);
  const float u = (float)t;
  const float q = u * u * fmaf(fmaf(fmaf(1.f / 120, u, 1.f / 24), u, 1.f / 6), u, 0.5f);
  return (1.0 + (t + (double)q)) * (kExp2Sixteenths[k & 15] * __longlong_as_double((long long)((k >> 4) + 1023) << 52));
}
// ln s for a normal s > 0: s = 2^e m, 1 <= m < 2, i = the inverse of the middle of m's sixteenth, and
// ln m = -ln i + ln(1 + r), r = i m - 1 exactly in two fp32 numbers, |r| <= 1/31.  A row with one
// token to choose has a sum of 1, and its total is the score itself.
__device__ __forceinline__ double ln64(double s) {
  const long long b = __double_as_longlong(s);
  const int e = (int)((b >> 52) & 2047) - 1023, k = (int)((b >> 48) & 15);
  const double m = __longlong_as_double((b & 0xFFFFFFFFFFFFFll) | (1023ll << 52));
  const float hi = (float)m, lo = (float)(m - (double)hi), i = kInverse[k];
  const float p = hi * i, r1 = p - 1.f, r2 = fmaf(lo, i, fmaf(hi, i, -p)), r = r1 + r2;
  const float q = r * r * fmaf(fmaf(fmaf(fmaf(fmaf(1.f / 7, r, -1.f / 6), r, 1.f / 5), r, -1.f / 4), r, 1.f / 3), r, -0.5f);
  const double rest = (b & 0xFFFFFFFFFFFFFll) == 0 ? 0.0 : kMinusLnInverse[k] + ((double)r1 + (double)(r2 + q));
  return fma((double)e, kLn2, rest);
}

// len^penalty for ranks that the tables cannot tell apart: a length itself is exact (so that total / length is
// the nearest double), any other power CUDA's.
__device__ __noinline__ double length_power(int len, float penalty) {
  return penalty == 1.f ? (double)len : pow((double)len, (double)penalty);
}
// Ranks of different lengths this many steps of a double apart (2^-28 of their size or more) are
// in the right order however the tables' 1e-10 fell.
constexpr u64 kClearSteps = 1ull << 24;
// Ranks of one length within this many steps may be equal once divided by the power itself, or be so only by the tables.
constexpr u64 kSameSteps = 8;
constexpr double kSmallInverse = 1e-200;  // below this products may underflow

// This shared-memory address in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(const void *p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(pa::smem_u32(p)));
  return a;
}
__device__ __forceinline__ void store_cluster(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Joins the warps' descending lists (one key per lane); the result is in warp 0.
__device__ __forceinline__ u64 join_warps(u64 k, BeamShared &sm, int warp, int lane, int lists) {
  sm.buf[warp][lane] = k;
  for (int n = lists >> 1; n >= 1; n >>= 1) {
    __syncthreads();
    if (warp < n) {
      k = merge32(k, sm.buf[warp + n][31 - lane], lane);
      sm.buf[warp][lane] = k;
    }
  }
  return k;
}

// The W-th best of the best keys of every G threads (0: there are not as many), and the best one's value.
template <int G>
__device__ u64 lower_bound(u64 k, BeamShared &sm, int W, int tid, float &top) {
  constexpr int kGroups = kBeamThreads / G, Q = kGroups / 32;
  const int lane = tid & 31;
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) {
    const u64 y = __shfl_xor_sync(~0u, k, o);
    k = k > y ? k : y;
  }
  __syncthreads();  // an earlier part's readers are done
  if (tid % G == 0) sm.best[tid / G] = k;
  if (tid == 0) sm.owners = sm.cands = 0;
  __syncthreads();
  // (the keys differ but for 0, of which any will do: a key's place is the number of larger ones)
  u64 mine[Q], tau = 0;
  int place[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    mine[q] = sm.best[32 * q + lane];
    place[q] = 0;
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const u64 y = sm.best[i];
#pragma unroll
    for (int q = 0; q < Q; ++q) place[q] += y > mine[q];
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const unsigned at_w = __ballot_sync(~0u, place[q] == W - 1), first = __ballot_sync(~0u, place[q] == 0);
    if (at_w != 0) tau = __shfl_sync(~0u, mine[q], __ffs(at_w) - 1);
    if (first != 0) top = key_value(__shfl_sync(~0u, mine[q], __ffs(first) - 1));
  }
  return tau;
}

// One part of one row: its list, maximum and sum go to slot `slot` of the first CTA.
template <typename T>
__device__ void beam_part(const BeamParams &p, BeamShared &sm, int64_t row, int part, int slot, bool wait) {
  constexpr int E = Vec<T>::E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowView<T> r(static_cast<const T *>(p.logits) + row * p.stride, p.V);
  const int lo = (int)((int64_t)r.nv * part / p.parts), hi = (int)((int64_t)r.nv * (part + 1) / p.parts);

  // ---- one pass: maximum, sum of 2^((x - m) log2 e), and the vector of the maximum
  float m = -INFINITY;
  int best = lo + tid;
  uint4 bv = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  pa::f32x2 sum = pa::pack2(0.f, 0.f), minus_m = sum;
  const pa::f32x2 log2e = pa::pack2(kLog2e, kLog2e);
  auto take = [&](const uint4 &v, int j) {
    const float mx = Vec<T>::max(v);
    if (mx > m) {
      const float f = pa::fast_exp2((m - mx) * kLog2e);
      sum = pa::mul2(sum, pa::pack2(f, f));
      minus_m = pa::pack2(-mx, -mx);
      m = mx;
      bv = v;
      best = j;
    }
    // the difference first: exact near the maximum, and in range at the types' lowest values
    // (while m is still -inf, -inf - 0 gives 0)
    pa::f32x2 t[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      float a, b;
      pa::unpack2(pa::mul2(pa::add2(pa::pack2(Vec<T>::get(v, 2 * e), Vec<T>::get(v, 2 * e + 1)), minus_m), log2e), a, b);
      t[e] = pa::pack2(pa::fast_exp2(a), pa::fast_exp2(b));
    }
#pragma unroll
    for (int n = E / 4; n >= 1; n >>= 1)
#pragma unroll
      for (int e = 0; e < n; ++e) t[e] = pa::add2(t[e], t[e + n]);
    sum = pa::add2(sum, t[0]);
  };
  int j = lo + tid;
  if (j < r.begin && j < hi) {  // what is fetched for the first vector begins before the row
    take(r.load(j), j);
    j += kBeamThreads;
  }
  const int whole = min(hi, r.whole);
  if (r.mis == 0) {
    for (; j + (kUnroll - 1) * kBeamThreads < whole; j += kUnroll * kBeamThreads) {
      const uint4 *src = r.aligned() + j;
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u] = __ldg(src + u * kBeamThreads);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) take(v[u], j + u * kBeamThreads);
    }
  } else {
    for (; j + (kCutUnroll - 1) * kBeamThreads < whole; j += kCutUnroll * kBeamThreads) {
      const uint4 *src = r.aligned() + j;
      uint4 v[kCutUnroll], w[kCutUnroll];
#pragma unroll
      for (int u = 0; u < kCutUnroll; ++u) {
        v[u] = __ldg(src + u * kBeamThreads);
        w[u] = __ldg(src + u * kBeamThreads + 1);
      }
#pragma unroll
      for (int u = 0; u < kCutUnroll; ++u) take(r.cut(v[u], w[u]), j + u * kBeamThreads);
    }
  }
  for (; j < hi; j += kBeamThreads) take(r.load(j), j);
  float s, s1;
  pa::unpack2(sum, s, s1);
  s += s1;
  const bool nan = s != s;  // a NaN or +inf among the elements
  u64 key = 0;
  if (lo + tid < hi) {
    int at = r.first(lo + tid);  // nothing above -inf: the first element
    if (m > -INFINITY) {
      at = r.first(best);
      bool found = false;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!found) {
          if (Vec<T>::get(bv, e) == m) found = true;
          else ++at;
        }
    }
    key = pair_key(m, at);
  }

  // ---- tau: the W-th of the best elements of every 16 threads, so at least W elements reach it.  With more
  // beams of every 8: the fewer groups there are to spare, the lower tau lies and the more elements reach it
  // (1 x 32 x 131072: 31.6 us with 8 against 60.3 with 16; 1 x 4 x 32001: 9.8 against 8.8)
  float top;
  const u64 tau = p.W <= 16 ? lower_bound<16>(key, sm, p.W, tid, top) : lower_bound<8>(key, sm, p.W, tid, top);
  // the threads whose best reaches it
  u64 *owners = &sm.buf[0][0];
  if (key >= tau && key != 0) owners[atomicAdd(&sm.owners, 1)] = key;
  // the part's sum: every thread's relative to the part's maximum, in fixed point (2^-36), so that
  // joining 512 of them loses nothing
  const float scaled = m == -INFINITY ? 0.f : s * pa::fast_exp2((m - top) * kLog2e);
  long long fixed = nan ? 0 : __float2ll_rn(scaled * 68719476736.f);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) fixed += __shfl_xor_sync(~0u, fixed, o);
  const bool wnan = __any_sync(~0u, nan);
  if (lane == 0) sm.wsum[warp] = wnan ? -1 : fixed;

  __syncthreads();

  // ---- the elements at or above tau, all of them with those threads: a warp looks through the vectors
  // of one, a lane per vector
  const int nowners = sm.owners;
  auto search = [&](auto &&found) {
    for (int i = warp; i < nowners; i += kBeamWarps) {
      const int oj = key_index(owners[i]) / E;
      for (int j0 = lo + (oj - lo) % kBeamThreads; j0 < hi; j0 += 32 * kBeamThreads) {
        const int64_t jl = (int64_t)j0 + (int64_t)lane * kBeamThreads;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        unsigned left = 0;  // this lane's elements at or above tau
        if (jl < hi) {
          v = r.load((int)jl);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = r.first((int)jl) + e;
            if (at < p.V && pair_key(Vec<T>::get(v, e), at) >= tau) left |= 1u << e;
          }
        }
        found(v, (int)jl, left);
      }
    }
  };
  auto element = [&](const uint4 &v, int jl, unsigned left) {  // the key of the first of `left`
    const int e = __ffs(left) - 1;
    float x = 0.f;
#pragma unroll
    for (int q = 0; q < E; ++q)
      if (q == e) x = Vec<T>::get(v, q);
    return pair_key(x, r.first(jl) + e);
  };
  search([&](const uint4 &v, int jl, unsigned left) {
    if (left == 0) return;
    for (int at = atomicAdd(&sm.cands, __popc(left)); left != 0 && at < kMaxCands; ++at, left &= left - 1) sm.cand[at] = element(v, jl, left);
  });
  if (wait) pa::cluster_wait();  // the first CTA runs: its shared memory can be written
  __syncthreads();
  // As a rule there are not many more than W: each is put in its place by counting the larger ones (joining
  // the warps' lists in every case cost 2 us more: 25.6 against 23.5).
  const int cands = sm.cands;
  if (cands <= kMaxCands) {
    if (tid < cands) {
      const u64 c = sm.cand[tid];
      int to = 0;
      for (int i = 0; i < cands; ++i) to += sm.cand[i] > c;
      if (to < kMaxBeams) store_cluster(in_first_cta(&sm.list[slot][to]), c);
    }
    if (tid >= cands && tid < kMaxBeams) store_cluster(in_first_cta(&sm.list[slot][tid]), (u64)0);
  } else {
    // many (long runs of equal or rising values): each warp keeps the best 32 of a share of the vectors in order, then they
    // are joined (64 x 32 x 1000 bf16: 187 us; 415 with elements counted and inserted one by one)
    u64 mine = 0, least = 0;
    const int first = lo + 32 * warp + lane;
    auto vector = [&](int j) { return j < hi ? r.load(j) : make_uint4(0u, 0u, 0u, 0u); };
    uint4 v = vector(first), next = vector(first + kBeamThreads);
    for (int jl = first; jl - lane < hi; jl += kBeamThreads) {
      const uint4 later = vector(jl + 2 * kBeamThreads);
      const u64 most = pair_key(Vec<T>::max(v), r.first(jl));
      if (__any_sync(~0u, jl < hi && most >= tau && most > least)) {
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          const int at = r.first(jl) + e;
          u64 k = jl < hi && at < p.V ? pair_key(Vec<T>::get(v, e), at) : 0ull;
          if (k < tau) k = 0;
          if (__any_sync(~0u, k > least)) {
            mine = take32(mine, k);
            least = __shfl_sync(~0u, mine, 31);
          }
        }
      }
      v = next;
      next = later;
    }
    __syncthreads();  // the owners have been read
    const u64 k = join_warps(mine, sm, warp, lane, kBeamWarps);
    if (warp == 0) store_cluster(in_first_cta(&sm.list[slot][lane]), k);
  }
  if (warp == 0) {
    long long t = lane < kBeamWarps ? sm.wsum[lane] : 0;
    const bool bad = __any_sync(~0u, t < 0);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
    if (lane == 0) {
      store_cluster(in_first_cta(&sm.max[slot]), top);
      store_cluster(in_first_cta(&sm.sum[slot]), (u64)(bad ? -1 : t));
    }
  }
}

// A total's rank: by the tables' inverse power, or with that power itself.
__device__ __forceinline__ double rank_of(const BeamParams &p, double total, double inv, bool careful) {
  if (p.penalty == 0.f || !is_finite(total)) return total;
  return careful ? total / inv : total * inv;
}
__device__ __forceinline__ double total_of(float c, float x, double lse) {
  const double t = (double)c + ((double)x - lse);
  return is_nan(t) ? -INFINITY : t;
}

// No continuation at a number: every candidate of beam b counts as -inf.
__device__ __forceinline__ bool is_dead(const BeamShared &sm, int b, float c, bool ended) {
  return c != c || c == -INFINITY || (!ended && !is_finite(sm.lse[b]));
}

// Every (beam, place) candidate's token, total and rank: a warp per beam, a lane per place.  Lane b has what beam
// b brings.
template <bool CAREFUL>
__device__ __forceinline__ void candidates(const BeamParams &p, BeamShared &sm, float cum, bool done) {
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < p.W; b += kBeamWarps) {
    const float c = __shfl_sync(~0u, cum, b);
    const bool ended = __shfl_sync(~0u, (int)done, b) != 0, dead = is_dead(sm, b, c, ended);
    int tok = lane, to = lane;
    double total = -INFINITY;
    if (!dead && ended) {
      tok = lane == 0 ? p.eos : (lane <= p.eos ? lane - 1 : lane);
      if (lane == 0) total = (double)c;
    } else if (!dead) {
      const u64 k = sm.list[b * p.parts][lane];
      tok = key_index(k);
      total = total_of(c, key_value(k), sm.lse[b]);
    }
    const u64 key = lane < p.W && lane < p.V ? rank_key(rank_of(p, total, sm.inv[b], CAREFUL)) : 0ull;
    if (CAREFUL) {
      to = 0;
      for (int j = 0; j < 32; ++j) {
        const u64 y = __shfl_sync(~0u, key, j);
        const int t = __shfl_sync(~0u, tok, j);
        to += y > key || (y == key && (t < tok || (t == tok && j < lane)));
      }
    }
    sm.rank[b][to] = key;
    sm.total[b][to] = (float)total;
    sm.token[b][to] = tok;
  }
}

// The num_beams best of all beams' candidates, by one warp: lane j has the j-th best's beam, place and rank, and
// lane b the rank of the first candidate of beam b that is left (0: none).
struct Choice {
  int from, place;
  u64 rank, left;
};
__device__ __forceinline__ Choice choose(const BeamParams &p, BeamShared &sm) {
  const int lane = threadIdx.x & 31;
  Choice x = {0, 0, 0ull, lane < p.W ? sm.rank[lane][0] : 0ull};
  int at = 0;
  for (int j = 0; j < p.W; ++j) {
    const uint32_t hi = (uint32_t)(x.left >> 32), top = __reduce_max_sync(~0u, hi);
    const uint32_t lo = hi == top ? (uint32_t)x.left : 0u, low = __reduce_max_sync(~0u, lo);
    const int win = __ffs(__ballot_sync(~0u, hi == top && lo == low && x.left != 0)) - 1;  // equal ranks: the lower beam
    const int p_win = __shfl_sync(~0u, at, max(win, 0));
    if (lane == j) {
      x.from = max(win, 0);
      x.place = p_win;
      x.rank = ((u64)top << 32) | low;
    }
    if (lane == win) {
      ++at;
      x.left = at < p.W ? sm.rank[lane][at] : 0ull;
    }
  }
  sm.used[lane] = at;
  return x;
}
// And what the caller gets of it; returns the length that lane j's has.
__device__ __forceinline__ int write_choice(const BeamParams &p, const BeamShared &sm, const Choice &x, int64_t me, bool done, int len) {
  const bool from_done = __shfl_sync(~0u, (int)done, x.from) != 0;
  const int from_len = __shfl_sync(~0u, len, x.from);
  if ((threadIdx.x & 31) < p.W) {
    const int tok = sm.token[x.from][x.place];
    p.tokens[me] = tok;
    p.parents[me] = x.from;
    p.scores_out[me] = sm.total[x.from][x.place];
    if (p.finished_out != nullptr) p.finished_out[me] = from_done || (p.eos >= 0 && tok == p.eos);
    if (p.lengths_out != nullptr) p.lengths_out[me] = from_len;
  }
  return from_len;
}

// The order of totals is that of the logits unless their rounding makes one of several logits, as with scores
// of -1e9 for beams that hardly exist: then the lower token comes first, which may not even be in the list.
// The first place of beam b's list from which that can be so (32: nowhere), for a warp.
template <typename T>
__device__ int open_from(const BeamParams &p, const BeamShared &sm, int b, float c) {
  const int lane = threadIdx.x & 31, n = min(p.W, p.V), i = min(lane + 1, 31);
  const u64 k = sm.list[b * p.parts][lane], next = sm.list[b * p.parts][i];
  bool near = lane + 1 < n && sm.rank[b][lane] - sm.rank[b][i] <= kSameSteps, differ = near && k >> 32 != next >> 32;
  if (lane == n - 1 && n < p.V) {
    // beyond the list: is the step from its last logit x to the next lower value (2^-24 or 2^-8 of x or more) within
    // 16 steps of a total (2^-50 of the largest of its terms or less)?
    auto exponent = [](float y) { return max((int)(__float_as_uint(y) >> 23 & 255u), 1); };
    const float x = key_value(k);
    const int largest = max(exponent(c), max(exponent((float)sm.lse[b]), exponent(x)));
    near = differ = x > -INFINITY && (c == INFINITY || exponent(x) + (sizeof(T) == 2 ? 16 : 0) + 22 <= largest);
  }
  const unsigned same = __ballot_sync(~0u, near), other = __ballot_sync(~0u, differ);
  if (other == 0) return 32;
  const unsigned apart = ~same & ((1u << (__ffs(other) - 1)) - 1u);  // equal ranks may begin before logits differ
  return 32 - __clz(apart);
}

// The candidates chosen from beam b's list at its lowest rank: of all the row's tokens with that rank they have to
// be the lowest.  The tokens' logits are an interval, whose lower end is found by bisection; each warp looks for the first
// in a stretch of the row, and their tokens and totals take the place of those in the list.  For the whole CTA.
template <typename T>
__device__ __noinline__ void lowest_tokens(const BeamParams &p, BeamShared &sm, int64_t row, int b, float c) {
  constexpr int E = Vec<T>::E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const u64 rank = sm.rank[b][p.W - 1];
  const int higher = __popc(__ballot_sync(~0u, sm.rank[b][lane] > rank)), need = sm.used[b] - higher;
  if (need <= 0 || rank == rank_key(-INFINITY)) return;
  const double lse = sm.lse[b], inv = sm.inv[b];
  const uint32_t last = (uint32_t)(sm.list[b * p.parts][p.W - 1] >> 32), top = (uint32_t)(sm.list[b * p.parts][higher] >> 32);
  uint32_t lo = (uint32_t)(pair_key(-INFINITY, 0) >> 32), hi = last;  // the lowest logit of this rank is one of [lo, hi]
  while (lo < hi) {
    const uint32_t step = (hi - lo + 31) / 32, at = min(lo + lane * step, hi);
    const double r = rank_of(p, total_of(c, key_value((u64)at << 32), lse), inv, true);
    const unsigned has = __ballot_sync(~0u, rank_key(r) == rank);
    if (has & 1u) {
      hi = lo;
    } else if (has != 0) {
      const uint32_t from = lo;
      lo = from + (__ffs(has) - 2) * step + 1;
      hi = min(from + (__ffs(has) - 1) * step, hi);
    } else {
      lo += 31 * step + 1;
    }
  }
  if (lo == top) return;  // one logit only, whose lowest tokens the list has
  const T *x = static_cast<const T *>(p.logits) + row * p.stride;
  const RowView<T> r(x, p.V);
  const int begin = (int)((int64_t)r.nv * warp / kBeamWarps), end = (int)((int64_t)r.nv * (warp + 1) / kBeamWarps);
  int got = 0;
  for (int j0 = begin; j0 < end && got < need; j0 += 32 * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + 32 * u + lane;
      v[u] = j < end ? r.load(j) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + 32 * u + lane;
      unsigned left = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t o = (uint32_t)(pair_key(Vec<T>::get(v[u], e), 0) >> 32);
        if (j < end && r.first(j) + e < p.V && o >= lo && o <= top) left |= 1u << e;
      }
      unsigned have;
      while (got < need && (have = __ballot_sync(~0u, left != 0)) != 0) {
        if (lane == __ffs(have) - 1) {
          sm.buf[warp][got] = (u64)(r.first(j) + __ffs(left) - 1);
          left &= left - 1;
        }
        ++got;
      }
    }
  }
  if (lane == 0) sm.wsum[warp] = got;
  __syncthreads();
  if (warp == 0 && lane < need) {
    int from = 0, k = lane;
    while (from < kBeamWarps && k >= (int)sm.wsum[from]) k -= (int)sm.wsum[from++];
    if (from < kBeamWarps) {
      const int token = (int)sm.buf[from][k];
      float y;
      if constexpr (sizeof(T) == 4)
        y = x[token];
      else
        y = __uint_as_float((uint32_t)x[token] << 16);
      sm.token[b][higher + lane] = token;
      sm.total[b][higher + lane] = (float)total_of(c, y, lse);
    }
  }
  __syncthreads();
}

// The choice where the first one is not certain to be right.  For the whole CTA.
template <typename T>
__device__ __noinline__ void choose_again(const BeamParams &p, BeamShared &sm, int64_t base, float cum, bool done, int len) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // what led here has been read
  if (warp == 0 && p.penalty != 0.f) sm.inv[lane] = length_power(max(len, 1), p.penalty);
  __syncthreads();
  candidates<true>(p, sm, cum, done);
  __syncthreads();
  Choice x = {};
  if (warp == 0) x = choose(p, sm);
  __syncthreads();
  for (int b = 0; b < p.W && p.V > p.W; ++b) {
    const float c = __shfl_sync(~0u, cum, b);
    const bool ended = __shfl_sync(~0u, (int)done, b) != 0;
    if (!ended && !is_dead(sm, b, c, ended)) lowest_tokens<T>(p, sm, base + b, b, c);
  }
  if (warp == 0) write_choice(p, sm, x, base + lane, done, len);
}

template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 2) beam_select_kernel(const __grid_constant__ BeamParams p) {
  __shared__ BeamShared sm;
  pa::pdl_wait();
  pa::cluster_arrive();
  const uint32_t C = pa::cluster_ctas(), rank = pa::cluster_rank();
  const int n = blockIdx.x / C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t base = (int64_t)n * p.W, me = base + lane;
  const bool mine = lane < p.W;
  // lane b: what beam b brings (read by all, used by the first CTA; the loads run ahead of the rows')
  const float cum = mine ? p.scores[me] : -INFINITY;
  const bool done = mine && p.finished != nullptr && p.finished[me] != 0;
  int len = mine && p.lengths != nullptr ? p.lengths[me] : 0;
  if (!done && len < INT_MAX) ++len;
  const int units = p.W * p.parts;
  bool waited = false;
  for (int u = rank; u < units; u += C) {
    beam_part<T>(p, sm, base + u / p.parts, u % p.parts, u, !waited);
    waited = true;
  }
  if (!waited) pa::cluster_wait();
  pa::cluster_arrive();
  if (rank != 0) return;
  // lane b of the last warp, while the others' lists arrive: the power of beam b's length
  if (warp == kBeamWarps - 1) sm.inv[lane] = p.penalty == 0.f ? 1.0 : exp64(-(double)p.penalty * ln64((double)max(len, 1)));
  pa::cluster_wait();

  // ---- the first CTA.  Lane u < units of warp 0: its part's sum relative to the row's maximum; then
  // lane b: beam b's lse.  The other warps join the rows' lists meanwhile.
  if (warp == 0) {
    if (lane < units) {
      const int s0 = lane / p.parts * p.parts;
      float M = sm.max[s0];
      for (int q = 1; q < p.parts; ++q) M = fmaxf(M, sm.max[s0 + q]);
      const long long t = sm.sum[lane];
      const double x = (double)t * (1.0 / 68719476736.0);
      sm.part[lane] = t < 0 ? (double)NAN : sm.max[lane] == M ? x : x * exp64((double)sm.max[lane] - (double)M);
    }
    __syncwarp();
    if (mine) {
      double sum = 0.0;
      float M = -INFINITY;
      for (int q = 0; q < p.parts; ++q) {
        sum += sm.part[lane * p.parts + q];
        M = fmaxf(M, sm.max[lane * p.parts + q]);
      }
      // a sum that is NaN or 0 (nothing above -inf) has no logarithm
      sm.lse[lane] = sum > 0.0 ? (double)M + ln64(sum) : (double)NAN;
    }
  } else if (p.parts > 1) {
    for (int b = warp - 1; b < p.W; b += kBeamWarps - 1) {
      u64 k = sm.list[b * p.parts][lane];
      for (int q = 1; q < p.parts; ++q) k = merge32(k, sm.list[b * p.parts + q][31 - lane], lane);
      sm.list[b * p.parts][lane] = k;
    }
  }
  __syncthreads();
  // The candidates are taken in the order of the logits, and ranked by total * length^-penalty from the tables.  Where
  // that leaves the order of the chosen open -- different logits of a beam with all but the same total, beams of different
  // lengths with ranks closer than the tables' error, so that of equal ranks not the lower token or beam might come
  // first -- it is done again, with total / length^penalty and the tokens of equal ranks in order.
  candidates<false>(p, sm, cum, done);
  __syncthreads();
  if (warp == 0) {
    const Choice x = choose(p, sm);
    const int from_len = write_choice(p, sm, x, me, done, len);
    // The chosen are in the order of their computed ranks, so two of different lengths have neighbours of different
    // lengths between them; what is left of a beam comes after its next candidate, which each lane compares with
    // the last of the chosen.  Two beams of one length are in the order of their totals, unless quotients round together
    // what the products do not, or the other way round.
    bool unsure = false;
    if (p.penalty != 0.f) {
      const u64 lowest = rank_key(-INFINITY);
      auto close = [&](int b, int n, u64 r, int b2, int n2, u64 r2) {  // r >= r2
        return b != b2 && r > lowest && r - r2 <= (n != n2 ? kClearSteps : kSameSteps);
      };
      const u64 next = __shfl_down_sync(~0u, x.rank, 1), last = __shfl_sync(~0u, x.rank, p.W - 1);
      const int next_from = __shfl_down_sync(~0u, x.from, 1), last_from = __shfl_sync(~0u, x.from, p.W - 1);
      const int next_len = __shfl_down_sync(~0u, from_len, 1), last_len = __shfl_sync(~0u, from_len, p.W - 1);
      unsure = mine && (sm.inv[lane] < kSmallInverse ||
                        (lane + 1 < p.W && close(x.from, from_len, x.rank, next_from, next_len, next)) ||
                        (x.left != 0 && close(last_from, last_len, last, lane, len, x.left)));
    }
    unsure = __any_sync(~0u, unsure);
    if (lane == 0) sm.unsure = unsure;
  } else {
    for (int b = warp - 1; b < p.W; b += kBeamWarps - 1) {
      const float c = __shfl_sync(~0u, cum, b);
      const bool ended = __shfl_sync(~0u, (int)done, b) != 0;
      const int open = ended || is_dead(sm, b, c, ended) ? 32 : open_from<T>(p, sm, b, c);
      if (lane == 0) sm.open[b] = open;
    }
  }
  __syncthreads();
  if (sm.unsure || __any_sync(~0u, mine && sm.used[lane] > sm.open[lane])) choose_again<T>(p, sm, base, cum, done, len);
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
// page, its share of the states.  Every CTA works the request's parents out by itself, a lane per beam,
// so that nothing has to be exchanged.  Copies only, bound by latency at the sizes of a step: 32 x 8 beams
// with 32 KB of mass each (20 MB, 2.9 us at a copy's rate) take 6.2 us, a request of four beams 2.6 us.
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const ReorderParams p) {
  pa::pdl_wait();
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

constexpr int kMaxCluster = 16;  // more than 8 needs the kernel's opt-in

// The current device's SM count, and its kernels' opt-in to clusters of 16, once per device; 0 for
// a device beyond those tracked, -1 when a call fails.
int beam_device() {
  static std::once_flag once[pa_host::kMaxDevices];
  static int sms[pa_host::kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev < 0 || dev >= pa_host::kMaxDevices) return 0;
  std::call_once(once[dev], [dev]() {
    int n = 0;
    const bool ok =
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
        cudaFuncSetAttribute(beam_select_kernel<float>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaFuncSetAttribute(beam_select_kernel<uint16_t>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    sms[dev] = ok ? n : -1;
  });
  return sms[dev];
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
  {
    using pa_host::Span;
    const bool f32 = a->logits_dtype == PA_LOGITS_F32;
    const uint64_t beams = (uint64_t)a->num_reqs * a->num_beams, stride = std::min<int64_t>(a->logits_stride, 1ll << 36);
    const Span logits = {a->logits, beams == 0 ? 0 : ((beams - 1) * stride + a->vocab) * (f32 ? 4 : 2)};
    const Span scores = {a->scores, 4 * beams}, finished = {a->finished, beams}, lengths = {a->lengths, 4 * beams};
    const Span tokens = {a->tokens, 4 * beams}, parents = {a->parents, 4 * beams}, scores_out = {a->scores_out, 4 * beams};
    const Span finished_out = {a->finished_out, beams}, lengths_out = {a->lengths_out, 4 * beams};
    // an output in place of its input is that input; a part of it is another request's
    auto unless = [](const Span &in, const Span &out) { return Span{in.p == out.p ? nullptr : in.p, in.n}; };
    if (pa_host::overlaps(tokens, {logits, scores, finished, lengths, parents, scores_out, finished_out, lengths_out}) ||
        pa_host::overlaps(parents, {logits, scores, finished, lengths, scores_out, finished_out, lengths_out}) ||
        pa_host::overlaps(scores_out, {logits, unless(scores, scores_out), finished, lengths, finished_out, lengths_out}) ||
        pa_host::overlaps(finished_out, {logits, scores, unless(finished, finished_out), lengths, lengths_out}) ||
        pa_host::overlaps(lengths_out, {logits, scores, finished, unless(lengths, lengths_out)}))
      return PA_ERR_INVALID_ARG;
  }
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
  p.eos = a->eos_token;
  p.penalty = a->length_penalty;
  const bool f32 = a->logits_dtype == PA_LOGITS_F32;
  const int sms = beam_device();
  if (sms < 1) return sms == 0 ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
  // CTAs per request: as many as keep one wave (two CTAs per SM) and have a beam or 16 KB of logits each.
  // 32 x 8 x 131072: 21.9 us with 8, 33.4 with 16, 28.7 with 4; 1 x 4 x 32001 fp32: 8.8 us with 16, 24.2 with
  // 1; 1 x 8 x 1000: 9.3 us with 8, 33.1 with 1; 64 x 4 x 32000: 10.9 with 4, 18.9 with 8.
  const int64_t bytes = (int64_t)a->num_beams * a->vocab * (f32 ? 4 : 2);
  int C = 1;
  while (C < kMaxCluster && (int64_t)a->num_reqs * C <= sms &&
         (C < a->num_beams || bytes / (2 * C) >= 16384))
    C *= 2;
  p.parts = C > a->num_beams ? C / a->num_beams : 1;
  const pa_host::Launch run(dim3((unsigned)a->num_reqs * C), dim3(kBeamThreads), 0, stream, C);
  const cudaError_t e = f32 ? cudaLaunchKernelEx(run.cfg(), beam_select_kernel<float>, p)
                            : cudaLaunchKernelEx(run.cfg(), beam_select_kernel<uint16_t>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
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
  const pa_host::Span parents = {a->parents, 4 * rows}, lens = {a->context_lens, 4 * rows}, table_out = {a->block_table_out, tbytes};
  if (pa_host::overlaps(table_out, {{a->block_table, tbytes}, parents, lens})) return PA_ERR_INVALID_ARG;
  int64_t widest = 0;
  for (int k = 0; k < a->num_states; ++k) {
    if (a->state_in[k] == nullptr || a->state_out[k] == nullptr || a->state_bytes[k] < 1 ||
        a->state_bytes[k] > (INT64_MAX >> 17))
      return PA_ERR_INVALID_ARG;
    const uint64_t n = rows * (uint64_t)a->state_bytes[k];
    if (pa_host::overlaps({a->state_out[k], n}, {{a->block_table, tbytes}, table_out, parents, lens}) ||
        pa_host::overlaps(table_out, {{a->state_in[k], n}}))
      return PA_ERR_INVALID_ARG;
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
  const pa_host::Launch run(dim3((unsigned)gx, a->num_reqs * a->num_beams), dim3(kReorderThreads), 0, stream);
  return cudaLaunchKernelEx(run.cfg(), beam_reorder_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
