// pa_mass.cu -- attention mass: pa_attn_mass adds one decode step's attention weights to the
// mass of the cached tokens.  See include/pa.h for the contract.
//
//   w[p] = sum over rows t, heads g of exp(sm_scale q[t][g] . k[p] k_scale[p] - lse[t][g])
//
// The K cache is read once per four query rows.  With the log-sum-exp known beforehand there is no
// running maximum, no second product and nothing to join: a 128-token tile of one (request, KV
// head) is
//   S[tok][n] = K[tok][:] . Q[n][:]   tcgen05.mma, M = 128 tokens, A = the tile as TMA left it
//                                     (K-major, 128-byte swizzle): kind::f8f6f4 on the cache's e4m3
//                                     bytes, kind::f16 on a bf16 cache
//   mass[tok] += sum_n 2^(S c - lse)  TMEM lane = token: a thread sums its token's columns in
//                                     registers, and the mass is read and written once, coalesced.
// For e4m3 keys a query row of 128 bf16 values is an e4m3 pair hi + lo / 32 at its own power of
// two, in two columns of N: exact for elements within 2^-14 of the row's largest, and within
// 2^-22 of that for smaller ones.  So N = 32 columns per query row (16 heads), or 16 for bf16.
//
// Warp roles (576 threads, one CTA per SM, each with an equal share of the tiles): warps 0-15 are four
// epilogue groups that take every fourth tile and convert the queries of the segment to come
// ((request, KV head, up to four rows) of the CTA's share); warp 16 gathers pages by TMA into a ring of
// stages; warp 17 issues the MMAs, up to two tiles ahead of each group.  Every wait is bounded.
//
// Bound by HBM: 132 B of keys and 8 B of mass per token against 4096 flop per query row.  Measured
// (GB300): 8 requests x 131072 tokens, 143 MB, 27.2 us (5.2 TB/s); from twice that size the steady
// rate is 6.66 TB/s, 0.98 of the 6.78 a copy measures, and some 6.6 us are launch, schedule, the
// first tile's way through the roles and the last one's.  What it took: one thread per token on
// fp32 arithmetic 173 us; this kernel with two epilogue groups and the MMAs issued by "lane 0"
// 37 us; issued by an elected lane 30 us (without that the issue alone took 270 cycles per MMA);
// launched ahead of the kernel before it 29 us; ring positions kept by counters, not by
// divisions, 27 us.  Keys marked to leave L2 first: without that 29.2 us.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kG = 16;            // query heads per KV head
constexpr int kD = pa_host::kD;
constexpr int kTile = 128;        // tokens per tile
constexpr int kMaxSeqs = 4096;
constexpr int kMaxQ = 64;
constexpr int kMaxPositions = 1 << 30;
// Query rows per pass over the keys.  A row costs no further key bytes within a pass: 16 x 65536 tokens take
// 28.1 us with one row and 31.6 us with four; eight rows would fill TMEM with one buffer for two groups.
constexpr int kRows = 4;
constexpr int kGroups = 4;        // epilogue groups of four warps
constexpr int kEpiWarps = 4 * kGroups;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kMaxStages = 12;
constexpr float kLog2e = 1.4426950408889634f;

struct MassParams {
  CUtensorMap tm_k;
  const uint16_t *q;
  const float *ks;
  const int32_t *bt, *L, *cu;
  const float *lse, *mass;
  float *out;
  uint32_t *status;
  int64_t num_pages;
  int32_t B, R, Hkv, ps, ps_shift, ppt, bt_stride, mass_stride, maxq;
  int32_t nstage, stage_bytes, qbuf_bytes;
  int32_t nbuf, buf_cols, tmem_cols;  // TMEM: nbuf buffers of buf_cols columns for each group
  float kfold, decay;  // kfold = sm_scale * log2 e (* k_scale_scalar)
};

// Shared memory: stages | 2 query operands | factors | barriers | requests (tile prefix, L, row0, q_len)
constexpr int kFactorBytes = 2 * kRows * 2 * kG * 4;  // per buffer and row: factor[16], -lse2[16]
constexpr int kSBars = 2 * kGroups;  // two buffers per group at most
constexpr int kNumBars = 2 * kMaxStages + 2 * kSBars + 2 + 2 + 2;
constexpr int kCtrlBytes = kFactorBytes + kNumBars * 8 + kMaxStages * 4 + 16 + (kThreads / 32) * 4 + 64;

struct MassSmem {
  uint8_t *base;
  uint32_t stages, q, factors, bars;
  uint32_t *valid;   // per stage: which of the tile's pages are loaded
  uint32_t *misc;    // [0] TMEM address, [1] abort
  int32_t *wsum;     // per-warp sums of the scan
  int32_t *tstart;   // [B + 1] tiles of the requests before, for one KV head
  int32_t *info;     // [B][3]: context length, first row, rows
};

__device__ __forceinline__ MassSmem carve(uint8_t *raw, const MassParams &p) {
  MassSmem s;
  s.base = raw;
  uint8_t *c = raw + (size_t)p.nstage * p.stage_bytes + 2 * (size_t)p.qbuf_bytes;
  s.stages = pa::smem_u32(raw);
  s.q = s.stages + p.nstage * p.stage_bytes;
  s.factors = pa::smem_u32(c);
  s.bars = s.factors + kFactorBytes;
  s.valid = reinterpret_cast<uint32_t *>(c + kFactorBytes + kNumBars * 8);
  s.misc = s.valid + kMaxStages;
  s.wsum = reinterpret_cast<int32_t *>(s.misc + 4);
  s.tstart = reinterpret_cast<int32_t *>(c + kCtrlBytes);
  s.info = s.tstart + p.B + 1;
  return s;
}

__device__ __forceinline__ uint32_t bar_full(const MassSmem &s, int i) { return s.bars + 8 * i; }
__device__ __forceinline__ uint32_t bar_empty(const MassSmem &s, int i) { return s.bars + 8 * (kMaxStages + i); }
__device__ __forceinline__ uint32_t bar_sfull(const MassSmem &s, int i) { return s.bars + 8 * (2 * kMaxStages + i); }
__device__ __forceinline__ uint32_t bar_sfree(const MassSmem &s, int i) { return s.bars + 8 * (2 * kMaxStages + kSBars + i); }
__device__ __forceinline__ uint32_t bar_qready(const MassSmem &s, int i) { return s.bars + 8 * (2 * kMaxStages + 2 * kSBars + i); }
__device__ __forceinline__ uint32_t bar_qfree(const MassSmem &s, int i) { return s.bars + 8 * (2 * kMaxStages + 2 * kSBars + 2 + i); }
__device__ __forceinline__ uint32_t bar_tdone(const MassSmem &s) { return s.bars + 8 * (2 * kMaxStages + 2 * kSBars + 4); }
__device__ __forceinline__ uint32_t bar_mmadone(const MassSmem &s) { return s.bars + 8 * (2 * kMaxStages + 2 * kSBars + 5); }

// What one request contributes, and what is wrong with it.
struct Request {
  int L, row0, ql;
};
__device__ __forceinline__ uint32_t read_request(const MassParams &p, int r, Request &q) {
  q.L = p.L[r];
  q.row0 = p.cu[r];
  q.ql = p.cu[r + 1] - q.row0;
  uint32_t fl = 0;
  if (q.L < 0 || q.L > p.mass_stride || ((int64_t)q.L + p.ps - 1) >> p.ps_shift > p.bt_stride)
    fl |= PA_DEV_BAD_CONTEXT;
  if (q.ql < 0 || q.ql > p.maxq || q.L < q.ql || q.row0 < 0 || q.row0 > p.R - q.ql) fl |= PA_DEV_BAD_QLEN;
  return fl;
}

// tstart[r]: the tiles of requests 0 .. r - 1 (per KV head); flagged requests and those without rows
// have none.  Returns the flags.
__device__ uint32_t scan_requests(const MassParams &p, const MassSmem &s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t flags = 0;
  int run = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int r = b0 + tid;
    int n = 0;
    if (r < p.B) {
      Request q;
      const uint32_t fl = read_request(p, r, q);
      flags |= fl;
      if (!fl && q.ql > 0) n = (q.L + kTile - 1) / kTile;
      s.info[3 * r] = q.L;
      s.info[3 * r + 1] = q.row0;
      s.info[3 * r + 2] = q.ql;
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s.wsum[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int v = s.wsum[w];
      before += w < warp ? v : 0;
      all += v;
    }
    if (r < p.B) s.tstart[r] = run + before + x - n;
    run += all;
  }
  if (tid == 0) s.tstart[p.B] = run;
  __syncthreads();
  return flags;
}

// A segment: tiles [t0, t1) of (request r, KV head h) against its query rows [tok0, tok0 + nr).
// Every role walks the same segments of the CTA's tiles [a, b), in order; the rows of a
// (request, head) beyond four come in further segments over the same tiles.
struct Segment {
  int r, h, t0, t1, tok0, nr;
  Request q;
};
struct Walk {
  int at, end;  // tiles of the call, over all heads (their mass takes 512 bytes each: fewer than 2^31)
  Segment s;
  bool open;
  __device__ Walk(int a, int b) : at(a), end(b), open(false) {}
  // The epilogue group of tile t: in turn over the CTA's tiles, so that short segments spread over the groups
  // too, and the same for all rows of a (request, head).
  __device__ __forceinline__ int group(int t) const { return (at + t - s.t0) & (kGroups - 1); }
  __device__ bool next(const MassParams &p, const MassSmem &sm) {
    if (open && s.tok0 + s.nr < s.q.ql) {
      s.tok0 += s.nr;
      s.nr = min(kRows, s.q.ql - s.tok0);
      return true;
    }
    const bool follows = open;
    if (open) at += s.t1 - s.t0;
    open = at < end;
    if (!open) return false;
    int lo = 0, hi = p.B - 1;  // the last request with tstart * Hkv <= at
    if (follows) {  // as a rule the same one (its next head) or the next (searched for: 44 us, not 33, for 2000 x 128)
      const int r = at < sm.tstart[s.r + 1] * p.Hkv ? s.r : s.r + 1;
      if (r < p.B && at < sm.tstart[r + 1] * p.Hkv) lo = hi = r;
    }
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sm.tstart[mid] * p.Hkv <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int begin = sm.tstart[lo], nt = sm.tstart[lo + 1] - begin, rem = at - begin * p.Hkv;
    s.r = lo;
    s.h = p.Hkv == 1 ? 0 : rem / nt;
    s.t0 = rem - s.h * nt;
    s.t1 = min(nt, s.t0 + (end - at));
    s.q = Request{sm.info[3 * lo], sm.info[3 * lo + 1], sm.info[3 * lo + 2]};
    s.tok0 = 0;
    s.nr = min(kRows, s.q.ql);
    return true;
  }
};

__device__ __forceinline__ void raise(const MassParams &p, uint32_t flag) {
  if (p.status != nullptr) atomicOr(p.status, flag);
}

// A tile's place in the ring of stages, and the parity of its use of it.
struct Place {
  int st = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int n, int nstage) {
    st += n;
    if (st >= 2 * nstage) {  // (a whole segment at once)
      parity ^= (uint32_t)(st / nstage) & 1u;
      st %= nstage;
    } else if (st >= nstage) {
      st -= nstage;
      parity ^= 1u;
    }
  }
};

// A bounded wait by a whole warp: false for all lanes if it gave up for one.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(~0u, pa::mbar_wait_bounded(bar, parity)) != 0;
}

// ---------------------------------------------------------------------------- producer

template <bool BF16>
__device__ void run_producer(const MassParams &p, const MassSmem &sm, int a, int b) {
  const int lane = threadIdx.x & 31;
  const int nb = 32 / p.ppt, slot = lane / p.ppt, kpg = lane - slot * p.ppt;
  const uint64_t pol = pa::l2_evict_first_policy();
  const uint32_t page_tx = (uint32_t)p.ps * (BF16 ? 2 * kD : kD) + (p.ks != nullptr ? 4u * p.ps : 0u);
  int i = 0;
  Place at;
  bool ok = true;
  Walk w(a, b);
  while (ok && w.next(p, sm)) {
    const Segment &s = w.s;
    const int np = (s.q.L + p.ps - 1) >> p.ps_shift;
    const int32_t *row = p.bt + (int64_t)s.r * p.bt_stride;
    // nb tiles' pages at a time, one per lane
    auto lookup = [&](int t) {
      const int idx = (t + slot) * p.ppt + kpg;
      return t + slot < s.t1 && idx < np ? row[idx] : -2;  // -2: past the context
    };
    int ahead = lookup(s.t0);
    for (int t = s.t0; t < s.t1 && ok; t += nb) {
      int phys = ahead;
      if (t + nb < s.t1) ahead = lookup(t + nb);
      if (phys != -2 && (phys < 0 || phys >= p.num_pages)) {
        raise(p, PA_DEV_BAD_PAGE);
        phys = -2;
      }
      const uint32_t valid = __ballot_sync(~0u, phys >= 0);
      const int32_t y = (phys * p.Hkv + s.h) * p.ps;  // the page's first row (unused where phys is -2)
      for (int j = 0; j < nb && t + j < s.t1; ++j, ++i) {
        const int src = j * p.ppt;
        // the stage's earlier tile has been released: the parity of that use, one before this one
        if (i >= p.nstage) ok = warp_wait(bar_empty(sm, at.st), at.parity ^ 1u);
        if (!ok) break;
        const uint32_t bits = (valid >> src) & ((1u << p.ppt) - 1u);
        const uint32_t dst = sm.stages + at.st * p.stage_bytes, fb = bar_full(sm, at.st);
        if (lane == src) {  // a page's first lane announces the tile's bytes, then each lane fetches its page
          sm.valid[at.st] = bits;
          pa::mbar_arrive_expect_tx(fb, __popc(bits) * page_tx);
        }
        __syncwarp();
        if (lane >= src && lane < src + p.ppt && phys >= 0) {
          const uint32_t off = kpg * p.ps * 128;
          pa::tma_load_2d(dst + off, &p.tm_k, 0, y, fb, pol);
          if (BF16) pa::tma_load_2d(dst + 16384 + off, &p.tm_k, 64, y, fb, pol);
          if (p.ks != nullptr) pa::bulk_load_hint(dst + 16384 + kpg * p.ps * 4, p.ks + y, p.ps * 4, fb, pol);
        }
        at.advance(1, p.nstage);
      }
    }
  }
  if (!ok) {
    if (lane == 0) {
      raise(p, PA_DEV_TIMEOUT);
      for (int k = max(0, i - p.nstage); k < i; ++k)  // copies in flight land before the CTA can exit
        pa::mbar_wait_bounded(bar_full(sm, k % p.nstage), (k / p.nstage) & 1);
    }
  }
}

// --------------------------------------------------------------------------------- MMA

__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// TMEM columns of group g's buffer k.
__device__ __forceinline__ uint32_t tmem_buf(const MassParams &p, int g, int k) {
  return (uint32_t)((g * p.nbuf + k) * p.buf_cols);
}

template <bool BF16>
__device__ void run_mma(const MassParams &p, const MassSmem &sm, int a, int b, uint32_t tm) {
  const int lane = threadIdx.x & 31;
  int seg = 0;
  Place at;
  int uses[kGroups] = {0, 0, 0, 0};  // each group's tiles so far
  bool ok = true;
  Walk w(a, b);
  while (ok && w.next(p, sm)) {
    const int qb = seg & 1;
    ok = warp_wait(bar_qready(sm, qb), (seg >> 1) & 1);
    const uint32_t q = sm.q + qb * p.qbuf_bytes;
    const int N = w.s.nr * (BF16 ? kG : 2 * kG);
    const uint32_t id = BF16 ? idesc_bf16(kTile, N) : pa::umma_idesc_e4m3(kTile, N, 0, 0);
    for (int t = w.s.t0; t < w.s.t1 && ok; ++t, at.advance(1, p.nstage)) {
      const int st = at.st, g = w.group(t);
      int n = 0;
#pragma unroll
      for (int x = 0; x < kGroups; ++x) n = x == g ? uses[x]++ : n;
      const int k = n & (p.nbuf - 1), u = n >> (p.nbuf - 1);  // one or two buffers
      ok = warp_wait(bar_full(sm, st), at.parity);
      if (ok && u > 0) ok = warp_wait(bar_sfree(sm, 2 * g + k), (u - 1) & 1);
      if (!ok) break;
      pa::tc_fence_after();
      const uint32_t ka = sm.stages + st * p.stage_bytes, d = tm + tmem_buf(p, g, k);
      if (pa::elect_one()) {
#pragma unroll
        for (int x = 0; x < (BF16 ? 8 : 4); ++x) {  // bf16: the second half of a row in its own 16 KB
          const uint64_t da = pa::umma_sdesc(ka + (BF16 ? (x >> 2) * 16384 + 32 * (x & 3) : 32 * x), 1024, 1024, 2);
          const uint64_t db = pa::umma_sdesc(q + (BF16 ? (x >> 2) * (p.qbuf_bytes >> 1) + 32 * (x & 3) : 32 * x), 1024, 1024, 2);
          if (BF16)
            pa::umma_f16(d, da, db, id, x > 0);
          else
            pa::umma_e4m3(d, da, db, id, x > 0);
        }
        pa::umma_commit(bar_sfull(sm, 2 * g + k));
        pa::umma_commit(bar_empty(sm, st));
        if (t + 1 == w.s.t1) pa::umma_commit(bar_qfree(sm, qb));
      }
      __syncwarp();
    }
    ++seg;
  }
  if (!ok && lane == 0) raise(p, PA_DEV_TIMEOUT);
  __syncwarp();
  if (pa::elect_one()) pa::umma_commit(bar_mmadone(sm));
  __syncwarp();
  if (!warp_wait(bar_mmadone(sm), 0) && lane == 0) raise(p, PA_DEV_TIMEOUT);
  if (!warp_wait(bar_tdone(sm), 0) && lane == 0) raise(p, PA_DEV_TIMEOUT);
  pa::tc_fence_after();
  pa::tmem_dealloc(tm, p.tmem_cols);
}

// ---------------------------------------------------------------------------- epilogue

// The segment's query rows as the MMA's B operand (K-major, 128-byte swizzle), and per (row, head) the
// factor of its scores and its -lse in base 2 (-inf where the row has no key: 2^(x - inf) = 0).
// `rot` shifts the work over the warps: a single row keeps one group busy, and a group per segment in turn
// leaves the others to their tiles (2000 x 128 tokens: 32.7 us without, 28.6 with).
template <bool BF16>
__device__ void convert_queries(const MassParams &p, const MassSmem &sm, const Segment &s, int qb, int rot) {
  const int etid = (threadIdx.x + rot) & (32 * kEpiWarps - 1);
  if ((etid & ~31) >= s.nr * kG * (BF16 ? 16 : 8)) {  // nothing for this warp
    if ((threadIdx.x & 31) == 0) pa::mbar_arrive(bar_qready(sm, qb));
    return;
  }
  const uint32_t dst = sm.q + qb * p.qbuf_bytes, fac = sm.factors + qb * (kFactorBytes / 2);
  const int64_t Hq = (int64_t)p.Hkv * kG;
  const int64_t qrow = (int64_t)(s.q.row0 + s.tok0) * Hq + s.h * kG;  // (row t, head g): + t Hq + g
  for (int u = etid; u < s.nr * kG; u += 32 * kEpiWarps) {
    const float l = p.lse[qrow + (u / kG) * Hq + u % kG];
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(fac + (u / kG) * (2 * kG * 4) + (kG + u % kG) * 4),
                 "f"(l == -INFINITY ? l : -l * kLog2e) : "memory");
  }
  if (BF16) {
    for (int u = etid; u < s.nr * kG * 16; u += 32 * kEpiWarps) {  // 16 bytes: 8 elements
      const int n = u >> 4, c = u & 15;
      const uint4 v = *reinterpret_cast<const uint4 *>(p.q + (qrow + (n / kG) * Hq + n % kG) * kD + 8 * c);
      pa::sts128(dst + (c >> 3) * (p.qbuf_bytes >> 1) + n * 128 + (((c & 7) ^ (n & 7)) << 4), v);
      if (c == 0)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(fac + (n / kG) * (2 * kG * 4) + (n % kG) * 4), "f"(p.kfold) : "memory");
    }
  } else {
    for (int u0 = 0; u0 < s.nr * kG * 8; u0 += 32 * kEpiWarps) {  // 16 elements; 8 lanes per (row, head)
      const int u = u0 + etid, n = u >> 3, c = u & 7;
      const bool live = u < s.nr * kG * 8;
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (live) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (qrow + (n / kG) * Hq + n % kG) * kD + 16 * c);
        x = src[0];
        y = src[1];
      }
      const uint32_t wd[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(pa::bf16lo(wd[j])), fabsf(pa::bf16hi(wd[j]))));
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
      if (!live) continue;
      // 2^sig puts the largest magnitude in [128, 256)
      int sig = 0;
      if (amax > 0.f) sig = min(max(7 - ((int)(__float_as_uint(amax) >> 23) - 127), -126), 126);
      const float up = __uint_as_float((uint32_t)(sig + 127) << 23);
      uint32_t hw[4] = {0u, 0u, 0u, 0u}, lw[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // word j: d = 16 c + 2 j, + 1
        const float y0 = pa::bf16lo(wd[j]) * up, y1 = pa::bf16hi(wd[j]) * up;
        const uint32_t hc = pa::pack_e4m3x2(y0, y1);
        float h0, h1;
        pa::e4m3x2_to_f32x2(hc, h0, h1);
        const uint32_t lc = pa::pack_e4m3x2((y0 - h0) * 32.f, (y1 - h1) * 32.f);
        hw[j >> 1] |= hc << (16 * (j & 1));
        lw[j >> 1] |= lc << (16 * (j & 1));
      }
      const int row = (n / kG) * 2 * kG + n % kG;  // hi; lo 16 rows on
      const uint32_t off = row * 128 + ((c ^ (row & 7)) << 4);
      pa::sts128(dst + off, make_uint4(hw[0], hw[1], hw[2], hw[3]));
      pa::sts128(dst + kG * 128 + off, make_uint4(lw[0], lw[1], lw[2], lw[3]));
      if (c == 0)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(fac + (n / kG) * (2 * kG * 4) + (n % kG) * 4),
                     "f"(p.kfold * __uint_as_float((uint32_t)(127 - sig) << 23)) : "memory");
    }
  }
  pa::fence_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) pa::mbar_arrive(bar_qready(sm, qb));
}

template <bool BF16>
__device__ void run_epilogue(const MassParams &p, const MassSmem &sm, int a, int b, uint32_t tm) {
  const int etid = threadIdx.x, lane = etid & 31, warp = etid >> 5, g = warp >> 2, quarter = warp & 3;
  const int tok = 32 * quarter + lane;  // of a tile: the TMEM lane
  const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
  int seg = 0, cnt = 0;
  Place begin;  // of the segment
  bool ok = true;
  Walk w(a, b), ahead(a, b);
  if (ahead.next(p, sm)) convert_queries<BF16>(p, sm, ahead.s, 0, 0);
  while (ok && w.next(p, sm)) {
    const Segment s = w.s;
    const int qb = seg & 1;
    if (ahead.next(p, sm)) {
      // segment seg - 1, which had the other buffers: its MMAs and every group are done
      if (seg >= 1) ok = warp_wait(bar_qfree(sm, qb ^ 1), ((seg - 1) >> 1) & 1);
      if (!ok) break;
      convert_queries<BF16>(p, sm, ahead.s, qb ^ 1, 128 * (seg + 1));
    }
    const uint32_t fac = sm.factors + qb * (kFactorBytes / 2);
    const int64_t mrow = ((int64_t)s.r * p.Hkv + s.h) * p.mass_stride;
    // What the mass of this thread's position in tile t was, asked for two of the group's tiles ahead.
    auto before = [&](int t) {
      const int pos = t * kTile + tok;
      if (t >= s.t1 || pos >= s.q.L) return 0.f;
      if (s.tok0 > 0) return p.out[mrow + pos];  // this thread's own sum over the rows before
      return pos < s.q.L - s.q.ql && p.decay != 0.f ? p.mass[mrow + pos] : 0.f;
    };
    const float keep = s.tok0 > 0 ? 1.f : p.decay;
    int t = s.t0 + ((g - w.group(s.t0)) & (kGroups - 1));  // the group's first tile
    float old0 = before(t), old1 = before(t + kGroups);
    Place at = begin;
    at.advance(t - s.t0, p.nstage);
    begin.advance(s.t1 - s.t0, p.nstage);
    // (by the warps that have no tile of it too: a parity tells a barrier's last two uses apart, not three)
    ok = warp_wait(bar_qready(sm, qb), (seg >> 1) & 1);
    for (; t < s.t1 && ok; t += kGroups, at.advance(kGroups, p.nstage)) {
      const int st = at.st, k = cnt & (p.nbuf - 1), pos = t * kTile + tok;
      const bool live = pos < s.q.L;
      const float old = keep * old0;
      old0 = old1;
      old1 = before(t + 2 * kGroups);
      ok = warp_wait(bar_full(sm, st), at.parity) &&
           warp_wait(bar_sfull(sm, 2 * g + k), (cnt >> (p.nbuf - 1)) & 1);
      if (!ok) break;
      ++cnt;
      float ks = 1.f;
      const uint32_t base = sm.stages + st * p.stage_bytes;
      if (!BF16 && p.ks != nullptr) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks) : "r"(base + 16384 + 4 * tok) : "memory");
      const bool valid = (sm.valid[st] >> (tok >> p.ps_shift)) & 1u;
      __syncwarp();
      if (lane == 0) pa::mbar_arrive(bar_empty(sm, st));
      pa::tc_fence_after();
      const pa::f32x2 ks2 = pa::pack2(ks, ks), lo_unit = pa::pack2(1.f / 32.f, 1.f / 32.f);
      float sum = 0.f;
      for (int x = 0; x < s.nr; ++x) {
        uint32_t hi[kG], lo[kG];
        const uint32_t col = tl + tmem_buf(p, g, k) + x * (BF16 ? kG : 2 * kG);
        pa::tmem_ld16_async(col, hi);
        if (!BF16) pa::tmem_ld16_async(col + kG, lo);
        pa::tmem_wait16(hi);
        if (!BF16) pa::tmem_wait16(lo);
        const uint32_t f = fac + x * (2 * kG * 4);
        pa::f32x2 part[2] = {pa::pack2(0.f, 0.f), pa::pack2(0.f, 0.f)};
#pragma unroll
        for (int j = 0; j < kG; j += 4) {
          const uint4 kv = pa::lds128(f + 4 * j), lv = pa::lds128(f + 4 * (kG + j));
          const uint32_t kf[4] = {kv.x, kv.y, kv.z, kv.w}, l2[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            pa::f32x2 d = pa::pack2(__uint_as_float(hi[j + e]), __uint_as_float(hi[j + e + 1]));
            if (!BF16) d = pa::fma2(pa::pack2(__uint_as_float(lo[j + e]), __uint_as_float(lo[j + e + 1])), lo_unit, d);
            const pa::f32x2 c = pa::mul2(pa::pack2(__uint_as_float(kf[e]), __uint_as_float(kf[e + 1])), ks2);
            d = pa::fma2(d, c, pa::pack2(__uint_as_float(l2[e]), __uint_as_float(l2[e + 1])));
            float d0, d1;
            pa::unpack2(d, d0, d1);
            part[e >> 1] = pa::add2(part[e >> 1], pa::pack2(pa::fast_exp2(d0), pa::fast_exp2(d1)));
          }
        }
        float p0, p1, p2, p3;
        pa::unpack2(part[0], p0, p1);
        pa::unpack2(part[1], p2, p3);
        if (pos < s.q.L - s.q.ql + s.tok0 + x + 1) sum += (p0 + p1) + (p2 + p3);
      }
      pa::tc_fence_before();
      __syncwarp();
      if (lane == 0) pa::mbar_arrive(bar_sfree(sm, 2 * g + k));
      if (live) p.out[mrow + pos] = old + (valid ? sum : 0.f);
    }
    if (ok && lane == 0) pa::mbar_arrive(bar_qfree(sm, qb));  // the factors have been read
    __syncwarp();
    ++seg;
  }
  if (!ok && lane == 0) raise(p, PA_DEV_TIMEOUT);
  pa::tc_fence_before();
  __syncwarp();
  if (lane == 0) pa::mbar_arrive(bar_tdone(sm));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) attn_mass_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t mis = pa::smem_u32(raw) & 1023u;
  const MassSmem sm = carve(raw + ((1024u - mis) & 1023u), p);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int k = 0; k < p.nstage; ++k) {
      pa::mbar_init(bar_full(sm, k), 1);
      pa::mbar_init(bar_empty(sm, k), 1 + 4);  // the MMAs' commit, the warps of the tile's group
    }
    for (int k = 0; k < kSBars; ++k) {
      pa::mbar_init(bar_sfull(sm, k), 1);
      pa::mbar_init(bar_sfree(sm, k), 4);
    }
    for (int k = 0; k < 2; ++k) {
      pa::mbar_init(bar_qready(sm, k), kEpiWarps);
      pa::mbar_init(bar_qfree(sm, k), 1 + kEpiWarps);  // the MMAs' commit, the epilogue's warps
    }
    pa::mbar_init(bar_tdone(sm), kEpiWarps);
    pa::mbar_init(bar_mmadone(sm), 1);
    pa::fence_barrier_init();
  }
  if (warp == kEpiWarps + 1) pa::tmem_alloc(pa::smem_u32(sm.misc), p.tmem_cols);
  pa::tc_fence_before();
  // Up to here the CTA may run beside the kernel before it (programmatic dependent launch): it has
  // read nothing.  The next kernel may start as soon as this one's inputs are complete.
  pa::pdl_wait();
  pa::pdl_launch_dependents();
  const uint32_t fl = scan_requests(p, sm);  // synchronises the CTA
  pa::tc_fence_after();
  if (blockIdx.x == 0 && fl) raise(p, fl);
  // this CTA's tiles: an equal share, the odd ones spread over the CTAs (all to the first ones: 0.3 us
  // more for 8 x 131072)
  const int total = sm.tstart[p.B] * p.Hkv, grid = (int)gridDim.x, cta = (int)blockIdx.x;
  const int each = total / grid, more = total - each * grid;
  const int a = cta * each + cta * more / grid, b = (cta + 1) * each + (cta + 1) * more / grid;
  if (a >= b) {  // the whole CTA
    if (warp == kEpiWarps + 1) pa::tmem_dealloc(sm.misc[0], p.tmem_cols);
    return;
  }
  const uint32_t tm = sm.misc[0];
  if (warp < kEpiWarps)
    run_epilogue<BF16>(p, sm, a, b, tm);
  else if (warp == kEpiWarps)
    run_producer<BF16>(p, sm, a, b);
  else
    run_mma<BF16>(p, sm, a, b, tm);
}

// ------------------------------------------------------------------------------- host

struct MassDevice {
  int sms = 0, smem = 0;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
};

// The current device's SM count and shared memory, the kernels' opt-in, and the tensor-map
// encoder, once per device; NULL when a call fails or the device is beyond those tracked.
const MassDevice *mass_device() {
  static std::once_flag once[pa_host::kMaxDevices];
  static MassDevice devs[pa_host::kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= pa_host::kMaxDevices) return nullptr;
  std::call_once(once[dev], [dev]() {
    MassDevice d;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaFuncSetAttribute(attn_mass_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem) != cudaSuccess ||
        cudaFuncSetAttribute(attn_mass_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem) != cudaSuccess ||
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      return;
    d.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    devs[dev] = d;
  });
  return devs[dev].encode != nullptr ? &devs[dev] : nullptr;
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
  if (a->group_size != kG || a->max_q_len > kMaxQ || a->num_seqs > kMaxSeqs || a->mass_stride > kMaxPositions)
    return PA_ERR_UNSUPPORTED;
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
  const uint64_t lens = (uint64_t)a->num_seqs * 4, heads = (uint64_t)a->num_rows * a->num_kv_heads * kG;
  if (pa_host::overlaps({a->mass_out, bytes}, {{a->q, heads * kD * 2}, {a->lse, heads * 4}, {a->context_lens, lens},
                                               {a->cu_seqlens_q, lens + 4}, {a->block_table, lens * a->block_table_stride}}))
    return PA_ERR_INVALID_ARG;
  if (a->num_seqs == 0 || a->num_rows == 0) return PA_OK;

  const MassDevice *dev = mass_device();
  if (dev == nullptr) return PA_ERR_CUDA;

  MassParams p;
  p.q = static_cast<const uint16_t *>(a->q);
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
  const bool bf16 = a->kv_dtype == PA_KV_BF16;
  p.ppt = kTile / a->page_size;
  p.kfold = (float)((double)a->sm_scale * 1.4426950408889634 *
                    (a->scale_mode == PA_SCALE_SCALAR ? (double)a->k_scale_scalar : 1.0));
  p.decay = a->decay;
  // Query operand and TMEM for the rows a segment can have (two buffers per group where 512 columns hold
  // them, so that a group's next tile is multiplied while it reads this one); as many stages as fit.
  const int nr = std::min(a->max_q_len, kRows);
  p.qbuf_bytes = nr * 2 * kG * 128;  // e4m3: 32 rows of 128 bytes; bf16: two halves of 16 rows
  p.buf_cols = nr * (bf16 ? kG : 2 * kG);
  p.nbuf = 2 * kGroups * p.buf_cols <= 512 ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < kGroups * p.nbuf * p.buf_cols) p.tmem_cols *= 2;
  p.stage_bytes = bf16 ? 32768 : 16384 + 1024;  // keys, then an e4m3 tile's scales
  const int fixed = 1024 + 2 * p.qbuf_bytes + kCtrlBytes + (4 * a->num_seqs + 1) * 4;
  p.nstage = std::min(kMaxStages, (dev->smem - fixed) / p.stage_bytes);
  if (p.nstage < 2) return PA_ERR_UNSUPPORTED;
  const size_t smem = (size_t)fixed + (size_t)p.nstage * p.stage_bytes;

  cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)(a->num_pages * a->num_kv_heads * a->page_size)};
  cuuint64_t strides[1] = {(cuuint64_t)(bf16 ? 2 * kD : kD)};
  cuuint32_t box[2] = {(cuuint32_t)(bf16 ? 64 : 128), (cuuint32_t)a->page_size};
  cuuint32_t estr[2] = {1, 1};
  if (dev->encode(&p.tm_k, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                  const_cast<void *>(a->k_cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return PA_ERR_CUDA;

  // One CTA per SM, or fewer where the mass rows cannot hold that many tiles
  const int64_t tiles = (int64_t)a->num_seqs * a->num_kv_heads * ((a->mass_stride + kTile - 1) / kTile);
  const int grid = (int)std::min<int64_t>(dev->sms, tiles);
  pa_host::Launch run(dim3((unsigned)grid), dim3(kThreads), smem, stream);
  const cudaError_t e = bf16 ? cudaLaunchKernelEx(run.cfg(), attn_mass_kernel<true>, p)
                             : cudaLaunchKernelEx(run.cfg(), attn_mass_kernel<false>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
