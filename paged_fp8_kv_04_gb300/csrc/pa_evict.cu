// pa_evict.cu -- eviction from the paged cache: pa_evict_select chooses the tokens that stay,
// pa_kv_compact moves them to the front of their pages.  See include/pa.h for the contract.
//
// The selection has little to read (4 B per position) and is bound by its dependent steps:
// measured on 16 rows x 131072 (8.4 MB, 1.3 us at HBM rate) 17.3 us, of which the masses take 2.5, a
// counting step 3 (counting, two exchanges of 0.5 to 0.7 each, the pick; two or three steps as a rule), counting
// and writing 3; some SMs have CTAs of two rows (8 rows: 13.9 us).  One CTA per row, bit by bit, took 475 us.
// The compaction is bound by HBM: 528 B and more per kept token.  32 x 8192 tokens into other pages, 142 MB,
// take 26.8 us (5.3 TB/s, 0.78 of a copy's rate); 8 x 4095 in place 6.1 us.  One CTA per row
// took 203 and 70 us; rows carried in registers 33 and 10 us.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <mutex>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kMaxRows = 65535;         // (request, KV head) pairs of a call
constexpr int kMaxPositions = 1 << 30;  // per (request, KV head) row

// --------------------------------------------------------------------------- selection

struct SelectParams {
  const float *mass;
  const int32_t *L;
  int32_t *keep, *new_lens;
  uint32_t *status;
  int32_t Hkv, stride, budget, first, recent;
};

// Unsigned keys in the order of the masses, from 1 (NaN) to that of +inf; -0 = +0.  0 stands for a
// position that is not a middle one.
__device__ __forceinline__ uint32_t mass_key(float m) {
  const uint32_t u = __float_as_uint(m + 0.f);
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return m != m ? 1u : k;
}

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;   // and twice that where it pays
constexpr int kMaxKeys = 32;     // keys a thread can hold
// Masses a thread has on their way where it holds no keys (one at a time: 55.7 us against 43.5 for 1 x 262144).
constexpr int kBatch = 16;

// A cluster of C CTAs per (request, KV head), each with one stretch of the positions, a warp with
// one stretch of those.  The masses are read once, as keys into registers, KPT per thread; rows
// beyond C * 512 * 32 positions (KPT 0) are read again instead.  The key T of the last middle token
// taken is found by counting keys in 2048 bins of the range that still holds it: the top 11 bits,
// then the 11 bits below them of the keys in one bin, then the last 10.  The CTAs' counts meet
// through distributed shared memory: each CTA sums its share of the bins and sends the sums to all, 16
// bytes per thread and direction in place of 64 KB per CTA.  They are asynchronous stores that the
// receiver counts: loads of what the others have left, or cluster barriers, measured a round trip more
// (8 rows x 131072: 16.1 us against 14.4).  A part or a sum is overwritten in the next step only by CTAs that
// have what its reader sent after reading it.  A bin that is taken whole ends the search early.  Then the
// kept positions are written in order: those above T and the first `need` equal to it, at offsets from
// the counts of the warps and CTAs before.
struct SelectShared {
  uint32_t hist[kBins];          // this CTA's keys
  uint32_t part[kBins];          // its share of the bins, from each CTA of the cluster
  uint32_t own[kBins / 2];       // and summed
  uint32_t all[kBins];           // the cluster's keys
  uint2 totals[2 * kMaxCluster];  // of each CTA: keys equal to T, and certain ones
  uint64_t bars[3];              // part, all, totals: what the cluster sends has arrived
  int weq[kSelWarps], wsure[kSelWarps], scan[kSelWarps];
  int pick[3];                   // the chosen bin, keys above it, keys in it
};

// Asynchronous stores to this shared-memory address in CTA `rank` of the cluster, which count towards
// the barrier `bar` there.
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(pa::smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void push_cluster(void *p, uint64_t *bar, uint32_t rank, const uint4 &v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(in_cta(p, rank)),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(in_cta(bar, rank))
               : "memory");
}
__device__ __forceinline__ void push_cluster(void *p, uint64_t *bar, uint32_t rank, const uint2 &v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(in_cta(p, rank)),
               "r"(v.x), "r"(v.y), "r"(in_cta(bar, rank))
               : "memory");
}

// A bounded wait for a phase of what the cluster sends; false if it gave up.
__device__ __forceinline__ bool wait_cluster(const uint64_t *bar, uint32_t parity) {
  const uint32_t a = pa::smem_u32(bar);
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > pa::kWaitCycles) return false;
  }
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The number of `eq` equal keys that stay when `before` of them come earlier.
__device__ __forceinline__ int ties_taken(int need, int before, int eq) { return min(max(need - before, 0), eq); }

template <int KPT>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const SelectParams p) {
  __shared__ __align__(16) SelectShared sm;
  pa::pdl_wait();
  const int C = (int)pa::cluster_ctas(), rank = (int)pa::cluster_rank();
  const int row = blockIdx.x / C, r = row / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float *m = p.mass + (int64_t)row * p.stride;
  // This warp's positions [wb, we) are cut from the row's capacity, not its length: its masses are on their
  // way while the length is (4 x 1000: 3.99 us, and 4.33 when they wait for it).
  const int stretch = (((p.stride + C * kSelWarps - 1) / (C * kSelWarps)) + 31) & ~31;
  const int wb = (int)min((int64_t)(rank * kSelWarps + warp) * stretch, (int64_t)p.stride);
  float x[KPT > 0 ? KPT : 1];
#pragma unroll
  for (int u = 0; u < KPT; ++u) {
    const int i = wb + 32 * u + lane;
    x[u] = i < p.stride ? m[i] : 0.f;
  }
  const int L = p.L[r];
  int32_t *keep = p.keep + (int64_t)row * p.budget;
  const bool bad = L < 0 || L > p.stride;
  const int n = bad ? 0 : min(L, p.budget);
  if (row == r * p.Hkv && rank == 0 && tid == 0) {
    p.new_lens[r] = n;
    if (bad && p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_CONTEXT);
  }
  const int gid = rank * kSelThreads + tid, gsz = C * kSelThreads;
  if (bad || n == L) {  // the same for the whole cluster
    for (int64_t i = gid; i < p.budget; i += gsz) keep[i] = i < n ? (int)i : -1;
    return;
  }
  if (C > 1 && tid == 0) {
    for (int b = 0; b < 3; ++b) pa::mbar_init(pa::smem_u32(&sm.bars[b]), 1);
    pa::fence_barrier_init();
    pa::mbar_arrive_expect_tx(pa::smem_u32(&sm.bars[2]), C * sizeof(uint2));
  }
  pa::cluster_arrive();
  // A wait for what the cluster sends.  Where one runs out (bounded: it does not) the request is flagged, and
  // no CTA leaves while another may still send to it.
  auto arrived = [&](int b, uint32_t parity) { return wait_cluster(&sm.bars[b], parity); };
  auto give_up = [&]() {
    if (tid == 0 && p.status != nullptr) atomicOr(p.status, PA_DEV_TIMEOUT);
    pa::cluster_sync();
  };
  // of the row the middle positions [mlo, mhi)
  const int we = (int)max((int64_t)wb, min((int64_t)wb + stretch, (int64_t)L));
  const int mlo = p.first, mhi = L - p.recent, want = p.budget - p.first - p.recent;

  // Position u of a lane is wb + 32 u + lane; the warp's middle ones are [lo, hi).
  const int lo = max(wb, mlo), hi = min(we, mhi);
  // the warp's keys in batches of kBatch loads in flight (KPT 0)
  auto batches = [&](int from, int to, auto &&each) {
    for (int i0 = from; i0 < to; i0 += 32 * kBatch) {
      float x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        x[u] = i >= lo && i < hi ? m[i] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        each(i, i >= lo && i < hi ? mass_key(x[u]) : 0u);
      }
    }
  };
  uint32_t key[KPT > 0 ? KPT : 1];
  if (KPT > 0) {
    const unsigned count = (unsigned)max(hi - lo, 0);
#pragma unroll
    for (int u = 0; u < KPT; ++u) key[u] = (unsigned)(wb + 32 * u + lane - lo) < count ? mass_key(x[u]) : 0u;
  }
  static_assert(kBins == 4 * kSelThreads, "four bins per thread");
  uint4 *hist4 = reinterpret_cast<uint4 *>(sm.hist) + tid;
  *hist4 = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  pa::cluster_wait();  // every CTA of the cluster runs: its shared memory can be written

  uint32_t T = 0xFFFFFFFFu;  // with want 0 nothing of the middle stays
  int need = 0;
  if (want > 0) {
    // keys in [base, base + span] are still open; 0 never is (the largest key is that of +inf)
    uint32_t base = 1, span = 0xFFFFFFFEu;
    need = want;
    for (int step = 0;; ++step) {
      const int shift = step == 0 ? 21 : step == 1 ? 10 : 0;
      if (KPT > 0) {
#pragma unroll
        for (int u = 0; u < KPT; ++u) {
          const uint32_t d = key[u] - base;
          if (d <= span) atomicAdd(sm.hist + (d >> shift), 1u);
        }
      } else {
        batches(lo, hi, [&](int, uint32_t k) {
          const uint32_t d = k - base;
          if (d <= span) atomicAdd(sm.hist + (d >> shift), 1u);
        });
      }
      __syncthreads();
      uint4 c = *hist4;
      *hist4 = make_uint4(0u, 0u, 0u, 0u);
      if (C > 1) {
        // four bins per thread, to the CTA that sums them, and the sums to all
        const int quads = kBins / 4 / C, q = tid / quads, e4 = tid - q * quads;
        if (tid == 0) {
          pa::mbar_arrive_expect_tx(pa::smem_u32(&sm.bars[0]), sizeof(sm.part));
          pa::mbar_arrive_expect_tx(pa::smem_u32(&sm.bars[1]), sizeof(sm.all));
        }
        push_cluster(sm.part + 4 * (rank * quads + e4), &sm.bars[0], q, c);
        bool ok = arrived(0, step & 1);
        if (tid < quads) {
          c = make_uint4(0u, 0u, 0u, 0u);
          for (int k = 0; k < C; ++k) {
            const uint4 x = *reinterpret_cast<const uint4 *>(sm.part + 4 * (k * quads + tid));
            c.x += x.x;
            c.y += x.y;
            c.z += x.z;
            c.w += x.w;
          }
          *reinterpret_cast<uint4 *>(sm.own + 4 * tid) = c;
        }
        if (__syncthreads_or(!ok)) return give_up();
        push_cluster(sm.all + 4 * (rank * quads + e4), &sm.bars[1], q, *reinterpret_cast<const uint4 *>(sm.own + 4 * e4));
        ok = arrived(1, step & 1);
        if (__syncthreads_or(!ok)) return give_up();
        c = *reinterpret_cast<const uint4 *>(sm.all + 4 * tid);
      }
      // the bin that holds the want-th key from the top (one thread finds it; none only if the masses change
      // under the call)
      int above = 0;
      const int four = (int)(c.x + c.y + c.z + c.w), incl = warp_scan(four, lane);
      if (lane == 31) sm.scan[warp] = incl;
      __syncthreads();
      const int w = lane < kSelWarps ? sm.scan[lane] : 0, wincl = warp_scan(w, lane);
      above += __shfl_sync(~0u, wincl, 31) - (__shfl_sync(~0u, wincl - w, warp) + incl);
      const uint32_t bins[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        if (above < need && need <= above + (int)bins[e]) {
          sm.pick[0] = 4 * tid + e;
          sm.pick[1] = above;
          sm.pick[2] = (int)bins[e];
        }
        above += (int)bins[e];
      }
      __syncthreads();
      base += (uint32_t)sm.pick[0] << shift;
      need -= sm.pick[1];
      T = base;
      if (shift == 0) break;  // T is the key, and `need` of its tokens stay
      if (need == sm.pick[2]) {  // the whole bin stays: everything from its lowest key on
        need = INT_MAX;
        break;
      }
      span = (1u << shift) - 1u;
    }
  }

  // ---- count, then write.  Bit u of `sure` and `eq`: position u stays; it has key T
  uint32_t sure = 0, eq = 0;
  int nsure = 0, neq = 0;
  const bool ends = wb < mlo || we > mhi;  // the warp has some of the first or the recent positions
  auto always = [&](int i) { return i < we && (i < mlo || i >= mhi); };
  if (KPT > 0) {
#pragma unroll
    for (int u = 0; u < KPT; ++u) {
      sure |= (uint32_t)(key[u] > T) << u;
      eq |= (uint32_t)(key[u] == T) << u;
    }
    if (ends)
#pragma unroll
      for (int u = 0; u < KPT; ++u) sure |= (uint32_t)always(wb + 32 * u + lane) << u;
    nsure = __popc(sure);
    neq = __popc(eq);
  } else {
    batches(wb, we, [&](int i, uint32_t k) {
      nsure += k > T || always(i);
      neq += k == T;
    });
  }
  nsure = __reduce_add_sync(~0u, nsure);
  neq = __reduce_add_sync(~0u, neq);
  if (lane == 0) {
    sm.wsure[warp] = nsure;
    sm.weq[warp] = neq;
  }
  __syncthreads();
  if (warp == 0) {
    const int e = __reduce_add_sync(~0u, lane < kSelWarps ? sm.weq[lane] : 0);
    const int y = __reduce_add_sync(~0u, lane < kSelWarps ? sm.wsure[lane] : 0);
    if (C == 1)
      sm.totals[0] = make_uint2((uint32_t)e, (uint32_t)y);
    else if (lane < C)
      push_cluster(&sm.totals[rank], &sm.bars[2], lane, make_uint2((uint32_t)e, (uint32_t)y));
  }
  if (__syncthreads_or(C > 1 && !arrived(2, 0))) return give_up();
  const uint2 ct = lane < C ? sm.totals[lane] : make_uint2(0u, 0u);
  const int ceq = (int)ct.x, ceq_before = warp_scan(ceq, lane) - ceq;
  const int ckept = (int)ct.y + ties_taken(need, ceq_before, ceq);
  const int cstart = warp_scan(ckept, lane) - ckept;
  int before = __shfl_sync(~0u, ceq_before, rank), at = __shfl_sync(~0u, cstart, rank);
  {
    const int e = lane < kSelWarps ? sm.weq[lane] : 0, eb = before + warp_scan(e, lane) - e;
    const int kept = (lane < kSelWarps ? sm.wsure[lane] : 0) + ties_taken(need, eb, e);
    const int start = at + warp_scan(kept, lane) - kept;
    before = __shfl_sync(~0u, eb, warp);
    at = __shfl_sync(~0u, start, warp);
  }
  const unsigned lt = (1u << lane) - 1u;
  auto emit = [&](int i, bool is_sure, bool is_eq) {
    const unsigned eqs = __ballot_sync(~0u, is_eq);
    const bool stays = is_sure || (is_eq && before + __popc(eqs & lt) < need);
    const unsigned st = __ballot_sync(~0u, stays);
    if (stays && at + __popc(st & lt) < p.budget) keep[at + __popc(st & lt)] = i;
    at += __popc(st);
    before += __popc(eqs);
  };
  if (KPT > 0) {
    if (before >= need || neq <= need - before) {  // none or all of the warp's equal keys stay: no ranks to count
      const uint32_t stays = before >= need ? sure : sure | eq;
#pragma unroll
      for (int u = 0; u < KPT; ++u) {
        const unsigned st = __ballot_sync(~0u, (stays >> u) & 1u);
        if ((stays >> u) & 1u) keep[at + __popc(st & lt)] = wb + 32 * u + lane;
        at += __popc(st);
      }
    } else {
#pragma unroll 1
      for (int u = 0; u < KPT; ++u) emit(wb + 32 * u + lane, (sure >> u) & 1u, (eq >> u) & 1u);
    }
  } else {
    batches(wb, we, [&](int i, uint32_t k) { emit(i, k > T || always(i), k == T); });
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
  int32_t Hkv, ps, ps_shift, keep_stride, bt_stride, dt_stride, m_stride, mo_stride;
};

constexpr int kMoveThreads = 256;
// K and V rows of a CTA's round in shared memory: three CTAs per SM.  Half of it gains 2% into other pages
// (26.6 us) and loses 20% in place (8.1 us).
constexpr int kMoveBytes = 65536;
constexpr int kMaxMoveCluster = 16;  // more than 8 needs the kernel's opt-in

// Tokens of a round: 256 with 128-byte rows, 128 with 256-byte ones.
template <int RC>
__host__ __device__ constexpr int move_tokens() { return kMoveBytes / (32 * RC); }

struct MoveShared {
  int32_t from[256];  // cache row of each token of the round, or -1: not to be written
  unsigned odd;       // destination pages (of the round) with a token that is not to be written
  unsigned moved;     // and those with one that is, and comes from elsewhere
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Contiguous bulk copy shared -> global (16-byte aligned addresses and size).
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// The request's new length, or 0 where it cannot be (flagged once).
__device__ __forceinline__ int new_length(const CompactParams &p, int r, bool flag) {
  const int n = p.new_lens[r];
  if (n < 0 || n > p.keep_stride || ((int64_t)n + p.ps - 1) >> p.ps_shift > p.dt_stride ||
      (p.mass != nullptr && n > p.mo_stride)) {
    if (flag && p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_KEEP);
    return 0;
  }
  return n;
}

// A round of a (request, KV head): T tokens, whose rows are gathered into shared memory with 16-byte
// asynchronous copies (all of a round's 64 KB in flight at once) and leave it as one bulk store of K and
// one of V per destination page, since the destinations are consecutive slots.  A thread per
// token looks its row up and carries its scales and mass.
//
// Into other pages each CTA moves one round.  In place the CTAs of a cluster share the rounds of a
// row: kept positions ascend, so keep[i] >= i, and the destinations of a round are sources of
// this round or an earlier one only.  So a round is written once every CTA has read its part of it
// (one cluster barrier), and the next may be read meanwhile: its sources lie further on.
template <int RC, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, 3) kv_compact_kernel(const CompactParams p) {
  constexpr int T = move_tokens<RC>(), kRow = 16 * RC;
  extern __shared__ __align__(128) uint8_t tile[];  // K rows, then V rows
  __shared__ MoveShared sm;
  pa::pdl_wait();
  const int tid = threadIdx.x;
  const int C = IN_PLACE ? (int)pa::cluster_ctas() : (int)gridDim.x, rank = IN_PLACE ? (int)pa::cluster_rank() : (int)blockIdx.x;
  const int64_t row = IN_PLACE ? blockIdx.x / C : blockIdx.y;
  const int h = (int)(row % p.Hkv), r = (int)(row / p.Hkv);
  const int n = new_length(p, r, rank == 0 && h == 0 && tid == 0);
  const int32_t *keep = p.keep + row * p.keep_stride;
  const uint32_t ks_at = pa::smem_u32(tile), vs_at = ks_at + T * kRow;
  const int64_t round = (int64_t)C * T;
  // every CTA of a cluster takes part in every round's barrier
  for (int64_t start = 0; start < n; start += round) {
    const int64_t first = start + (int64_t)rank * T, i = first + tid;
    if (!IN_PLACE && first >= n) return;
    if (tid == 0) sm.odd = sm.moved = 0;
    __syncthreads();
    float kx = 0.f, vx = 0.f, mx = 0.f;
    int from = -1, to = -1;
    bool moves = false;
    if (tid < T && i < n) {
      const int s = keep[i], prev = i > 0 ? keep[i - 1] : -1;
      const int dp = p.dt[(int64_t)r * p.dt_stride + (i >> p.ps_shift)];
      if (s <= prev || s < i || s >> p.ps_shift >= p.bt_stride || (p.mass != nullptr && s >= p.m_stride)) {
        if (p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_KEEP);
      } else {
        const int sp = p.bt[(int64_t)r * p.bt_stride + (s >> p.ps_shift)];
        if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) {
          if (p.status != nullptr) atomicOr(p.status, PA_DEV_BAD_PAGE);
        } else {
          from = ((sp * p.Hkv + h) << p.ps_shift) + (s & (p.ps - 1));
          to = ((dp * p.Hkv + h) << p.ps_shift) + (int)(i & (p.ps - 1));
          moves = !IN_PLACE || s != i;
          if (moves) {
            if (p.ks != nullptr) {
              kx = p.ks[from];
              vx = p.vs[from];
            }
            if (p.mass != nullptr) mx = p.mass[row * p.m_stride + s];
          }
        }
      }
      const unsigned seg = 1u << (tid >> p.ps_shift);
      if (from < 0) atomicOr(&sm.odd, seg);
      if (moves) atomicOr(&sm.moved, seg);
    }
    if (tid < T) sm.from[tid] = from;
    __syncthreads();
    const unsigned moved = sm.moved, odd = sm.odd;
#pragma unroll 4
    for (int u = tid; u < T * RC; u += kMoveThreads) {
      const int t = u / RC, c = u % RC, f = sm.from[t];
      if (f >= 0 && (moved >> (t >> p.ps_shift)) & 1u) {
        cp_async16(ks_at + 16 * u, p.k + (int64_t)f * kRow + 16 * c);
        cp_async16(vs_at + 16 * u, p.v + (int64_t)f * kRow + 16 * c);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // what was read and copied through the generic proxy comes before the bulk stores
    asm volatile("fence.proxy.async;" ::: "memory");
    if (IN_PLACE)
      pa::cluster_sync();
    else
      __syncthreads();
    if (moves) {
      if (p.ks != nullptr) {
        p.ks[to] = kx;
        p.vs[to] = vx;
      }
      if (p.mass != nullptr) p.mass_out[row * p.mo_stride + i] = mx;
    }
    // page tid of the round: its rows go out together, or one by one where some must not be written
    if (tid < T >> p.ps_shift && (moved >> tid) & 1u) {
      const int64_t slot = first + ((int64_t)tid << p.ps_shift);
      const int cnt = (int)min((int64_t)p.ps, n - slot);
      const int dp = p.dt[(int64_t)r * p.dt_stride + (slot >> p.ps_shift)];
      const int at = tid << p.ps_shift;
      if (!((odd >> tid) & 1u)) {
        const int64_t dst = ((int64_t)(dp * p.Hkv + h) << p.ps_shift) * kRow;
        bulk_store(p.k + dst, ks_at + at * kRow, cnt * kRow);
        bulk_store(p.v + dst, vs_at + at * kRow, cnt * kRow);
      } else {
        for (int t = at; t < at + cnt; ++t) {
          if (sm.from[t] < 0) continue;
          const int64_t dst = (((int64_t)(dp * p.Hkv + h) << p.ps_shift) + t - at) * kRow;
          bulk_store(p.k + dst, ks_at + t * kRow, kRow);
          bulk_store(p.v + dst, vs_at + t * kRow, kRow);
        }
      }
      asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    if (!IN_PLACE) return;
    __syncthreads();  // the tile is free again
  }
}

// Clusters of more than 8 CTAs.
template <typename Params>
bool wide_opt_in(void (*kernel)(Params)) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
}
bool move_opt_in(void (*kernel)(CompactParams)) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveBytes) == cudaSuccess && wide_opt_in(kernel);
}

// The current device's SM count, and its kernels' opt-ins, once per device; 0 for a
// device beyond those tracked, -1 when a call fails.
int evict_device() {
  static std::once_flag once[pa_host::kMaxDevices];
  static int sms[pa_host::kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev < 0 || dev >= pa_host::kMaxDevices) return 0;
  std::call_once(once[dev], [dev]() {
    int n = 0;
    const bool ok = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
                    move_opt_in(kv_compact_kernel<8, true>) && move_opt_in(kv_compact_kernel<16, true>) &&
                    move_opt_in(kv_compact_kernel<8, false>) && move_opt_in(kv_compact_kernel<16, false>) &&
                    wide_opt_in(evict_select_kernel<4>) && wide_opt_in(evict_select_kernel<16>) &&
                    wide_opt_in(evict_select_kernel<kMaxKeys>) && wide_opt_in(evict_select_kernel<0>);
    sms[dev] = ok ? n : -1;
  });
  return sms[dev];
}

}  // namespace

extern "C" pa_status_t pa_evict_select(const pa_evict_select_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_kv_heads < 1 || a->mass_stride < 1 || a->budget < 1 || a->keep_first < 0 ||
      a->keep_recent < 0 || (int64_t)a->keep_first + a->keep_recent > a->budget || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (a->num_kv_heads > pa_host::kMaxHeads || (int64_t)a->num_seqs * a->num_kv_heads > kMaxRows ||
      a->mass_stride > kMaxPositions)
    return PA_ERR_UNSUPPORTED;
  if (a->mass == nullptr || a->context_lens == nullptr || a->keep == nullptr || a->new_lens == nullptr ||
      (const int32_t *)a->new_lens == a->context_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(a->mass, 4) || !aligned(a->context_lens, 4) || !aligned(a->keep, 4) ||
      !aligned(a->new_lens, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  const uint64_t lens = (uint64_t)a->num_seqs * 4, cells = lens * a->num_kv_heads;
  const pa_host::Span mass = {a->mass, cells * a->mass_stride}, old = {a->context_lens, lens};
  const pa_host::Span keep = {a->keep, cells * a->budget}, made = {a->new_lens, lens};
  if (pa_host::overlaps(made, {old, mass, keep}) || pa_host::overlaps(keep, {old, mass})) return PA_ERR_INVALID_ARG;
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
  const int sms = evict_device();
  if (sms < 1) return sms == 0 ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
  // CTAs per row: more while each keeps 2048 positions and all run at once (two per SM), or
  // while a row's keys do not fit their registers.  16 rows x 131072: 17.3 us with 8 CTAs per row; 4 rows x
  // 1000: 4.0 us with one CTA; 1 x 4096 6.5 with two, 1 x 2048 4.2 with one and 6.3 with two.
  const int64_t rows = (int64_t)a->num_seqs * a->num_kv_heads;
  auto fits = [&](int ctas) { return a->mass_stride <= (int64_t)ctas * kSelThreads * kMaxKeys; };
  int C = 1;
  while (C < kMaxCluster && a->mass_stride / (2 * C) >= 2048 && (rows * 2 * C <= 2 * sms || !fits(C))) C *= 2;
  // 16 CTAs where each has an SM for itself (4 rows x 131072: 11.4 us against 14.4), or where the keys then
  // fit after all (1 row x 262144: 12.6 us against 43.5 with 8, 16 rows 29.5 against 43.6).
  if (C == kMaxCluster && a->mass_stride / (2 * C) >= 2048 && (rows * 2 * C <= sms || (!fits(C) && fits(2 * C)))) C *= 2;
  // The keys a warp's stretch of the longest row gives each lane.  The loops are unrolled over the keys a
  // lane can have, so fewer is faster for short rows (4 x 1000: +1.9 us with 16, +4.4 with 32), and keeping
  // them beats reading them again (16 x 131072: 17.3 us with 32, twice that re-read).
  const int64_t warps = (int64_t)C * kSelWarps;
  const int64_t keys = (((int64_t)a->mass_stride + warps - 1) / warps + 31) / 32;
  const pa_host::Launch run(dim3((unsigned)(rows * C)), dim3(kSelThreads), 0, stream, C);
  const cudaError_t e = keys <= 4          ? cudaLaunchKernelEx(run.cfg(), evict_select_kernel<4>, p)
                        : keys <= 16       ? cudaLaunchKernelEx(run.cfg(), evict_select_kernel<16>, p)
                        : keys <= kMaxKeys ? cudaLaunchKernelEx(run.cfg(), evict_select_kernel<kMaxKeys>, p)
                                           : cudaLaunchKernelEx(run.cfg(), evict_select_kernel<0>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
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
  if ((int64_t)a->num_seqs * a->num_kv_heads > kMaxRows) return PA_ERR_UNSUPPORTED;
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
    const uint64_t lens = (uint64_t)a->num_seqs * 4;
    if (pa_host::overlaps({a->mass_out, rows * a->mass_out_stride},
                          {{a->keep, rows * a->keep_stride}, {a->new_lens, lens}, {a->block_table, lens * a->block_table_stride},
                           {a->dst_block_table, in_place ? 0 : lens * a->dst_block_table_stride}}))
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
  p.keep_stride = a->keep_stride;
  p.bt_stride = a->block_table_stride;
  p.dt_stride = in_place ? a->block_table_stride : a->dst_block_table_stride;
  p.m_stride = a->mass_stride;
  p.mo_stride = a->mass_out_stride;
  const bool wide = a->kv_dtype == PA_KV_BF16;
  const int tokens = wide ? move_tokens<16>() : move_tokens<8>();
  const int64_t rows = (int64_t)a->num_seqs * a->num_kv_heads;
  const int sms = evict_device();
  if (sms < 1) return sms == 0 ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
  const int64_t rounds = ((int64_t)a->keep_stride + tokens - 1) / tokens;
  if (!in_place) {
    const pa_host::Launch run(dim3((unsigned)rounds, (unsigned)rows), dim3(kMoveThreads), kMoveBytes, stream);
    const cudaError_t e = wide ? cudaLaunchKernelEx(run.cfg(), kv_compact_kernel<16, false>, p)
                               : cudaLaunchKernelEx(run.cfg(), kv_compact_kernel<8, false>, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  // CTAs per row: more while all rows' CTAs run at once (three per SM, with room for the clusters'
  // placement: two) and there are rounds for them (8 rows x 4095: 6.5 us with 16, 8.4 with 8, 14.9 with 4)
  int C = 1;
  while (C < kMaxMoveCluster && rows * C <= sms && C < rounds) C *= 2;
  const pa_host::Launch run(dim3((unsigned)(rows * C)), dim3(kMoveThreads), kMoveBytes, stream, C);
  const cudaError_t e = wide ? cudaLaunchKernelEx(run.cfg(), kv_compact_kernel<16, true>, p)
                             : cudaLaunchKernelEx(run.cfg(), kv_compact_kernel<8, true>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
