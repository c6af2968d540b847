// pa_evict.cu -- eviction from the paged cache: pa_evict_select chooses the tokens that stay,
// pa_kv_compact moves them to the front of their pages.  See include/pa.h for the contract.
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

// Unsigned keys in the order of the masses: NaN lowest, -0 = +0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kStageKeys = 49152;  // keys a CTA can hold in shared memory (192 KB)

// A cluster of C CTAs per (request, KV head), each with one stretch of the positions.  The masses
// are read once, as keys into shared memory (rows beyond C * kStageKeys are read again instead).
// The key T of the last middle token taken is found by counting keys in 2048 bins of the
// range that still holds it: at first the range of the middle's keys (so the bins are as fine as the
// data allow, and shared-memory counters rarely collide), then one bin of the step before; three
// steps narrow 2^32 to a single key.  The CTAs' counts meet through distributed shared memory,
// one cluster barrier per step.  Then the kept positions are written in order: those above T and
// the first `need` equal to it, at offsets from the counts of the warps and CTAs before.
struct SelectShared {
  uint32_t hist[2][kBins];
  uint32_t range[2];             // this CTA's smallest and largest middle key
  int total[2];                  // this CTA's keys equal to T, and certain ones
  uint32_t wlo[kSelWarps], whi[kSelWarps];
  int weq[kSelWarps], wsure[kSelWarps], scan[kSelWarps];
  int pick[3];                   // the chosen bin, keys above it, keys in it
};

// 8 bytes at this shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint2 load_cluster(const void *p, uint32_t rank) {
  uint32_t a;
  uint2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(pa::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
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

template <bool STAGED>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) SelectShared sm;
  const int C = (int)pa::cluster_ctas(), rank = (int)pa::cluster_rank();
  const int row = blockIdx.x / C, r = row / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  // this CTA's positions, and of them the middle ones
  const int S = ((L + C - 1) / C + 31) & ~31;
  const int begin = (int)min((int64_t)rank * S, (int64_t)L), end = (int)min((int64_t)begin + S, (int64_t)L);
  const int mlo = max(begin, p.first), mhi = min(end, L - p.recent), want = p.budget - p.first - p.recent;
  const float *m = p.mass + (int64_t)row * p.stride;
  auto key_at = [&](int i) { return STAGED ? keys[i - begin] : mass_key(m[i]); };

  uint32_t T = 0xFFFFFFFFu;  // with want 0 nothing of the middle stays
  int need = 0;
  if (want > 0) {
    uint32_t klo = 0xFFFFFFFFu, khi = 0;
    for (int i0 = mlo + tid; i0 < mhi; i0 += 8 * kSelThreads) {  // eight loads in flight
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = i0 + u * kSelThreads < mhi ? m[i0 + u * kSelThreads] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kSelThreads;
        if (i >= mhi) break;
        const uint32_t k = mass_key(x[u]);
        if (STAGED) keys[i - begin] = k;
        klo = min(klo, k);
        khi = max(khi, k);
      }
    }
    klo = __reduce_min_sync(~0u, klo);
    khi = __reduce_max_sync(~0u, khi);
    if (lane == 0) {
      sm.wlo[warp] = klo;
      sm.whi[warp] = khi;
    }
    for (int b = tid; b < kBins; b += kSelThreads) sm.hist[0][b] = 0;
    __syncthreads();
    if (warp == 0) {
      klo = __reduce_min_sync(~0u, sm.wlo[lane]);
      khi = __reduce_max_sync(~0u, sm.whi[lane]);
      if (lane == 0) {
        sm.range[0] = klo;
        sm.range[1] = khi;
      }
    }
    pa::cluster_sync();
    const uint2 kr = lane < C ? load_cluster(sm.range, lane) : make_uint2(0xFFFFFFFFu, 0u);
    uint32_t base = __reduce_min_sync(~0u, kr.x);
    uint32_t span = __reduce_max_sync(~0u, kr.y) - base;  // keys in [base, base + span] are still open
    need = want;
    for (int step = 0;; ++step) {
      if (span == 0) {  // one key left: it is T, and `need` of its tokens stay
        T = base;
        break;
      }
      uint32_t *hist = sm.hist[step & 1];
      const int shift = max(0, 21 - __clz(span));  // (span >> shift) < 2048
      for (int i = mlo + tid; i < mhi; i += kSelThreads) {
        const uint32_t d = key_at(i) - base;
        if (d <= span) atomicAdd(hist + (d >> shift), 1u);
      }
      pa::cluster_sync();
      // bins 2 tid and 2 tid + 1 over the cluster; prefix sums from the top
      uint2 c = make_uint2(0u, 0u), x[kMaxCluster];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) x[q] = q < C ? load_cluster(hist + 2 * tid, q) : make_uint2(0u, 0u);
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        c.x += x[q].x;
        c.y += x[q].y;
      }
      for (int b = tid; b < kBins; b += kSelThreads) sm.hist[(step + 1) & 1][b] = 0;  // read by all a step ago
      const int mine = (int)(c.x + c.y), upto = warp_scan(mine, lane);
      if (lane == 31) sm.scan[warp] = upto;
      __syncthreads();
      const int w = sm.scan[lane], wincl = warp_scan(w, lane);
      const int all = __shfl_sync(~0u, wincl, 31), below = __shfl_sync(~0u, wincl - w, warp);
      const int above1 = all - (below + upto);  // keys in bins above 2 tid + 1
      const int above0 = above1 + (int)c.y;
      if (above1 < need && need <= above0) {
        sm.pick[0] = 2 * tid + 1;
        sm.pick[1] = above1;
        sm.pick[2] = (int)c.y;
      } else if (above0 < need && need <= above0 + (int)c.x) {
        sm.pick[0] = 2 * tid;
        sm.pick[1] = above0;
        sm.pick[2] = (int)c.x;
      }
      __syncthreads();
      base += (uint32_t)sm.pick[0] << shift;
      need -= sm.pick[1];
      if (need == sm.pick[2]) {  // the whole bin stays: everything from its lowest key on
        T = base;
        need = INT_MAX;
        break;
      }
      span = (1u << shift) - 1u;
    }
  }
  __syncthreads();

  // ---- each warp's stretch: count, then write
  const int wl = ((end - begin + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int wb = min(begin + warp * wl, end), we = min(wb + wl, end);
  auto classify = [&](int i, bool &sure, bool &eq) {
    sure = eq = false;
    if (i >= we) return;
    if (i < mlo || i >= mhi) {
      sure = true;  // not in the middle: one of the first or of the recent
    } else if (want > 0) {
      const uint32_t k = key_at(i);
      sure = k > T;
      eq = k == T;
    }
  };
  int nsure = 0, neq = 0;
  for (int i = wb + lane; i - lane < we; i += 32) {
    bool sure, eq;
    classify(i, sure, eq);
    nsure += sure;
    neq += eq;
  }
  nsure = __reduce_add_sync(~0u, nsure);
  neq = __reduce_add_sync(~0u, neq);
  if (lane == 0) {
    sm.wsure[warp] = nsure;
    sm.weq[warp] = neq;
  }
  __syncthreads();
  if (warp == 0) {
    const int e = __reduce_add_sync(~0u, sm.weq[lane]), u = __reduce_add_sync(~0u, sm.wsure[lane]);
    if (lane == 0) {
      sm.total[0] = e;
      sm.total[1] = u;
    }
  }
  pa::cluster_sync();
  const uint2 ct = lane < C ? load_cluster(sm.total, lane) : make_uint2(0u, 0u);
  pa::cluster_arrive();  // no CTA leaves before the others have read its totals
  const int ceq = (int)ct.x, ceq_before = warp_scan(ceq, lane) - ceq;
  const int ckept = (int)ct.y + ties_taken(need, ceq_before, ceq);
  const int cstart = warp_scan(ckept, lane) - ckept;
  int before = __shfl_sync(~0u, ceq_before, rank), at = __shfl_sync(~0u, cstart, rank);
  {
    const int e = sm.weq[lane], eb = before + warp_scan(e, lane) - e;
    const int kept = sm.wsure[lane] + ties_taken(need, eb, e), start = at + warp_scan(kept, lane) - kept;
    before = __shfl_sync(~0u, eb, warp);
    at = __shfl_sync(~0u, start, warp);
  }
  const unsigned lt = (1u << lane) - 1u;
  for (int i = wb + lane; i - lane < we; i += 32) {
    bool sure, eq;
    classify(i, sure, eq);
    const unsigned eqs = __ballot_sync(~0u, eq);
    const bool stays = sure || (eq && before + __popc(eqs & lt) < need);
    const unsigned st = __ballot_sync(~0u, stays);
    if (stays) keep[at + __popc(st & lt)] = i;
    at += __popc(st);
    before += __popc(eqs);
  }
  pa::cluster_wait();
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
constexpr int kMoveBytes = 65536;    // K and V rows of a CTA's round in shared memory: three CTAs per SM
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

bool move_opt_in(void (*kernel)(CompactParams)) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveBytes) == cudaSuccess &&
         cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
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
                    cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kStageKeys * (int)sizeof(uint32_t)) == cudaSuccess &&
                    move_opt_in(kv_compact_kernel<8, true>) && move_opt_in(kv_compact_kernel<16, true>) &&
                    move_opt_in(kv_compact_kernel<8, false>) && move_opt_in(kv_compact_kernel<16, false>);
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
  const int sms = evict_device();
  if (sms < 1) return sms == 0 ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
  // CTAs per row: more while each keeps 2048 positions and all run at once (one per SM), or
  // while a row's keys do not fit their shared memory
  const int64_t rows = (int64_t)a->num_seqs * a->num_kv_heads;
  int C = 1;
  while (C < kMaxCluster && a->mass_stride / (2 * C) >= 2048 &&
         (rows * 2 * C <= sms || a->mass_stride > (int64_t)C * kStageKeys))
    C *= 2;
  const int64_t stretch = ((((int64_t)a->mass_stride + C - 1) / C) + 31) & ~(int64_t)31;
  const bool staged = stretch <= kStageKeys;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = staged ? (size_t)stretch * sizeof(uint32_t) : 0;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = staged ? cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, p)
                               : cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, p);
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
  (void)cudaGetLastError();  // drop an earlier, unrelated launch error
  const bool wide = a->kv_dtype == PA_KV_BF16;
  const int tokens = wide ? move_tokens<16>() : move_tokens<8>();
  const int64_t rows = (int64_t)a->num_seqs * a->num_kv_heads;
  const int sms = evict_device();
  if (sms < 1) return sms == 0 ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
  const int64_t rounds = ((int64_t)a->keep_stride + tokens - 1) / tokens;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = kMoveBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  if (!in_place) {
    cfg.gridDim = dim3((unsigned)rounds, (unsigned)rows);
    const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, kv_compact_kernel<16, false>, p)
                               : cudaLaunchKernelEx(&cfg, kv_compact_kernel<8, false>, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  // CTAs per row: more while all rows' CTAs run at once (three per SM, with room for the clusters'
  // placement: two) and there are rounds for them
  int C = 1;
  while (C < kMaxMoveCluster && rows * C <= sms && C < rounds) C *= 2;
  cfg.gridDim = dim3((unsigned)(rows * C));
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, kv_compact_kernel<16, true>, p)
                             : cudaLaunchKernelEx(&cfg, kv_compact_kernel<8, true>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
