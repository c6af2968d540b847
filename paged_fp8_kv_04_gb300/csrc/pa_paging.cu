// pa_paging.cu -- pages of the cache for requests that grow and back from those that shrink:
// pa_page_assign and pa_page_release.  See include/pa.h for the contract.
//
// Both are a prefix sum over the requests' pages followed by work per row (a slot, a position and, where the
// row opens a page, a table entry) or per page.  Every CTA scans all the requests by itself, which costs less than an
// exchange, and takes its share of the rows.  The lengths and the count of free pages may be updated in place, so no CTA may write
// them before all have read them.  Few rows: one cluster, whose barrier tells.  Many rows: CTAs all over the GPU, and a second
// launch of one CTA for what is updated in place (32 x 8192 tokens: 16.2 us in one cluster, 4.6 so).
//
// Bound by latency: 12 bytes per row, and a chain of lengths -> scan -> page -> slot.  32 tokens 2.6 us, 262144 tokens 4.6 us, 200000
// pages given back 3.5 us (back to back; an empty kernel 1.5).
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kMaxThreads = 1024;
constexpr int kMaxCluster = 16;
constexpr int kMaxSeqs = 1 << 30;  // requests are counted in 32 bits, chunks of them ahead

struct AssignParams {
  const int32_t *L, *cu, *free_pages, *num_free;
  int32_t *bt, *num_free_out, *new_lens, *pos;
  int64_t *slots;
  uint32_t *status;
  int32_t num_pages, B, rows, bt_stride, shift, capacity;
  int32_t write_rows;  // 0: lengths and count alone; those are left to another launch where new_lens is NULL
};

struct ReleaseParams {
  const int32_t *L, *new_lens, *bt, *num_free;
  int32_t *free_pages, *num_free_out;
  uint32_t *status;
  int32_t num_pages, B, bt_stride, shift, capacity;
  int32_t write_pages;  // 0: the count alone, which is left to another launch where num_free_out is NULL
};

// This CTA's place among those that share the work: of a cluster, whose barrier they pass when they have read what may be
// updated in place, or of the grid.
template <bool WIDE>
struct Team {
  int rank = (int)blockIdx.x, ranks = (int)gridDim.x;  // (a cluster is the whole grid)
  __device__ __forceinline__ void have_read() {
    if constexpr (!WIDE) pa::cluster_arrive();
  }
  __device__ __forceinline__ void all_have_read() {
    if constexpr (!WIDE) pa::cluster_wait();
  }
};

__device__ __forceinline__ void raise(uint32_t *status, uint32_t flags) {
  if (flags != 0 && status != nullptr) atomicOr(status, flags);
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// Inclusive sum over the CTA's threads (a multiple of 32 of them); `all` becomes the total.
__device__ __forceinline__ int64_t scan(int64_t x, int64_t *sums, int64_t &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of the chunk before have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  // the warps' sums in turn, in every warp (one by one in every thread: 13.5 us, not 9.5, for 3000 requests of a token)
  int64_t y = lane < warps ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(~0u, y, o);
    if (lane >= o) y += z;
  }
  all = __shfl_sync(~0u, y, 31);
  const int64_t before = __shfl_sync(~0u, y, max(warp - 1, 0));
  return x + (warp > 0 ? before : 0);
}

// The last of at[0 .. n] that is not above x (ascending), or -1.  It is looked for at `guess` first.
__device__ __forceinline__ int find(const int32_t *at, int n, int x, int guess) {
  int lo = -1, hi = n;
  if (guess >= 0 && guess < n && at[guess] <= x && x < at[guess + 1]) return guess;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// R rows per thread and step, 32 apart: R independent chains in flight.
template <int R, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads) page_assign_kernel(const __grid_constant__ AssignParams p) {
  __shared__ int64_t sums[kMaxThreads / 32];
  __shared__ int32_t cu_s[kMaxThreads + 1], len_s[kMaxThreads], have_s[kMaxThreads], base_s[kMaxThreads];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  Team<WIDE> team;
  pa::pdl_wait();
  pa::pdl_launch_dependents();
  const int stack = min(max(*p.num_free, 0), p.capacity);
  uint32_t flags = 0;
  // The requests of a chunk, one per thread, are read a chunk ahead.
  int na = 0, nb = 0, nL = 0;
  auto read = [&](int r) {
    if (r < p.B) {
      na = p.cu[r];
      nb = p.cu[r + 1];
      nL = p.L[r];
    }
  };
  read(tid);
  // Ascending within 0 .. rows, or nobody is served: then every row has one owner at most.
  bool bad = false;
  for (int r = tid; r < p.B; r += threads) {
    const int a = p.cu[r], b = p.cu[r + 1];
    bad |= a < 0 || b < a || b > p.rows;
  }
  const bool ascends = __syncthreads_or(bad) == 0;
  if (!ascends) flags |= PA_DEV_BAD_QLEN;

  int64_t run = 0;  // pages that the requests so far have asked for
  int taken = 0;    // and what was taken
  int r0 = 0;
  do {
    const int n = min(threads, p.B - r0), r = r0 + tid;
    int L = 0, have = 0;
    int64_t need = 0;
    bool good = false;
    const int a = na, b = nb;
    if (tid < n) {
      L = nL;
      if (ascends) {
        const int64_t end = (int64_t)L + (b - a);
        good = L >= 0 && end <= INT_MAX && pages_of(end, p.shift) <= p.bt_stride;
        if (!good) flags |= PA_DEV_BAD_CONTEXT;
        if (good) {
          have = (int)pages_of(L, p.shift);
          need = pages_of(end, p.shift) - have;
        }
      }
      cu_s[tid] = a;
      if (tid == n - 1) cu_s[n] = b;
      len_s[tid] = L;
      have_s[tid] = have;
    }
    read(r + threads);
    int64_t all;
    const int64_t upto = run + scan(need, sums, all);  // synchronises the CTA
    const bool served = good && (need == 0 || upto <= stack);
    if (good && !served) flags |= PA_DEV_PAGE_POOL;
    if (tid < n) base_s[tid] = served ? (need == 0 ? 0 : (int)(upto - need)) : -1;
    team.have_read();  // this chunk's lengths
    // what was taken: the last of those served (they are the first of those that asked)
    taken = max(taken, __reduce_max_sync(~0u, served && need > 0 ? (int)upto : 0));
    run += all;
    __syncthreads();

    const bool last = r0 + threads >= p.B;
    const int lo = r0 == 0 || !ascends ? 0 : cu_s[0], hi = p.write_rows == 0 ? 0 : last || !ascends ? p.rows : cu_s[n];
    const int strip = 32 * R, warps = team.ranks * (threads >> 5);
    // (64 bits: the last strip may pass 2^31)
    for (int64_t s = lo + (int64_t)strip * (team.rank * (threads >> 5) + (tid >> 5)); s < hi && (ascends || r0 == 0);
         s += (int64_t)strip * warps) {
      int j[R], id[R], at[R];
      bool opens[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t row = s + 32 * k + lane;
        j[k] = -1;
        id[k] = -1;
        at[k] = 0;
        opens[k] = false;
        if (row < hi && ascends && p.B > 0) {
          j[k] = find(cu_s, n, (int)row, (int)row - lo);  // (a token each)
          if (j[k] >= n) j[k] = -1;
        }
        if (j[k] >= 0) {
          at[k] = (int)((uint32_t)len_s[j[k]] + (uint32_t)((int)row - cu_s[j[k]]));
          const int base = base_s[j[k]];
          if (base >= 0) {
            const int col = at[k] >> p.shift, more = col - have_s[j[k]];
            opens[k] = more >= 0 && (at[k] & ((1 << p.shift) - 1)) == 0;
            id[k] = more >= 0 ? p.free_pages[stack - 1 - (base + more)] : p.bt[(int64_t)(r0 + j[k]) * p.bt_stride + col];
          } else {
            j[k] = -1;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t row = s + 32 * k + lane;
        if (row >= hi) continue;
        if (opens[k]) p.bt[(int64_t)(r0 + j[k]) * p.bt_stride + (at[k] >> p.shift)] = id[k];
        const bool page = id[k] >= 0 && id[k] < p.num_pages;
        if (j[k] >= 0 && !page) flags |= PA_DEV_BAD_PAGE;
        p.slots[row] = !page ? -1 : ((int64_t)id[k] << p.shift) + (at[k] & ((1 << p.shift) - 1));
        if (p.pos != nullptr) p.pos[row] = at[k];
      }
    }
    team.all_have_read();  // this chunk's lengths, and the count of free pages
    if (team.rank == 0 && tid < n && p.new_lens != nullptr) p.new_lens[r] = served ? L + (b - a) : L;
    __syncthreads();  // the chunk's arrays have been read
    r0 += threads;
  } while (r0 < p.B);

  if (team.rank == 0 && p.num_free_out != nullptr) {
    __shared__ int32_t most;
    if (tid == 0) most = 0;
    __syncthreads();
    if (lane == 0 && taken > 0) atomicMax(&most, taken);
    __syncthreads();
    if (tid == 0) *p.num_free_out = stack - most;
  }
  flags = __reduce_or_sync(~0u, flags);
  if (lane == 0) raise(p.status, flags);
}

template <int R, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads) page_release_kernel(const __grid_constant__ ReleaseParams p) {
  __shared__ int64_t sums[kMaxThreads / 32];
  __shared__ int32_t from_s[kMaxThreads + 1], col_s[kMaxThreads];
  __shared__ int32_t most;
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  Team<WIDE> team;
  pa::pdl_wait();
  pa::pdl_launch_dependents();
  const int stack = min(max(*p.num_free, 0), p.capacity), room = p.capacity - stack;
  team.have_read();
  uint32_t flags = 0;
  int64_t run = 0;  // pages of the requests so far
  int given = 0;
  for (int r0 = 0; r0 < p.B; r0 += threads) {
    const int n = min(threads, p.B - r0), r = r0 + tid;
    int64_t back = 0;
    int col = 0;
    if (tid < n) {
      const int L = p.L[r], m = p.new_lens[r];
      if (L < 0 || m < 0 || pages_of(L, p.shift) > p.bt_stride) {
        flags |= PA_DEV_BAD_CONTEXT;
      } else if (m < L) {
        col = (int)pages_of(m, p.shift);
        back = pages_of(L, p.shift) - col;
      }
    }
    int64_t all;
    const int64_t upto = run + scan(back, sums, all);
    const bool fits = upto <= room;
    if (!fits && back > 0) flags |= PA_DEV_PAGE_POOL;
    // the page, of all that are given back, with which the request's begin; past the end of those that fit: none
    if (tid == 0) most = given;
    __syncthreads();
    const int mine = __reduce_max_sync(~0u, fits ? (int)upto : 0);
    if (lane == 0) atomicMax(&most, mine);
    if (tid < n) {
      from_s[tid] = (int)min(upto - back, (int64_t)INT_MAX);
      col_s[tid] = col;
    }
    __syncthreads();
    const int end = most;  // (in pages; those of this chunk begin at `given`)
    const int strip = 32 * R, warps = team.ranks * (threads >> 5);
    for (int64_t s = given + (int64_t)strip * (team.rank * (threads >> 5) + (tid >> 5)); s < end && p.write_pages != 0; s += (int64_t)strip * warps) {
      int id[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t f = s + 32 * k + lane;
        if (f < end) {
          const int j = find(from_s, n - 1, (int)f, -1);
          id[k] = p.bt[(int64_t)(r0 + j) * p.bt_stride + col_s[j] + ((int)f - from_s[j])];
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t f = s + 32 * k + lane;
        if (f >= end) continue;
        if (id[k] < 0 || id[k] >= p.num_pages) flags |= PA_DEV_BAD_PAGE;
        p.free_pages[stack + f] = id[k];
      }
    }
    given = end;
    run += all;
    __syncthreads();  // the chunk's arrays have been read
  }
  team.all_have_read();  // the count of free pages
  if (team.rank == 0 && tid == 0 && p.num_free_out != nullptr) *p.num_free_out = stack + given;
  flags = __reduce_or_sync(~0u, flags);
  if (lane == 0) raise(p.status, flags);
}

// The current device's SM count, looked up with the kernels' opt-in to clusters of 16 once per device; 0 if a call fails.
int paging_device() {
  static std::atomic<int> known[pa_host::kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= pa_host::kMaxDevices) return 0;
  if ((sms = known[dev].load(std::memory_order_acquire)) > 0) return sms;
  for (const void *f : {(const void *)page_assign_kernel<1, false>, (const void *)page_assign_kernel<4, false>,
                        (const void *)page_release_kernel<1, false>, (const void *)page_release_kernel<4, false>})
    if (cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  known[dev].store(sms, std::memory_order_release);
  return sms;
}

// CTAs, threads of each and items per thread for `items` rows or pages of `seqs` requests.
struct Shape {
  int ctas, threads, each;
  bool wide;
};
constexpr int64_t kWide = 16384;  // more items than this go to the whole GPU
Shape shape_of(int64_t items, int64_t seqs, int sms) {
  Shape s{1, kMaxThreads, 1, false};
  if (items > kWide) {
    const int64_t ctas = (items + 2047) / 2048;
    return Shape{(int)(ctas < 2 * sms ? ctas : 2 * sms), seqs <= 512 ? 512 : kMaxThreads, 4, true};
  }
  const int64_t most = items > seqs ? items : seqs;
  if (most <= 512) {
    s.threads = most <= 128 ? 128 : 512;
    return s;
  }
  while (s.ctas < kMaxCluster && (int64_t)s.ctas * kMaxThreads < items) s.ctas *= 2;
  if (items > (int64_t)s.ctas * kMaxThreads) s.each = 4;
  return s;
}

template <typename P>
cudaError_t launch(void (*one)(P), void (*four)(P), void (*wide)(P), const Shape &s, const P &p, void *stream) {
  const pa_host::Launch run(dim3((unsigned)s.ctas), dim3((unsigned)s.threads), 0, stream, s.wide ? 0 : s.ctas);
  return cudaLaunchKernelEx(run.cfg(), s.wide ? wide : s.each == 1 ? one : four, p);
}

}  // namespace

extern "C" pa_status_t pa_page_assign(const pa_page_assign_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_seqs > kMaxSeqs || a->num_rows < 0 || a->block_table_stride < 1 || a->free_capacity < 1 || a->num_pages < 1 ||
      a->num_pages > INT_MAX || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (pa_host::log2_page(a->page_size) < 0) return PA_ERR_UNSUPPORTED;
  if (a->cu_seqlens_q == nullptr || a->free_pages == nullptr || a->num_free == nullptr || a->num_free_out == nullptr ||
      (a->num_seqs > 0 && (a->context_lens == nullptr || a->block_table == nullptr || a->new_lens == nullptr)) ||
      (a->num_rows > 0 && a->slot_mapping == nullptr))
    return PA_ERR_INVALID_ARG;
  if (!aligned(a->context_lens, 4) || !aligned(a->cu_seqlens_q, 4) || !aligned(a->block_table, 4) || !aligned(a->free_pages, 4) ||
      !aligned(a->num_free, 4) || !aligned(a->num_free_out, 4) || !aligned(a->new_lens, 4) || !aligned(a->slot_mapping, 8) ||
      !aligned(a->positions, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  using pa_host::Span;
  const uint64_t lens = (uint64_t)a->num_seqs * 4, rows = (uint64_t)a->num_rows;
  const Span L{a->context_lens, lens}, cu{a->cu_seqlens_q, lens + 4}, table{a->block_table, lens * a->block_table_stride},
      pages{a->free_pages, (uint64_t)a->free_capacity * 4}, count{a->num_free, 4}, left{a->num_free_out, 4}, grown{a->new_lens, lens},
      slots{a->slot_mapping, rows * 8}, pos{a->positions, rows * 4}, none{nullptr, 0};
  if (pa_host::overlaps(table, {L, cu, pages, count, left, grown, slots, pos}) ||
      pa_host::overlaps(left, {a->num_free_out == a->num_free ? none : count, L, cu, pages, grown, slots, pos}) ||
      pa_host::overlaps(grown, {a->new_lens == a->context_lens ? none : L, cu, pages, count, slots, pos}) ||
      pa_host::overlaps(slots, {L, cu, pages, count, pos}) || pa_host::overlaps(pos, {L, cu, pages, count}))
    return PA_ERR_INVALID_ARG;
  if (a->num_seqs == 0 && a->num_rows == 0 && a->num_free_out == a->num_free) return PA_OK;
  const int sms = paging_device();
  if (sms < 1) return PA_ERR_CUDA;
  AssignParams p;
  p.L = a->context_lens;
  p.cu = a->cu_seqlens_q;
  p.free_pages = a->free_pages;
  p.num_free = a->num_free;
  p.bt = a->block_table;
  p.num_free_out = a->num_free_out;
  p.new_lens = a->new_lens;
  p.pos = a->positions;
  p.slots = a->slot_mapping;
  p.status = a->status;
  p.num_pages = (int32_t)a->num_pages;
  p.B = a->num_seqs;
  p.rows = a->num_rows;
  p.bt_stride = a->block_table_stride;
  p.shift = pa_host::log2_page(a->page_size);
  p.capacity = a->free_capacity;
  p.write_rows = 1;
  const Shape s = shape_of(a->num_rows, a->num_seqs, sms);
  const bool later = s.wide && (a->num_free_out == a->num_free || a->new_lens == a->context_lens);  // no cluster: a launch of its own
  if (later) {
    p.new_lens = nullptr;
    p.num_free_out = nullptr;
  }
  cudaError_t e = launch(page_assign_kernel<1, false>, page_assign_kernel<4, false>, page_assign_kernel<4, true>, s, p, stream);
  if (later && e == cudaSuccess) {
    p.new_lens = a->new_lens;
    p.num_free_out = a->num_free_out;
    p.write_rows = 0;
    e = launch(page_assign_kernel<1, false>, page_assign_kernel<4, false>, page_assign_kernel<4, true>, shape_of(0, a->num_seqs, sms), p, stream);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status_t pa_page_release(const pa_page_release_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_seqs > kMaxSeqs || a->block_table_stride < 1 || a->free_capacity < 1 || a->num_pages < 1 || a->num_pages > INT_MAX ||
      a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (pa_host::log2_page(a->page_size) < 0) return PA_ERR_UNSUPPORTED;
  if (a->free_pages == nullptr || a->num_free == nullptr || a->num_free_out == nullptr ||
      (a->num_seqs > 0 && (a->context_lens == nullptr || a->new_lens == nullptr || a->block_table == nullptr)))
    return PA_ERR_INVALID_ARG;
  if (!aligned(a->context_lens, 4) || !aligned(a->new_lens, 4) || !aligned(a->block_table, 4) || !aligned(a->free_pages, 4) ||
      !aligned(a->num_free, 4) || !aligned(a->num_free_out, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  using pa_host::Span;
  const uint64_t lens = (uint64_t)a->num_seqs * 4;
  const Span L{a->context_lens, lens}, grown{a->new_lens, lens}, table{a->block_table, lens * a->block_table_stride},
      pages{a->free_pages, (uint64_t)a->free_capacity * 4}, count{a->num_free, 4}, left{a->num_free_out, 4}, none{nullptr, 0};
  if (pa_host::overlaps(pages, {L, grown, table, count, left}) ||
      pa_host::overlaps(left, {a->num_free_out == a->num_free ? none : count, L, grown, table}))
    return PA_ERR_INVALID_ARG;
  if (a->num_seqs == 0 && a->num_free_out == a->num_free) return PA_OK;
  const int sms = paging_device();
  if (sms < 1) return PA_ERR_CUDA;
  ReleaseParams p;
  p.L = a->context_lens;
  p.new_lens = a->new_lens;
  p.bt = a->block_table;
  p.num_free = a->num_free;
  p.free_pages = a->free_pages;
  p.num_free_out = a->num_free_out;
  p.status = a->status;
  p.num_pages = (int32_t)a->num_pages;
  p.B = a->num_seqs;
  p.bt_stride = a->block_table_stride;
  p.shift = pa_host::log2_page(a->page_size);
  p.capacity = a->free_capacity;
  // how many pages come back is not known here: what the tables and the stack can hold
  const int64_t table_pages = (int64_t)a->num_seqs * a->block_table_stride;
  p.write_pages = 1;
  const Shape s = shape_of(table_pages < a->free_capacity ? table_pages : a->free_capacity, a->num_seqs, sms);
  const bool later = s.wide && a->num_free_out == a->num_free;
  if (later) p.num_free_out = nullptr;
  cudaError_t e = launch(page_release_kernel<1, false>, page_release_kernel<4, false>, page_release_kernel<4, true>, s, p, stream);
  if (later && e == cudaSuccess) {
    p.num_free_out = a->num_free_out;
    p.write_pages = 0;
    e = launch(page_release_kernel<1, false>, page_release_kernel<4, false>, page_release_kernel<4, true>, shape_of(0, a->num_seqs, sms), p, stream);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
