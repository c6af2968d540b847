// pa_prompt.cu -- causal attention over whole packed prompts: pa_prompt_attn.  See include/pa.h for
// the contract.
//
//   S = Q K^T        tcgen05.mma kind::f16, M = 128 rows, N = 128 keys, both operands from shared memory as TMA left
//                    them (K-major, 128-byte swizzle)
//   P = 2^(c S - m)  a thread per row: TMEM lane = row.  c = sm_scale log2 e; m follows the row's maximum, but only
//                    when it has grown by more than 2^8: until then the weights exceed 1 by that much at most, and nothing
//                    has to be scaled again.  The sum of the weights is fp32, taken before they are rounded
//   O += P V         kind::f16 with P as the A operand in TMEM, in the columns that S had (bf16 because V is: a
//                    rounding of 2^-8 of a weight at most, as that of the output), V as the B operand, MN-major, as TMA left it
//
// Rows of a tile are (token, head of the group) pairs, 128 / group_size tokens with all query heads of a KV head: they
// share its keys, short prompts fill a tile as well as long ones do, and the diagonal cuts few tokens.  A CTA has two tiles (a unit),
// so that the tensor core works on one while the other's weights are computed: PV0 S0' | PV1 S1' | ...  Where there are fewer units
// than SMs a unit's tiles go to a CTA each, and its two slots take the even and the odd blocks of keys.  Of many short sequences
// a CTA takes several units, claimed from the launch queue, whose first scores are there when the rows of the one before are written.
//
// Warp roles (384 threads): warps 0-3 and 4-7 are the softmax of slots 0 and 1; warp 8 finds the units and fetches tiles by TMA; one
// lane of warp 9 issues the MMAs; warps 10 and 11 look through the values of the blocks that the diagonal or the sequence's end cuts: an
// infinity or NaN there must not reach rows that do not attend it (0 * inf), so it is replaced by 0, and rows that do attend it
// get it in the epilogue.  Every wait for a barrier in memory is bounded; warps that gave up still come to the named barriers that they
// share with others (agreed, unit_comes), so that nobody stays there.  TMEM is released on every path.
//
// Bound by the tensor core at what its power allows: 2600 cycles for two tiles and a block (16.8 MFLOP), of 2054 that the MMAs take
// on constant data, hardly fewer with the softmax left out (2520), and a cuBLAS product of 8192^3 comes to the same rate.  32768
// tokens x 16 heads 2360 to 2420 us in a few calls (1.81 to 1.86 PFLOP/s; cuBLAS 1.89), 2600 in a loop of seconds (1.69; cuBLAS 1.70),
// 16384 605 us in a few; shorter ones by what a CTA takes beside its blocks (some 5 us alone, 2 to 3 between units of one CTA) and by SMs
// that are done early: 2048 tokens 21 us, 13 prompts of 200 .. 4001 tokens x 4 KV heads 200 us in a few calls (0.79 of the rate) and 214
// to 227 in a loop, 300 of 100 tokens x 16 heads 64 us (36 by its bytes), 16 tokens 6.2 us.
// These are of the kernel as it stands; comparisons, here and beside the code, of the step that they decided.
// Measured on the way: one warp per tile to issue the MMAs 821 us, not 738, for 16384 tokens (both tiles' softmax at once); weights
// worked out with the maximum so far while the block's own is found 637, not 597; keys split over a cluster of two CTAs and joined
// through shared memory 23.4 us, not 21, for 2048 tokens.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

using pa_host::aligned;

constexpr int kD = pa_host::kD;
constexpr int kM = 128;           // rows of a tile
constexpr int kN = 128;           // keys of a block
constexpr int kSoftWarps = 8;     // four per tile
constexpr int kThreads = 384;
constexpr int kRegs = 168;        // per thread at launch: 384 * 168 = 256 * 216 + 128 * 72
constexpr int kMaxSeqs = 4096;
constexpr int kMaxGroup = 64;
constexpr int kMaxRows = 1 << 24;
constexpr int kOperand = kM * kD * 2;  // bytes of a tile or block: two halves of 64 elements a row
constexpr int kMaxStages = 5;     // blocks of keys and values in flight
// One unit to a CTA: five.  CTAs that go on with further units: four, and room for outputs on their way while the next unit's
// queries come in.
template <bool LOOP>
constexpr int kStages = LOOP ? 4 : kMaxStages;
constexpr int kMinSplit = 1;      // blocks that a unit has more than to be split into its tiles (3: 512 tokens x 16 heads 9.9 us, not 8.9)
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;     // log2 of what the weights may exceed 1 by

struct PromptParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_o;  // tm_o: a bf16 output, in boxes like the queries'

  const int32_t *cu;
  const uint16_t *v;  // for the epilogue of values that are not finite
  void *out;
  float *lse;
  uint32_t *status;
  int64_t v_stride;
  int32_t B, T, Hkv, G, tokens;  // tokens of a tile
  int32_t out_f32;
  int32_t sms;
  int32_t first_split, aside;  // the first unit index that may be split; blocks' worth of units that a CTA takes beside its keys
  uint64_t per_span;           // ceil(2^40 / (2 tokens)): x / (2 tokens) = x per_span / 2^40 for x < 2^25
  float fold;  // sm_scale * log2 e
};

// Shared memory: two query tiles, the ring of K and V blocks (and with LOOP 16 KB of either tile's output), barriers and the
// schedule's scratch.
constexpr int kRing = 2 * kOperand, kOut = kRing + kStages<true> * kOperand;
constexpr int kBars = kRing + kMaxStages * kOperand;
static_assert(kOut + kOperand <= kBars, "the outputs on their way lie in place of a stage");
enum {
  B_QFULL = 0,                      // [2] the tile's queries have landed
  B_QFREE = B_QFULL + 2,            // [2] the tile's last S is complete
  B_FULL = B_QFREE + 2,             // [stages]
  B_EMPTY = B_FULL + kMaxStages,    // [stages]
  B_S = B_EMPTY + kMaxStages,       // [2] S is complete
  B_P = B_S + 2,                    // [2][2] half of P is in TMEM (and O scaled)
  B_O = B_P + 4,                    // [2] PV is complete
  B_CUT = B_O + 2,                  // [2] the values of the unit's first or second cut block have landed
  B_CLEAN = B_CUT + 2,              // [2] and been looked through
  B_UNIT = B_CLEAN + 2,             // [4] the unit has been found
  B_LEFT = B_UNIT + 4,              // [4] every warp that the unit was found for is done with it
  B_CLAIM = B_LEFT + 4,             // the answer of the launch queue
  B_END = B_CLAIM + 1,              // the load warp posts no more units
  B_DONE = B_END + 1,               // the softmax warps are done with TMEM
  B_MMA = B_DONE + 1,               // every MMA is complete
  kNumBars = B_MMA + 1
};
constexpr int kMisc = (kBars + 8 * kNumBars + 15) / 16 * 16;  // TMEM address, padding, a sequence
constexpr int kDirty = kMisc + 16;           // [4 units][2 warps] dirty blocks
constexpr int kClaim = kDirty + 32;          // the launch queue's answer
constexpr int kPosted = kClaim + 16;         // [4] units
constexpr int kRed = kPosted + 4 * 48;       // [2][warps] of the schedule's sums
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr int kSmem = kRed + 2 * 4 * (kThreads / 32) + 1024;
// Both slots' maxima and sums of a tile that has two, [2][128] each: over the second tile's queries, or (LOOP) the outputs.
template <bool LOOP>
constexpr int kBoth = LOOP ? kOut : kOperand;

// TMEM columns: S of tile t at 128 t, O at 256 + 128 t; P over S.  The CTA has all of them, so they begin at 0.
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr uint32_t idesc(int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// The wait for the loads so far, of which these 32 registers are defined only now.
__device__ __forceinline__ void tmem_wait32(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
      : "memory");
}
// 16 columns
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's stores have read their rows, or are complete.
__device__ __forceinline__ void bulk_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_write_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void raise(const PromptParams &p, uint32_t flag) {
  if (p.status != nullptr) atomicOr(p.status, flag);
}

// A bounded wait by a whole warp: false for all lanes if it gave up for one.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(~0u, pa::mbar_wait_bounded(bar, parity)) != 0;
}

// A CTA's share, all keys of up to two tiles of a sequence and KV head.  It has two slots, each with its softmax warps and its
// columns of TMEM: one for either tile, or (solo) both for one tile, with the even and the odd blocks of its keys.
struct Unit {
  int row0, len, h;        // the sequence's first row and length, the KV head
  int tok0, tok1;          // the first token of either slot's tile
  int nb0, nb1;            // either slot's key blocks (0: no tokens)
  int blocks, cut;         // key blocks in all, and the first that the diagonal cuts: two of them at most, since a unit has
                           // 256 tokens and begins with a block, or has 128 or fewer
  bool solo;
  __device__ __forceinline__ int nb(int t) const { return t ? nb1 : nb0; }
  __device__ __forceinline__ int tok(int t) const { return t ? tok1 : tok0; }
  __device__ __forceinline__ int block(int t, int j) const { return solo ? 2 * j + t : j; }  // a slot's j-th
};

// What the units before this one have used, in phases of the barriers.
struct Past {
  int ring = 0;              // blocks of keys and values
  int units = 0, q0 = 0, q1 = 0, b0 = 0, b1 = 0;  // units, of either tile units with queries of it, of either slot key blocks
  int cut1 = 0;              // units with a second cut block (all have a first one)
  __device__ __forceinline__ int q(int t) const { return t ? q1 : q0; }
  __device__ __forceinline__ int b(int t) const { return t ? b1 : b0; }
  __device__ __forceinline__ int cut(int k) const { return k ? cut1 : units; }
  __device__ __forceinline__ void add(const Unit &u) {
    ring += 2 * u.blocks;
    units += 1;
    q0 += u.nb0 > 0;
    q1 += u.nb1 > 0 && !u.solo;
    b0 += u.nb0;
    b1 += u.nb1;
    cut1 += u.blocks > u.cut + 1;
  }
};

// ---------------------------------------------------------------------------- schedule

// The sum over the CTA's threads, or their maximum, in all of them.  `turn` alternates between calls.
__device__ __forceinline__ int reduce_all(int v, bool most, int *red, int turn) {
  const int warp = threadIdx.x >> 5;
  v = most ? __reduce_max_sync(~0u, v) : __reduce_add_sync(~0u, v);
  if ((threadIdx.x & 31) == 0) red[turn * (kThreads / 32) + warp] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int x = red[turn * (kThreads / 32) + w];
    all = most ? max(all, x) : all + x;
  }
  return all;
}

// The units of the call, those with the most keys first: unit j of a sequence has j + 1 times the keys of its first, and the GPU's
// last CTAs should be short ones.  Units of index c or more number N(c) for one KV head, the sum of max(0, n_s - c) over the
// sequences: the x-th unit's index is the largest c with N(c) > x, and it belongs to the (x - N(c + 1))-th of the sequences that
// have such a unit.
// OWN sequences to each thread: of a warp by itself, up to 32 OWN sequences, or (ALL) of the CTA, which every call synchronises.
//
// While there are SMs without a unit the longest units are split into their two tiles, a CTA each, which takes half the time: its
// keys are dealt to both slots.  So many more may be split that the shortest units come last, to the SMs that are done first: of units
// of 1, 2, ... n times the same keys, s = (2 SMs - units - what a CTA takes beside its keys, about 4 blocks) / 3 makes the longest
// whole one and two short ones in turn take the same time.  Not more of them than there are units below a third of the longest's
// index.  (2048 tokens x 16 heads: 22.6 us, 24.1 with as many as there are idle SMs, 26.5 without; 1024: 12.5, 15.8 without.)
template <int OWN, bool ALL>
struct Schedule {
  const PromptParams &p;
  uint8_t *smem;
  int n[OWN];  // units of each sequence
  int total, units, splits = 0, turn = 0;  // units for one head and for all

  __device__ __forceinline__ Schedule(const PromptParams &params, uint8_t *shared) : p(params), smem(shared) {}

  __device__ __forceinline__ int reduce(int v, bool most) {
    if constexpr (!ALL) return most ? __reduce_max_sync(~0u, v) : __reduce_add_sync(~0u, v);
    turn ^= 1;
    return reduce_all(v, most, reinterpret_cast<int *>(smem + kRed), turn);
  }
  // N(c), for one head
  __device__ __forceinline__ int from(int c) {
    int v = 0;
#pragma unroll
    for (int i = 0; i < OWN; ++i) v += max(0, n[i] - c);
    return reduce(v, false);
  }
  __device__ __forceinline__ int longest() {
    int top = 0;
#pragma unroll
    for (int i = 0; i < OWN; ++i) top = max(top, n[i]);
    return reduce(top, true);
  }

  __device__ __forceinline__ void start() {
    const int tid = threadIdx.x, lane = tid & 31, span = 2 * p.tokens;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int s = ALL ? tid + i * kThreads : lane + 32 * i;
      n[i] = 0;
      if (s < p.B) {
        const int a = p.cu[s], b = p.cu[s + 1];
        if (a < 0 || b < a || b > p.T)
          bad = true;
        else
          n[i] = (int)(((uint64_t)(b - a + span - 1) * p.per_span) >> 40);
      }
    }
    if (bad && blockIdx.x == 0) raise(p, PA_DEV_BAD_QLEN);
    total = from(0);
    units = total * p.Hkv;
    if (units > 0 && units < 2 * p.sms) {
      const int few = longest() / 3;
      const int longer = from(p.first_split) * p.Hkv, rest = from(few) * p.Hkv;  // that may be split; but the shortest
      const int idle = p.sms - units, even = (p.sms + idle - p.aside) / 3;
      splits = max(0, min(longer, max(idle, min(even, p.sms - rest))));
    }
  }

  // The x-th share: false if there are fewer, or it is an empty tile.
  __device__ __forceinline__ bool find(int x, Unit &u) {
    const int tid = threadIdx.x, lane = tid & 31, span = 2 * p.tokens;
    const int tile = x < 2 * splits ? x & 1 : -1;
    x = x < 2 * splits ? x >> 1 : x - splits;
    if (x >= units) return false;
    u.h = p.Hkv == 1 ? 0 : x % p.Hkv;
    x = p.Hkv == 1 ? x : x / p.Hkv;
    int lo = 0, above = 0;  // N(lo) > x >= above = N(hi)
    if (p.B == 1) {
      lo = total - 1 - x;
      above = x;
    } else {
      int hi = longest();
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, count = from(mid);
        if (count > x) {
          lo = mid;
        } else {
          hi = mid;
          above = count;
        }
      }
    }
    // the (x - above)-th of those with more than lo units
    int s = 0;
    if constexpr (!ALL) {
      int k = x - above;
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const uint32_t have = __ballot_sync(~0u, n[i] > lo);
        const uint32_t it = __ballot_sync(~0u, n[i] > lo && __popc(have & ((1u << lane) - 1u)) == k);
        if (it != 0) s = 32 * i + __ffs(it) - 1;
        k -= __popc(have);
      }
    } else {  // thread by thread
      int *red = reinterpret_cast<int *>(smem + kRed);
      volatile int *found = reinterpret_cast<volatile int *>(smem + kMisc + 8);
      int mine = 0;
#pragma unroll
      for (int i = 0; i < OWN; ++i) mine += n[i] > lo;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();  // the last sum has been read
      if (lane == 31) red[tid >> 5] = upto;
      __syncthreads();
      for (int w = 0; w < (tid >> 5); ++w) upto += red[w];
      int at = x - above - (upto - mine);
      if (at >= 0 && at < mine) {
#pragma unroll
        for (int i = 0; i < OWN; ++i)
          if (n[i] > lo && at-- == 0) *found = tid + i * kThreads;
      }
      __syncthreads();
      s = *found;
    }
    u.row0 = p.cu[s];
    u.len = p.cu[s + 1] - u.row0;
    auto blocks_of = [&](int first) { return first < u.len ? (min(u.len, first + p.tokens) + kN - 1) / kN : 0; };
    u.cut = lo * span / kN;
    u.solo = tile >= 0;
    if (u.solo) {
      u.tok0 = u.tok1 = lo * span + tile * p.tokens;
      u.blocks = blocks_of(u.tok0);
      u.nb0 = (u.blocks + 1) >> 1;
      u.nb1 = u.blocks >> 1;
    } else {
      u.tok0 = lo * span;
      u.tok1 = u.tok0 + p.tokens;
      u.nb0 = blocks_of(u.tok0);
      u.nb1 = blocks_of(u.tok1);
      u.blocks = max(u.nb0, u.nb1);
    }
    return u.blocks > 0;  // (a sequence's last unit may have but one tile)
  }
};

// The next CTA of the grid that has not been launched yet, to be run by this one in its place: asked for by one thread, the answer
// is there when the barrier's phase is complete.  Its index, or -1 if there is none left.
__device__ __forceinline__ void claim_next(uint32_t answer, uint32_t bar) {
  pa::mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer), "r"(bar) : "memory");
}
__device__ __forceinline__ int claimed(uint32_t answer) {
  uint32_t x, any;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\tld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\tselp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
      : "=r"(x), "=r"(any)
      : "r"(answer)
      : "memory");
  return any ? (int)x : -1;
}

// The units that the load warp has found for the others: a place for each of the last four, and two barriers: found, and left by all.
// (A slot without a tile of its own runs ahead of the other, or lags behind it, by any number of units.)
struct Slot {
  int row0, len, h, tok0, tok1, nb0, nb1, blocks, cut, solo, pad[2];
};
constexpr int kUnits = 4;
__device__ __forceinline__ void post_unit(uint8_t *smem, int round, const Unit &u, bool some) {
  Slot *s = reinterpret_cast<Slot *>(smem + kPosted) + (round & (kUnits - 1));
  *s = Slot{u.row0, u.len, u.h, u.tok0, u.tok1, u.nb0, u.nb1, some ? u.blocks : 0, u.cut, (int)u.solo, {0, 0}};
}
__device__ __forceinline__ bool posted_unit(const uint8_t *smem, int round, Unit &u) {
  const Slot s = reinterpret_cast<const Slot *>(smem + kPosted)[round & (kUnits - 1)];
  u = Unit{s.row0, s.len, s.h, s.tok0, s.tok1, s.nb0, s.nb1, s.blocks, s.cut, s.solo != 0};
  return s.blocks > 0;
}

// Whether the load warp posts that unit, for a whole warp that has given up: posted, or the load warp has ended without.  The answer is that
// of the warps that have seen the unit come: warps of a unit meet at named barriers, which know no time.  All waits of the load warp are
// bounded, and it fails at the first that others do not serve any more.
__device__ __forceinline__ bool unit_comes(uint32_t bars, int round) {
  const long long t0 = clock64();
  bool ended, comes;
  do {
    ended = __all_sync(~0u, pa::mbar_try_wait(bars + 8 * B_END, 0));
    comes = __all_sync(~0u, pa::mbar_try_wait(bars + 8 * (B_UNIT + (round & (kUnits - 1))), (round / kUnits) & 1));
  } while (!ended && !comes && !__any_sync(~0u, clock64() - t0 > 8 * pa::kWaitCycles));
  return comes;
}

// ------------------------------------------------------------------------------- roles

__device__ __forceinline__ uint32_t bar_full(uint32_t bars, int stage) { return bars + 8 * (B_FULL + stage); }

// Block i of the unit (keys and values in turn) into its place of the ring, by one thread.
template <int STAGES>
__device__ __forceinline__ void load_block(const PromptParams &p, const Unit &u, int ring, uint32_t base, uint32_t bars, int i) {
  const int stage = (ring + i) % STAGES;
  const uint32_t bar = bar_full(bars, stage), dst = base + kRing + stage * kOperand;
  pa::mbar_arrive_expect_tx(bar, kOperand);
  for (int x = 0; x < 2; ++x)
    tma_load_3d(dst + x * (kOperand / 2), i & 1 ? &p.tm_v : &p.tm_k, 64 * x, u.h, u.row0 + (i >> 1) * kN, bar);
}
__device__ __forceinline__ void load_queries(const PromptParams &p, const Unit &u, int t, uint32_t base, uint32_t bars) {
  pa::mbar_arrive_expect_tx(bars + 8 * (B_QFULL + t), (uint32_t)p.G * p.tokens * kD * 2);
  for (int x = 0; x < 2; ++x)
    tma_load_3d(base + t * kOperand + x * (kOperand / 2), &p.tm_q, 64 * x, u.h * p.G, u.row0 + u.tok(t), bars + 8 * (B_QFULL + t));
}

// The loads of a unit, in the order of their use: as many blocks as the ring holds do not wait for anything in the first unit.
// `done` counts what has been asked for.
struct Loads {
  int blocks = 0, q0 = 0, q1 = 0, claims = 0;
};
template <int STAGES>
__device__ bool load_unit(const PromptParams &p, const Unit &u, const Past &past, uint32_t base, uint32_t bars, Loads &done) {
  const int lane = threadIdx.x & 31, tiles = u.solo ? 1 : 2;
  auto block = [&](int i) {
    const int e = past.ring + i;
    if (e >= STAGES && !warp_wait(bars + 8 * (B_EMPTY + e % STAGES), (e / STAGES - 1) & 1)) return false;
    if (lane == 0) load_block<STAGES>(p, u, past.ring, base, bars, i);
    __syncwarp();
    ++done.blocks;
    return true;
  };
  for (int t = 0; t < tiles; ++t) {
    if (u.nb(t) > 0) {
      if (past.q(t) > 0 && !warp_wait(bars + 8 * (B_QFREE + t), (past.q(t) - 1) & 1)) return false;
      if (lane == 0) load_queries(p, u, t, base, bars);
      __syncwarp();
      ++(t ? done.q1 : done.q0);
    }
    if (t == 0 && !block(0)) return false;
  }
  for (int i = 1; i < 2 * u.blocks; ++i)
    if (!block(i)) return false;
  return true;
}

// Copies in flight land before the CTA can exit: what a load warp that gave up may have left.
template <int STAGES>
__device__ void drain(uint32_t bars, const Loads &done) {
  for (int e = max(0, done.blocks - STAGES); e < done.blocks; ++e) pa::mbar_wait_bounded(bar_full(bars, e % STAGES), (e / STAGES) & 1);
  if (done.q0 > 0) pa::mbar_wait_bounded(bars + 8 * B_QFULL, (done.q0 - 1) & 1);
  if (done.q1 > 0) pa::mbar_wait_bounded(bars + 8 * (B_QFULL + 1), (done.q1 - 1) & 1);
  if (done.claims > 0) pa::mbar_wait_bounded(bars + 8 * B_CLAIM, (done.claims - 1) & 1);
}

// A bounded wait of a whole warp whose control flow stays uniform: what the MMAs' operands are computed from then stays
// in uniform registers, where the instructions want them.
__device__ __forceinline__ bool uniform_wait(uint32_t bar, uint32_t parity) {
  if (__all_sync(~0u, pa::mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(~0u, pa::mbar_try_wait(bar, parity)))
    if (__any_sync(~0u, clock64() - t0 > pa::kWaitCycles)) return false;
  return true;
}

// D (+)= A B with the low words of the shared-memory descriptors, whose high words are the same for all: 1024 bytes between
// groups of 8 rows, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__host__ __device__ constexpr uint32_t desc_low(uint32_t lead) { return (lead >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accumulate), "r"(kDescHigh));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accumulate), "r"(kDescHigh));
}

// What the MMA warp needs of a unit, in uniform registers.
struct Work {
  int nb0, nb1, cut, ring, units, cut1;
  int uses[4];  // units before it with queries of either tile, blocks before it of either slot
  bool solo;
  __device__ __forceinline__ void set(const Unit &u, const Past &past) {
    nb0 = __reduce_max_sync(~0u, u.nb0);
    nb1 = __reduce_max_sync(~0u, u.nb1);
    cut = __reduce_max_sync(~0u, u.cut);
    ring = __reduce_max_sync(~0u, past.ring);
    units = __reduce_max_sync(~0u, past.units);
    cut1 = __reduce_max_sync(~0u, past.cut1);
    uses[0] = __reduce_max_sync(~0u, past.q0);
    uses[1] = __reduce_max_sync(~0u, past.q1);
    uses[2] = __reduce_max_sync(~0u, past.b0);
    uses[3] = __reduce_max_sync(~0u, past.b1);
    solo = __any_sync(~0u, u.solo);
  }
  __device__ __forceinline__ int nb(int t) const { return t ? nb1 : nb0; }
  __device__ __forceinline__ int block(int t, int j) const { return solo ? 2 * j + t : j; }
  __device__ __forceinline__ bool last_of(int t, int j) const { return solo || t == 1 || j >= nb1; }  // the slot that reads a block last
};

// The MMAs of a unit, both slots: PV0 S0' PV1 S1' of every block, S' being the slot's next one's.  The waits for what the next
// product reads come half way through the one before, where the tensor core has MMAs left (before them instead: 620 us, not 613,
// for 16384 tokens x 16 heads).
template <int STAGES>
__device__ bool issue_mmas(const Work &w, uint32_t base, uint32_t bars) {
  // (14 bits of the address)
  const uint32_t q_at = (base >> 4) & 0x3FFFu, ring_at = q_at + (kRing >> 4);
  const uint32_t q_low = q_at | desc_low(1024), k_low = ring_at | desc_low(1024), v_low = ring_at | desc_low(kOperand / 2);
  auto arrived = [&](int bar, int phase) { return uniform_wait(bars + 8 * bar, (uint32_t)phase & 1u); };
  auto fetched = [&](const Work &w, int i) {  // block i of the unit's (keys and values in turn) has landed
    const int e = w.ring + i;
    if (!arrived(B_FULL + e % STAGES, e / STAGES)) return false;
    const int k = (i >> 1) - w.cut;
    if ((i & 1) != 0 && k >= 0) {  // values to be looked through
      if (pa::elect_one()) pa::mbar_arrive(bars + 8 * (B_CUT + k));
      __syncwarp();
    }
    return true;
  };
  auto scores = [&](const Work &w, int t, int j, bool values) {  // S of the slot's j-th block; `values`: half way through, those have landed
    const int i = 2 * w.block(t, j), stage = (w.ring + i) % STAGES;
    const uint32_t q = q_low + (w.solo ? 0 : t) * (kOperand >> 4), k = k_low + stage * (kOperand >> 4);
    if (pa::elect_one()) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t off = (32 * x) >> 4;
        mma_ss(128 * t, q + off, k + off, idesc(0), x > 0);
      }
    }
    __syncwarp();
    const bool ok = !values || fetched(w, i + 1);
    if (pa::elect_one()) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t off = (kOperand / 2 + 32 * x) >> 4;
        mma_ss(128 * t, q + off, k + off, idesc(0), 1);
      }
      pa::umma_commit(bars + 8 * (B_S + t));
      if (w.last_of(t, j)) pa::umma_commit(bars + 8 * (B_EMPTY + stage));
      // the last S that reads a tile's queries: either slot's own, or (solo) the last block's of both
      if (w.solo ? i + 2 == 2 * (w.nb0 + w.nb1) : j + 1 == w.nb(t)) pa::umma_commit(bars + 8 * (B_QFREE + (w.solo ? 0 : t)));
    }
    __syncwarp();
    return ok;
  };
  auto begin = [&](const Work &w) {
    if (!arrived(B_QFULL, w.uses[0]) || !fetched(w, 0)) return false;
    pa::tc_fence_after();
    scores(w, 0, 0, false);
    return true;
  };
  if (w.nb0 > 0 && !begin(w)) return false;
  if (w.nb1 > 0) {
    if (w.solo ? !fetched(w, 2) : !arrived(B_QFULL + 1, w.uses[1])) return false;
    pa::tc_fence_after();
    scores(w, 1, 0, false);
  }
  if (!fetched(w, 1) || (w.solo && w.nb1 > 0 && !fetched(w, 3))) return false;
  const int blocks = max(w.nb0, w.nb1);
  for (int j = 0; j < blocks; ++j) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int nb = w.nb(t), b = w.block(t, j), stage = (w.ring + 2 * b + 1) % STAGES;
      if (j >= nb) continue;
      if (b >= w.cut && (w.solo || t == 0 || j >= w.nb0) && !arrived(B_CLEAN + b - w.cut, b > w.cut ? w.cut1 : w.units)) return false;
      const uint32_t v = v_low + stage * (kOperand >> 4);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!arrived(B_P + 2 * t + half, w.uses[2 + t] + j)) return false;
        pa::tc_fence_after();
        if (pa::elect_one()) {
#pragma unroll
          for (int x = 4 * half; x < 4 * half + 4; ++x)  // 16 keys: two groups of 8 rows; the two halves of head_dim 16 KB apart
            mma_ts(256 + 128 * t, 128 * t + 8 * x, v + x * (2048 >> 4), idesc(1), j > 0 || x > 0);
          if (half == 1) {
            pa::umma_commit(bars + 8 * (B_O + t));
            if (w.last_of(t, j)) pa::umma_commit(bars + 8 * (B_EMPTY + stage));
          }
        }
        __syncwarp();
        // the next block's keys: of either slot's, or the same for both
        const bool another = w.solo || t == 1 ? j + 1 < nb : j + 1 < blocks;
        if (half == 0 && another && (w.solo || t == 0 || j >= w.nb0) && !fetched(w, 2 * w.block(t, j + 1))) return false;
      }
      // over P of this block, which the product before reads: a thread's MMAs run in order
      if (j + 1 < nb && !scores(w, t, j + 1, w.last_of(t, j + 1))) return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7F80u) == 0x7F80u; }

// Whether one of the eight bf16 values of w is an infinity or NaN: an exponent of ones carries into the sign's place.
__device__ __forceinline__ uint32_t any_not_finite(const uint4 &w) {
  constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
  return (((w.x & kExp) + kOne) | ((w.y & kExp) + kOne) | ((w.z & kExp) + kOne) | ((w.w & kExp) + kOne)) & 0x80008000u;
}

// Values of the unit's blocks that the diagonal or the sequence's end cuts.
template <int STAGES>
__device__ bool clean_unit(const Unit &u, const Past &past, uint32_t bars, uint8_t *smem) {
  constexpr int kBatch = 8;
  const int lane = threadIdx.x & 31, half = (threadIdx.x >> 5) - kCleanWarp;
  uint32_t dirty = 0;
  for (int j = u.cut; j < u.blocks; ++j) {
    // In the first unit a stage's first use: its barrier has one phase until these values have been looked through.  Else the
    // MMA warp tells; and it is waited for there too, afterwards, since a wait knows a phase from the next one alone.
    const int e = past.ring + 2 * j + 1;
    const bool first = past.units == 0 && e < STAGES;
    const uint32_t told = bars + 8 * (B_CUT + j - u.cut), phase = past.cut(j - u.cut) & 1;
    if (!(first ? warp_wait(bar_full(bars, e), 0) : warp_wait(told, phase))) return false;
    uint4 *at = reinterpret_cast<uint4 *>(smem + kRing + (e % STAGES) * kOperand + half * (kOperand / 2)) + lane;
    bool own = false;  // one of the sequence's own
#pragma unroll 1
    for (int c0 = 0; c0 < kOperand / 32; c0 += 32 * kBatch) {  // pieces of this half
      uint4 w[kBatch];
      uint32_t any = 0;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) w[b] = at[c0 + 32 * b];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) any |= any_not_finite(w[b]);
      if (any == 0) continue;
#pragma unroll 1
      for (int b = 0; b < kBatch; ++b) {
        uint32_t *v = reinterpret_cast<uint32_t *>(at + c0 + 32 * b);
        for (int e = 0; e < 4; ++e) {
          const bool lo = not_finite(v[e]), hi = not_finite(v[e] >> 16);
          if (!lo && !hi) continue;
          v[e] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
          own |= j * kN + ((c0 + 32 * b + lane) >> 3) < u.len;  // 8 pieces a row
        }
      }
    }
    dirty |= __any_sync(~0u, own) ? 1u << (j - u.cut) : 0u;
    // (the unit's word, read by the softmax warps once its last product is complete)
    if (lane == 0) reinterpret_cast<volatile uint32_t *>(smem + kDirty)[2 * (past.units & (kUnits - 1)) + half] = dirty;
    pa::fence_async_smem();
    __syncwarp();
    if (lane == 0) pa::mbar_arrive(bars + 8 * (B_CLEAN + j - u.cut));
    if (first && !warp_wait(told, phase)) return false;
  }
  return true;
}

// The infinities and NaN among the values that a row attends and that were replaced by 0: into its output, which this
// thread has written.  Rare, so it is simple: a thread walks up to 256 keys x 128 elements, two bytes at a time.  A weight of 0 is not told from
// others here: the infinity is added (0 * inf would be NaN, as it is in blocks that no row is cut in).
__device__ __noinline__ void add_not_finite(const uint16_t *v, int64_t v_stride, void *out, bool out_f32, uint32_t dirty, int cut, int token) {
  for (int i = cut * kN; i <= token; ++i) {
    if (!(dirty >> (i / kN - cut) & 1u)) continue;
    for (int d = 0; d < kD; ++d) {
      const uint16_t bits = v[i * v_stride + d];
      if (!not_finite(bits)) continue;
      const float x = __uint_as_float((uint32_t)bits << 16);
      if (out_f32) {
        static_cast<float *>(out)[d] += x;
      } else {
        uint16_t *o = static_cast<uint16_t *>(out) + d;
        *o = (uint16_t)(pa::pack_bf16x2(__uint_as_float((uint32_t)*o << 16) + x, 0.f) & 0xFFFFu);
      }
    }
  }
}

template <int N>
__device__ __forceinline__ float peak_of(const uint32_t *s) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < N; k += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e] = max3(top[e], __uint_as_float(s[k + 2 * e]), __uint_as_float(s[k + 2 * e + 1]));
  return max3(fmaxf(top[0], top[1]), top[2], top[3]);
}

// 2^(c s - m) of N columns as bf16 pairs; they are added, before the rounding, to the half block's sums.
struct Sums {
  pa::f32x2 part[2] = {pa::pack2(0.f, 0.f), pa::pack2(0.f, 0.f)};
  __device__ __forceinline__ float all() const {
    float x, y;
    pa::unpack2(pa::add2(part[0], part[1]), x, y);
    return x + y;
  }
};
template <int N>
__device__ __forceinline__ void weights(const uint32_t *s, float c, float m, uint32_t *w, Sums &sums) {
  const pa::f32x2 c2 = pa::pack2(c, c), m2 = pa::pack2(-m, -m);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    float a, b;
    pa::unpack2(pa::fma2(pa::pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, m2), a, b);
    a = pa::fast_exp2(a);
    b = pa::fast_exp2(b);
    sums.part[(e >> 1) & 1] = pa::add2(sums.part[(e >> 1) & 1], pa::pack2(a, b));
    w[e >> 1] = pa::pack_bf16x2(a, b);
  }
}

__device__ __forceinline__ void published(uint32_t bar) {
  tmem_wait_st();
  pa::tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) pa::mbar_arrive(bar);
}

// A row of a tile: TMEM lane and thread.  A warp's rows are in the order of their tokens.
struct Row {
  int row, tk, token;  // of the tile, its token of the tile and of the sequence
  bool live;
  int first, last;     // tokens of the sequence: of the warp's first row, and of its last one that is live (or less)
  uint32_t lanes;      // of the warp, in a TMEM address
};
__device__ __forceinline__ Row row_of(const PromptParams &p, const Unit &u, int tk, int tk0, int tk1) {  // tk0, tk1: of the warp's first and last row
  const int warp = threadIdx.x >> 5;
  Row r;
  r.row = 32 * (warp & 3) + (threadIdx.x & 31);
  r.tk = tk;
  r.token = u.tok(warp >> 2) + r.tk;
  r.live = r.tk < p.tokens && r.token < u.len;
  r.first = u.tok(warp >> 2) + tk0;
  r.last = tk0 < p.tokens ? min(u.tok(warp >> 2) + min(tk1, p.tokens - 1), u.len - 1) : -1;
  r.lanes = (uint32_t)(32 * (warp & 3)) << 16;
  return r;
}

// 32 columns of S from the g-th, -inf where a row does not attend.
__device__ __forceinline__ void cut_scores(const Row &r, int key0, int g, uint32_t s_at, uint32_t (&s)[32]) {
  tmem_ld32(s_at + 32 * g, s);
  tmem_wait32(s);
  key0 += 32 * g;
  if (r.first - key0 >= 31) return;
  const int seen = r.token - key0;  // a bit for each column (0.1 us less than comparisons, for 128 tokens)
  const uint32_t bits = seen >= 31 ? ~0u : seen < 0 ? 0u : (2u << seen) - 1u;
#pragma unroll
  for (int k = 0; k < 32; ++k) s[k] = (bits >> k) & 1u ? s[k] : 0xFF800000u;
}

// Where a row's scores grew by more than the slack: O and l are scaled.
__device__ __forceinline__ bool raise_max(float peak, uint32_t o_at, uint32_t bar_o, uint32_t phase_o, float &m, float &l) {
  const bool grown = peak > m + kSlack;
  if (!__any_sync(~0u, grown)) return true;
  const float alpha = grown ? pa::fast_exp2(m - peak) : 1.f;
  if (grown) m = peak;
  l *= alpha;
  if (!warp_wait(bar_o, phase_o)) return false;
  pa::tc_fence_after();
  uint32_t w[32];
#pragma unroll 1
  for (int k = 0; k < kD; k += 32) {
    tmem_ld32(o_at + k, w);
    tmem_wait32(w);
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
    tmem_st32(o_at + k, w);
  }
  return true;
}

// The weights of all blocks; m: what is subtracted from the scaled scores, in units of log2, l: the weights' sum.
template <bool LOOP>
__device__ bool run_softmax(const PromptParams &p, const Unit &u, const Past &past, const Row &r, uint32_t bars, float &m, float &l) {
  const int t = threadIdx.x >> 7, nb = u.nb(t), before = past.b(t);
  const uint32_t s_at = r.lanes + 128 * t, o_at = r.lanes + 256 + 128 * t, bar_o = bars + 8 * (B_O + t), bar_p = bars + 8 * (B_P + 2 * t);
  const int first = u.tok(t);
  const float c = p.fold;
  m = -INFINITY;
  l = 0.f;
  for (int j = 0; j < nb; ++j) {
    if (!warp_wait(bars + 8 * (B_S + t), (before + j) & 1)) return false;
    pa::tc_fence_after();
    const int key0 = u.block(t, j) * kN;
    const uint32_t phase_o = (before + j - 1) & 1;
    // The diagonal may cut it.  LOOP, whose units are many and short: 32 columns at a time, read twice, and those that no row of the
    // warp attends cost nothing (300 x 100 tokens x 16 heads 65 us, 73 as below; one prompt of 512 8.6 us, not 8.3).
    if (LOOP && key0 + kN > first) {
      const int groups = min(max(r.last - key0 + 32, 0) >> 5, kN / 32);
      float peak = -INFINITY;
#pragma unroll 1
      for (int g = 0; g < groups; ++g) {
        uint32_t s[32];
        cut_scores(r, key0, g, s_at, s);
        peak = fmaxf(peak, peak_of<32>(s));
      }
      peak *= c;
      if (j == 0)
        m = fmaxf(peak, -FLT_MAX);  // (scores of -inf alone: weights of 0, not of 2^(inf - inf), so that a later block counts)
      else if (!raise_max(peak, o_at, bar_o, phase_o, m, l))
        return false;
      Sums sums;
#pragma unroll 1
      for (int g = 0; g < kN / 32; ++g) {  // over S of columns that have been read twice
        uint32_t w[16];
        if (g < groups) {
          uint32_t s[32];
          cut_scores(r, key0, g, s_at, s);
          weights<32>(s, c, m, w, sums);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0u;
        }
        tmem_st16(s_at + 16 * g, w);
        if (g & 1) {
          published(bar_p + 4 * (g - 1));
          l += sums.all();  // (in the order of whole blocks: the same bits)
          sums = Sums();
        }
      }
      continue;
    }
    uint32_t s[kN], w[32];
#pragma unroll
    for (int k = 0; k < kN; k += 32) tmem_ld32(s_at + k, s + k);
#pragma unroll
    for (int k = 0; k < kN; k += 32) tmem_wait32(s + k);
    if (!LOOP && key0 + kN > first) {  // the diagonal may cut this block (a bit for each column: 0.1 us less than comparisons, for 128 tokens)
      const int seen = r.token - key0;
#pragma unroll
      for (int k0 = 0; k0 < kN; k0 += 32) {
        const uint32_t bits = seen >= k0 + 31 ? ~0u : seen < k0 ? 0u : (2u << (seen - k0)) - 1u;
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k0 + k] = (bits >> k) & 1u ? s[k0 + k] : 0xFF800000u;
      }
    }
    const float peak = peak_of<kN>(s) * c;
    if (j == 0)
      m = fmaxf(peak, -FLT_MAX);
    else if (!raise_max(peak, o_at, bar_o, phase_o, m, l))
      return false;
    Sums first_half, second_half;
    weights<kN / 2>(s, c, m, w, first_half);
    l += first_half.all();
    tmem_st32(s_at, w);
    published(bar_p);  // its product begins while the second half is worked out
    weights<kN / 2>(s + kN / 2, c, m, w, second_half);
    l += second_half.all();
    tmem_st32(s_at + kN / 4, w);
    published(bar_p + 8);
  }
  return true;
}

// N columns of a tile's O, scaled; of a solo tile, whose other slot's lie 128 columns on, the sum of both.
template <int N>
__device__ __forceinline__ void o_columns(uint32_t at, bool solo, float mine, float others, uint32_t *o) {
#pragma unroll
  for (int k = 0; k < N; k += 32) tmem_ld32(at + k, o + k);
  if (solo) {
    uint32_t x[N];
#pragma unroll
    for (int k = 0; k < N; k += 32) tmem_ld32(at + 128 + k, x + k);
#pragma unroll
    for (int k = 0; k < N; k += 32) tmem_wait32(o + k);
#pragma unroll
    for (int k = 0; k < N; k += 32) tmem_wait32(x + k);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), mine, __uint_as_float(x[e]) * others));
  } else {
#pragma unroll
    for (int k = 0; k < N; k += 32) tmem_wait32(o + k);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * mine);
  }
}

// The tile's rows: O / l and the log-sum-exp.  A solo tile's O is the sum of both slots', which lie in the same lanes of TMEM: each
// slot's warps join half of its columns.
// The rows go through shared memory, 128 bytes of each at a time, as the tensor map has them (128-byte swizzle): in place of the
// tile's queries, whose last S is complete, or (LOOP) where the next unit's queries are not.  Stored from the lanes, row by row, each
// store took 32 cycles and a tile 4000.
template <bool LOOP>
__device__ void write_tile(const PromptParams &p, const Unit &u, const Past &past, const Row &r, float m, float l, uint8_t *smem) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = warp >> 2, hq = p.Hkv * p.G;
  const int first = u.tok(t);
  const uint32_t o_at = r.lanes + 256 + (u.solo ? 0 : 128 * t);
  float mine = 1.f, others = 0.f;  // what O of slot 0 (or of the tile's own) and that of slot 1 count
  const bool leader = warp == 4 * t && lane == 0;  // the tile's stores are this thread's
  auto together = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(2 + t) : "memory"); };  // the slot's four warps
  auto both = [&]() { asm volatile("bar.sync 4, 256;" ::: "memory"); };
  if (u.solo) {
    float *ms = reinterpret_cast<float *>(smem + kBoth<LOOP>), *ls = ms + 2 * kM;
    if (LOOP) {  // (the stores of the unit before have read that place)
      if (leader) bulk_read_wait();
      both();
    }
    ms[t * kM + r.row] = m;
    ls[t * kM + r.row] = l;
    both();
    pa::tc_fence_after();
    const float m0 = ms[r.row], m1 = ms[kM + r.row], l0 = ls[r.row], l1 = ls[kM + r.row];
    if (LOOP) both();  // read by both before rows are written there
    m = fmaxf(m0, m1);
    mine = pa::fast_exp2(m0 - m);
    others = pa::fast_exp2(m1 - m);
    l = l0 * mine + l1 * others;
  }
  // A slot looks at the bits of its own blocks alone: the warps of slot 0 would read that of slot 1's last block before it is set, after,
  // or some of them either way, and part at the barriers below.  Its own bits are final: they are written before the block's B_CLEAN,
  // which the MMA warp waits for before the block's product, and this warp has waited for the last of those (B_O).  A solo tile's
  // blocks are both slots', which both() has joined.
  const volatile uint32_t *dirt = reinterpret_cast<const volatile uint32_t *>(smem + kDirty) + 2 * (past.units & (kUnits - 1));
  uint32_t dirty = dirt[0] | dirt[1];
  if (!u.solo) dirty &= (1u << (u.nb(t) - u.cut)) - 1u;
  const int64_t at = (int64_t)(u.row0 + r.token) * hq + u.h * p.G + (r.row - r.tk * p.G);
  const bool writes = r.live && !(u.solo && t == 1);  // a row's lse, and what else is one thread's
  if (writes && p.lse != nullptr) p.lse[at] = (m + log2f(l)) * kLn2;
  float inv;  // (to 1 unit of the last place; a division 0.7 us more for 300 x 100 tokens x 16 heads)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(l));
  mine *= inv;
  others *= inv;
  const bool whole = !p.out_f32 && first + p.tokens <= u.len;  // else the tile's box reaches past the sequence
  const int size = p.out_f32 ? 4 : 2, cols = 128 / size;
  int pass = 0;
#pragma unroll 1
  for (int k0 = u.solo ? t * cols : 0; k0 < kD; k0 += u.solo ? 2 * cols : cols, ++pass) {
    // (solo: the slots' passes take turns, and so do the two places)
    uint8_t *rows = LOOP ? smem + kOut + t * (kOperand / 2) : smem + (u.solo ? 0 : t * kOperand) + ((u.solo ? t : pass) & 1) * (kOperand / 2);
    uint4 *row = reinterpret_cast<uint4 *>(rows + r.row * 128);
    auto ready = [&]() {
      if (LOOP) {  // the store before, of this unit or the last one, has read its rows
        if (leader) bulk_read_wait();
        together();
      }
    };
    if (p.out_f32) {
      uint32_t o[32];
      o_columns<32>(o_at + k0, u.solo, mine, others, o);
      ready();
#pragma unroll
      for (int e = 0; e < 8; ++e) row[e ^ (r.row & 7)] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
    } else {
      // (LOOP: short code, since many units are short ones; 600 x 60 tokens x 16 heads 84 us, 87 with 64 at a time; but a prompt of
      // 1024 11.4 us, not 11.2)
      constexpr int kCols = LOOP ? 32 : 64;
#pragma unroll 1
      for (int k = 0; k < 64; k += kCols) {
        uint32_t o[kCols];
        o_columns<kCols>(o_at + k0 + k, u.solo, mine, others, o);
        if (k == 0) ready();
#pragma unroll
        for (int e = 0; e < kCols / 8; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pa::pack_bf16x2(__uint_as_float(o[8 * e + 2 * i]), __uint_as_float(o[8 * e + 2 * i + 1]));
          row[(k / 8 + e) ^ (r.row & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (whole) {
      pa::fence_async_smem();
      together();
      if (leader) {
        tma_store_3d(&p.tm_o, pa::smem_u32(rows), k0, u.h * p.G, u.row0 + first);
        bulk_commit();
      }
    } else {  // 128 bytes of a row to 8 lanes; a warp's rows are its own
      const int where = r.live ? r.tk * hq + r.row - r.tk * p.G : -1;  // from the tile's first row and head
      const int64_t origin = (int64_t)(u.row0 + first) * hq + u.h * p.G;
      __syncwarp();
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const int q = 4 * i + (lane >> 3), dst = __shfl_sync(~0u, where, q), row = 32 * (warp & 3) + q;
        const uint4 v = *reinterpret_cast<const uint4 *>(rows + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
        if (dst >= 0) *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + ((origin + dst) * kD + k0) * size + (lane & 7) * 16) = v;
      }
      __syncwarp();
    }
  }
  if (LOOP && u.solo) {
    // Either slot has read columns of both slots' O: neither publishes weights of the next unit, whose product would be written over
    // them, before the other has read its own.
    pa::tc_fence_before();
    both();
  }
  if (dirty != 0) {  // (the same for both slots of a solo tile)
    if (leader) bulk_write_wait();
    if (u.solo)
      both();
    else
      together();  // the tile has been written
    if (writes)
      add_not_finite(p.v + u.row0 * p.v_stride + u.h * kD, p.v_stride, static_cast<uint8_t *>(p.out) + at * kD * size, p.out_f32, dirty,
                     u.cut, r.token);
  }
}

// Whether none of the warps that write a tile together gave up: they write it, or none of them does.
__device__ __forceinline__ bool agreed(bool ok, bool solo, int t) {
  int r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((int)ok), "r"(solo ? 4 : 2 + t), "r"(solo ? 256 : 128)
               : "memory");
  return r != 0;
}

// What a warp that gave up owes to others of its slot, or (solo) of both: it comes to the barriers of the units that are posted still,
// from this one on.  (As many as there are places for them at most: it leaves none.)
__device__ __noinline__ void come_to_barriers(uint8_t *smem, uint32_t bars, int round, int t) {
  Unit u;
  for (; unit_comes(bars, round) && posted_unit(smem, round, u); ++round) agreed(false, u.solo, t);
}

// OWN, ALL: how the schedule is worked out.  LOOP: CTAs go on with further units, whose first scores are there when the rows of
// the one before have been written; else a CTA for each.
template <int OWN, bool ALL, bool LOOP>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
  constexpr int STAGES = kStages<LOOP>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (pa::smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = pa::smem_u32(smem), bars = base + kBars;
  // (from lane 0, so that the roles' control flow and the MMAs' operands are known to be uniform: 650 us, else 620, for
  // 16384 tokens x 16 heads)
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == kLoadWarp && lane == 0) {
    prefetch_map(&p.tm_q);
    prefetch_map(&p.tm_k);
    prefetch_map(&p.tm_v);
    for (int i = 0; i < kNumBars; ++i)
      pa::mbar_init(bars + 8 * i, i >= B_P && i < B_P + 4 ? 4 : i == B_DONE ? kSoftWarps : i >= B_CLEAN && i < B_CLEAN + 2 ? 2
                                                              : i >= B_LEFT && i < B_LEFT + 4 ? kThreads / 32 - 1 : 1);
    pa::fence_barrier_init();
  }
  if (warp == kMmaWarp) pa::tmem_alloc(base + kMisc, kTmemCols);
  __syncwarp();  // (before the register split, which whole warps take)
  // The load warp finds the CTA's units, the first one before the others need anything of it.  The units come in descending order.
  Unit u;
  Past past;
  bool ok = true, more = false;
  int round = 0;
  Schedule<OWN, ALL> schedule(p, smem);
  auto post = [&]() {
    if (lane == 0) {
      post_unit(smem, round, u, more);
      pa::mbar_arrive(bars + 8 * (B_UNIT + (round & (kUnits - 1))));
    }
    __syncwarp();
  };
  auto begin = [&]() {
    pa::pdl_wait();
    pa::pdl_launch_dependents();
    if (ALL || warp == kLoadWarp) {
      schedule.start();
      more = schedule.find((int)blockIdx.x, u);
      if (!ALL) post();
    }
    pa::tc_fence_before();
    if (warp == kLoadWarp)  // (it needs nothing of the others)
      asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
    else
      asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    pa::tc_fence_after();
    if (!ALL && warp != kLoadWarp) more = posted_unit(smem, 0, u);
  };
  auto next = [&]() {  // the unit after this one, if there is one
    if (LOOP) {
      __syncwarp();
      if (lane == 0) pa::mbar_arrive(bars + 8 * (B_LEFT + (round & (kUnits - 1))));
    }
    past.add(u);
    ++round;
    more = false;
    if (LOOP) {
      ok = warp_wait(bars + 8 * (B_UNIT + (round & (kUnits - 1))), (round / kUnits) & 1);
      more = ok && posted_unit(smem, round, u);
    }
  };
  if (warp < kSoftWarps) {
    pa::regs_inc<216>();
    begin();
    if (!more) return;
    const int t = warp >> 2, tk = (threadIdx.x & (kM - 1)) / p.G;
    const int tk0 = __shfl_sync(~0u, tk, 0), tk1 = __shfl_sync(~0u, tk, 31);
    while (more) {
      const Row r = row_of(p, u, tk, tk0, tk1);
      float m, l;
      ok = run_softmax<LOOP>(p, u, past, r, bars, m, l);
      if (ok && u.nb(t) > 0) ok = warp_wait(bars + 8 * (B_O + t), (past.b(t) + u.nb(t) - 1) & 1);
      pa::tc_fence_after();
      ok = agreed(ok, u.solo, t);
      if (!ok) break;
      if (u.nb(t) > 0) write_tile<LOOP>(p, u, past, r, m, l, smem);
      pa::tc_fence_before();  // O has been read before the next unit's weights are published
      next();
    }
    if (LOOP && !ok)  // with its slot (`more`), or while it waited for a unit
      come_to_barriers(smem, bars, more ? round + 1 : round, t);
    if (lane == 0) {
      bulk_read_wait();
      pa::mbar_arrive(bars + 8 * B_DONE);
    }
  } else {
    pa::regs_dec<72>();
    begin();
    if (!more) {
      if (warp == kMmaWarp) pa::tmem_dealloc(0, kTmemCols);
      return;
    }
    if (warp == kLoadWarp) {
      Loads done;
      while (more) {
        ok = load_unit<STAGES>(p, u, past, base, bars, done);
        if (!ok || !LOOP) break;
        // The CTA that would come next: asked for when the last loads of this unit have been (some two blocks before its end).
        if (lane == 0) claim_next(base + kClaim, bars + 8 * B_CLAIM);
        __syncwarp();
        ++done.claims;
        past.add(u);
        ok = warp_wait(bars + 8 * B_CLAIM, round & 1);
        if (!ok) break;
        const int x = claimed(base + kClaim);
        __syncwarp();
        ++round;
        if (round >= kUnits) ok = warp_wait(bars + 8 * (B_LEFT + (round & (kUnits - 1))), (round / kUnits - 1) & 1);
        if (!ok) break;
        more = x >= 0 && schedule.find(x, u);
        pa::fence_async_smem();  // the answer has been read
        post();
      }
      if (LOOP && lane == 0) pa::mbar_arrive(bars + 8 * B_END);
      if (!ok && lane == 0) drain<STAGES>(bars, done);
    } else if (warp == kMmaWarp) {
      pa::tc_fence_after();
      while (ok && more) {
        Work w;
        w.set(u, past);
        ok = issue_mmas<STAGES>(w, base, bars);
        if (ok) next();
      }
      if (pa::elect_one()) pa::umma_commit(bars + 8 * B_MMA);
      __syncwarp();
      ok = warp_wait(bars + 8 * B_MMA, 0) & ok;
      ok = warp_wait(bars + 8 * B_DONE, 0) & ok;
      pa::tc_fence_after();
      pa::tmem_dealloc(0, kTmemCols);
    } else {
      while (ok && more) {
        ok = clean_unit<STAGES>(u, past, bars, smem);
        if (ok) next();
      }
    }
  }
  if (!ok && lane == 0) raise(p, PA_DEV_TIMEOUT);
}

// ------------------------------------------------------------------------------- host

struct PromptDevice {
  int sms = 0;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
};

// The kernels' opt-in and the tensor-map encoder, once per device; NULL when a call fails, the kernel was not built
// with the registers that its split counts on, or the device is beyond those tracked.
const PromptDevice *prompt_device() {
  static std::once_flag once[pa_host::kMaxDevices];
  static PromptDevice devs[pa_host::kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= pa_host::kMaxDevices) return nullptr;
  std::call_once(once[dev], [dev]() {
    PromptDevice d;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return;
    for (const void *f : {(const void *)prompt_attn_kernel<1, false, false>, (const void *)prompt_attn_kernel<1, true, false>,
                          (const void *)prompt_attn_kernel<11, true, false>, (const void *)prompt_attn_kernel<1, false, true>,
                          (const void *)prompt_attn_kernel<4, false, true>, (const void *)prompt_attn_kernel<32, false, true>}) {
      cudaFuncAttributes at;
      if (cudaFuncGetAttributes(&at, f) != cudaSuccess || at.numRegs != kRegs ||
          cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        return;
    }
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      return;
    d.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    devs[dev] = d;
  });
  return devs[dev].encode != nullptr ? &devs[dev] : nullptr;
}

// [rows][heads][128] bf16 with `stride` elements between rows, in boxes of 64 elements x box_heads x box_rows.
bool encode_rows(const PromptDevice *dev, CUtensorMap *map, const void *at, int rows, int heads, int64_t stride, int box_heads, int box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)(2 * kD), (cuuint64_t)(2 * stride)};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t each[3] = {1, 1, 1};
  return dev->encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(at), dims, strides, box, each,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" pa_status_t pa_prompt_attn(const pa_prompt_attn_args_t *a, void *stream) {
  if (a == nullptr) return PA_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_rows < 0 || a->num_kv_heads < 1 || a->group_size < 1 || !(a->sm_scale > 0.f) ||
      !std::isfinite(a->sm_scale) || (a->out_dtype != PA_OUT_BF16 && a->out_dtype != PA_OUT_F32) || a->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (a->head_dim != kD || a->num_kv_heads > pa_host::kMaxHeads || a->group_size > kMaxGroup || a->num_seqs > kMaxSeqs ||
      a->num_rows > kMaxRows)
    return PA_ERR_UNSUPPORTED;
  const int heads = a->num_kv_heads * a->group_size;
  const int64_t q_row = (int64_t)heads * kD, k_row = (int64_t)a->num_kv_heads * kD;
  constexpr int64_t kMost = 1ll << 38;  // elements between rows: a tensor map's stride is below 2^40 bytes
  if (a->q_stride < q_row || a->k_stride < k_row || a->v_stride < k_row || a->q_stride > kMost || a->k_stride > kMost || a->v_stride > kMost)
    return PA_ERR_INVALID_ARG;
  if (a->q == nullptr || a->k == nullptr || a->v == nullptr || a->cu_seqlens == nullptr || a->out == nullptr) return PA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16) || a->q_stride % 8 != 0 ||
      a->k_stride % 8 != 0 || a->v_stride % 8 != 0 || !aligned(a->cu_seqlens, 4) || !aligned(a->lse, 4) || !aligned(a->status, 4))
    return PA_ERR_ALIGN;
  using pa_host::Rows;
  const int64_t n = a->num_rows, size = a->out_dtype == PA_OUT_F32 ? 4 : 2, cus = ((int64_t)a->num_seqs + 1) * 4;
  const Rows q{a->q, n, q_row * 2, a->q_stride * 2}, k{a->k, n, k_row * 2, a->k_stride * 2}, v{a->v, n, k_row * 2, a->v_stride * 2},
      out{a->out, 1, n * q_row * size, n * q_row * size}, lse{a->lse, 1, n * heads * 4, n * heads * 4}, cu{a->cu_seqlens, 1, cus, cus};
  for (const Rows &in : {q, k, v, cu})
    if (pa_host::rows_overlap(out, in) || pa_host::rows_overlap(lse, in)) return PA_ERR_INVALID_ARG;
  if (pa_host::rows_overlap(out, lse)) return PA_ERR_INVALID_ARG;
  if (a->num_seqs == 0 || n == 0) return PA_OK;

  const PromptDevice *dev = prompt_device();
  if (dev == nullptr) return PA_ERR_CUDA;
  PromptParams p;
  p.cu = a->cu_seqlens;
  p.v = static_cast<const uint16_t *>(a->v);
  p.out = a->out;
  p.lse = a->lse;
  p.status = a->status;
  p.v_stride = a->v_stride;
  p.B = a->num_seqs;
  p.T = a->num_rows;
  p.Hkv = a->num_kv_heads;
  p.G = a->group_size;
  p.tokens = kM / a->group_size;
  p.out_f32 = a->out_dtype == PA_OUT_F32;
  p.fold = (float)((double)a->sm_scale * 1.4426950408889634);
  p.sms = dev->sms;
  const int64_t span = 2 * p.tokens;
  p.first_split = (int)((kMinSplit * kN + span - 1) / span);
  p.aside = (int)(4 * kN * a->num_kv_heads / span);
  p.per_span = ((1ull << 40) + span - 1) / span;
  if (!encode_rows(dev, &p.tm_q, a->q, a->num_rows, heads, a->q_stride, p.G, p.tokens) ||
      !encode_rows(dev, &p.tm_k, a->k, a->num_rows, a->num_kv_heads, a->k_stride, 1, kN) ||
      !encode_rows(dev, &p.tm_v, a->v, a->num_rows, a->num_kv_heads, a->v_stride, 1, kN) ||
      !encode_rows(dev, &p.tm_o, a->out, a->num_rows, heads, q_row, p.G, p.tokens))
    return PA_ERR_CUDA;
  // A CTA for every unit there can be, and for those that may be split (while there are fewer units than twice the SMs).  CTAs
  // without a share exit.  Where CTAs would come to an SM one after the other, a CTA takes several units in turn: as many units as SMs
  // (16 x 2048 tokens x 16 heads 191 us, 238 without, 16384 600 and 613, 64 x 40 10.6 and 13.2), or of several sequences two thirds of
  // that (4 x 400 10.7 and 12.8, 2 x 1024 15.4 and 17.5; but 4 x 330 9.2 and 8.5).  Units of one sequence are of all lengths, and the
  // split ones fill such gaps (1800 tokens 19.8 and 17.2).  The load warps of these CTAs work out the schedule alone, which holds for
  // up to 1024 sequences.
  const int64_t units = (n + a->num_seqs * (span - 1)) / span * a->num_kv_heads;
  const bool loop = a->num_seqs <= 1024 && (units >= dev->sms || (a->num_seqs > 1 && 3 * units >= 2 * dev->sms));
  const int64_t grid = std::max(units, std::min<int64_t>(2 * units, 4 * dev->sms));
  const pa_host::Launch run(dim3((unsigned)grid), dim3(kThreads), kSmem, stream);
  cudaError_t e;
  if (loop)
    e = a->num_seqs <= 32    ? cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<1, false, true>, p)
        : a->num_seqs <= 128 ? cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<4, false, true>, p)
                             : cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<32, false, true>, p);
  else
    e = a->num_seqs <= 32         ? cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<1, false, false>, p)
        : a->num_seqs <= kThreads ? cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<1, true, false>, p)
                                  : cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<11, true, false>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
