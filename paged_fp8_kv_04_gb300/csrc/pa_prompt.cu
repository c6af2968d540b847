// pa_prompt.cu -- causal attention over whole packed prompts: pa_prompt_attn.  See include/pa.h for
// the contract.
//
//   S = Q K^T        tcgen05.mma kind::f16, M = 128 rows, N = 128 keys, both operands from shared memory as TMA left
//                    them (K-major, 128-byte swizzle)
//   P = 2^(c S - m)  a thread per row: TMEM lane = row.  c = sm_scale log2 e; m follows the row's maximum, but only
//                    when it has grown by more than 2^8: until then the weights exceed 1 by that much at most, and nothing
//                    has to be scaled again.  The sum of the weights is fp32, taken before they are rounded
//   O += P V         kind::f16 with P as the A operand in TMEM, in the columns that S had (bf16 because V is: a
//                    rounding of 2^-9 per weight, as that of the output), V as the B operand, MN-major, as TMA left it
//
// Rows of a tile are (token, head of the group) pairs, 128 / group_size tokens with all query heads of a KV head: they
// share its keys, short prompts fill a tile as well as long ones do, and the diagonal cuts few tokens.  A CTA has two tiles, so that the
// tensor core works on one while the other's weights are computed: S0 S1 | PV0 S0' PV1 S1' | ...
//
// Warp roles (384 threads): warps 0-3 and 4-7 are the softmax of tiles 0 and 1; warp 8 fetches tiles by TMA; warp 9
// issues the MMAs; warps 10 and 11 look through the values of the blocks that the diagonal or the sequence's end cuts: an
// infinity or NaN there must not reach rows that do not attend it (0 * inf), so it is replaced by 0, and rows that do attend it
// get it in the epilogue.  Every wait is bounded; TMEM is released on every path.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

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
constexpr int kStages = 5;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;     // log2 of what the weights may exceed 1 by

struct PromptParams {
  CUtensorMap tm_q, tm_k, tm_v;
  const int32_t *cu;
  const uint16_t *v;  // for the epilogue of values that are not finite
  void *out;
  float *lse;
  uint32_t *status;
  int64_t v_stride;
  int32_t B, T, Hkv, G, tokens;  // tokens of a tile
  int32_t out_f32;
  float fold;  // sm_scale * log2 e
};

// Shared memory: two query tiles, the ring of K and V blocks, barriers and the schedule's scratch.
constexpr int kRing = 2 * kOperand;
constexpr int kBars = kRing + kStages * kOperand;
enum {
  B_QFULL = 0,                      // [2] the tile's queries
  B_FULL = 2,                       // [kStages]
  B_EMPTY = B_FULL + kStages,       // [kStages]
  B_S = B_EMPTY + kStages,          // [2] S is complete
  B_P = B_S + 2,                    // [2] P is in TMEM (and O scaled)
  B_O = B_P + 2,                    // [2] PV is complete
  B_CLEAN = B_O + 2,                // [2] the values have been looked through: of the first and second cut block
  B_CUT = B_CLEAN + 2,              // [2] the values of a cut block, in place of B_FULL
  B_DONE = B_CUT + 2,               // the softmax warps are done with TMEM
  B_MMA = B_DONE + 1,               // every MMA is complete
  kNumBars = B_MMA + 1
};
constexpr int kMisc = kBars + 8 * kNumBars;  // TMEM address, dirty blocks, sequence, padding
constexpr int kRed = kMisc + 16;             // [2][warps] of the schedule's sums
constexpr int kSmem = kRed + 2 * 4 * (kThreads / 32) + 1024;

// TMEM columns: S of tile t at 128 t, O at 256 + 128 t; P over S.
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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands, K = 16.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void raise(const PromptParams &p, uint32_t flag) {
  if (p.status != nullptr) atomicOr(p.status, flag);
}

// A bounded wait by a whole warp: false for all lanes if it gave up for one.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(~0u, pa::mbar_wait_bounded(bar, parity)) != 0;
}

// A CTA's share: two tiles of one sequence and KV head.
struct Unit {
  int row0, len, tok0, h;  // the sequence's first row and length, the unit's first token
  // Key blocks of each tile (0: no tokens) and of both, and the first that the diagonal cuts: two of them at most, since a
  // unit has 256 tokens and begins with a block, or has 128 or fewer.
  int nb[2], blocks, cut;
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

// The x-th unit of the call for one KV head, the units with the most keys first: unit j of a sequence has j + 1 times the
// keys of its first, and the GPU's last CTAs should be short ones.  Units of index c or more number N(c), the sum
// of max(0, n_s - c) over the sequences: the unit's index is the largest c with N(c) > x, and it belongs to the
// (x - N(c + 1))-th of the sequences that have such a unit.  Synchronises the CTA; false if there are fewer units.
template <int KS>
__device__ bool locate(const PromptParams &p, int x, uint8_t *smem, Unit &u) {
  const int tid = threadIdx.x, span = 2 * p.tokens;
  int *red = reinterpret_cast<int *>(smem + kRed);
  volatile int *found = reinterpret_cast<volatile int *>(smem + kMisc + 8);
  int n[KS], sum = 0, top = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const int s = tid + i * kThreads;
    n[i] = 0;
    if (s < p.B) {
      const int a = p.cu[s], b = p.cu[s + 1];
      if (a < 0 || b < a || b > p.T)
        bad = true;
      else
        n[i] = (b - a + span - 1) / span;
    }
    sum += n[i];
    top = max(top, n[i]);
  }
  if (bad && blockIdx.x == 0) raise(p, PA_DEV_BAD_QLEN);
  const int total = reduce_all(sum, false, red, 0);
  if (x >= total) return false;
  int lo = 0, above = 0;  // N(lo) > x >= above = N(hi)
  if (p.B == 1) {
    lo = total - 1 - x;
    above = x;
  } else {
    int hi = reduce_all(top, true, red, 1), turn = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      int v = 0;
#pragma unroll
      for (int i = 0; i < KS; ++i) v += max(0, n[i] - mid);
      const int count = reduce_all(v, false, red, turn);
      turn ^= 1;
      if (count > x) {
        lo = mid;
      } else {
        hi = mid;
        above = count;
      }
    }
  }
  // the (x - above)-th of those with more than lo units, thread by thread
  int mine = 0;
#pragma unroll
  for (int i = 0; i < KS; ++i) mine += n[i] > lo;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, upto, o);
    if ((tid & 31) >= o) upto += y;
  }
  __syncthreads();  // the last sum has been read
  if ((tid & 31) == 31) red[tid >> 5] = upto;
  __syncthreads();
  for (int w = 0; w < (tid >> 5); ++w) upto += red[w];
  int at = x - above - (upto - mine);
  if (at >= 0 && at < mine) {
#pragma unroll
    for (int i = 0; i < KS; ++i)
      if (n[i] > lo && at-- == 0) *found = tid + i * kThreads;
  }
  __syncthreads();
  const int s = *found;
  u.row0 = p.cu[s];
  u.len = p.cu[s + 1] - u.row0;
  u.tok0 = lo * span;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = u.tok0 + t * p.tokens;
    u.nb[t] = first < u.len ? (min(u.len, first + p.tokens) + kN - 1) / kN : 0;
  }
  u.blocks = max(u.nb[0], u.nb[1]);
  u.cut = u.tok0 / kN;
  return true;
}

// ------------------------------------------------------------------------------- roles

// The barrier that block i of the ring (keys and values in turn) lands on.  Values of cut blocks have one of their own,
// since the warps that look through them follow no others; nothing comes after them in their stages.
__device__ __forceinline__ uint32_t bar_landed(const Unit &u, uint32_t bars, int i, uint32_t &parity) {
  const bool cut = (i & 1) != 0 && (i >> 1) >= u.cut;
  parity = cut ? 0 : (i / kStages) & 1;
  return bars + 8 * (cut ? B_CUT + (i >> 1) - u.cut : B_FULL + i % kStages);
}
__device__ __forceinline__ bool landed(const Unit &u, uint32_t bars, int i) {
  uint32_t parity;
  const uint32_t bar = bar_landed(u, bars, i, parity);
  return warp_wait(bar, parity);
}

__device__ void run_producer(const PromptParams &p, const Unit &u, uint32_t base, uint32_t bars) {
  const int lane = threadIdx.x & 31;
  const uint32_t qbytes = (uint32_t)p.G * p.tokens * kD * 2;
  if (lane == 0) {
    for (int t = 0; t < 2; ++t) {
      if (u.nb[t] == 0) continue;
      pa::mbar_arrive_expect_tx(bars + 8 * (B_QFULL + t), qbytes);
      for (int x = 0; x < 2; ++x)
        tma_load_3d(base + t * kOperand + x * (kOperand / 2), &p.tm_q, 64 * x, u.h * p.G, u.row0 + u.tok0 + t * p.tokens,
                    bars + 8 * (B_QFULL + t));
    }
  }
  bool ok = true;
  int i = 0;
  for (; i < 2 * u.blocks && ok; ++i) {
    const int st = i % kStages, use = i / kStages;
    if (use > 0) ok = warp_wait(bars + 8 * (B_EMPTY + st), (use - 1) & 1);
    if (!ok) break;
    if (lane == 0) {
      uint32_t parity;
      const uint32_t bar = bar_landed(u, bars, i, parity), dst = base + kRing + st * kOperand;
      pa::mbar_arrive_expect_tx(bar, kOperand);
      for (int x = 0; x < 2; ++x)
        tma_load_3d(dst + x * (kOperand / 2), i & 1 ? &p.tm_v : &p.tm_k, 64 * x, u.h, u.row0 + (i >> 1) * kN, bar);
    }
    __syncwarp();
  }
  if (!ok && lane == 0) {
    raise(p, PA_DEV_TIMEOUT);
    for (int t = 0; t < 2; ++t)  // copies in flight land before the CTA can exit
      if (u.nb[t] > 0) pa::mbar_wait_bounded(bars + 8 * (B_QFULL + t), 0);
    for (int k = max(0, i - kStages); k < i; ++k) {
      uint32_t parity;
      const uint32_t bar = bar_landed(u, bars, k, parity);
      pa::mbar_wait_bounded(bar, parity);
    }
  }
}

__device__ void run_mma(const PromptParams &p, const Unit &u, uint32_t base, uint32_t bars, uint32_t tm) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  auto stage = [&](int i) { return base + kRing + (i % kStages) * kOperand; };
  auto scores = [&](int t, int j, bool last) {  // S_t of block j; `last`: nobody else reads its keys
    if (pa::elect_one()) {
      const uint32_t q = base + t * kOperand, k = stage(2 * j);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t off = (x >> 2) * (kOperand / 2) + 32 * (x & 3);
        pa::umma_f16(tm + 128 * t, pa::umma_sdesc(q + off, 1024, 1024, 2), pa::umma_sdesc(k + off, 1024, 1024, 2), idesc(0), x > 0);
      }
      pa::umma_commit(bars + 8 * (B_S + t));
      if (last) pa::umma_commit(bars + 8 * (B_EMPTY + (2 * j) % kStages));
    }
    __syncwarp();
  };
  // the tile that reads a block last: 1 if it has the block
  auto last_of = [&](int j) { return j < u.nb[1] ? 1 : 0; };
  for (int t = 0; t < 2 && ok; ++t)
    if (u.nb[t] > 0) {
      ok = warp_wait(bars + 8 * (B_QFULL + t), 0) && landed(u, bars, 0);
      if (!ok) break;
      pa::tc_fence_after();
      scores(t, 0, t == last_of(0));
    }
  for (int j = 0; j < u.blocks && ok; ++j) {
    ok = landed(u, bars, 2 * j + 1);
    if (ok && j >= u.cut) ok = warp_wait(bars + 8 * (B_CLEAN + j - u.cut), 0);
    for (int t = 0; t < 2 && ok; ++t) {
      if (j >= u.nb[t]) continue;
      ok = warp_wait(bars + 8 * (B_P + t), j & 1);
      if (!ok) break;
      pa::tc_fence_after();
      if (pa::elect_one()) {
        const uint32_t v = stage(2 * j + 1);
#pragma unroll
        for (int x = 0; x < 8; ++x)  // 16 keys: two groups of 8 rows; the two halves of head_dim 16 KB apart
          umma_ts(tm + 256 + 128 * t, tm + 128 * t + 8 * x, pa::umma_sdesc(v + 2048 * x, kOperand / 2, 1024, 2), idesc(1), j > 0 || x > 0);
        pa::umma_commit(bars + 8 * (B_O + t));
        if (t == last_of(j)) pa::umma_commit(bars + 8 * (B_EMPTY + (2 * j + 1) % kStages));
      }
      __syncwarp();
      if (j + 1 < u.nb[t]) {  // over P of this block, which the product before reads: MMAs run in order
        ok = landed(u, bars, 2 * j + 2);
        if (!ok) break;
        scores(t, j + 1, t == last_of(j + 1));
      }
    }
  }
  if (!ok && lane == 0) raise(p, PA_DEV_TIMEOUT);
  __syncwarp();
  if (pa::elect_one()) pa::umma_commit(bars + 8 * B_MMA);
  __syncwarp();
  if (!warp_wait(bars + 8 * B_MMA, 0) && lane == 0) raise(p, PA_DEV_TIMEOUT);
  if (!warp_wait(bars + 8 * B_DONE, 0) && lane == 0) raise(p, PA_DEV_TIMEOUT);
  pa::tc_fence_after();
  pa::tmem_dealloc(tm, kTmemCols);
}

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7F80u) == 0x7F80u; }

// Values of the blocks that the diagonal or the sequence's end cuts, by two warps.
__device__ void run_clean(const PromptParams &p, const Unit &u, uint32_t base, uint32_t bars, uint8_t *smem) {
  const int tid = threadIdx.x & 63, lane = tid & 31;
  for (int j = u.cut; j < u.blocks; ++j) {
    const int i = 2 * j + 1, st = i % kStages;
    if (!landed(u, bars, i)) {
      if (lane == 0) raise(p, PA_DEV_TIMEOUT);
      return;
    }
    const uint32_t at = base + kRing + st * kOperand;
    bool own = false;  // one of the sequence's own
    for (int c = tid; c < kOperand / 16; c += 64) {
      uint4 w = pa::lds128(at + 16 * c);
      uint32_t v[4] = {w.x, w.y, w.z, w.w};
      bool any = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool lo = not_finite(v[e]), hi = not_finite(v[e] >> 16);
        any |= lo || hi;
        v[e] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
      }
      if (any) {
        pa::sts128(at + 16 * c, make_uint4(v[0], v[1], v[2], v[3]));
        own |= j * kN + ((c & (kOperand / 32 - 1)) >> 3) < u.len;  // 8 pieces a row, in each half
      }
    }
    if (own) atomicOr(reinterpret_cast<unsigned *>(smem + kMisc + 4), 1u << (j - u.cut));
    pa::fence_async_smem();
    __syncwarp();
    if (lane == 0) pa::mbar_arrive(bars + 8 * (B_CLEAN + j - u.cut));
  }
}

__device__ void run_softmax(const PromptParams &p, const Unit &u, uint32_t bars, uint32_t tm, const uint8_t *smem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = warp >> 2;
  const int row = 32 * (warp & 3) + lane;
  const uint32_t lanes = tm + ((uint32_t)(32 * (warp & 3)) << 16), s_at = lanes + 128 * t, o_at = lanes + 256 + 128 * t;
  const int first = u.tok0 + t * p.tokens, tk = row / p.G, token = first + tk, nb = u.nb[t];
  const bool live = tk < p.tokens && token < u.len;
  const float c = p.fold;
  float m = 0.f, l = 0.f;  // m: what is subtracted, in units of log2
  bool ok = true;
  for (int j = 0; j < nb; ++j) {
    ok = warp_wait(bars + 8 * (B_S + t), j & 1);
    if (!ok) break;
    pa::tc_fence_after();
    uint32_t s[kN];
#pragma unroll
    for (int k = 0; k < kN; k += 32) tmem_ld32(s_at + k, s + k);
#pragma unroll
    for (int k = 0; k < kN; k += 32) tmem_wait32(s + k);
    if ((j + 1) * kN > first) {  // the diagonal may cut this block
      const int seen = token - j * kN;
#pragma unroll
      for (int k = 0; k < kN; ++k) s[k] = k <= seen ? s[k] : 0xFF800000u;
    }
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < kN; k += 4)
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], __uint_as_float(s[k + e]));
    const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
    if (j == 0) {
      m = peak;
    } else {
      const bool grown = peak > m + kSlack;
      if (__any_sync(~0u, grown)) {
        const float alpha = grown ? pa::fast_exp2(m - peak) : 1.f;
        if (grown) m = peak;
        l *= alpha;
        ok = warp_wait(bars + 8 * (B_O + t), (j - 1) & 1);
        if (!ok) break;
        pa::tc_fence_after();
#pragma unroll
        for (int k = 0; k < kD; k += 32) {
          uint32_t o[32];
          tmem_ld32(o_at + k, o);
          tmem_wait32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(o_at + k, o);
        }
      }
    }
    const pa::f32x2 c2 = pa::pack2(c, c), m2 = pa::pack2(-m, -m);
    pa::f32x2 part[2] = {pa::pack2(0.f, 0.f), pa::pack2(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < kN; k += 64) {
      uint32_t w[32];
#pragma unroll
      for (int e = 0; e < 64; e += 2) {
        float a, b;
        pa::unpack2(pa::fma2(pa::pack2(__uint_as_float(s[k + e]), __uint_as_float(s[k + e + 1])), c2, m2), a, b);
        a = pa::fast_exp2(a);
        b = pa::fast_exp2(b);
        part[(e >> 1) & 1] = pa::add2(part[(e >> 1) & 1], pa::pack2(a, b));
        w[e >> 1] = pa::pack_bf16x2(a, b);
      }
      tmem_st32(s_at + (k >> 1), w);
    }
    float x0, x1;
    pa::unpack2(pa::add2(part[0], part[1]), x0, x1);
    l += x0 + x1;
    tmem_wait_st();
    pa::tc_fence_before();
    __syncwarp();
    if (lane == 0) pa::mbar_arrive(bars + 8 * (B_P + t));
  }
  if (ok && nb > 0) ok = warp_wait(bars + 8 * (B_O + t), (nb - 1) & 1);
  if (ok && nb > 0) {
    pa::tc_fence_after();
    const uint32_t dirty = *reinterpret_cast<const volatile uint32_t *>(smem + kMisc + 4);
    const int64_t at = (int64_t)(u.row0 + token) * (p.Hkv * p.G) + u.h * p.G + (row - tk * p.G);
    const float inv = 1.f / l;
    if (live && p.lse != nullptr) p.lse[at] = (m + log2f(l)) * kLn2;
#pragma unroll
    for (int k = 0; k < kD; k += 32) {
      uint32_t o[32];
      tmem_ld32(o_at + k, o);
      tmem_wait32(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
      if (dirty != 0 && live) {  // infinities and NaN among the values that were replaced by 0
        for (int j = u.cut; j < nb; ++j) {
          if (!(dirty >> (j - u.cut) & 1u)) continue;
          for (int i = j * kN; i <= token && i < (j + 1) * kN; ++i) {
            const uint16_t *v = p.v + (int64_t)(u.row0 + i) * p.v_stride + u.h * kD + k;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (not_finite(v[e])) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float((uint32_t)v[e] << 16));
          }
        }
      }
      if (live) {
        if (p.out_f32) {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<float *>(p.out) + at * kD + k);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pa::pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at * kD + k);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
      }
    }
  }
  if (!ok && lane == 0) raise(p, PA_DEV_TIMEOUT);
  pa::tc_fence_before();
  __syncwarp();
  if (lane == 0) pa::mbar_arrive(bars + 8 * B_DONE);
}

// KS: sequences per thread in the schedule.
template <int KS>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (pa::smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = pa::smem_u32(smem), bars = base + kBars;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool soft = i == B_P || i == B_P + 1;
      pa::mbar_init(bars + 8 * i, soft ? 4 : i == B_CLEAN || i == B_CLEAN + 1 ? 2 : i == B_DONE ? kSoftWarps : 1);
    }
    *reinterpret_cast<uint32_t *>(smem + kMisc + 4) = 0;
    pa::fence_barrier_init();
  }
  pa::pdl_wait();
  pa::pdl_launch_dependents();
  Unit u;
  const int x = p.Hkv == 1 ? blockIdx.x : blockIdx.x / p.Hkv;
  if (!locate<KS>(p, x, smem, u)) return;
  u.h = (int)blockIdx.x - x * p.Hkv;
  if (warp == 9) pa::tmem_alloc(base + kMisc, kTmemCols);
  pa::tc_fence_before();
  __syncthreads();
  pa::tc_fence_after();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t *>(smem + kMisc);
  if (warp < kSoftWarps) {
    pa::regs_inc<216>();
    run_softmax(p, u, bars, tm, smem);
  } else {
    pa::regs_dec<72>();
    if (warp == 8)
      run_producer(p, u, base, bars);
    else if (warp == 9)
      run_mma(p, u, base, bars, tm);
    else
      run_clean(p, u, base, bars, smem);
  }
}

// ------------------------------------------------------------------------------- host

struct PromptDevice {
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
    for (const void *f : {(const void *)prompt_attn_kernel<1>, (const void *)prompt_attn_kernel<11>}) {
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
  if (!encode_rows(dev, &p.tm_q, a->q, a->num_rows, heads, a->q_stride, p.G, p.tokens) ||
      !encode_rows(dev, &p.tm_k, a->k, a->num_rows, a->num_kv_heads, a->k_stride, 1, kN) ||
      !encode_rows(dev, &p.tm_v, a->v, a->num_rows, a->num_kv_heads, a->v_stride, 1, kN))
    return PA_ERR_CUDA;
  // as many CTAs as there can be units: those without one exit
  const int64_t span = 2 * p.tokens, units = (n + a->num_seqs * (span - 1)) / span;
  const pa_host::Launch run(dim3((unsigned)(units * a->num_kv_heads)), dim3(kThreads), kSmem, stream);
  const cudaError_t e = a->num_seqs <= kThreads ? cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<1>, p)
                                                : cudaLaunchKernelEx(run.cfg(), prompt_attn_kernel<11>, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
