// pa_host.cuh -- host-side argument checks shared by the cache operators (pa_mass.cu,
// pa_evict.cu, pa_beam.cu).
#pragma once

#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "pa.h"

namespace pa_host {

constexpr int kD = 128;           // head_dim
constexpr int kMaxHeads = 64;     // KV heads
constexpr int kMaxDevices = 64;   // devices whose kernel attributes are tracked

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int log2_page(int ps) {
  switch (ps) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

// The cache's shape and mode: the limits every operator on it shares.
inline pa_status_t check_cache(int64_t num_pages, int num_kv_heads, int head_dim, int page_size,
                               int kv_dtype, int scale_mode) {
  if (num_pages < 1 || num_kv_heads < 1) return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_FP8_E4M3 && kv_dtype != PA_KV_BF16) return PA_ERR_INVALID_ARG;
  if (num_kv_heads > kMaxHeads || head_dim != kD || log2_page(page_size) < 0) return PA_ERR_UNSUPPORTED;
  if (kv_dtype == PA_KV_FP8_E4M3 ? (scale_mode != PA_SCALE_SCALAR && scale_mode != PA_SCALE_PER_TOKEN)
                                 : scale_mode != PA_SCALE_NONE)
    return PA_ERR_UNSUPPORTED;
  if (num_pages > INT32_MAX / ((int64_t)num_kv_heads * page_size)) return PA_ERR_CAPACITY;
  return PA_OK;
}

// A launch configuration: with programmatic dependent launch (each of these kernels begins with
// griddepcontrol.wait, so that only its launch overlaps the end of the kernel before it), and with
// clusters of `cluster` CTAs where that is more than 0.
class Launch {
 public:
  Launch(dim3 grid, dim3 block, size_t smem, void *stream, int cluster = 0) {
    cfg_.gridDim = grid;
    cfg_.blockDim = block;
    cfg_.dynamicSmemBytes = smem;
    cfg_.stream = static_cast<cudaStream_t>(stream);
    attr_[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr_[0].val.programmaticStreamSerializationAllowed = 1;
    attr_[1].id = cudaLaunchAttributeClusterDimension;
    attr_[1].val.clusterDim.x = cluster;
    attr_[1].val.clusterDim.y = attr_[1].val.clusterDim.z = 1;
    cfg_.attrs = attr_;
    cfg_.numAttrs = cluster > 0 ? 2 : 1;
  }
  const cudaLaunchConfig_t *cfg() const { return &cfg_; }

 private:
  cudaLaunchConfig_t cfg_ = {};
  cudaLaunchAttribute attr_[2] = {};
};

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// The memory of one tensor of a call; absent ones have no bytes.
struct Span {
  const void *p;
  uint64_t n;
};
// Whether an output shares a byte with one of the call's other tensors: several CTAs read what others write, in no order.
inline bool overlaps(const Span &out, std::initializer_list<Span> others) {
  if (out.p == nullptr || out.n == 0) return false;
  for (const Span &o : others)
    if (o.p != nullptr && o.n != 0 && overlap(out.p, out.n, o.p, o.n)) return true;
  return false;
}

}  // namespace pa_host
