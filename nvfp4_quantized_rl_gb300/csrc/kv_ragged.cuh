// Packed rows of several sequences and the cache rows they belong to (the ragged append in quantize.cu, the read in
// kv_read.cu).
#pragma once

#include "common.cuh"

namespace nvfp4rl {

struct RaggedArgs {
  const int32_t* offsets;  // [B + 1]: sequence b has packed rows [offsets[b], offsets[b + 1])
  const int32_t* pos;      // [B] or null (0): cache row of its first one
  int64_t B, T, Lmax;
};

nvfp4rl_status launch_kv_append_ragged(const void* k, const void* v, int dtype, int64_t ldk, int64_t ldv, int64_t Hkv,
                                       int64_t D, const RaggedArgs& r, const float* gk, const float* gv, uint8_t* kc,
                                       uint8_t* ks, uint8_t* vc, uint8_t* vs, const DeviceInfo& dev, cudaStream_t st);
nvfp4rl_status launch_kv_read(const uint8_t* kc, const uint8_t* ks, const float* gk, const uint8_t* vc, const uint8_t* vs,
                              const float* gv, int64_t Hkv, int64_t D, const RaggedArgs& r, void* k, void* v, int dtype,
                              int64_t ldk, int64_t ldv, const DeviceInfo& dev, cudaStream_t st);

#ifdef __CUDACC__
constexpr int64_t kNoSequence = -1, kNoCacheRow = -2;

// Cache row (b Lmax + token) of packed row t; kNoSequence for rows of no sequence, kNoCacheRow for a place
// outside [0, Lmax). Sequences without rows are passed over. Any contents of offsets and pos give an answer within
// the cache.
__device__ __forceinline__ int64_t ragged_cache_row(const RaggedArgs& r, int64_t t) {
  int64_t lo = 0, hi = r.B + 1;  // how many offsets are at most t
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(r.offsets + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  if (lo == 0 || lo > r.B) return kNoSequence;
  const int64_t b = lo - 1;
  const int64_t at = t - __ldg(r.offsets + b) + (r.pos ? static_cast<int64_t>(__ldg(r.pos + b)) : int64_t(0));
  return at >= 0 && at < r.Lmax ? b * r.Lmax + at : kNoCacheRow;
}
#endif

}  // namespace nvfp4rl
