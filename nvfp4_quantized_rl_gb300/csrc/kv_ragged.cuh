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
constexpr int kRaggedThreads = 256;

// How many of the offsets are at most t: by one thread, or by 32 lanes together (a 33-way search: latency for few rows).
__device__ __forceinline__ int64_t offsets_passed(const RaggedArgs& r, int64_t t) {
  int64_t lo = 0, hi = r.B + 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(r.offsets + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int64_t offsets_passed_warp(const RaggedArgs& r, int64_t t) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = r.B + 1;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) >> 5, at = lo + (lane + 1) * step - 1;
    const bool passed = at < hi && __ldg(r.offsets + at) <= t;
    lo += __popc(__ballot_sync(0xFFFFFFFFu, passed)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Cache row (b Lmax + token) of packed row t, which `passed` offsets are at most; kNoSequence for rows of no sequence,
// kNoCacheRow for a place outside [0, Lmax). Sequences without rows are passed over. Any contents of offsets and pos give
// an answer within the cache.
__device__ __forceinline__ int64_t ragged_cache_row(const RaggedArgs& r, int64_t t, int64_t passed) {
  if (passed == 0 || passed > r.B) return kNoSequence;
  const int64_t b = passed - 1;
  const int64_t at = t - __ldg(r.offsets + b) + (r.pos ? static_cast<int64_t>(__ldg(r.pos + b)) : int64_t(0));
  return at >= 0 && at < r.Lmax ? b * r.Lmax + at : kNoCacheRow;
}

// The cache rows of packed rows t0 .. t0 + n - 1, n at most kRaggedThreads, by a CTA of that many threads, for all of it
// (a barrier on both sides).
__device__ __forceinline__ void ragged_cache_rows(const RaggedArgs& r, int64_t t0, int n, int64_t* rows) {
  __syncthreads();
  if (n <= kRaggedThreads / 32) {
    const int i = threadIdx.x >> 5;
    if (i < n) {
      const int64_t passed = offsets_passed_warp(r, t0 + i);
      if ((threadIdx.x & 31) == 0) rows[i] = ragged_cache_row(r, t0 + i, passed);
    }
  } else if (threadIdx.x < n) {
    rows[threadIdx.x] = ragged_cache_row(r, t0 + threadIdx.x, offsets_passed(r, t0 + threadIdx.x));
  }
  __syncthreads();
}
#endif

}  // namespace nvfp4rl
