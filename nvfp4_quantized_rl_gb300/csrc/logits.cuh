// Shared pieces of the logits operators (logprobs.cu, logprobs_grad.cu).
#pragma once

#include "common.cuh"

namespace nvfp4rl {

// A logit at or below -2^100 is masked (p = 0); one above 2^100 (or NaN) spoils its row. With scale
// within [2^-20, 2^20] every product scale * log2(e) * x of the others stays finite.
constexpr float kLogitBound = 1.2676506002282294e30f;  // 2^100
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLog2ELow = 1.9259629911e-8f;  // log2 e - kLog2E
constexpr float kLn2 = 0.6931471805599453f;
// Columns: a thread's fp32 sum then has at most 16384 terms per lane (in CTAs of 128 threads; of 256: 8192).
constexpr int64_t kMaxVocab = int64_t(1) << 22;
constexpr int kMaxListed = 256;  // alternatives or listed teacher columns per row

// 2^x (ex2.approx: about 2 ulp; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float logit(const uint16_t* x, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(x[i]) << 16);
}
__device__ __forceinline__ float logit(const float* x, int64_t i) { return x[i]; }
__device__ __forceinline__ void store_logit(uint16_t* y, int64_t i, float v) {
  y[i] = static_cast<uint16_t>(f32_to_bf16_bits(v));
}
__device__ __forceinline__ void store_logit(float* y, int64_t i, float v) { y[i] = v; }

// Two fp32 values in one 64-bit register, for the packed fp32 instructions (one issue for two results).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// 16 bytes of logits, not kept in L1 (each is used once). An ordinary load: a gradient may lie over them.
__device__ __forceinline__ uint4 ld_logits16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Logits per 16-byte vector, and the element of a vector at which the row at p starts.
template <typename T>
constexpr int kVecOf = 16 / static_cast<int>(sizeof(T));
template <typename T>
__device__ __forceinline__ int vec_phase(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % kVecOf<T>);
}

struct LogitsArgs {
  const void* x;
  int64_t M, V, ld;
  float scale;
  // log-probs
  const int32_t* tokens;
  int k;
  float *logp, *entropy, *lse;
  int32_t* top_ids;
  float* top_logp;
  // distillation: k listed columns per row
  const int32_t* ids;
  const float* teacher;
  bool tail;
  float *loss, *lse_tail;
};

struct LogitsGradArgs {
  const void* x;
  int64_t M, V, ld;
  float scale;
  const int32_t* tokens;
  const float *lse, *entropy, *dlogp, *dentropy;
  const int32_t* ids;
  const float* teacher;
  int k;
  bool tail;
  const float *lse_tail, *dloss;
  void* dx;
  int64_t ldd;
  float low;  // set by the launch
};

nvfp4rl_status launch_logprobs(const LogitsArgs& a, int dtype, const DeviceInfo& dev, cudaStream_t st);
nvfp4rl_status launch_logprobs_grad(const LogitsGradArgs& a, int dtype, const DeviceInfo& dev, cudaStream_t st);

// ---- a teacher's row, one entry to a thread of a CTA of kW warps ----

constexpr int kListWarps = 8;  // of the widest CTA
static_assert(32 * kListWarps >= kMaxListed, "one thread per listed column");

// Block reductions with one barrier each; `red` (kW values of its own for every use in a row) is free again
// after the CTA's next barrier.
template <int kW>
__device__ __forceinline__ float cta_max(float v, float* red) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) v = fmaxf(v, red[i]);
  return v;
}
template <int kW>
__device__ __forceinline__ float2 cta_sum(float2 v, float2* red) {
  v = make_float2(warp_sum(v.x), warp_sum(v.y));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kW; ++i) v = make_float2(v.x + red[i].x, v.y + red[i].y);
  return v;
}

// The bucket's mass and Q = sum q + q_0. `any`: an entry counts (NORMALIZED: one above -inf).
struct TeacherRow {
  float q0, mass;
  bool any;
};

struct TeacherShared {
  float top[kListWarps];
  float2 sum[kListWarps];
};

// This thread's entry: column id (-1: none, or skipped) with log-prob l; gives its q and ln q. All threads call.
// 1 - sum q would lose the digits of a small rest in 32 bits: the largest q enters as -expm1(l).
template <int kW>
__device__ __forceinline__ TeacherRow teacher_row(TeacherShared& sh, int id, float l, bool tail, float& q, float& lq) {
  const bool counts = id >= 0;
  // a NaN hides from the maximum, and shows in the sums
  const float top = cta_max<kW>(counts ? l : -INFINITY, sh.top);
  if (!tail) {
    q = counts && l != -INFINITY ? expf(l - top) : 0.0f;
    const float total = cta_sum<kW>(make_float2(q, 0.0f), sh.sum).x;
    q /= total;
    lq = (l - top) - logf(total);
    return TeacherRow{0.0f, total != total ? NAN : 1.0f, total != 0.0f};
  }
  q = counts ? expf(l) : 0.0f;
  lq = l;
  // the others' sum, and how many hold the largest
  const float2 sum = cta_sum<kW>(make_float2(l == top ? 0.0f : q, counts && l == top ? 1.0f : 0.0f), sh.sum);
  const float largest = expf(top), others = fmaf(fmaxf(sum.y - 1.0f, 0.0f), largest, sum.x);
  const float rest = -expm1f(top) - others, q0 = rest < 0.0f ? 0.0f : rest;
  return TeacherRow{q0, (largest + others) + q0, true};
}

}  // namespace nvfp4rl
