// Rows of an NVFP4 KV cache as bf16 or fp32 (sm_103a): value = E2M1 code x E4M3 block scale x g.
//
// Pure traffic: 0.5625 bytes in and 2 (4) out per element. A CTA takes eight packed rows, looks up their cache rows
// once, and walks their words of eight codes; a token's heads and blocks lie one after another in the cache and in the
// output alike, so that a word's place needs no head or block index. Code times scale is exact in f16 (at
// most six significant bits), the product with g is rounded to fp32 and, for bf16, from there.
#include "kv_ragged.cuh"

namespace nvfp4rl {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTile = 8;    // packed rows per CTA
constexpr int kReadAhead = 4;   // words in flight per thread

struct ReadArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const float *gk, *gv;
  void *k, *v;
  int64_t ldk, ldv;
  uint32_t words;  // words of eight codes in a token's row of K (or V): Hkv D / 8
  RaggedArgs r;
};

// Eight E2M1 codes times one E4M3 scale byte, exactly, as four f16 pairs (low half: the lower element).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&d)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 s;\n\t"
      "cvt.rn.f16x2.e4m3x2 s, %5;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
      "mul.rn.f16x2 %0, %0, s;\n\t"
      "mul.rn.f16x2 %1, %1, s;\n\t"
      "mul.rn.f16x2 %2, %2, s;\n\t"
      "mul.rn.f16x2 %3, %3, s;\n\t}"
      : "=&r"(d[0]), "=&r"(d[1]), "=&r"(d[2]), "=&r"(d[3])
      : "r"(w), "h"(static_cast<uint16_t>(scale | (scale << 8))));
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t p) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(p));
  return f;
}

template <int kDtype>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
  __shared__ int64_t rows[kReadTile];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kReadTile;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(kReadTile), a.r.T - t0));
  if (threadIdx.x < tokens) rows[threadIdx.x] = ragged_cache_row(a.r, t0 + threadIdx.x);
  __syncthreads();
  const float gk = __ldg(a.gk), gv = __ldg(a.gv);
  const uint32_t per = 2 * a.words, total = tokens * per;
  for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kReadAhead * kReadThreads) {
    uint32_t word[kReadAhead], scale[kReadAhead], at[kReadAhead], tok[kReadAhead];
    bool is_v[kReadAhead], live[kReadAhead];
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) {
      const uint32_t i = i0 + j * kReadThreads;
      tok[j] = i / per;
      const uint32_t u = i - tok[j] * per;
      is_v[j] = u >= a.words;
      at[j] = is_v[j] ? u - a.words : u;
      live[j] = i < total && rows[i < total ? tok[j] : 0] != kNoSequence;
      word[j] = scale[j] = 0;
      if (live[j] && rows[tok[j]] >= 0) {
        const int64_t w = rows[tok[j]] * a.words + at[j];
        word[j] = __ldg(reinterpret_cast<const uint32_t*>(is_v[j] ? a.vc : a.kc) + w);
        scale[j] = __ldg((is_v[j] ? a.vs : a.ks) + (w >> 1));
      }
    }
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) {
      if (!live[j]) continue;
      const float g = is_v[j] ? gv : gk;
      uint32_t h[4];
      decode8(word[j], scale[j], h);
      float2 f[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[q] = f16x2_floats(h[q]);
        f[q].x *= g;
        f[q].y *= g;
      }
      const int64_t e = (t0 + tok[j]) * (is_v[j] ? a.ldv : a.ldk) + static_cast<int64_t>(at[j]) * 8;
      if constexpr (kDtype == NVFP4RL_BF16) {
        uint4 o;
        o.x = pack_bf16x2(f[0].x, f[0].y);
        o.y = pack_bf16x2(f[1].x, f[1].y);
        o.z = pack_bf16x2(f[2].x, f[2].y);
        o.w = pack_bf16x2(f[3].x, f[3].y);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v[j] ? a.v : a.k) + e) = o;
      } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(is_v[j] ? a.v : a.k) + e);
        o[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        o[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
      }
    }
  }
}

}  // namespace

nvfp4rl_status launch_kv_read(const uint8_t* kc, const uint8_t* ks, const float* gk, const uint8_t* vc, const uint8_t* vs,
                              const float* gv, int64_t Hkv, int64_t D, const RaggedArgs& r, void* k, void* v, int dtype,
                              int64_t ldk, int64_t ldv, const DeviceInfo&, cudaStream_t st) {
  ReadArgs a{kc, ks, vc, vs, gk, gv, k, v, ldk, ldv, static_cast<uint32_t>(Hkv * D / 8), r};
  const dim3 grid(static_cast<unsigned>((r.T + kReadTile - 1) / kReadTile));
  const cudaError_t e = dtype == NVFP4RL_BF16 ? launch_pdl(kv_read_kernel<NVFP4RL_BF16>, grid, dim3(kReadThreads), 0, st, a)
                                              : launch_pdl(kv_read_kernel<NVFP4RL_F32>, grid, dim3(kReadThreads), 0, st, a);
  if (e != cudaSuccess) return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace nvfp4rl
