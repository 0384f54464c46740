// Rows of an NVFP4 KV cache as bf16 or fp32 (sm_103a): value = E2M1 code x E4M3 block scale x g.
//
// Pure traffic: 0.5625 bytes in and 2 (4) out per element. Each CTA of one wave takes an equal stretch of the packed rows
// of K or V, looks up their cache rows once, and walks their pieces of 8 (4) codes, 16 bytes of output each; a token's heads
// and blocks lie one after another in the cache and in the output alike, so that a piece's place needs no head or block
// index. Code times scale is exact in f16 (at most six significant bits), the product with g is rounded to fp32 and, for
// bf16, from there.
//
// 65536 rows of 8 heads of 128 to bf16 take 60 us and 30000 to fp32 50 us, 0.85 and 0.82 of the measured copy bandwidth;
// with a CTA for each eight rows and divisions for each piece 64 us. Five CTAs of four pieces in flight a thread hide the
// loads; four of eight take 63 us.
#include <algorithm>

#include "kv_ragged.cuh"

namespace nvfp4rl {
namespace {

constexpr int kReadCtas = 5;   // per SM
constexpr int kMinRows = 2;    // of a CTA, where there are as many
constexpr int kReadAhead = 4;  // pieces in flight per thread

struct ReadArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const float *gk, *gv;
  void *k, *v;
  int64_t ldk, ldv;
  uint32_t pieces;  // of a token's row of K (or V)
  RaggedArgs r;
};

// Four E2M1 codes times one E4M3 scale byte, exactly, as two f16 pairs (low half: the lower element).
__device__ __forceinline__ void decode4(uint32_t w, uint32_t scale, uint32_t (&d)[2]) {
  asm("{\n\t.reg .b8 b0, b1;\n\t.reg .b32 s;\n\t"
      "cvt.rn.f16x2.e4m3x2 s, %3;\n\t"
      "mov.b16 {b0, b1}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "mul.rn.f16x2 %0, %0, s;\n\t"
      "mul.rn.f16x2 %1, %1, s;\n\t}"
      : "=&r"(d[0]), "=&r"(d[1])
      : "h"(static_cast<uint16_t>(w)), "h"(static_cast<uint16_t>(scale | (scale << 8))));
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t p) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(p));
  return f;
}

template <int kDtype>
__global__ void __launch_bounds__(kRaggedThreads, kReadCtas) kv_read_kernel(const ReadArgs a) {
  __shared__ int64_t rows[kRaggedThreads];
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const uint8_t *codes = is_v ? a.vc : a.kc, *scales = is_v ? a.vs : a.ks;
  const float g = __ldg(is_v ? a.gv : a.gk);
  const int64_t ld = is_v ? a.ldv : a.ldk;
  constexpr int kCodes = kDtype == NVFP4RL_BF16 ? 8 : 4;
  const uint32_t pieces = a.pieces, step_tok = kRaggedThreads / pieces, step_at = kRaggedThreads - step_tok * pieces;
  const int64_t end = a.r.T * (blockIdx.x + 1) / gridDim.x;
  for (int64_t t0 = a.r.T * blockIdx.x / gridDim.x; t0 < end; t0 += kRaggedThreads) {
    const uint32_t n = static_cast<uint32_t>(min(static_cast<int64_t>(kRaggedThreads), end - t0));
    ragged_cache_rows(a.r, t0, n, rows);
    uint32_t tok = threadIdx.x / pieces, at = threadIdx.x - tok * pieces;  // the thread's next piece: at in tok's row
    while (tok < n) {
      uint32_t word[kReadAhead], scale[kReadAhead], out_at[kReadAhead], out_tok[kReadAhead];
      bool live[kReadAhead];
#pragma unroll
      for (int j = 0; j < kReadAhead; ++j) {
        const int64_t row = tok < n ? rows[tok] : kNoSequence;
        out_tok[j] = tok;
        out_at[j] = at;
        live[j] = row != kNoSequence;
        word[j] = scale[j] = 0;
        if (row >= 0) {
          const int64_t w = row * pieces + at;
          if constexpr (kCodes == 8) word[j] = __ldg(reinterpret_cast<const uint32_t*>(codes) + w);
          else word[j] = __ldg(reinterpret_cast<const uint16_t*>(codes) + w);
          scale[j] = __ldg(scales + w / (16 / kCodes));
        }
        tok += step_tok;
        at += step_at;
        if (at >= pieces) {
          at -= pieces;
          ++tok;
        }
      }
#pragma unroll
      for (int j = 0; j < kReadAhead; ++j) {
        if (!live[j]) continue;
        float2 f[kCodes / 2];
#pragma unroll
        for (int q = 0; q < kCodes / 4; ++q) {
          uint32_t h[2];
          decode4(word[j] >> (16 * q), scale[j], h);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 x = f16x2_floats(h[i]);
            f[2 * q + i] = make_float2(x.x * g, x.y * g);
          }
        }
        const int64_t e = (t0 + out_tok[j]) * ld + static_cast<int64_t>(out_at[j]) * kCodes;
        if constexpr (kDtype == NVFP4RL_BF16) {
          uint4 o;
          o.x = pack_bf16x2(f[0].x, f[0].y);
          o.y = pack_bf16x2(f[1].x, f[1].y);
          o.z = pack_bf16x2(f[2].x, f[2].y);
          o.w = pack_bf16x2(f[3].x, f[3].y);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v : a.k) + e) = o;
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(is_v ? a.v : a.k) + e) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        }
      }
    }
  }
}

}  // namespace

nvfp4rl_status launch_kv_read(const uint8_t* kc, const uint8_t* ks, const float* gk, const uint8_t* vc, const uint8_t* vs,
                              const float* gv, int64_t Hkv, int64_t D, const RaggedArgs& r, void* k, void* v, int dtype,
                              int64_t ldk, int64_t ldv, const DeviceInfo& dev, cudaStream_t st) {
  ReadArgs a{kc, ks, vc, vs, gk, gv, k, v, ldk, ldv, static_cast<uint32_t>(Hkv * D / (dtype == NVFP4RL_BF16 ? 8 : 4)), r};
  const int64_t wave = static_cast<int64_t>(dev.sm_count) * kReadCtas / 2;
  const dim3 grid(static_cast<unsigned>(std::min((r.T + kMinRows - 1) / kMinRows, wave)), 2);
  const cudaError_t e = dtype == NVFP4RL_BF16 ? launch_pdl(kv_read_kernel<NVFP4RL_BF16>, grid, dim3(kRaggedThreads), 0, st, a)
                                              : launch_pdl(kv_read_kernel<NVFP4RL_F32>, grid, dim3(kRaggedThreads), 0, st, a);
  if (e != cudaSuccess) return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace nvfp4rl
