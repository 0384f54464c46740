// Log-probs of given tokens, entropy and top alternatives of rows of logits, and the divergence from a
// teacher's listed log-probs (sm_103a). One CTA per row.
#include "logits.cuh"

namespace nvfp4rl {
namespace {

constexpr int kThreads = 256;

__device__ float block_max(float v, float* red) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kThreads / 32; ++i) v = fmaxf(v, red[i]);
  __syncthreads();
  return v;
}

__device__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) v += red[i];
  __syncthreads();
  return v;
}

// Order of the alternatives as one integer: larger value first, then the lower column (-0 = +0).
__device__ unsigned long long rank_key(float v, int64_t col) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t u = (b >> 31) ? ~b : (b | 0x80000000u);
  return (static_cast<unsigned long long>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(col));
}

template <typename T, bool kDistill>
__global__ void __launch_bounds__(kThreads) logits_row_kernel(const LogitsArgs a) {
  __shared__ float red[kThreads / 32];
  __shared__ int32_t ids_s[kMaxListed];
  __shared__ float q_s[kMaxListed], lq_s[kMaxListed];
  __shared__ TeacherRow teacher_s;
  __shared__ unsigned long long best;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  const int tid = threadIdx.x;
  int64_t token = -1;
  if (kDistill) {
    if (tid < 32) {
      const TeacherRow t = teacher_row(a.ids + row * a.k, a.teacher + row * a.k, a.k, a.V, a.tail, ids_s, q_s, lq_s);
      if (tid == 0) teacher_s = t;
    }
    __syncthreads();
    if (!teacher_s.any) {
      if (tid == 0) {
        a.loss[row] = 0.0f;
        if (a.lse) a.lse[row] = 0.0f;
        if (a.tail && a.lse_tail) a.lse_tail[row] = 0.0f;
      }
      return;
    }
  } else if (a.tokens) {
    token = a.tokens[row];
    if (token < 0 || token >= a.V) {
      if (tid == 0) {
        if (a.logp) a.logp[row] = 0.0f;
        if (a.entropy) a.entropy[row] = 0.0f;
        if (a.lse) a.lse[row] = 0.0f;
      }
      for (int i = tid; i < a.k; i += kThreads) {
        a.top_ids[row * a.k + i] = -1;
        a.top_logp[row * a.k + i] = -INFINITY;
      }
      return;
    }
  }
  const float c = a.scale * kLog2E;
  // the sums run over the columns that are not listed apart (TAIL), relative to their own maximum: a tail
  // far below the row's maximum keeps its digits
  const auto apart = [&](int64_t j) {
    bool in = false;
    if (kDistill && a.tail)
      for (int i = 0; i < a.k; ++i) in |= ids_s[i] == j;
    return in;
  };
  float m = -kLogitBound;
  bool nan = false;
  for (int64_t j = tid; j < a.V; j += kThreads) {
    const float v = logit(x, j);
    nan |= v != v || v > kLogitBound;
    if (!apart(j)) m = fmaxf(m, v);
  }
  nan = __syncthreads_or(nan);
  m = block_max(m, red);
  const float R = m * c;
  float s = 0.0f, w = 0.0f;
  for (int64_t j = tid; j < a.V; j += kThreads) {
    const float v = logit(x, j);
    if (v <= -kLogitBound || apart(j)) continue;
    const float t = fmaf(v, c, -R), e = exp2_approx(t);
    s += e;
    w = fmaf(e, t, w);
  }
  s = block_sum(s, red);
  w = block_sum(w, red);
  if (nan) s = NAN;
  if (kDistill) {
    const float s_tail = s;
    float m2 = m;
    if (a.tail) {
      for (int i = tid; i < a.k; i += kThreads)
        if (ids_s[i] >= 0) m2 = fmaxf(m2, logit(x, ids_s[i]));
      m2 = block_max(m2, red);
    }
    const float R2 = m2 * c, down = R - R2;
    if (a.tail) {
      float more = 0.0f;
      for (int i = tid; i < a.k; i += kThreads) {
        bool first = ids_s[i] >= 0;
        for (int j = 0; j < i; ++j) first &= ids_s[j] != ids_s[i];
        if (!first) continue;
        const float v = logit(x, ids_s[i]);
        if (v > -kLogitBound) more += exp2_approx(fmaf(v, c, -R2));
      }
      s = fmaf(s_tail, exp2_approx(down), block_sum(more, red));
    }
    const bool empty = s == 0.0f;
    const float ln_s = logf(s), ln_tail = logf(s_tail);
    float part = 0.0f;
    for (int i = tid; i < a.k; i += kThreads) {
      if (ids_s[i] < 0 || q_s[i] == 0.0f) continue;
      const float v = logit(x, ids_s[i]);
      const float lp = empty || v <= -kLogitBound ? -INFINITY : fmaf(v, c, -R2) * kLn2 - ln_s;
      part += q_s[i] * (lq_s[i] - lp);
    }
    part = block_sum(part, red);
    if (tid == 0) {
      if (a.tail && teacher_s.q0 > 0.0f && s_tail > 0.0f)
        part += teacher_s.q0 * (logf(teacher_s.q0) - (fmaf(down, kLn2, ln_tail) - ln_s));
      a.loss[row] = s != s ? NAN : part;
      if (a.lse) a.lse[row] = empty ? -INFINITY : fmaf(R2, kLn2, ln_s);
      if (a.tail && a.lse_tail) a.lse_tail[row] = s_tail == 0.0f ? -INFINITY : fmaf(R, kLn2, ln_tail);
    }
    return;
  }
  const bool empty = s == 0.0f;
  const float ln_s = logf(s);
  const float lse = empty ? -INFINITY : fmaf(R, kLn2, ln_s);
  if (tid == 0) {
    if (a.logp) {
      const float v = logit(x, token);
      a.logp[row] = s != s ? NAN : empty || v <= -kLogitBound ? -INFINITY : fmaf(v, c, -R) * kLn2 - ln_s;
    }
    if (a.entropy) {
      const float h = empty ? 0.0f : ln_s - kLn2 * (w / s);
      a.entropy[row] = h < 0.0f ? 0.0f : h;
    }
    if (a.lse) a.lse[row] = lse;
  }
  unsigned long long prev = ~0ull;
  for (int i = 0; i < a.k; ++i) {
    if (tid == 0) best = 0;
    __syncthreads();
    unsigned long long b = 0;
    if (s == s)
      for (int64_t j = tid; j < a.V; j += kThreads) {
        const float v = logit(x, j);
        const unsigned long long key = v > -kLogitBound ? rank_key(v, j) : 0ull;
        if (key < prev && key > b) b = key;
      }
    atomicMax(&best, b);
    __syncthreads();
    prev = best;
    if (tid == 0) {
      const int32_t id = prev ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(prev)) : -1;
      a.top_ids[row * a.k + i] = id;
      a.top_logp[row * a.k + i] =
          s != s ? NAN : id < 0 ? -INFINITY : fmaf(logit(x, id), c, -R) * kLn2 - ln_s;
    }
    __syncthreads();
  }
}

template <typename T, bool kDistill>
nvfp4rl_status launch(const LogitsArgs& a, cudaStream_t st) {
  if (launch_pdl(logits_row_kernel<T, kDistill>, dim3(static_cast<unsigned>(a.M)), dim3(kThreads), 0, st, a) !=
      cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace

nvfp4rl_status launch_logprobs(const LogitsArgs& a, int dtype, const DeviceInfo&, cudaStream_t st) {
  const bool distill = a.ids != nullptr;
  if (dtype == NVFP4RL_BF16) return distill ? launch<uint16_t, true>(a, st) : launch<uint16_t, false>(a, st);
  return distill ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace nvfp4rl
