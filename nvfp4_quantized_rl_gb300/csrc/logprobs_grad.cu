// Gradients of the token log-probs, the entropy and the top-k distillation loss to the logits (sm_103a).
// Elementwise given the forward call's lse; one CTA per row.
#include "logits.cuh"

namespace nvfp4rl {
namespace {

constexpr int kThreads = 256;

template <typename T, bool kDistill>
__global__ void __launch_bounds__(kThreads) logits_grad_kernel(const LogitsGradArgs a) {
  __shared__ int32_t ids_s[kMaxListed];
  __shared__ float q_s[kMaxListed], lq_s[kMaxListed];
  __shared__ TeacherRow teacher_s;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  T* dx = static_cast<T*>(a.dx) + row * a.ldd;
  const int tid = threadIdx.x;
  const float c = a.scale * kLog2E;
  const float lse = a.lse[row];
  bool dead = lse == -INFINITY;
  int64_t token = -1;
  // p_j (alpha + beta t_j), t_j = log2 p_j, and `hit` more at the token
  float alpha = 0.0f, beta = 0.0f, hit = 0.0f, R = lse * kLog2E, mass = 0.0f;
  if (kDistill) {
    if (tid < 32) {
      const TeacherRow t = teacher_row(a.ids + row * a.k, a.teacher + row * a.k, a.k, a.V, a.tail, ids_s, q_s, lq_s);
      if (tid == 0) teacher_s = t;
    }
    __syncthreads();
    const float d = a.dloss[row] * a.scale;
    dead |= !teacher_s.any || a.dloss[row] == 0.0f;
    hit = d;
    mass = teacher_s.mass;
    alpha = mass * d;
    if (a.tail) {
      const float rest = a.lse_tail[row];
      if (rest == -INFINITY) {
        mass -= teacher_s.q0;
        alpha = 0.0f;
      } else {
        // (Q - q0 / p0) p = (Q p0 - q0) exp(z - lse_tail): nothing overflows for a tiny p0
        alpha = (mass * expf(rest - lse) - teacher_s.q0) * d;
        R = rest * kLog2E;
      }
    }
  } else {
    if (a.tokens) {
      token = a.tokens[row];
      dead |= token < 0 || token >= a.V;
    }
    const float dl = a.dlogp ? a.dlogp[row] : 0.0f, dh = a.dentropy ? a.dentropy[row] : 0.0f;
    dead |= dl == 0.0f && dh == 0.0f;
    hit = dl * a.scale;
    alpha = -a.scale * (a.dentropy ? fmaf(dh, a.entropy[row], dl) : dl);
    beta = -a.scale * dh * kLn2;
  }
  for (int64_t j = tid; j < a.V; j += kThreads) {
    float g = 0.0f;
    if (!dead) {
      const float v = fmaxf(logit(x, j), -kLogitBound);
      const float t = fmaf(v, c, -R), e = v <= -kLogitBound ? 0.0f : exp2_approx(t);
      g = e * fmaf(beta, t, alpha);
      if (j == token) g += hit;
      if (kDistill) {
        float q = 0.0f;
        bool in = false;
        for (int i = 0; i < a.k; ++i)
          if (ids_s[i] == j) {
            q += q_s[i];
            in = true;
          }
        if (in) g = hit * ((v <= -kLogitBound ? 0.0f : mass * exp2_approx(fmaf(v, c, -lse * kLog2E))) - q);
      }
      if (lse != lse) g = NAN;
    }
    store_logit(dx, j, g);
  }
}

template <typename T, bool kDistill>
nvfp4rl_status launch(const LogitsGradArgs& a, cudaStream_t st) {
  if (launch_pdl(logits_grad_kernel<T, kDistill>, dim3(static_cast<unsigned>(a.M)), dim3(kThreads), 0, st, a) !=
      cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace

nvfp4rl_status launch_logprobs_grad(const LogitsGradArgs& a, int dtype, const DeviceInfo&, cudaStream_t st) {
  const bool distill = a.ids != nullptr;
  if (dtype == NVFP4RL_BF16) return distill ? launch<uint16_t, true>(a, st) : launch<uint16_t, false>(a, st);
  return distill ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace nvfp4rl
