// Argument blocks and launchers of the loss operators (losses.cu).
#pragma once

#include "common.cuh"

namespace nvfp4rl {

// Tokens per warp step of the loss kernels. Each (step, sequence) pair that shares a token has a slot of
// partial sums of its own, at index step + sequence: both only grow along the packed tokens, so the
// ceil(n / kLossStep) + sequences slots suffice.
constexpr int kLossStep = 256;

inline int64_t loss_steps(int64_t n) { return (n + kLossStep - 1) / kLossStep; }
// Policy loss: 256 bytes for the ticket, then 32 bytes per slot and per sequence. Preference loss: 16 per slot.
inline size_t policy_workspace_bytes(int64_t n, int64_t B) {
  return 256 + static_cast<size_t>(loss_steps(n) + 2 * B) * 32;
}
inline size_t preference_workspace_bytes(int64_t n, int64_t pairs) {
  return 256 + static_cast<size_t>(loss_steps(n) + 2 * pairs) * 16;
}

// A real number as the sum of two floats.
struct SplitFloat {
  float hi, lo;
};

struct PolicyArgs {
  const float *logp, *logp_old, *logp_ref, *adv, *weights;
  const uint8_t* mask;
  const int32_t* offsets;
  int64_t n, B;
  bool adv_per_token;
  SplitFloat ln_low, ln_high, ln_dual;  // ln(1 - eps_low), ln(1 + eps_high), ln c (c = 0: +inf)
  float low, high, dual;                // 1 - eps_low, 1 + eps_high, c
  float kl;
  int mode;
  float norm;
  // forward
  float *loss, *stats, *coef;
  void* ws;
  // backward
  const float *coef_in, *dloss;
  float* dlogp;
};

struct PreferenceArgs {
  const float *logp, *logp_ref;
  const uint8_t* mask;
  const int32_t* offsets;
  int64_t n, pairs;
  float beta, margin, smoothing;
  bool mean;
  float *loss, *rewards, *coef;
  void* ws;
  const float *coef_in, *dloss;
  float* dlogp;
};

nvfp4rl_status launch_policy_loss(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st);
nvfp4rl_status launch_policy_loss_grad(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st);
nvfp4rl_status launch_preference_loss(const PreferenceArgs& a, const DeviceInfo& dev, cudaStream_t st);
nvfp4rl_status launch_preference_loss_grad(const PreferenceArgs& a, const DeviceInfo& dev, cudaStream_t st);

}  // namespace nvfp4rl
