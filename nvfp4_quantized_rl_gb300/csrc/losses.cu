// Losses over packed token log-probs (sm_103a): the clipped policy loss with a KL term and the
// preference loss of paired log ratios, forward and backward. include/nvfp4rl.h states the formulas.
//
// All four stream a few fp32 arrays once, so HBM (or L2) bounds them. A warp takes a step of 256
// consecutive tokens (coalesced 4-byte loads at any alignment, eight per array in flight per lane) and
// walks the sequences that meet the step; it sums each one's tokens over its lanes and leaves the sums in the
// slot (step + sequence). A second kernel adds a sequence's slots in order, one warp to a sequence, and the
// CTA that finishes last joins the sequences. No floating-point atomics: equal inputs give equal bits.
//
// Ratios next to a bound: whether r = e^d lies above 1 + eps is decided as d > ln(1 + eps), with d the exact
// difference of the two log-probs (two floats, from one TwoSum) and the logarithm split into two floats, so
// that clipping does not depend on the rounding of d or of the exponential.
#include "losses.cuh"

namespace nvfp4rl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kPerLane = kLossStep / 32;

// a + b as a float and its rounding error, exactly (both finite).
__device__ __forceinline__ SplitFloat two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float v = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
// Sum of two split floats to about 44 bits.
__device__ __forceinline__ SplitFloat split_add(SplitFloat a, SplitFloat b) {
  const SplitFloat s = two_sum(a.hi, b.hi);
  if (!isfinite(s.hi)) return {s.hi, 0.0f};  // infinities add up to what they are; their tails would be NaN
  const float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s.hi, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, s.hi))};
}
__device__ __forceinline__ SplitFloat warp_sum_split(SplitFloat v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = split_add(v, SplitFloat{__shfl_xor_sync(0xFFFFFFFFu, v.hi, o), __shfl_xor_sync(0xFFFFFFFFu, v.lo, o)});
  return v;
}

__device__ __forceinline__ bool above(SplitFloat d, SplitFloat t) { return d.hi > t.hi || (d.hi == t.hi && d.lo > t.lo); }
__device__ __forceinline__ bool below(SplitFloat d, SplitFloat t) { return d.hi < t.hi || (d.hi == t.hi && d.lo < t.lo); }

// e^x - x - 1 >= 0: its power series up to x^9 below 1/2 (truncated at 2e-9 of the sum), where the
// difference would lose x's digits.
__device__ __forceinline__ float expm1_less(float x) {
  if (fabsf(x) >= 0.5f) return expm1f(x) - x;
  float p = fmaf(x, 1.0f / 362880.0f, 1.0f / 40320.0f);
  p = fmaf(x, p, 1.0f / 5040.0f);
  p = fmaf(x, p, 1.0f / 720.0f);
  p = fmaf(x, p, 1.0f / 120.0f);
  p = fmaf(x, p, 1.0f / 24.0f);
  p = fmaf(x, p, 1.0f / 6.0f);
  p = fmaf(x, p, 0.5f);
  return x * x * p;
}

// How many of offsets[0 .. count) are at most t: whole warp, 32 probes a round.
__device__ __forceinline__ int64_t count_up_to(const int32_t* __restrict__ offsets, int64_t count, int64_t t) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = count;  // the answer is in [lo, hi]
  while (hi > lo) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + lane * step;
    const bool le = at < hi && __ldg(offsets + at) <= t;
    const int hits = __popc(__ballot_sync(0xFFFFFFFFu, le));
    if (hits == 0) return lo;
    hi = min(hi, lo + hits * step);
    lo += (hits - 1) * step + 1;
  }
  return lo;
}

// The sequences of tokens [t0, t1), in order: f(b, s, e) for the part [s, e) that sequence b has of them;
// b = -1 for tokens of no sequence. Whole warp. Offsets that fall are answered with some split of the
// tokens, each in one part.
template <class F>
__device__ __forceinline__ void for_sequences(const int32_t* __restrict__ offsets, int64_t B, int64_t t0, int64_t t1,
                                              F&& f) {
  int64_t t = t0;
  while (t < t1) {
    const int64_t c = count_up_to(offsets, B + 1, t);
    const int64_t b = c > B ? -1 : c - 1;
    int64_t e = c > B ? t1 : min(t1, static_cast<int64_t>(__ldg(offsets + c)));
    e = max(e, t + 1);
    f(b, t, e);
    t = e;
  }
}

// ---- the policy loss ------------------------------------------------------------------------------------

// What one token of the policy loss gives: its clipped term -w min(..), the estimate e^x - x - 1 of the divergence
// from the reference, the gradient of term + kl estimate to logp, whether clipping took the term, r and e^d - d - 1.
struct Token {
  float term, div, grad, ratio, drift;
  bool clipped;
};

template <bool kGrad>
__device__ __forceinline__ Token policy_token(const PolicyArgs& a, float lp, float lo, float ref, float adv, float w) {
  Token t;
  const SplitFloat d = two_sum(lp, -lo);
  const float e = expf(d.hi);
  t.ratio = isfinite(d.hi) && isfinite(e) ? fmaf(e, d.lo, e) : e;
  const bool over = adv > 0.0f && above(d, a.ln_high);
  const bool under = adv < 0.0f && below(d, a.ln_low);
  const bool far = adv < 0.0f && above(d, a.ln_dual);
  t.clipped = over || under || far;
  const float used = far ? a.dual : over ? a.high : under ? a.low : t.ratio;
  t.term = adv == 0.0f ? 0.0f : -(w * (used * adv));
  t.grad = t.clipped ? 0.0f : t.term;
  t.div = 0.0f;
  if (a.logp_ref) {
    const float x = ref - lp;
    if constexpr (kGrad) t.grad = fmaf(-a.kl, expm1f(x), t.grad);
    else t.div = expm1_less(x);
  }
  if constexpr (!kGrad) t.drift = expm1_less(d.hi);
  return t;
}

// Slots and sequences hold the same eight floats. A slot: sums of term, div, drift and ratio, then the numbers of
// tokens and of clipped ones. A sequence: term and div as split floats, then drift, ratio and the two numbers.
struct SlotSums {
  float4 a, b;
};

__global__ void __launch_bounds__(kThreads) policy_sums_kernel(const PolicyArgs a, unsigned int* __restrict__ ticket,
                                                               SlotSums* __restrict__ slots) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0u;  // for the kernel behind this one
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  const int64_t t0 = s * kLossStep, t1 = min(a.n, t0 + kLossStep);
  if (t0 >= a.n) return;
  float lp[kPerLane], lo[kPerLane], ref[kPerLane], w[kPerLane], adv[kPerLane];
  bool live[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int64_t t = t0 + 32 * j + lane;
    const bool in = t < t1;
    live[j] = in && (!a.mask || __ldg(a.mask + t) != 0);
    lp[j] = in ? __ldg(a.logp + t) : 0.0f;
    lo[j] = in ? __ldg(a.logp_old + t) : 0.0f;
    ref[j] = a.logp_ref && in ? __ldg(a.logp_ref + t) : 0.0f;
    w[j] = a.weights && in ? __ldg(a.weights + t) : 1.0f;
    adv[j] = a.adv_per_token && in ? __ldg(a.adv + t) : 0.0f;
  }
  for_sequences(a.offsets, a.B, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    if (b < 0) return;
    const float seq_adv = a.adv_per_token ? 0.0f : __ldg(a.adv + b);
    float term = 0.0f, div = 0.0f, drift = 0.0f, ratio = 0.0f;
    uint32_t counts = 0;  // tokens, and clipped ones from bit 16 on: at most 256 of each
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int64_t t = t0 + 32 * j + lane;
      if (live[j] && t >= from && t < to) {
        const Token k = policy_token<false>(a, lp[j], lo[j], ref[j], a.adv_per_token ? adv[j] : seq_adv, w[j]);
        term += k.term;
        div += k.div;
        drift += k.drift;
        ratio += k.ratio;
        counts += k.clipped ? 0x10001u : 1u;
      }
    }
    counts = __reduce_add_sync(0xFFFFFFFFu, counts);
    term = warp_sum(term);
    div = warp_sum(div);
    drift = warp_sum(drift);
    ratio = warp_sum(ratio);
    if (lane == 0)
      slots[s + b] = {make_float4(term, div, drift, ratio),
                      make_float4(static_cast<float>(counts & 0xFFFFu), static_cast<float>(counts >> 16), 0.0f, 0.0f)};
  });
}

// Sums of sequence b's slots, in lanes' strides and then a tree: get(slot, i) is the i-th of kN numbers of a slot.
template <int kN, class Get>
__device__ __forceinline__ void sum_slots(const int32_t* __restrict__ offsets, int64_t n, int64_t b, SplitFloat (&v)[kN],
                                          Get&& get) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = {0.0f, 0.0f};
  const int64_t s = min(max(static_cast<int64_t>(__ldg(offsets + b)), int64_t(0)), n);
  const int64_t e = min(max(static_cast<int64_t>(__ldg(offsets + b + 1)), int64_t(0)), n);
  if (e <= s) return;
  for (int64_t k = s / kLossStep + (threadIdx.x & 31); k <= (e - 1) / kLossStep; k += 32) get(k + b, v);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = warp_sum_split(v[i]);
}

__global__ void __launch_bounds__(kThreads) policy_join_kernel(const PolicyArgs a, unsigned int* __restrict__ ticket,
                                                               const SlotSums* __restrict__ slots,
                                                               SlotSums* __restrict__ seqs) {
  __shared__ SplitFloat part[7][kWarpsPerCta];
  __shared__ int last;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarpsPerCta;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + warp; b < a.B; b += warps) {
    SplitFloat v[6];
    sum_slots<6>(a.offsets, a.n, b, v, [&](int64_t i, SplitFloat (&u)[6]) {
      const float4 x = __ldcg(&slots[i].a), y = __ldcg(&slots[i].b);
      const float z[6] = {x.x, x.y, x.z, x.w, y.x, y.y};
#pragma unroll
      for (int k = 0; k < 6; ++k) u[k] = split_add(u[k], {z[k], 0.0f});
    });
    if (lane == 0)
      seqs[b] = {make_float4(v[0].hi, v[0].lo, v[1].hi, v[1].lo), make_float4(v[2].hi, v[3].hi, v[4].hi, v[5].hi)};
  }
  __threadfence();  // this thread's sequences are visible before the CTA's ticket
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();  // and every other CTA's from here on
  // term, div, drift, ratio, tokens, clipped, sequences with a token
  SplitFloat v[7];
#pragma unroll
  for (int i = 0; i < 7; ++i) v[i] = {0.0f, 0.0f};
  for (int64_t b = threadIdx.x; b < a.B; b += kThreads) {
    const float4 x = __ldcg(&seqs[b].a), y = __ldcg(&seqs[b].b);
    SplitFloat term{x.x, x.y}, div{x.z, x.w};
    if (a.mode == NVFP4RL_LOSS_SEQ_MEAN) {
      const float len = fmaxf(y.z, 1.0f);
      term = {term.hi / len, term.lo / len};
      div = {div.hi / len, div.lo / len};
    }
    v[0] = split_add(v[0], term);
    v[1] = split_add(v[1], div);
    v[2] = split_add(v[2], {y.x, 0.0f});
    v[3] = split_add(v[3], {y.y, 0.0f});
    v[4] = split_add(v[4], {y.z, 0.0f});
    v[5] = split_add(v[5], {y.w, 0.0f});
    v[6] = split_add(v[6], {y.z > 0.0f ? 1.0f : 0.0f, 0.0f});
  }
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const SplitFloat t = warp_sum_split(v[i]);
    if (lane == 0) part[i][warp] = t;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    v[i] = part[i][0];
    for (int w = 1; w < kWarpsPerCta; ++w) v[i] = split_add(v[i], part[i][w]);
  }
  const float tokens = v[4].hi, there = v[6].hi, per_token = 1.0f / fmaxf(tokens, 1.0f);
  const float share = a.mode == NVFP4RL_LOSS_TOKEN_MEAN ? fmaxf(tokens, 1.0f)
                      : a.mode == NVFP4RL_LOSS_SEQ_MEAN ? fmaxf(there, 1.0f) : a.norm;
  if (threadIdx.x == 0) {
    const float policy = v[0].hi / share, div = v[1].hi / share;
    const float loss = a.logp_ref && a.kl != 0.0f ? fmaf(a.kl, div, policy) : policy;
    a.loss[0] = loss;
    if (a.stats) {
      a.stats[0] = loss;
      a.stats[1] = policy;
      a.stats[2] = div;
      a.stats[3] = v[5].hi * per_token;
      a.stats[4] = v[2].hi * per_token;
      a.stats[5] = v[3].hi * per_token;
      a.stats[6] = tokens;
      a.stats[7] = there;
    }
  }
  if (!a.coef) return;
  for (int64_t b = threadIdx.x; b < a.B; b += kThreads) {
    float c = 1.0f / share;
    if (a.mode == NVFP4RL_LOSS_SEQ_MEAN) c = 1.0f / (fmaxf(__ldcg(&seqs[b].b).z, 1.0f) * share);
    a.coef[b] = c;
  }
}

__global__ void __launch_bounds__(kThreads) policy_grad_kernel(const PolicyArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  const int64_t t0 = s * kLossStep, t1 = min(a.n, t0 + kLossStep);
  if (t0 >= a.n) return;
  const float dloss = a.dloss ? __ldg(a.dloss) : 1.0f;
  float lp[kPerLane], lo[kPerLane], ref[kPerLane], w[kPerLane], adv[kPerLane];
  bool live[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int64_t t = t0 + 32 * j + lane;
    const bool in = t < t1;
    live[j] = in && (!a.mask || __ldg(a.mask + t) != 0);
    lp[j] = in ? __ldg(a.logp + t) : 0.0f;
    lo[j] = in ? __ldg(a.logp_old + t) : 0.0f;
    ref[j] = a.logp_ref && in ? __ldg(a.logp_ref + t) : 0.0f;
    w[j] = a.weights && in ? __ldg(a.weights + t) : 1.0f;
    adv[j] = a.adv_per_token && in ? __ldg(a.adv + t) : 0.0f;
  }
  for_sequences(a.offsets, a.B, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    const float seq_adv = b < 0 || a.adv_per_token ? 0.0f : __ldg(a.adv + b);
    const float c = b < 0 ? 0.0f : dloss * __ldg(a.coef_in + b);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int64_t t = t0 + 32 * j + lane;
      if (t < from || t >= to) continue;
      float g = 0.0f;
      if (b >= 0 && live[j])
        g = c * policy_token<true>(a, lp[j], lo[j], ref[j], a.adv_per_token ? adv[j] : seq_adv, w[j]).grad;
      a.dlogp[t] = g;
    }
  });
}

// ---- the preference loss ----------------------------------------------------------------------------------

// A slot: the sum of logp - logp_ref over the counted tokens as a split float, and their number.
__global__ void __launch_bounds__(kThreads) preference_sums_kernel(const PreferenceArgs a, float4* __restrict__ slots) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  const int64_t t0 = s * kLossStep, t1 = min(a.n, t0 + kLossStep);
  if (t0 >= a.n) return;
  float lp[kPerLane], ref[kPerLane];
  bool live[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int64_t t = t0 + 32 * j + lane;
    const bool in = t < t1;
    live[j] = in && (!a.mask || __ldg(a.mask + t) != 0);
    lp[j] = in ? __ldg(a.logp + t) : 0.0f;
    ref[j] = a.logp_ref && in ? __ldg(a.logp_ref + t) : 0.0f;
  }
  for_sequences(a.offsets, 2 * a.pairs, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    if (b < 0) return;
    SplitFloat v{0.0f, 0.0f};
    uint32_t tokens = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int64_t t = t0 + 32 * j + lane;
      if (live[j] && t >= from && t < to) {
        SplitFloat d = two_sum(lp[j], -ref[j]);
        if (!isfinite(d.hi)) d.lo = 0.0f;
        v = split_add(v, d);
        ++tokens;
      }
    }
    v = warp_sum_split(v);
    tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
    if (lane == 0) slots[s + b] = make_float4(v.hi, v.lo, static_cast<float>(tokens), 0.0f);
  });
}

// One warp to a pair.
__global__ void __launch_bounds__(kThreads) preference_join_kernel(const PreferenceArgs a,
                                                                   const float4* __restrict__ slots) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t p = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  if (p >= a.pairs) return;
  SplitFloat total[2];
  float share[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    SplitFloat v[2];
    sum_slots<2>(a.offsets, a.n, 2 * p + side, v, [&](int64_t i, SplitFloat (&u)[2]) {
      const float4 x = __ldcg(slots + i);
      u[0] = split_add(u[0], {x.x, x.y});
      u[1] = split_add(u[1], {x.z, 0.0f});
    });
    total[side] = v[0];
    share[side] = 1.0f;
    if (a.mean) {
      // the quotient with what its rounding left
      const float len = fmaxf(v[1].hi, 1.0f), q = v[0].hi / len;
      total[side] = {q, isfinite(q) ? (fmaf(-q, len, v[0].hi) + v[0].lo) / len : 0.0f};
      share[side] = 1.0f / len;
    }
  }
  if ((threadIdx.x & 31) != 0) return;
  const SplitFloat d = split_add(total[0], {-total[1].hi, -total[1].lo});
  const float h = isfinite(d.hi) ? fmaf(a.beta, d.hi, fmaf(a.beta, d.lo, -a.margin)) : a.beta * d.hi - a.margin;
  // ln(1 + e^-|h|), sigma(|h|) and sigma(-|h|)
  const float e = expf(-fabsf(h)), tail = log1pf(e), big = 1.0f / (1.0f + e), small = e * big;
  const float lose = fmaxf(-h, 0.0f) + tail;  // -ln sigma(h)
  const float win = fmaxf(h, 0.0f) + tail;    // -ln sigma(-h)
  float loss = (1.0f - a.smoothing) * lose;
  if (a.smoothing > 0.0f) loss = fmaf(a.smoothing, win, loss);
  if (h != h) loss = h;
  a.loss[p] = loss;
  if (a.rewards) {
    a.rewards[2 * p] = fmaf(a.beta, total[0].hi, a.beta * total[0].lo);
    a.rewards[2 * p + 1] = fmaf(a.beta, total[1].hi, a.beta * total[1].lo);
  }
  if (a.coef) {
    const float up = h >= 0.0f ? big : small, down = h >= 0.0f ? small : big;  // sigma(h), sigma(-h)
    float slope = fmaf(a.smoothing, up, -(1.0f - a.smoothing) * down);
    if (h != h) slope = h;
    a.coef[2 * p] = a.beta * slope * share[0];
    a.coef[2 * p + 1] = -(a.beta * slope) * share[1];
  }
}

__global__ void __launch_bounds__(kThreads) preference_grad_kernel(const PreferenceArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  const int64_t t0 = s * kLossStep, t1 = min(a.n, t0 + kLossStep);
  if (t0 >= a.n) return;
  bool live[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int64_t t = t0 + 32 * j + lane;
    live[j] = t < t1 && (!a.mask || __ldg(a.mask + t) != 0);
  }
  for_sequences(a.offsets, 2 * a.pairs, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    const float c = b < 0 ? 0.0f : __ldg(a.coef_in + b) * (a.dloss ? __ldg(a.dloss + (b >> 1)) : 1.0f);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int64_t t = t0 + 32 * j + lane;
      if (t >= from && t < to) a.dlogp[t] = live[j] ? c : 0.0f;
    }
  });
}

dim3 warps_grid(int64_t warps) {
  return dim3(static_cast<unsigned>(std::max<int64_t>(1, (warps + kWarpsPerCta - 1) / kWarpsPerCta)));
}

}  // namespace

nvfp4rl_status launch_policy_loss(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  auto* ticket = static_cast<unsigned int*>(a.ws);
  auto* slots = reinterpret_cast<SlotSums*>(static_cast<uint8_t*>(a.ws) + 256);
  SlotSums* seqs = slots + loss_steps(a.n) + a.B;
  if (launch_pdl(policy_sums_kernel, warps_grid(loss_steps(a.n)), dim3(kThreads), 0, st, a, ticket, slots) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  if (launch_status() != NVFP4RL_OK) return NVFP4RL_ERR_CUDA;
  dim3 grid = warps_grid(a.B);
  grid.x = std::min(grid.x, static_cast<unsigned>(dev.sm_count) * 4u);
  if (launch_pdl(policy_join_kernel, grid, dim3(kThreads), 0, st, a, ticket, static_cast<const SlotSums*>(slots), seqs) !=
      cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

nvfp4rl_status launch_policy_loss_grad(const PolicyArgs& a, const DeviceInfo&, cudaStream_t st) {
  if (launch_pdl(policy_grad_kernel, warps_grid(loss_steps(a.n)), dim3(kThreads), 0, st, a) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

nvfp4rl_status launch_preference_loss(const PreferenceArgs& a, const DeviceInfo&, cudaStream_t st) {
  auto* slots = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.ws) + 256);
  if (a.n > 0) {
    if (launch_pdl(preference_sums_kernel, warps_grid(loss_steps(a.n)), dim3(kThreads), 0, st, a, slots) != cudaSuccess)
      return NVFP4RL_ERR_CUDA;
    if (launch_status() != NVFP4RL_OK) return NVFP4RL_ERR_CUDA;
  }
  if (launch_pdl(preference_join_kernel, warps_grid(a.pairs), dim3(kThreads), 0, st, a,
                 static_cast<const float4*>(slots)) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

nvfp4rl_status launch_preference_loss_grad(const PreferenceArgs& a, const DeviceInfo&, cudaStream_t st) {
  if (launch_pdl(preference_grad_kernel, warps_grid(loss_steps(a.n)), dim3(kThreads), 0, st, a) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace nvfp4rl
