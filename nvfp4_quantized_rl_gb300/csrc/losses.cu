// Losses over packed token log-probs (sm_103a): the clipped policy loss with a KL term and the
// preference loss of paired log ratios, forward and backward. include/nvfp4rl.h states the formulas.
//
// All four stream a few fp32 arrays once, so HBM (or L2) would bound them; the policy loss's arithmetic, some 110 instructions
// a token, half of them compares and selects, and its loads' latency do. A warp takes steps of 256 consecutive tokens
// (coalesced 4-byte loads at any alignment, eight per array in flight per lane), computes its eight tokens per lane in pairs
// (packed fp32) and without branches, walks the sequences that meet the step, sums each one's tokens over its lanes and
// leaves the sums in the slot (step + sequence). A second kernel adds a sequence's slots in order, one warp to a sequence,
// and the CTA that finishes last joins the sequences; small batches do both in one CTA. No floating-point atomics: equal
// inputs give equal bits.
//
// 4 Mi tokens in 512 sequences with every term, 88 MB, forward and backward: 57 us from a cold L2 (0.23 of the measured copy
// bandwidth), 46 us again and again on arrays that the L2 holds; 2 Mi tokens in 2048 sequences of the preference loss, 27 MB: 24
// and 16 us. (Cold: a graph of one pass behind a write of 256 MB, of which a graph's start takes up to 7 us.) Steps that led here,
// on arrays in L2, one pass to a graph: branches in the token 137 us; tokens one at a time and expf 65; a warp for each step
// 58; one wave of warps that each take a stretch of the steps and load the next step ahead 54. The backward pass evaluates the
// forward's exponentials again: what a token gives is not kept.
//
// Ratios next to a bound: whether r = e^d lies above 1 + eps is decided as d > ln(1 + eps), with d the exact
// difference of the two log-probs (two floats, from one TwoSum) and the logarithm split into two floats, so
// that clipping does not depend on the rounding of d or of the exponential.
#include <climits>

#include "logits.cuh"
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

// The same for two tokens at a time, in the packed fp32 instructions.
__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }
__device__ __forceinline__ F2 minus2(F2 a, F2 b) { return fma2(b, both(-1.0f), a); }  // a - b, rounded once
// a - b and its rounding error, exactly (finite).
__device__ __forceinline__ void two_diff2(F2 a, F2 b, F2& hi, F2& lo) {
  hi = minus2(a, b);
  const F2 v = minus2(hi, a);
  lo = minus2(minus2(a, minus2(hi, v)), add2(b, v));
}
__device__ __forceinline__ F2 pick2(bool p0, bool p1, F2 a, F2 b) {  // a where p holds, else b
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(p0 ? a0 : b0, p1 ? a1 : b1);
}
__device__ __forceinline__ F2 inside2(F2 x, float bound, F2 a, F2 b) {  // a where |x| < bound, else b (NaN: b)
  float x0, x1;
  unpack2(x, x0, x1);
  return pick2(fabsf(x0) < bound, fabsf(x1) < bound, a, b);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^(x + low), |low| at most an ulp of x: 2^t with t the rounded x log2(e), times 1 + what t's rounding and `low` left. The
// hardware's 2^t is within 2^-22, what is left out of the correction below 2^-33. From |x| = ln(2^128) on 2^t by itself, which
// is infinite or below 2^-127 (or NaN), as it should be.
__device__ __forceinline__ F2 exp_pair(F2 x, F2 low) {
  constexpr float kHead = 1.44269504f, kTail = static_cast<float>(1.4426950408889634 - static_cast<double>(kHead));
  const F2 minus_t = mul2(x, both(-kHead));
  const F2 left = fma2(x, both(kTail), fma2(x, both(kHead), minus_t));
  const F2 rest = fma2(left, both(0.693147181f), low);
  float t0, t1;
  unpack2(minus_t, t0, t1);
  const F2 e = pack2(ex2(-t0), ex2(-t1));
  return inside2(x, 88.72284f, fma2(e, rest, e), e);
}
// (e^x - x - 1) / x^2: the power series up to x^9 (for |x| < 1/2, where it is truncated at 2e-9 of the sum and the
// difference would lose x's digits).
__device__ __forceinline__ F2 exp_series2(F2 x) {
  F2 p = fma2(x, both(1.0f / 362880.0f), both(1.0f / 40320.0f));
  p = fma2(x, p, both(1.0f / 5040.0f));
  p = fma2(x, p, both(1.0f / 720.0f));
  p = fma2(x, p, both(1.0f / 120.0f));
  p = fma2(x, p, both(1.0f / 24.0f));
  p = fma2(x, p, both(1.0f / 6.0f));
  return fma2(x, p, both(0.5f));
}
// e^x - x - 1 >= 0 and e^x - 1, with ex = e^x.
__device__ __forceinline__ F2 expm1_less2(F2 x, F2 ex) {
  return inside2(x, 0.5f, mul2(mul2(x, x), exp_series2(x)), minus2(add2(ex, both(-1.0f)), x));
}
__device__ __forceinline__ F2 expm1_2(F2 x, F2 ex) {
  return inside2(x, 0.5f, fma2(mul2(x, x), exp_series2(x), x), add2(ex, both(-1.0f)));
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

// 32 sequences from the one that holds token t0 on: lane l has the end of sequence first + l (first -1: tokens ahead of all
// sequences). Made once per step; a walk over the step's sequences then takes a shuffle each.
struct Window {
  int64_t first;
  int end;
};
__device__ __forceinline__ Window window_at(const int32_t* __restrict__ offsets, int64_t B, int64_t t0) {
  const int64_t c = count_up_to(offsets, B + 1, t0), at = c + (threadIdx.x & 31);
  return {c - 1, at <= B ? __ldg(offsets + at) : INT_MAX};
}

// The sequences of tokens [t0, t1), in order: f(b, s, e) for the part [s, e) that sequence b has of them;
// b = -1 for tokens of no sequence. Whole warp. The window is of t0 or earlier tokens, and moves on where it ends. Offsets
// that fall are answered with some split of the
// tokens, each in one part.
template <class F>
__device__ __forceinline__ void for_sequences(const int32_t* __restrict__ offsets, int64_t B, Window& w, int64_t t0,
                                              int64_t t1, F&& f) {
  int64_t t = t0, seen = -1;
  const uint32_t behind = __ballot_sync(0xFFFFFFFFu, w.end > t0);
  int k = behind ? __ffs(behind) - 1 : 32;
  while (t < t1) {
    if (k == 32) {  // more sequences (or empty ones) than the window has
      if (t == seen) {  // offsets that fall: the rest is of no sequence
        f(int64_t(-1), t, t1);
        return;
      }
      w = window_at(offsets, B, t);
      seen = t;
      k = 0;
    }
    const int64_t e = min(t1, static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, w.end, k)));
    const int64_t b = w.first + k;
    ++k;
    if (e <= t) continue;
    f(b < B ? b : int64_t(-1), t, e);
    t = e;
  }
}

// ---- the policy loss ------------------------------------------------------------------------------------

// What two tokens of the policy loss give: their clipped terms -w min(..) (0 instead of a product with an infinity where the
// advantage is 0), the estimates e^x - x - 1 of the divergence from the reference, the gradients of term + kl estimate to logp,
// r, e^d - d - 1, and whether clipping took the terms.
struct Pair {
  F2 term, div, grad, ratio, drift;
  bool clipped[2];
};

// Where clipping acts for one sign of the advantage: above `over` the ratio is `cap`, below `under` it is 1 - eps_low. Made
// once per sequence.
struct Clip {
  SplitFloat over, under;
  float cap;
};
__device__ __forceinline__ Clip clip_for(const PolicyArgs& a, float adv) {
  Clip c;
  const bool gain = adv > 0.0f;
  c.over = gain ? a.ln_high : a.ln_dual;
  c.under = gain ? SplitFloat{-INFINITY, 0.0f} : a.ln_low;
  c.cap = gain ? a.high : a.dual;
  if (adv == 0.0f) c.over = {INFINITY, 0.0f}, c.under = {-INFINITY, 0.0f};
  return c;
}

template <bool kGrad, bool kRef>
__device__ __forceinline__ Pair policy_pair(const PolicyArgs& a, const Clip& c0, const Clip& c1, F2 lp, F2 lo, F2 ref, float adv0,
                                            float adv1, F2 w) {
  Pair t;
  F2 hi, low;
  two_diff2(lp, lo, hi, low);
  t.ratio = exp_pair(hi, low);
  SplitFloat d0, d1;
  unpack2(hi, d0.hi, d1.hi);
  unpack2(low, d0.lo, d1.lo);
  const bool over0 = above(d0, c0.over), under0 = below(d0, c0.under), over1 = above(d1, c1.over), under1 = below(d1, c1.under);
  t.clipped[0] = over0 || under0;
  t.clipped[1] = over1 || under1;
  if constexpr (kGrad) {
    const F2 term = mul2(w, mul2(t.ratio, pack2(-adv0, -adv1)));
    t.grad = pick2(t.clipped[0] || adv0 == 0.0f, t.clipped[1] || adv1 == 0.0f, both(0.0f), term);
    if constexpr (kRef) {
      const F2 x = minus2(ref, lp);
      t.grad = fma2(both(-a.kl), expm1_2(x, exp_pair(x, both(0.0f))), t.grad);
    }
  } else {
    const F2 used = pick2(over0, over1, pack2(c0.cap, c1.cap), pick2(under0, under1, both(a.low), t.ratio));
    t.term = pick2(adv0 == 0.0f, adv1 == 0.0f, both(0.0f), mul2(w, mul2(used, pack2(-adv0, -adv1))));
    t.drift = expm1_less2(hi, t.ratio);
    if constexpr (kRef) {
      const F2 x = minus2(ref, lp);
      t.div = expm1_less2(x, exp_pair(x, both(0.0f)));
    }
  }
  return t;
}

// A step's tokens of this lane: token 32 j + lane of the step, with its advantage and whether it counts (nonzero).
template <bool kRef, bool kTok>
struct Step {
  float lp[kPerLane], lo[kPerLane], ref[kRef ? kPerLane : 1], w[kPerLane], adv[kTok ? kPerLane : 1];
  uint8_t mask[kPerLane];
};

// One array of a step, `count` tokens long, from its first token of this lane on: constant offsets, no bounds in whole steps.
template <class T>
__device__ __forceinline__ void load_array(const T* __restrict__ p, int count, T (&v)[kPerLane]) {
  if (count == kLossStep) {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) v[j] = __ldg(p + 32 * j);
  } else {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) v[j] = 32 * j + static_cast<int>(threadIdx.x & 31) < count ? __ldg(p + 32 * j) : T(0);
  }
}
// Whether the lane's tokens are there and not masked.
__device__ __forceinline__ void load_mask(const uint8_t* __restrict__ mask, int64_t at, int count, uint8_t (&m)[kPerLane]) {
  if (mask) {
    load_array(mask + at, count, m);
  } else {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) m[j] = 32 * j + static_cast<int>(threadIdx.x & 31) < count;
  }
}
__device__ __forceinline__ uint32_t mask_bits(const uint8_t (&m)[kPerLane]) {
  uint32_t live = 0;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) live |= m[j] ? 1u << j : 0u;
  return live;
}

template <bool kRef, bool kTok>
__device__ __forceinline__ void load_step(const PolicyArgs& a, int64_t t0, Step<kRef, kTok>& s) {
  const int64_t at = t0 + (threadIdx.x & 31);
  const int count = static_cast<int>(min(a.n - t0, static_cast<int64_t>(kLossStep)));
  load_array(a.logp + at, count, s.lp);
  load_array(a.logp_old + at, count, s.lo);
  if constexpr (kRef) load_array(a.logp_ref + at, count, s.ref);
  if constexpr (kTok) load_array(a.adv + at, count, s.adv);
  if (a.weights) {
    load_array(a.weights + at, count, s.w);
  } else {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) s.w[j] = 1.0f;
  }
  load_mask(a.mask, at, count, s.mask);
}

// A warp's equal stretch of the steps: f(s, step, window) for each, the next one's loads under way meanwhile.
template <bool kRef, bool kTok, class F>
__device__ __forceinline__ void for_steps(const PolicyArgs& a, F&& f) {
  const int64_t steps = (a.n + kLossStep - 1) / kLossStep, warps = static_cast<int64_t>(gridDim.x) * kWarpsPerCta;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5), end = steps * (w + 1) / warps;
  int64_t s = steps * w / warps;
  if (s >= end) return;
  Step<kRef, kTok> next;
  load_step(a, s * kLossStep, next);
  Window win = window_at(a.offsets, a.B, s * kLossStep);
#pragma unroll 1
  for (; s < end; ++s) {
    const Step<kRef, kTok> st = next;
    if (s + 1 < end) load_step(a, (s + 1) * kLossStep, next);
    f(s, st, win);
  }
}

// Bit j: token 32 j + lane of the step is in [lo, hi), parts of 0 .. 256.
__device__ __forceinline__ uint32_t part_mask(int lo, int hi) {
  const int lane = threadIdx.x & 31;
  const auto before = [lane](int end) { return (1u << ((end - lane + 31) >> 5)) - 1u; };  // rows of 32 with 32 j + lane < end
  return before(hi) & ~before(lo);
}

// A slot: sums of term, div, drift and ratio, then the numbers of tokens and of clipped ones. A sequence: term and div as
// split floats, drift and ratio (heads), the two numbers.
struct SlotSums {
  float v[4];
  uint32_t tokens, clipped, unused[2];
};
struct SeqSums {
  SplitFloat term, div;
  float drift, ratio;
  uint32_t tokens, clipped;
};
static_assert(sizeof(SlotSums) == 32 && sizeof(SeqSums) == 32, "as policy_workspace_bytes has them");

template <bool kRef, bool kTok>
__device__ __forceinline__ void policy_step(const PolicyArgs& a, int64_t s, const Step<kRef, kTok>& st, Window& win,
                                            SlotSums* __restrict__ slots) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = s * kLossStep, t1 = min(a.n, t0 + kLossStep);
  const uint32_t there = mask_bits(st.mask);
  for_sequences(a.offsets, a.B, win, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    if (b < 0) return;
    const int lo = static_cast<int>(from - t0), hi = static_cast<int>(to - t0);
    const uint32_t live = there & part_mask(lo, hi);
    F2 u[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
    uint32_t clipped = 0;
    // tokens j and j + 1 of the lane
    const auto pair = [&](int j, const Clip& c0, const Clip& c1, float adv0, float adv1) {
      const F2 ref = kRef ? pack2(st.ref[kRef ? j : 0], st.ref[kRef ? j + 1 : 0]) : both(0.0f);
      const Pair k = policy_pair<false, kRef>(a, c0, c1, pack2(st.lp[j], st.lp[j + 1]), pack2(st.lo[j], st.lo[j + 1]), ref,
                                              adv0, adv1, pack2(st.w[j], st.w[j + 1]));
      const bool in0 = live >> j & 1, in1 = live >> (j + 1) & 1;
      const F2 none = both(0.0f);
      u[0] = add2(u[0], pick2(in0, in1, k.term, none));
      if constexpr (kRef) u[1] = add2(u[1], pick2(in0, in1, k.div, none));
      u[2] = add2(u[2], pick2(in0, in1, k.drift, none));
      u[3] = add2(u[3], pick2(in0, in1, k.ratio, none));
      clipped |= (k.clipped[0] ? 1u << j : 0u) | (k.clipped[1] ? 2u << j : 0u);
    };
    if constexpr (kTok) {
#pragma unroll
      for (int j = 0; j < kPerLane; j += 2) pair(j, clip_for(a, st.adv[j]), clip_for(a, st.adv[j + 1]), st.adv[j], st.adv[j + 1]);
    } else {
      const float adv = __ldg(a.adv + b);
      const Clip clip = clip_for(a, adv);
      if (hi - lo >= kLossStep / 4) {  // most tokens of the step: all eight side by side
#pragma unroll
        for (int j = 0; j < kPerLane; j += 2) pair(j, clip, clip, adv, adv);
      } else {  // a short sequence: only the rows of tokens that it meets
#pragma unroll
        for (int j = 0; j < kPerLane; j += 2)
          if (32 * j + 64 > lo && 32 * j < hi) pair(j, clip, clip, adv, adv);
      }
    }
    // the numbers of tokens and, from bit 16 on, of clipped ones: at most 256 of each in a step
    const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, __popc(live) | __popc(live & clipped) << 16);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x, y;
      unpack2(u[i], x, y);
      v[i] = kRef || i != 1 ? warp_sum(x + y) : 0.0f;
    }
    if (lane == 0) slots[s + b] = {{v[0], v[1], v[2], v[3]}, c & 0xFFFFu, c >> 16, {0u, 0u}};
  });
}

// The slots of sequence b: of the steps that hold its tokens.
struct SlotRange {
  int64_t first, end;
};
__device__ __forceinline__ SlotRange slot_range(const int32_t* __restrict__ offsets, int64_t n, int64_t b) {
  const int64_t s = min(max(static_cast<int64_t>(__ldg(offsets + b)), int64_t(0)), n);
  const int64_t e = min(max(static_cast<int64_t>(__ldg(offsets + b + 1)), int64_t(0)), n);
  const int64_t first = s / kLossStep + b;
  return {first, e > s ? (e - 1) / kLossStep + b + 1 : first};
}

// Sequence b of the policy loss: its slots in lanes' strides, then a tree. Whole warp.
__device__ __forceinline__ void policy_sequence(int64_t b, SlotRange of, const SlotSums* __restrict__ slots,
                                                SeqSums* __restrict__ seqs) {
  const int lane = threadIdx.x & 31;
  SplitFloat v[4] = {{0.0f, 0.0f}, {0.0f, 0.0f}, {0.0f, 0.0f}, {0.0f, 0.0f}};
  uint32_t tokens = 0, clipped = 0;
#pragma unroll 2
  for (int64_t k = of.first + lane; k < of.end; k += 32) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(slots + k));
    const uint2 c = __ldcg(reinterpret_cast<const uint2*>(&slots[k].tokens));
    const float u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = split_add(v[i], {u[i], 0.0f});
    tokens += c.x;
    clipped += c.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = warp_sum_split(v[i]);
  tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
  clipped = __reduce_add_sync(0xFFFFFFFFu, clipped);
  if (lane == 0) seqs[b] = {v[0], v[1], v[2].hi, v[3].hi, tokens, clipped};
}

// The sequences' sums to the loss, the statistics and the coefficients. Whole CTA.
__device__ __forceinline__ void policy_finish(const PolicyArgs& a, const SeqSums* __restrict__ seqs) {
  __shared__ SplitFloat part[4][32];
  __shared__ uint32_t parts[3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  SplitFloat v[4] = {{0.0f, 0.0f}, {0.0f, 0.0f}, {0.0f, 0.0f}, {0.0f, 0.0f}};
  uint32_t c[3] = {0, 0, 0};  // tokens, clipped, sequences with a token: at most 2^31
  for (int64_t b = threadIdx.x; b < a.B; b += blockDim.x) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(seqs + b));
    const float2 y = __ldcg(reinterpret_cast<const float2*>(&seqs[b].drift));
    const uint2 z = __ldcg(reinterpret_cast<const uint2*>(&seqs[b].tokens));
    SplitFloat term{x.x, x.y}, div{x.z, x.w};
    if (a.mode == NVFP4RL_LOSS_SEQ_MEAN) {
      const float len = fmaxf(static_cast<float>(z.x), 1.0f);
      term = {term.hi / len, term.lo / len};
      div = {div.hi / len, div.lo / len};
    }
    v[0] = split_add(v[0], term);
    v[1] = split_add(v[1], div);
    v[2] = split_add(v[2], {y.x, 0.0f});
    v[3] = split_add(v[3], {y.y, 0.0f});
    c[0] += z.x;
    c[1] += z.y;
    c[2] += z.x > 0 ? 1u : 0u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const SplitFloat t = warp_sum_split(v[i]);
    if (lane == 0) part[i][warp] = t;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t t = __reduce_add_sync(0xFFFFFFFFu, c[i]);
    if (lane == 0) parts[i][warp] = t;
  }
  __syncthreads();
  // every warp joins the warps alike: the coefficients need the numbers
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = warp_sum_split(lane < warps ? part[i][lane] : SplitFloat{0.0f, 0.0f});
#pragma unroll
  for (int i = 0; i < 3; ++i) c[i] = __reduce_add_sync(0xFFFFFFFFu, lane < warps ? parts[i][lane] : 0u);
  const float tokens = static_cast<float>(c[0]), there = static_cast<float>(c[2]), many = fmaxf(tokens, 1.0f);
  const float share = a.mode == NVFP4RL_LOSS_TOKEN_MEAN ? many : a.mode == NVFP4RL_LOSS_SEQ_MEAN ? fmaxf(there, 1.0f) : a.norm;
  if (threadIdx.x == 0) {
    const float policy = v[0].hi / share, div = v[1].hi / share;
    const float loss = a.logp_ref && a.kl != 0.0f ? fmaf(a.kl, div, policy) : policy;
    a.loss[0] = loss;
    if (a.stats) {
      a.stats[0] = loss;
      a.stats[1] = policy;
      a.stats[2] = div;
      a.stats[3] = static_cast<float>(c[1]) / many;
      a.stats[4] = v[2].hi / many;
      a.stats[5] = v[3].hi / many;
      a.stats[6] = tokens;
      a.stats[7] = there;
    }
  }
  if (!a.coef) return;
  const float same = 1.0f / share;
  for (int64_t b = threadIdx.x; b < a.B; b += blockDim.x)
    a.coef[b] = a.mode == NVFP4RL_LOSS_SEQ_MEAN
                    ? 1.0f / (fmaxf(static_cast<float>(__ldcg(&seqs[b].tokens)), 1.0f) * share)
                    : same;
}

// Per SM: two of 128 registers, which hold two steps (three of 80 spill them: 74 us instead of 54).
constexpr int kPolicyCtas = 2;

template <bool kRef, bool kTok>
__global__ void __launch_bounds__(kThreads, kPolicyCtas) policy_sums_kernel(const PolicyArgs a, unsigned int* __restrict__ ticket,
                                                                            SlotSums* __restrict__ slots) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0u;  // for the kernel behind this one
  for_steps<kRef, kTok>(a, [&](int64_t s, const Step<kRef, kTok>& st, Window& win) { policy_step(a, s, st, win, slots); });
}

__global__ void __launch_bounds__(kThreads) policy_join_kernel(const PolicyArgs a, unsigned int* __restrict__ ticket,
                                                               const SlotSums* __restrict__ slots,
                                                               SeqSums* __restrict__ seqs) {
  __shared__ int last;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarpsPerCta;
  int64_t b = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  // ahead of the wait for the slots: the offsets, complete before the kernel ahead let this one start
  SlotRange of{0, 0};
  if (b < a.B) of = slot_range(a.offsets, a.n, b);
  griddep_wait();
  griddep_launch_dependents();
  while (b < a.B) {
    policy_sequence(b, of, slots, seqs);
    b += warps;
    if (b < a.B) of = slot_range(a.offsets, a.n, b);
  }
  __threadfence();  // this thread's sequences are visible before the CTA's ticket
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();  // and every other CTA's from here on
  policy_finish(a, seqs);
}

// The whole of the loss in one CTA of 16 warps, for batches of at most as many steps and sequences: one launch instead of two,
// and no ticket (1843 tokens in 8 sequences 7.7 instead of 9.6 us, 4000 in 8 8.5 instead of 9.2; in a second round of steps
// 8000 took 12.4 instead of 8.3, and 32 warps, with half the registers, 10.6 for the 1843).
constexpr int kOneWarps = 16;

template <bool kRef, bool kTok>
__global__ void __launch_bounds__(32 * kOneWarps) policy_one_kernel(const PolicyArgs a, SlotSums* __restrict__ slots,
                                                                    SeqSums* __restrict__ seqs) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int64_t t0 = static_cast<int64_t>(warp) * kLossStep;
  if (t0 < a.n) {
    Step<kRef, kTok> st;
    load_step(a, t0, st);
    Window win = window_at(a.offsets, a.B, t0);
    policy_step(a, warp, st, win, slots);
  }
  __syncthreads();
  if (warp < a.B) policy_sequence(warp, slot_range(a.offsets, a.n, warp), slots, seqs);
  __syncthreads();
  policy_finish(a, seqs);
}

template <bool kRef, bool kTok>
__device__ __forceinline__ void policy_grad_step(const PolicyArgs& a, float dloss, int64_t s, const Step<kRef, kTok>& st,
                                                 Window& win) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = s * kLossStep, t1 = min(a.n, t0 + kLossStep);
  const uint32_t there = mask_bits(st.mask);
  float* out = a.dlogp + t0 + lane;
  for_sequences(a.offsets, a.B, win, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    const int lo = static_cast<int>(from - t0), hi = static_cast<int>(to - t0);
    const float coef = b < 0 ? 0.0f : dloss * __ldg(a.coef_in + b);
    const float seq_adv = b < 0 || kTok ? 0.0f : __ldg(a.adv + b);
    const Clip seq_clip = clip_for(a, seq_adv);
    const uint32_t part = part_mask(lo, hi), live = b >= 0 ? there & part : 0u;
#pragma unroll
    for (int j = 0; j < kPerLane; j += 2) {
      if (32 * j + 64 <= lo || 32 * j >= hi) continue;
      const float adv0 = kTok ? st.adv[kTok ? j : 0] : seq_adv, adv1 = kTok ? st.adv[kTok ? j + 1 : 0] : seq_adv;
      const Clip c0 = kTok ? clip_for(a, adv0) : seq_clip, c1 = kTok ? clip_for(a, adv1) : seq_clip;
      const F2 ref = kRef ? pack2(st.ref[kRef ? j : 0], st.ref[kRef ? j + 1 : 0]) : both(0.0f);
      const Pair k = policy_pair<true, kRef>(a, c0, c1, pack2(st.lp[j], st.lp[j + 1]), pack2(st.lo[j], st.lo[j + 1]), ref, adv0,
                                             adv1, pack2(st.w[j], st.w[j + 1]));
      float g0, g1;
      unpack2(mul2(both(coef), k.grad), g0, g1);
      if (part >> j & 1) out[32 * j] = live >> j & 1 ? g0 : 0.0f;
      if (part >> (j + 1) & 1) out[32 * j + 32] = live >> (j + 1) & 1 ? g1 : 0.0f;
    }
  });
}

template <bool kRef, bool kTok>
__global__ void __launch_bounds__(kThreads, kPolicyCtas) policy_grad_kernel(const PolicyArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const float dloss = a.dloss ? __ldg(a.dloss) : 1.0f;
  for_steps<kRef, kTok>(a, [&](int64_t s, const Step<kRef, kTok>& st, Window& win) { policy_grad_step(a, dloss, s, st, win); });
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
  const int count = static_cast<int>(t1 - t0);
  float lp[kPerLane], ref[kPerLane];
  load_array(a.logp + t0 + lane, count, lp);
  if (a.logp_ref) {
    load_array(a.logp_ref + t0 + lane, count, ref);
  } else {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) ref[j] = 0.0f;
  }
  uint8_t m[kPerLane];
  load_mask(a.mask, t0 + lane, count, m);
  Window win = window_at(a.offsets, 2 * a.pairs, t0);
  const uint32_t live = mask_bits(m);
  for_sequences(a.offsets, 2 * a.pairs, win, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    if (b < 0) return;
    const int lo = static_cast<int>(from - t0), hi = static_cast<int>(to - t0);
    // heads and rounding errors, in two sums side by side; an infinite head keeps no tail
    SplitFloat v[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    uint32_t tokens = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int i = 32 * j + lane;
      const bool in = (live >> j & 1) && i >= lo && i < hi;
      const SplitFloat d = two_sum(in ? lp[j] : 0.0f, in ? -ref[j] : 0.0f);  // logp - logp_ref, exactly
      const SplitFloat h = two_sum(v[j & 1].hi, d.hi);
      v[j & 1] = {h.hi, v[j & 1].lo + (h.lo + d.lo)};
      tokens += in ? 1u : 0u;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!isfinite(v[i].hi)) v[i].lo = 0.0f;
    const SplitFloat sum = warp_sum_split(split_add(v[0], v[1]));
    tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
    if (lane == 0) slots[s + b] = make_float4(sum.hi, sum.lo, static_cast<float>(tokens), 0.0f);
  });
}

// One warp to a pair.
__global__ void __launch_bounds__(kThreads) preference_join_kernel(const PreferenceArgs a,
                                                                   const float4* __restrict__ slots) {
  const int64_t p = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  SlotRange of[2] = {{0, 0}, {0, 0}};
  if (a.n > 0 && p < a.pairs) {  // ahead of the wait for the slots, as in policy_join_kernel
#pragma unroll
    for (int side = 0; side < 2; ++side) of[side] = slot_range(a.offsets, a.n, 2 * p + side);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (p >= a.pairs) return;
  SplitFloat total[2];
  float share[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    SplitFloat v[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // the sum and the number of tokens
    for (int64_t k = of[side].first + (threadIdx.x & 31); k < of[side].end; k += 32) {
      const float4 x = __ldcg(slots + k);
      v[0] = split_add(v[0], {x.x, x.y});
      v[1] = split_add(v[1], {x.z, 0.0f});
    }
    v[0] = warp_sum_split(v[0]);
    v[1] = warp_sum_split(v[1]);
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
  uint8_t m[kPerLane];
  load_mask(a.mask, t0 + lane, static_cast<int>(t1 - t0), m);
  Window win = window_at(a.offsets, 2 * a.pairs, t0);
  const uint32_t live = mask_bits(m);
  float* out = a.dlogp + t0 + lane;
  for_sequences(a.offsets, 2 * a.pairs, win, t0, t1, [&](int64_t b, int64_t from, int64_t to) {
    const int lo = static_cast<int>(from - t0), hi = static_cast<int>(to - t0);
    const float c = b < 0 ? 0.0f : __ldg(a.coef_in + b) * (a.dloss ? __ldg(a.dloss + (b >> 1)) : 1.0f);
    if (lo == 0 && hi == kLossStep) {
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) out[32 * j] = live >> j & 1 ? c : 0.0f;
      return;
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
      if (32 * j + lane >= lo && 32 * j + lane < hi) out[32 * j] = live >> j & 1 ? c : 0.0f;
  });
}

dim3 warps_grid(int64_t warps) {
  return dim3(static_cast<unsigned>(std::max<int64_t>(1, (warps + kWarpsPerCta - 1) / kWarpsPerCta)));
}

}  // namespace

namespace {

// One wave of CTAs at most: each warp takes a stretch of the steps.
dim3 policy_grid(int64_t n, const DeviceInfo& dev) {
  dim3 grid = warps_grid(loss_steps(n));
  grid.x = std::min(grid.x, static_cast<unsigned>(dev.sm_count * kPolicyCtas));
  return grid;
}

template <bool kRef, bool kTok>
nvfp4rl_status policy_forward(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  auto* ticket = static_cast<unsigned int*>(a.ws);
  auto* slots = reinterpret_cast<SlotSums*>(static_cast<uint8_t*>(a.ws) + 256);
  auto* seqs = reinterpret_cast<SeqSums*>(slots + loss_steps(a.n) + a.B);
  if (loss_steps(a.n) <= kOneWarps && a.B <= kOneWarps) {
    if (launch_pdl(policy_one_kernel<kRef, kTok>, dim3(1), dim3(32 * kOneWarps), 0, st, a, slots, seqs) != cudaSuccess)
      return NVFP4RL_ERR_CUDA;
    return launch_status();
  }
  if (launch_pdl(policy_sums_kernel<kRef, kTok>, policy_grid(a.n, dev), dim3(kThreads), 0, st, a, ticket, slots) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  if (launch_status() != NVFP4RL_OK) return NVFP4RL_ERR_CUDA;
  dim3 grid = warps_grid(a.B);
  grid.x = std::min(grid.x, static_cast<unsigned>(dev.sm_count) * 4u);
  if (launch_pdl(policy_join_kernel, grid, dim3(kThreads), 0, st, a, ticket, static_cast<const SlotSums*>(slots), seqs) !=
      cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

template <bool kRef, bool kTok>
nvfp4rl_status policy_backward(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (launch_pdl(policy_grad_kernel<kRef, kTok>, policy_grid(a.n, dev), dim3(kThreads), 0, st, a) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace

nvfp4rl_status launch_policy_loss(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (a.logp_ref) return a.adv_per_token ? policy_forward<true, true>(a, dev, st) : policy_forward<true, false>(a, dev, st);
  return a.adv_per_token ? policy_forward<false, true>(a, dev, st) : policy_forward<false, false>(a, dev, st);
}

nvfp4rl_status launch_policy_loss_grad(const PolicyArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (a.logp_ref && a.kl != 0.0f)
    return a.adv_per_token ? policy_backward<true, true>(a, dev, st) : policy_backward<true, false>(a, dev, st);
  return a.adv_per_token ? policy_backward<false, true>(a, dev, st) : policy_backward<false, false>(a, dev, st);
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
