// Gradients of the token log-probs, the entropy and the top-k distillation loss to the logits (sm_103a).
//
// Given the forward call's lse (and entropy, lse_tail) the gradient is elementwise: with t = log2 p_j = x c - R,
// c = scale log2 e, R = lse log2 e,
//   token log-prob and entropy:  dx_j = 2^t (alpha + beta t) [+ scale dlogp at the token],
//     alpha = -scale (dlogp + dentropy H), beta = -scale dentropy ln 2;
//   distillation, unlisted columns:  dx_j = alpha 2^t; NORMALIZED: alpha = scale dloss, R as above; TAIL: the factor
//     Q - q_0 / p_0 would overflow for a small p_0, so alpha = scale dloss (Q p_0 - q_0) with R = lse_tail log2 e;
//   listed columns:  dx_j = scale dloss (Q p_j - q_j), written over the above after a block barrier.
// Bound by HBM: each logit is read once, each gradient written once (4096 x 152064 bf16 with entropy, an eighth of
// the rows padding, 333 us, 1.03 of the copy rate counted in the bytes it cannot do without, all rows live 346 us;
// distillation with 64 listed 376 us, 0.98, with 200, whose CTAs of 256 threads spill 40 bytes, 436-444 us). A CTA takes
// a chunk of one row, 16-byte vectors aligned for the stores; where the row of logits starts at another element of
// a vector than the row of gradients, a vector is put together from two aligned loads by funnel shifts (the second one
// hits L1/L2). Vectors at a row's ends, whose 16 bytes are not all inside it, go element by element. A list costs every
// chunk the same (the teacher's row, the barriers): chunks of four steps where the CTAs suffice (eight: 378 us);
// an fp32 batch of 100 rows of 128257 with 128 listed stays at 0.69 (19.1 us): 1600 CTAs, of which 1368 run at once.
// Rows of scores past 2^12, where lse itself is too coarse, get their sums anew from one CTA (far_row): 4096 x 152064 bf16 of
// them 2.0 ms with entropy, 2.8-2.9 ms with 64 listed, 2.1-2.2 ms with 200 (more threads); one alone 0.16, 0.58, 0.17 ms.
#include "logits.cuh"

namespace nvfp4rl {
namespace {

constexpr int64_t kListCtas = 4 * kNumSMsHint;

// The 8 (bf16) or 4 (fp32) logits that start s elements into the 32 bytes (a, b).
template <typename T>
__device__ __forceinline__ uint4 shift_vec(uint4 a, uint4 b, int s) {
  const int words = sizeof(T) == 2 ? s >> 1 : s;  // uniform over the row
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (words & 1) {
#pragma unroll
    for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
  }
  if (words & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  const uint32_t odd = sizeof(T) == 2 ? (s & 1) * 16 : 0;
  return make_uint4(__funnelshift_r(w[0], w[1], odd), __funnelshift_r(w[1], w[2], odd),
                    __funnelshift_r(w[2], w[3], odd), __funnelshift_r(w[3], w[4], odd));
}

// x is clamped at low = -2^17 / c, where 2^t is 0 (|R| is below 2^13) and beta t finite: 0 beta t has to be 0.
struct RowCoef {
  float c, c_low, R, alpha, beta, low;
};

// Past 2^12 lse as a 32-bit number takes more than 2^-13 from p (past 2^24 it holds no trace of ln s): far_row takes the
// row. (Not for -inf, NaN.)
__device__ __forceinline__ bool is_far(float lse) { return fabsf(lse) > 0x1p12f && fabsf(lse) < INFINITY; }

// t = x c - R, with the rounding of c made good for fp32 logits (29 2^-24 of p at z = 20; a bf16 result does not show it).
template <typename T>
__device__ __forceinline__ float score(float v, const RowCoef& r) {
  return fmaf(v, r.c, sizeof(T) == 4 ? fmaf(v, r.c_low, -r.R) : -r.R);
}

// What the rounding of R = lse log2 e took: p = 2^(x c - R) times this, which goes into a row's factors.
__device__ __forceinline__ float ref_factor(float lse, float R) {
  const float low = fmaf(lse, kLog2E, -R) + lse * kLog2ELow, d = -low * kLn2;
  return fabsf(d) < 0.01f ? fmaf(fmaf(0.5f * d, d, d), 1.0f, 1.0f) : expf(d);
}

// One element, with the roundings of the packed form (no contraction): the bits do not depend on where a row lies.
template <typename T, bool kEntropy>
__device__ __forceinline__ float grad1(float v, const RowCoef& r) {
  if (kEntropy || sizeof(T) == 4) v = fmaxf(v, r.low);
  const float t = score<T>(v, r), e = exp2_approx(t);
  return __fmul_rn(e, kEntropy ? fmaf(r.beta, t, r.alpha) : r.alpha);
}

template <typename T, bool kEntropy>
__device__ __forceinline__ F2 grad2(float lo, float hi, const RowCoef& r) {
  if (kEntropy || sizeof(T) == 4) {
    lo = fmaxf(lo, r.low);
    hi = fmaxf(hi, r.low);
  }
  const F2 x = pack2(lo, hi), ref = pack2(-r.R, -r.R);
  const F2 t = fma2(x, pack2(r.c, r.c), sizeof(T) == 4 ? fma2(x, pack2(r.c_low, r.c_low), ref) : ref);
  float t0, t1;
  unpack2(t, t0, t1);
  const F2 e = pack2(exp2_approx(t0), exp2_approx(t1));
  return mul2(e, kEntropy ? fma2(pack2(r.beta, r.beta), t, pack2(r.alpha, r.alpha)) : pack2(r.alpha, r.alpha));
}

// The gradients of one vector; `hit` is added at element `at` (none: outside [0, VEC)).
template <typename T, bool kEntropy>
__device__ __forceinline__ uint4 grad_vec(uint4 x, const RowCoef& r, int at, float hit) {
  constexpr int VEC = kVecOf<T>;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float g[VEC];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    float lo, hi;
    if (sizeof(T) == 2) {
      lo = __uint_as_float(bf16_lo_bits(w[i]));
      hi = __uint_as_float(bf16_hi_bits(w[i]));
    } else {
      lo = __uint_as_float(w[(2 * i) & 3]);
      hi = __uint_as_float(w[(2 * i + 1) & 3]);
    }
    unpack2(grad2<T, kEntropy>(lo, hi, r), g[2 * i], g[2 * i + 1]);
  }
  if (static_cast<unsigned>(at) < static_cast<unsigned>(VEC)) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i == at) g[i] = __fadd_rn(g[i], hit);
  }
  if (sizeof(T) == 2)
    return make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4 % VEC], g[5 % VEC]),
                      pack_bf16x2(g[6 % VEC], g[7 % VEC]));
  return make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
}

// A row whose lse does not hold its sums: one CTA forms them anew, relative to the maxima, and writes the whole row.
struct FarShared {
  float hit, mass, q0;
  float dh, h;          // scale dentropy, entropy
  int token;
};
struct FarReduce {
  float top[2][kListWarps];
  float2 sum[kListWarps];
};

// f takes every column and its logit, in groups of at most 8 per thread; `end` is called after each group.
template <typename T, int NT, typename F, typename E>
__device__ __forceinline__ void for_row(const T* x, int V, const F& f, const E& end) {
  for (int j0 = threadIdx.x; j0 < V; j0 += 8 * NT) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = j0 + u * NT < V ? logit(x, j0 + u * NT) : -INFINITY;
#pragma unroll 1
    for (int u = 0; u < 8 && j0 + u * NT < V; ++u) {
      f(j0 + u * NT, v[0]);
#pragma unroll
      for (int i = 0; i < 7; ++i) v[i] = v[i + 1];
    }
    end();
  }
}
template <typename T, int NT, typename F>
__device__ __forceinline__ void for_row(const T* x, int V, const F& f) {
  for_row<T, NT>(x, V, f, [] {});
}

// A sum that keeps what its additions lose: 65536 equal terms in one chain (64 threads, the longest rows) drift by
// 2^-11 of the sum, which would go into every gradient of the row; groups of 8 added this way stay within 10 2^-24.
struct LongSum {
  float s, lost;
  __device__ __forceinline__ void add(float v) {
    const float y = __fsub_rn(v, lost), t = __fadd_rn(s, y);
    lost = __fsub_rn(__fsub_rn(t, s), y);
    s = t;
  }
};

template <typename T, int NT, bool kEntropy, bool kList>
__device__ __forceinline__ void far_row(const LogitsGradArgs& a, const T* x, T* dx, const int32_t* ids_s, const float* q_s,
                                        const FarShared& sh, FarReduce& red) {
  const float hit = sh.hit, dh = sh.dh, h = sh.h;
  const int token = sh.token;
  const int V = static_cast<int>(a.V);
  const float c = a.scale * kLog2E;
  const bool tail = kList && a.tail;
  const auto listed = [&](int j) {
    bool in = false;
    for (int i = 0; i < a.k && !in; i += 4) {
      const int4 id = *reinterpret_cast<const int4*>(ids_s + i);
      in = id.x == j || id.y == j || id.z == j || id.w == j;
    }
    return in;
  };
  // listed columns: thread i holds entry i; the first entry of a column writes it, with the sum of all
  int mine = -1;
  float mine_x = -INFINITY, mine_q = 0.0f;
  if (kList && threadIdx.x < a.k && ids_s[threadIdx.x] >= 0) {
    mine = ids_s[threadIdx.x];
    mine_x = logit(x, mine);
    for (int i = 0; i < a.k; ++i) {
      if (ids_s[i] != mine) continue;
      mine_q += q_s[i];
      if (i < static_cast<int>(threadIdx.x)) mine = -1;
    }
  }
  float m = -kLogitBound, m_rest = -kLogitBound;
  for_row<T, NT>(x, V, [&](int j, float v) {
    m = fmaxf(m, v);
    if (tail && v > m_rest && !listed(j)) m_rest = v;
  });
  m = cta_max<NT / 32>(m, red.top[0]);
  m_rest = cta_max<NT / 32>(m_rest, red.top[1]);
  const auto exp_from = [&](float v, float top) {
    return v <= -kLogitBound || v > top ? 0.0f : exp2_approx((v - top) * c);
  };
  LongSum all{0.0f, 0.0f}, rest{0.0f, 0.0f};
  float2 s = make_float2(0.0f, 0.0f);
  for_row<T, NT>(
      x, V,
      [&](int, float v) {
        s.x += exp_from(v, m);
        if (tail) s.y += exp_from(v, m_rest);
      },
      [&] {
        all.add(s.x);
        if (tail) rest.add(s.y);
        s = make_float2(0.0f, 0.0f);
      });
  s = make_float2(all.s, rest.s);
  // the listed columns' terms come out of the second sum: at most k of 1, beside at least one unlisted of 1
  if (tail && mine >= 0) s.y -= exp_from(mine_x, m_rest);
  s = cta_sum<NT / 32>(s, red.sum);
  const float ln_s = logf(s.x), to_p = 1.0f / s.x, to_b = tail && m_rest > -kLogitBound ? sh.q0 / s.y : 0.0f;
  for_row<T, NT>(x, V, [&](int j, float v) {
    const float p = exp_from(v, m) * to_p;
    float g;
    if (kList) {
      g = hit * fmaf(sh.mass, p, -(exp_from(v, m_rest) * to_b));
    } else {
      g = hit * ((j == token ? 1.0f : 0.0f) - p);
      if (kEntropy && p > 0.0f) g -= dh * p * (fmaf(v - m, a.scale, -ln_s) + h);
    }
    store_logit(dx, j, g);
  });
  if (kList) {
    __syncthreads();
    if (mine >= 0) store_logit(dx, mine, hit * fmaf(sh.mass, exp_from(mine_x, m) * to_p, -mine_q));
  }
}

// The same as a call, which spares the token form's loop (4096 x 152064 334 us, inlined 337; the list's is better inlined: 376, 380).
template <typename T, int NT, bool kEntropy>
__device__ __noinline__ void far_row_called(const LogitsGradArgs& a, const T* x, T* dx, const FarShared& sh, FarReduce& red) {
  far_row<T, NT, kEntropy, false>(a, x, dx, nullptr, nullptr, sh, red);
}

// NT: threads, at least as many as listed columns; kU: vectors per thread and step; kEntropy: the entropy term (token form only); kList: distillation;
// kShift: rows of logits and gradients start at different elements of a vector (somewhere in the call).
template <typename T, int NT, int kU, bool kEntropy, bool kList, bool kShift>
__global__ void __launch_bounds__(NT) logits_grad_kernel(const LogitsGradArgs a, unsigned chunks, int steps) {
  constexpr int VEC = kVecOf<T>;
  __shared__ __align__(16) int32_t ids_s[kList ? kMaxListed : 4];
  __shared__ float q_s[kList ? kMaxListed : 1];
  __shared__ TeacherShared teacher_s;
  __shared__ FarShared far_s;
  __shared__ FarReduce far_red;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x / chunks;
  // vectors and columns in 32 bits: V <= 2^22
  const int V = static_cast<int>(a.V);
  const int v_begin = static_cast<int>(blockIdx.x % chunks) * steps * (kU * NT);
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  T* dx = static_cast<T*>(a.dx) + row * a.ldd;
  const int tid = threadIdx.x;
  const int out_phase = vec_phase(dx);
  const int s = kShift ? (vec_phase(x) - out_phase) & (VEC - 1) : 0;
  const float lse = a.lse[row];
  bool dead = lse == -INFINITY;
  const float c = a.scale * kLog2E, R = lse * kLog2E, f = ref_factor(lse, R);
  RowCoef r{c, fmaf(a.scale, kLog2E, -c) + a.scale * kLog2ELow, R, 0.0f, 0.0f, a.low};
  const float rest = kList && a.tail ? a.lse_tail[row] : 0.0f;
  const bool far = is_far(lse) || is_far(rest);
  float hit = 0.0f, mass = 0.0f;
  int token = -1;
  // listed columns of this chunk: thread i holds entry i
  int mine = -1;
  float mine_x = 0.0f;
  uint4 in[kU], in2[kShift ? kU : 1];
  bool whole[kU];
  const auto load_step = [&](int step) {
    const int v0 = v_begin + step * (kU * NT) + tid;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int col = (v0 + u * NT) * VEC - out_phase;
      // every byte of the loads and of the store lies inside the row
      whole[u] = kShift && s ? col >= s && col - s + 2 * VEC <= V : col >= 0 && col + VEC <= V;
      if (whole[u] && !dead) {
        in[u] = ld_logits16(x + col - s);
        if (kShift && s) in2[u] = ld_logits16(x + col - s + VEC);
      }
    }
  };
  if (kList) {
    // all of these are under way together: the row's scalars, its list, the first vectors and the listed logits of
    // this chunk
    const float d = a.dloss[row];
    int id = -1;
    float l = -INFINITY, q, lq;
    if (tid < a.k) {
      id = a.ids[row * a.k + tid];
      l = a.teacher[row * a.k + tid];
    }
    dead |= d == 0.0f;
    load_step(0);
    if (id >= V) id = -1;
    if (id >= 0) {
      const int v = (id + out_phase) / VEC - v_begin;
      if (v >= 0 && v < steps * (kU * NT)) {
        mine = id;
        mine_x = logit(x, id);
      }
    }
    ids_s[tid] = id >= 0 ? id : -1;
    // its barriers: the listed logits are read before a gradient in their place may be written
    const TeacherRow t = teacher_row<NT / 32>(teacher_s, id >= 0 ? id : -1, l, a.tail, q, lq);
    q_s[tid] = q;
    dead |= !__syncthreads_or(id >= 0) || !t.any;
    hit = d * a.scale;
    mass = t.mass;
    r.alpha = mass * hit * f;
    if (a.tail) {
      if (rest == -INFINITY) {
        mass -= t.q0;  // no bucket; the unlisted columns are masked
        r.alpha = 0.0f;
      } else {
        r.R = rest * kLog2E;
        r.alpha = (mass * expf(rest - lse) - t.q0) * hit * ref_factor(rest, r.R);
      }
    }
    if (far && tid == 0) far_s = FarShared{hit, mass, t.q0, 0.0f, 0.0f, -1};
    if (dead) mine = -1;
  } else {
    const float dl = a.dlogp ? a.dlogp[row] : 0.0f, dh = kEntropy ? a.dentropy[row] : 0.0f;
    if (a.tokens) {
      token = a.tokens[row];
      dead |= token < 0 || token >= V;
    }
    dead |= dl == 0.0f && dh == 0.0f;
    hit = dl * a.scale;
    r.alpha = -a.scale * (kEntropy ? fmaf(dh, a.entropy[row], dl) : dl) * f;
    r.beta = -a.scale * dh * kLn2 * f;
  }
  const bool anew = far && !dead;
  if (anew) {
    if (!kList && tid == 0)
      far_s = FarShared{hit, 0.0f, 0.0f, kEntropy ? a.scale * a.dentropy[row] : 0.0f, kEntropy ? a.entropy[row] : 0.0f,
                        token};
    __syncthreads();
  }
  for (int step = 0; step < steps && !anew; ++step) {
    const int v0 = v_begin + step * (kU * NT) + tid;
    if (!kList || step > 0) load_step(step);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int col = (v0 + u * NT) * VEC - out_phase;
      if (whole[u]) {
        uint4 g = make_uint4(0, 0, 0, 0);
        if (!dead) {
          const uint4 xin = kShift && s ? shift_vec<T>(in[u], in2[kShift ? u : 0], s) : in[u];
          g = grad_vec<T, kEntropy>(xin, r, kList || token < 0 ? -1 : token - col, hit);
        }
        __stcs(reinterpret_cast<uint4*>(dx + col), g);
      } else if (col < V) {
        for (int j = max(col, 0); j < min(col + VEC, V); ++j) {
          float g = 0.0f;
          if (!dead) {
            g = grad1<T, kEntropy>(logit(x, j), r);
            if (!kList && j == token) g = __fadd_rn(g, hit);
          }
          store_logit(dx, j, g);
        }
      }
    }
  }
  if (kList) {
    __syncthreads();  // the chunk's dense values are written
    if (mine >= 0 && !anew) {
      // a column listed more than once is written by its first entry, with the sum of all
      float q = 0.0f;
      bool first = true;
      for (int i = 0; i < a.k; i += 4) {  // four ids a load; behind the k-th they are -1
        const int4 id = *reinterpret_cast<const int4*>(ids_s + i);
        if (id.x == mine || id.y == mine || id.z == mine || id.w == mine) {
          const int same[4] = {id.x, id.y, id.z, id.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (same[j] == mine) {
              first &= i + j >= tid;
              q += q_s[i + j];
            }
        }
      }
      r.R = R;
      const float p = mine_x <= -kLogitBound && lse == lse ? 0.0f : exp2_approx(score<T>(mine_x, r)) * f;
      if (first) store_logit(dx, mine, hit * (fmaf(mass, p, -q)));
    }
  }
  if (anew && v_begin == 0) {
    if (kList)
      far_row<T, NT, kEntropy, kList>(a, x, dx, ids_s, q_s, far_s, far_red);
    else
      far_row_called<T, NT, kEntropy>(a, x, dx, far_s, far_red);
  }
}

template <typename T, int NT, int kU, bool kEntropy, bool kList>
cudaError_t launch(const LogitsGradArgs& a, bool shift, unsigned grid, unsigned chunks, int steps, cudaStream_t st) {
  if (shift)
    return launch_pdl(logits_grad_kernel<T, NT, kU, kEntropy, kList, true>, dim3(grid), dim3(NT), 0, st, a, chunks,
                      steps);
  return launch_pdl(logits_grad_kernel<T, NT, kU, kEntropy, kList, false>, dim3(grid), dim3(NT), 0, st, a, chunks,
                    steps);
}

template <typename T, int NT>
nvfp4rl_status launch_width(const LogitsGradArgs& a, cudaStream_t st) {
  constexpr int64_t VEC = kVecOf<T>;
  const auto phase = [](const void* p) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) / sizeof(T)) % VEC; };
  const bool shift = phase(a.x) != phase(a.dx) || (a.M > 1 && a.ld % VEC != a.ldd % VEC);
  const int64_t vecs = (a.V + 2 * VEC - 2) / VEC;  // of the row, at its worst phase
  const bool wide = a.M * ((vecs + 4 * NT - 1) / (4 * NT)) >= 4 * kNumSMsHint;
  const int64_t per_step = (wide ? 4 : 1) * NT;
  // a list costs its chunk a fixed part: larger chunks, where enough CTAs are left
  int64_t steps = 1;
  while (a.ids && wide && steps < 4 && a.M * ((vecs + 2 * steps * per_step - 1) / (2 * steps * per_step)) >= kListCtas) steps *= 2;
  while (steps * per_step < vecs && a.M * ((vecs + steps * per_step - 1) / (steps * per_step)) > (int64_t(1) << 30))
    steps *= 2;
  const int64_t chunks = (vecs + steps * per_step - 1) / (steps * per_step);
  const unsigned grid = static_cast<unsigned>(a.M * chunks), ch = static_cast<unsigned>(chunks);
  const int n = static_cast<int>(steps);
  cudaError_t e;
  if constexpr (NT > 64) {
    if (!a.ids) {
      if (wide)
        e = a.dentropy ? launch<T, NT, 4, true, false>(a, shift, grid, ch, n, st)
                       : launch<T, NT, 4, false, false>(a, shift, grid, ch, n, st);
      else
        e = a.dentropy ? launch<T, NT, 1, true, false>(a, shift, grid, ch, n, st)
                       : launch<T, NT, 1, false, false>(a, shift, grid, ch, n, st);
      return e == cudaSuccess ? launch_status() : NVFP4RL_ERR_CUDA;
    }
  }
  e = wide ? launch<T, NT, 4, false, true>(a, shift, grid, ch, n, st) : launch<T, NT, 1, false, true>(a, shift, grid, ch, n, st);
  return e == cudaSuccess ? launch_status() : NVFP4RL_ERR_CUDA;
}

// As many threads as the list has entries, at least 64: with 64 listed, 256, 128 and 64 threads took 381, 370, 371 us at
// 4096 x 152064 bf16, 39, 20, 14.5 us at 4096 x 1001. Without a list 256 for long rows (4096 x 152064, every row live, no
// entropy: 351.2 us, with 128 352.7), 128 for short ones (6.6 us at 4096 x 1001, with 256 9.1).
template <typename T>
nvfp4rl_status launch_type(const LogitsGradArgs& a, cudaStream_t st) {
  if (a.ids && a.k <= 64) return launch_width<T, 64>(a, st);
  const bool narrow = a.ids ? a.k <= 128 : a.V <= 4096 * kVecOf<T>;
  return narrow ? launch_width<T, 128>(a, st) : launch_width<T, 256>(a, st);
}

}  // namespace

nvfp4rl_status launch_logprobs_grad(const LogitsGradArgs& a0, int dtype, const DeviceInfo&, cudaStream_t st) {
  LogitsGradArgs a = a0;
  a.low = -0x1p17f / (a.scale * kLog2E);
  return dtype == NVFP4RL_BF16 ? launch_type<uint16_t>(a, st) : launch_type<float>(a, st);
}

}  // namespace nvfp4rl