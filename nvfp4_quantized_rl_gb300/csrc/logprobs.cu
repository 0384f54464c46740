// Log-probs of given tokens, entropy and top alternatives of rows of logits, and the divergence from a
// teacher's listed log-probs (sm_103a). One pass over the logits.
//
// Every thread keeps a running reference R = c max(x) (c = scale log2 e), s = sum 2^t and w = sum 2^t t of the logits it
// has seen, t = x c - R; a larger maximum rescales them. Over a row (R, s, w) merge by
// s 2^(R_i - R), (w + (R_i - R) s) 2^(R_i - R), and
//   lse = R ln 2 + ln s,   ln p_j = t_j ln 2 - ln s,   entropy = ln s - ln 2 (w / s).
// R is rounded, which shifts every t and s alike and drops out, but past 2^24 (a row, or a thread's part of one, of nothing
// but -1e10 or -1e30) 2^t would overflow: there t = (x - max) c, and R has a low part.
// A masked logit (at or below -2^100) gives 2^t = 0; where t itself is summed it is clamped to -2^100, which keeps t
// finite. A thread that has seen nothing else adds nothing. A NaN stays in s.
//
// Each logit is read once: bound by HBM (8192 x 152064 bf16 with entropy 352 us, 1.04 of the copy rate), and near it by
// issue slots, which is why the arithmetic is packed (8 instructions for two logits) and nothing else runs in the loop.
// A thread takes 5 x 16 bytes a step; several CTAs of 64 to 256 threads on an SM, a row to each, hide one another's row
// ends. What did not help: a cp.async ring that runs ahead over the rows' ends (410 us for 367 at the time: its copies
// and shared-memory loads cost issue slots), loading a step ahead into registers, and CTAs that stay for several rows.
// Few rows are split over clusters of 2 to 8 CTAs, whose sums and alternatives meet in the first CTA's shared memory
// (one row with 20 alternatives 8 us).
//
// Alternatives: the loop only keeps the upper half of each thread's maximum per step. At the row's end the k-th largest
// of those maxima (of the threads' first, then by a histogram of the steps') bounds the k-th largest logit from below;
// the few thread-steps that reach it are read again, dealt out over the CTA, and the logits above the bound go to a
// list in shared memory as 64-bit keys (value order, then the lower column). A list that is too long is cut by a
// histogram; the rest is ranked by counting. The result does not depend on the order of the appends. 64 of each of
// 2048 x 152064 bf16: 116 us, 0.79 of the copy rate (93 us without any), bound by the latency of the row's end; testing
// every logit against a bound in the loop took 164 us. Rows of equal logits are dearer (2048 rows of zeros 139 us).
//
// Distillation with a tail bucket: listed columns are marked in a bit map in shared memory and masked as they are
// read, so that the streamed sum is the tail's own, relative to its own maximum; the listed ones are gathered and
// added at the end. 1 - sum p would lose a small tail. 4096 x 152064 bf16, 64 listed: 192 us, 0.96 of the copy rate.
#include <atomic>

#include "logits.cuh"

namespace nvfp4rl {
namespace {

constexpr int kThreads = 256;                      // of the widest CTA
constexpr int kU = 5;                              // vectors per thread and step
constexpr int kBlock = 32;                         // steps whose maxima are kept (one bit each in a mask)
constexpr int kParts = 1024;                       // thread-steps read again together
constexpr int kMaxCluster = 8;
constexpr int kMapColumns = 1 << 18;               // columns per bit map (32 KB)
constexpr float kFarRef = 0x1p24f;                 // |R| above which R's rounding is a whole score or more
static_assert(kThreads >= kMaxListed && kThreads == 32 * kListWarps, "one thread per listed column");

enum Mode { kLogprobs = 0, kNormalized = 1, kTailBucket = 2 };

// ---- clusters ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address, in CTA `rank`, of what p is in this CTA's shared memory.
__device__ __forceinline__ uint32_t map_shared(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// ---- keys: larger value first, then the lower column; 0 is no key ----

__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are one value
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t u) { return __uint_as_float((u >> 31) ? (u & 0x7FFFFFFFu) : ~u); }
__device__ __forceinline__ unsigned long long rank_key(float v, int col) {
  return (static_cast<unsigned long long>(order_bits(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ int key_column(unsigned long long key) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

// The alternatives' shared memory of a CTA of NT threads.
template <int NT>
struct TopShared {
  static constexpr int kWarps = NT / 32;
  static constexpr int kMaxKept = NT;                      // a cut leaves at most this many keys, one to a thread
  static constexpr int kCandidates = NT / 2 * 8 + kMaxKept;  // one vector of half the threads beside a list that was cut
  static constexpr int kBins = 4 * NT;
  static constexpr int kLogBins = NT == 256 ? 10 : NT == 128 ? 9 : 8;
  static_assert(1 << kLogBins == kBins && kCandidates % 2 == 0, "four bins to a thread; keys are read in pairs");
  unsigned long long key[kCandidates];
  unsigned long long kept[kMaxKept];
  uint4 vec[NT];  // a thread's vector with candidates, to take single elements from
  uint16_t step_max[kBlock][NT];  // the upper half of every thread's maximum in each step of a block
  uint16_t part[kParts];                // step * NT + thread of those that hold candidates
  int bins[kBins];
  unsigned long long ends[2 * kWarps];
  int warp_sum[kWarps];
  uint32_t warp_bound[kWarps], warp_top[kWarps];
  int count, kept_count, above, with, bin, part_count;
  // of the cluster's first CTA, with more than one: what every CTA kept, k keys each
  __device__ __forceinline__ unsigned long long* merged() { return reinterpret_cast<unsigned long long*>(this + 1); }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float a) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The bin that holds the want-th largest entry of the histogram, and how many entries lie above it and with it. Left as
// they are where the histogram holds fewer. Called after a barrier, ends with one.
template <int NT>
__device__ void find_bin(TopShared<NT>& sh, int want) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 b4 = reinterpret_cast<const int4*>(sh.bins)[NT - 1 - tid];  // from the top: bins kBins - 1 - 4 tid and the three below
  const int sum = (b4.x + b4.y) + (b4.z + b4.w);
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sh.warp_sum[warp] = scan;
  __syncthreads();
  int above = scan - sum;
#pragma unroll
  for (int i = 0; i < TopShared<NT>::kWarps; ++i)
    if (i < warp) above += sh.warp_sum[i];
  if (above < want && above + sum >= want) {  // in one of this thread's bins
    int bin = TopShared<NT>::kBins - 1 - 4 * tid, in = b4.w;
    if (above + in < want) --bin, above += in, in = b4.z;
    if (above + in < want) --bin, above += in, in = b4.y;
    if (above + in < want) --bin, above += in, in = b4.x;
    sh.bin = bin;
    sh.above = above;
    sh.with = above + in;
  }
  __syncthreads();
}

// Cuts a list of n keys, more than kMaxKept, to those that include the k largest: at most min(k + 32, kMaxKept), in
// key[0 .. count). Returns the lower bound that the cut used (0: nothing was cut). All threads of the CTA call, after a
// barrier that follows the last append. For keys in any range, equal values among them.
template <int NT>
__device__ unsigned long long cut_long(TopShared<NT>& sh, int n, int k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, most = min(k + 32, TopShared<NT>::kMaxKept);
  unsigned long long lo = ~0ull, hi = 0;
  int keys = 0;
  for (int j = tid; j < n; j += NT) {
    const unsigned long long key = sh.key[j];
    if (key) {
      ++keys;
      lo = min(lo, key);
      hi = max(hi, key);
    }
  }
  keys = __reduce_add_sync(0xFFFFFFFFu, keys);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  if (lane == 0) {
    sh.ends[2 * warp] = lo;
    sh.ends[2 * warp + 1] = hi;
    sh.warp_sum[warp] = keys;
  }
  if (tid == 0) sh.kept_count = 0;
  auto* bins4 = reinterpret_cast<int4*>(sh.bins);
  bins4[tid] = make_int4(0, 0, 0, 0);
  __syncthreads();
  keys = 0;
#pragma unroll
  for (int i = 0; i < TopShared<NT>::kWarps; ++i) {
    keys += sh.warp_sum[i];
    lo = min(lo, sh.ends[2 * i]);
    hi = max(hi, sh.ends[2 * i + 1]);
  }
  unsigned long long cut = 0;
  if (keys > most) {
    int want = k;  // of the keys in [lo, hi]: those above are in
    while (true) {
      const int bits = 64 - __clzll(static_cast<long long>(hi - lo));
      const int shift = max(bits - TopShared<NT>::kLogBins, 0);  // (hi - lo) >> shift < kBins
      for (int j = tid; j < n; j += NT) {
        const unsigned long long key = sh.key[j];
        if (key >= lo && key <= hi) atomicAdd(&sh.bins[static_cast<int>((key - lo) >> shift)], 1);
      }
      __syncthreads();
      find_bin(sh, want);
      cut = lo + (static_cast<unsigned long long>(sh.bin) << shift);
      // keys at or above the cut: k - want of earlier rounds, and `with` (one key per bin at shift 0: k)
      if (k - want + sh.with <= most || shift == 0) break;
      want -= sh.above;
      hi = min(hi, cut + ((1ull << shift) - 1));
      lo = cut;
      bins4[tid] = make_int4(0, 0, 0, 0);
      __syncthreads();
    }
  }
  for (int j = tid; j < n; j += NT) {
    const unsigned long long key = sh.key[j];
    if (key && key >= cut) sh.kept[atomicAdd(&sh.kept_count, 1)] = key;
  }
  __syncthreads();
  const int kept = sh.kept_count;
  for (int i = tid; i < kept; i += NT) sh.key[i] = sh.kept[i];
  if (tid == 0) sh.count = kept;
  __syncthreads();
  return cut;
}

// The same for a list whose values lie above thr and at most at the threads' maxima m: one histogram of the values'
// order bits, without the reductions of the keys' range, and cut_long only where too many keys share the cut's bin.
template <int NT>
__device__ unsigned long long cut_values(TopShared<NT>& sh, int n, int k, float thr, float m) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, most = min(k + 32, TopShared<NT>::kMaxKept);
  const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, order_bits(m));
  if (lane == 0) sh.warp_bound[warp] = top;
  if (tid == 0) {
    sh.kept_count = 0;
    sh.bin = 0;  // fewer than k: all stay
    sh.with = n;
  }
  auto* bins4 = reinterpret_cast<int4*>(sh.bins);
  bins4[tid] = make_int4(0, 0, 0, 0);
  __syncthreads();
  const uint32_t lo = order_bits(thr);
  uint32_t hi = lo;
#pragma unroll
  for (int i = 0; i < TopShared<NT>::kWarps; ++i) hi = max(hi, sh.warp_bound[i]);
  const int shift = max(32 - TopShared<NT>::kLogBins - __clz((hi - lo) | 1u), 0);  // (hi - lo) >> shift < kBins
  for (int j = tid; j < n; j += NT)
    atomicAdd(&sh.bins[(static_cast<uint32_t>(sh.key[j] >> 32) - lo) >> shift], 1);
  __syncthreads();
  find_bin(sh, k);
  if (sh.with > most) {
    __syncthreads();
    return cut_long(sh, n, k);
  }
  const uint32_t cut = lo + (static_cast<uint32_t>(sh.bin) << shift);
  for (int j = tid; j < n; j += NT) {
    const unsigned long long key = sh.key[j];
    if (static_cast<uint32_t>(key >> 32) >= cut) sh.kept[atomicAdd(&sh.kept_count, 1)] = key;
  }
  __syncthreads();
  const int kept = sh.kept_count;
  if (tid < kept) sh.key[tid] = sh.kept[tid];
  if (tid == 0) sh.count = kept;
  __syncthreads();
  return static_cast<unsigned long long>(cut) << 32;
}

// The k largest of at most kMaxKept keys, in order, in sh.key[0 .. count): every key counts those above it, with 4, 2 or 1
// threads to a key, two keys a load. Returns the k-th (0: there are fewer). Called as cut_long.
template <int NT>
__device__ unsigned long long sort_short(TopShared<NT>& sh, int n, int k) {
  const int p = n <= NT / 4 ? 2 : n <= NT / 2 ? 1 : 0, parts = 1 << p;
  const int i = static_cast<int>(threadIdx.x) >> p, part = threadIdx.x & (parts - 1);
  const unsigned long long key = i < n ? sh.key[i] : 0ull;
  int rank = 0;
  if (__any_sync(0xFFFFFFFFu, key != 0)) {
    const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(sh.key);
#pragma unroll 4
    for (int j = part; 2 * j < n; j += parts) {
      const ulonglong2 v = pairs[j];
      rank += (v.x > key) + (v.y > key && 2 * j + 1 < n);
    }
    for (int o = 1; o < parts; o <<= 1) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, o);
  }
  const bool in = part == 0 && key && rank < k;
  const int kept = __syncthreads_count(in);
  if (in) sh.key[rank] = key;
  if (threadIdx.x == 0) sh.count = kept;
  __syncthreads();
  return kept == k ? sh.key[k - 1] : 0ull;
}

// Of `lists` sorted lists of k keys each (0 where there is none, at the end) those that can be among the k largest, into
// sh.key: ceil(k / lists) keys of every list reach the least of the lists' ceil(k / lists)-th keys.
template <int NT>
__device__ void gather_lists(TopShared<NT>& sh, const unsigned long long* from, int lists, int k) {
  const int each = (k + lists - 1) / lists, tid = threadIdx.x;
  unsigned long long bound = ~0ull;
  for (int l = 0; l < lists; ++l) bound = min(bound, from[l * k + each - 1]);
  if (tid == 0) sh.count = 0;
  __syncthreads();
  for (int i = tid; i < lists * k; i += NT) {
    const unsigned long long key = from[i];
    if (key && key >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < TopShared<NT>::kCandidates) sh.key[at] = key;
    }
  }
  __syncthreads();
  if (sh.count <= TopShared<NT>::kCandidates) return;
  // Too many reach the bound (it is 0 where a list is short; or most of the largest are in few of the lists, as in a rising
  // row): list by list, cut to a list's length each time.
  int n = 0;
  __syncthreads();
  for (int l = 0; l < lists; ++l) {
    if (tid < k) sh.key[n + tid] = from[l * k + tid];
    __syncthreads();
    cut_long(sh, n + k, k);
    n = sh.count;
    __syncthreads();
  }
}

// The k largest of the list, in order, in key[0 .. count). Counting costs n^2 / 3 instructions of a warp, a cut about 1200.
template <int NT>
__device__ void sort_list(TopShared<NT>& sh, int k) {
  int n = sh.count;
  if (n > TopShared<NT>::kMaxKept) {
    cut_long(sh, n, k);
    n = sh.count;
  }
  sort_short(sh, n, k);
}

// ---- the streamed sums ----

// s, w relative to the largest logit m
struct RowSum {
  float m, s, w;
};

// The reference of a maximum m: R = fl(m c), and its low part, kept where R is far.
__device__ __forceinline__ float ref_of(float m, float c) { return __fmul_rn(m, c); }
__device__ __forceinline__ float ref_low(float m, float R, float c) { return fabsf(R) > kFarRef ? fmaf(m, c, -R) : 0.0f; }
// The score of x relative to m.
__device__ __forceinline__ float score_from(float x, float m, float c) {
  const float R = ref_of(m, c);
  return fmaf(x, c, -R) - ref_low(m, R, c);
}
// The reference of a relative to that of b. (Far bf16 maxima are equal or 2^15 scores apart: no low parts.)
template <typename T>
__device__ __forceinline__ float ref_diff(float a, float Ra, float b, float Rb, float c) {
  const float d = Ra - Rb;
  return sizeof(T) == 4 ? d + (ref_low(a, Ra, c) - ref_low(b, Rb, c)) : d;
}
// The same for a <= b, no lower than where 2^d is 0: d s stays finite.
template <typename T>
__device__ __forceinline__ float ref_down(float a, float Ra, float b, float Rb, float c) {
  return fmaxf(ref_diff<T>(a, Ra, b, Rb, c), -16384.0f);
}
// ln sum exp: scale m and ln s, without what the rounding of a near R put into s.
__device__ __forceinline__ float ref_lse(float m, float c, float scale, float ln_s) {
  const float R = ref_of(m, c);
  return fmaf(m, scale, fabsf(R) > kFarRef ? ln_s : fmaf(-fmaf(m, c, -R), kLn2, ln_s));
}

// a, relative to a maximum m of several.
template <typename T>
__device__ __forceinline__ RowSum moved(const RowSum& a, float m, float c) {
  const float d = ref_down<T>(a.m, ref_of(a.m, c), m, ref_of(m, c), c), f = exp2_approx(d);
  return RowSum{m, a.s * f, fmaf(d, a.s, a.w) * f};
}
// The sum of n parts, n <= N, in their order.
template <typename T, int N>
__device__ __forceinline__ RowSum merged(const RowSum* parts, int n, float c) {
  float m = parts[0].m;
#pragma unroll
  for (int i = 1; i < N; ++i)
    if (i < n) m = max_nan(m, parts[i].m);
  RowSum sum{m, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) {
      const RowSum a = moved<T>(parts[i], m, c);
      sum.s += a.s;
      sum.w += a.w;
    }
  return sum;
}

template <typename T>
__device__ __forceinline__ uint4 masked_vec() {
  const uint32_t w = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  return make_uint4(w, w, w, w);
}

__device__ __forceinline__ float elem(const uint32_t (&w)[4], int i, uint16_t) {
  return __uint_as_float((i & 1) ? bf16_hi_bits(w[i >> 1]) : bf16_lo_bits(w[i >> 1]));
}
__device__ __forceinline__ float elem(const uint32_t (&w)[4], int i, float) { return __uint_as_float(w[i & 3]); }

template <typename T>
__device__ __forceinline__ void set_masked(uint32_t (&w)[4], int i) {
  if (sizeof(T) == 2)
    w[i >> 1] = (i & 1) ? (w[i >> 1] & 0x0000FFFFu) | 0xFF800000u : (w[i >> 1] & 0xFFFF0000u) | 0x0000FF80u;
  else
    w[i & 3] = 0xFF800000u;
}

__device__ __forceinline__ uint4 clamp_masked(const uint4& x, uint16_t) {
  constexpr uint32_t kLow = 0xF180F180u;  // -2^100, twice
  return make_uint4(max_nan_bf16x2(x.x, kLow), max_nan_bf16x2(x.y, kLow), max_nan_bf16x2(x.z, kLow),
                    max_nan_bf16x2(x.w, kLow));
}
__device__ __forceinline__ uint4 clamp_masked(const uint4& x, float) {
  const auto f = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), -kLogitBound)); };
  return make_uint4(f(x.x), f(x.y), f(x.z), f(x.w));
}
// x - m. Rounding to bf16 is free here: bf16 logits below a far m are 2^15 scores or more below it.
__device__ __forceinline__ uint4 minus_max(const uint4& x, float m, uint16_t) {
  const uint32_t m2 = (__float_as_uint(m) >> 16) * 0x10001u;
  const auto f = [&](uint32_t w) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(m2));
    return r;
  };
  return make_uint4(f(x.x), f(x.y), f(x.z), f(x.w));
}
__device__ __forceinline__ uint4 minus_max(const uint4& x, float m, float) {
  const auto f = [&](uint32_t w) { return __float_as_uint(__uint_as_float(w) - m); };
  return make_uint4(f(x.x), f(x.y), f(x.z), f(x.w));
}
__device__ __forceinline__ float vector_max(const uint4& x, uint16_t) {
  const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(x.x, x.y), max_nan_bf16x2(x.z, x.w));
  return max_nan(__uint_as_float(bf16_lo_bits(m)), __uint_as_float(bf16_hi_bits(m)));
}
__device__ __forceinline__ float vector_max(const uint4& x, float) {
  return max_nan(max_nan(__uint_as_float(x.x), __uint_as_float(x.y)), max_nan(__uint_as_float(x.z), __uint_as_float(x.w)));
}

// The vector at column col of a row of V: what lies outside is masked.
template <typename T>
__device__ __forceinline__ uint4 load_edge(const T* x, int col, int V) {
  constexpr int VEC = kVecOf<T>;
  if (col >= 0 && col + VEC <= V) return ld_logits16(x + col);
  uint4 r = masked_vec<T>();
#pragma unroll 1
  for (int i = VEC - 1; i >= 0; --i) {  // the elements enter at the low end, the last one first
    const bool in = col + i >= 0 && col + i < V;
    if (sizeof(T) == 2) {
      const uint32_t b = in ? __float_as_uint(logit(x, col + i)) >> 16 : 0xFF80u;
      r = make_uint4((r.x << 16) | b, __funnelshift_l(r.x, r.y, 16), __funnelshift_l(r.y, r.z, 16),
                     __funnelshift_l(r.z, r.w, 16));
    } else {
      r = make_uint4(in ? __float_as_uint(logit(x, col + i)) : 0xFF800000u, r.x, r.y, r.z);
    }
  }
  return r;
}

struct Shared {
  RowSum sums[kThreads / 32];
  RowSum parts[kMaxCluster];
};
struct ListShared {
  int32_t ids[kMaxListed];
  TeacherShared teacher;
  float top[kListWarps];
  float2 sum[2][kListWarps];
};

// The elements of a vector above the bound, as a mask: bit (i >> 1) + 16 (i & 1) for element i. The bound is rounded
// down to bf16 (a negative one away from zero): no candidate is lost, the keys decide.
__device__ __forceinline__ uint32_t above_mask(const uint4& x, float thr, uint16_t) {
  const uint32_t b = __float_as_uint(thr), t = (b >> 16) + (b > 0x80000000u && (b & 0xFFFFu)), t2 = t | (t << 16);
  const auto gt = [&](uint32_t w) {
    uint32_t r;
    asm("set.gt.u32.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(t2));
    return r;
  };
  return (gt(x.x) & 0x00010001u) | (gt(x.y) & 0x00020002u) | (gt(x.z) & 0x00040004u) | (gt(x.w) & 0x00080008u);
}
__device__ __forceinline__ uint32_t above_mask(const uint4& x, float thr, float) {
  return (__uint_as_float(x.x) > thr ? 0x00001u : 0u) | (__uint_as_float(x.y) > thr ? 0x10000u : 0u) |
         (__uint_as_float(x.z) > thr ? 0x00002u : 0u) | (__uint_as_float(x.w) > thr ? 0x20000u : 0u);
}

// The vector's columns above the bound go to the list; a full list drops them (the caller sees it by the count).
template <int NT, typename T>
__device__ __forceinline__ void append(TopShared<NT>& sh, const uint4& x, int col, float thr) {
  uint32_t mask = above_mask(x, thr, T());
  if (!mask) return;
  int at = atomicAdd(&sh.count, __popc(mask));
  sh.vec[threadIdx.x] = x;
  const T* mine = reinterpret_cast<const T*>(&sh.vec[threadIdx.x]);
  do {
    const int bit = __ffs(mask) - 1, i = 2 * (bit & 15) + (bit >> 4);
    mask &= mask - 1;
    if (at < TopShared<NT>::kCandidates) sh.key[at] = rank_key(logit(mine, i), col + i);
    ++at;
  } while (mask);
}

// The bound that a cut at `cut` gives: later columns with its value rank behind the k kept.
__device__ __forceinline__ void raise(float& thr, unsigned long long cut) {
  if (cut) thr = fmaxf(thr, order_value(static_cast<uint32_t>(cut >> 32)));
}

// The value before the least one with these upper 16 order bits (-0 is +0).
template <typename T>
__device__ __forceinline__ float before(uint32_t t) {
  t -= t == 0x8000u ? 2u : t > 0u ? 1u : 0u;
  return order_value(sizeof(T) == 2 ? t << 16 : (t << 16) | 0xFFFFu);
}

// A lower bound of the k-th largest logit, for columns above it: every warp's ceil(k / 8)-th largest thread maximum, to 16
// bits; at least k maxima reach the least of them, and the bound is the value before that one.
template <int NT, typename T>
__device__ __forceinline__ float first_bound(TopShared<NT>& sh, float m, int k) {
  const uint32_t key = order_bits(fmaxf(m, -kLogitBound)) >> 16;
  const int each = (k + TopShared<NT>::kWarps - 1) / TopShared<NT>::kWarps;
  uint32_t t = __reduce_max_sync(0xFFFFFFFFu, key);
  if (each <= 4) {  // the next smaller maximum, till enough reach it
    int reach = __popc(__ballot_sync(0xFFFFFFFFu, key == t));
    while (reach < each) {
      t = __reduce_max_sync(0xFFFFFFFFu, key < t ? key : 0u);
      reach = __popc(__ballot_sync(0xFFFFFFFFu, key >= t));
    }
  } else {
    uint32_t low = __reduce_min_sync(0xFFFFFFFFu, key);  // all reach it
#pragma unroll 1
    for (uint32_t step = 0x80000000u >> __clz((t - low) | 1u); step; step >>= 1)
      if (low + step <= t && __popc(__ballot_sync(0xFFFFFFFFu, key >= low + step)) >= each) low += step;
    t = low;
  }
  if ((threadIdx.x & 31) == 0) sh.warp_bound[threadIdx.x >> 5] = t;
  reinterpret_cast<int4*>(sh.bins)[threadIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TopShared<NT>::kWarps; ++i) t = min(t, sh.warp_bound[i]);
  return fmaxf(before<T>(t), -kLogitBound);  // of NaN: the bound
}

// A step's maximum of this thread, in order, to 16 bits (rounded down).
template <int NT>
__device__ __forceinline__ uint32_t step_order(const TopShared<NT>& sh, int step) {
  return order_bits(__uint_as_float(static_cast<uint32_t>(sh.step_max[step][threadIdx.x]) << 16)) >> 16;
}

// Whether this thread's logits of a step may exceed the bound: exactly for bf16, with a rounded maximum for fp32.
template <int NT, typename T>
__device__ __forceinline__ bool may_exceed(const TopShared<NT>& sh, int step, float thr) {
  if (sizeof(T) == 2) return __uint_as_float(static_cast<uint32_t>(sh.step_max[step][threadIdx.x]) << 16) > thr;
  return step_order(sh, step) >= max(order_bits(thr) >> 16, (order_bits(-kLogitBound) >> 16) + 1);  // not the masked
}

// Where the first bound lets many more than k steps pass (mask: this thread's): the k-th largest of all the block's step
// maxima is a lower bound too, found by one histogram of them. Returns the steps that pass it.
template <int NT, typename T>
__device__ uint32_t refine_bound(TopShared<NT>& sh, uint32_t mask, int k, float& thr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int all = __reduce_add_sync(0xFFFFFFFFu, __popc(mask));
  uint32_t hi = 0;
  for (uint32_t left = mask; left; left &= left - 1) hi = max(hi, step_order(sh, __ffs(left) - 1));
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  if (lane == 0) {
    sh.warp_sum[warp] = all;
    sh.warp_top[warp] = hi;
  }
  __syncthreads();
  int steps = 0;
#pragma unroll
  for (int i = 0; i < TopShared<NT>::kWarps; ++i) {
    steps += sh.warp_sum[i];
    hi = max(hi, sh.warp_top[i]);
  }
  if (steps <= k + 48) return mask;
  const uint32_t lo = order_bits(thr) >> 16;
  const int shift = max(32 - TopShared<NT>::kLogBins - __clz((hi - lo) | 1u), 0);  // (hi - lo) >> shift < kBins
  for (uint32_t left = mask; left; left &= left - 1)
    atomicAdd(&sh.bins[(step_order(sh, __ffs(left) - 1) - lo) >> shift], 1);
  __syncthreads();
  find_bin(sh, k);
  const uint32_t t = lo + (static_cast<uint32_t>(sh.bin) << shift);  // at least k steps reach it
  uint32_t pass = 0;
  for (uint32_t left = mask; left; left &= left - 1)
    if (step_order(sh, __ffs(left) - 1) >= t) pass |= left & (0u - left);
  thr = fmaxf(thr, before<T>(t));
  return pass;
}

// CTAs to an SM. Five of 256 threads where 48 registers do: 2048 x 152064 bf16 (floor 92 us), without alternatives, 4
// vectors and 4 CTAs 106 us, 4 and 5 99 us, 5 and 5 96 us, 6 and 5 98 us, 8 and 4 99 us. With 64 alternatives: 4 CTAs of
// 256 threads 124 us, 5 163 us (spills), 6, 7, 8 CTAs of 128 threads 134, 119, 121 us. fp32 takes the same numbers: 4096 x
// 152064 (floor 367 us) with entropy 355 us, with 20 and 64 alternatives 382 and 408 us; its entropy kernels, its
// alternatives with 256 threads and the bf16 tail kernels spill 4 to 12 bytes at these bounds.
template <bool kTop, int NT>
constexpr int kPerSm = NT == 256 ? (kTop ? 4 : 5) : NT == 128 ? (kTop ? 7 : 10) : (kTop ? 13 : 18);

// kEntropy: w is kept; kTop: alternatives are listed (both kLogprobs only).
template <typename T, int kMode, bool kEntropy, bool kTop, int NT>
__global__ void __launch_bounds__(NT, kPerSm<kTop, NT>) logits_row_kernel(const LogitsArgs a, uint32_t cluster) {
  constexpr int VEC = kVecOf<T>;
  constexpr bool kDistill = kMode != kLogprobs;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  TopShared<NT>& top = *reinterpret_cast<TopShared<NT>*>(dyn);                  // kTop
  ListShared& list = *reinterpret_cast<ListShared*>(dyn);               // kDistill
  uint32_t* map = reinterpret_cast<uint32_t*>(dyn + sizeof(ListShared));  // kTailBucket
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
  const int64_t row = blockIdx.x / cluster;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = static_cast<int>(a.V), k = a.k;
  const int phase = vec_phase(x);
  const int vecs = (V + phase + VEC - 1) / VEC;  // vector v: columns v VEC - phase ..
  const int share = (vecs + static_cast<int>(cluster) - 1) / static_cast<int>(cluster);
  const int v_begin = static_cast<int>(rank) * share, v_end = min(v_begin + share, vecs);
  uint4 in[kU];
  const auto load_step = [&](int v0) {
    if (v0 * VEC >= phase && v0 + kU * NT <= v_end && (v0 + kU * NT) * VEC - phase <= V) {
      const T* at = x + ((v0 + tid) * VEC - phase);
#pragma unroll
      for (int u = 0; u < kU; ++u) in[u] = ld_logits16(at + u * (NT * VEC));
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int v = v0 + u * NT + tid;
        in[u] = v < v_end ? load_edge(x, v * VEC - phase, V) : masked_vec<T>();
      }
    }
  };
  load_step(v_begin);  // beside what the row needs else
  constexpr int kMapVecs = kMapColumns / VEC / (kU * NT) * (kU * NT);
  int map_begin = v_begin;  // first vector of the bit map
  const auto clear_map = [&]() {
    const int words = (min(v_end - map_begin, kMapVecs) * VEC + 31) / 32;
    for (int i = tid; i < words; i += NT) map[i] = 0;
  };
  // listed columns: thread i holds entry i
  int id = -1, token = -1;
  float listed_l = -INFINITY, listed_x = -INFINITY;
  const auto mark_map = [&]() -> bool {  // whether the column was marked already
    const int v = id >= 0 ? (id + phase) / VEC : -1;
    if (v < map_begin || v >= min(v_end, map_begin + kMapVecs)) return false;
    const int bit = id + phase - map_begin * VEC;
    const uint32_t was = atomicOr(&map[bit >> 5], 1u << (bit & 31));
    return was >> (bit & 31) & 1u;
  };
  bool twice = true;  // a column may be listed twice
  if (kDistill) {
    if (tid < k) {
      id = a.ids[row * k + tid];
      listed_l = a.teacher[row * k + tid];
      if (id < 0 || id >= V) id = -1;
      list.ids[tid] = id;
    }
    if (kMode == kTailBucket) clear_map();
    if (!__syncthreads_or(id >= 0)) {  // in every CTA of the cluster
      if (rank == 0 && tid == 0) {
        a.loss[row] = 0.0f;
        if (a.lse) a.lse[row] = 0.0f;
        if (kMode == kTailBucket && a.lse_tail) a.lse_tail[row] = 0.0f;
      }
      return;
    }
    if (rank == 0 && id >= 0) listed_x = logit(x, id);
    if (kMode == kTailBucket) {
      twice = __syncthreads_or(mark_map());
      twice |= cluster > 1 || v_end - v_begin > kMapVecs;  // other maps may know of others
    }
  } else if (a.tokens) {
    token = a.tokens[row];
    if (token < 0 || token >= V) {
      if (rank == 0) {
        if (tid == 0) {
          if (a.logp) a.logp[row] = 0.0f;
          if (a.entropy) a.entropy[row] = 0.0f;
          if (a.lse) a.lse[row] = 0.0f;
        }
        if (kTop)
          for (int i = tid; i < k; i += NT) {
            a.top_ids[row * k + i] = -1;
            a.top_logp[row * k + i] = -INFINITY;
          }
      }
      return;
    }
  }

  if (cluster > 1) cluster_arrive();
  const float at_token = kMode == kLogprobs && tid == 0 && token >= 0 ? logit(x, token) : 0.0f;
  const float c = a.scale * kLog2E;
  float m = -kLogitBound, R = ref_of(m, c), thr = -kLogitBound;
  F2 s2 = pack2(0.0f, 0.0f), w2 = pack2(0.0f, 0.0f);
  const F2 c2 = pack2(c, c);
  if (kTop && tid == 0) top.count = top.part_count = 0;
  int block_begin = v_begin;  // first vector of the block

  const auto warp_sums = [&]() {  // the warp's sums to shared memory; a barrier has to follow
    float lo, hi, wlo, whi;
    unpack2(s2, lo, hi);
    unpack2(w2, wlo, whi);
    RowSum sum = moved<T>(RowSum{m, lo + hi, wlo + whi}, warp_max_nan(m), c);
    sum.s = warp_sum(sum.s);
    if (kEntropy) sum.w = warp_sum(sum.w);
    if (lane == 0) sh.sums[warp] = sum;
  };

  for (int v0 = v_begin; v0 < v_end; v0 += kU * NT) {
    if (kMode == kTailBucket && v0 - map_begin >= kMapVecs) {  // the listed columns of the next kMapVecs vectors
      __syncthreads();
      map_begin = v0;
      clear_map();
      __syncthreads();
      mark_map();
      __syncthreads();
    }
    if (v0 > v_begin) load_step(v0);
    if (kMode == kTailBucket) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int v = v0 + u * NT + tid;
        if (v < v_end) {
          const int at = (v - map_begin) * VEC;
          const uint32_t bits = (map[at >> 5] >> (at & 31)) & ((1u << VEC) - 1u);
          if (bits) {
            uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (bits >> i & 1) set_masked<T>(w, i);
            in[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    if (kEntropy) {  // masked logits clamped to -2^100: 2^t t has to be 0 there (2^t alone is, for -inf too)
#pragma unroll
      for (int u = 0; u < kU; ++u) in[u] = clamp_masked(in[u], T());
    }
    float cm = vector_max(in[0], T());
#pragma unroll
    for (int u = 1; u < kU; ++u) cm = max_nan(cm, vector_max(in[u], T()));
    if (!(cm <= m)) {  // larger, or NaN (which stays)
      const float Rn = ref_of(cm, c), d = ref_down<T>(m, R, cm, Rn, c), f = exp2_approx(d);
      const F2 f2 = pack2(f, f);
      if (kEntropy) w2 = mul2(fma2(pack2(d, d), s2, w2), f2);
      s2 = mul2(s2, f2);
      R = Rn;
      m = max_nan(m, cm);  // a NaN stays: no listed value lies above the largest m (cut_values)
    }
    if (!(m <= -kLogitBound)) {
      float ref = -R;
      if (fabsf(R) > kFarRef) {
#pragma unroll
        for (int u = 0; u < kU; ++u) in[u] = minus_max(in[u], m, T());
        ref = 0.0f;
      }
      const F2 r2 = pack2(ref, ref);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const F2 t = fma2(pack2(elem(w, 2 * i, T()), elem(w, 2 * i + 1, T())), c2, r2);
          float t0, t1;
          unpack2(t, t0, t1);
          const F2 e = pack2(exp2_approx(t0), exp2_approx(t1));
          s2 = add2(s2, e);
          if (kEntropy) w2 = fma2(e, t, w2);
        }
      }
    }
    if (kTop) {
      const int step = (v0 - block_begin) / (kU * NT);
      top.step_max[step][tid] = static_cast<uint16_t>(__float_as_uint(cm) >> 16);
      if (step < kBlock - 1 && v0 + kU * NT < v_end) continue;
      if (v0 + kU * NT >= v_end) warp_sums();
      // The block's end (of the row, but for the longest): the steps that hold a candidate are read again.
      if (block_begin == v_begin)
        thr = first_bound<NT, T>(top, m, k);  // and the bins are clear
      else
        __syncthreads();  // part_count is 0
      uint32_t mask = 0;
      for (int i = 0; i <= step; ++i)
        if (may_exceed<NT, T>(top, i, thr)) mask |= 1u << i;
      if (block_begin == v_begin) mask = refine_bound<NT, T>(top, mask, k, thr);
      // The thread-steps with candidates are listed, and their vectors dealt out to the threads: all loads of a row's
      // end go out together (thread by thread their latencies would add up, 6000 cycles under load).
      if (mask) {
        int at = atomicAdd(&top.part_count, __popc(mask));
        for (uint32_t left = mask; left; left &= left - 1, ++at)
          if (at < kParts) top.part[at] = static_cast<uint16_t>((__ffs(left) - 1) * NT + tid);
      }
      __syncthreads();
      const int parts = top.part_count;
      if (parts <= kParts) {
        constexpr int kBatch = 2;
        for (int i = tid; i < parts * kU; i += kBatch * NT) {
          uint4 y[kBatch];
          int col[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int q = i + j * NT;
            y[j] = masked_vec<T>();
            col[j] = 0;
            if (q < parts * kU) {
              const int part = top.part[q / kU];
              const int v = block_begin + (part / NT * kU + q % kU) * NT + part % NT;
              col[j] = v * VEC - phase;
              if (v < v_end) y[j] = load_edge(x, col[j], V);
            }
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (vector_max(y[j], T()) > thr) append<NT, T>(top, y[j], col[j], thr);
        }
      }
      __syncthreads();
      if (tid == 0) top.part_count = 0;
      const int n = parts <= kParts ? top.count : TopShared<NT>::kCandidates + 1;
      if (n > TopShared<NT>::kCandidates) {
        // More than find a place (equal values): what the block appended goes, and it is appended again in parts
        // that a list that was cut can take, one vector of half the threads. The first cuts raise the bound, and what
        // cannot exceed it any more is passed over.
        const int from = block_begin * VEC - phase;
        const int held = min(top.count, TopShared<NT>::kCandidates);
        for (int i = tid; i < held; i += NT)
          if (key_column(top.key[i]) >= from) top.key[i] = 0;
        __syncthreads();
        raise(thr, cut_long(top, held, k));
#pragma unroll 1
        for (int i = 0; i <= step; ++i) {
          if (!__syncthreads_or(may_exceed<NT, T>(top, i, thr))) continue;
#pragma unroll 1
          for (int half = 0; half < 2 * kU; ++half) {
            const int v = block_begin + (i * kU + (half >> 1)) * NT + tid;
            const bool mine = tid / (NT / 2) == (half & 1) && v < v_end && may_exceed<NT, T>(top, i, thr);
            if (!__syncthreads_or(mine)) continue;
            if (mine) {
              const int col = v * VEC - phase;
              append<NT, T>(top, load_edge(x, col, V), col, thr);
            }
            __syncthreads();
            const int now = top.count;
            if (now > TopShared<NT>::kMaxKept) raise(thr, cut_long(top, now, k));
            __syncthreads();
          }
        }
      } else if (v0 + kU * NT < v_end && n > k) {
        raise(thr, cut_values(top, n, k, thr, m));
      }
      block_begin = v0 + kU * NT;
    }
  }

  // the CTA's sums, then the cluster's, in a fixed order
  if (!kTop || v_begin >= v_end) {
    warp_sums();
    __syncthreads();
  }
  RowSum sum = merged<T, NT / 32>(sh.sums, NT / 32, c);
  if (kTop) {
    if (top.count > 128) cut_values(top, top.count, k, thr, m);
    sort_list(top, k);
  }
  if (cluster > 1) {
    cluster_wait();  // every CTA has started (the arrival at the kernel's start): its shared memory is there
    if (tid == 0) {
      const uint32_t at = map_shared(&sh.parts[rank], 0);
      st_cluster(at, sum.m);
      st_cluster(at + 4, sum.s);
      st_cluster(at + 8, sum.w);
    }
    if (kTop && tid < k) st_cluster(map_shared(top.merged() + rank * k + tid, 0), tid < top.count ? top.key[tid] : 0ull);
    cluster_arrive();
    cluster_wait();
    if (rank > 0) return;
    sum = merged<T, kMaxCluster>(sh.parts, static_cast<int>(cluster), c);
    if (kTop) {
      gather_lists(top, top.merged(), static_cast<int>(cluster), k);
      sort_list(top, k);
    }
  }
  if (sum.m > kLogitBound) sum.s = NAN;  // a logit above 2^100

  if (kDistill) {
    float q, lq;
    const TeacherRow t = teacher_row<NT / 32>(list.teacher, id, listed_l, kMode == kTailBucket, q, lq);
    const float s_tail = sum.s;
    const float R1 = ref_of(sum.m, c);
    float m2 = sum.m;
    if (kMode == kTailBucket) {
      m2 = fmaxf(m2, cta_max<NT / 32>(fmaxf(listed_x, -kLogitBound), list.top));
      const bool bad = listed_x != listed_x || listed_x > kLogitBound;
      bool once = id >= 0 && listed_x > -kLogitBound;  // the first entry of its column
      if (once && twice)
        for (int j = 0; j < tid; ++j) once &= list.ids[j] != id;
      const float e = bad ? NAN : once ? exp2_approx(score_from(listed_x, m2, c)) : 0.0f;
      sum.s = fmaf(s_tail, exp2_approx(ref_down<T>(sum.m, R1, m2, ref_of(m2, c), c)), cta_sum<NT / 32>(make_float2(e, 0.0f), list.sum[0]).x);
    }
    const bool empty = sum.s == 0.0f;
    const float ln_s = logf(sum.s);
    float part = 0.0f;
    if (id >= 0 && q != 0.0f) {
      const float lp = empty || listed_x <= -kLogitBound ? -INFINITY : score_from(listed_x, m2, c) * kLn2 - ln_s;
      part = q * (lq - lp);
    }
    part = cta_sum<NT / 32>(make_float2(part, 0.0f), list.sum[1]).x;
    if (tid == 0) {
      const float ln_tail = logf(s_tail);
      if (kMode == kTailBucket && t.q0 > 0.0f && s_tail > 0.0f)
        part += t.q0 * (logf(t.q0) - (fmaf(ref_diff<T>(sum.m, R1, m2, ref_of(m2, c), c), kLn2, ln_tail) - ln_s));
      // NORMALIZED with every l_i at -inf: the row does not count
      a.loss[row] = !t.any ? 0.0f : sum.s != sum.s ? NAN : part;
      if (a.lse) a.lse[row] = !t.any ? 0.0f : empty ? -INFINITY : ref_lse(m2, c, a.scale, ln_s);
      if (kMode == kTailBucket && a.lse_tail)
        a.lse_tail[row] = sum.s != sum.s ? NAN : s_tail == 0.0f ? -INFINITY : ref_lse(sum.m, c, a.scale, ln_tail);
    }
    return;
  }

  const bool bad = sum.s != sum.s, empty = sum.s == 0.0f;
  const float ln_s = logf(sum.s);
  if (tid == 0) {
    if (a.logp)
      a.logp[row] = bad ? NAN : empty || at_token <= -kLogitBound ? -INFINITY
                                                                  : score_from(at_token, sum.m, c) * kLn2 - ln_s;
    if (kEntropy) {
      const float h = empty ? 0.0f : ln_s - kLn2 * (sum.w / sum.s);
      a.entropy[row] = h < 0.0f ? 0.0f : h;
    }
    if (a.lse) a.lse[row] = empty ? -INFINITY : ref_lse(sum.m, c, a.scale, ln_s);
  }
  if (kTop && tid < k) {
    const unsigned long long key = tid < top.count && !bad ? top.key[tid] : 0ull;
    a.top_ids[row * k + tid] = key ? key_column(key) : -1;
    a.top_logp[row * k + tid] =
        bad ? NAN : key ? score_from(order_value(static_cast<uint32_t>(key >> 32)), sum.m, c) * kLn2 - ln_s : -INFINITY;
  }
}

template <typename T, int kMode, bool kEntropy, bool kTop, int NT>
nvfp4rl_status launch(const LogitsArgs& a, unsigned cluster, const DeviceInfo& dev, cudaStream_t st) {
  size_t smem = kTop ? sizeof(TopShared<NT>) + (cluster > 1 ? static_cast<size_t>(cluster) * a.k * 8 : 0) : kMode == kLogprobs ? 0 : sizeof(ListShared);
  if (kMode == kTailBucket) {
    const int64_t share = (a.V + 2 * kVecOf<T>) / cluster + 2 * kVecOf<T>;
    smem += align_up(static_cast<size_t>(std::min<int64_t>(share, kMapColumns) + 31) / 8 + 4, 16);
  }
  auto* kernel = logits_row_kernel<T, kMode, kEntropy, kTop, NT>;
  if (kTop || kMode == kTailBucket) {  // more than 48 KB of shared memory with the static part: asked for once per device
    static std::atomic<uint64_t> asked{0};
    const uint64_t bit = uint64_t(1) << (dev.device & 63);
    if (!(asked.load(std::memory_order_relaxed) & bit)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess)
        return NVFP4RL_ERR_CUDA;
      asked.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.M) * cluster);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, cluster) == cudaSuccess ? launch_status() : NVFP4RL_ERR_CUDA;
}

template <typename T, int NT>
nvfp4rl_status launch_width(const LogitsArgs& a, unsigned cluster, const DeviceInfo& dev, cudaStream_t st) {
  if (a.ids) return a.tail ? launch<T, kTailBucket, false, false, NT>(a, cluster, dev, st)
                           : launch<T, kNormalized, false, false, NT>(a, cluster, dev, st);
  if (a.k > 0)
    return a.entropy ? launch<T, kLogprobs, true, true, NT>(a, cluster, dev, st)
                     : launch<T, kLogprobs, false, true, NT>(a, cluster, dev, st);
  return a.entropy ? launch<T, kLogprobs, true, false, NT>(a, cluster, dev, st)
                   : launch<T, kLogprobs, false, false, NT>(a, cluster, dev, st);
}

// Threads per row, of rows that are not split: narrow CTAs, more of them, where there are enough rows to fill the SMs, the
// rows are short or their ends dear. Measured with 256, 128, 64 threads, bf16, in us (ent: entropy, top: 20 alternatives,
// tail: 32 listed): 400 x 16000 ent 6.7, 5.3, 6.6, top 9.4, 7.9, 9.8, tail 9.1, 7.4, 9.4; 1064 x 8000 ent 7.4, 6.6, 6.6,
// top 14.1, 9.3, 9.8, tail 10.9, 9.3, 8.1; 2128 x 16000 ent 19.1, 16.6, 16.0, top 30.4, 22.7, 17.9, tail 25.0, 19.7, 19.0;
// 760 x 50257 ent 15.4, 16.9, 23.0, top 24.3, 21.0, 26.9, tail 19.0, 18.9, 26.3; 400 x 152064 ent 30.7, 34.7, 54.1, top 29.5,
// 36.0, 59.7; 2128 x 152064 ent 99, 108, 108, top 115.8, 109.5, 109.6, tail 104, 117, 140. fp32 rows go by their vectors, as bf16 rows of
// twice their length.
int width_of(const LogitsArgs& a, int64_t vecs, int sms) {
  const bool list = a.ids != nullptr, top = !list && a.k > 0;
  int w = 256;
  if (a.M > 2 * sms) {
    if (vecs > 12288)
      w = top && a.M > 4 * sms ? 128 : 256;
    else if (top)
      w = a.M <= 4 * sms && vecs > 2560 ? 256 : a.M > 8 * sms && vecs <= 5120 ? 64 : 128;
    else
      w = a.M > 6 * sms && vecs <= 2560 ? 64 : list || vecs <= 5120 ? 128 : 256;
  }
  // a narrow CTA's list holds as many keys, its teacher as many entries, as it has threads
  const int least = top ? a.k + 32 : list ? a.k : 0;
  while (w < 256 && least > w) w *= 2;
  return w;
}

template <typename T>
nvfp4rl_status launch_type(const LogitsArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  // CTAs per row: two to an SM at most, and no share below a vector to a thread. 152064 columns, 5 alternatives: 64 rows with 8 CTAs
  // each 11.6 us, with 4 10.1, with 2 11.9; 152 rows with 2 15.9 us, with 1 20.0; 200 rows with 2 23.1 us, with 1 22.2.
  unsigned cluster = kMaxCluster;
  while (cluster > 1 && (a.M * cluster > 2 * dev.sm_count || a.V < static_cast<int64_t>(cluster) * kThreads * kVecOf<T>))
    cluster /= 2;
  switch (cluster > 1 ? 256 : width_of(a, a.V / kVecOf<T>, dev.sm_count)) {
    case 64: return launch_width<T, 64>(a, cluster, dev, st);
    case 128: return launch_width<T, 128>(a, cluster, dev, st);
    default: return launch_width<T, 256>(a, cluster, dev, st);
  }
}

}  // namespace

nvfp4rl_status launch_logprobs(const LogitsArgs& a, int dtype, const DeviceInfo& dev, cudaStream_t st) {
  return dtype == NVFP4RL_BF16 ? launch_type<uint16_t>(a, dev, st) : launch_type<float>(a, dev, st);
}

}  // namespace nvfp4rl
