// Decode attention over shared prefixes (sm_103a): every sequence of a group attends to its group's prefix cache and
// to its own cache, out = softmax(scale q K^T) V over both together.
//
// The group's (sequence, query head) rows of one KV head make the M of two matrix products with the prefix, so
// that each cached row is read, decoded and multiplied once for all of them: prefix_attention_kernel on the 5th-generation
// tensor cores. The own caches go through the decode kernel (attention.cu) as partial results, and
// kv_prefix_join_kernel joins a row's partials: (max, sum, O) each, as an online softmax does.
//
// prefix_attention_kernel: one persistent CTA per SM. A tile is up to 128 rows (whole sequences) of one group and KV head;
// the 128-token blocks of all tiles lie in one row, and each CTA takes an equal stretch of it, whatever the lengths,
// so that one long prefix keeps every SM busy. Up to eight KV heads are walked side by side, a CTA each over the same blocks:
// their rows of a token share the lines that DRAM gives (a head alone has 64 bytes of codes and 8 of scales there: it read
// 570 MB where 276 do). A
// stretch is one segment per tile; stretch c's segment in tile t leaves its partial in slot c + t of its head (both only grow
// along the stretch).
// Per block, in a pipeline of warps:
//   - four warps decode K and four V: one thread to a token row, 128 codes to f16 (exact: code x scale has at most
//     six significant bits), stored in the 128-byte swizzle of the MMA operands. Each warp copies its own 32 rows into a ring
//     of its own (cp.async, three blocks ahead; zeros behind the prefix's end, which makes those tokens' values zero),
//     four lanes to a row of 64 bytes. (With one warp's tensor copies of 64-byte rows a block took 2200 clocks.)
//   - one warp issues S = Q K^T (tcgen05, f16, 128 x 128 x 128) and one O += P V, V as it lies ([token][dim]: MN-major): one
//     warp for both spent as long on its waits as the tensor cores on the products;
//   - two groups of four warps take every second block each, so that one group's exponentials run under the other's and under
//     the products. A thread owns a row: the maximum of its 128 scores, then p = 2^(s - ref), P in f16 over S's own TMEM
//     columns. ref only moves when the maximum has grown by more than 2^8 (then O is scaled, once the products so far
//     are complete); a row's two threads hand it on from block to block. p is scaled by 2^6, so that f16 keeps 2^-30 of the
//     largest, and stays below 2^14.
//   TMEM: three S / P buffers and O, so that the scores of block n + 2 can follow the values of block n - 1 and are there
//   when the softmax of block n ends.
// A block takes 0.94 us (1800 clocks) in long stretches, 0.44 of the measured copy bandwidth, and a call 18 to 25 us beside its
// blocks (256 sequences behind sixteen prefixes, 154 us). What bounds it is the dependent chain scores - softmax - values with three
// blocks in flight: no unit is full. (Copies that left out work, of a build that read the heads one after another and took 125 us
// where this one takes 112: without the decoding 113, without exponentials and half of the maximum 116, with an eighth of the
// products 111 to 121, without the copies 118, without any of these 78.) Rows as M take 128 columns of TMEM to a score buffer and
// a whole tile's time whatever their number; rows as N would not, and is not built.
// Q enters as f16 scaled per row by a power of two that puts its largest element in [2^14, 2^15): exact down to 2^-31 of it. P is
// f16: results differ from those of an fp32 P by up to 8e-4 (relative), their distance from 64 bits stays that of
// the rounding to bf16, 1.7e-3.
#include <climits>
#include <map>
#include <mutex>

#include "common.cuh"
#include "logits.cuh"
#include "sm100.cuh"

namespace nvfp4rl {
namespace {

using namespace sm100;

constexpr int kDim = 128;
constexpr int kBlock = 128;  // tokens
constexpr int kRows = 128;   // rows of a tile
constexpr int kStages = 3;   // blocks of codes in a decoding warp's ring
constexpr int kWarpRows = 32, kCodeRow = kDim / 2, kScaleRow = kDim / 16;        // what a decoding warp copies
constexpr int kSlotBytes = kWarpRows * (kCodeRow + kScaleRow);                   // its code rows, then its scale rows
constexpr int kTileBytes = kBlock * kDim * 2;  // an f16 operand: two panels of 64 columns, 128 bytes to a row
constexpr int kPanel = kTileBytes / 2;
constexpr int kSmemBytes = kTileBytes /*Q*/ + 4 * kTileBytes /*K, V twice*/ + 8 * kStages * kSlotBytes + 1024 /*alignment*/;
// warps: 0-3 and 4-7 softmax (every second block each), 8-11 decode K, 12-15 decode V, 16 scores, 17 values, 18 segments, one
// idle that fills the warpgroup
constexpr int kScoreWarp = 16, kValueWarp = 17, kWalkWarp = 18, kThreads = 20 * 32;
// KV heads side by side: this many, or the largest power of two below that divides their number (256 sequences: 161 us,
// one head after the other 165).
constexpr int kBeside = 8;
constexpr int kSegments = 8, kSegmentReaders = 18;  // a ring of segments, read by warps 0-17
// Registers by warpgroup, out of the 96 that each of the 640 threads starts with.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 136, kDecodeRegs = 72, kOtherRegs = 64;
static_assert(2 * kSoftmaxRegs + 2 * kDecodeRegs + kOtherRegs <= 5 * kLaunchRegs, "within the launch's registers");
static_assert(kSoftmaxRegs >= kLaunchRegs && kDecodeRegs <= kLaunchRegs && kOtherRegs <= kLaunchRegs, "inc raises, dec lowers");
constexpr uint32_t kOcol = 384, kTmemCols = 512;  // S / P of blocks n % 3 from column 128 (n % 3) on, then O
constexpr float kSlack = 8.0f, kLift = 6.0f;                 // log2 units
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kSmemBytes <= 227 * 1024 - 2048, "fits one CTA's shared memory beside the static part");

struct Bars {
  uint64_t k_full[2], v_full[2];  // by n & 1, as the operands
  // by n % 3, as the S / P buffers. A barrier that two blocks' phases could pass before a waiter looks would be misread; here
  // block n + 3 needs the values of block n in O, and those the scores and P of block n.
  uint64_t s_done[3];   // the scores are there, and the K operand free
  uint64_t p_full[3];
  uint64_t pv_done[3];  // the block is in O, and its V operand and P free
  uint64_t ref_done[4][2];        // by quarter of the rows and n & 1: the rows' references of block n stand
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t q_full, stat_full, o_full, o_free, drain[2];
};

// A group of sequences as the tiles see it.
struct Group {
  int first, members;  // its sequences
  int tile0, tiles;    // the tiles before it, its own
  int unit0, units;    // the blocks of all tiles and head sets before it, its own
  int p, blocks;       // the prefix (-1: none) and its blocks
};

// Sizes that keep every count below 2^31: the host refuses larger ones.
struct Groups {
  const int32_t *offsets, *lens;
  int P, Lp, B, Hkv;
  int per_tile;   // sequences of a tile
  int max_tiles;  // P + B / per_tile
  int beside;     // KV heads that as many CTAs walk side by side, and the sets of that many
  int sets;
};

// The 32 groups from p0 on, one per lane, behind `tiles0` tiles and `units0` blocks, which move on. Whole warp. Offsets are
// clamped to the batch, lengths to the cache and tiles to their largest number, so that any contents give places inside
// the batch, the cache and the workspace.
__device__ __forceinline__ Group scan_groups(const Groups& a, int p0, int& tiles0, int& units0) {
  const int lane = threadIdx.x & 31;
  Group g{0, 0, 0, 0, 0, 0, p0 + lane, 0};
  if (g.p < a.P) {
    const int first = __ldg(a.offsets + g.p), end = __ldg(a.offsets + g.p + 1), len = __ldg(a.lens + g.p);
    g.first = min(max(first, 0), a.B);
    g.members = max(min(max(end, 0), a.B) - g.first, 0);
    g.blocks = (min(max(len, 0), a.Lp) + kBlock - 1) / kBlock;
    g.tiles = (g.members + a.per_tile - 1) / a.per_tile;
  }
  const auto sum_up_to = [&](int v) {  // with this lane's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  int upto = tiles0 + sum_up_to(g.tiles);
  g.tile0 = min(upto - g.tiles, a.max_tiles);
  g.tiles = min(upto, a.max_tiles) - g.tile0;
  tiles0 = __shfl_sync(0xFFFFFFFFu, upto, 31);
  g.units = g.tiles * g.blocks * a.sets;
  upto = units0 + sum_up_to(g.units);
  g.unit0 = upto - g.units;
  units0 = __shfl_sync(0xFFFFFFFFu, upto, 31);
  return g;
}

// The group of the first lane in `lanes`; p = -1 for none.
__device__ __forceinline__ Group pick_group(const Group& g, uint32_t lanes) {
  if (!lanes) return {0, 0, 0, 0, 0, 0, -1, 0};
  const int l = __ffs(lanes) - 1;
  Group r;
  r.first = __shfl_sync(0xFFFFFFFFu, g.first, l);
  r.members = __shfl_sync(0xFFFFFFFFu, g.members, l);
  r.tile0 = __shfl_sync(0xFFFFFFFFu, g.tile0, l);
  r.tiles = __shfl_sync(0xFFFFFFFFu, g.tiles, l);
  r.unit0 = __shfl_sync(0xFFFFFFFFu, g.unit0, l);
  r.units = __shfl_sync(0xFFFFFFFFu, g.units, l);
  r.p = __shfl_sync(0xFFFFFFFFu, g.p, l);
  r.blocks = __shfl_sync(0xFFFFFFFFu, g.blocks, l);
  return r;
}

// The first group for which f(group) holds, and the number of all blocks where it is wanted (else the search ends there).
template <class F>
__device__ __forceinline__ Group find_group(const Groups& a, int* total, F&& f) {
  int tiles0 = 0, units0 = 0;
  Group found{0, 0, 0, 0, 0, 0, -1, 0};
#pragma unroll 1
  for (int p0 = 0; p0 < a.P; p0 += 32) {
    const Group g = scan_groups(a, p0, tiles0, units0);
    if (found.p < 0) found = pick_group(g, __ballot_sync(0xFFFFFFFFu, g.p < a.P && f(g)));
    if (!total && found.p >= 0) break;
  }
  if (total) *total = units0;
  return found;
}

// How the blocks are shared out: the first `extra` CTAs take each + 1 of them, the others each.
struct Shares {
  int ctas, each, extra;
  __device__ __forceinline__ Shares(int total, int grid) {
    ctas = min(grid, max(total, 1));
    each = total / ctas;
    extra = total - each * ctas;
  }
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, extra); }
  __device__ __forceinline__ int owner(int u) const {
    const int head = extra * (each + 1);
    return u < head ? u / (each + 1) : extra + (u - head) / each;  // u < total, so each > 0 behind the head
  }
};

// A CTA's part of a tile.
struct Segment {
  int p, kvh, first_seq, members;  // members: the tile's sequences
  int slot, block0, blocks, len;   // blocks 0: there is no further segment
};

// Walks a CTA's stretch of blocks, segment by segment. One warp does it and hands the segments to the others through a ring
// in shared memory: the walk's state in the registers of every warp would spill.
struct Walk {
  Group g;        // the group of block u
  int u, end;     // blocks to come
  int tile, set;  // of u, within the group
  int block0;     // and its place in the tile: 0 but for the CTA's first
  __device__ __forceinline__ Segment next(const Groups& a) {
    Segment s{0, 0, 0, 0, 0, 0, 0, 0};
    if (u >= end) return s;
    if (u - g.unit0 >= g.units) {
      const int want = u;
      g = find_group(a, nullptr, [want](const Group& x) { return want >= x.unit0 && want - x.unit0 < x.units; });
      if (g.p < 0) return s;
      tile = set = 0;
    }
    s.p = g.p;
    const int which = static_cast<int>(blockIdx.x) % a.beside, cta = static_cast<int>(blockIdx.x) / a.beside;
    s.kvh = set * a.beside + which;
    s.first_seq = g.first + tile * a.per_tile;
    s.members = min(a.per_tile, g.members - tile * a.per_tile);
    s.slot = (cta + (g.tile0 + tile) * a.sets + set) * a.beside + which;
    s.block0 = block0;
    s.blocks = min(g.blocks - block0, end - u);
    s.len = min(max(__ldg(a.lens + g.p), 0), a.Lp);
    block0 = 0;
    u += s.blocks;
    if (++set == a.sets) {
      set = 0;
      ++tile;
    }
    return s;
  }
};

// The walk of the CTAs c (`beside` of them, a head of each set each) of `grid`. Whole warp.
__device__ __forceinline__ Walk begin_walk(const Groups& a, int grid, int c) {
  Walk w;
  int total = 0, tiles0 = 0;
  Group g = scan_groups(a, 0, tiles0, total);
#pragma unroll 1
  for (int p0 = 32; p0 < a.P; p0 += 32) scan_groups(a, p0, tiles0, total);
  const Shares shares(total, grid);
  w.u = w.end = 0;
  w.tile = w.set = w.block0 = 0;
  w.g = g;
  if (total == 0 || c >= shares.ctas) return w;
  const int begin = shares.begin(c);
  w.u = begin;
  w.end = shares.begin(c + 1);
  const auto here = [begin](const Group& x) { return begin >= x.unit0 && begin - x.unit0 < x.units; };
  w.g = pick_group(g, __ballot_sync(0xFFFFFFFFu, g.p < a.P && here(g)));
  if (w.g.p < 0) w.g = find_group(a, nullptr, here);  // behind the first 32 groups
  const int in = begin - w.g.unit0, row = in / w.g.blocks;
  w.block0 = in - row * w.g.blocks;
  w.tile = row / a.sets;
  w.set = row - w.tile * a.sets;
  return w;
}

// Partial results: O as [slot][kDim / 4][kRows] groups of four floats (32 rows write 512 bytes at once), maximum (log2 units)
// and sum as [slot][kRows].
__device__ __forceinline__ int64_t part_at(int64_t slot, int four, int row) { return (slot * (kDim / 4) + four) * kRows + row; }

struct PrefixArgs {
  const uint16_t* q;
  int64_t ldq;
  const uint8_t *kc, *ks, *vc, *vs;
  const float* gk;
  Groups groups;
  int heads;
  float scale;
  float4* part;
  float2* stats;
  uint32_t* status;
};

// Instruction descriptor, kind::f16: f16 A and B, fp32 D; transpose_b: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, bool transpose_b) {
  return (1u << 4) | (transpose_b ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The eight products of a block, K = 16 each, as one instruction sequence with two additions per product: the operands
// then stay warp-uniform, and the issuing warp keeps the tensor cores fed.
// D = A B^T, both in shared memory, K-major: 32 bytes further along the swizzled rows per product, the second panel after four.
__device__ __forceinline__ void mma8_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred f, t;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "add.u64 x, %1, 2;\n\tadd.u64 y, %2, 2;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 4;\n\tadd.u64 y, %2, 4;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, 6;\n\tadd.u64 y, %2, 6;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, %4;\n\tadd.u64 y, %2, %4;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, %5;\n\tadd.u64 y, %2, %5;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, %6;\n\tadd.u64 y, %2, %6;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u64 x, %1, %7;\n\tadd.u64 y, %2, %7;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(kPanel >> 4), "n"((kPanel >> 4) + 2), "n"((kPanel >> 4) + 4), "n"((kPanel >> 4) + 6)
      : "memory");
}
// D += A B, A in TMEM (8 columns per product), B MN-major in shared memory (16 rows of 128 bytes).
__device__ __forceinline__ void mma8_values(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 x, %1, 8;\n\tadd.u64 y, %2, 128;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.u32 x, %1, 16;\n\tadd.u64 y, %2, 256;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.u32 x, %1, 24;\n\tadd.u64 y, %2, 384;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.u32 x, %1, 32;\n\tadd.u64 y, %2, 512;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.u32 x, %1, 40;\n\tadd.u64 y, %2, 640;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.u32 x, %1, 48;\n\tadd.u64 y, %2, 768;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.u32 x, %1, 56;\n\tadd.u64 y, %2, 896;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 8 or 16 bytes, or as many zeros.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8u : 0u) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// 2^x (about 2 ulp; below 2^-126 zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Placed behind tmem_ld_wait: no use of these 32 loaded registers is moved ahead of it.
__device__ __forceinline__ void loaded32(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// Eight E2M1 codes times one scale pair (the same E4M3 value in both halves), exactly, to f16, stored at a.
__device__ __forceinline__ void decode8_store(uint32_t a, uint32_t w, uint32_t scale) {
  uint32_t d[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
      "mul.rn.f16x2 %0, %0, %5;\n\t"
      "mul.rn.f16x2 %1, %1, %5;\n\t"
      "mul.rn.f16x2 %2, %2, %5;\n\t"
      "mul.rn.f16x2 %3, %3, %5;\n\t}"
      : "=&r"(d[0]), "=&r"(d[1]), "=&r"(d[2]), "=&r"(d[3])
      : "r"(w), "r"(scale));
  sts128(a, d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

// The 16-byte unit u of a ring's code row i lies at code_unit: eight rows' units of one number are in eight different
// banks groups then, for the thread that reads a row and for the four that copy it.
__device__ __forceinline__ uint32_t code_unit(int i, int u) { return kCodeRow * i + ((u ^ ((i >> 1) & 3)) << 4); }

// One token row, row i of the warp's slot: 128 codes and 8 scale bytes to f16 in the operand row at `row`, in the 128-byte
// swizzle: 16-byte chunk c of a panel lies at chunk c ^ (row & 7), chunk[k] being the place of chunk k < 4 in bytes.
__device__ __forceinline__ void decode_row(uint32_t slot, uint32_t row, const uint32_t (&chunk)[4], int i) {
  const uint2 s = lds64(slot + kWarpRows * kCodeRow + kScaleRow * i);
  uint4 c[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) c[u] = lds128(slot + code_unit(i, u));
  uint32_t at[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) at[k] = row + (chunk[k & 3] ^ (16 * (k & 4)));
#pragma unroll
  for (int u = 0; u < 4; ++u) {  // 32 codes: two scale blocks
    const uint32_t two = e4m3x2_f16((u < 2 ? s.x : s.y) >> (16 * (u & 1)));
    const uint32_t s0 = __byte_perm(two, two, 0x1010), s1 = __byte_perm(two, two, 0x3232);
    const uint32_t* p = at + 4 * (u & 1);
    const uint32_t panel = (u >> 1) * kPanel;
    decode8_store(p[0] + panel, c[u].x, s0);
    decode8_store(p[1] + panel, c[u].y, s0);
    decode8_store(p[2] + panel, c[u].z, s1);
    decode8_store(p[3] + panel, c[u].w, s1);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prefix_attention_kernel(const PrefixArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ float row_scale[kRows], row_ref[kRows];
  __shared__ Segment segs[kSegments];
  __shared__ float2 stat[2][2][kRows];  // by the parity of the segment
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t qs = base, kvs = base + kTileBytes, ring = kvs + 4 * kTileBytes;  // K 0, K 1, V 0, V 1
  const auto bar = [&](uint64_t& b) { return smem_addr(&b); };
  if (warp == kScoreWarp) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.k_full[i]), 4);
      mbar_init(bar(bars.v_full[i]), 4);
      for (int q = 0; q < 4; ++q) mbar_init(bar(bars.ref_done[q][i]), 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(bars.s_done[i]), 1);
      mbar_init(bar(bars.p_full[i]), 4);
      mbar_init(bar(bars.pv_done[i]), 1);
    }
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(bar(bars.seg_full[i]), 1);
      mbar_init(bar(bars.seg_empty[i]), kSegmentReaders);
    }
    mbar_init(bar(bars.q_full), 4);
    mbar_init(bar(bars.stat_full), 8);
    mbar_init(bar(bars.o_full), 1);
    mbar_init(bar(bars.o_free), 8);
    mbar_init(bar(bars.drain[0]), 1);
    mbar_init(bar(bars.drain[1]), 1);
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  // a wait of the whole warp; false (for all lanes) when it ran out
  const auto wait = [&](uint64_t& b, uint32_t parity, uint32_t code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&b), parity, a.status, code));
  };
  // segment i of the CTA, and its slot's release by this warp
  const auto segment = [&](uint32_t i, uint32_t code) -> const Segment& {
    ok = ok && wait(bars.seg_full[i % kSegments], (i / kSegments) & 1, code);
    return segs[i % kSegments];
  };
  const auto release = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bars.seg_empty[i % kSegments]));
  };

  if (warp < 8) {
    // ---- softmax: one thread to a row, group x = warp / 4 takes every second block of the CTA
    more_registers<kSoftmaxRegs>();
    const int x = warp >> 2, r = threadIdx.x & (kRows - 1);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t ocol = tmem + lanes + kOcol;
    const float gk = __ldg(a.gk);
    const int member = r / a.heads, head = r - member * a.heads;
    uint32_t n0 = 0, n_q = 0;  // blocks before this segment; segments
    uint4 qv[16];              // the next segment's row of Q, loaded ahead of the last one's end
    const auto load_q = [&](const Segment& t) {
      const bool there = member < t.members;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (there ? (t.first_seq + member) * a.ldq + static_cast<int64_t>(t.kvh * a.heads + head) * kDim : 0));
#pragma unroll
      for (int i = 0; i < 16; ++i) qv[i] = __ldg(src + i);
    };
    if (x == 0) {
      const Segment& t = segment(0, kStatusTimeoutEpilogue);
      if (ok && t.blocks > 0) load_q(t);
    }
    while (true) {
      const Segment s = segment(n_q, kStatusTimeoutEpilogue);
      if (!ok || s.blocks == 0) break;
      release(n_q);
      const int rows = s.members * a.heads;
      if (x == 0) {  // Q: every earlier product with the old one is complete (stat_full)
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          top = __vmaxu2(__vmaxu2(__vmaxu2(top, qv[i].x & 0x7FFF7FFFu), qv[i].y & 0x7FFF7FFFu),
                         __vmaxu2(qv[i].z & 0x7FFF7FFFu, qv[i].w & 0x7FFF7FFFu));
        const int e = static_cast<int>(max(top & 0xFFFFu, top >> 16) >> 7);  // biased exponent of the largest
        const float up = __uint_as_float(static_cast<uint32_t>(min(max(268 - e, 1), 254)) << 23);
        // S is taken times |scale gk| below: the sign goes into Q. A row with a NaN or an infinity has no softmax: it is all
        // NaN, and so are its scores, its sum and its result. Rows that do not exist are 0 times the batch's first row, which
        // they load (0, or NaN: nothing of them is stored; loads of none instead took small calls 0.3 us).
        const float f = member >= s.members ? 0.0f : e == 255 ? NAN : (a.scale < 0.0f) != (gk < 0.0f) ? -up : up;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = pack_f16(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f);
          sts128(qs + (i >> 3) * kPanel + 128 * r + (((i & 7) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
        }
        // at least 2^-100: a masked score, -inf, stays that where the scale or gk is 0 (a NaN stays)
        const float to_log2 = fabsf(a.scale) * fabsf(gk) * kLog2e / up;
        row_scale[r] = to_log2 < 0x1p-100f ? 0x1p-100f : to_log2;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.q_full));
      }
      ok = wait(bars.q_full, n_q & 1, kStatusTimeoutEpilogue);
      if (!ok) break;
      const float sl2 = row_scale[r];
      const int tokens = s.len - s.block0 * kBlock;  // to the prefix's end
      const bool work = (warp & 3) * 32 < rows;  // a warp of rows that do not exist only keeps the pace
      const int j0 = (n0 & 1) == static_cast<uint32_t>(x) ? 0 : 1;
      float ref = -INFINITY;  // the reference of this thread's sum
      F2 sum = pack2(0.0f, 0.0f);
      for (int j = j0; j < s.blocks; j += 2) {
        const uint32_t n = n0 + j, third = n / 3, buf = n - 3 * third;
        const uint32_t scol = tmem + lanes + 128 * buf;
        ok = wait(bars.s_done[buf], third & 1, kStatusTimeoutEpilogue);
        if (!ok) break;
        tc_fence_after();
        if (work) {
          // Loops that stay loops: the code of the six kinds of warps has to stay in the instruction caches.
          const int valid = tokens - j * kBlock;  // tokens of this block
          if (valid < kBlock) {                   // the prefix's end: scores behind it become -inf
#pragma unroll 1
            for (int col = valid & ~15; col < kBlock; col += 16) {
              uint32_t u[16];
              tmem_ld16(scol + col, u);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (col + i >= valid) u[i] = 0xFF800000u;
              tmem_st16(scol + col, u);
            }
            tmem_st_wait();
          }
          uint32_t v[32], w[32];
          float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int col = 0; col < kBlock; col += 64) {
            tmem_ld32(scol + col, v);
            tmem_ld32(scol + col + 32, w);
            tmem_ld_wait();
            loaded32(v);
            loaded32(w);
#pragma unroll
            for (int i = 0; i < 32; ++i) m[i & 3] = max3(m[i & 3], __uint_as_float(v[i]), __uint_as_float(w[i]));
          }
          const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * sl2;
          // the reference: the last block's, or this one's maximum where that has grown past it
          float now = top;
          if (j > 0) {
            ok = wait(bars.ref_done[warp & 3][x ^ 1], ((n - 1) >> 1) & 1, kStatusTimeoutEpilogue);
            if (!ok) break;
            const float last = row_ref[r];
            const bool grew = top > last + kSlack;
            if (!grew) now = last;
            if (__any_sync(0xFFFFFFFFu, grew)) {
              // what is summed up so far moves to the new reference, with every product up to block n - 1 complete
              const uint32_t before = (n - 1) / 3;
              ok = wait(bars.pv_done[n - 1 - 3 * before], before & 1, kStatusTimeoutEpilogue);
              if (!ok) break;
              tc_fence_after();
              const float f = ex2(last - now);
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tmem_ld16(ocol + 16 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(ocol + 16 * c, o);
              }
            }
          }
          row_ref[r] = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bars.ref_done[warp & 3][x]));
          if (now != ref) {
            const float f = ex2(ref - now);
            sum = mul2(sum, pack2(f, f));
            ref = now;
          }
          const F2 scale2 = pack2(sl2, sl2), shift2 = pack2(kLift - ref, kLift - ref);
          const auto powers = [&](const uint32_t* u, int col) {  // p of 32 columns
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float e0, e1;
              unpack2(fma2(pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), scale2, shift2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum = add2(sum, pack2(e0, e1));
              p[i] = pack_f16(e0, e1);
            }
            tmem_st16(scol + col / 2, p);
          };
          // P of columns c .. c + 31 lies over scores from c / 2 on, which have been loaded by then
          tmem_ld32(scol, v);
#pragma unroll 1
          for (int col = 0; col < kBlock; col += 64) {
            tmem_ld_wait();
            loaded32(v);
            tmem_ld32(scol + col + 32, w);
            powers(v, col);
            tmem_ld_wait();
            loaded32(w);
            if (col == 0) tmem_ld32(scol + 64, v);
            powers(w, col + 32);
          }
          tmem_st_wait();
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bars.ref_done[warp & 3][x]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.p_full[buf]));
      }
      if (!ok) break;
      if (x == 0) {
        const Segment& t = segment(n_q + 1, kStatusTimeoutEpilogue);
        if (!ok) break;
        if (t.blocks > 0) load_q(t);
      }
      ok = wait(bars.o_full, n_q & 1, kStatusTimeoutEpilogue);
      if (!ok) break;
      tc_fence_after();
      float s0, s1;
      unpack2(sum, s0, s1);
      stat[n_q & 1][x][r] = make_float2(ref, s0 + s1);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.stat_full));
      ok = wait(bars.stat_full, n_q & 1, kStatusTimeoutEpilogue);
      if (!ok) break;
      // the row's sums of both groups, the later reference being O's; this thread writes 64 of its dims
      if (work) {
        const float2 t0 = stat[n_q & 1][0][r], t1 = stat[n_q & 1][1][r];
        const float M = fmaxf(t0.x, t1.x);  // -inf for a group without a block
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
          tmem_ld16(ocol + 64 * x + 16 * c, o);
          tmem_ld_wait();
          if (r < rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a.part[part_at(s.slot, 16 * x + 4 * c + i, r)] =
                  make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                              __uint_as_float(o[4 * i + 3]));
          }
        }
        if (x == 0 && r < rows)
          a.stats[static_cast<int64_t>(s.slot) * kRows + r] = make_float2(M - kLift, ex2(t0.x - M) * t0.y + ex2(t1.x - M) * t1.y);
      }
      n0 += s.blocks;
      ++n_q;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.o_free));
    }
  } else if (warp < kScoreWarp) {
    // ---- decoding: warps 8-11 K, 12-15 V; one thread to a token
    fewer_registers<kDecodeRegs>();
    const bool is_v = warp >= 12;
    const int r = threadIdx.x & (kBlock - 1);
    uint64_t* full = is_v ? bars.v_full : bars.k_full;
    const uint8_t* codes = is_v ? a.vc : a.kc;
    const uint8_t* scales = is_v ? a.vs : a.ks;
    const uint32_t slots = ring + (warp - 8) * (kStages * kSlotBytes), out = kvs + (is_v ? 2 * kTileBytes : 0) + 128 * r;
    uint32_t chunk[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) chunk[k] = (k ^ (r & 7)) << 4;
    const int row0 = r & ~31;  // of the warp's rows in a block
    // The copies run three blocks ahead of the decoding: `left` blocks of segment seg - 1 are still to come, `tokens` tokens from
    // the warp's first row of the next one on, which the lane's pointers are at. A group of copies is closed per block
    // whether there is one or not.
    const int64_t code_step = static_cast<int64_t>(a.groups.Hkv) * kCodeRow;
    const int64_t scale_step = static_cast<int64_t>(a.groups.Hkv) * kScaleRow;
    const uint8_t *from = codes, *scale_from = scales;
    uint32_t seg = 0, copied = 0;
    int left = 0, tokens = 0;
    bool more = true;
    const auto copy_next = [&]() {
      if (more && left == 0) {
        const Segment& s = segment(seg, kStatusTimeoutDequant);
        left = s.blocks;
        more = ok && left > 0;
        if (more) {
          const int t0 = s.block0 * kBlock + row0;
          const int64_t at = (static_cast<int64_t>(s.p) * a.groups.Lp + t0) * a.groups.Hkv + s.kvh;
          tokens = s.len - t0;
          from = codes + at * kCodeRow + (lane >> 2) * code_step + 16 * (lane & 3);
          scale_from = scales + at * kScaleRow + lane * scale_step;
          release(seg);
        }
        ++seg;
      }
      if (more) {
        const uint32_t slot = slots + (copied % kStages) * kSlotBytes;
        const uint32_t to = slot + code_unit(lane >> 2, lane & 3), scale_to = slot + kWarpRows * kCodeRow + kScaleRow * lane;
        if (tokens >= kWarpRows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async16(to + 8 * kCodeRow * i, from + 8 * i * code_step, true);
          cp_async8(scale_to, scale_from, true);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool there = 8 * i + (lane >> 2) < tokens;
            cp_async16(to + 8 * kCodeRow * i, there ? from + 8 * i * code_step : codes, there);
          }
          cp_async8(scale_to, lane < tokens ? scale_from : scales, lane < tokens);
        }
        from += kBlock * code_step;
        scale_from += kBlock * scale_step;
        tokens -= kBlock;
        --left;
        ++copied;
      }
      cp_async_commit();
    };
    for (int i = 0; i < kStages; ++i) copy_next();
    for (uint32_t n = 0; ok && n < copied; ++n) {
      const uint32_t buf = n & 1;
      cp_async_wait<kStages - 1>();
      __syncwarp();
      if (n >= 2) {  // the operand's last product, of block n - 2, is complete
        const uint32_t third = (n - 2) / 3;
        ok = wait((is_v ? bars.pv_done : bars.s_done)[n - 2 - 3 * third], third & 1, kStatusTimeoutDequant);
        if (!ok) break;
      }
      decode_row(slots + (n % kStages) * kSlotBytes, out + buf * kTileBytes, chunk, lane);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(full[buf]));
      copy_next();
    }
    cp_async_wait<0>();  // every copy has landed before the CTA leaves
  } else {
    fewer_registers<kOtherRegs>();
    // what the issuing warps make of a value that is the same in every lane: the shuffle tells the compiler, which then
    // keeps the products' operands in uniform registers
    const auto uniform = [](uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
    // the products in flight of an issuing warp end before shared memory and TMEM go
    const auto drain = [&](uint64_t& b) {
      if (elect_one()) mma_commit(bar(b));
      __syncwarp();
      mbar_wait(bar(b), 0, a.status, kStatusTimeoutDrain);
    };
    if (warp == kScoreWarp) {
      // ---- S = Q K^T, issued by one elected lane of the converged warp
      constexpr uint32_t idesc = idesc_f16_f32(kRows, kBlock, false);
      const uint64_t qdesc = smem_desc(qs, 16, 1024, 2);
      const uint32_t tmem_u = uniform(tmem);
      uint32_t n = 0;
      for (uint32_t i = 0; ok; ++i) {
        const int blocks = segment(i, kStatusTimeoutMma).blocks;
        if (!ok || blocks == 0) break;
        release(i);
        ok = wait(bars.q_full, i & 1, kStatusTimeoutMma);
        for (int j = 0; j < blocks && ok; ++j, ++n) {
          const uint32_t x = uniform(n & 1), third = n / 3, buf = uniform(n - 3 * third);
          ok = wait(bars.k_full[x], (n >> 1) & 1, kStatusTimeoutMma);
          // the buffer is free: the values of block n - 3 are in O
          if (ok && n >= 3) ok = wait(bars.pv_done[buf], (third & 1) ^ 1, kStatusTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma8_scores(tmem_u + 128 * buf, qdesc, smem_desc(kvs + x * kTileBytes, 16, 1024, 2), idesc);
            mma_commit(bar(bars.s_done[buf]));
          }
          __syncwarp();
        }
      }
      if (!ok) drain(bars.drain[0]);
    } else if (warp == kValueWarp) {
      // ---- O += P V
      constexpr uint32_t idesc = idesc_f16_f32(kRows, kDim, true);
      const uint32_t tmem_u = uniform(tmem);
      uint32_t n = 0;
      for (uint32_t i = 0; ok; ++i) {
        const int blocks = segment(i, kStatusTimeoutMma).blocks;
        if (!ok || blocks == 0) break;
        release(i);
        for (int j = 0; j < blocks && ok; ++j, ++n) {
          const uint32_t x = uniform(n & 1), third = n / 3, buf = uniform(n - 3 * third);
          ok = wait(bars.v_full[x], (n >> 1) & 1, kStatusTimeoutMma) && wait(bars.p_full[buf], third & 1, kStatusTimeoutMma);
          // the first products into O: the last segment's has been read
          if (ok && j == 0 && i > 0) ok = wait(bars.o_free, (i - 1) & 1, kStatusTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            // V is [token][dim]: the contiguous dims are N (two panels), eight tokens to 1024 bytes
            mma8_values(tmem_u + kOcol, tmem_u + 128 * buf, smem_desc(kvs + (2 + x) * kTileBytes, kPanel, 1024, 2), idesc,
                        j > 0 ? 1u : 0u);
            mma_commit(bar(bars.pv_done[buf]));
            if (j == blocks - 1) mma_commit(bar(bars.o_full));
          }
          __syncwarp();
        }
      }
      if (!ok) drain(bars.drain[1]);
    } else if (warp == kWalkWarp) {
      // ---- segments
      Walk walk = begin_walk(a.groups, gridDim.x / a.groups.beside, blockIdx.x / a.groups.beside);
      for (uint32_t i = 0; ok; ++i) {
        const Segment s = walk.next(a.groups);
        ok = wait(bars.seg_empty[i % kSegments], ((i / kSegments) & 1) ^ 1, kStatusTimeoutProducer);
        if (!ok) break;
        if (lane == 0) {
          segs[i % kSegments] = s;
          mbar_arrive(bar(bars.seg_full[i % kSegments]));
        }
        __syncwarp();
        if (s.blocks == 0) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial results of every (sequence, query head); one warp per row, four dims per lane. A row that attends to
// nothing is 0.
struct JoinArgs {
  const float4* part;
  const float2* stats;
  int grid;  // stretches of the prefix kernel
  Groups groups;
  OwnPartials own;
  const int32_t* lens;
  int64_t Lmax;
  int Hq, heads;
  const float* gv;
  uint16_t* out;
};

// A warp per row; kAhead partials in flight. Sixteen where the rows are no more than the warps that then fit the GPU (1792 rows of
// up to 17 partials: the whole call 42 us, by fours 47), four where more rows at a time do better (10240 of about 5:
// 165 us, by sixteens 173).
constexpr int kJoinFew = 16;  // warps per SM
template <int kAhead>
__global__ void __launch_bounds__(128) kv_prefix_join_kernel(const JoinArgs a) {
  // Ahead of the wait for the partials: the offsets and lengths, which were complete before the prefix kernel's CTAs let any
  // kernel behind it start.
  const int fours = (a.Hq + 3) / 4;  // CTAs of a sequence: one per four heads
  const int b = blockIdx.x / fours, h = (blockIdx.x - b * fours) * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (h >= a.Hq) return;
  // the row's partials: slots s0 .. of the prefix kernel, then the spans of its own cache
  const int own_len = a.own.part ? __ldg(a.lens + b) : 0;
  int total;
  const Group g = find_group(a.groups, &total, [b](const Group& x) { return b >= x.first && b - x.first < x.members; });
  const int kvh = h / a.heads, r = h - kvh * a.heads;
  int64_t s0 = 0;
  int tile_row = 0, npre = 0, nown = 0;
  if (g.p >= 0) {
    const int tile = (b - g.first) / a.groups.per_tile, set = kvh / a.groups.beside;
    if (g.blocks > 0 && tile < g.tiles) {
      const int u0 = g.unit0 + (tile * a.groups.sets + set) * g.blocks;
      const Shares shares(total, a.grid);
      const int c0 = shares.owner(u0);
      tile_row = (b - g.first - tile * a.groups.per_tile) * a.heads + r;
      s0 = (c0 + (g.tile0 + tile) * a.groups.sets + set) * a.groups.beside + kvh % a.groups.beside;
      npre = shares.owner(u0 + g.blocks - 1) - c0 + 1;
    }
  }
  const float* own = nullptr;
  if (a.own.part) {
    nown = static_cast<int>(a.own.spans(min(max(static_cast<int64_t>(own_len), int64_t(0)), a.Lmax)));
    own = a.own.part + ((static_cast<int64_t>(b) * a.groups.Hkv + kvh) * a.own.nsplit * kOwnRows + r) * kOwnFloats;
  }
  griddep_wait();
  griddep_launch_dependents();
  const int n = npre + nown;
  const auto own_at = [&](int i) { return own + static_cast<int64_t>(i - npre) * kOwnRows * kOwnFloats; };
  float M = -INFINITY, L = 0.0f, O[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i0 = 0; i0 < n; i0 += 32) {  // a lane to a partial's statistics
    const int i = i0 + lane, count = min(32, n - i0);
    float2 t = make_float2(-INFINITY, 0.0f);
    if (i < npre) t = a.stats[(s0 + i * a.groups.beside) * kRows + tile_row];
    else if (i < n) t = make_float2(own_at(i)[0], own_at(i)[1]);
    const float m = fmaxf(M, warp_max(t.x));
    // an empty partial is (-inf, 0); a maximum passes over NaN, so that one of a row of NaN is (-inf, NaN)
    if (m == -INFINITY && !__any_sync(0xFFFFFFFFu, t.y != 0.0f)) continue;
    const float keep = ex2(M - m), f = ex2(t.x - m);
    L = L * keep + warp_sum(f * t.y);
#pragma unroll
    for (int q = 0; q < 4; ++q) O[q] *= keep;
    M = m;
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int at = i0 + k0 + k;
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // the four rows of a CTA's warps share their sectors in L1
        if (k0 + k < count)
          v[k] = at < npre ? a.part[part_at(s0 + at * a.groups.beside, lane, tile_row)]
                           : reinterpret_cast<const float4*>(own_at(at) + 4)[lane];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, (k0 + k) & 31);  // past the end: times zeros
        O[0] = fmaf(w, v[k].x, O[0]);
        O[1] = fmaf(w, v[k].y, O[1]);
        O[2] = fmaf(w, v[k].z, O[2]);
        O[3] = fmaf(w, v[k].w, O[3]);
      }
    }
  }
  const float inv = L == 0.0f ? 0.0f : __ldg(a.gv) / L;  // a NaN stays
  reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(b) * a.Hq + h) * kDim)[lane] =
      make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
}

// Tiles of all groups, at most, and partial results of the prefix kernel: at most one per CTA more than tiles times heads.
int64_t most_tiles(int64_t B, int64_t heads, int64_t P) { return P + B / (kRows / heads); }
int64_t prefix_slots(int64_t B, int64_t Hkv, int64_t heads, int64_t P) { return kPlanSMs + most_tiles(B, heads, P) * Hkv; }
size_t prefix_bytes(int64_t slots) { return static_cast<size_t>(slots) * kRows * (kDim * sizeof(float) + sizeof(float2)); }

}  // namespace

size_t prefix_attention_workspace_bytes(int64_t B, int64_t Hkv, int64_t Lmax, int64_t heads, int64_t P) {
  return prefix_bytes(prefix_slots(B, Hkv, heads, P)) + own_partials_bytes(B, Hkv, Lmax);
}

// The kernels count (tile, head, block) triples in 32 bits.
bool prefix_attention_fits(int64_t B, int64_t Hkv, int64_t heads, int64_t P, int64_t Lp) {
  return (Lp + kBlock - 1) / kBlock <= INT32_MAX / (most_tiles(B, heads, P) * Hkv);
}

nvfp4rl_status launch_prefix_attention(const PrefixAttnArgs& p, const DeviceInfo& dev, cudaStream_t st) {
  const int heads = static_cast<int>(p.Hq / p.Hkv);
  const int64_t tiles = most_tiles(p.B, heads, p.P), slots = prefix_slots(p.B, p.Hkv, heads, p.P);
  auto* part = static_cast<float4*>(p.workspace);
  auto* stats = reinterpret_cast<float2*>(part + slots * kRows * (kDim / 4));
  auto* own = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + prefix_bytes(slots));
  int beside = kBeside;
  while (p.Hkv % beside != 0) beside /= 2;
  const Groups groups{p.groups, p.prefix_lens, static_cast<int>(p.P), static_cast<int>(p.Lp), static_cast<int>(p.B),
                      static_cast<int>(p.Hkv), kRows / heads, static_cast<int>(tiles), beside, static_cast<int>(p.Hkv) / beside};
  {
    static std::mutex mu;
    static std::map<int, bool> set;
    std::lock_guard<std::mutex> lock(mu);
    bool& done = set[dev.device];
    if (!done) {
      if (cudaFuncSetAttribute(prefix_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
        return NVFP4RL_ERR_CUDA;
      done = true;
    }
  }
  // no more CTAs than blocks there can be, so that few leave SMs to the kernel behind
  const int64_t units = tiles * groups.sets * ((p.Lp + kBlock - 1) / kBlock);
  const int most = std::min(dev.sm_count, kPlanSMs) / beside;
  const int stretches = static_cast<int>(std::min<int64_t>(std::max<int64_t>(units, 1), most));
  const PrefixArgs a{p.q, p.ldq, p.pkc, p.pks, p.pvc, p.pvs, p.gk, groups, heads, p.scale, part, stats, dev.status};
  if (launch_pdl(prefix_attention_kernel, dim3(static_cast<unsigned>(stretches * beside)), dim3(kThreads), kSmemBytes, st, a) !=
      cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  nvfp4rl_status s = launch_status();
  if (s != NVFP4RL_OK) return s;
  OwnPartials partials{nullptr, 0};
  if (p.Lmax > 0) {
    s = launch_own_partials(p, own, &partials, dev, st);
    if (s != NVFP4RL_OK) return s;
  }
  const JoinArgs j{part, stats, stretches, groups, partials, p.lens, p.Lmax, static_cast<int>(p.Hq), heads, p.gv, p.out};
  const bool few = p.B * p.Hq <= static_cast<int64_t>(kJoinFew) * dev.sm_count;
  const auto join = few ? kv_prefix_join_kernel<16> : kv_prefix_join_kernel<4>;
  if (launch_pdl(join, dim3(static_cast<unsigned>(p.B * ((p.Hq + 3) / 4))), dim3(128), 0, st, j) != cudaSuccess)
    return NVFP4RL_ERR_CUDA;
  return launch_status();
}

}  // namespace nvfp4rl
