// tree_attention.cu -- attention of several new tokens per sequence (a drafted
// tree or chain) over the paged key-value cache and over one another.
//
//   s_tj = scale * q_t . k_j over the cache's rows j < len and over the new
//   tokens j that t sees (a mask, or j <= t);
//   out_t = sum_j exp(s_tj - lse_t) v_j,   lse_t = log sum_j exp(s_tj)
//
// Bound: bytes of the cache while rows are few, the two products (4 * head_dim
// operations per row and key) when they are many.  The new tokens of a sequence
// and the G query heads of a key-value head are rows of one matrix (row =
// token * G + head), so that a key read once meets all of them: at a few tokens
// they fill the 128 rows of a tcgen05 tile.
//
// The work is cut by cost: all (sequence, key-value head, 256 rows, key tile)
// units in order form one line, with the cost of a segment's start and end, that
// the CTAs, one per SM, share out evenly.  It is computed on the device from the
// lengths and offsets.  A CTA whose stretch begins or ends inside a segment
// leaves its partial (m, l, o) in the workspace, and a second small kernel joins
// the partials in CTA order.
//
//   warps 0-3, 4-7  softmax of tile 0, tile 1: a thread owns a row, reads its
//                   128 scores from tensor memory, keeps the reference m and
//                   the sum l in registers and writes the weights back as bf16
//                   over the scores; then the tile's outputs
//   4 or 8 more     loads: q and k, v tiles through a ring.  Pages may be of any
//                   size, so rows are gathered with cp.async; bytes of an E4M3
//                   cache pass through a ring of their own and are widened on
//                   the way (exact), keys to bf16 as the queries are, values to
//                   fp16, which takes a fifth of the instructions
//   two more        issue S_i = Q_i K^T and O_i += P_i V of tile 0, tile 1
//   one more        finds the CTA's next items
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (head_dim each).
// Of more than 128 rows the two tiles are rows 0-127 and 128-255 and go through
// all keys.  Up to 128 rows both are the same rows and take every other key
// tile; their outputs are added at the end.  Either way one tile's products run
// while the other's softmax is computed.
//
// Roundings: scores, m, l, O are fp32; the weights 2^(s - m) are rounded to bf16
// for the product with v, l sums the unrounded ones.  With an E4M3 cache the
// weights of its rows are rounded to fp16 instead.  They are taken 2^7 times as
// large there: m lies at most 2^8 below the maximum, so they reach 2^15 of fp16's
// 2^16, and one is lost to the product only below 2^-32 of the largest (without the
// factor below 2^-25, and 130000 of those are a third of a percent of the sum, which
// keeps them).  O is in units of the head's value scale while its tiles are of the
// cache, and takes the scale before the first tile of new tokens, whose values are
// bf16 (or at the end): a scale may be of any size and sign, or 0.
//
// A masked weight is 0, but 0 * NaN is NaN: rows past a length read as zeros, and
// the values of new tokens that some row of the item does not see are looked
// through before the product; elements that are not finite are replaced by 0 there
// and added back in the end to the rows that do see them.
//
// Measured: 48 sequences to 8192 rows, 25 nodes, 40/8 heads of 128: 99 us = 0.76 of
// the copy rate (a segment's start and end cost two to three tiles); 64 x 6000
// rows E4M3, 61 nodes, 28/4 heads: 394 us where the products take 179 (215 with the
// rows that fill 512): a tile's chain, 2700 cycles of softmax, then the second
// half of its values' product and the next scores, 1700, beside the widening
// (issue 53%, tensor pipe 38%); 96 sequences to 2500 rows, 30 nodes, 32/8 heads of
// 64: 74 us where the bytes take 28 (five to nine segments a CTA, each 11000 cycles
// for three tiles: a chain of latencies); a chain of 5 over 777 rows 12.6 us, of
// which a call without work takes 10.2.  Long chains: 512 new tokens over 8192
// rows, 4 sequences, 28/4 heads 214 us = 0.62 of the bf16 rate (E4M3 rows 249 us, 32/8
// heads of 64 over E4M3 rows 242 us = 0.31), 131072 tokens of one
// head 3.23 ms = 0.73.  What made it so: instruction fetches bound the first forms
// (1.9 warps of a scheduler waited for one), so that code is small and in loops:
// E4M3 829 us with every kind of load inlined where it is used, 753 us in one
// place each, 713 us without a polling wait, 507 us with the widening as a loop;
// bf16 108 to 101 us with the softmax as loops.  Loads that announce themselves
// (130 to 109 us), four warps each for keys and values of an E4M3 cache (510 to
// 428 us) and products of the parts of a tile that hold keys (79 to 77 us) came on
// top; then values as fp16, whole tiles 64 keys at a time and one place for each
// product in the issuers (422 to 398 us; long chains 257 to 219 us).
#include "attention.cuh"
#include "qerl_internal.h"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace qerl {
namespace {

constexpr int kRows = 128;   // rows of a query tile, keys of a key tile
constexpr int kBlock = 256;  // rows of a segment
constexpr float kSlack = 8.0f;
// Base-2 factor of all weights, and so of l and O: of the partials too.
template <bool kFp8>
constexpr float kAbove = kFp8 ? 7.0f : 0.0f;
constexpr int kMaxCtas = 160;
constexpr int kSegmentCost = 2;  // of a segment's start and end, in key tiles
constexpr int kMaxTokens = 1 << 20;  // of a sequence

struct TreeParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const uint8_t *kp, *vp;
  const float *k_scale, *v_scale;
  const int* table;
  int64_t ld_table, num_pages;
  int page_size, page_shift;  // shift < 0: not a power of two
  int64_t capacity;           // max_pages * page_size
  const int *cu, *lengths;
  const unsigned long long* mask;  // null: j <= t
  int words;
  int num_seqs, tokens, heads, kv_heads, group;
  unsigned group_inverse;  // ceil(2^32 / group), 0 for a group of 1
  float scale_log2;
  __nv_bfloat16* out;
  int64_t ldo;
  float* lse;
  int4* jobs;   // [CTA]: (sequence, key-value head, first row, partials) of the segment begun in its stretch; 0: whole
  float* part;  // [CTA][2]: of the segment begun before its stretch, of the one begun in it; see slot_floats
  int slot_rows;
  int* status;
};

// A partial: o as [head_dim / 4][slot_rows] of 4 floats, then m and l.
__host__ __device__ __forceinline__ int64_t slot_floats(int slot_rows, int head_dim) {
  return static_cast<int64_t>(slot_rows) * (head_dim + 2);
}

template <int D, bool kFp8>
struct Shape {
  // Four warps bring the keys and then the values of a tile; of an E4M3 cache,
  // which takes them longer, four the keys and four the values.
  static constexpr int kLoadWarps = kFp8 ? 8 : 4;
  static constexpr int kThreads = 384 + 32 * kLoadWarps;
  // At launch 512 threads have 128 registers each, 640 have 96:
  // 256 * 184 + 128 * 88 + 128 * 56 = 512 * 128, 256 * 136 + 256 * 72 + 128 * 64 = 640 * 96.
  // (A share above the launch's goes by setmaxnreg.inc, one below by .dec, and their
  // sum stays within the launch's: anything else faults or waits forever.)
  static constexpr int kSoftmaxRegs = kFp8 ? 136 : 184, kLoadRegs = kFp8 ? 72 : 88, kOtherRegs = kFp8 ? 64 : 56;
  static_assert(kSoftmaxRegs * 256 + kLoadRegs * 32 * kLoadWarps + kOtherRegs * 128 <= kThreads * (kFp8 ? 96 : 128) &&
                    kSoftmaxRegs >= (kFp8 ? 96 : 128) && kLoadRegs <= (kFp8 ? 96 : 128) && kOtherRegs <= (kFp8 ? 96 : 128),
                "shares of the launch's registers");
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kTile = kPanels * kPanel;
  // Slots of the keys' and of the values' ring.
  static constexpr unsigned kKeySlots = kFp8 ? 2 * (128 / D) : D == 128 ? 2 : 5;
  static constexpr unsigned kValueSlots = kFp8 ? 2 * (128 / D) : D == 128 ? 3 : 5;
  static constexpr unsigned kSlots = kKeySlots + kValueSlots;
  // Slots and phases of a tile's loads repeat after so many tiles.
  static constexpr unsigned kLaps = 2 * kKeySlots * kValueSlots;
  static constexpr unsigned kRaw = kFp8 ? 2 : 0;  // tiles as they lie in the cache: keys, values
  static constexpr uint32_t kRawTile = kRows * D;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kRawRing = kRing + kSlots * kTile;
  // (m, l) of shared rows, 1 KB a query tile, behind the outputs in the second buffer of the queries if they fit.
  static constexpr uint32_t kMl = kTile >= 18432 ? kTile + 16384 : kRawRing + kRaw * kRawTile;
  static constexpr uint32_t kBars = kRawRing + kRaw * kRawTile + (kTile >= 18432 ? 0 : 2048);
  static constexpr uint32_t kSmem = 1024 + kBars + 768;
};

// Four E4M3 bytes -> four bf16 (exact): the exponent and mantissa as bf16's,
// which is 2^-120 of the value (subnormals too), times 2^120.  NaN's bits give
// +-480 here; the caller looks for them.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);  // each byte atop 16 bits
  const uint32_t x = (a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), y = (b & 0x80008000u) | ((b >> 4) & 0x07F007F0u);
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x7B807B80u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x7B807B80u));
}
// The barrier takes this thread's arrival when its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// NaN where a byte of w is E4M3's NaN.
__device__ __forceinline__ void nan_bytes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if ((w & 0x7Fu) == 0x7Fu) lo = (lo & 0xFFFF0000u) | 0x7FFFu;
  if ((w & 0x7F00u) == 0x7F00u) lo = (lo & 0x0000FFFFu) | 0x7FFF0000u;
  if ((w & 0x7F0000u) == 0x7F0000u) hi = (hi & 0xFFFF0000u) | 0x7FFFu;
  if ((w & 0x7F000000u) == 0x7F000000u) hi = (hi & 0x0000FFFFu) | 0x7FFF0000u;
}

// mbar_wait_a in fewer instructions: this kernel waits in some thirty places, and
// what runs once an item is fetched cold.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const long long t0 = clock64();
  while (!mbar_try_wait_hint_a(bar, parity, QERL_WAIT_HINT_NS)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > QERL_WAIT_LIMIT) {
      *abort_flag = 1;
      record_error(status, QERL_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The warp that finds the items is up to two ahead, and an item may last as long
// as the cache is long: it waits until another role gives up (or some 2000 s).
__device__ __forceinline__ bool wait_patiently(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  for (int i = 0; i < (1 << 27); ++i) {
    if (mbar_try_wait_hint_a(bar, parity, QERL_WAIT_HINT_NS)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  record_error(status, QERL_ERR_TIMEOUT);
  return false;
}

// Units of the outputs over an E4M3 cache once they have the value scale: large beside
// a large one, whose product with sums of some 2^41 would overflow.
__device__ __forceinline__ float value_unit(float scale) { return fabsf(scale) > 0x1p40f ? 0x1p64f : 1.0f; }

// A sequence's place on the line.
struct Sequence {
  int start, n, len;  // its first new token, their count, its rows in the cache
  int blocks, ctx, tiles;  // segments per key-value head; key tiles of the cache, of all keys
  // Key tiles of a segment.  In order, a block sees the new tokens up to its last row's.
  __device__ __forceinline__ int needed(const TreeParams& p, int block) const {
    if (p.mask != nullptr || block + 1 >= blocks) return tiles;
    return ctx + (block * kBlock + kBlock - 1) / p.group / kRows + 1;
  }
  // Cost of the segments of a key-value head's first `count` blocks.  In order,
  // block i sees floor((2 i + 1) / group) + 1 tiles of new tokens; with i = a * group + b
  // the quotient is 2 a, one more from b = group / 2 on.
  __device__ __forceinline__ long long before(const TreeParams& p, int count) const {
    if (p.mask != nullptr || count == 0) return static_cast<long long>(count) * (tiles + kSegmentCost);
    const long long inner = min(count, blocks - 1);
    const int a = static_cast<int>(inner) / p.group, b = static_cast<int>(inner) - a * p.group, z = p.group >> 1;
    const long long quotients =
        static_cast<long long>(a) * (a - 1) * p.group + static_cast<long long>(a) * (p.group - z + 2 * b) + max(b - z, 0);
    return inner * (ctx + 1 + kSegmentCost) + quotients + (count == blocks ? tiles + kSegmentCost : 0);
  }
  __device__ __forceinline__ long long cost(const TreeParams& p) const {
    return n > 0 ? p.kv_heads * before(p, blocks) : 0;
  }
};
// false: its offsets break the rules.
__device__ __forceinline__ bool sequence(const TreeParams& p, int s, Sequence& q) {
  q.start = p.cu[s];
  const int end = p.cu[s + 1], len = p.lengths[s];
  if (q.start < 0 || end < q.start || end > p.tokens || end - q.start > kMaxTokens) return false;
  q.n = end - q.start;
  q.len = len < 0 ? 0 : len > p.capacity ? static_cast<int>(p.capacity) : len;
  q.blocks = (q.n * p.group + kBlock - 1) / kBlock;
  q.ctx = q.len == 0 ? 0 : (q.len - 1) / kRows + 1;
  q.tiles = q.ctx + (q.n + kRows - 1) / kRows;
  return true;
}

// A piece of a segment: key tiles [t0, t1).  Its rows begin at row0 = token0 * group + head0.
struct Item {
  int start, n, len, seq, kv_head, row0, t0, t1, slot, token0, head0;  // slot -1: the whole segment
};
// Token and head (within the group) of row row0 + x of the sequence's, x < 256.
// The product with the rounded inverse is exact for numerators below 2^32 / 1024.
__device__ __forceinline__ int token_of(const TreeParams& p, const Item& it, int x, int& head) {
  const unsigned n = it.head0 + x;
  const int q = p.group_inverse == 0 ? n : __umulhi(n, p.group_inverse);
  head = n - q * p.group;
  return it.token0 + q;
}
constexpr int kItemInts = 12;

template <int D, bool kFp8>
__global__ void __launch_bounds__((Shape<D, kFp8>::kThreads), 1) tree_kernel(const __grid_constant__ TreeParams p) {
  using S = Shape<D, kFp8>;
  constexpr int kThreads = S::kThreads, kLoadWarps = S::kLoadWarps;
  constexpr int kIssuer = 8 + kLoadWarps, kFinder = kIssuer + 2;  // warps
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (sbase - raw);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // uniform to the compiler too
  const float kInf = __int_as_float(0x7f800000);

  const uint32_t bars = sbase + S::kBars;
  auto full = [&](unsigned s) { return bars + 8u * s; };
  auto empty = [&](unsigned s) { return bars + 8u * (S::kSlots + s); };
  const uint32_t misc = bars + 16u * S::kSlots;
  auto s_full = [&](int i) { return misc + 8u * i; };
  auto p_full = [&](int i, int part) { return misc + 8u * (2 + 2 * i + part); };
  auto o_full = [&](int i) { return misc + 8u * (6 + i); };
  auto turn = [&](int i) { return misc + 8u * (8 + i); };
  const uint32_t q_full = misc + 8u * 10;
  const uint32_t q_free = misc + 8u * 11;    // the last scores are computed
  auto out_free = [&](int e) { return misc + 8u * (12 + e); };  // the outputs of an even, odd item have left
  auto ml_full = [&](int i) { return misc + 8u * (14 + i); };
  auto ml_empty = [&](int i) { return misc + 8u * (16 + i); };
  auto item_full = [&](int e) { return misc + 8u * (18 + e); };
  auto item_empty = [&](int e) { return misc + 8u * (20 + e); };
  const uint32_t done = misc + 8u * 22;
  const uint32_t tmem_holder = misc + 8u * 23;
  uint8_t* misc_gen = gen + S::kBars + 16 * S::kSlots;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc_gen + 8 * 23 + 4);
  volatile int* dirty = reinterpret_cast<volatile int*>(misc_gen + 8 * 24);       // [4]: item k's at k & 3 is k + 1
  volatile int* items = reinterpret_cast<volatile int*>(misc_gen + 8 * 26);       // [2][kItemInts]
  volatile long long* sums = reinterpret_cast<volatile long long*>(misc_gen + 8 * 38);  // [20], then the place found
  volatile int* place = reinterpret_cast<volatile int*>(misc_gen + 8 * 58);       // sequence, bad offsets
  volatile long long* inside_seq = reinterpret_cast<volatile long long*>(misc_gen + 8 * 59);
  volatile unsigned* begun = reinterpret_cast<volatile unsigned*>(misc_gen + 8 * 60);
  // Tile n's keys (part 0) and values (part 1): slot and phase of the barriers.
  auto slot_of = [&](int part, unsigned n) { return part == 0 ? n % S::kKeySlots : S::kKeySlots + n % S::kValueSlots; };
  auto phase_of = [&](int part, unsigned n) { return (part == 0 ? n / S::kKeySlots : n / S::kValueSlots) & 1; };
  auto slot_at = [&](int part, unsigned n) { return sbase + S::kRing + slot_of(part, n) * S::kTile; };
  // Waits for a load of tile n, the `count`-th of all (modulo 2^32).  A barrier's
  // phase is only told from the one before, and where the tiles take turns an
  // issuer does not look at every load: so first that the slot was given to this
  // load, then that it is there.
  auto wait_load = [&](int part, unsigned n, unsigned count) -> bool {
    if (static_cast<int>(begun[part] - count) <= 0) {
      const long long t0 = clock64();
      while (static_cast<int>(begun[part] - count) <= 0) {
        __nanosleep(40);  // (a warp that polls takes issue slots and instruction fetches from the loads)
        if (*abort_flag) return false;
        if (clock64() - t0 > QERL_WAIT_LIMIT) {
          *abort_flag = 1;
          record_error(p.status, QERL_ERR_TIMEOUT);
          return false;
        }
      }
    }
    return wait_for(full(slot_of(part, n)), phase_of(part, n), abort_flag, p.status);
  };

  if (threadIdx.x == 0) {
    for (unsigned s = 0; s < S::kSlots; ++s) {
      mbar_init_a(full(s), 128);
      mbar_init_a(empty(s), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_a(s_full(i), 1);
#ifdef QERL_TEST_HOOKS
      mbar_init_a(p_full(i, 0), 4 + (g_test_extra_arrival ? 1 : 0));
#else
      mbar_init_a(p_full(i, 0), 4);
#endif
      mbar_init_a(p_full(i, 1), 4);
      mbar_init_a(o_full(i), 1);
      mbar_init_a(turn(i), 1);
      mbar_init_a(ml_full(i), 4);
      mbar_init_a(ml_empty(i), 4);
      mbar_init_a(item_full(i), 1);
      mbar_init_a(item_empty(i), 10 + kLoadWarps);  // 8 softmax warps, the loads and 2 issuers
    }
    mbar_init_a(q_full, 128);
    mbar_init_a(q_free, 2);
    mbar_init_a(out_free(0), 8);
    mbar_init_a(out_free(1), 8);
    begun[0] = begun[1] = 0;
    mbar_init_a(done, 2);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) dirty[i] = 0;
    place[1] = 0;
    fence_mbarrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *reinterpret_cast<volatile uint32_t*>(misc_gen + 8 * 23), 0);

  griddep_wait();

  // ---- this CTA's stretch of the line ---------------------------------------
  constexpr int kWarps = kThreads / 32;
  auto scan = [&](long long v) -> long long {  // inclusive over the block
#pragma unroll 1
    for (int i = 1; i < 32; i <<= 1) {
      const long long up = __shfl_up_sync(~0u, v, i);
      if (lane >= i) v += up;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    long long w = lane < kWarps ? sums[lane] : 0;
#pragma unroll 1
    for (int i = 1; i < kWarps; i <<= 1) {
      const long long up = __shfl_up_sync(~0u, w, i);
      if (lane >= i) w += up;
    }
    const long long before = __shfl_sync(~0u, w, warp > 0 ? warp - 1 : 0);
    return warp > 0 ? v + before : v;
  };
  auto total_of = [&]() -> long long {  // of the last scan
    long long w = lane < kWarps ? sums[lane] : 0;
#pragma unroll 1
    for (int i = 16; i > 0; i >>= 1) w += __shfl_xor_sync(~0u, w, i);
    return w;
  };
  Sequence sq;
  long long total = 0, begin = 0, end = 0, each = 0, extra = 0, inside = 0;
  int seq = 0;
  bool busy = false;
  auto stretch = [&](long long c) -> long long { return each * c + (c < extra ? c : extra); };
  // Even stretches; a tile belongs to the stretch in which its place lies.
  auto divide = [&]() {
    const long long ctas = total < gridDim.x ? total : gridDim.x;
    each = ctas > 0 ? quotient(total, ctas) : 0;
    extra = total - each * ctas;  // the first `extra` are one longer
    busy = blockIdx.x < ctas;
    begin = stretch(blockIdx.x);
    end = stretch(blockIdx.x + 1);
  };
  // One sequence that breaks the rules leaves nothing to do: the offsets around
  // it may lie before those of other sequences, and two CTAs would then write
  // the same rows.
  auto cost_of = [&](int b, bool& bad) -> long long {
    const bool fine = sequence(p, b, sq);
    const int len = p.lengths[b];
    if (!fine || len < 0 || len > p.capacity || (p.mask != nullptr && sq.n > static_cast<int64_t>(p.words) * 64))
      record_error(p.status, QERL_ERR_RANGE);
    bad |= !fine;
    return fine ? sq.cost(p) : 0;
  };
  if (p.num_seqs <= 32) {  // the warp that finds the items alone, without a barrier
    if (warp == kFinder) {
      bool bad = false;
      const long long mine = lane < p.num_seqs ? cost_of(lane, bad) : 0;
      long long incl = mine;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const long long up = __shfl_up_sync(~0u, incl, i);
        if (lane >= i) incl += up;
      }
      total = __any_sync(~0u, bad) ? 0 : __shfl_sync(~0u, incl, 31);
      divide();
      const unsigned hit = __ballot_sync(~0u, incl - mine <= begin && begin < incl);
      seq = hit != 0 ? __ffs(hit) - 1 : 0;
      inside = begin - __shfl_sync(~0u, incl - mine, seq);
      int* const fields = reinterpret_cast<int*>(&sq);  // that lane's, to all
#pragma unroll
      for (int f = 0; f < static_cast<int>(sizeof(Sequence) / sizeof(int)); ++f) fields[f] = __shfl_sync(~0u, fields[f], seq);
    }
  } else {
    bool bad = false;
    long long mine = 0, first_cost = 0;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.num_seqs; b += kThreads) {
      const long long c = cost_of(b, bad);
      if (b == threadIdx.x) first_cost = c;
      mine += c;
    }
    if (bad) place[1] = 1;
    long long incl = scan(mine);
    total = place[1] ? 0 : total_of();
    divide();
    if (p.num_seqs <= kThreads) {
      if (busy && incl - mine <= begin && begin < incl) {
        place[0] = threadIdx.x;
        *inside_seq = begin - (incl - mine);
      }
    } else if (busy) {
      long long base = 0;
      for (int b0 = 0;; b0 += kThreads) {  // ends: begin < total, the sum of all
        const int b = b0 + threadIdx.x;
        mine = b0 == 0 ? first_cost : b < p.num_seqs && sequence(p, b, sq) ? sq.cost(p) : 0;
        incl = scan(mine) + base;
        const long long next = base + total_of();
        if (begin < next) {
          if (incl - mine <= begin && begin < incl) {
            place[0] = b;
            *inside_seq = begin - (incl - mine);
          }
          break;
        }
        base = next;
      }
    }
    __syncthreads();
    seq = place[0];
    inside = *inside_seq;
    if (warp == kFinder && busy) sequence(p, seq, sq);
  }
  // The kernel that joins partials may be set up; it begins when this one has ended.
  griddep_launch_dependents();

  struct Work {
    Item it;
    bool shared;  // the two query tiles are the same rows and take every other key tile
    int ctx;
    // key tiles of query tile i, and the j-th of them
    __device__ __forceinline__ int count(int i) const {
      const int n = it.t1 - it.t0;
      return shared ? (n + 1 - i) >> 1 : n;
    }
    __device__ __forceinline__ int tile(int i, int j) const { return it.t0 + (shared ? 2 * j + i : j); }
    // 32-key parts of key tile t that hold keys: the products and the softmax leave out the rest.
    __device__ __forceinline__ int parts(int t) const {
      const int keys = t < ctx ? it.len - t * kRows : it.n - (t - ctx) * kRows;
      return keys >= kRows ? 4 : (keys + 31) >> 5;
    }
  };
  auto take = [&](int k, Work& w) -> bool {
    const int e = k & 1;
    // (a warp goes on or gives up as a whole, here and at every wait of a whole warp)
    if (!__all_sync(~0u, wait_for(item_full(e), (k >> 1) & 1, abort_flag, p.status))) return false;
    const volatile int* it = items + e * kItemInts;
    w.it = {it[0], it[1], it[2], it[3], it[4], it[5], it[6], it[7], it[8], it[9], it[10]};
    w.shared = w.it.n * p.group - w.it.row0 <= kRows;
    w.ctx = w.it.len == 0 ? 0 : (w.it.len - 1) / kRows + 1;
    __syncwarp();
    if (lane == 0) mbar_arrive_a(item_empty(e));
    return w.it.n > 0;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
    const int i = warp >> 2;               // query tile
    const int r = (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + i * 128, o_t = tmem + lanes + 256 + i * D, o_other = tmem + lanes + 256 + (1 - i) * D;
    bool ok = true;
    // Tiles of this query tile; all tiles before this item, for their slots and
    // phases (they may pass 2^32, which is no multiple of the laps) and modulo 2^32.
    unsigned tiles_done = 0, n0 = 0, count0 = 0;
    int outputs_done = 0, exchanges = 0;
    Work w;
    for (int k = 0; ok && take(k, w); ++k) {
      const int mine_n = w.count(i);
      const int row = w.it.row0 + (w.shared ? 0 : i * kRows) + r;  // of the sequence's rows
      const int rows = w.it.n * p.group;
      int row_head;
      const int row_token = token_of(p, w.it, row - w.it.row0, row_head);
      const int token = row < rows ? row_token : 0;
      // The reference in base-2 units and as a score (of the cache's tiles or of the
      // new tokens', whose units may differ), and the sum of 2^(s - m).  The
      // reference is taken from the scores before their product with c: a fused
      // product would leave the rounding of a large m in the exponent, which
      // overflows from scores of 2^31 on.
      float mc = -kInf, ref = -kInf, l = 0.0f;
      bool ref_fresh = false;
      float unit = 1.0f, v_scale = 1.0f, c_ctx = fabsf(p.scale_log2);  // v_scale in units of `unit`
      if (kFp8) {
        if (p.k_scale != nullptr) c_ctx = fabsf(p.scale_log2 * p.k_scale[w.it.kv_head]);
        if (p.v_scale != nullptr) v_scale = p.v_scale[w.it.kv_head];
        unit = value_unit(v_scale);
        v_scale /= unit;
      }
      // Not 0: a masked score of -inf times 0 would be NaN (1e-37 times any score below 1e29 is as good as 0).
      // A key scale of NaN stays.
      if (c_ctx < 1e-37f) c_ctx = 1e-37f;
      const float c_new = fmaxf(fabsf(p.scale_log2), 1e-37f);
      // Bits of the keys 32 q .. 32 q + 31 of key tile t that this row attends to, for
      // its weights and for what is added back in the end; a mask's words are looked up
      // together, for their latencies.
      auto sees = [&](int t, uint32_t (&keep)[4]) {
        auto below = [](int n) -> uint32_t { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };
        const bool fresh = t >= w.ctx;
        unsigned long long word[2] = {~0ull, ~0ull};
        int limit = fresh ? w.it.n - (t - w.ctx) * kRows : w.it.len - t * kRows;  // keys of the tile
        if (fresh && p.mask != nullptr) {
          const int at = 2 * (t - w.ctx);
          const unsigned long long* src = p.mask + (static_cast<int64_t>(w.it.start) + token) * p.words + at;
          word[0] = at < p.words ? src[0] : 0;
          word[1] = at + 1 < p.words ? src[1] : 0;
        } else if (fresh) {
          limit = min(limit, token + 1 - (t - w.ctx) * kRows);
        }
        if (fresh && row >= rows) limit = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) keep[q] = static_cast<uint32_t>(word[q >> 1] >> (32 * (q & 1))) & below(limit - q * 32);
      };
      // The first tile of new tokens of which this item's rows may not see all.
      const int first_hidden = w.ctx + (p.mask == nullptr ? (w.it.token0 + 1) / kRows : 0);
      // The mask's words are on their way to the L1 cache during the tiles before.
      if (p.mask != nullptr && row < rows)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.mask + (static_cast<int64_t>(w.it.start) + token) * p.words));
      // The values of a tile of new tokens, looked through
      // for elements that are not finite; a thread takes one token's row.
      auto clean_values = [&](int t) -> bool {  // of the item's t-th tile
        if (!__all_sync(~0u, wait_load(1, n0 + t, count0 + t))) return false;
        const uint32_t at_row = slot_at(1, n0 + t) + r * 128;
        // x * 0 + sum is NaN from the first x that is not finite
        uint32_t sum = 0;
#pragma unroll
        for (int q = 0; q < S::kPanels * 8; ++q) {
          const uint4 a = lds128(at_row + (q >> 3) * kPanel + (((q & 7) ^ (r & 7)) << 4));
          sum = times0_plus(a.x, sum);
          sum = times0_plus(a.y, sum);
          sum = times0_plus(a.z, sum);
          sum = times0_plus(a.w, sum);
        }
        if ((sum & 0x7FFF7FFFu) != 0) {
          dirty[k & 3] = k + 1;
#pragma unroll 1
          for (int q = 0; q < S::kPanels * 8; ++q) {
            const uint32_t at = at_row + (q >> 3) * kPanel + (((q & 7) ^ (r & 7)) << 4);
            const uint4 x = lds128(at);
            uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((a[e] & 0x7F800000u) == 0x7F800000u) a[e] &= 0x0000FFFFu;
              if ((a[e] & 0x7F80u) == 0x7F80u) a[e] &= 0xFFFF0000u;
            }
            sts128(at, make_uint4(a[0], a[1], a[2], a[3]));
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        return true;
      };
      // One key tile: scores in, weights out, l and (rarely) the reference moved.
      // Both passes are loops over 32 keys, which read the scores twice: code
      // that runs through once a tile is fetched as slowly as it runs.
      // Whole tiles have code of their own (kWhole) where they go on for long, of an
      // E4M3 cache, or of a bf16 cache where the products hold the kernel (more than
      // 128 rows): 64 keys at a time, the last 64 of the first pass still in
      // registers for the second (4 x 512 tokens over 8192 rows, 28/4 heads: 250 us,
      // in common code 257; for 128 rows and few tiles a segment the second code
      // costs more fetches than it saves: 96 sequences with heads of 64 90 against 76).
      // All 128 scores in registers: 2% faster there, 8% slower in the others.
      constexpr int kAny = 0, kPartial = 1, kWhole = 2;
      auto step = [&](auto kind, int j, int parts, bool hides, bool fresh, const uint32_t (&keep)[4]) {
        constexpr int kKind = decltype(kind)::value;
        const bool masked = kKind == kPartial || (kKind == kAny && hides);
        auto load = [&](int q, float (&x)[32]) {
          tmem_ld32(s_t + q * 32, x);
          tmem_ld_wait();
          pin<32>(x);
          if (masked) {
            const uint32_t bits = q < 2 ? (q == 0 ? keep[0] : keep[1]) : (q == 2 ? keep[2] : keep[3]);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((bits & (1u << e)) == 0) x[e] = -kInf;
          }
        };
        float top = -kInf;
        auto largest = [&](const float* x) {
          float t2[2] = {top, x[0]};
#pragma unroll
          for (int e = 1; e < 29; e += 4) {
            t2[0] = max3(t2[0], x[e], x[e + 1]);
            t2[1] = max3(t2[1], x[e + 2], x[e + 3]);
          }
          t2[0] = max3(t2[0], x[29], x[30]);
          top = max3(t2[0], t2[1], x[31]);
        };
        float x64[64];  // of a whole tile, a half
        if (kKind == kWhole) {
#pragma unroll 1
          for (int half = 1; half >= 0; --half) {
            tmem_ld32(s_t + half * 64, x64);
            tmem_ld32(s_t + half * 64 + 32, x64 + 32);
            tmem_ld_wait();
            pin<64>(x64);
            largest(x64);
            largest(x64 + 32);
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < parts; ++q) {
            float x[32];
            load(q, x);
            largest(x);
          }
        }
        const float c = kFp8 && !fresh ? c_ctx : c_new;
        bool scales = false;
        if (kFp8 && fresh != ref_fresh) {
          ref = mc == -kInf ? -kInf : mc / c;
          ref_fresh = fresh;
          scales = v_scale != 1.0f;
        }
        // A row moves its own reference only: what its neighbours in the warp see rounds none of its weights.
        const bool moves = (top - ref) * c > kSlack;
        if (__any_sync(~0u, moves) || scales) {
          if (j > 0) {
            float f = moves ? ex2((ref - top) * c) : 1.0f;
            l *= f;
            if (kFp8 && scales) f *= v_scale;
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              float v[16];
              tmem_ld16(o_t + q * 16, v);
              tmem_ld_wait();
              pin<16>(v);
              uint32_t y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(v[e] * f);
              tmem_st_x16(o_t + q * 16, y);
            }
          }
          if (moves) {
            ref = top;
            mc = top * c;
          }
        }
        uint64_t part[2] = {0, 0};  // two chains of two fp32 sums
        const float sub = ref == -kInf ? 0.0f : ref;
        const uint64_t c2 = pair(c, c), sub2 = pair(-sub, -sub);
        const float raise = kAbove<kFp8> - (kFp8 && fresh && unit != 1.0f ? 64.0f : 0.0f);
        const uint64_t raise2 = pair(raise, raise);
        auto weigh = [&](const float* x, int q) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, b;
            unpair(fma2(add2(pair(x[2 * e], x[2 * e + 1]), sub2), c2, raise2), a, b);
            a = ex2(a);
            b = ex2(b);
            part[e & 1] = add2(part[e & 1], pair(a, b));
            // weights of an E4M3 cache's rows: fp16, as those rows are
            y[e] = kFp8 && (kKind == kWhole || !fresh) ? pack_f16(a, b) : pack_bf16(a, b);
          }
          tmem_st_x16(s_t + q * 16, y);
        };
        auto announce = [&](bool half, bool all) {  // half of the keys, or all: the product with v may begin
          if (half || all) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && half) mbar_arrive_a(p_full(i, 0));
            if (lane == 0 && all) mbar_arrive_a(p_full(i, 1));
          }
        };
        if (kKind == kWhole) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            if (half == 1) {
              tmem_ld32(s_t + 64, x64);
              tmem_ld32(s_t + 96, x64 + 32);
              tmem_ld_wait();
              pin<64>(x64);
            }
            weigh(x64, 2 * half);
            weigh(x64 + 32, 2 * half + 1);
            announce(half == 0, half == 1);
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < parts; ++q) {
            float x[32];
            load(q, x);
            weigh(x, q);
            announce(q == 1 || (q == 0 && parts == 1), q + 1 == parts);
          }
        }
        float s0, s1;
        unpair(add2(part[0], part[1]), s0, s1);
        l += kFp8 && fresh ? (s0 + s1) * unit : s0 + s1;
      };

      for (int j = 0; j < mine_n; ++j) {
        const int t = w.tile(i, j);
        const bool fresh = t >= w.ctx, masked = fresh ? t >= first_hidden : w.it.len - t * kRows < kRows;
        uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked) sees(t, keep);  // (while the scores are computed)
        ok = __all_sync(~0u, wait_for(s_full(i), (tiles_done + j) & 1, abort_flag, p.status));
        if (ok && fresh && masked) ok = clean_values(t - w.it.t0);
        if (!ok) break;
        tc_fence_after();
        if (masked || (kFp8 ? fresh : w.shared))
          step(std::integral_constant<int, kFp8 ? kPartial : kAny>{}, j, w.parts(t), kFp8 || masked, fresh, keep);
        else
          step(std::integral_constant<int, kWhole>{}, j, 4, false, !kFp8 && fresh, keep);
      }
      tiles_done += mine_n;
      n0 = (n0 + w.it.t1 - w.it.t0) % S::kLaps;
      count0 += w.it.t1 - w.it.t0;
      if (mine_n > 0) {
        ok = __all_sync(~0u, ok && wait_for(o_full(i), outputs_done & 1, abort_flag, p.status));
        ++outputs_done;
      }
      if (!ok) break;
      tc_fence_after();
      // (a tile's last keys tell whether its outputs have the value scale)
      float f_own = kFp8 && !ref_fresh ? v_scale : 1.0f, f_other = 0.0f;
      const bool both = w.shared && w.count(1) > 0;
      if (both) {
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sbase + S::kMl + i * 1024 + r * 8), "f"(mc), "f"(l) : "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_a(ml_full(i));
        ok = __all_sync(~0u, wait_for(ml_full(1 - i), exchanges & 1, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        float m2, l2;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(m2), "=f"(l2)
                     : "r"(sbase + S::kMl + (1 - i) * 1024 + r * 8)
                     : "memory");
        const float top = fmaxf(mc, m2);
        const float w_own = weight_of(mc, top);
        f_other = weight_of(m2, top);
        // the same sum in the same order on both sides
        l = i == 0 ? w_own * l + f_other * l2 : f_other * l2 + w_own * l;
        mc = top;
        f_own *= w_own;
        if (kFp8 && w.tile(1 - i, w.count(1 - i) - 1) < w.ctx) f_other *= v_scale;
      }
      const bool live = row < rows;
      const bool fix = __any_sync(~0u, dirty[k & 3] == k + 1);
      const float f = l == 0.0f ? 0.0f : unit / l;
      const bool whole = w.it.slot < 0;
      float* slot = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (whole ? 0 : w.it.slot)) * slot_floats(p.slot_rows, D);
      const int slot_row = row - w.it.row0;
      // Shared rows: each tile's warps take half of the columns, tile 0's all of them if tile 1 had no keys.
      const int c0 = both && i == 1 ? D / 2 : 0, c1 = both ? c0 + D / 2 : w.shared && i == 1 ? 0 : D;
      // Outputs pass through the tile's own queries, or through the buffer that shared rows leave free.
      const uint32_t stage = sbase + (w.shared ? S::kTile + i * 8192 : i * S::kTile) + (warp & 3) * 2048;
      const int head0 = w.it.kv_head * p.group;
#pragma unroll 1
      for (int col = c0; col < c1; col += 32) {
        float v[32];
        tmem_ld32(o_t + col, v);
        if (both) {
          float y[32];
          tmem_ld32(o_other + col, y);
          tmem_ld_wait();
          pin<32>(v);
          pin<32>(y);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            v[e] = i == 0 ? f_own * v[e] + f_other * y[e] : f_other * y[e] + f_own * v[e];
        } else {
          tmem_ld_wait();
          pin<32>(v);
          if (kFp8) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= f_own;
          }
        }
        if (fix) {
          // A lane looks through one of 32 tokens, then the warp goes through those with something to add back.
#pragma unroll 1
          for (int t = max(w.it.t0, first_hidden); t < w.it.t1; ++t) {
            uint32_t bits[4];
            sees(t, bits);
#pragma unroll 1
            for (int q = 0; q < 4 && (t - w.ctx) * kRows + q * 32 < w.it.n; ++q) {
              const uint32_t keep = q < 2 ? (q == 0 ? bits[0] : bits[1]) : (q == 2 ? bits[2] : bits[3]);
              const int node = (t - w.ctx) * kRows + q * 32;
              const __nv_bfloat16* src = p.v + (static_cast<int64_t>(w.it.start) + node) * p.ldv + w.it.kv_head * D + col;
              uint32_t sum = 0;
              if (node + lane < w.it.n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint4 a = *reinterpret_cast<const uint4*>(src + lane * p.ldv + e * 8);
                  sum = times0_plus(a.x, sum);
                  sum = times0_plus(a.y, sum);
                  sum = times0_plus(a.z, sum);
                  sum = times0_plus(a.w, sum);
                }
              }
              uint32_t found = __ballot_sync(~0u, (sum & 0x7FFF7FFFu) != 0) & __reduce_or_sync(~0u, keep);
              while (found != 0) {
                const int x = __ffs(found) - 1;
                found &= found - 1;
                const float mine = __bfloat162float(src[x * p.ldv + lane]);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float y = __shfl_sync(~0u, mine, e);
                  if ((keep >> x & 1) != 0 && !(fabsf(y) < kInf)) v[e] += y;
                }
              }
            }
          }
        }
        if (whole) {
          // Through shared memory, so that a store covers 64 bytes of a row.
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sts128(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4),
                   make_uint4(pack_bf16(v[8 * e] * f, v[8 * e + 1] * f), pack_bf16(v[8 * e + 2] * f, v[8 * e + 3] * f),
                              pack_bf16(v[8 * e + 4] * f, v[8 * e + 5] * f),
                              pack_bf16(v[8 * e + 6] * f, v[8 * e + 7] * f)));
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at = q * 8 + (lane >> 2), ch = lane & 3;
            const uint4 y = lds128(stage + at * 64 + ((ch ^ ((at >> 1) & 3)) << 4));
            const int g = row - lane + at;
            int hd;
            const int tk = token_of(p, w.it, g - w.it.row0, hd);
            if (g < rows)
              *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(w.it.start) + tk) * p.ldo +
                                        static_cast<int64_t>(head0 + hd) * D + col + ch * 8) = y;
          }
          __syncwarp();
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            __stcg(reinterpret_cast<float4*>(slot) + static_cast<int64_t>(col / 4 + e) * p.slot_rows + slot_row,
                   make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
        }
      }
      if (live && c0 == 0 && c1 > 0) {
        if (!whole) {
          __stcg(slot + static_cast<int64_t>(D) * p.slot_rows + slot_row, mc);
          __stcg(slot + static_cast<int64_t>(D + 1) * p.slot_rows + slot_row, l);
        } else if (p.lse != nullptr) {
          p.lse[(static_cast<int64_t>(w.it.start) + token) * p.heads + head0 + row_head] =
              l == 0.0f ? -kInf : (mc + (log2f(l) - kAbove<kFp8>)) * 0.69314718055994530942f;
        }
      }
      if (both) {  // the other tile's warps still read this tile's outputs and (m, l)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_a(ml_empty(i));
        ok = __all_sync(~0u, wait_for(ml_empty(1 - i), exchanges & 1, abort_flag, p.status));
        ++exchanges;
        if (!ok) break;
        tc_fence_after();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_a(out_free(k & 1));
    }
  } else if (warp < kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kLoadRegs));
    // Four warps bring 32 rows each of a tile; a barrier takes an arrival of every
    // thread, which comes by itself when the thread's copies have landed.
    const int lw = (warp - 8) & 3, group = (warp - 8) >> 2;  // E4M3: group 0 the keys and the queries, 1 the values
    unsigned n = 0;      // the next tile, but for laps dropped
    unsigned count = 0;  // the same of all tiles (modulo 2^32)
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(~0u, wait_for(bar, parity, abort_flag, p.status));
    };
    auto passed = [&](uint32_t bar, uint32_t parity) -> bool { return __all_sync(~0u, mbar_test_wait_a(bar, parity)); };
    auto next_slot = [&](int part) -> bool {  // waits for the slot of tile n's load
      if (n >= (part == 0 ? S::kKeySlots : S::kValueSlots) && !wait(empty(slot_of(part, n)), phase_of(part, n) ^ 1))
        return false;
      if (lw == 0 && lane == 0) begun[part] = count + 1;
      return true;
    };
    // 16-byte chunks of this warp's rows of a tile of bf16 rows (lane x's row at src; null: zeros).
    auto copy_rows = [&](uint32_t tile_at, const void* src) {
      constexpr int kChunks = D / 8;
      const int ch = lane % kChunks;
      const uint32_t to = tile_at + (ch >> 3) * kPanel;
#pragma unroll 4
      for (int q = 0; q < kChunks; ++q) {
        const int at = (q * 32 + lane) / kChunks, row = lw * 32 + at;
        const uint8_t* from =
            reinterpret_cast<const uint8_t*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(src), at));
        const bool real = from != nullptr;
        cp_async_16(to + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                    real ? from + ch * 16 : reinterpret_cast<const uint8_t*>(p.q), real ? 16 : 0);
      }
    };
    // The same of E4M3 rows, as they are, to this group's part of the raw ring;
    // every thread reads back what it wrote.
    constexpr int kRawChunks = D / 16;
    auto raw_at = [&](int q) { return sbase + S::kRawRing + group * S::kRawTile + ((q * 4 + lw) * 32 + lane) * 16; };
    auto copy_raw = [&](int q, const void* src) {
      const uint8_t* from = reinterpret_cast<const uint8_t*>(
          __shfl_sync(~0u, reinterpret_cast<unsigned long long>(src), (q * 32 + lane) / kRawChunks));
      const bool real = from != nullptr;
      cp_async_16(raw_at(q), real ? from + lane % kRawChunks * 16 : reinterpret_cast<const uint8_t*>(p.q), real ? 16 : 0);
    };
    // The raw tile, which has landed, into its slot, and the next one in its place.
    auto widen = [&](const void* next, bool more) {
      // A chunk becomes two, of which a lane of the second panel writes the later
      // one first: the eight lanes of a row then fall into eight bank groups.
      const int ch = 2 * (lane % kRawChunks);
      const bool swap = (ch >> 3) != 0;
      const uint32_t to = slot_at(group, n) + (ch >> 3) * kPanel;
      constexpr int kTogether = 2;  // chunks at a time, for their latencies; a loop, as its code would not stay in the cache
#pragma unroll 1
      for (int q0 = 0; q0 < kRawChunks; q0 += kTogether) {
        uint32_t x[kTogether][4];
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
          const uint4 v = lds128(raw_at(q0 + q));
          x[q][0] = swap ? v.z : v.x;
          x[q][1] = swap ? v.w : v.y;
          x[q][2] = swap ? v.x : v.z;
          x[q][3] = swap ? v.y : v.w;
        }
        uint32_t y[kTogether][8];
        if (group == 1) {
#pragma unroll
          for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16(x[q][e], y[q][2 * e], y[q][2 * e + 1]);
        } else {
          uint32_t nan = 0;
#pragma unroll
          for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) nan |= (x[q][e] & 0x7F7F7F7Fu) + 0x01010101u;
          const bool some = (nan & 0x80808080u) != 0;
#pragma unroll
          for (int q = 0; q < kTogether; ++q) {
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_bf16(x[q][e], y[q][2 * e], y[q][2 * e + 1]);
            if (some) {
#pragma unroll
              for (int e = 0; e < 4; ++e) nan_bytes_to_bf16(x[q][e], y[q][2 * e], y[q][2 * e + 1]);
            }
          }
        }
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
          const int row = lw * 32 + ((q0 + q) * 32 + lane) / kRawChunks;
          const uint32_t first = to + row * 128 + ((((ch & 7) + (swap ? 1 : 0)) ^ (row & 7)) << 4);
          sts128(first, make_uint4(y[q][0], y[q][1], y[q][2], y[q][3]));
          sts128(first ^ 16, make_uint4(y[q][4], y[q][5], y[q][6], y[q][7]));
        }
        if (more) {
#pragma unroll
          for (int q = 0; q < kTogether; ++q) copy_raw(q0 + q, next);
        }
      }
      mbar_arrive_a(full(slot_of(group, n)));
    };
    // Only slots, phases and whether the first lap is over are used of n.
    auto drop_laps = [&]() {
      if (n >= 2 * S::kLaps) n -= (n / S::kLaps - 1) * S::kLaps;
    };
    bool shared_before = false, more = true;
    Work w;
    for (int k = 0; ok && more; ++k) {
      more = take(k, w);
      const Item& it = w.it;
      // Lane x's rows of keys and values of key tile t: key 32 lw + x.  Its
      // page's number is fetched a tile ahead and looked at when its rows are due.
      int page_next = 0;
      auto page_index = [&](int key) { return p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size; };
      auto fetch_page = [&](int t) {
        const int key = t * kRows + lw * 32 + lane % 32;
        if (t < it.t1 && t < w.ctx && key < it.len) page_next = p.table[it.seq * p.ld_table + page_index(key)];
      };
      const void *src_k = nullptr, *src_v = nullptr;
      auto find_rows = [&](int t) {
        src_k = src_v = nullptr;
        if (t < w.ctx) {
          const int key = t * kRows + lw * 32 + lane % 32;
          if (key >= it.len) return;
          const int64_t page = page_next;
          if (page < 0 || page >= p.num_pages) {
            record_error(p.status, QERL_ERR_RANGE);
            return;
          }
          const int64_t row = key - static_cast<int64_t>(page_index(key)) * p.page_size;
          const int64_t at = ((page * p.kv_heads + it.kv_head) * p.page_size + row) * (D * (kFp8 ? 1 : 2));
          src_k = p.kp + at;
          src_v = p.vp + at;
        } else {
          const int node = (t - w.ctx) * kRows + lw * 32 + lane % 32;
          if (node >= it.n) return;
          src_k = p.k + (static_cast<int64_t>(it.start) + node) * p.ldk + it.kv_head * D;
          src_v = p.v + (static_cast<int64_t>(it.start) + node) * p.ldv + it.kv_head * D;
        }
      };
      // The buffers of the queries.  Rows that both query tiles share lie in the
      // first, free with the last scores of the item before if that was such a
      // one too; outputs pass through the second, or through both.  (The item
      // before the last is always waited for, so that no barrier is a phase
      // further than the one asked for.)
      const bool with_scores = w.shared && shared_before;
      shared_before = w.shared;
      auto queries_free = [&](bool block) -> bool {
        if (k >= 2) {
          const uint32_t bar = out_free(k & 1), parity = ((k >> 1) & 1) ^ 1;
          if (!(block ? wait(bar, parity) : passed(bar, parity))) return false;
        }
        if (k == 0) return true;
        const uint32_t bar = with_scores ? q_free : out_free((k - 1) & 1);
        const uint32_t parity = (with_scores ? k - 1 : (k - 1) >> 1) & 1;
        return block ? wait(bar, parity) : passed(bar, parity);
      };
      drop_laps();
      if (!more) break;
      fetch_page(it.t0);
      auto load_queries = [&]() {
#pragma unroll 1
        for (int i = 0; i < (w.shared ? 1 : 2); ++i) {
          const int row = it.row0 + i * kRows + lw * 32 + lane;
          const void* src = nullptr;
          if (row < it.n * p.group) {
            int head;
            const int token = token_of(p, it, row - it.row0, head);
            src = p.q + (static_cast<int64_t>(it.start) + token) * p.ldq +
                  static_cast<int64_t>(it.kv_head * p.group + head) * D;
          }
          copy_rows(sbase + i * S::kTile, src);
        }
        cp_async_arrive(q_full);
      };
      if (kFp8) {
        // The first raw tile on its way, the queries, then tile after tile, each
        // making room for the next.  Nothing is kept back from the others here.
        bool raw = it.t0 < w.ctx;
        find_rows(it.t0);
        const void* src = group == 0 ? src_k : src_v;
        if (raw) {
#pragma unroll 2
          for (int q = 0; q < kRawChunks; ++q) copy_raw(q, src);
        }
        fetch_page(it.t0 + 1);
        if (group == 0) {
          ok = queries_free(true);
          if (!ok) break;
          load_queries();
        }
#pragma unroll 1
        for (int t = it.t0; t < it.t1; ++t) {
          const void* next = nullptr;
          if (t + 1 < it.t1) {
            find_rows(t + 1);
            next = group == 0 ? src_k : src_v;
            fetch_page(t + 2);
          }
          const bool raw_next = t + 1 < it.t1 && t + 1 < w.ctx;
          ok = next_slot(group);
          if (!ok) break;
          if (raw) {
            cp_async_wait_all();
            widen(next, raw_next);
          } else {
            copy_rows(slot_at(group, n), src);
            cp_async_arrive(full(slot_of(group, n)));
          }
          ++n;
          ++count;
          src = next;
          raw = raw_next;
        }
      } else {
        // The queries as soon as their buffers are free, but no later than the
        // third tile: nothing gives the slots of an item back without them.
        static_assert(S::kKeySlots >= 2 && S::kValueSlots >= 2, "two tiles may come before the queries");
        bool asked = false;
#pragma unroll 1
        for (int u = 0; u <= 2 * (it.t1 - it.t0); ++u) {
          const int t = it.t0 + (u >> 1), part = u & 1;
          const bool tail = t == it.t1, due = u == 4 || tail;
          if (!asked && queries_free(due)) {
            asked = true;
            load_queries();
          }
          ok = asked || !due;
          if (!ok || tail) break;
          if (part == 0) {
            find_rows(t);
            fetch_page(t + 1);
          }
          ok = next_slot(part);
          if (!ok) break;
          copy_rows(slot_at(part, n), part == 0 ? src_k : src_v);
          cp_async_arrive(full(slot_of(part, n)));
          n += part;
          count += part;
        }
      }
    }
    cp_async_wait_all();  // every copy lands before the CTA exits
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
    if (warp < kFinder) {
      const uint32_t leader = elect_lane();
      // Each issues the products of one query tile.
      const int i = warp - kIssuer;
      const uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);  // v: rows along the contraction
      // A slot is free after two arrivals: one of each issuer where both use it,
      // or both of the one that does.
      auto release = [&](int part, unsigned n, bool alone) {
        commit(leader, empty(slot_of(part, n)));
        if (alone && leader) mbar_arrive_a(empty(slot_of(part, n)));
      };
      unsigned n0 = 0, count0 = 0, tiles_done = 0, turns = 0;
      bool ok = true, first_turn = i == 0;  // of tile 0: nobody hands it over
      Work w;
      for (int k = 0; ok && take(k, w); ++k) {
        const int n = w.count(i);
        // Of every item, with or without tiles of this one: a barrier's phase is only told from the one before.
        ok = __all_sync(~0u, wait_for(q_full, k & 1, abort_flag, p.status));
        if (!ok) break;
        if (n == 0) {
          if (leader) mbar_arrive_a(q_free);
        } else {
          const float ks = kFp8 && p.k_scale != nullptr ? p.k_scale[w.it.kv_head] : 1.0f;
          auto tile_of = [&](int j) { return static_cast<unsigned>(w.tile(i, j) - w.it.t0); };
          auto wait_part = [&](int part, int j) { return wait_load(part, n0 + tile_of(j), count0 + tile_of(j)); };
          // One place each for the two products, as code is fetched cold at every item,
          // and in a turn nothing but waits and products until the next scores are
          // on their way: the softmax of this tile waits for them.
          const uint32_t qa = sbase + (w.shared ? 0 : i * S::kTile);
          for (int j = -1; j < n; ++j) {
            const bool more = j + 1 < n;
            const int t = j < 0 ? 0 : w.tile(i, j), t_next = more ? w.tile(i, j + 1) : 0;
            const uint32_t va = j < 0 ? 0 : slot_at(1, n0 + tile_of(j)), ka = more ? slot_at(0, n0 + tile_of(j + 1)) : 0;
            const int steps = j < 0 ? 0 : 2 * w.parts(t);
            // rows of an E4M3 cache and their weights are fp16
            const uint32_t id_v = kFp8 && t < w.ctx ? id_o & ~(9u << 7) : id_o;
            // a negative factor of the scores: the product is negated
            const bool negative = p.scale_log2 < 0.0f != (t_next < w.ctx && ks < 0.0f);
            const uint32_t id_k = idesc_bf16_f32(128, more ? 32 * w.parts(t_next) : 32) | (negative ? 1u << 13 : 0u);
            if (j >= 0) {
              ok = wait_part(1, j);
              if (!w.shared) {
                // Turns, as the two tiles would fall into step: both in the softmax, then both at the tensor
                // core (without turns 4 x 512 tokens over 8192 rows 269 us, handed on before the scores 247,
                // behind them 226, in their midst, so that the other's products follow at once, 223).
                ok = ok && (!more || wait_part(0, j + 1));
                if (ok && !first_turn) ok = wait_for(turn(i), (turns - (i == 0 ? 1 : 0)) & 1, abort_flag, p.status);
                first_turn = false;
                ++turns;
              }
#pragma unroll 1
              for (int half = 0; half < 2; ++half) {
                ok = __all_sync(~0u, ok && wait_for(p_full(i, half), (tiles_done + j) & 1, abort_flag, p.status));
                if (!ok) break;
                if (half == 0) fence_proxy_async_smem();
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  if (4 * half + kk < steps)
                    mma_ts(leader, tmem + 256 + i * D, tmem + i * 128 + half * 32 + kk * 8,
                           sw128_mnmajor_desc(va + half * 8192 + kk * 2048), id_v, j > 0 || half > 0 || kk > 0 ? 1u : 0u);
              }
              if (!ok) break;
            }
            if (more) {
              if (w.shared || j < 0) {
                if (j >= 0) release(1, n0 + tile_of(j), true);
                ok = __all_sync(~0u, wait_part(0, j + 1));
                if (!ok) break;
                // (the loads are ordinary writes of other threads, seen here through the barrier)
                fence_proxy_async_smem();
                tc_fence_after();
              }
#pragma unroll
              for (int d = 0; d < S::kPanels; ++d)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma_ss(leader, tmem + i * 128, sw128_kmajor_desc(qa + d * kPanel + kk * 32),
                         sw128_kmajor_desc(ka + d * kPanel + kk * 32), id_k, d + kk > 0 ? 1u : 0u);
                  if (d * 4 + kk + 1 == 2 * S::kPanels && !w.shared && j >= 0 && leader)
                    mbar_arrive_a(turn(1 - i));
                }
              commit(leader, s_full(i));
            } else {
              commit(leader, o_full(i));
            }
            if (!w.shared && !more && leader) mbar_arrive_a(turn(1 - i));
            if (j >= 0 && !(w.shared && more)) release(1, n0 + tile_of(j), w.shared);
            if (more) release(0, n0 + tile_of(j + 1), w.shared);
            if (j + 2 == n) commit(leader, q_free);
          }
        }
        tiles_done += n;
        n0 = (n0 + w.it.t1 - w.it.t0) % S::kLaps;
        count0 += w.it.t1 - w.it.t0;
      }
      commit(leader, done);  // also after an expired wait: arrives once the issued MMAs are done
    } else if (warp == kFinder) {
      // The items of this CTA's stretch, ahead of the others.
      auto owner = [&](long long pos) -> int {  // the CTA whose stretch holds a place
        const long long wide = extra * (each + 1);
        return static_cast<int>(pos < wide ? quotient(pos, each + 1) : extra + quotient(pos - wide, each));
      };
      int4 job = make_int4(0, 0, 0, 0);
      int k = 0;
      auto put = [&](const Item& it) -> bool {
        const int e = k & 1;
        if (k >= 2 && !__all_sync(~0u, wait_patiently(item_empty(e), ((k >> 1) & 1) ^ 1, abort_flag, p.status)))
          return false;
        if (lane == 0) {
          const int v[11] = {it.start, it.n,  it.len,  it.seq,    it.kv_head, it.row0,
                             it.t0,    it.t1, it.slot, it.token0, it.head0};
#pragma unroll
          for (int x = 0; x < 11; ++x) items[e * kItemInts + x] = v[x];
          mbar_arrive_a(item_full(e));
        }
        __syncwarp();
        ++k;
        return true;
      };
      bool go = busy;
      if (go) {
        int b = seq;
        const long long wide = sq.before(p, sq.blocks);  // of a key-value head
        int kv_head = static_cast<int>(quotient(inside, wide)), block = 0;
        inside -= kv_head * wide;
        for (int beyond = sq.blocks; beyond - block > 1;) {  // the block in which the place lies
          const int middle = block + (beyond - block) / 2;
          (sq.before(p, middle) <= inside ? block : beyond) = middle;
        }
        int t = static_cast<int>(inside - sq.before(p, block));
        for (long long pos = begin; go && pos < end;) {
          const long long base = pos - t;
          const int needed = sq.needed(p, block);
          const int t1 = static_cast<int>(min(static_cast<long long>(needed), t + (end - pos)));
          if (t < t1) {
            const bool whole = t == 0 && t1 == needed;
            go = put({sq.start, sq.n, sq.len, b, kv_head, block * kBlock, t, t1, whole ? -1 : t == 0 ? 1 : 0,
                      block * kBlock / p.group, block * kBlock % p.group});
            if (t == 0 && !whole)
              job = make_int4(b, kv_head, block * kBlock, owner(base + needed - 1) - static_cast<int>(blockIdx.x) + 1);
          }
          pos = base + needed + kSegmentCost;
          t = 0;
          if (++block == sq.blocks) {
            block = 0;
            if (++kv_head == p.kv_heads) {
              kv_head = 0;
              for (++b; b < p.num_seqs; b += 32) {  // the next sequence with new tokens
                const bool some = b + lane < p.num_seqs && p.cu[b + lane + 1] > p.cu[b + lane];
                const unsigned which = __ballot_sync(~0u, some);
                if (which != 0) {
                  b += __ffs(which) - 1;
                  break;
                }
              }
              if (b >= p.num_seqs) break;
              sequence(p, b, sq);
            }
          }
        }
      }
      if (!busy || go) put({});
      if (lane == 0) p.jobs[blockIdx.x] = job;
    }
  }
  __syncwarp();
  {  // every MMA is done before the tensor memory goes back (bounded)
    volatile int no_abort = 0;
    if (!wait_patiently(done, 0, abort_flag, p.status)) wait_for(done, 0, &no_abort, p.status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

// Block (c, y): 16 columns of the segment that CTA c began and others went on with.
template <int D, bool kFp8>
__global__ void __launch_bounds__(kBlock) join_kernel(const __grid_constant__ TreeParams p) {
  griddep_wait();
  const int4 job = p.jobs[blockIdx.x];
  if (job.w == 0) return;
  const int start = p.cu[job.x], rows = (p.cu[job.x + 1] - start) * p.group;
  const int row = job.z + threadIdx.x;
  if (row >= rows) return;
  const float kInf = __int_as_float(0x7f800000);
  const int64_t slot = slot_floats(p.slot_rows, D);
  // The first partial is in the second slot of its CTA, the others in the first of theirs.
  auto part = [&](int c) { return p.part + (2 * (static_cast<int64_t>(blockIdx.x) + c) + (c == 0 ? 1 : 0)) * slot; };
  constexpr int kBatch = 4;  // partials in flight
  float top = -kInf, sum = 0.0f;
  float acc[16] = {};
  for (int c0 = 0; c0 < job.w; c0 += kBatch) {
    float m[kBatch], l[kBatch];
    float4 v[kBatch][4];
    float up = top;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      m[q] = -kInf;
      l[q] = 0.0f;
      if (c0 + q < job.w) {
        const float* src = part(c0 + q);
        m[q] = __ldcg(src + static_cast<int64_t>(D) * p.slot_rows + threadIdx.x);
        l[q] = __ldcg(src + static_cast<int64_t>(D + 1) * p.slot_rows + threadIdx.x);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[q][e] = __ldcg(reinterpret_cast<const float4*>(src) +
                           static_cast<int64_t>(blockIdx.y * 4 + e) * p.slot_rows + threadIdx.x);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[q][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) up = fmaxf(up, m[q]);
    const float f0 = weight_of(top, up);
    top = up;
    sum *= f0;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] *= f0;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const float f = weight_of(m[q], top);
      sum += f * l[q];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[4 * e] += f * v[q][e].x;
        acc[4 * e + 1] += f * v[q][e].y;
        acc[4 * e + 2] += f * v[q][e].z;
        acc[4 * e + 3] += f * v[q][e].w;
      }
    }
  }
  const int token = row / p.group, head = job.y * p.group + row - token * p.group;
  const float f = sum == 0.0f ? 0.0f : (kFp8 && p.v_scale != nullptr ? value_unit(p.v_scale[job.y]) : 1.0f) / sum;
  uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(start) + token) * p.ldo +
                                        static_cast<int64_t>(head) * D + blockIdx.y * 16);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    dst[e] = make_uint4(pack_bf16(acc[8 * e] * f, acc[8 * e + 1] * f), pack_bf16(acc[8 * e + 2] * f, acc[8 * e + 3] * f),
                        pack_bf16(acc[8 * e + 4] * f, acc[8 * e + 5] * f),
                        pack_bf16(acc[8 * e + 6] * f, acc[8 * e + 7] * f));
  if (blockIdx.y == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(start) + token) * p.heads + head] =
        sum == 0.0f ? -kInf : (top + (log2f(sum) - kAbove<kFp8>)) * 0.69314718055994530942f;
}

template <int D, bool kFp8>
qerl_status launch(const TreeParams& p, int grid, int dev, cudaStream_t s) {
  using S = Shape<D, kFp8>;
  static std::atomic<uint64_t> ready{0};  // one bit per device: the attribute belongs to the device's function
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if ((ready.load() & bit) == 0) {
    if (cudaFuncSetAttribute(tree_kernel<D, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
        cudaSuccess)
      return QERL_ERR_CUDA;
    ready.fetch_or(bit);
  }
  if (launch_dependent(tree_kernel<D, kFp8>, dim3(static_cast<unsigned>(grid)), S::kThreads, S::kSmem, s, p) !=
      cudaSuccess)
    return QERL_ERR_CUDA;
  return cuda_status(
      launch_dependent(join_kernel<D, kFp8>, dim3(static_cast<unsigned>(grid), D / 16), kBlock, 0, s, p));
}

// Rows of a partial: no segment has more.
int slot_rows(int64_t tokens, int group) {
  return static_cast<int>(std::min<int64_t>(kBlock, (tokens * group + 31) / 32 * 32));
}

}  // namespace

size_t tree_attention_workspace_bytes(int64_t tokens, int num_heads, int num_kv_heads, int head_dim) {
  const size_t slot = slot_floats(slot_rows(tokens, num_heads / num_kv_heads), head_dim) * sizeof(float);
  return kWsHeaderBytes + align_up(kMaxCtas * sizeof(int4), 256) + 2 * kMaxCtas * slot;
}

qerl_status launch_tree_attention(const TreeAttentionArgs& a, cudaStream_t s) {
  const qerl_kv_cache& c = *a.cache;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QERL_ERR_CUDA;
  TreeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.kp = static_cast<const uint8_t*>(c.k);
  p.vp = static_cast<const uint8_t*>(c.v);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.table = c.page_table;
  p.ld_table = c.ld_table;
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.page_shift = (c.page_size & (c.page_size - 1)) == 0 ? __builtin_ctz(c.page_size) : -1;
  p.capacity = c.max_pages * c.page_size;
  p.cu = a.cu_tokens;
  p.lengths = a.lengths;
  p.mask = reinterpret_cast<const unsigned long long*>(a.mask);
  p.words = a.mask_words;
  p.num_seqs = static_cast<int>(c.num_seqs);
  p.tokens = static_cast<int>(a.tokens);
  p.heads = a.num_heads;
  p.kv_heads = c.num_kv_heads;
  p.group = a.num_heads / c.num_kv_heads;
  p.group_inverse = p.group == 1 ? 0 : static_cast<unsigned>(((uint64_t{1} << 32) + p.group - 1) / p.group);
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ldo = a.ldo;
  p.lse = a.lse;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  p.jobs = reinterpret_cast<int4*>(ws + kWsHeaderBytes);
  p.part = reinterpret_cast<float*>(ws + kWsHeaderBytes + align_up(kMaxCtas * sizeof(int4), 256));
  p.slot_rows = slot_rows(a.tokens, p.group);
  const int grid = std::min(sms, kMaxCtas);
  if (c.head_dim == 128)
    return c.dtype == QERL_E4M3 ? launch<128, true>(p, grid, dev, s) : launch<128, false>(p, grid, dev, s);
  return c.dtype == QERL_E4M3 ? launch<64, true>(p, grid, dev, s) : launch<64, false>(p, grid, dev, s);
}

}  // namespace qerl

#ifdef QERL_TEST_HOOKS
// Test-only build: this file's wait limit, and one arrival too many expected on
// the barriers that announce the first half of a tile's weights.
extern "C" QERL_API int qerl_test_set_tree_hooks(long long wait_limit_cycles, int extra_arrival) {
  if (cudaMemcpyToSymbol(qerl::g_test_wait_limit, &wait_limit_cycles, sizeof(wait_limit_cycles)) != cudaSuccess)
    return 1;
  return cudaMemcpyToSymbol(qerl::g_test_extra_arrival, &extra_arrival, sizeof(extra_arrival)) != cudaSuccess ? 1 : 0;
}
#endif
