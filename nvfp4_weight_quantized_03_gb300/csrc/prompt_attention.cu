// prompt_attention.cu -- causal attention of packed whole prompts on the
// tensor cores.
//
//   s_ij = scale * q_i . k_j,  j <= i within the sequence;
//   out_i = sum_j exp(s_ij - lse_i) v_j,   lse_i = log sum_j exp(s_ij)
//
// Bound: the two products, 4 * head_dim operations per (i, j <= i, head).
//
// A CTA per SM takes items of 256 query rows of one head as two tiles of 128
// rows and walks the keys in tiles of 128: one key tile in shared memory serves
// both, and the tensor core has one query tile's products to run while the
// other tile's softmax is computed.
//   warps 0-3, 4-7  softmax of tile 0, tile 1: a thread owns a row, reads its
//                   128 scores from tensor memory, keeps the reference m and
//                   the sum l in registers and writes the weights back as bf16
//                   over the scores, where the second product reads them; then
//                   the tile's outputs
//   warp 8          TMA: q, then k, v tiles through a ring
//   warps 9, 10     issue S_i = Q_i K^T and O_i += P_i V of tile 0, tile 1
//   warp 11         finds the CTA's next items
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (head_dim each).
//
// The reference m moves only when a score passes it by 2^8 (base-2 units), so
// rescaling O (a round trip through the registers) is rare; 2^(s - m) and the
// sums stay far inside fp32's and bf16's range.
//
// Roundings: scores, m, l, O are fp32.  The weights 2^(s - m) are rounded to
// bf16 for the product with v (the tensor core takes both operands in one
// type, and v is bf16); l sums the unrounded weights.
//
// A masked weight is 0, but 0 * NaN is NaN: the value rows of the diagonal
// tile (the only one with masked keys) are looked through before the product,
// non-finite elements are replaced by 0 there and added back in the epilogue
// to the rows that do attend to them.
//
// Measured, 8192 rows x 40 heads of 128 (687 GFLOP; 364 us at the rate of a
// large bf16 product): one issuer for both tiles 594 us, an issuer each with
// descriptors in uniform registers 502 us, the value product begun at half of
// the weights 492 us, persistent CTAs 467 us, items found ahead and outputs in
// whole lines 421 us in a captured graph, 428 us a call (1.61 to 1.63 PFLOP/s).
// Short prompts are further away (28/4 heads: 4 of 2000 rows 91 us = 0.66 of the
// rate, 12 to 3001 0.56, 16 to 500 29 us = 0.31): half of a diagonal tile's
// products are masked, and an item's end, where the softmax warps also write the
// outputs, takes about 2000 cycles.  What is left is the tiles' own chain
// (scores, softmax, weights, products: 2860 cycles a pair of tiles where the
// products take 2048).  Heads of 64 have half the products per exponential and
// are held by the softmax: 2400 cycles a pair, of which the exponentials of
// both tiles take 1024 and their issue 1320 on each scheduler.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "qerl_internal.h"
#include "qerl_ptx.cuh"

namespace qerl {
namespace {

constexpr int kRows = 128;   // rows of a query tile, keys of a key tile
constexpr int kBlock = 256;  // query rows of a CTA
// Two softmax warpgroups and one for the rest, which gives registers to them:
// at launch 384 threads have 168 each; 256 * 224 + 128 * 56 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
constexpr uint32_t kPanel = kRows * 128;  // 128 rows of 64 bf16, 128-byte swizzle
constexpr float kSlack = 8.0f;
// The longest sequence.  A wait may last two items (the loads and the finder are
// done that much before the last outputs), and an item takes 1430 cycles per key
// tile: 2^24 rows stay 5 times below the wait limit of 4e9 cycles, which would
// otherwise report a timeout for a call that is only long.
constexpr int kMaxRows = 1 << 24;

struct PromptParams {
  const __nv_bfloat16* v;  // for the epilogue of a tile with non-finite values
  int64_t ldv;
  const int* cu;
  int num_seqs;
  int tokens, heads, group;
  float c;       // |scale| * log2(e)
  int negative;  // scale < 0: the first product is negated
  __nv_bfloat16* out;
  int64_t ldo;
  float* lse;
  int* status;
};
struct PromptMaps {
  CUtensorMap q, k, v;
};

template <int D>
struct Shape {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kTile = kPanels * kPanel;
  static constexpr unsigned kSlots = D == 128 ? 4 : 8;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kStage = kRing + kSlots * kTile;  // 64 output columns of each query tile
  static constexpr uint32_t kBars = kStage + 2 * kPanel;
  static constexpr uint32_t kSmem = 1024 + kBars + 384;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// x * 0 + c for two bf16
__device__ __forceinline__ uint32_t times0_plus(uint32_t x, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(c));
  return d;
}
// Two fp32 operations in one instruction, each rounded as a single one.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 16 or 32 columns of this thread's lane without waiting for them.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Ties registers to this place: their readers cannot be moved above it (and so
// not above the wait for the load that fills them).
template <int N>
__device__ __forceinline__ void pin(float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile(""
                 : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                   "+f"(v[i + 6]), "+f"(v[i + 7]));
}

// Descriptor of an operand whose rows run along the contraction (v: [key][64
// elements] panels): 128-byte swizzle, 8-key groups 1024 B apart (stride
// offset), the next 64 elements one panel on (leading offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(kPanel >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// The issuing warps stay converged and one lane's predicate guards each
// instruction: descriptors then live in uniform registers.  From a branch that
// one lane takes, every product paid for moving them there (85 instead of 60
// cycles between products of 64 cycles).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}

// Where the counters of the ring's loads and of a tile's steps begin.  A CTA
// counts over all its items, so they may pass 2^32: they are unsigned, and only
// their residues (slot and phase) are used, which the wrap keeps because 2^32 is
// a multiple of two laps of the ring.  The start is too.
#ifdef QERL_TEST_HOOKS
__device__ unsigned g_test_first_count = 0;
#define QERL_FIRST_COUNT g_test_first_count
#else
#define QERL_FIRST_COUNT 0u
#endif

// The work of a CTA: query rows [row0, row0 + 256) of one sequence.
struct Item {
  int start, len, t;  // the sequence's first row and length; the block's index in it
};

// The blocks of sequence s; -1 if its offsets break the rules.
__device__ __forceinline__ int blocks_of(const PromptParams& p, int s, int& start, int& len) {
  start = p.cu[s];
  const int end = p.cu[s + 1];
  len = 0;
  if (start < 0 || end < start || end > p.tokens || end - start > kMaxRows) return -1;
  len = end - start;
  return (len + kBlock - 1) / kBlock;
}

// All sequences' blocks in the order of their cost: those of index `level`
// within their sequence in the order of the sequences, level descending (the
// last blocks to start are the cheapest).  find() is called by a whole warp
// with ranks that do not decrease and goes on from where it was, so a CTA's
// calls together look at each (level, sequence) once at most.  The sequences are
// taken in up to 32 groups, and a level passes over the groups that have no
// block in it.  A group that is looked through has one, so the ranks between a
// CTA's items bound the steps between them: of 2^20 sequences with one long one
// among them a level takes 1024 steps where all of them take 32768 (at a few
// hundred cycles a step, the 304 levels that may lie between two items of one
// head would take most of the 4e9 cycles that a wait may last).
struct Finder {
  int level, s0;
  int group_shift;  // a group: 32 << group_shift sequences
  int group_most;   // lane g's: the most blocks of a sequence of group g
  int64_t passed;   // blocks before sequence s0 of this level

  // One sequence that breaks the rules leaves nothing to find: the offsets
  // around it may lie before those of other sequences, and two CTAs would then
  // write the same rows.
  __device__ __forceinline__ void begin(const PromptParams& p) {
    const int lane = threadIdx.x & 31;
    int start, len;
    bool bad = false;
    group_shift = 0;
    while ((1024 << group_shift) < p.num_seqs) ++group_shift;
    group_most = 0;
    for (int g = 0; (g << group_shift) * 32 < p.num_seqs; ++g) {
      const int end = min(((g + 1) << group_shift) * 32, p.num_seqs);
      int most = 0;
      for (int s = ((g << group_shift) * 32) + lane; s < end; s += 32) {
        const int n = blocks_of(p, s, start, len);
        most = max(most, n);
        bad |= n < 0;
      }
      most = __reduce_max_sync(~0u, most);
      if (lane == g) group_most = most;
    }
    if (bad) record_error(p.status, QERL_ERR_RANGE);
    level = __any_sync(~0u, bad) ? -1 : __reduce_max_sync(~0u, group_most) - 1;
    s0 = 0;
    passed = 0;
  }
  __device__ __forceinline__ bool find(const PromptParams& p, int64_t rank, Item& it) {
    const int lane = threadIdx.x & 31;
    for (; level >= 0; --level, s0 = 0) {
      const unsigned groups = __ballot_sync(~0u, group_most > level);
      for (; s0 < p.num_seqs; s0 += 32) {
        const int g = s0 >> (group_shift + 5);
        if ((groups >> g & 1) == 0) {  // to the group's end
          s0 = (((g + 1) << group_shift) - 1) * 32;
          continue;
        }
        int start = 0, len = 0;
        const bool has = s0 + lane < p.num_seqs && blocks_of(p, s0 + lane, start, len) > level;
        const unsigned mask = __ballot_sync(~0u, has);
        const int n = __popc(mask);
        if (rank - passed < n) {
          const unsigned mine = __ballot_sync(~0u, has && __popc(mask & ((1u << lane) - 1)) == rank - passed);
          const int src = __ffs(mine) - 1;
          it.t = level;
          it.start = __shfl_sync(~0u, start, src);
          it.len = __shfl_sync(~0u, len, src);
          return true;
        }
        passed += n;
      }
    }
    return false;
  }
};

// A CTA works through items (query blocks x heads) until none are left; the
// softmax, the issuers and the loads each run ahead as far as their buffers
// allow, so an item's first loads and products overlap the end of the one
// before it.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptMaps maps, const PromptParams p) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (sbase - raw);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // uniform to the compiler too

  const uint32_t bars = sbase + S::kBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S::kSlots + s); };
  const uint32_t misc = bars + 16u * S::kSlots;
  auto s_full = [&](int i) { return misc + 8u * i; };
  auto p_full = [&](int i, int part) { return misc + 8u * (2 + 2 * i + part); };
  auto o_full = [&](int i) { return misc + 8u * (6 + i); };
  auto turn = [&](int i) { return misc + 8u * (8 + i); };
  auto q_full = [&](int i) { return misc + 8u * (10 + i); };
  auto q_empty = [&](int i) { return misc + 8u * (12 + i); };
  auto item_full = [&](int e) { return misc + 8u * (14 + e); };
  auto item_empty = [&](int e) { return misc + 8u * (16 + e); };
  const uint32_t done = misc + 8u * 18;
  const uint32_t tmem_holder = misc + 8u * 19;
  uint8_t* misc_gen = gen + S::kBars + 16 * S::kSlots;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc_gen + 8 * 19 + 4);
  volatile int* dirty = reinterpret_cast<volatile int*>(misc_gen + 8 * 20);         // [4]: item k's at k & 3 is k + 1
  volatile int* items = reinterpret_cast<volatile int*>(misc_gen + 8 * 20 + 16);    // [2][4]

  if (threadIdx.x == 0) {
    for (unsigned s = 0; s < S::kSlots; ++s) {
      mbar_init_a(full(s), 1);
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
      mbar_init_a(q_full(i), 1);
      mbar_init_a(q_empty(i), 1);
      mbar_init_a(item_full(i), 1);
      mbar_init_a(item_empty(i), 11);  // 8 softmax warps, the loads and 2 issuers
    }
    mbar_init_a(done, 2);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) dirty[i] = 0;
    fence_mbarrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *reinterpret_cast<volatile uint32_t*>(misc_gen + 8 * 19), 0);

  griddep_wait();

  // The item in hand, read from the ring by a whole warp; false: no more.
  struct Work {
    Item it;
    int head, n0, n1;  // key tiles of query tile 0, 1 (0: it has no rows)
  };
  auto take = [&](int k, Work& w) -> bool {
    const int e = k & 1;
    // (a warp goes on or gives up as a whole, here and at every wait of a whole warp)
    if (!__all_sync(~0u, mbar_wait_a(item_full(e), (k >> 1) & 1, abort_flag, p.status))) return false;
    w.it.start = items[e * 4];
    w.it.len = items[e * 4 + 1];
    w.it.t = items[e * 4 + 2];
    w.head = items[e * 4 + 3];
    w.n0 = 2 * w.it.t + 1;
    w.n1 = w.it.t * kBlock + kRows < w.it.len ? 2 * w.it.t + 2 : 0;
    __syncwarp();
    if (lane == 0) mbar_arrive_a(item_empty(e));
    return w.it.len > 0;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2;               // query tile
    const int r = (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + i * 128, o_t = tmem + lanes + 256 + i * D;
    const float kInf = __int_as_float(0x7f800000);
    bool ok = true;
    unsigned tiles_done = QERL_FIRST_COUNT, u0 = QERL_FIRST_COUNT;  // of this query tile; loads of the ring before this item
    int outputs_done = 0;
    Work w;
    for (int k = 0; ok && take(k, w); ++k) {
      const int mine = i == 0 ? w.n0 : w.n1;
      float mc = -kInf, l = 0.0f;  // the reference in base-2 units and the sum of 2^(s - m)
      // The values of the diagonal tile (load u of the ring), looked through for
      // elements that are not finite; a thread takes one key's row.
      auto clean_values = [&](unsigned u) -> bool {
        const unsigned s = u % S::kSlots;
        if (!__all_sync(~0u, mbar_wait_a(full(s), (u / S::kSlots) & 1, abort_flag, p.status))) return false;
        const uint32_t row = sbase + S::kRing + s * S::kTile + r * 128;
        // x * 0 + sum is NaN from the first x that is not finite
        uint32_t sum = 0;
#pragma unroll
        for (int q = 0; q < S::kPanels * 8; ++q) {
          const uint4 w = lds128(row + (q >> 3) * kPanel + (((q & 7) ^ (r & 7)) << 4));
          sum = times0_plus(w.x, sum);
          sum = times0_plus(w.y, sum);
          sum = times0_plus(w.z, sum);
          sum = times0_plus(w.w, sum);
        }
        const bool bad = (sum & 0x7FFF7FFFu) != 0;
        if (bad) {
          dirty[k & 3] = k + 1;
          for (int q = 0; q < S::kPanels * 8; ++q) {
            const uint32_t at = row + (q >> 3) * kPanel + (((q & 7) ^ (r & 7)) << 4);
            uint4 w = lds128(at);
            uint32_t a[4] = {w.x, w.y, w.z, w.w};
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
      auto step = [&](int j) {
        float x[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(s_t + q * 32, x + q * 32);
        tmem_ld_wait();
        pin<128>(x);
        if (j + 1 == mine) {  // the diagonal tile: keys past r are left out
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t keep = r >= q * 32 + 31 ? ~0u : r < q * 32 ? 0u : (2u << (r - q * 32)) - 1;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((keep & (1u << e)) == 0) x[q * 32 + e] = -kInf;
          }
        }
        const uint64_t c2 = pair(p.c, p.c);
        uint64_t sums[2];  // two chains of two fp32 sums
        uint32_t w[32];
        auto weights = [&](int half) {
          const float sub = mc == -kInf ? 0.0f : mc;
          const uint64_t sub2 = pair(-sub, -sub);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float a, b;
            unpair(fma2(pair(x[half * 64 + 2 * e], x[half * 64 + 2 * e + 1]), c2, sub2), a, b);
            a = ex2(a);
            b = ex2(b);
            sums[e & 1] = add2(sums[e & 1], pair(a, b));
            w[e] = pack_bf16(a, b);
          }
        };
        auto hand_over = [&](int half) {  // half of the keys: the product with v may begin
          tmem_st_x32(s_t + half * 32, w);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_a(p_full(i, half));
        };
        // Heads of 64, whose products are short, wait for the softmax: the
        // first half's weights are then taken against the reference as it
        // stands while the maximum is found, and seldom taken again (5000
        // rows x 32 heads: 164 us, without 171; heads of 128 lose 2%).
        constexpr bool kEarly = D == 64;
        sums[0] = sums[1] = 0;
        if (kEarly) weights(0);
        float t4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t4[q] = max3(x[q * 32], x[q * 32 + 1], x[q * 32 + 2]);
#pragma unroll
          for (int e = 3; e < 31; e += 2) t4[q] = max3(t4[q], x[q * 32 + e], x[q * 32 + e + 1]);
          t4[q] = fmaxf(t4[q], x[q * 32 + 31]);
        }
        const float top = max3(fmaxf(t4[0], t4[1]), t4[2], t4[3]);
        const float tc = top == -kInf ? -kInf : top * p.c;
        if (__any_sync(~0u, tc > mc + kSlack)) {
          const float up = fmaxf(mc, tc);
          if (j > 0) {
            const float f = mc == up ? 1.0f : ex2(mc - up);
            l *= f;
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
          mc = up;
          if (kEarly) {
            sums[0] = sums[1] = 0;
            weights(0);
          }
        }
        if (!kEarly) weights(0);
        hand_over(0);
        weights(1);
        hand_over(1);
        float s0, s1;
        unpair(add2(sums[0], sums[1]), s0, s1);
        l += s0 + s1;
      };

      for (int j = 0; j < mine; ++j) {
        if (j + 1 == mine) ok = clean_values(u0 + 2 * j + 1);  // while the scores are computed
        ok = __all_sync(~0u, ok && mbar_wait_a(s_full(i), (tiles_done + j) & 1, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        step(j);
      }
      tiles_done += mine;
      u0 += 2 * max(w.n0, w.n1);
      if (mine > 0) {
        ok = __all_sync(~0u, ok && mbar_wait_a(o_full(i), outputs_done & 1, abort_flag, p.status));
        ++outputs_done;
        tc_fence_after();
        const int rs = w.it.t * kBlock + i * kRows + r;  // row in the sequence
        const bool live = ok && rs < w.it.len;
        const bool fix = dirty[k & 3] == k + 1;
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t row = static_cast<int64_t>(w.it.start) + rs;
        // 64 columns at a time through shared memory, so that a store covers
        // whole lines (a thread's own row, 16 bytes a store, took 4 times as
        // long).  Each warp uses its own 32 rows of the buffer.
        const uint32_t stage = sbase + S::kStage + i * kPanel + (warp & 3) * 32 * 128;
        const int first = rs - lane;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          float v[64];
          tmem_ld32(o_t + h * 64, v);
          tmem_ld32(o_t + h * 64 + 32, v + 32);
          tmem_ld_wait();
          pin<64>(v);
          if (fix && live) {
            for (int j = (w.n0 - 1) * kRows; j <= rs; ++j) {
              const __nv_bfloat16* src =
                  p.v + static_cast<int64_t>(w.it.start + j) * p.ldv + w.head / p.group * D + h * 64;
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                const float y = __bfloat162float(src[e]);
                if (!(fabsf(y) < kInf)) v[e] += y;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sts128(stage + lane * 128 + ((e ^ (lane & 7)) << 4),
                   make_uint4(pack_bf16(v[8 * e] * f, v[8 * e + 1] * f), pack_bf16(v[8 * e + 2] * f, v[8 * e + 3] * f),
                              pack_bf16(v[8 * e + 4] * f, v[8 * e + 5] * f),
                              pack_bf16(v[8 * e + 6] * f, v[8 * e + 7] * f)));
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 32; q += 4) {
            const int at = q + (lane >> 3), ch = lane & 7;
            const uint4 y = lds128(stage + at * 128 + ((ch ^ (at & 7)) << 4));
            if (ok && first + at < w.it.len)
              *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(w.it.start) + first + at) * p.ldo + w.head * D +
                                        h * 64 + ch * 8) = y;
          }
          __syncwarp();
        }
        if (live && p.lse != nullptr)
          p.lse[row * p.heads + w.head] = l == 0.0f ? -kInf : (mc + log2f(l)) * 0.69314718055994530942f;
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      unsigned issued = QERL_FIRST_COUNT, used = 0;  // loads; slots of the ring that hold one
      int q_loads[2] = {0, 0};
      Work w;
      for (int k = 0; take(k, w); ++k) {
        bool ok = true;
        if (lane == 0) {
          const int n = max(w.n0, w.n1);
          for (int u = 0; ok && u < 2 * n; ++u) {  // k, v, k, v, ...
            const unsigned s = issued % S::kSlots;
            if (used == S::kSlots) ok = mbar_wait_a(empty(s), ((issued / S::kSlots) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            mbar_arrive_expect_tx_a(full(s), S::kTile);
            const uint32_t dst = sbase + S::kRing + s * S::kTile;
#pragma unroll
            for (int d = 0; d < S::kPanels; ++d)
              tma_load_2d(dst + d * kPanel, (u & 1) ? &maps.v : &maps.k, w.head / p.group * D + d * 64,
                          w.it.start + (u >> 1) * kRows, full(s));
            ++issued;
            if (used < S::kSlots) ++used;
            if (u > 0) continue;
            // After the first keys, the queries (their buffers come free with the last scores of the item before).
            for (int i = 0; ok && i < (w.n1 > 0 ? 2 : 1); ++i) {
              if (q_loads[i] > 0) ok = mbar_wait_a(q_empty(i), (q_loads[i] - 1) & 1, abort_flag, p.status);
              if (!ok) break;
              mbar_arrive_expect_tx_a(q_full(i), S::kTile);
#pragma unroll
              for (int d = 0; d < S::kPanels; ++d)
                tma_load_2d(sbase + i * S::kTile + d * kPanel, &maps.q, w.head * D + d * 64,
                            w.it.start + w.it.t * kBlock + i * kRows, q_full(i));
              ++q_loads[i];
            }
          }
        }
        if (!__shfl_sync(~0u, static_cast<int>(ok), 0)) break;
      }
      if (lane == 0) {
        // Every issued copy lands before the CTA exits (after an expired wait too).
        volatile int no_abort = 0;
        for (int i = 0; i < 2; ++i)
          if (q_loads[i] > 0) mbar_wait_a(q_full(i), (q_loads[i] - 1) & 1, &no_abort, p.status);
        for (unsigned s = 0; s < used; ++s) {
          const unsigned last = issued - 1 - ((issued - 1 - s) % S::kSlots);
          mbar_wait_a(full(s), (last / S::kSlots) & 1, &no_abort, p.status);
        }
      }
    } else if (warp < 11) {
      const uint32_t leader = elect_lane();
      // Warp 9 + i issues the products of query tile i.  An issuer is held up
      // while the tensor core works its products off; with one issuer for
      // both tiles its waits left the tensor core idle for a quarter of the
      // time.
      const int i = warp - 9;
      const uint32_t id_s = idesc_bf16_f32(128, 128) | (p.negative ? 1u << 13 : 0u);
      const uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);  // v: rows along the contraction
      auto slot = [&](unsigned u) { return sbase + S::kRing + (u % S::kSlots) * S::kTile; };
      auto wait_slot = [&](unsigned u) {
        return mbar_wait_a(full(u % S::kSlots), (u / S::kSlots) & 1, abort_flag, p.status);
      };
      auto scores = [&](unsigned u) {
        const uint32_t qa = sbase + i * S::kTile, ka = slot(u);
#pragma unroll
        for (int d = 0; d < S::kPanels; ++d)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(leader, tmem + i * 128, sw128_kmajor_desc(qa + d * kPanel + kk * 32),
                   sw128_kmajor_desc(ka + d * kPanel + kk * 32), id_s, d + kk > 0 ? 1u : 0u);
        commit(leader, s_full(i));
      };
      auto values = [&](unsigned u, int part, bool more) {
        const uint32_t va = slot(u);
#pragma unroll
        for (int kk = 4 * part; kk < 4 * part + 4; ++kk)
          mma_ts(leader, tmem + 256 + i * D, tmem + i * 128 + kk * 8, sw128_mnmajor_desc(va + kk * 2048), id_o,
                 more || kk > 0 ? 1u : 0u);
      };
      // A slot is free when both issuers have released it; one whose tile
      // does not use it (fewer key tiles, or no rows) just arrives.
      auto release = [&](unsigned u, bool used) {
        if (used) {
          commit(leader, empty(u % S::kSlots));
        } else if (leader) {
          mbar_arrive_a(empty(u % S::kSlots));
        }
      };
      unsigned u0 = QERL_FIRST_COUNT, tiles_done = QERL_FIRST_COUNT, turns = QERL_FIRST_COUNT;
      int q_used = 0;
      bool ok = true, first_turn = i == 0;  // of tile 0: nobody hands it over
      Work w;
      for (int k = 0; ok && take(k, w); ++k) {
        const int mine = i == 0 ? w.n0 : w.n1, n = max(w.n0, w.n1);
        if (mine > 0) {
          ok = mbar_wait_a(q_full(i), q_used & 1, abort_flag, p.status);
          ++q_used;
        }
        ok = __all_sync(~0u, ok && wait_slot(u0));
        if (!ok) break;
        tc_fence_after();
        if (mine > 0) scores(u0);
        if (mine == 1) commit(leader, q_empty(i));
        release(u0, mine > 0);
        for (int j = 0; j < n; ++j) {
          ok = wait_slot(u0 + 2 * j + 1) && (j + 1 >= n || wait_slot(u0 + 2 * j + 2));
          // Turns: tile 0's products of a key tile, then tile 1's, then tile
          // 0's of the next.  Without them the two tiles fall into step, both
          // in the softmax and then both at the tensor core.
          if (ok && w.n1 > 0) {
            if (!first_turn) ok = mbar_wait_a(turn(i), (turns - (i == 0 ? 1 : 0)) & 1, abort_flag, p.status);
            first_turn = false;
            ++turns;
          }
          if (ok && j < mine) ok = mbar_wait_a(p_full(i, 0), (tiles_done + j) & 1, abort_flag, p.status);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          if (j < mine) {
            tc_fence_after();
            values(u0 + 2 * j + 1, 0, j > 0);
            ok = __all_sync(~0u, mbar_wait_a(p_full(i, 1), (tiles_done + j) & 1, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            values(u0 + 2 * j + 1, 1, true);
          }
          release(u0 + 2 * j + 1, j < mine);
          if (j + 1 < mine) scores(u0 + 2 * j + 2);
          if (j + 2 == mine) commit(leader, q_empty(i));
          if (w.n1 > 0 && leader) mbar_arrive_a(turn(1 - i));
          if (j + 1 == mine) commit(leader, o_full(i));
          if (j + 1 < n) release(u0 + 2 * j + 2, j + 1 < mine);
        }
        tiles_done += mine;
        u0 += 2 * n;
      }
      commit(leader, done);  // also after an expired wait: arrives once the issued MMAs are done
    } else {
      // Warp 11 finds the items, ahead of the others.  They are dealt out in
      // rounds, every other round backwards.
      Finder finder;
      finder.begin(p);
      for (int k = 0;; ++k) {
        const int64_t g = gridDim.x, c = blockIdx.x;
        const int64_t idx = k * g + ((k & 1) ? g - 1 - c : c);
        const int e = k & 1;
        Item it{0, 0, 0};
        const bool have = finder.find(p, idx / p.heads, it);
        const bool free = k < 2 || mbar_wait_a(item_empty(e), ((k >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!__all_sync(~0u, free)) break;
        if (lane == 0) {
          items[e * 4] = it.start;
          items[e * 4 + 1] = have ? it.len : 0;
          items[e * 4 + 2] = it.t;
          items[e * 4 + 3] = static_cast<int>(idx % p.heads);
          mbar_arrive_a(item_full(e));
        }
        __syncwarp();
        if (!have) break;
      }
    }
  }
  __syncwarp();
  {  // every MMA is done before the tensor memory goes back (bounded)
    volatile int no_abort = 0;
    mbar_wait_a(done, 0, &no_abort, p.status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load();
  if (f == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    fn.store(f);
  }
  return f;
}

// Rows of `width` bf16 (stride ld), read in boxes of 64 columns x 128 rows.
bool rows_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t ld) {
  const auto enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, kRows}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
qerl_status launch(const PromptMaps& maps, const PromptParams& p, int64_t grid, int dev, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // one bit per device: the attribute belongs to the device's function
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if ((ready.load() & bit) == 0) {
    if (cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem) !=
        cudaSuccess)
      return QERL_ERR_CUDA;
    ready.fetch_or(bit);
  }
  return cuda_status(
      launch_dependent(prompt_kernel<D>, dim3(static_cast<unsigned>(grid)), kThreads, Shape<D>::kSmem, s, maps, p));
}

}  // namespace

size_t prompt_attention_workspace_bytes(int64_t, int, int, int, int64_t) { return kWsHeaderBytes; }

qerl_status launch_prompt_attention(const PromptAttentionArgs& a, cudaStream_t s) {
  PromptMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const int64_t qw = static_cast<int64_t>(a.num_heads) * a.head_dim, kw = static_cast<int64_t>(a.num_kv_heads) * a.head_dim;
  if (!rows_map(&maps.q, a.q, qw, a.tokens, a.ldq) || !rows_map(&maps.k, a.k, kw, a.tokens, a.ldk) ||
      !rows_map(&maps.v, a.v, kw, a.tokens, a.ldv))
    return QERL_ERR_CUDA;
  PromptParams p{};
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.ldv = a.ldv;
  p.cu = a.cu_seqlens;
  p.num_seqs = static_cast<int>(a.num_seqs);
  p.tokens = static_cast<int>(a.tokens);
  p.heads = a.num_heads;
  p.group = a.num_heads / a.num_kv_heads;
  p.negative = a.scale < 0.0f;
  // Not 0: a masked score of -inf times 0 would be NaN (1e-37 times any score below 1e29 is as good as 0).
  p.c = std::max((a.scale < 0.0f ? -a.scale : a.scale) * 1.44269504088896340736f, 1e-37f);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ldo = a.ldo;
  p.lse = a.lse;
  p.status = &static_cast<WsHeader*>(a.workspace)->status;
  // Every sequence has at most one block that is not full.
  const int64_t blocks = a.tokens / kBlock + std::min(a.num_seqs, a.tokens);
  if (blocks * a.num_heads > INT32_MAX) return QERL_ERR_UNSUPPORTED_SHAPE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QERL_ERR_CUDA;
  const int64_t grid = std::min<int64_t>(blocks * a.num_heads, sms);  // one resident CTA per SM
  return a.head_dim == 128 ? launch<128>(maps, p, grid, dev, s) : launch<64>(maps, p, grid, dev, s);
}

}  // namespace qerl

#ifdef QERL_TEST_HOOKS
// Test-only build: where the counters begin (a multiple of 16).
extern "C" QERL_API int qerl_test_set_prompt_first_count(unsigned count) {
  if (count % 16 != 0) return 1;
  return cudaMemcpyToSymbol(qerl::g_test_first_count, &count, sizeof(count)) != cudaSuccess ? 1 : 0;
}

// Test-only build: this file's wait limit, and one arrival too many expected on
// the barriers that announce the first half of a tile's weights.
extern "C" QERL_API int qerl_test_set_prompt_hooks(long long wait_limit_cycles, int extra_arrival) {
  if (cudaMemcpyToSymbol(qerl::g_test_wait_limit, &wait_limit_cycles, sizeof(wait_limit_cycles)) != cudaSuccess)
    return 1;
  return cudaMemcpyToSymbol(qerl::g_test_extra_arrival, &extra_arrival, sizeof(extra_arrival)) != cudaSuccess ? 1 : 0;
}
#endif
