// decode_attention.cu -- attention of one new token per sequence over the
// paged key-value cache, or over a window of it.
//
//   s_j = scale * q . k_j,  j < len;   o = sum_j exp(s_j - lse) v_j,
//   lse = log sum_j exp(s_j)
// (a window of w rows and n sinks: of these j those with j >= len - w or j < n,
// which the tiles take as if they lay side by side; nothing else differs: 192
// sequences to 12000 rows, window 4096, 64 sinks, 40/8 heads 336 us = 0.96 of the
// copy rate, one of 50001 rows with a window of 1000 9.2 us, of which the call
// takes most)
// for every query head; the G = num_heads / num_kv_heads query heads of a
// key-value head read its rows together.  One pass: the running reference m
// (a maximum in base-2 units), the sum l of 2^(s - m) and the unnormalised
// output stay in registers.
//
// Bound: bytes of the cache (G multiply-adds per byte).  The work is cut by
// cost, not by sequences: all (sequence, key-value head, key tile) units in
// order form one line, weighted by their rows and the cost of a segment's start
// and join, that the resident CTAs share out evenly.  It is computed on the
// device from the lengths, so ragged batches balance and no host copy of the
// lengths is needed.  A CTA whose stretch begins or ends inside a (sequence,
// head) leaves its partial (m, l, o) in the workspace; the last of that
// head's CTAs to arrive joins the partials in CTA order (the result does not
// depend on the arrival order).
//
// Measured (in a captured graph): 128 x 6000 rows, 40/8 heads of 128, E4M3:
// 249 us = 0.93 of the copy rate; 64 ragged to 8192, 28/4, bf16: 72 us = 0.88;
// 1 x 100003, 40/8, bf16: 71 us = 0.85 (3 us before the first rows, the CTAs
// finish 12 us apart, 5 us of join); 256 ragged to 1500, 32/8 heads of 64: 49 us
// = 0.85.  Furthest from the rate are two column tiles over an E4M3 cache (64 x
// 6000 rows: 12/1 heads of 128 31 us = 0.48, 45/3 heads of 64 42 us = 0.52): 255
// and 168 registers leave 2 and 3 warps to a scheduler, which issues in 35% and
// 49% of its cycles and otherwise waits for each warp's chain.  Steps: the
// join with more than one partial in flight 96 -> 84 us on the long sequence;
// the stretch by cost, the segments' joins by one warp while the others go on,
// and the stream marked evict-first (it leaves the code and the partials in L2)
// 84 -> 73 us; many partials joined in two levels 73 -> 72 us (one sequence of
// 8000 rows 18.3 -> 12.8 us).
//
// A warp owns kKeys keys of every tile and its own ring of cp.async stages, so
// the key loop has no CTA barrier.  Products run on mma.sync.m16n8k16 with the
// keys (then the head's elements) as the 16-row operand and the query heads as
// the 8 columns: up to 8 heads fill the tile, where heads as rows would leave
// half of it empty.  A tcgen05 tile needs 64 or 128 rows, which G <= 16 heads
// do not fill.
//
// Roundings: scores, m, l and o are fp32.  bf16 cache: 2^(s - m) enters the
// value product as bf16 high + bf16 low (16 bits), which costs 8 more MMAs per
// 16 keys where the memory is the bound anyway.  E4M3 cache: keys and values
// are exact in fp16, q is scaled by a power of two per head to the top of
// fp16's range (exact unless an element is 2^31 below the head's largest),
// 2^(s - m) is rounded to fp16 (half a step 2^-11).  There m lies 2^7 below the
// maximum it was taken from, so that weights up to 2^15 use fp16's range: one
// is lost to the product only below 2^-32 of the largest (with m at the maximum
// below 2^-25, and 100000 of those are a third of a percent of the sum, which
// keeps them).
#include "attention.cuh"
#include "qerl_internal.h"

#include <algorithm>
#include <atomic>

namespace qerl {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Partials at the front of the workspace, in a region of one size for every
// shape: the counters behind it then lie at the same place for all calls that
// share a workspace, and are zero between them.
constexpr size_t kPartBytes = size_t{6} << 20;
constexpr int kMaxCtas = 1024;
constexpr size_t kGroupBytes = 2 * kMaxCtas * sizeof(unsigned);
// A segment of more CTAs than kDirect is joined in groups of kGroup CTAs first,
// by the last of each group to arrive: one CTA alone took 9 us for 76 partials.
constexpr int kDirect = 16, kGroup = 8;
// How far (base 2) a score may pass the reference m before m moves: 2^8 keeps
// the fp32 sums and the fp16 probabilities in range, and most steps then skip
// the maximum's reduction and the rescaling.
constexpr float kSlack = 8.0f;
// How far m lies below the maximum when it moves.
template <bool kFp8>
constexpr float kBelow = kFp8 ? 7.0f : 0.0f;

struct DecodeParams {
  const __nv_bfloat16* q;
  int64_t ldq;
  const uint8_t *kp, *vp;
  const float *k_scale, *v_scale;
  const int* table;
  int64_t ld_table, num_pages;
  int page_size, page_shift;  // shift < 0: not a power of two
  int64_t capacity;           // max_pages * page_size
  int num_seqs, heads, kv_heads, group;
  int zgroups, zheads;  // a key-value head's query heads in zgroups parts of zheads
  const int* lengths;
  int sinks, seen;  // a window: the rows j < sinks and the last ones, at most `seen` rows in all
  float scale_log2;
  __nv_bfloat16* out;
  int64_t ldo;
  float* lse;
  float* part;         // [CTA][2][NT * 8][D + 4]: of the segment begun before its stretch, of the one begun in it
  unsigned* counters;  // [num_seqs * kv_heads * zgroups], zero between calls
  unsigned* group_counters;  // [CTA][2], zero between calls
  int* status;
};

template <int D, bool kFp8, int NT>
struct Shape {
  static constexpr int kRow = D * (kFp8 ? 1 : 2);  // bytes of a cache row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kKeys = kRow >= 256 ? 16 : 32;  // per warp and stage
  static constexpr int kTile = kKeys * kWarps;
  // The line's unit of cost is 16 keys; a (sequence, head) costs about one and a
  // half tiles more for its start and its join (heads of 64, 256 sequences of
  // 93 to 1500 rows: half a tile 65 us, one 59 us, one and a half 55.5 us, two
  // 56.6 us).
  static constexpr int kTileCost = kTile / 16;
  static constexpr int kSegmentCost = kTileCost * 3 / 2;
  static constexpr int kStage = 2 * kKeys * kRow;  // K then V
  // CTAs per SM and stages per warp fill the shared memory.  Short rows leave
  // the warps waiting on their own chain of steps more than on memory: heads of
  // 64, bf16, three CTAs with 2 stages 51 us, two with 3 55.5 us; E4M3 (64 x
  // 6000 rows, 32/8 heads) four with 2 stages 75 us, three with 4 79 us.
  static constexpr int kCtas = kStage == 4096 ? (NT == 1 ? 4 : 3) : D == 64 && NT == 1 ? 3 : 2;
  static constexpr int kStages = kStage == 4096 ? (NT == 1 ? 2 : 3) : NT == 1 && D == 128 ? 3 : 2;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kOStride = D + 4;  // columns 2c, 2c+1 of 8 rows fall in 32 banks
  static constexpr int kJoin = kWarps * NT * 8 * kOStride * 4;
  static constexpr int kSmem = kRing + kJoin;
  static constexpr int kPartRow = D + 4;  // o; (m, l) of a CTA's partial; (m, l) of a group's sum
};

// Physical 16-byte chunk of a row in shared memory: 8 rows of one logical
// chunk fall into 8 different bank groups.
template <int kRow>
__device__ __forceinline__ uint32_t at_chunk(int row, int chunk) {
  if (kRow == 64) return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
  return static_cast<uint32_t>(row * kRow + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t o;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(v));
  return o;
}
template <bool kFp8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kFp8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// cp_async_16 with an L2 cache policy.
__device__ __forceinline__ void cp_async_16_hint(uint32_t smem_dst, const void* gsrc, uint32_t src_bytes, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(smem_dst), "l"(gsrc),
               "r"(src_bytes), "l"(pol)
               : "memory");
}

__device__ __forceinline__ unsigned atomic_add_acq_rel(unsigned* p, unsigned v) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Named barriers of the join (0 is __syncthreads), one of each for even and one
// for odd segments: the warp that joined a segment does not wait before the
// next one and may be a whole segment ahead, where its arrival must not count
// for the barrier the others are still at.
__device__ __forceinline__ int join_full(int segment) { return 1 + (segment & 1); }
__device__ __forceinline__ int join_free(int segment) { return 3 + (segment & 1); }
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

// A place on the line of work: key tile `tile` of `tiles` of (sequence b, part
// hz of its kv_heads * zgroups), which begins at `pos`.
struct Cursor {
  int b, hz, tile, tiles, len;
  int skip;  // the rows that a window leaves out, behind the sinks
  long long pos;
};

__device__ __forceinline__ int kept_length(const DecodeParams& p, int b) {
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.capacity ? static_cast<int>(p.capacity) : n;
}
// The rows of a sequence that its token attends to.
template <bool kWindow>
__device__ __forceinline__ int live_length(const DecodeParams& p, int b) {
  const int n = kept_length(p, b);
  return kWindow ? min(n, p.seen) : n;
}
template <bool kWindow>
__device__ __forceinline__ void set_length(const DecodeParams& p, Cursor& c) {
  const int n = kept_length(p, c.b);
  c.len = kWindow ? min(n, p.seen) : n;
  c.skip = n - c.len;
}

template <typename S>
__device__ __forceinline__ int segment_cost(int len) {
  return (len - 1) / 16 + 1 + S::kSegmentCost;
}

// The next tile on the line; b == num_seqs past its end.
template <typename S, bool kWindow>
__device__ __forceinline__ void advance(const DecodeParams& p, Cursor& c) {
  if (++c.tile < c.tiles) {
    c.pos += S::kTileCost;
    return;
  }
  c.pos += segment_cost<S>(c.len) - (c.tiles - 1) * S::kTileCost;
  c.tile = 0;
  if (++c.hz < p.kv_heads * p.zgroups) return;
  c.hz = 0;
  while (++c.b < p.num_seqs) {
    set_length<kWindow>(p, c);
    if (c.len > 0) {
      c.tiles = (c.len - 1) / S::kTile + 1;
      return;
    }
  }
}

template <int D, bool kFp8, int NT, bool kWindow>
__global__ void __launch_bounds__(kThreads, (Shape<D, kFp8, NT>::kCtas)) decode_kernel(const DecodeParams p) {
  using S = Shape<D, kFp8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long red[kWarps];
  __shared__ long long found[2];
  __shared__ float ml[kWarps][NT * 8][2];
  __shared__ int4 pending[2];  // (b, hz, first CTA, CTAs) of a segment to join, by slot
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hz_all = p.kv_heads * p.zgroups;
  const uint32_t ring = smem_u32(smem) + warp * (S::kStages * S::kStage);
  float* o_join = reinterpret_cast<float*>(smem + S::kRing);
  const float kInf = __int_as_float(0x7f800000);
  if (tid < 2) pending[tid] = make_int4(0, 0, 0, 0);  // before the loop's first barrier

  griddep_wait();

  // ---- this CTA's stretch of the line ---------------------------------------
  auto cost = [&](int b) -> long long {
    if (b >= p.num_seqs) return 0;
    const int n = live_length<kWindow>(p, b);
    return n > 0 ? static_cast<long long>(segment_cost<S>(n)) * hz_all : 0;
  };
  auto scan = [&](long long v) -> long long {  // inclusive over the warp
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const long long up = __shfl_up_sync(~0u, v, i);
      if (lane >= i) v += up;
    }
    return v;
  };
  // A sequence without keys: zeros and lse = -inf, shared out over the CTAs.
  for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x) {
    const int n = p.lengths[b];
    if (tid == 0 && (n < 0 || n > p.capacity)) record_error(p.status, QERL_ERR_RANGE);
    if (n > 0 && p.capacity > 0) continue;
    for (int i = tid; i < p.heads * D / 8; i += kThreads)
      *reinterpret_cast<uint4*>(p.out + b * p.ldo + i * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr)
      for (int i = tid; i < p.heads; i += kThreads) p.lse[static_cast<int64_t>(b) * p.heads + i] = -kInf;
  }
  long long total = 0, incl = 0, mine = 0;
  if (p.num_seqs <= 32) {  // every warp for itself, no barrier
    mine = cost(lane);
    incl = scan(mine);
    total = __shfl_sync(~0u, incl, 31);
  } else {
    for (int b = tid; b < p.num_seqs; b += kThreads) total += cost(b);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) total += __shfl_xor_sync(~0u, total, i);
    if (lane == 0) red[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += red[i];
  }
  if (total == 0) return;
  // Even stretches of the line; a tile belongs to the stretch in which it
  // begins.  None is shorter than a tile, so that every CTA between the owners
  // of a segment's first and last tile has a tile of it (the join counts them).
  const long long most = quotient(total, S::kTileCost);
  const long long ctas = most < 1 ? 1 : most < gridDim.x ? most : gridDim.x;
  if (blockIdx.x >= ctas) return;
  const long long each = quotient(total, ctas), extra = total - each * ctas;  // the first `extra` are one longer
  auto stretch = [&](long long c) -> long long { return each * c + (c < extra ? c : extra); };
  auto owner = [&](long long pos) -> int {  // the CTA whose stretch holds a place
    const long long wide = extra * (each + 1);
    return static_cast<int>(pos < wide ? quotient(pos, each + 1) : extra + quotient(pos - wide, each));
  };
  const long long begin = stretch(blockIdx.x), end = stretch(blockIdx.x + 1);
  // The sequence that holds `begin`, and the place in it.
  Cursor cur;
  long long inside;
  if (p.num_seqs <= 32) {
    const unsigned hit = __ballot_sync(~0u, incl - mine <= begin && begin < incl);
    cur.b = __ffs(hit) - 1;
    inside = begin - __shfl_sync(~0u, incl - mine, cur.b);
  } else {
    long long base = 0;
    for (int b0 = 0;; b0 += kThreads) {
      mine = cost(b0 + tid);
      incl = scan(mine);
      __syncthreads();
      if (lane == 31) red[warp] = incl;
      __syncthreads();
      long long before = base, all = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += red[i];
        all += red[i];
      }
      incl += before;
      if (begin < base + all) {  // uniform: in this block of sequences
        if (incl - mine <= begin && begin < incl) {
          found[0] = b0 + tid;
          found[1] = begin - (incl - mine);
        }
        __syncthreads();
        break;
      }
      base += all;
    }
    cur.b = static_cast<int>(found[0]);
    inside = found[1];
  }
  set_length<kWindow>(p, cur);
  cur.tiles = (cur.len - 1) / S::kTile + 1;
  {
    const int segment = segment_cost<S>(cur.len);
    cur.hz = static_cast<int>(quotient(inside, segment));
    const int in_segment = static_cast<int>(inside - static_cast<long long>(cur.hz) * segment);
    cur.tile = (in_segment + S::kTileCost - 1) / S::kTileCost;  // the first that begins here or later
    cur.pos = begin - in_segment + cur.tile * S::kTileCost;
    if (cur.tile >= cur.tiles) {
      cur.tile = cur.tiles - 1;
      cur.pos = begin - in_segment + cur.tile * S::kTileCost;
      advance<S, kWindow>(p, cur);
    }
  }
  if (cur.b >= p.num_seqs || cur.pos >= end) return;  // no tile begins in this stretch

  // ---- loads ----------------------------------------------------------------
  // Byte offset of this lane's key row of the cursor's tile; -1 past the length
  // or for a page number outside the cache (the row then reads as zeros).
  auto lookup = [&](const Cursor& c) -> int64_t {
    int64_t key = static_cast<int64_t>(c.tile) * S::kTile + warp * S::kKeys + (lane & (S::kKeys - 1));
    if (key >= c.len) return -1;
    // The tiles run over the visible rows as if they lay side by side.
    if (kWindow && key >= p.sinks) key += c.skip;
    const int pi = p.page_shift >= 0 ? static_cast<int>(key) >> p.page_shift : static_cast<int>(key) / p.page_size;
    const int64_t page = p.table[c.b * p.ld_table + pi];
    if (page < 0 || page >= p.num_pages) {
      record_error(p.status, QERL_ERR_RANGE);
      return -1;
    }
    return ((page * p.kv_heads + c.hz / p.zgroups) * p.page_size + (key - static_cast<int64_t>(pi) * p.page_size)) *
           S::kRow;
  };
  const uint64_t once = l2_policy_evict_first();  // the stream leaves the kernel's code in L2
  auto issue = [&](int stage, int64_t off) {
    const uint32_t base_a = ring + stage * S::kStage;
    constexpr int kPer = S::kKeys * S::kChunks / 32;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int row = (i * 32 + lane) / S::kChunks, chunk = lane % S::kChunks;
      const int64_t o = __shfl_sync(~0u, off, row);
      const uint32_t dst = base_a + at_chunk<S::kRow>(row, chunk);
      // a row of zeros: nothing is read, from an address that is memory all the same
      const bool real = o >= 0;
      const void* none = p.q;
      cp_async_16_hint(dst, real ? p.kp + o + chunk * 16 : none, real ? 16 : 0, once);
      cp_async_16_hint(dst + S::kKeys * S::kRow, real ? p.vp + o + chunk * 16 : none, real ? 16 : 0, once);
    }
  };
  // The page numbers of the first stages are fetched together, later ones a
  // step before their rows.
  Cursor ahead = cur;
  int64_t offs[S::kStages];
  bool more[S::kStages];
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) {
    if (s > 0 && more[s - 1]) advance<S, kWindow>(p, ahead);
    more[s] = (s == 0 || more[s - 1]) && ahead.b < p.num_seqs && ahead.pos < end;
    offs[s] = more[s] ? lookup(ahead) : -1;
  }
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (more[s]) issue(s, offs[s]);
    cp_async_commit();
  }
  int64_t off = offs[S::kStages - 1];
  bool to_load = more[S::kStages - 1];

  // ---- the key loop ----------------------------------------------------------
  constexpr int KS = D / 16;  // 16-element steps of a head
  constexpr int MT = S::kKeys / 16;
  const int t4 = lane & 3, g8 = lane >> 2;
  uint32_t qf[NT][KS][2];
  float mult[NT][2];
  float o[NT][KS][4];
  float m[NT][2], l[NT][2];
  // This thread's words of the queries of a (sequence, head): for the bf16
  // cache elements 2 t4, 2 t4 + 1 and 8 more on of every 16; for the E4M3 cache
  // 4 t4 .. 4 t4 + 3 (the order the bytes of a key arrive in).
  auto load_q = [&](const Cursor& c, uint32_t (&w)[NT][KS][2]) {
    const int kvh = c.hz / p.zgroups, z = c.hz - kvh * p.zgroups;
    const int nheads = min(p.zheads, p.group - z * p.zheads);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + g8;
      const __nv_bfloat16* src =
          p.q + c.b * p.ldq + static_cast<int64_t>(kvh * p.group + z * p.zheads + (h < nheads ? h : 0)) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (kFp8) {
          const uint2 v = *reinterpret_cast<const uint2*>(src + ks * 16 + 4 * t4);
          w[nt][ks][0] = v.x;
          w[nt][ks][1] = v.y;
        } else {
          w[nt][ks][0] = *reinterpret_cast<const uint32_t*>(src + ks * 16 + 2 * t4);
          w[nt][ks][1] = *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8 + 2 * t4);
        }
      }
    }
  };
  // With one column tile there are registers to fetch the next segment's
  // queries during the last tile of this one.
  constexpr bool kAheadQ = NT == 1;
  uint32_t qn[NT][KS][2];
  load_q(cur, qn);
  bool fresh = true;
  int stage = 0;
  const long long first_pos = cur.pos;
  constexpr int64_t kSlot = static_cast<int64_t>(NT * 8) * S::kPartRow;
  // Output elements d .. d + 3 of the h-th head of a segment from its (m, l, o).
  auto finish = [&](int b, int hz, int h, int d, float top, float sum, const float4& v) {
    const int kv = hz / p.zgroups;
    const int head = kv * p.group + (hz - kv * p.zgroups) * p.zheads + h;
    const float vs = kFp8 && p.v_scale != nullptr ? p.v_scale[kv] : 1.0f;
    const float f = sum == 0.0f ? 0.0f : vs / sum;
    uint2 w;
    w.x = pack_bf16(v.x * f, v.y * f);
    w.y = pack_bf16(v.z * f, v.w * f);
    *reinterpret_cast<uint2*>(p.out + b * p.ldo + static_cast<int64_t>(head) * D + d) = w;
    if (d == 0 && p.lse != nullptr)
      p.lse[static_cast<int64_t>(b) * p.heads + head] = sum == 0.0f ? -kInf : (top + log2f(sum)) * 0.69314718055994530942f;
  };
  int segments = 0;
  bool last = false;
  while (!last) {
    const int kvh = cur.hz / p.zgroups, z = cur.hz - kvh * p.zgroups;
    const int head0 = kvh * p.group + z * p.zheads;
    const int nheads = min(p.zheads, p.group - z * p.zheads);
    if (fresh) {
      fresh = false;
      if (!kAheadQ && cur.pos != first_pos) load_q(cur, qn);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (!kFp8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            qf[nt][ks][0] = qn[nt][ks][0];
            qf[nt][ks][1] = qn[nt][ks][1];
          }
          mult[nt][0] = mult[nt][1] = p.scale_log2;
        } else {
          float amax = 0.0f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            amax = fmaxf(amax, fmaxf(fabsf(bf_lo(qn[nt][ks][0])), fabsf(bf_hi(qn[nt][ks][0]))));
            amax = fmaxf(amax, fmaxf(fabsf(bf_lo(qn[nt][ks][1])), fabsf(bf_hi(qn[nt][ks][1]))));
          }
          amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
          // amax in [2^e, 2^(e+1)) goes to [2^14, 2^15); beside an infinite
          // element the finite ones are scaled as if of its size, and stay
          // finite.  Both factors are normal numbers.
          const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -112), 127);
          const float down = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
          const float up = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            qf[nt][ks][0] = pack_f16(bf_lo(qn[nt][ks][0]) * down, bf_hi(qn[nt][ks][0]) * down);
            qf[nt][ks][1] = pack_f16(bf_lo(qn[nt][ks][1]) * down, bf_hi(qn[nt][ks][1]) * down);
          }
          const float f = p.scale_log2 * (p.k_scale != nullptr ? p.k_scale[kvh] : 1.0f) * up;
          mult[nt][0] = __shfl_sync(~0u, f, 8 * t4);      // head 2 t4
          mult[nt][1] = __shfl_sync(~0u, f, 8 * t4 + 4);  // head 2 t4 + 1
        }
        m[nt][0] = m[nt][1] = -kInf;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][ks][i] = 0.0f;
      }
    }
    const bool last_tile = cur.tile + 1 == cur.tiles;
    Cursor next = cur;
    advance<S, kWindow>(p, next);
    last = next.b >= p.num_seqs || next.pos >= end;
    if (kAheadQ && last_tile && !last) load_q(next, qn);
    // Refill the stage the previous step emptied, then wait for this one.
    {
      const int fill = stage == 0 ? S::kStages - 1 : stage - 1;
      if (to_load) {
        issue(fill, off);
        advance<S, kWindow>(p, ahead);
        to_load = ahead.b < p.num_seqs && ahead.pos < end;
        if (to_load) off = lookup(ahead);
      }
      cp_async_commit();
      cp_async_wait_group<S::kStages - 1>();
      __syncwarp();
    }
    const uint32_t k_a = ring + stage * S::kStage, v_a = k_a + S::kKeys * S::kRow;

    // scores: keys x heads
    float x[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nt][mt][i] = 0.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int c2 = 0; c2 < S::kChunks / 2; ++c2) {
        uint32_t r[4];
        ldsm4(k_a + at_chunk<S::kRow>(mt * 16 + (lane & 15), 2 * c2 + (lane >> 4)), r);
        if (!kFp8) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<false>(x[nt][mt], r, qf[nt][c2][0], qf[nt][c2][1]);
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t a[4];
            e4m3x4_to_f16(r[2 * half], a[0], a[2]);
            e4m3x4_to_f16(r[2 * half + 1], a[1], a[3]);
            const int ks = (2 * c2 + half) % KS;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<true>(x[nt][mt], a, qf[nt][ks][0], qf[nt][ks][1]);
          }
        }
      }
    }
    const int64_t key0 = static_cast<int64_t>(cur.tile) * S::kTile + warp * S::kKeys;
    const int keys_left = static_cast<int>(cur.len - key0 < S::kKeys ? cur.len - key0 : S::kKeys);  // may be <= 0
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2] = {-kInf, -kInf};
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = x[nt][mt][i] * mult[nt][i & 1];
          if (mt * 16 + g8 + (i >> 1) * 8 >= keys_left) v = -kInf;
          x[nt][mt][i] = v;
          top[i & 1] = fmaxf(top[i & 1], v);
        }
      // (the difference is exact where it matters; the sum would be rounded up to let
      // weights of an E4M3 cache reach 2^16, infinity in fp16, at scores of 2^27)
      grow |= top[0] - m[nt][0] > kBelow<kFp8> + kSlack || top[1] - m[nt][1] > kBelow<kFp8> + kSlack;
    }
    if (__any_sync(~0u, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = -kInf;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) top = fmaxf(top, fmaxf(x[nt][mt][c], x[nt][mt][c + 2]));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
          top = fmaxf(m[nt][c], top - kBelow<kFp8>);
          const float f = m[nt][c] == -kInf ? 1.0f : ex2(m[nt][c] - top);  // no sum yet (or NaN, kept) at -inf
          m[nt][c] = top;
          l[nt][c] *= f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            o[nt][ks][c] *= f;
            o[nt][ks][c + 2] *= f;
          }
        }
    }
    // probabilities as the 8-column operand: heads x keys after the transpose
    uint32_t ph[NT][MT][2], pl[NT][MT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] == -kInf ? 0.0f : m[nt][0], m1 = m[nt][1] == -kInf ? 0.0f : m[nt][1];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float a = ex2(x[nt][mt][2 * r] - m0), b = ex2(x[nt][mt][2 * r + 1] - m1);
          l[nt][0] += a;
          l[nt][1] += b;
          if (kFp8) {
            ph[nt][mt][r] = transpose8(pack_f16(a, b));
          } else {
            const uint32_t hi = pack_bf16(a, b);
            ph[nt][mt][r] = transpose8(hi);
            pl[nt][mt][r] = transpose8(pack_bf16(a - bf_lo(hi), b - bf_hi(hi)));
          }
        }
    }
    // o (elements x heads) += V^T (elements x keys) P^T (keys x heads)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int c2 = 0; c2 < S::kChunks / 2; ++c2) {
        uint32_t r[4];
        if (!kFp8) {
          ldsm4_t(v_a + at_chunk<S::kRow>(mt * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * c2 + ((lane >> 3) & 1)), r);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<false>(o[nt][c2], r, ph[nt][mt][0], ph[nt][mt][1]);
            mma16816<false>(o[nt][c2], r, pl[nt][mt][0], pl[nt][mt][1]);
          }
        } else {
          // A 16-bit unit holds elements 2j, 2j+1 of one key: unzip the pair of
          // keys into one word per element (rows j and j + 8 of the tile).
          ldsm4_t(v_a + at_chunk<S::kRow>(mt * 16 + (lane & 15), 2 * c2 + (lane >> 4)), r);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t a[4];
            e4m3x4_to_f16(__byte_perm(r[2 * half], 0, 0x3120), a[0], a[1]);
            e4m3x4_to_f16(__byte_perm(r[2 * half + 1], 0, 0x3120), a[2], a[3]);
            const int ks = (2 * c2 + half) % KS;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<true>(o[nt][ks], a, ph[nt][mt][0], ph[nt][mt][1]);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage before it is refilled
    stage = stage + 1 == S::kStages ? 0 : stage + 1;

    // ---- end of a (sequence, head) or of the stretch -------------------------
    // The warps leave their (m, l, o) in shared memory and go on; one of them,
    // another each time, waits for the others' and joins them.
    if (last_tile || last) {
      if (segments > 0 && warp != ((segments - 1) & (kWarps - 1))) bar_sync(join_free(segments));  // its last joiner has read it
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float s = l[nt][c];
          s += __shfl_xor_sync(~0u, s, 4);
          s += __shfl_xor_sync(~0u, s, 8);
          s += __shfl_xor_sync(~0u, s, 16);
          const int h = nt * 8 + 2 * t4 + c;
          if (g8 == 0) {
            ml[warp][h][0] = m[nt][c];
            ml[warp][h][1] = s;
          }
          float* dst = o_join + (warp * NT * 8 + h) * S::kOStride;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            dst[ks * 16 + (kFp8 ? 2 * g8 : g8)] = o[nt][ks][c];
            dst[ks * 16 + (kFp8 ? 2 * g8 + 1 : g8 + 8)] = o[nt][ks][c + 2];
          }
        }
      __syncwarp();
      if (warp != (segments & (kWarps - 1))) {
        bar_arrive(join_full(segments));
      } else {
        bar_sync(join_full(segments));
        const long long seg_begin = cur.pos - static_cast<long long>(cur.tile) * S::kTileCost;  // its first tile
        const bool whole = seg_begin >= begin && last_tile;
        const int slot_index = seg_begin < begin ? 0 : 1;
        float* slot = p.part + (2 * static_cast<int64_t>(blockIdx.x) + slot_index) * kSlot;
        for (int i = lane; i < nheads * (D / 4); i += 32) {
          const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
          float top = -kInf;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][h][0]);
          float sum = 0.0f;
          float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = weight_of(ml[w][h][0], top);
            const float4 v = *reinterpret_cast<const float4*>(o_join + (w * NT * 8 + h) * S::kOStride + d);
            sum += f * ml[w][h][1];
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
          }
          if (whole) {
            finish(cur.b, cur.hz, h, d, top, sum, acc);
          } else {
            __stcg(reinterpret_cast<float4*>(slot + h * D + d), acc);
            if (d == 0) __stcg(reinterpret_cast<float2*>(slot + NT * 8 * D + 2 * h), make_float2(top, sum));
          }
        }
        __syncwarp();
        if (!last) bar_arrive(join_free(segments + 1));
        if (!whole && lane == 0) {
          // The CTAs that hold tiles of this segment; the last of them to come
          // here adds their partials when its own tiles are done.
          const int c0 = owner(seg_begin), c1 = owner(seg_begin + static_cast<long long>(cur.tiles - 1) * S::kTileCost);
          const int parts = c1 - c0 + 1;
          const int lead = parts <= kDirect ? 0 : (static_cast<int>(blockIdx.x) - c0) / kGroup * kGroup;
          const int group = parts <= kDirect ? parts : min(kGroup, parts - lead);
          unsigned* counter = parts <= kDirect ? p.counters + static_cast<int64_t>(cur.b) * hz_all + cur.hz
                                               : p.group_counters + 2 * (c0 + lead) + (lead == 0 ? 1 : 0);
          // Release of this warp's partial, acquire of the others'.
          if (atomic_add_acq_rel(counter, 1u) == static_cast<unsigned>(group - 1)) {
            *counter = 0;  // ready for the next call
            pending[slot_index] = make_int4(cur.b, cur.hz, c0 + lead, parts <= kDirect ? parts : group | lead << 8 | parts << 18);
          }
        }
        __syncwarp();
      }
      ++segments;
      fresh = true;
    }
    cur = next;
  }
  cp_async_wait_group<0>();

  // ---- segments (or groups of their CTAs) whose last partial this CTA brought --
  // A partial's slot is 1 in the CTA that began the segment and 0 in the others,
  // which came to it from before.  Kept short: this code runs once, and its
  // fetch is part of its time.
  __syncthreads();
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int4 job = pending[s];
    if (job.w == 0) continue;
    // .w: the number of partials, or group | lead << 8 | parts << 18
    const bool grouped = job.w > kDirect;
    const int parts = job.w >> 18, lead = (job.w >> 8) & 1023;
    int first_cta = job.z, first_slot = grouped && lead > 0 ? 0 : 1, count = grouped ? job.w & 255 : job.w, stride = 1;
    bool sums_of_groups = false;  // the second level
    const int part0 = job.y % p.zgroups, nheads = min(p.zheads, p.group - part0 * p.zheads);
#pragma unroll 1
    for (;;) {
      float* first = p.part + (2 * static_cast<int64_t>(first_cta) + first_slot) * kSlot;
      const int ml_at = NT * 8 * (sums_of_groups ? D + 2 : D);
      const bool last_level = !grouped || sums_of_groups;
#pragma unroll 1
      for (int i = tid; i < nheads * (D / 4); i += kThreads) {
        const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
        float top = -kInf, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        constexpr int kBatch = 16;  // partials in flight
#pragma unroll 1
        for (int c0 = 0; c0 < count; c0 += kBatch) {
          float2 e[kBatch];
          float4 v[kBatch];
          float up = top;
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            const int c = c0 + q;
            const float* slot = first + (c == 0 ? 0 : 2 * c * stride - first_slot) * kSlot;
            e[q] = make_float2(-kInf, 0.0f);
            v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c < count) {
              e[q] = __ldcg(reinterpret_cast<const float2*>(slot + ml_at + 2 * h));
              v[q] = __ldcg(reinterpret_cast<const float4*>(slot + h * D + d));
            }
          }
#pragma unroll
          for (int q = 0; q < kBatch; ++q) up = fmaxf(up, e[q].x);
          const float f0 = weight_of(top, up);
          top = up;
          sum *= f0;
          acc.x *= f0;
          acc.y *= f0;
          acc.z *= f0;
          acc.w *= f0;
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            const float f = weight_of(e[q].x, top);
            sum += f * e[q].y;
            acc.x += f * v[q].x;
            acc.y += f * v[q].y;
            acc.z += f * v[q].z;
            acc.w += f * v[q].w;
          }
        }
        if (last_level) {
          finish(job.x, job.y, h, d, top, sum, acc);
        } else {
          // into the first partial's slot; its (m, l), which other threads still read, stays
          __stcg(reinterpret_cast<float4*>(first + h * D + d), acc);
          if (d == 0) __stcg(reinterpret_cast<float2*>(first + NT * 8 * (D + 2) + 2 * h), make_float2(top, sum));
        }
      }
      if (last_level) break;
      // The group's sum is there; the last group of the segment goes on to join them.
      __syncthreads();
      if (tid == 0) {
        const int groups = (parts + kGroup - 1) / kGroup;
        unsigned* counter = p.counters + static_cast<int64_t>(job.x) * hz_all + job.y;
        const bool mine = atomic_add_acq_rel(counter, 1u) == static_cast<unsigned>(groups - 1);
        if (mine) *counter = 0;
        found[0] = mine;
      }
      __syncthreads();
      if (!found[0]) break;
      first_cta = job.z - lead;
      first_slot = 1;
      count = (parts + kGroup - 1) / kGroup;
      stride = kGroup;
      sums_of_groups = true;
    }
    __syncthreads();  // found is free
  }
}

template <int D, bool kFp8, int NT, bool kWindow>
qerl_status launch(const DecodeParams& p, int sms, int dev, cudaStream_t s) {
  using S = Shape<D, kFp8, NT>;
  static std::atomic<uint64_t> ready{0};  // one bit per device: the attribute belongs to the device's function
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if ((ready.load() & bit) == 0) {
    if (cudaFuncSetAttribute(decode_kernel<D, kFp8, NT, kWindow>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem) != cudaSuccess)
      return QERL_ERR_CUDA;
    ready.fetch_or(bit);
  }
  constexpr int kFit = static_cast<int>(kPartBytes / (2 * NT * 8 * S::kPartRow * sizeof(float)));
  int64_t grid = std::min({S::kCtas * sms, kFit, kMaxCtas});
  const int64_t rows = kWindow ? std::min<int64_t>(p.capacity, p.seen) : p.capacity;
  const int64_t most = static_cast<int64_t>(p.num_seqs) * p.kv_heads * p.zgroups * ((rows + S::kTile - 1) / S::kTile);
  if (most < grid) grid = most > 0 ? most : 1;
  return cuda_status(
      launch_dependent(decode_kernel<D, kFp8, NT, kWindow>, dim3(static_cast<unsigned>(grid)), kThreads, S::kSmem, s, p));
}

template <bool kWindow>
qerl_status launch_for(const DecodeParams& p, int head_dim, bool f8, bool one, int sms, int dev, cudaStream_t s) {
  if (head_dim == 128) {
    if (f8) return one ? launch<128, true, 1, kWindow>(p, sms, dev, s) : launch<128, true, 2, kWindow>(p, sms, dev, s);
    return one ? launch<128, false, 1, kWindow>(p, sms, dev, s) : launch<128, false, 2, kWindow>(p, sms, dev, s);
  }
  if (f8) return one ? launch<64, true, 1, kWindow>(p, sms, dev, s) : launch<64, true, 2, kWindow>(p, sms, dev, s);
  return one ? launch<64, false, 1, kWindow>(p, sms, dev, s) : launch<64, false, 2, kWindow>(p, sms, dev, s);
}

struct Split {
  int zgroups, zheads, tiles;
};
// A key-value head's query heads: up to 8 in one column tile, up to 16 in two;
// more are cut into equal parts that read the cache once each.
Split split_heads(int group) {
  Split s;
  s.zgroups = (group + 15) / 16;
  s.zheads = (group + s.zgroups - 1) / s.zgroups;
  s.zgroups = (group + s.zheads - 1) / s.zheads;
  s.tiles = s.zheads > 8 ? 2 : 1;
  return s;
}

size_t counter_bytes(int64_t num_seqs, int num_kv_heads, const Split& s) {
  return align_up(static_cast<size_t>(num_seqs) * num_kv_heads * s.zgroups * sizeof(unsigned), 256);
}

}  // namespace

size_t decode_attention_workspace_bytes(int64_t num_seqs, int num_heads, int num_kv_heads) {
  const Split s = split_heads(num_heads / num_kv_heads);
  return kWsHeaderBytes + kPartBytes + kGroupBytes + counter_bytes(num_seqs, num_kv_heads, s);
}

qerl_status launch_decode_attention(const DecodeAttentionArgs& a, cudaStream_t s) {
  const qerl_kv_cache& c = *a.cache;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QERL_ERR_CUDA;
  const Split sp = split_heads(a.num_heads / c.num_kv_heads);
  DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.ldq = a.ldq;
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
  p.num_seqs = static_cast<int>(c.num_seqs);
  p.heads = a.num_heads;
  p.kv_heads = c.num_kv_heads;
  p.group = a.num_heads / c.num_kv_heads;
  p.zgroups = sp.zgroups;
  p.zheads = sp.zheads;
  p.lengths = a.lengths;
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ldo = a.ldo;
  p.lse = a.lse;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  p.part = reinterpret_cast<float*>(ws + kWsHeaderBytes);
  p.group_counters = reinterpret_cast<unsigned*>(ws + kWsHeaderBytes + kPartBytes);
  p.counters = p.group_counters + 2 * kMaxCtas;
  const bool f8 = c.dtype == QERL_E4M3;
  const bool one = sp.tiles == 1;
  // A window that no sequence outgrows leaves nothing out.
  p.sinks = a.sinks;
  p.seen = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(a.window) + a.sinks, INT32_MAX));
  if (a.window > 0 && p.seen < p.capacity) return launch_for<true>(p, c.head_dim, f8, one, sms, dev, s);
  return launch_for<false>(p, c.head_dim, f8, one, sms, dev, s);
}

}  // namespace qerl
