// cache_pages.cu -- pages of the key-value cache: forking sequences and
// compacting the pool.
//
// Fork: the child's table row takes the parent's full pages; the rows of the
// parent's last page, if it is not full, are copied to a page of the child's own.
// Compaction: of the pages in use, the i-th (ascending) with a number at or past
// their count L moves into the i-th unused number below L.
//
// Bound: bytes, each copied row once in and once out.  Measured: 384 children of 48
// parents (53 MB) 12.4 us = 0.63 of the copy rate; 1336 pages of 256 KB moved
// (700 MB) 125 us = 0.82, of which the marks and numbers take some 15 us; a million
// pages of 1 KB in use of two 1.73 ms, where the bytes take 0.30: one block numbers
// the pool.
#include "qerl_internal.h"
#include "qerl_ptx.cuh"

#include <algorithm>

namespace qerl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpPiece = 4096;  // bytes that a warp copies at a time: 8 loads of 16 bytes a lane in flight

// `bytes` (a multiple of 16, at most kWarpPiece) from one place to another, by a warp.
__device__ __forceinline__ void warp_copy(const uint8_t* src, uint8_t* dst, int bytes) {
  const int lane = threadIdx.x & 31;
  uint4 v[kWarpPiece / 512];
#pragma unroll
  for (int i = 0; i < kWarpPiece / 512; ++i)
    if ((i * 32 + lane) * 16 < bytes) v[i] = *reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16);
#pragma unroll
  for (int i = 0; i < kWarpPiece / 512; ++i)
    if ((i * 32 + lane) * 16 < bytes) *reinterpret_cast<uint4*>(dst + (i * 32 + lane) * 16) = v[i];
}

struct PoolParams {
  uint8_t *k, *v;
  int row_bytes, kv_heads, page_size;
  int64_t num_pages;
  int* table;
  int64_t ld_table, num_seqs, max_pages;
  int* status;
};

struct ForkParams {
  PoolParams pool;
  const int *parents, *children, *lengths, *new_pages;
};

constexpr int kForkCtas = 4;  // per SM

// Block (x, y): child x's piece y of the (k or v, head, part of its rows) to copy;
// the blocks of y == 0 also write the child's table row.
__global__ void __launch_bounds__(kThreads, kForkCtas) fork_kernel(const ForkParams p) {
  griddep_wait();
  const PoolParams& c = p.pool;
  const int64_t i = blockIdx.x;
  const int parent = p.parents[i], child = p.children[i], length = p.lengths[i], fresh = p.new_pages[i];
  bool bad = parent < 0 || parent >= c.num_seqs || child < 0 || child >= c.num_seqs || parent == child || length < 0 ||
             length > c.max_pages * c.page_size;
  const int full = bad ? 0 : length / c.page_size, rest = bad ? 0 : length - full * c.page_size;
  const int* from = c.table + parent * c.ld_table;
  int last = 0;
  if (rest > 0) {
    last = from[full];
    bad = last < 0 || last >= c.num_pages || fresh < 0 || fresh >= c.num_pages;
  }
  // Every block looks through the full pages' entries, as nothing of a bad item is
  // written (a negative one is a page given up, and passed on).
  for (int j = threadIdx.x; j < full; j += kThreads) bad |= from[j] >= c.num_pages;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(c.status, QERL_ERR_RANGE);
    return;
  }
  if (blockIdx.y == 0) {
    int* to = c.table + child * c.ld_table;
    for (int j = threadIdx.x; j < full; j += kThreads) to[j] = from[j];
    if (rest > 0 && threadIdx.x == 0) to[full] = fresh;
  }
  // The rows of one head lie side by side: rest * row_bytes bytes, in pieces for a warp each.
  const int64_t bytes = static_cast<int64_t>(rest) * c.row_bytes;
  const int pieces = static_cast<int>((bytes + kWarpPiece - 1) / kWarpPiece);
  const int64_t units = 2ll * c.kv_heads * pieces;
  const int64_t head_bytes = static_cast<int64_t>(c.page_size) * c.row_bytes;
  for (int64_t u = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += gridDim.y * (kThreads / 32)) {
    const int head = static_cast<int>(u / pieces);
    const int64_t at = static_cast<int64_t>(u - static_cast<int64_t>(head) * pieces) * kWarpPiece;
    uint8_t* pages = head < c.kv_heads ? c.k : c.v;
    const int h = head < c.kv_heads ? head : head - c.kv_heads;
    warp_copy(pages + (static_cast<int64_t>(last) * c.kv_heads + h) * head_bytes + at,
              pages + (static_cast<int64_t>(fresh) * c.kv_heads + h) * head_bytes + at,
              static_cast<int>(min(bytes - at, static_cast<int64_t>(kWarpPiece))));
  }
}

struct CompactParams {
  PoolParams pool;
  const int* lengths;
  int* new_table;
  int64_t ld_new;
  int* live_pages;
  uint8_t* used;   // [num_pages]: 1 where a sequence holds the page; zero at the call's start
  int* number;     // [num_pages]: the new number of a page in use
  int *from, *to;  // [num_pages / 2]: the moves
  int* moves;      // their count
};

// Entries of sequence s that hold pages.
__device__ __forceinline__ int64_t held(const CompactParams& p, int64_t s, bool record) {
  const int64_t n = p.lengths[s], most = p.pool.max_pages * p.pool.page_size;
  if (record && (n < 0 || n > most)) record_error(p.pool.status, QERL_ERR_RANGE);
  return n < 0 ? 0 : (min(n, most) + p.pool.page_size - 1) / p.pool.page_size;
}

constexpr int kEntries = 1024;  // table entries of a row that a block takes at a time

__global__ void __launch_bounds__(kThreads) mark_kernel(const CompactParams p) {
  griddep_wait();
  const PoolParams& c = p.pool;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kEntries;
  for (int64_t s = blockIdx.y; s < c.num_seqs; s += gridDim.y) {
    const int64_t end = min(held(p, s, first == 0 && threadIdx.x == 0), first + kEntries);
    for (int64_t j = first + threadIdx.x; j < end; j += kThreads) {
      const int page = c.table[s * c.ld_table + j];
      if (page >= c.num_pages) record_error(c.status, QERL_ERR_RANGE);
      if (page >= 0 && page < c.num_pages) p.used[page] = 1;
    }
  }
}

constexpr int kScanThreads = 1024;

// Sum over the block of `mine` before this thread, and of all.
__device__ __forceinline__ int block_before(int mine, int* warps, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int up = __shfl_up_sync(~0u, incl, i);
    if (lane >= i) incl += up;
  }
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int w = lane < kScanThreads / 32 ? warps[lane] : 0;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int up = __shfl_up_sync(~0u, w, i);
    if (lane >= i) w += up;
  }
  all = __shfl_sync(~0u, w, 31);
  const int before = __shfl_sync(~0u, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return incl - mine + (warp > 0 ? before : 0);
}

// The block that numbers the pages of a small table also marks them: 114 entries
// 9.1 us, with the launches for it 14.5 us; 12288 entries 130.5 us, with them 125.4.
constexpr int64_t kMarkEntries = 4096, kMarkPages = 131072;

// New numbers and the list of moves, by one block: thread t takes the t-th part
// of the pool, in words of 16 pages.
template <bool kMark>
__global__ void __launch_bounds__(kScanThreads) number_kernel(const CompactParams p) {
  __shared__ int warps[kScanThreads / 32];
  griddep_wait();
  const int64_t n = p.pool.num_pages, words = (n + 15) / 16;  // the array is padded with zeros to whole words
  if (kMark) {
    const PoolParams& c = p.pool;
    for (int64_t w = threadIdx.x; w < words; w += kScanThreads)
      reinterpret_cast<uint4*>(p.used)[w] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const int width = static_cast<int>(c.max_pages), entries = static_cast<int>(c.num_seqs * c.max_pages);
    if (width == 0)  // no entry's thread looks at the lengths
      for (int s = threadIdx.x; s < c.num_seqs; s += kScanThreads) held(p, s, true);
    for (int e = threadIdx.x; e < entries; e += kScanThreads) {
      const int s = e / width, j = e - s * width;
      const int page = c.table[s * c.ld_table + j];
      if (j >= held(p, s, j == 0)) continue;
      if (page >= c.num_pages) record_error(c.status, QERL_ERR_RANGE);
      if (page >= 0 && page < c.num_pages) p.used[page] = 1;
    }
    __syncthreads();
  }
  const int64_t each = (words + kScanThreads - 1) / kScanThreads;
  const int64_t w0 = min(threadIdx.x * each, words), w1 = min(w0 + each, words);
  const uint4* used = reinterpret_cast<const uint4*>(p.used);
  auto count = [](const uint4& v) { return __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w); };
  int mine = 0;
#pragma unroll 4
  for (int64_t w = w0; w < w1; ++w) mine += count(used[w]);
  int live;
  int before = block_before(mine, warps, live);  // pages in use before this thread's
  // A page in use with number q has `before` pages in use before it; an unused
  // one below the count of those in use, q - before unused ones.
  int low = 0;  // of this thread's pages in use, those that stay
  for (int64_t w = w0; w < w1; ++w) {
    const uint4 v = used[w];
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
      const int64_t q = w * 16 + e;
      if (q >= n) break;
      if (x[e >> 2] >> (8 * (e & 3)) & 1) {
        if (q < live) {
          p.number[q] = static_cast<int>(q);
          ++low;
        }
        ++before;
      } else if (q < live) {
        p.to[q - before] = static_cast<int>(q);
      }
    }
  }
  int stay;
  block_before(low, warps, stay);
  const int moves = live - stay;
  // (its barriers also made p.to visible to the whole block)
  before -= mine;
  for (int64_t w = w0; w < w1; ++w) {
    if (w * 16 + 15 < live) {
      before += count(used[w]);
      continue;
    }
    const uint4 v = used[w];
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
      const int64_t q = w * 16 + e;
      if ((x[e >> 2] >> (8 * (e & 3)) & 1) == 0) continue;
      if (q >= live) {
        const int i = before - stay;
        p.from[i] = static_cast<int>(q);
        p.number[q] = p.to[i];
      }
      ++before;
    }
  }
  if (threadIdx.x == 0) {
    *p.moves = moves;
    *p.live_pages = live;
  }
}

// The new table, and the pages that move.  No page is both read and written: the
// moved ones lie past the count of those in use, their new places below it.
__global__ void __launch_bounds__(kThreads, 4) move_kernel(const CompactParams p) {
  griddep_wait();
  const PoolParams& c = p.pool;
  const int64_t chunks = (c.max_pages + kEntries - 1) / kEntries;
  for (int64_t b = blockIdx.x; b < c.num_seqs * chunks; b += gridDim.x) {
    const int64_t s = b / chunks, first = (b - s * chunks) * kEntries;
    const int64_t end = held(p, s, false), last = min(first + kEntries, c.max_pages);
    for (int64_t j = first + threadIdx.x; j < last; j += kThreads) {
      const int page = c.table[s * c.ld_table + j];
      p.new_table[s * p.ld_new + j] = j < end && page >= 0 && page < c.num_pages ? p.number[page] : page;
    }
  }
  const int64_t page_bytes = static_cast<int64_t>(c.kv_heads) * c.page_size * c.row_bytes;
  const int64_t pieces = (page_bytes + kWarpPiece - 1) / kWarpPiece;
  const int64_t units = 2 * pieces * *p.moves;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t page = u / pieces, at = (u - page * pieces) * kWarpPiece;
    uint8_t* pages = page & 1 ? c.v : c.k;
    warp_copy(pages + p.from[page >> 1] * page_bytes + at, pages + p.to[page >> 1] * page_bytes + at,
              static_cast<int>(min(page_bytes - at, static_cast<int64_t>(kWarpPiece))));
  }
}

PoolParams pool_of(const qerl_kv_cache& c, int* status) {
  PoolParams p{};
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.row_bytes = c.head_dim * (c.dtype == QERL_E4M3 ? 1 : 2);
  p.kv_heads = c.num_kv_heads;
  p.page_size = c.page_size;
  p.num_pages = c.num_pages;
  p.table = const_cast<int*>(c.page_table);
  p.ld_table = c.ld_table;
  p.num_seqs = c.num_seqs;
  p.max_pages = c.max_pages;
  p.status = status;
  return p;
}

// The workspace of a compaction, behind its header.
struct CompactLayout {
  size_t used, number, from, to, moves, bytes;
};
CompactLayout compact_layout(int64_t num_pages) {
  const size_t n = static_cast<size_t>(num_pages);
  CompactLayout l{};
  l.used = kWsHeaderBytes;
  l.number = l.used + align_up(n, 256);
  l.from = l.number + align_up(4 * n, 256);
  l.to = l.from + align_up(2 * n + 4, 256);
  l.moves = l.to + align_up(2 * n + 4, 256);
  l.bytes = l.moves + 256;
  return l;
}

}  // namespace

qerl_status launch_kv_fork(const KvForkArgs& a, cudaStream_t s) {
  ForkParams p{};
  p.pool = pool_of(*a.cache, a.status);
  p.parents = a.parents;
  p.children = a.children;
  p.lengths = a.lengths;
  p.new_pages = a.new_pages;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QERL_ERR_CUDA;
  // Blocks per child: for a whole page 8 pieces at a time, but no more than twice
  // what is resident together, as each looks its child up first (384 children of
  // up to 64 rows, 8 heads of 128: 11.9 us, as many as are resident 16.5 us,
  // without a limit 12.9 us; 12.4 us since every block also looks through the
  // full pages' numbers).
  const int64_t pieces = 2ll * p.pool.kv_heads *
                         ((static_cast<int64_t>(p.pool.page_size) * p.pool.row_bytes + kWarpPiece - 1) / kWarpPiece);
  const int64_t whole = (pieces + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t y = std::max<int64_t>(1, std::min({whole, int64_t{64}, 2 * kForkCtas * static_cast<int64_t>(sms) / a.count}));
  return cuda_status(launch_dependent(fork_kernel, dim3(static_cast<unsigned>(a.count), static_cast<unsigned>(y)),
                                      kThreads, 0, s, p));
}

size_t kv_compact_workspace_bytes(int64_t num_pages) { return compact_layout(num_pages).bytes; }

qerl_status launch_kv_compact(const KvCompactArgs& a, cudaStream_t s) {
  const qerl_kv_cache& c = *a.cache;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const CompactLayout l = compact_layout(c.num_pages);
  CompactParams p{};
  p.pool = pool_of(c, &reinterpret_cast<WsHeader*>(ws)->status);
  p.lengths = a.lengths;
  p.new_table = a.new_table;
  p.ld_new = a.ld_new;
  p.live_pages = a.live_pages;
  p.used = ws + l.used;
  p.number = reinterpret_cast<int*>(ws + l.number);
  p.from = reinterpret_cast<int*>(ws + l.from);
  p.to = reinterpret_cast<int*>(ws + l.to);
  p.moves = reinterpret_cast<int*>(ws + l.moves);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QERL_ERR_CUDA;
  const int64_t chunks = (c.max_pages + kEntries - 1) / kEntries;
  if (c.num_seqs * c.max_pages <= kMarkEntries && c.num_pages <= kMarkPages) {
    if (launch_dependent(number_kernel<true>, dim3(1), kScanThreads, 0, s, p) != cudaSuccess) return QERL_ERR_CUDA;
  } else {
    if (cudaMemsetAsync(p.used, 0, l.number - l.used, s) != cudaSuccess) return QERL_ERR_CUDA;
    if (c.num_seqs > 0) {  // without entries or pages too: lengths and numbers outside are recorded there
      const dim3 grid(static_cast<unsigned>(std::max<int64_t>(chunks, 1)),
                      static_cast<unsigned>(std::min<int64_t>(c.num_seqs, 65535)));
      if (launch_dependent(mark_kernel, grid, kThreads, 0, s, p) != cudaSuccess) return QERL_ERR_CUDA;
    }
    if (launch_dependent(number_kernel<false>, dim3(1), kScanThreads, 0, s, p) != cudaSuccess) return QERL_ERR_CUDA;
  }
  return cuda_status(launch_dependent(move_kernel, dim3(static_cast<unsigned>(4 * sms)), kThreads, 0, s, p));
}

}  // namespace qerl
