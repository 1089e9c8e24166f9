// kv_cache.cu -- rotary position embedding of q and k with the append of k and
// v to the paged cache, in one pass over the rows the q/k/v linears produced.
//
// Token t of sequence s at position p, pair i of a head (half = rot_dim / 2):
//   theta = p * inv_freq[i]
//   (x[i], x[i + half]) -> (x[i] cos - x[i + half] sin, x[i + half] cos + x[i] sin)
// in fp32 with one rounding to bf16 (and, for the cache, one rounding of the
// fp32 value to the cache's type: the 8-bit cache holds sat(value * (1 / scale)),
// the reciprocal taken once in fp32).
//
// Bound: bytes.  Every q, k, v element is read once and written once or twice.
// A CTA takes one token at a time (grid-stride); a thread takes the same item of
// every token, two 16-byte chunks of one head: the two halves of 8 pairs, or 2
// chunks that are only copied, so its addresses are worked out once.  What a
// token needs is on its way during the token before: a thread copies its own
// item to shared memory (cp.async), the angles go to the other of two buffers,
// the page number and the position it depends on follow one and two tokens
// ahead.  Measured on 10517 tokens of 28 + 2 x 4 heads of 128 (205 MB, 30 us at
// the copy rate): page after position after token 68 us, fetched ahead 58 us,
// rows through shared memory at 5 CTAs per SM 42 us, the angles a token ahead
// 37 us (5.5 TB/s).  An E4M3 cache: 9132 tokens of 40 + 2 x 8 heads (262 MB,
// 38.5 us) 56 us; with fewer threads and the same two stages less is in flight,
// and warps wait for loads in a third of their cycles.
#include "qerl_internal.h"
#include "qerl_ptx.cuh"

#include <algorithm>
#include <atomic>
#include <cuda_bf16.h>

namespace qerl {
namespace {

constexpr int kMaxHalf = 64;  // rot_dim / 2
constexpr int kStages = 2;
// Threads per SM that the launch bounds leave room for.  The E4M3 conversions
// need the registers of two thirds (9132 tokens of 40 + 2 x 8 heads: 56 us, with
// 1536 threads 60 us); without them more threads win (10517 tokens of 28 + 2 x 4
// heads: 37 us against 39).
template <bool kE4m3>
constexpr int kThreadsPerSm = kE4m3 ? 1024 : 1536;

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t ldq, ldk, ldv;
  __nv_bfloat16 *q_out, *k_out;
  int64_t ldqo, ldko;
  int64_t tokens;
  int heads, kv_heads, dim, half;
  const int *seq_ids, *positions;
  const double* inv_freq;
  bool has_cache;  // false: rotation only
  uint8_t *k_pages, *v_pages;  // null for a cache of no pages
  const float *k_scale, *v_scale;
  const int* table;
  int64_t num_seqs, ld_table, num_pages, max_pages;
  int page_size;
  int* status;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two fp32 values times `inverse` -> E4M3 (nearest even, saturating, NaN kept), in the low 16 bits.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi, float inverse) {
  const float a = lo * inverse, b = hi * inverse;
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(h)
      : "f"(b), "f"(a));
  return h;
}

template <bool kE4m3>
__global__ void __launch_bounds__(512, kThreadsPerSm<kE4m3> / 512) rope_append_kernel(const AppendParams p) {
  extern __shared__ __align__(16) uint4 ring[];  // [stage][chunk][thread]
  __shared__ __align__(16) float cs[2][kMaxHalf], sn[2][kMaxHalf];
  const int tid = threadIdx.x;
  // Turns per position as a 64-bit binary fraction: the product with the
  // position keeps exactly the bits below one turn, so far positions lose
  // nothing (an fp32 angle would be off by 1e-3 rad at position 1e4).
  uint64_t turn = 0;
  griddep_wait();
  if (tid < p.half) {
    const double t = p.inv_freq[tid] * 0.15915494309189533577;  // 1 / (2 pi)
    turn = static_cast<uint64_t>(__double2ull_rn((t - floor(t)) * 18446744073709551616.0));
  }
  // This thread's item: kind 0 q, 1 k, 2 v; e0, e1 the chunks' element offsets
  // within the head.
  const int per_head = p.dim >> 4;  // items of a head
  const int items = (p.heads + 2 * p.kv_heads) * per_head;
  const int item = static_cast<int>(blockIdx.y * blockDim.x) + tid;
  int head = item / per_head;
  const int sub = item - head * per_head, rot_items = p.half >> 3;
  const int kind = head < p.heads ? 0 : head < p.heads + p.kv_heads ? 1 : 2;
  head -= kind == 0 ? 0 : kind == 1 ? p.heads : p.heads + p.kv_heads;
  const bool rot = kind < 2 && sub < rot_items;
  const int e0 = rot ? sub * 8 : kind == 2 ? sub * 16 : 2 * p.half + (sub - rot_items) * 16;
  const int e1 = rot ? p.half + sub * 8 : e0 + 8;
  const bool active = item < items && (kind < 2 || p.has_cache);
  const int64_t step = gridDim.x;
  const __nv_bfloat16* src = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + head * p.dim;
  const int64_t ld = kind == 0 ? p.ldq : kind == 1 ? p.ldk : p.ldv;
  __nv_bfloat16* dst = kind == 0 ? p.q_out : kind == 1 ? p.k_out : nullptr;
  const int64_t ldd = kind == 0 ? p.ldqo : p.ldko;
  if (dst != nullptr) dst += head * p.dim + blockIdx.x * ldd;
  uint8_t* pages = kind == 1 ? p.k_pages : kind == 2 ? p.v_pages : nullptr;
  // One division a thread: 16 per item and token took longer than the rows
  // (9132 tokens of 40 + 2 x 8 heads: 66 us, so 0.59 of the copy rate).  The
  // reciprocal of a scale near either end of fp32's range leaves it (that of a
  // subnormal scale is infinite, and would make NaN of a zero): such a scale,
  // and then every value, is first moved by 2^64.  That is exact but for values
  // whose quotients saturate or are far below E4M3's smallest.
  float inverse = 1.0f, move = 1.0f;
  if (kE4m3 && active && kind > 0) {
    const float* sc = kind == 1 ? p.k_scale : p.v_scale;
    if (sc != nullptr) {
      const float scale = sc[head];
      move = fabsf(scale) < 0x1p-64f ? 0x1p64f : fabsf(scale) > 0x1p64f ? 0x1p-64f : 1.0f;
      inverse = 1.0f / (scale * move);
    }
  }
  // The place of token t in the cache: its page number, or -1.
  auto page_of = [&](int64_t t, int pos) -> int {
    if (!p.has_cache || pos < 0) return -1;
    const int64_t s = p.seq_ids != nullptr ? p.seq_ids[t] : t;
    const int pi = pos / p.page_size;
    return s >= 0 && s < p.num_seqs && pi < p.max_pages ? p.table[s * p.ld_table + pi] : -1;
  };
  const uint32_t ring_a = smem_u32(ring) + tid * 16;
  const uint32_t chunk_bytes = blockDim.x * 16;
  int64_t t = blockIdx.x, t_fetch = t;
  src += t * ld;
  auto fetch = [&](int stage) {
    if (active && t_fetch < p.tokens) {
      cp_async_16(ring_a + stage * 2 * chunk_bytes, src + e0, 16);
      cp_async_16(ring_a + (stage * 2 + 1) * chunk_bytes, src + e1, 16);
    }
    cp_async_commit();
    t_fetch += step;
    src += step * ld;
  };
  for (int s = 0; s < kStages - 1; ++s) fetch(s);
  int buf = 0, stage = 0;
  int pos = p.positions[t], pos_next = t + step < p.tokens ? p.positions[t + step] : -1;
  auto angles = [&](int at, int b) {
    if (tid < p.half && at >= 0) {
      const uint64_t a = turn * static_cast<uint64_t>(at);
      // the top 32 bits as a signed fraction of half a turn, in [-1, 1)
      const float x = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578125e-10f;
      sincospif(x, &sn[b][tid], &cs[b][tid]);
    }
  };
  angles(pos, 0);
  int page = page_of(t, pos), page_next = -1, pos_later = -1;
  for (; t < p.tokens; t += step, dst = dst == nullptr ? dst : dst + step * ldd, pos = pos_next, page = page_next, pos_next = pos_later) {
    page_next = t + step < p.tokens ? page_of(t + step, pos_next) : -1;
    pos_later = t + 2 * step < p.tokens ? p.positions[t + 2 * step] : -1;
    cp_async_wait_group<kStages - 2>();
    const uint4 w0 = lds128(ring_a + stage * 2 * chunk_bytes), w1 = lds128(ring_a + (stage * 2 + 1) * chunk_bytes);
    fetch((stage + kStages - 1) & (kStages - 1));  // the stage that this thread read in the step before
    stage = (stage + 1) & (kStages - 1);
    __syncthreads();  // the angles of this token; those of the token before are no longer read
    buf ^= 1;
    angles(pos_next, buf);  // of the next one, so that nobody waits for them
    if (pos < 0) continue;  // padding
    const bool placed = page >= 0 && page < p.num_pages;  // never without pages
    if (tid == 0 && p.has_cache && !placed) record_error(p.status, QERL_ERR_RANGE);
    if (active) {
      uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, b[4] = {w1.x, w1.y, w1.z, w1.w}, c0[2] = {0, 0}, c1[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float xl = bf_lo(a[i]), xh = bf_hi(a[i]), yl = bf_lo(b[i]), yh = bf_hi(b[i]);
        if (rot) {
          const float2 c = reinterpret_cast<const float2*>(&cs[buf ^ 1][e0])[i];
          const float2 s = reinterpret_cast<const float2*>(&sn[buf ^ 1][e0])[i];
          const float rl = xl * c.x - yl * s.x, rh = xh * c.y - yh * s.y;
          yl = yl * c.x + xl * s.x;
          yh = yh * c.y + xh * s.y;
          xl = rl;
          xh = rh;
          a[i] = pack_bf16(xl, xh);
          b[i] = pack_bf16(yl, yh);
        }
        if (kE4m3 && kind > 0) {
          if (move != 1.0f) {
            xl *= move;
            xh *= move;
            yl *= move;
            yh *= move;
          }
          c0[i >> 1] |= pack_e4m3(xl, xh, inverse) << (16 * (i & 1));
          c1[i >> 1] |= pack_e4m3(yl, yh, inverse) << (16 * (i & 1));
        }
      }
      if (dst != nullptr) {
        *reinterpret_cast<uint4*>(dst + e0) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4*>(dst + e1) = make_uint4(b[0], b[1], b[2], b[3]);
      }
      if (pages != nullptr && placed) {
        const int64_t at = ((static_cast<int64_t>(page) * p.kv_heads + head) * p.page_size + pos % p.page_size) * p.dim;
        if (kE4m3) {
          *reinterpret_cast<uint2*>(pages + at + e0) = make_uint2(c0[0], c0[1]);
          *reinterpret_cast<uint2*>(pages + at + e1) = make_uint2(c1[0], c1[1]);
        } else {
          __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(pages) + at;
          *reinterpret_cast<uint4*>(d + e0) = make_uint4(a[0], a[1], a[2], a[3]);
          *reinterpret_cast<uint4*>(d + e1) = make_uint4(b[0], b[1], b[2], b[3]);
        }
      }
    }
  }
  cp_async_wait_group<0>();
}

}  // namespace

qerl_status launch_rope_append(const RopeAppendArgs& a, cudaStream_t s) {
  AppendParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.k_out = static_cast<__nv_bfloat16*>(a.k_out);
  p.ldqo = a.ldqo;
  p.ldko = a.ldko;
  p.tokens = a.tokens;
  p.heads = a.q != nullptr ? a.num_heads : 0;
  p.kv_heads = a.num_kv_heads;
  p.dim = a.head_dim;
  p.half = a.rot_dim / 2;
  p.seq_ids = a.seq_ids;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  bool e4m3 = false;
  if (a.cache != nullptr) {
    const qerl_kv_cache& c = *a.cache;
    e4m3 = c.dtype == QERL_E4M3;
    p.has_cache = true;
    p.k_pages = static_cast<uint8_t*>(c.k);
    p.v_pages = static_cast<uint8_t*>(c.v);
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.table = c.page_table;
    p.num_seqs = c.num_seqs;
    p.ld_table = c.ld_table;
    p.num_pages = c.num_pages;
    p.max_pages = c.max_pages;
    p.page_size = c.page_size;
  }
  p.status = a.status;
  // One item a thread; more than 512 are cut into equal parts.
  const int items = (p.heads + 2 * p.kv_heads) * (p.dim / 16);
  const int parts = (items + 511) / 512;
  const int threads = std::max(kMaxHalf, ((items + parts - 1) / parts + 31) / 32 * 32);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QERL_ERR_CUDA;
  const int64_t most = static_cast<int64_t>(sms) * ((e4m3 ? kThreadsPerSm<true> : kThreadsPerSm<false>) / threads);
  const dim3 grid(static_cast<unsigned>(a.tokens < most ? a.tokens : most), static_cast<unsigned>(parts));
  const size_t smem = static_cast<size_t>(kStages) * 2 * threads * 16;
  const void* kernel = e4m3 ? reinterpret_cast<const void*>(rope_append_kernel<true>)
                            : reinterpret_cast<const void*>(rope_append_kernel<false>);
  static std::atomic<uint64_t> ready[2];  // one bit per device: the attribute belongs to the device's function
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if ((ready[e4m3].load() & bit) == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * 2 * 512 * 16) != cudaSuccess)
      return QERL_ERR_CUDA;
    ready[e4m3].fetch_or(bit);
  }
  return cuda_status(
      launch_dependent(e4m3 ? rope_append_kernel<true> : rope_append_kernel<false>, grid, threads, smem, s, p));
}

}  // namespace qerl
