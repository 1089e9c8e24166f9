// kv_cache.cu -- rotary position embedding of q and k with the append of k and
// v to the paged cache, in one pass over the rows the q/k/v linears produced.
//
// Token t of sequence s at position p, pair i of a head (half = rot_dim / 2):
//   theta = p * inv_freq[i]
//   (x[i], x[i + half]) -> (x[i] cos - x[i + half] sin, x[i + half] cos + x[i] sin)
// in fp32 with one rounding to bf16 (and, for the cache, one rounding of the
// fp32 value to the cache's type: the 8-bit cache holds sat(value / scale)).
//
// Bound: bytes.  Every q, k, v element is read once and written once or twice.
// A CTA takes one token at a time (grid-stride); a thread takes one item = two
// 16-byte chunks of one head: the two halves of 8 pairs, or 2 chunks that are
// only copied, so a thread's loads do not wait for the angles.
#include "qerl_internal.h"
#include "qerl_ptx.cuh"

#include <cuda_bf16.h>

namespace qerl {
namespace {

constexpr int kMaxHalf = 64;  // rot_dim / 2

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t ldq, ldk, ldv;
  __nv_bfloat16 *q_out, *k_out;
  int64_t ldqo, ldko;
  int64_t tokens;
  int heads, kv_heads, dim, half;
  const int *seq_ids, *positions;
  const double* inv_freq;
  // The cache; k_pages null: rotation only.
  uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int* table;
  int64_t num_seqs, ld_table, num_pages, max_pages;
  int page_size;
  int* status;
};

__device__ __forceinline__ void unpack8(uint4 w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// Eight fp32 values -> E4M3 (nearest even, saturating, NaN kept) of value / scale.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float scale) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __fdiv_rn(f[2 * i], scale), b = __fdiv_rn(f[2 * i + 1], scale);
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
        : "=r"(h[i])
        : "f"(b), "f"(a));
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <bool kE4m3>
__global__ void __launch_bounds__(512) rope_append_kernel(const AppendParams p) {
  __shared__ __align__(16) float cs[2][kMaxHalf], sn[2][kMaxHalf];
  const int tid = threadIdx.x;
  // Turns per position as a 64-bit binary fraction: the product with the
  // position keeps exactly the bits below one turn, so far positions lose
  // nothing (an fp32 angle would be off by 1e-3 rad at position 1e4).
  uint64_t turn = 0;
  if (tid < p.half) {
    const double t = p.inv_freq[tid] * 0.15915494309189533577;  // 1 / (2 pi)
    turn = static_cast<uint64_t>(__double2ull_rn((t - floor(t)) * 18446744073709551616.0));
  }
  const int per_head = p.dim >> 4;  // items of a head
  const int rot_items = p.half >> 3;
  const int items = (p.heads + 2 * p.kv_heads) * per_head;
  // The place of token t in the cache: its page number, or -1.
  auto page_of = [&](int64_t t, int pos) -> int {
    if (p.k_pages == nullptr || pos < 0) return -1;
    const int64_t s = p.seq_ids != nullptr ? p.seq_ids[t] : t;
    const int64_t pi = pos / p.page_size;
    return s >= 0 && s < p.num_seqs && pi < p.max_pages ? p.table[s * p.ld_table + pi] : -1;
  };
  int buf = 0;
  // A token's position and page number, which depend on one another, are
  // fetched while the tokens before it are worked on.
  int64_t t = blockIdx.x;
  int pos = p.positions[t], pos_next = t + gridDim.x < p.tokens ? p.positions[t + gridDim.x] : -1;
  int page = page_of(t, pos);
  for (int page_next = -1, pos_later = -1; t < p.tokens; t += gridDim.x, pos = pos_next, page = page_next, pos_next = pos_later) {
    const int64_t t1 = t + gridDim.x, t2 = t1 + gridDim.x;
    page_next = t1 < p.tokens ? page_of(t1, pos_next) : -1;
    pos_later = t2 < p.tokens ? p.positions[t2] : -1;
    if (pos < 0) continue;  // padding: uniform over the CTA
    for (int it = tid, first = 1;; it += blockDim.x, first = 0) {
      const int head = it / per_head, sub = it - head * per_head;
      // 0: q, 1: k, 2: v
      const int kind = head < p.heads ? 0 : head < p.heads + p.kv_heads ? 1 : 2;
      const int hh = kind == 0 ? head : kind == 1 ? head - p.heads : head - p.heads - p.kv_heads;
      const bool rot = kind < 2 && sub < rot_items;
      // element offsets of the item's two chunks within the head
      const int e0 = rot ? sub * 8 : kind == 2 ? sub * 16 : 2 * p.half + (sub - rot_items) * 16;
      const int e1 = rot ? p.half + sub * 8 : e0 + 8;
      const bool live = it < items && (kind < 2 || p.k_pages != nullptr);
      uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
      if (live) {
        const __nv_bfloat16* src = kind == 0 ? p.q + t * p.ldq : kind == 1 ? p.k + t * p.ldk : p.v + t * p.ldv;
        src += static_cast<int64_t>(hh) * p.dim;
        w0 = *reinterpret_cast<const uint4*>(src + e0);
        w1 = *reinterpret_cast<const uint4*>(src + e1);
      }
      if (first) {  // while the first item's rows arrive
        if (tid < p.half) {
          const uint64_t a = turn * static_cast<uint64_t>(pos);
          // the top 32 bits as a signed fraction of half a turn, in [-1, 1)
          const float x = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578125e-10f;
          sincospif(x, &sn[buf][tid], &cs[buf][tid]);
        }
        __syncthreads();  // the angles of this token; two buffers, so one barrier a token
      }
      if (it >= items) break;
      if (!live) continue;
      const bool placed = page >= 0 && page < p.num_pages;
      float a[8], b[8];
      unpack8(w0, a);
      unpack8(w1, b);
      if (rot) {
        float c[8], s[8];
        const float4* c4 = reinterpret_cast<const float4*>(&cs[buf][sub * 8]);
        const float4* s4 = reinterpret_cast<const float4*>(&sn[buf][sub * 8]);
        *reinterpret_cast<float4*>(c) = c4[0];
        *reinterpret_cast<float4*>(c + 4) = c4[1];
        *reinterpret_cast<float4*>(s) = s4[0];
        *reinterpret_cast<float4*>(s + 4) = s4[1];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = a[i], y = b[i];
          a[i] = x * c[i] - y * s[i];
          b[i] = y * c[i] + x * s[i];
        }
        w0 = pack8_bf16(a);
        w1 = pack8_bf16(b);
      }
      __nv_bfloat16* dst = kind == 0 ? p.q_out + t * p.ldqo
                           : kind == 1 && p.k_out != nullptr ? p.k_out + t * p.ldko
                                                             : nullptr;
      if (dst != nullptr) {
        dst += static_cast<int64_t>(hh) * p.dim;
        *reinterpret_cast<uint4*>(dst + e0) = w0;
        *reinterpret_cast<uint4*>(dst + e1) = w1;
      }
      if (kind >= 1 && placed) {
        uint8_t* pages = kind == 1 ? p.k_pages : p.v_pages;
        const int64_t at =
            ((static_cast<int64_t>(page) * p.kv_heads + hh) * p.page_size + pos % p.page_size) * p.dim;
        if (kE4m3) {
          const float* sc = kind == 1 ? p.k_scale : p.v_scale;
          const float scale = sc != nullptr ? sc[hh] : 1.0f;
          *reinterpret_cast<uint2*>(pages + at + e0) = pack8_e4m3(a, scale);
          *reinterpret_cast<uint2*>(pages + at + e1) = pack8_e4m3(b, scale);
        } else {
          __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(pages) + at;
          *reinterpret_cast<uint4*>(d + e0) = w0;
          *reinterpret_cast<uint4*>(d + e1) = w1;
        }
      }
    }
    if (tid == 0 && p.k_pages != nullptr && (page < 0 || page >= p.num_pages)) record_error(p.status, QERL_ERR_RANGE);
    buf ^= 1;
  }
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
  // One item a thread where the CTA's 512 threads allow it.
  const int items = (p.heads + 2 * p.kv_heads) * (p.dim / 16);
  int threads = (items + 31) / 32 * 32;
  threads = threads > 512 ? 512 : threads < kMaxHalf ? kMaxHalf : threads;
  const int64_t most = 152 * 8;
  const unsigned grid = static_cast<unsigned>(a.tokens < most ? a.tokens : most);
  if (e4m3)
    rope_append_kernel<true><<<grid, threads, 0, s>>>(p);
  else
    rope_append_kernel<false><<<grid, threads, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}

}  // namespace qerl
