// Exact attention of new tokens over a paged cache held in 8 bits (e4m3 with a
// scale for each page and K/V head). First form: one CTA per (token, K/V head),
// a warp per query head, a lane per key of 32.
#pragma once

#include "fa_append_kernel.cuh"

namespace fa {

enum : unsigned int { kRolePagedWalk = 33 };

struct PagedParams {
  const __nv_bfloat16* q;          // [T_q, H, d]
  __nv_bfloat16* o;
  float* lse;                      // [H, T_q]
  long long q_t, q_h, o_t, o_h;    // element strides
  const uint8_t* cache[2];
  long long c_page[2], c_head[2], c_row[2];   // bytes
  const float* scale[2];           // [num_pages, H_kv]
  const int* table;                // [B, max_pages]
  const int* lens;                 // [B]
  const int* cu;                   // [B + 1]
  int B, H, H_kv, G, T_q, num_pages, page, max_pages, causal;
  float scale_log2;                // of the scores, with its sign
};

__device__ __forceinline__ void paged_bad(int b) {
  if (atomicCAS(&g_status_word, 0u, kStatusBadOffsets) == 0u) {
    g_status_info[0] = kRolePagedWalk;
    g_status_info[1] = static_cast<unsigned int>(b);
    g_status_info[2] = g_status_info[3] = 0u;
  }
}

template <int HD>
__global__ void __launch_bounds__(128) fa_paged_kernel(const PagedParams p) {
  __shared__ float sq[4][HD];
  __shared__ int found[4];
  constexpr int kPer = HD / 32;
  const int t = blockIdx.x, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += 128) {
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    const bool fits = c0 >= 0 && c0 <= c1 && c1 <= p.T_q;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      const int len = p.lens[b];
      if (!fits || len < 0 || len > p.max_pages * p.page) paged_bad(b);
    }
    if (fits && c0 <= t && t < c1) {
      found[1] = c0;
      found[2] = c1;
      found[0] = b;
    }
  }
  __syncthreads();
  const int b = found[0];
  if (b < 0) return;
  const int room = p.max_pages * p.page;
  const int n_kv = max(0, min(room, p.lens[b]));
  const int end = p.causal ? min(n_kv, max(0, n_kv - (found[2] - found[1]) + (t - found[1]) + 1)) : n_kv;
  for (int g = warp; g < p.G; g += 4) {
    const int h = kvh * p.G + g;
    const __nv_bfloat16* q = p.q + t * p.q_t + h * p.q_h;
    __syncwarp();
    for (int i = lane; i < HD; i += 32) sq[warp][i] = __bfloat162float(q[i]) * p.scale_log2;
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      float s = -INFINITY, sv = 0.f;
      long long v_row = 0;
      if (j < end) {
        const int id = p.table[static_cast<long long>(b) * p.max_pages + j / p.page], r = j % p.page;
        if (id < 0 || id >= p.num_pages) {
          paged_bad(b);
        } else {
          const uint8_t* k = p.cache[0] + id * p.c_page[0] + kvh * p.c_head[0] + r * p.c_row[0];
          v_row = id * p.c_page[1] + kvh * p.c_head[1] + r * p.c_row[1];
          s = 0.f;
          for (int i = 0; i < HD; i += 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(k + i);
            const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 lo = from_e4m3x2(c[e] & 0xffffu), hi = from_e4m3x2(c[e] >> 16);
              const float* x = &sq[warp][i + 4 * e];
              s = fmaf(lo.x, x[0], fmaf(lo.y, x[1], fmaf(hi.x, x[2], fmaf(hi.y, x[3], s))));
            }
          }
          s *= p.scale[0][static_cast<long long>(id) * p.H_kv + kvh];
          sv = p.scale[1][static_cast<long long>(id) * p.H_kv + kvh];
        }
      }
      float mt = s;
      bool nan = s != s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      nan = __any_sync(0xffffffffu, nan);
      const float m_new = nan ? NAN : fmaxf(m, mt);
      if (m_new == -INFINITY) continue;
      const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new), w = exp2f(s - m_new);
      m = m_new;
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = l * alpha + sum;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] *= alpha;
      const float wv = w * sv;
      for (int k = 0; k < min(32, end - j0); ++k) {
        const float x = __shfl_sync(0xffffffffu, wv, k);
        const uint8_t* v = p.cache[1] + __shfl_sync(0xffffffffu, v_row, k) + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
          const float2 c = from_e4m3x2(*reinterpret_cast<const uint16_t*>(v + e));
          acc[e] = fmaf(x, c.x, acc[e]);
          acc[e + 1] = fmaf(x, c.y, acc[e + 1]);
        }
      }
    }
    const bool none = m == -INFINITY;
    const float inv = none ? 0.f : 1.f / l;
    __nv_bfloat16* o = p.o + t * p.o_t + h * p.o_h + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = __float2bfloat16(acc[e] * inv);
    if (lane == 0) p.lse[static_cast<long long>(h) * p.T_q + t] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
}

}  // namespace fa
