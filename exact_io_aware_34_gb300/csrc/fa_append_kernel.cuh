// New keys and values of a batch into the pages of an 8-bit cache, the keys
// (and the queries beside them) rotated to their positions on the way. sm_103a.
//
// What is written. New token i of the n_b of sequence b takes place
// p = len_b - n_b + i of it: row p % page of page table[b][p / page]. A page's
// rows of one K/V head share a scale, a power of two 2^e, and hold
//   code = e4m3(x / scale),  e the smallest with max |x| <= 448 * 2^e
// (-100 at least), x the rotated key or the value in float32: rounded once. A
// page that holds older rows keeps their scale if it suffices; else they are
// brought to the new one, code * old / new rounded again, which between powers
// of two is exact but for values that become subnormal. Values that are not
// finite are stored as NaN and have no part in the scale.
//
// Work. The rows that one call adds to one page, of one head, of K or of V, are
// a CTA's work: their largest value decides about all of them. Lengths are
// known to the device alone, so the grid has room for every way to cut T tokens
// into pages: with T <= T / page + 2 B one place per token, of which those work
// that begin a page or a sequence (a decode step: all of them); else sequence b
// has the places from cu[b] / page + 2 b on, at least as many as it touches pages.
// Behind them stand the CTAs that rotate queries.
#pragma once

#include <cuda_fp8.h>

#include "fa_rope_kernel.cuh"

namespace fa {

enum : unsigned int { kRoleAppend = 29 };

struct AppendParams {
  const __nv_bfloat16* kv[2];      // K, V [T, H_kv, d]
  long long in_t[2], in_h[2];
  uint8_t* cache[2];               // e4m3 [num_pages, H_kv, page, d]
  long long c_page[2], c_head[2], c_row[2];   // bytes
  float* scale[2];                 // [num_pages, H_kv]
  const int* cu;                   // [B + 1]
  const int* table;                // [B, max_pages]
  const int* lens;                 // [B], with the new tokens
  const int* positions;            // [T] or null: the token's place in its sequence
  const double* inv_freq;          // [rot / 2]
  RopeTensor q;                    // q.heads = 0: none
  int B, H_kv, T, d, num_pages, page, max_pages, rot, interleaved;
  int per_token;                   // places: 1 one per token, 0 by page
  int places, q_tokens;            // q_tokens: tokens of a query CTA
  int q_split;                     // query CTAs that share their tokens
  float factor;
};

__device__ __forceinline__ void append_bad(int b) {
  if (atomicCAS(&g_status_word, 0u, kStatusBadOffsets) == 0u) {
    g_status_info[0] = kRoleAppend;
    g_status_info[1] = static_cast<unsigned int>(b);
    g_status_info[2] = g_status_info[3] = 0u;
  }
}

// Whether sequence b's offsets and length fit each other and the buffers.
__device__ __forceinline__ bool append_fits(const AppendParams& p, int c0, int c1, int len) {
  return c0 >= 0 && c0 <= c1 && c1 <= p.T && len >= c1 - c0 &&
         len <= static_cast<long long>(p.max_pages) * p.page;
}

// Two codes, and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3)));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
}

// The smallest power of two s >= 2^-100 with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float least_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -100) + 127) << 23);
}

template <int kThreads, int kItems>
__global__ void __launch_bounds__(kThreads) fa_append_kernel(const AppendParams p) {
  __shared__ __align__(16) float2 cs[kRopeTokens * 64];
  __shared__ int found[4], at[kRopeTokens], skip[kRopeTokens];
  __shared__ float warp_max[kThreads / 32];
  const int half = p.rot / 2;
  const int kv_ctas = p.places * p.H_kv * 2;

  if (static_cast<int>(blockIdx.x) >= kv_ctas) {
    // ------------------------------------------------------------ queries
    const int w0 = static_cast<int>(blockIdx.x) - kv_ctas, part = w0 % p.q_split;
    const int t0 = w0 / p.q_split * p.q_tokens, n = min(p.q_tokens, p.T - t0);
    if (threadIdx.x < kRopeTokens) skip[threadIdx.x] = 1;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      const int c0 = p.cu[b], c1 = p.cu[b + 1];
      if (c0 >= t0 + n || c1 <= t0) continue;
      const int len = p.lens[b];
      if (!append_fits(p, c0, c1, len)) continue;
      for (int t = max(c0, t0); t < min(c1, t0 + n); ++t) {
        at[t - t0] = p.positions ? p.positions[t] : len - (c1 - t);
        skip[t - t0] = 0;
      }
    }
    __syncthreads();
    for (int w = threadIdx.x; w < n * half; w += kThreads) {
      const int k = w / half, j = w - k * half;
      if (!skip[k]) cs[w] = turn(at[k], turns_of(p.inv_freq[j]), p.factor);
    }
    __syncthreads();
    rope_rows(p.q, t0, n, p.d, p.rot, p.interleaved != 0, cs, skip, part * kThreads + threadIdx.x,
              p.q_split * kThreads);
    return;
  }

  // -------------------------------------------------------------- keys, values
  const int which = static_cast<int>(blockIdx.x) & 1, u = static_cast<int>(blockIdx.x) >> 1;
  const int place = u / p.H_kv, head = u - place * p.H_kv;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  const bool check = blockIdx.x == 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    const bool mine = p.per_token ? c0 <= place && place < c1
                                  : c0 / p.page + 2 * b <= place && place < c1 / p.page + 2 * b + 2;
    if (!mine && !check) continue;
    const int len = p.lens[b];
    if (!append_fits(p, c0, c1, len)) {
      append_bad(b);
    } else if (mine) {
      found[0] = b;
      found[1] = c0;
      found[2] = c1;
      found[3] = len;
    }
  }
  __syncthreads();
  const int b = found[0];
  if (b < 0) return;
  const int c0 = found[1], len = found[3], before = len - (found[2] - c0);
  int p0, p1;                      // places [p0, p1) of the sequence, all in one page
  if (p.per_token) {
    p0 = before + (place - c0);
    if (place != c0 && p0 % p.page != 0) return;
    p1 = min(len, (p0 / p.page + 1) * p.page);
  } else {
    const int k = before / p.page + (place - (c0 / p.page + 2 * b));
    p0 = max(before, k * p.page);
    p1 = min(len, (k + 1) * p.page);
    if (p0 >= p1) return;
  }
  const int id = p.table[static_cast<long long>(b) * p.max_pages + p0 / p.page];
  if (id < 0 || id >= p.num_pages) {
    if (threadIdx.x == 0) append_bad(b);
    return;
  }
  const int row0 = p0 % p.page, rows = p1 - p0, t0 = c0 + (p0 - before);
  float* scale_at = p.scale[which] + static_cast<long long>(id) * p.H_kv + head;
  const float old = row0 > 0 ? *scale_at : 0.f;
  const bool turns = which == 0 && half > 0;
  const int items = p.d / 16;
  const __nv_bfloat16* in = p.kv[which] + t0 * p.in_t[which] + head * p.in_h[which];
  uint8_t* out = p.cache[which] + id * p.c_page[which] + head * p.c_head[which];

  float x[kItems][16];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int w = threadIdx.x + k * kThreads, r = w / items, i = w - r * items;
    if (r >= rows) break;
    const RopeItem it = rope_item(i, which == 0 ? p.rot : 0, p.interleaved != 0);
    unpack8(*reinterpret_cast<const uint4*>(in + r * p.in_t[which] + it.c0), x[k]);
    unpack8(*reinterpret_cast<const uint4*>(in + r * p.in_t[which] + it.c1), x[k] + 8);
    if (turns && i < p.rot / 16) {
      const int position = p.positions ? p.positions[t0 + r] : p0 + r;
      float2 t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = turn(position, turns_of(p.inv_freq[8 * i + e]), p.factor);
      rope_turn(x[k], t, p.interleaved != 0);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (fabsf(x[k][e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[k][e]));
      else x[k][e] = __uint_as_float(0x7fffffffu);      // NaN
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();                 // (the old scale has been read, too)
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
  const float scale = fmaxf(least_scale(amax), old);
  if (threadIdx.x == 0) *scale_at = scale;
  // (A scale that other code left here need not be a power of two.)
  const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0u;
  const float inv = 1.f / scale;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int w = threadIdx.x + k * kThreads, r = w / items, i = w - r * items;
    if (r >= rows) break;
    const RopeItem it = rope_item(i, which == 0 ? p.rot : 0, p.interleaved != 0);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) y[f] = exact ? x[k][4 * e + f] * inv : x[k][4 * e + f] / scale;
      c[e] = to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16;
    }
    uint8_t* dst = out + (row0 + r) * p.c_row[which];
    *reinterpret_cast<uint2*>(dst + it.c0) = make_uint2(c[0], c[1]);
    *reinterpret_cast<uint2*>(dst + it.c1) = make_uint2(c[2], c[3]);
  }
  if (row0 > 0 && scale != old) {
    const float ratio = old / scale;
    for (int w = threadIdx.x; w < row0 * items; w += kThreads) {
      const int r = w / items, i = w - r * items;
      uint4* at16 = reinterpret_cast<uint4*>(out + r * p.c_row[which] + 16 * i);
      uint4 v = *at16;
      uint32_t* c = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 lo = from_e4m3x2(c[e] & 0xffffu), hi = from_e4m3x2(c[e] >> 16);
        c[e] = to_e4m3x2(lo.x * ratio, lo.y * ratio) | to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
      }
      *at16 = v;
    }
  }
}

}  // namespace fa
