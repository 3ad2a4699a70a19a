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
// Work. The rows that one call adds to one page, of one head, of K or of V,
// belong together: their largest value decides about all of them. They are the
// work of one warp, or, where many rows meet large pages, of page / 16 warps: 16 rows
// a warp stay in registers between the maximum and the rounding (more are read
// again). Lengths are known to the device alone, so the grid has room for every
// way to cut T tokens into pages: with T <= T / page + 2 B one place per token, of
// which those work that begin a page or a sequence (a decode step: all of them);
// else sequence b has the places from cu[b] / page + 2 b on, at least as many as it
// touches pages. Between them stand the CTAs that rotate queries (fa_rope_kernel's rows).
//
// What bounds it. A decode step is one chain: offsets, table, rows and old scale,
// maximum, rounding (2 tokens 3.8 us, 64 tokens 4.1; a page's angles once
// for the CTA's heads, a division of places by pages once for a block). Prompts pass every
// row through registers once: 8414 tokens, 32 query heads on 8, pages of 16 rows,
// 47.5 us, 4.0 TB/s (0.59 of a copy). Larger pages take longer, 32 rows 52 us, 64 rows 58, 128 rows
// 70: a head's page is then the work of 2, 4 or 8 warps, a CTA has 4, 2 or 1 heads instead of 8, and its
// angles (16, 32 or 64 KB instead of 8) serve only those. With 16 rows half of the time is computing (46 % of issue
// slots busy) in chains of load, rotation, maximum and rounding, which is why the CTAs of
// the queries, which wait for memory, stand between the others and not behind (50.7 us).
// Rows fetched before the angles are computed cost registers and with them
// CTAs (75 us); 8 rows a warp changed nothing (46-48); three CTAs per SM gave
// 44.5, and 4.8 instead of 4.1 for a decode step.
#pragma once

#include <cuda_fp8.h>

#include "fa_rope_kernel.cuh"

namespace fa {

namespace ptx {
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
}  // namespace ptx

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
  RopeRows q;                      // queries (q.x.heads = 0: none)
  int B, H_kv, T, d, num_pages, page, max_pages, rot, interleaved;
  int per_token;                   // places: 1 one per token, 0 by page
  int places;
  int warps;                       // of a head: 1, 2, 4 or 8
  int head_groups;                 // CTAs of a place, each with 8 / warps heads
  int query_ctas, period;
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

constexpr int kAppendThreads = 256;
// Dynamic shared memory at most: the angles of a page's rows (or kRopeAngles for queries).
constexpr int kAppendMaxSmem = 128 * 64 * static_cast<int>(sizeof(float2));

// Up to 16 rows of a head as kItems items of 16 columns a lane, rotated. Lane l's
// item k is item l % items of row (l / items) + k * (32 / items), items = HD / 16.
template <int HD>
struct AppendRows {
  static constexpr int kPerRow = HD / 16, kRowStep = 32 / kPerRow, kItems = 16 / kRowStep;
  float x[kItems][16];
  float amax;                      // of the finite values

  // cs: the rows' angles (keys).
  __device__ __forceinline__ void load(const AppendParams& p, const float2* cs, int which, int head, int t0, int rows) {
    const int lane = threadIdx.x & 31, row0 = lane / kPerRow, i = lane % kPerRow;
    const bool inter = p.interleaved != 0, turns = which == 0 && i < p.rot / 16;
    const RopeItem it = rope_item(i, which == 0 ? p.rot : 0, inter);
    const __nv_bfloat16* in = p.kv[which] + t0 * p.in_t[which] + head * p.in_h[which];
    uint4 v[kItems][2];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = row0 + k * kRowStep;
      v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        v[k][0] = *reinterpret_cast<const uint4*>(in + r * p.in_t[which] + it.c0);
        v[k][1] = *reinterpret_cast<const uint4*>(in + r * p.in_t[which] + it.c1);
      }
    }
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = row0 + k * kRowStep;
      if (k > 0 && k * kRowStep >= rows) {     // (no lane has a row here)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[k][e] = 0.f;
        continue;
      }
      unpack8(v[k][0], x[k]);
      unpack8(v[k][1], x[k] + 8);
      if (turns && r < rows) {
        float2 t[8];
        item_angles(t, cs + r * (p.rot / 2), i, p.rot);
        rope_turn(x[k], t, inter);
      }
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) m = ptx::max_nan(m, fabsf(x[k][e]));
      if (!(m <= 3.402823466e38f)) {
        m = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (fabsf(x[k][e]) <= 3.402823466e38f) m = fmaxf(m, fabsf(x[k][e]));
          else x[k][e] = __uint_as_float(0x7fffffffu);      // NaN
        }
      }
      amax = fmaxf(amax, m);
    }
  }

  // In units of the scale. (One that other code left here need not be a power of two.)
  __device__ __forceinline__ void divide(float scale) {
    if ((__float_as_uint(scale) & 0x7fffffu) == 0u) {
      const float inv = 1.f / scale;
#pragma unroll
      for (int k = 0; k < kItems; ++k)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[k][e] *= inv;
    } else {
#pragma unroll
      for (int k = 0; k < kItems; ++k)
#pragma unroll 1
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((e >> 2) == q) x[k][e] /= scale;
    }
  }

  // To the page's rows from `out` on.
  __device__ __forceinline__ void store(const AppendParams& p, int which, uint8_t* out, int rows) const {
    const int lane = threadIdx.x & 31, row0 = lane / kPerRow, i = lane % kPerRow;
    const RopeItem it = rope_item(i, which == 0 ? p.rot : 0, p.interleaved != 0);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = row0 + k * kRowStep;
      if (r >= rows) break;
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = to_e4m3x2(x[k][4 * e], x[k][4 * e + 1]) | to_e4m3x2(x[k][4 * e + 2], x[k][4 * e + 3]) << 16;
      uint8_t* dst = out + r * p.c_row[which];
      *reinterpret_cast<uint2*>(dst + it.c0) = make_uint2(c[0], c[1]);
      *reinterpret_cast<uint2*>(dst + it.c1) = make_uint2(c[2], c[3]);
    }
  }
};

template <int HD>
__global__ void __launch_bounds__(kAppendThreads) fa_append_kernel(const AppendParams p) {
  constexpr int kThreads = kAppendThreads;
  extern __shared__ __align__(16) float2 cs[];
  __shared__ int found, at[kRopeMaxTokens], skip[kRopeMaxTokens];
  __shared__ float warp_max[8];
  ptx::grid_wait();
  ptx::grid_next();
  const int half = p.rot / 2;
  // Query CTAs wait for memory, the others mostly compute: every p.period-th CTA is a query CTA while there are any.
  int cta = static_cast<int>(blockIdx.x);
  const int turn_of = (cta + 1) / p.period;        // query CTAs up to this one
  const bool query = turn_of * p.period == cta + 1 && turn_of <= p.query_ctas;
  cta = query ? turn_of - 1 : cta - min(turn_of, p.query_ctas);

  if (query) {
    // ------------------------------------------------------------ queries
    const int t0 = cta * p.q.tokens, n = min(p.q.tokens, p.T - t0);
    rope_rows<kThreads>(p.q, t0, n, cs, skip, [&] {
      if (threadIdx.x < kRopeMaxTokens) skip[threadIdx.x] = 1;
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
        if (!skip[k]) cs[k * half + angle_at(j, p.rot)] = turn(at[k], turns_of(p.inv_freq[j]), p.factor);
      }
      __syncthreads();
    });
    return;
  }

  // -------------------------------------------------------------- keys, values
  const int which = cta & 1, u = cta >> 1;
  const int place = p.head_groups == 1 ? u : u / p.head_groups, group = u - place * p.head_groups;
  const bool check = cta == 0;
  // A decode step's token t is sequence t's; else all threads look for the place's sequence.
  int b = -1, c0 = 0, c1 = 0, len = 0;
  if (p.per_token && place < p.B) {
    c0 = p.cu[place];
    c1 = p.cu[place + 1];
    if (c0 == place && c1 == place + 1) {
      len = p.lens[place];
      if (append_fits(p, c0, c1, len)) b = place;
    }
  }
  if (b < 0 || check) {            // (the same in all threads)
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < p.B; s += kThreads) {
      const int s0 = p.cu[s], s1 = p.cu[s + 1];
      const bool mine = p.per_token ? s0 <= place && place < s1
                                    : s0 / p.page + 2 * s <= place && place < s1 / p.page + 2 * s + 2;
      if (!mine && !check) continue;
      const int n = p.lens[s];
      if (!append_fits(p, s0, s1, n)) {
        append_bad(s);
      } else if (mine) {
        atomicMax(&found, s);      // (offsets that decrease in between may give a place to several)
      }
    }
    __syncthreads();
    b = found;
    if (b >= 0) {
      c0 = p.cu[b];
      c1 = p.cu[b + 1];
      len = p.lens[b];
    }
  }
  if (b < 0) return;
  const int before = len - (c1 - c0);
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
  // Warp `sub` of the head's takes every p.warps-th block of 16 rows.
  const int warp = threadIdx.x >> 5, sub = warp & (p.warps - 1), head = group * (8 / p.warps) + warp / p.warps;
  const bool live = head < p.H_kv;
  const int row0 = p0 % p.page, rows = p1 - p0, t0 = c0 + (p0 - before);
  // The angles of the keys' rows, for all heads of the CTA.
  if (which == 0 && half > 0) {
    for (int w = threadIdx.x; w < rows * half; w += kThreads) {
      const int k = w / half, j = w - k * half;
      cs[k * half + angle_at(j, p.rot)] =
          turn(p.positions ? p.positions[t0 + k] : p0 + k, turns_of(p.inv_freq[j]), p.factor);
    }
    __syncthreads();
  }
  if (id < 0 || id >= p.num_pages) {
    if (threadIdx.x == 0) append_bad(b);
    return;
  }
  float* scale_at = p.scale[which] + static_cast<long long>(id) * p.H_kv + head;
  const float old = live && row0 > 0 ? *scale_at : 0.f;
  uint8_t* out = p.cache[which] + id * p.c_page[which] + head * p.c_head[which];
  AppendRows<HD> x;
  float amax = 0.f, scale = 0.f;
  // First the largest value, then the rounding; rows of more than one block are read again for it.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int r = 16 * sub; r < rows && live; r += 16 * p.warps) {
      if (pass == 0 || rows > 16 * p.warps) {
        x.load(p, cs + r * half, which, head, t0 + r, min(16, rows - r));
        amax = fmaxf(amax, x.amax);
      }
      if (pass == 1) {
        x.divide(scale);
        x.store(p, which, out + (row0 + r) * p.c_row[which], min(16, rows - r));
      }
    }
    if (pass == 1) break;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncwarp();                  // (every lane has read the old scale)
    if (p.warps > 1) {
      if ((threadIdx.x & 31) == 0) warp_max[warp] = amax;
      __syncthreads();
      for (int w = 0; w < p.warps; ++w) amax = fmaxf(amax, warp_max[warp - sub + w]);
    }
    scale = fmaxf(least_scale(amax), old);
    if (live && sub == 0 && (threadIdx.x & 31) == 0) *scale_at = scale;
  }
  if (!live) return;
  if (row0 > 0 && scale != old) {
    const float ratio = old / scale;
    constexpr int kPerRow = HD / 16;
    for (int w = sub * 32 + (threadIdx.x & 31); w < row0 * kPerRow; w += 32 * p.warps) {
      const int r = w / kPerRow, i = w % kPerRow;
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
