// Rotary positions: each pair (a, b) of a head's first `rot` columns turned by
// an angle proportional to its token's position,
//   a' = f (a cos t - b sin t),  b' = f (a sin t + b cos t),  t = position * inv_freq[j],
// and for the gradient the transposed rotation (sin t -> -sin t). sm_103a.
//
// Angles. position * inv_freq in float32 is off by 0.06 at position 10^6. Here
// a frequency becomes turns per position in 64-bit fixed point; position times
// that, modulo 2^64, is the angle modulo one turn, exactly but for position *
// 2^-64 turns: one integer product per angle.
// Its top 32 bits, as a signed fraction of half a turn, go through sincospif.
//
// What bounds it: memory, one read and one write of every element. A CTA takes
// about 40 KB of rows (a few tokens, all heads of both tensors); its angles are
// computed once, into shared memory, for all heads, while the first rows are on
// their way. A thread keeps its columns for all its rows. Measured: 8192 tokens x 40 heads of 128 columns,
// strided, 29.2 us, 5.7 TB/s (0.85 of a copy); 16001 tokens x 20 heads of 64
// columns, half of them rotated, 17.7 us, 4.6 TB/s; 37 tokens 2.1 us, a launch.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fa_varlen_kernel.cuh"

namespace fa {

namespace ptx {
// Programmatic dependent launches: what follows waits until the grids before
// have ended and their writes are visible; the next grid may be scheduled.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
}  // namespace ptx

// Turns per position (modulo 1) in 2^-64, cut: the 53 bits of inv_freq times
// 2^66 / 2 pi, in integers (the SM has few float64 units: with them this took an
// eighth of the time of a large call).
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
  const int ex = static_cast<int>(bits >> 52) & 0x7ff;
  const uint64_t m = ((bits & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0ull)) << 11;
  constexpr uint64_t kC = 0xa2f9836e4e441529ull;            // floor(2^66 / 2 pi)
  const uint64_t hi = __umul64hi(m, kC), lo = m * kC;
  const int s = (ex ? ex : 1) - 1024;
  const uint64_t r = s <= 0 ? (s > -64 ? hi >> -s : 0ull) : s < 64 ? hi << s | lo >> (64 - s) : 0ull;
  return bits >> 63 ? 0ull - r : r;
}

// f cos, f sin of position * inv_freq.
__device__ __forceinline__ float2 turn(int position, uint64_t turns, float factor) {
  const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(at >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c * factor, s * factor);
}

// 16 columns of a head as two pieces of 8, so that every pair lies in one
// item: item i < rot / 16 holds the pairs 8 i .. 8 i + 7, the others pass.
struct RopeItem {
  int c0, c1;        // first columns of the pieces
};
__device__ __forceinline__ RopeItem rope_item(int i, int rot, bool interleaved) {
  if (i >= rot / 16 || interleaved) return RopeItem{16 * i, 16 * i + 8};
  return RopeItem{8 * i, 8 * i + rot / 2};
}

// A token's angles as pairs of (f cos, f sin), so that neighbouring items' are
// neighbours: those of the pairs 8 i + 2 e and 8 i + 2 e + 1 at [e][i], `rot / 16`
// items. This is where pair j of a token lies, in float2.
__device__ __forceinline__ int angle_at(int j, int rot) { return ((j & 7) >> 1) * (rot / 8) + (j >> 3) * 2 + (j & 1); }
__device__ __forceinline__ void item_angles(float2 (&t)[8], const float2* cs, int i, int rot) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = *reinterpret_cast<const float4*>(cs + e * (rot / 8) + 2 * i);
    t[2 * e] = make_float2(v.x, v.y);
    t[2 * e + 1] = make_float2(v.z, v.w);
  }
}

// The pairs of an item, in place; cs[e] belongs to its pair e.
__device__ __forceinline__ void rope_turn(float (&x)[16], const float2 (&cs)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 t = cs[e];
      const float a = x[2 * e], b = x[2 * e + 1];
      x[2 * e] = a * t.x - b * t.y;
      x[2 * e + 1] = a * t.y + b * t.x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 t = cs[e];
      const float a = x[e], b = x[8 + e];
      x[e] = a * t.x - b * t.y;
      x[8 + e] = a * t.y + b * t.x;
    }
  }
}

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                    ptx::pack_bf16x2(x[6], x[7]));
}

struct RopeTensor {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  long long in_t, in_h, out_t, out_h;    // element strides of tokens and heads
  int heads;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeAngles = 1024;        // pairs of a CTA's tokens

// The rows of a CTA's tokens: all heads of x, then of y, token by token.
struct RopeRows {
  RopeTensor x, y;           // y.heads = 0: none
  int T, d, rot, interleaved;
  int tokens;                // of a CTA
  unsigned inv_heads;        // ceil(2^32 / (x.heads + y.heads)), for several tokens a CTA and more than one head
};

struct RopeParams {
  RopeRows r;
  const int* positions;      // [T]
  const double* inv_freq;    // [rot / 2]
  int transpose;
  float factor;
};

// Rotates the rows of the tokens t0 .. t0 + n - 1, whose angles `angles` writes
// to cs, rot / 2 a token (see angle_at; all threads call it, behind their first loads).
// Tokens with skip[token] != 0, as `angles` left it, are left alone.
template <int kThreads, class Angles>
__device__ __forceinline__ void rope_rows(const RopeRows& p, int t0, int n, const float2* cs, const int* skip,
                                          Angles angles) {
  constexpr int kBatch = 4;
  const int items = p.d / 16, heads = p.x.heads + p.y.heads, rows = n * heads;
  const int step = kThreads / items, row0 = threadIdx.x / items, i = threadIdx.x - row0 * items;
  const bool inter = p.interleaved != 0, turns = i < p.rot / 16;
  const RopeItem it = rope_item(i, p.rot, inter);
  const bool idle = row0 >= step;            // (threads beyond the last whole row)
  bool first = true;
#pragma unroll 1
  for (int r0 = row0; first || r0 < rows; r0 += kBatch * step) {
    uint4 v[kBatch][2];
    __nv_bfloat16* out[kBatch];
    int token[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * step;
      token[k] = -1;
      if (r < rows && !idle) {
        const int t = p.tokens == 1 ? 0 : heads == 1 ? r : static_cast<int>(__umulhi(static_cast<unsigned>(r), p.inv_heads));
        int h = r - t * heads;
        const bool second = h >= p.x.heads;
        const RopeTensor& a = second ? p.y : p.x;
        if (second) h -= p.x.heads;
        const __nv_bfloat16* in = a.in + (t0 + t) * a.in_t + h * a.in_h;
        out[k] = a.out + (t0 + t) * a.out_t + h * a.out_h;
        token[k] = t;
        v[k][0] = *reinterpret_cast<const uint4*>(in + it.c0);
        v[k][1] = *reinterpret_cast<const uint4*>(in + it.c1);
      }
    }
    if (first) angles();
    first = false;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (token[k] < 0 || (skip && skip[token[k]])) continue;
      if (turns) {
        float x[16];
        unpack8(v[k][0], x);
        unpack8(v[k][1], x + 8);
        float2 t[8];
        item_angles(t, cs + token[k] * (p.rot / 2), i, p.rot);
        rope_turn(x, t, inter);
        v[k][0] = pack8(x);
        v[k][1] = pack8(x + 8);
      }
      *reinterpret_cast<uint4*>(out[k] + it.c0) = v[k][0];
      *reinterpret_cast<uint4*>(out[k] + it.c1) = v[k][1];
    }
  }
}

__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  __shared__ __align__(16) float2 cs[kRopeAngles];
  ptx::grid_wait();
  ptx::grid_next();
  const int t0 = blockIdx.x * p.r.tokens, n = min(p.r.tokens, p.r.T - t0), half = p.r.rot / 2;
  rope_rows<kRopeThreads>(p.r, t0, n, cs, nullptr, [&] {
    for (int w = threadIdx.x; w < n * half; w += kRopeThreads) {
      const int k = w / half, j = w - k * half;
      float2 t = turn(p.positions[t0 + k], turns_of(p.inv_freq[j]), p.factor);
      if (p.transpose) t.y = -t.y;
      cs[k * half + angle_at(j, p.r.rot)] = t;
    }
    __syncthreads();
  });
}

}  // namespace fa
