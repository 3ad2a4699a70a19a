// Rotary positions: each pair (a, b) of a head's first `rot` columns turned by
// an angle proportional to its token's position,
//   a' = f (a cos t - b sin t),  b' = f (a sin t + b cos t),  t = position * inv_freq[j],
// and for the gradient the transposed rotation (sin t -> -sin t). sm_103a.
//
// Angles. position * inv_freq in float32 is off by 0.06 at position 10^6. Here
// a frequency becomes turns per position in 64-bit fixed point; position times
// that, modulo 2^64, is the angle modulo one turn, exactly but for the
// frequency's own rounding (2^-53 of itself): one integer product per angle.
// Its top 32 bits, as a signed fraction of half a turn, go through sincospif.
//
// Work. A CTA takes a few tokens and all heads of both tensors: the angles of
// its tokens are computed once, into shared memory, and used for every head.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fa_varlen_kernel.cuh"

namespace fa {

// Turns per position (modulo 1) in 2^-64.
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;      // / 2 pi
  t -= floor(t);
  // (t may round up to 1, which is 0.)
  return t < 1.0 ? static_cast<uint64_t>(t * 18446744073709551616.0) : 0ull;
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

// The pairs of an item, in place; cs[e] belongs to its pair e.
__device__ __forceinline__ void rope_turn(float (&x)[16], const float2* cs, bool interleaved) {
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

struct RopeParams {
  RopeTensor x, y;           // y.heads = 0: none
  const int* positions;      // [T]
  const double* inv_freq;    // [rot / 2]
  int T, d, rot, interleaved, transpose;
  int tokens;                // of a CTA, at most kRopeTokens
  float factor;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;
constexpr int kRopeMaxPairs = 128;

// `n` tokens from t0 on, whose angles stand in cs [tokens][rot / 2]; rows with
// skip[token] != 0 are left alone.
__device__ __forceinline__ void rope_rows(const RopeTensor& t, int t0, int n, int d, int rot, bool interleaved,
                                          const float2* cs, const int* skip, int first, int step) {
  const int items = d / 16, per_token = t.heads * items;
  for (int w = first; w < n * per_token; w += step) {
    const int k = w / per_token, r = w - k * per_token, h = r / items, i = r - h * items;
    if (skip && skip[k]) continue;
    const RopeItem it = rope_item(i, rot, interleaved);
    const __nv_bfloat16* in = t.in + (t0 + k) * t.in_t + h * t.in_h;
    __nv_bfloat16* out = t.out + (t0 + k) * t.out_t + h * t.out_h;
    uint4 v0 = *reinterpret_cast<const uint4*>(in + it.c0), v1 = *reinterpret_cast<const uint4*>(in + it.c1);
    if (i < rot / 16) {
      float x[16];
      unpack8(v0, x);
      unpack8(v1, x + 8);
      rope_turn(x, cs + k * (rot / 2) + 8 * i, interleaved);
      v0 = pack8(x);
      v1 = pack8(x + 8);
    }
    *reinterpret_cast<uint4*>(out + it.c0) = v0;
    *reinterpret_cast<uint4*>(out + it.c1) = v1;
  }
}

__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  __shared__ __align__(16) float2 cs[kRopeTokens * kRopeMaxPairs];
  const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.T - t0), half = p.rot / 2;
  for (int w = threadIdx.x; w < n * half; w += kRopeThreads) {
    const int k = w / half, j = w - k * half;
    float2 t = turn(p.positions[t0 + k], turns_of(p.inv_freq[j]), p.factor);
    if (p.transpose) t.y = -t.y;
    cs[w] = t;
  }
  __syncthreads();
  const int first = blockIdx.y * kRopeThreads + threadIdx.x, step = gridDim.y * kRopeThreads;
  rope_rows(p.x, t0, n, p.d, p.rot, p.interleaved != 0, cs, nullptr, first, step);
  if (p.y.heads) rope_rows(p.y, t0, n, p.d, p.rot, p.interleaved != 0, cs, nullptr, first, step);
}

}  // namespace fa
