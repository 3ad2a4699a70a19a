// (Units of many rows.)
#pragma once

#include "fa_paged_kernel.cuh"

namespace fa {

template <int HD, int N>
struct PagedWideCfg {
  static constexpr int kThreads = 256;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kStages = N == 16 ? (HD == 128 ? 3 : 5) : (HD == 128 ? 2 : 4);
  static constexpr int kTileBytes = 128 * HD;          // K or V
  static constexpr int kPBytes = N * 128;              // hi or lo
  static constexpr int kQBytes = N * HD;
  // With d = 64 the M side of V^T P^T is V's 64 columns and 64 lanes that nobody
  // reads, fed from the 8 KB behind the tile: the last one has a pad.
  static constexpr int kPad = HD == 64 ? kTileBytes : 0;
  static constexpr int kSmemBytes = 2 * kPBytes + 2 * kQBytes + kStages * 2 * kTileBytes + kPad + 1024;
  static constexpr uint32_t kTmemCols = N == 16 ? 64 : 256;
  static constexpr uint32_t kColS = 0;                 // two buffers
  static constexpr uint32_t kColO = 2 * N;
  static constexpr uint32_t kSwizzle = HD == 128 ? 2 : 4;
  static constexpr uint32_t kAtom = 8 * HD;            // eight rows
  static constexpr int kRegsSoftmax = 200;
  static constexpr int kRegsControl = 56;
  static_assert(2 * (kSmemBytes + 5 * 1024) <= 228 * 1024, "two CTAs per SM");
};

// x[i] over the 32 lanes of a warp for 16 values at a time: lane l returns the sum of value l % 16.
__device__ __forceinline__ float lanes_sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int h = 8; h > 0; h >>= 1) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h], mine = up ? v[i + h] : v[i];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, send, h);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

template <int HD, int N>
__global__ void __launch_bounds__(PagedWideCfg<HD, N>::kThreads, PagedWideCfg<HD, N>::kCtasPerSm)
    fa_paged_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedParams p) {
  using C = PagedWideCfg<HD, N>;
  constexpr int kChunks = N / 16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_k_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_v_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_p_full;
  __shared__ __align__(8) uint64_t bar_o_full;
  __shared__ __align__(8) uint64_t bar_q_full;
  __shared__ __align__(8) uint64_t bar_job_full[2];
  __shared__ __align__(8) uint64_t bar_job_empty[2];
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PagedJob jobs[2];
  __shared__ __align__(16) float page_scale[C::kStages][2][8];   // K, V scales of a tile's pages
  __shared__ __align__(16) float row_scale[N];      // of S, by row: the scores' scale over the query row's
  __shared__ __align__(16) int row_lim[N];          // keys the row sees
  __shared__ __align__(16) float red[4][N];         // by warp
  __shared__ __align__(16) float row_max[N];        // the tile's maximum - kPagedTop
  __shared__ __align__(16) float row_fac[N];        // 2^(that - reference)
  __shared__ __align__(16) float row_fac_o[2][N];   // that times the tile's largest V scale, for two tiles
  __shared__ __align__(16) float row_corr[2][N];    // what the sums before are multiplied by first
  __shared__ int corr_any[2];
  __shared__ int warp_sum[C::kThreads / 32];
  __shared__ int start_b, start_cum;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShape& sh = p.s;
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sP = smem_base, sQ = sP + 2 * C::kPBytes, sKV = sQ + 2 * C::kQBytes;
  static_assert((2 * C::kPBytes) % 1024 == 0 && (2 * C::kQBytes) % 1024 == 0, "tiles begin on swizzle atoms");

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_k_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_v_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 6);   // warps 0-5
      corr_any[t] = 0;
    }
    ptx::mbar_init(ptx::smem_u32(&bar_p_full), 128);
    ptx::mbar_init(ptx::smem_u32(&bar_o_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_q_full), 128);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    abort_flag = 0;
    start_b = sh.B;
    start_cum = 0;
    p.split[blockIdx.x].n = 0;
    ptx::fence_mbar_init();
  }
  // (Of pages above 16 rows only the first places are ever written.)
  if (threadIdx.x < C::kStages * 16) (&page_scale[0][0][0])[threadIdx.x] = 0.f;
  if (warp == 5) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }

  // The line's length and where this CTA's piece begins (as in fa_prefix_kernel).
  int sum = 0;
  for (int b = threadIdx.x; b < sh.B; b += C::kThreads) sum += paged_seq(p, b).places(sh);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  int seq_sum = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) seq_sum += warp_sum[w];
  const int copies = sh.H_kv * sh.ht;              // of a sequence's places
  const int total = seq_sum * copies;
  const int x_begin = line_begin(total, sh.ctas, blockIdx.x), x_end = line_begin(total, sh.ctas, blockIdx.x + 1);
  const bool check = blockIdx.x == 0;
  if (check || x_end > x_begin) {
    const int target = x_begin / copies;
    int base = 0;
    for (int b0 = 0; b0 < sh.B; b0 += C::kThreads) {
      const int b = b0 + threadIdx.x;
      int nu = 0;
      if (b < sh.B) {
        nu = paged_seq(p, b).places(sh);
        if (check) {
          const int c0 = p.cu[b], c1 = p.cu[b + 1], len = p.lens[b];
          if (c0 < 0 || c0 > c1 || c1 > sh.T_q || len < 0 || len > sh.max_pages << sh.page_shift) paged_bad(b);
        }
      }
      int incl = nu;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      __syncthreads();
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      int before = base, chunk = 0;
#pragma unroll
      for (int w = 0; w < C::kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        chunk += warp_sum[w];
      }
      const int excl = before + incl - nu;
      if (nu > 0 && excl <= target && target < excl + nu) {
        start_b = b;
        start_cum = excl;
      }
      base += chunk;
      if (!check && base > target) break;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  volatile int* abort_ptr = &abort_flag;

  if (warp >= 4) ptx::setmaxnreg_dec<C::kRegsControl>();
  if (warp < 4) {
    // ------------------------------------------------------------ softmax and sums
    ptx::setmaxnreg_inc<C::kRegsSoftmax>();
    const int tid = threadIdx.x;                   // this thread's key of a tile, and its column of O
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem_base + lane_addr + C::kColO;
    const uint32_t tS0 = tmem_base + lane_addr + C::kColS;
    const int page_slot = tid >> sh.page_shift;
    uint8_t* generic = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
    int g = 0;                                     // tiles so far
    bool stop = false;
    for (int n = 0; !stop; ++n) {
      bool ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr,
                                   kUnitWaits * p.timeout_ns, kRolePagedSoftmax);
      // (All four warps leave together: a named barrier must not be left waiting.)
      if (ptx::softmax_any(!ok)) break;
      const PagedJob job = jobs[n & 1];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (job.b < 0) break;
      const int nch = (job.rows + 15) >> 4;        // 16-row chunks in use

      // The query rows, as hi and lo in the swizzled K-major layout.
      {
        constexpr int kLanes = HD / 16;            // threads of a row, 16 elements each
        const int part = tid % kLanes;
#pragma unroll 1
        for (int r = tid / kLanes; r < 16 * nch; r += 128 / kLanes) {
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
          const int ti = r / job.heads, hi = r - ti * job.heads;
          const bool live = r < job.rows;
          if (live) {
            const __nv_bfloat16* src = p.q + (job.token + ti) * p.q_t + (job.head + hi) * p.q_h + 16 * part;
            unpack8(*reinterpret_cast<const uint4*>(src), x);
            unpack8(*reinterpret_cast<const uint4*>(src + 8), x + 8);
          }
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (fabsf(x[e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[e]));
            else x[e] = __uint_as_float(0x7fffffffu);
          }
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // 2^k with the largest element in [128, 256)
          const int k = amax > 0.f ? max(-120, min(120, 134 - static_cast<int>(__float_as_uint(amax) >> 23))) : 0;
          const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
          uint32_t hi4[4], lo4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            hi4[e] = lo4[e] = 0;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const float a = x[4 * e + 2 * f] * up, b = x[4 * e + 2 * f + 1] * up;
              const uint32_t h = to_e4m3x2(a, b);
              const float2 back = from_e4m3x2(h);
              hi4[e] |= h << (16 * f);
              lo4[e] |= to_e4m3x2(a - back.x, b - back.y) << (16 * f);
            }
          }
          const uint32_t at = static_cast<uint32_t>(r) * HD +
                              ((part ^ (HD == 128 ? r & 7 : (r >> 1) & 3)) << 4);
          *reinterpret_cast<uint4*>(generic + (sQ - smem_base) + at) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(generic + (sQ - smem_base) + C::kQBytes + at) =
              make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          if (part == 0) {
            row_scale[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            row_lim[r] = live ? min(job.n_keys, sh.causal ? job.lim0 + ti : job.lim0) : 0;
          }
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bar_q_full));
      const int all_see = min(job.n_keys, job.lim0);   // keys that every row sees
      ptx::softmax_any(false);                         // row_scale and row_lim stand

      float acc[N], lsum[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = lsum[i] = 0.f;
      float ref = -INFINITY;                           // of row tid (tid < N): exponents in the sums are relative to it
      // Adds O^T of the tile before (number g - 1).
      auto add_tile = [&](int buf) {
        ptx::tc_fence_after();
        const bool corr = corr_any[buf] != 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c < nch) {
            uint32_t o[16];
            ptx::tmem_ld16(tO + 16 * c, o);
            ptx::tmem_ld_wait();
            ptx::reg_fence16(o);
            if (corr) {
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[16 * c + i] *= row_corr[buf][16 * c + i];
            }
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&row_fac_o[buf][16 * c + i]);
              acc[16 * c + i] = fmaf(__uint_as_float(o[i]), f.x, acc[16 * c + i]);
              acc[16 * c + i + 1] = fmaf(__uint_as_float(o[i + 1]), f.y, acc[16 * c + i + 1]);
              acc[16 * c + i + 2] = fmaf(__uint_as_float(o[i + 2]), f.z, acc[16 * c + i + 2]);
              acc[16 * c + i + 3] = fmaf(__uint_as_float(o[i + 3]), f.w, acc[16 * c + i + 3]);
            }
          }
        }
        ptx::tc_fence_before();
      };
      for (int j = job.j0; j < job.j1; ++j, ++g) {
        const int stage = g % C::kStages, buf = g & 1;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_full[buf]), (g >> 1) & 1, abort_ptr, p.timeout_ns,
                                kRolePagedSoftmax);
        if (ok)
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_v_full[stage]), (g / C::kStages) & 1, abort_ptr, p.timeout_ns,
                                  kRolePagedSoftmax);
        ptx::tc_fence_after();
        const int key = j * 128 + tid;
        const bool masked = (j + 1) * 128 > all_see;
        const uint32_t tS = tS0 + buf * N;
        float v_top = 0.f, k_sc = 0.f, v_log = 0.f, v_out = 1.f;
        if (ok) {
          const float4 a = *reinterpret_cast<const float4*>(&page_scale[stage][1][0]);
          const float4 b = *reinterpret_cast<const float4*>(&page_scale[stage][1][4]);
          v_top = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
          k_sc = page_scale[stage][0][page_slot];
          // The key's V scale relative to the tile's largest; below 2^-60 it counts as that.
          const float rel = page_scale[stage][1][page_slot] / (v_top > 0.f ? v_top : 1.f);
          v_log = rel < 8.673617379884035e-19f ? -60.f : ptx::lg2_approx(rel);
          v_out = ptx::ex2_approx(-v_log);
        }
        auto scores = [&](int c, float (&x)[16]) {
          uint32_t s[16];
          ptx::tmem_ld16(tS + 16 * c, s);
          ptx::tmem_ld_wait();
          ptx::reg_fence16(s);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&row_scale[16 * c + i]);
            x[i] = fmaf(__uint_as_float(s[i]), f.x * k_sc, v_log);
            x[i + 1] = fmaf(__uint_as_float(s[i + 1]), f.y * k_sc, v_log);
            x[i + 2] = fmaf(__uint_as_float(s[i + 2]), f.z * k_sc, v_log);
            x[i + 3] = fmaf(__uint_as_float(s[i + 3]), f.w * k_sc, v_log);
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (key >= row_lim[16 * c + i]) x[i] = -INFINITY;
          }
        };
        if (ok) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (c < nch) {
              float x[16];
              scores(c, x);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = ptx::warp_max_nan(x[i]);
              if (lane == 0) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                  *reinterpret_cast<float4*>(&red[warp][16 * c + i]) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
              }
            }
          }
          if (tid == 0) corr_any[buf] = 0;
          // V rows behind the unit's keys may hold anything, and a weight of zero does not cancel a NaN.
          if (key >= job.n_keys) {
            uint4* row = reinterpret_cast<uint4*>(generic + (sKV - smem_base) + (2 * stage + 1) * C::kTileBytes + tid * HD);
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        stop = ptx::softmax_any(!ok);
        if (stop) break;
        if (tid < 16 * nch) {
          const float m = ptx::max_nan(ptx::max_nan(red[0][tid], red[1][tid]), ptx::max_nan(red[2][tid], red[3][tid])) -
                          kPagedTop;
          float fac = 0.f, corr = 1.f;
          if (m != -INFINITY) {
            if (!(m - ref <= kPagedJump)) {            // (also the first tile with keys, and NaN)
              corr = ptx::ex2_approx(ref - m);
              if (ref != -INFINITY) corr_any[buf] = 1;
              ref = m;
            }
            fac = ptx::ex2_approx(m - ref);
          }
          row_max[tid] = m == -INFINITY ? 0.f : m;
          row_fac[tid] = fac;
          row_fac_o[buf][tid] = fac * v_top;
          row_corr[buf][tid] = corr;
        }
        // O^T of the tile before, while the maxima are joined
        if (j > job.j0) {
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_o_full), (g - 1) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
          if (ok) add_tile(buf ^ 1);
        }
        stop = ptx::softmax_any(!ok);
        if (stop) break;
        const bool corr = corr_any[buf] != 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c < nch) {
            float x[16];
            scores(c, x);
            uint32_t hi4[4], lo4[4];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 m = *reinterpret_cast<const float4*>(&row_max[16 * c + i]);
              const float4 f = *reinterpret_cast<const float4*>(&row_fac[16 * c + i]);
              float w[4] = {ptx::ex2_approx(x[i] - m.x), ptx::ex2_approx(x[i + 1] - m.y),
                            ptx::ex2_approx(x[i + 2] - m.z), ptx::ex2_approx(x[i + 3] - m.w)};
              if (corr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) lsum[16 * c + i + e] *= row_corr[buf][16 * c + i + e];
              }
              lsum[16 * c + i] = fmaf(w[0], f.x * v_out, lsum[16 * c + i]);
              lsum[16 * c + i + 1] = fmaf(w[1], f.y * v_out, lsum[16 * c + i + 1]);
              lsum[16 * c + i + 2] = fmaf(w[2], f.z * v_out, lsum[16 * c + i + 2]);
              lsum[16 * c + i + 3] = fmaf(w[3], f.w * v_out, lsum[16 * c + i + 3]);
              float h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = __uint_as_float(__float_as_uint(w[e]) & 0xfff00000u);
              hi4[i / 4] = to_e4m3x2(h[0], h[1]) | to_e4m3x2(h[2], h[3]) << 16;
              lo4[i / 4] = to_e4m3x2(w[0] - h[0], w[1] - h[1]) | to_e4m3x2(w[2] - h[2], w[3] - h[3]) << 16;
            }
            // [16 rows][key][16 bytes]: N-major without swizzle
            uint4* at = reinterpret_cast<uint4*>(generic + c * 2048 + tid * 16);
            *at = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
            *reinterpret_cast<uint4*>(generic + C::kPBytes + c * 2048 + tid * 16) =
                make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full));
      }
      if (stop) break;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_o_full), (g - 1) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
      stop = ptx::softmax_any(!ok);
      if (stop) break;
      add_tile((g - 1) & 1);
      // The sums of weights over the 128 threads.
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c < nch) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = lsum[16 * c + i];
          const float l = lanes_sum16(v, lane);
          if (lane < 16) red[warp][16 * c + lane] = l;
        }
      }
      ptx::softmax_any(false);
      if (tid < 16 * nch) {
        const float l = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
        const bool none = l == 0.f;
        row_max[tid] = none ? 0.f : 1.f / l;
        const float lse = none ? -INFINITY : (ref + __log2f(l)) * 0.69314718055994530942f;
        if (tid < job.rows) {
          if (job.slot >= 0) {
            p.Lp[static_cast<size_t>(job.slot) * N + tid] = lse;
          } else {
            const int ti = tid / job.heads;
            p.lse[static_cast<long long>(job.head + tid - ti * job.heads) * sh.T_q + job.token + ti] = lse;
          }
        }
      }
      ptx::softmax_any(false);
      if (tid < HD) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c < nch) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = 16 * c + i;
              if (r < job.rows) {
                const float o = acc[r] * row_max[r];
                if (job.slot >= 0) {
                  p.Op[(static_cast<size_t>(job.slot) * N + r) * HD + tid] = o;
                } else {
                  const int ti = r / job.heads;
                  p.o[(job.token + ti) * p.o_t + (job.head + r - ti * job.heads) * p.o_h + tid] = __float2bfloat16(o);
                }
              }
            }
          }
        }
      }
      ptx::softmax_any(false);      // (row_max and red are used again)
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t policy = p.keep ? ptx::policy_evict_last() : ptx::policy_evict_first();
    const int per_tile = 128 >> sh.page_shift, in_page = 1 << sh.page_shift;
    int it = 0, loads = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, kUnitWaits * p.timeout_ns,
                              kRolePagedProducer);
      if (!ok) break;
      const PagedJob job = jobs[n & 1];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (job.b < 0) break;
      const int* table = p.table + static_cast<long long>(job.b) * sh.max_pages;
      const int entries = (job.n_keys + in_page - 1) >> sh.page_shift;
      int id = -1, id_next = -1;
      float sk = 0.f, sv = 0.f;
      // One lane a page: its number, and then its scales; the next 32 are asked for a batch ahead.
      auto entry = [&](int e) { return e < entries ? table[e] : -1; };
      id_next = entry(job.j0 * per_tile + lane);
      for (int j = job.j0; j < job.j1 && ok; ++j, ++it) {
        const int in_batch = (j - job.j0) * per_tile & 31;
        if (in_batch == 0) {
          const int e = j * per_tile + lane;
          id = id_next;
          const bool good = id >= 0 && id < sh.num_pages;
          sk = sv = 0.f;
          if (e < entries) {
            if (good) {
              sk = p.k_scale[static_cast<long long>(id) * sh.H_kv + job.kvh];
              sv = p.v_scale[static_cast<long long>(id) * sh.H_kv + job.kvh];
            } else {
              paged_bad(job.b);
              id = sh.num_pages;            // outside the tensor: reads as zeros
            }
          } else {
            id = -1;
          }
          id_next = entry(e + 32);
        }
        const int stage = it % C::kStages;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_empty[stage]), ((it / C::kStages) & 1) ^ 1u, abort_ptr,
                                p.timeout_ns, kRolePagedProducer);
        if (!ok) break;
        const int slot = lane - in_batch;
        const bool mine = slot >= 0 && slot < per_tile;
        if (mine) {
          page_scale[stage][0][slot] = sk;
          page_scale[stage][1][slot] = sv;
        }
        const bool copy = mine && id >= 0;
        const int n_copies = __popc(__ballot_sync(0xffffffffu, copy));
        const uint32_t bytes = static_cast<uint32_t>(n_copies) << sh.page_shift;
        const uint32_t k_full = ptx::smem_u32(&bar_k_full[stage]), v_full = ptx::smem_u32(&bar_v_full[stage]);
        __syncwarp();
        const bool drop_k = 2 * it == p.drop_load, drop_v = 2 * it + 1 == p.drop_load;   // test hook
        if (lane == 0) {
          if (!drop_k) ptx::mbar_arrive_expect_tx(k_full, bytes * HD);
          if (!drop_v) ptx::mbar_arrive_expect_tx(v_full, bytes * HD);
        }
        __syncwarp();
        if (copy) {
          const uint32_t to = sKV + 2 * stage * C::kTileBytes + (static_cast<uint32_t>(slot * HD) << sh.page_shift);
          if (!drop_k) ptx::tma_load_4d(to, &tmK, k_full, 0, 0, job.kvh, id, policy);
          if (!drop_v) ptx::tma_load_4d(to + C::kTileBytes, &tmV, v_full, 0, 0, job.kvh, id, policy);
        }
        __syncwarp();
        loads = it + 1;
      }
    }
    if (__any_sync(0xffffffffu, !ok || *abort_ptr)) {
      for (int i = loads > C::kStages ? loads - C::kStages : 0; i < loads; ++i) {
        if (2 * i != p.drop_load) drain_wait(ptx::smem_u32(&bar_k_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
        if (2 * i + 1 != p.drop_load)
          drain_wait(ptx::smem_u32(&bar_v_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t dq = ptx::desc_of(sQ, 16, C::kAtom, C::kSwizzle);
    const uint64_t dp = ptx::desc_of(sP, 128, 2048, 0);
    bool ok = true;
    int g0 = 0;             // tiles of the jobs before
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, kUnitWaits * p.timeout_ns,
                              kRolePagedMma);
      if (!ok) break;
      const int b = jobs[n & 1].b, tiles = jobs[n & 1].j1 - jobs[n & 1].j0, rows = jobs[n & 1].rows;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (b < 0) break;
      const int nn = (rows + 15) & ~15;
      const uint32_t idesc_qk = ptx::idesc_e4m3_f32(128, 0, false, false) | static_cast<uint32_t>(nn >> 3) << 17;
      const uint32_t idesc_pv = ptx::idesc_e4m3_f32(128, 0, true, true) | static_cast<uint32_t>(nn >> 3) << 17;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_full), n & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
      // Step t: S of tile t, then O of tile t - 2 (whose weights are written meanwhile).
      auto qk = [&](int t) {
        const int g = g0 + t, stage = g % C::kStages;
        if (!wait_warp_or_abort(ptx::smem_u32(&bar_k_full[stage]), (g / C::kStages) & 1, abort_ptr, p.timeout_ns,
                                kRolePagedMma))
          return false;
        ptx::tc_fence_after();
        const uint64_t dk = ptx::desc_of(sKV + 2 * stage * C::kTileBytes, 16, C::kAtom, C::kSwizzle);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int k = 0; k < HD / 32; ++k)
            ptx::mma_f8_warp(tmem_base + C::kColS + (g & 1) * N, ptx::desc_lo(dk) + 2 * k, ptx::desc_hi(dk),
                             ptx::desc_lo(dq) + part * (C::kQBytes >> 4) + 2 * k, ptx::desc_hi(dq), idesc_qk,
                             part + k > 0 ? 1u : 0u);
        ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full[g & 1]));
        return true;
      };
      for (int t = 0; t < 2 && t < tiles && ok; ++t) ok = qk(t);
      for (int t = 0; t < tiles && ok; ++t) {
        const int g = g0 + t, stage = g % C::kStages;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full), g & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t dv = ptx::desc_of(sKV + (2 * stage + 1) * C::kTileBytes, C::kTileBytes, C::kAtom, C::kSwizzle);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::mma_f8_warp(tmem_base + C::kColO, ptx::desc_lo(dv) + k * (32 * HD >> 4), ptx::desc_hi(dv),
                             ptx::desc_lo(dp) + part * (C::kPBytes >> 4) + k * 32, ptx::desc_hi(dp), idesc_pv,
                             part + k > 0 ? 1u : 0u);
        ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full));
        ptx::mma_commit_warp(ptx::smem_u32(&bar_empty[stage]));
        if (t + 2 < tiles) ok = qk(t + 2);
      }
      g0 += tiles;
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------------ units
    if (lane == 0) {
      int x = x_begin, b = start_b, u = 0, i = 0, from = 0;
      PagedSeq q{};
      bool more = x < x_end && b < sh.B;
      if (more) {
        q = paged_seq(p, b);
        const int places = q.places(sh), y = x - start_cum * copies;
        more = places > 0 && y >= 0 && y < places * copies;
        if (more) {
          u = y / places;
          const int rem = y - u * places;
          int lo = q.first, hi = q.groups;           // before(lo) <= rem < before(hi)
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (q.before(sh, mid) <= rem) lo = mid;
            else hi = mid;
          }
          i = lo;
          from = rem - q.before(sh, i);
        }
      }
      for (int n = 0;; ++n) {
        PagedJob job;
        job.b = -1;
        int end = 0;
        while (more && x < x_end && job.b < 0) {
          const int keys = q.keys(sh, i), tiles = (keys + 127) >> 7, places = kPagedCost + tiles;
          // (Only lengths that change under the call can lead out of the unit. It ends then, with undefined results.)
          if (keys <= 0 || from >= places) {
            more = false;
            break;
          }
          const int to = min(places, from + (x_end - x));
          end = x - from + places - 1;               // the unit's last place
          x += to - from;
          job.j0 = max(0, from - kPagedCost);
          job.j1 = max(0, to - kPagedCost);
          if (job.j1 > job.j0) {
            const int kvh = u / sh.ht, h0 = (u - kvh * sh.ht) * sh.hp, t0 = i * sh.tp;
            job.b = b;
            job.kvh = kvh;
            job.token = q.c0 + t0;
            job.head = kvh * sh.G + h0;
            job.heads = min(sh.hp, sh.G - h0);
            job.rows = job.heads * min(sh.tp, q.n_q - t0);
            job.lim0 = sh.causal ? q.n_kv - q.n_q + t0 + 1 : q.n_kv;
            job.n_keys = keys;
            job.slot = job.j0 == 0 && job.j1 == tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (job.j0 == 0 ? 1 : 0);
          }
          from = to;
          if (to == places) {                        // on to the next unit
            from = 0;
            if (++i == q.groups) {
              i = q.first;
              if (++u == copies) {
                u = 0;
                do {
                  if (++b >= sh.B) break;
                  q = paged_seq(p, b);
                } while (q.first >= q.groups);
                more = b < sh.B;
                i = q.first;
              }
            }
          }
        }
        if (!wait_or_abort(ptx::smem_u32(&bar_job_empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr,
                           kUnitWaits * p.timeout_ns, kRolePagedWalk))
          break;
        jobs[n & 1] = job;
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[n & 1]));
        if (job.b < 0) break;
        if (job.slot >= 0 && job.j0 == 0) {
          PagedSplit s{};
          s.n = line_owner(total, sh.ctas, end) - static_cast<int>(blockIdx.x) + 1;
          s.token = job.token;
          s.head = job.head;
          s.heads = job.heads;
          s.rows = job.rows;
          p.split[blockIdx.x] = s;
        }
      }
    }
    __syncwarp();
  }

  // The merge may be scheduled now; it waits for this grid's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace fa
