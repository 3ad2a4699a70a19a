// Exact attention of new tokens over a paged cache held in 8 bits (e4m3 with a
// scale for each page and K/V head), for units of few rows: single tokens of a
// batch of answers, a few drafted tokens. sm_103a, tcgen05 (8-bit operands) +
// TMEM + TMA.
//
// 8-bit operands on both sides. K and V go from memory to the tensor core as
// they are stored; no thread converts them. The other operand, a bf16 query row
// or a row of probabilities, enters as the sum of two e4m3 numbers, its first
// four significant bits and the rest to four more (hi, lo): the products
// K (q_hi + q_lo) and V (p_hi + p_lo) accumulate in the same place. bf16 has
// eight significant bits: a query row, scaled by a power of two so that its
// largest element lies in [128, 256), is exact but for elements below 2^-9 of
// that (off by 2^-17 of it at most). A probability is cut to four bits and its
// rest rounded to four: off by at most 2^-8 of itself, as if rounded to bf16,
// or where it is small by 2^-17 of the largest among its 32 keys.
//
// Transposed tiles. A 128-key tile is the M side of both products,
//   S^T[key, row] = K Q^T,    O^T[column, row] = V^T P^T,
// so that few query rows (the N side, 16) leave no lane of the softmax idle: a
// thread has one key and all rows. V is read as it lies (M-major).
//
// A warp for itself. The K side of one 8-bit product is 32 keys: the keys of
// one warp. So each of the four warps takes its rows' maxima over its own 32
// lanes alone (redux.sync), writes its P relative to them, and has its own
// O^T in tensor memory; every 32 keys have 8 bits for themselves, however far
// below the row's largest weight they lie. The four O^T are added to a sum in
// registers (a thread has one column of O for all rows) by the factors
// 2^(warp's maximum - reference). The sums of weights stay per thread until the
// unit's end. Within a tile no warp waits for another but through the
// tensor core, and the O^T of a tile are added after the next tile's P
// is written: the products' latency is never waited for.
//
// Scales. A key's score is S times its page's K scale; log2 of its V scale
// (relative to the larger one of its warp's pages) is added to the exponent, so
// P carries it, and is taken out of the sum of weights again.
//
// Work: see fa_paged_common.cuh. Rows of a unit are consecutive tokens x the heads of a
// group, row = token * heads + head; N (4, 8 or 16) bounds them.
//
// Per CTA (256 threads, two CTAs per SM): warps 0-3 softmax and sums, warp 4
// TMA producer, warp 5 MMA issuer, warp 6 walks the line, warp 7 idle.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

namespace ptx {
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else if constexpr (N == 8) {
    tmem_ld8(taddr, r);
  } else {
    tmem_ld16(taddr, r);
  }
}
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
}  // namespace ptx

template <int HD, int N>
struct PagedCfg {
  static constexpr int kRows = 16;                     // the N side of the products
  static constexpr int kThreads = 256;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kStages = HD == 128 ? 3 : 5;    // pairs of tiles
  static constexpr int kTileBytes = 128 * HD;          // K or V
  static constexpr int kPBytes = kRows * 128;          // hi or lo
  static constexpr int kQBytes = kRows * HD;
  // With d = 64 the M side of V^T P^T is V's 64 columns and 64 lanes that nobody
  // reads, fed from the 8 KB behind the tile: the last one has a pad.
  static constexpr int kPad = HD == 64 ? kTileBytes : 0;
  static constexpr int kSmemBytes = 4 * kPBytes + 2 * kQBytes + kStages * 2 * kTileBytes + kPad + 1024;
  static constexpr uint32_t kTmemCols = 256;
  static constexpr uint32_t kColS = 0;                 // two buffers
  static constexpr uint32_t kColO = 2 * kRows;         // two buffers x four warps
  static constexpr uint32_t kSwizzle = HD == 128 ? 2 : 4;
  static constexpr uint32_t kAtom = 8 * HD;            // eight rows
  static_assert(kColO + 8 * kRows <= kTmemCols, "tensor memory");
  static_assert(2 * (kSmemBytes + 4 * 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int HD, int N>
__global__ void __launch_bounds__(PagedCfg<HD, N>::kThreads, PagedCfg<HD, N>::kCtasPerSm)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedParams p) {
  using C = PagedCfg<HD, N>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_k_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_v_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_o_full[2];
  __shared__ __align__(8) uint64_t bar_q_full;
  __shared__ __align__(8) uint64_t bar_job_full[2];
  __shared__ __align__(8) uint64_t bar_job_empty[2];
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PagedJob jobs[2];
  __shared__ __align__(16) float page_scale[C::kStages][2][8];   // K, V scales of a tile's pages
  __shared__ __align__(16) float row_scale[16];         // of S, by row: the scores' scale over the query row's
  __shared__ __align__(16) int row_lim[16];             // keys the row sees
  // By tile (modulo 4: a warp may be three tiles behind the first to write), warp and row: the maximum - kPagedTop.
  __shared__ __align__(16) float warp_max[4][4][N];
  __shared__ float warp_top[4][4];                      // the larger V scale of the warp's pages
  __shared__ __align__(16) float factor[4][4][N];       // by reading warp: what the four O^T are multiplied by
  __shared__ __align__(16) float corr[4][N];
  __shared__ float sums[2][4][2][16];                   // by unit (modulo 2) and warp: sums of weights, what they are relative to
  __shared__ int warp_sum[C::kThreads / 32];
  __shared__ int start[2];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShape& sh = p.s;
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sP = smem_base, sQ = sP + 4 * C::kPBytes, sKV = sQ + 2 * C::kQBytes;
  static_assert((4 * C::kPBytes) % 1024 == 0 && (2 * C::kQBytes) % 1024 == 0, "tiles begin on swizzle atoms");

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_k_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_v_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_p_full[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_o_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 6);   // warps 0-5
    }
    ptx::mbar_init(ptx::smem_u32(&bar_q_full), 128);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    abort_flag = 0;
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
  ptx::tc_fence_before();
  const PagedLine line = paged_line<C::kThreads>(p, warp_sum, start);
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  volatile int* abort_ptr = &abort_flag;

  if (warp < 4) {
    // ------------------------------------------------------------ softmax and sums
    const int tid = threadIdx.x;                   // this thread's key of a tile, and its column of O
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS0 = tmem_base + lane_addr + C::kColS, tO0 = tmem_base + lane_addr + C::kColO;
    const int page_slot = tid >> sh.page_shift;
    const int slot0 = warp * 32 >> sh.page_shift, slot1 = (warp * 32 + 31) >> sh.page_shift;   // the warp's pages
    uint8_t* generic = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
    int g = 0;                                     // tiles so far
    for (int n = 0;; ++n) {
      bool ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr,
                                   kUnitWaits * p.timeout_ns, kRolePagedSoftmax);
      PagedJob job;
      job.b = -1;
      if (ok) {
        job = jobs[n & 1];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      }
      if (job.b >= 0) {
        // The query rows, as hi and lo in the swizzled K-major layout.
        constexpr int kLanes = HD / 16;            // threads of a row, 16 elements each
        const int part = tid % kLanes, r = tid / kLanes;
        if (r < 16) {
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
          const uint32_t at =
              static_cast<uint32_t>(r) * HD + ((part ^ (HD == 128 ? r & 7 : (r >> 1) & 3)) << 4);
          *reinterpret_cast<uint4*>(generic + (sQ - smem_base) + at) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(generic + (sQ - smem_base) + C::kQBytes + at) =
              make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          if (part == 0) {
            row_scale[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            row_lim[r] = live ? min(job.n_keys, sh.causal ? job.lim0 + ti : job.lim0) : 0;
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&bar_q_full));
      }
      // row_scale and row_lim stand. (All four warps leave together: a named barrier must not be left waiting.)
      if (ptx::softmax_any(job.b < 0)) break;
      const int all_see = min(job.n_keys, job.lim0);   // keys that every row sees

      float acc[N], lsum[N], lref[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc[i] = lsum[i] = 0.f;
        lref[i] = -INFINITY;
      }
      float ref = -INFINITY;                           // of row lane % N: what acc is relative to, the same in all warps
      // Adds the four O^T of tile `t` (of this CTA).
      auto add_tile = [&](int t) {
        const int buf = t & 1;
        // (The P of a tile is complete when every warp has written its maxima.)
        if (!wait_warp_or_abort(ptx::smem_u32(&bar_p_full[buf]), (t >> 1) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax))
          return false;
        {
          // Lane l has (warp, row) = l / N, l % N (and 32 more with N = 16).
          float m[N == 16 ? 2 : 1], top = -INFINITY;
#pragma unroll
          for (int k = 0; k < (N == 16 ? 2 : 1); ++k) {
            const int at = min(lane + 32 * k, 4 * N - 1);
            m[k] = (&warp_max[t & 3][0][0])[at];
            top = ptx::max_nan(top, m[k]);
          }
#pragma unroll
          for (int o = N; o < (N == 4 ? 16 : 32); o <<= 1) top = ptx::max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
          const bool jump = top != -INFINITY && !(top - ref <= kPagedJump);   // (also the first tile with keys, and NaN)
          if (__any_sync(0xffffffffu, jump)) {
            if (lane < N) corr[warp][lane] = jump ? ptx::ex2_approx(ref - top) : 1.f;
            if (jump) ref = top;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] *= corr[warp][i];
          }
#pragma unroll
          for (int k = 0; k < (N == 16 ? 2 : 1); ++k) {
            const int at = lane + 32 * k;
            if (at < 4 * N)
              (&factor[warp][0][0])[at] = m[k] == -INFINITY ? 0.f : ptx::ex2_approx(m[k] - ref) * warp_top[t & 3][at / N];
          }
          __syncwarp();
        }
        if (!wait_warp_or_abort(ptx::smem_u32(&bar_o_full[buf]), (t >> 1) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax))
          return false;
        ptx::tc_fence_after();
        constexpr int kAtOnce = N == 16 ? 1 : 4;       // (registers)
#pragma unroll
        for (int w0 = 0; w0 < 4; w0 += kAtOnce) {
          uint32_t o[kAtOnce][N];
#pragma unroll
          for (int w = 0; w < kAtOnce; ++w) ptx::tmem_ld<N>(tO0 + (buf * 4 + w0 + w) * C::kRows, o[w]);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int w = 0; w < kAtOnce; ++w) {
            ptx::reg_fence<N>(o[w]);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(__uint_as_float(o[w][i]), factor[warp][w0 + w][i], acc[i]);
          }
        }
        __syncwarp();                                  // (factor is used again)
        return true;
      };
      for (int j = job.j0; j < job.j1; ++j, ++g) {
        const int stage = g % C::kStages, buf = g & 1;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_full[buf]), (g >> 1) & 1, abort_ptr, p.timeout_ns,
                                kRolePagedSoftmax);
        if (ok)
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_v_full[stage]), (g / C::kStages) & 1, abort_ptr, p.timeout_ns,
                                  kRolePagedSoftmax);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[N];
        ptx::tmem_ld<N>(tS0 + buf * C::kRows, s);
        const int key = j * 128 + tid;
        const float k_sc = page_scale[stage][0][page_slot], v_sc = page_scale[stage][1][page_slot];
        // The key's V scale relative to the larger one of its warp's pages; below 2^-60 of that it counts as that.
        float v_top = v_sc, v_log = 0.f, v_out = 1.f;
        if (slot0 != slot1) {
          v_top = fmaxf(page_scale[stage][1][slot0], page_scale[stage][1][slot1]);
          const float rel = v_sc / (v_top > 0.f ? v_top : 1.f);
          v_log = rel < 8.673617379884035e-19f ? -60.f : ptx::lg2_approx(rel);
          v_out = ptx::ex2_approx(-v_log);
        }
        ptx::tmem_ld_wait();
        ptx::reg_fence<N>(s);
        float x[N], m[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fmaf(__uint_as_float(s[i]), row_scale[i] * k_sc, v_log);
        if ((j + 1) * 128 > all_see) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (key >= row_lim[i]) x[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = ptx::warp_max_nan(x[i]) - kPagedTop;
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4*>(&warp_max[g & 3][warp][i]) = make_float4(m[i], m[i + 1], m[i + 2], m[i + 3]);
          warp_top[g & 3][warp] = v_top;
        }
        uint32_t hi4[4] = {0u, 0u, 0u, 0u}, lo4[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          float w[4], h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mi = m[i + e];
            w[e] = ptx::ex2_approx(x[i + e] - (mi == -INFINITY ? 0.f : mi));
            if (mi != -INFINITY && !(mi - lref[i + e] <= kPagedJump)) {
              lsum[i + e] *= lref[i + e] == -INFINITY ? 0.f : ptx::ex2_approx(lref[i + e] - mi);
              lref[i + e] = mi;
            }
            const float f = mi == -INFINITY ? 0.f : ptx::ex2_approx(mi - lref[i + e]);
            lsum[i + e] = fmaf(w[e], f * v_out, lsum[i + e]);
            h[e] = __uint_as_float(__float_as_uint(w[e]) & 0xfff00000u);
          }
          hi4[i / 4] = to_e4m3x2(h[0], h[1]) | to_e4m3x2(h[2], h[3]) << 16;
          lo4[i / 4] = to_e4m3x2(w[0] - h[0], w[1] - h[1]) | to_e4m3x2(w[2] - h[2], w[3] - h[3]) << 16;
        }
        // [key][16 bytes]: N-major without swizzle
        uint8_t* to = generic + buf * 2 * C::kPBytes + tid * 16;
        *reinterpret_cast<uint4*>(to) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
        *reinterpret_cast<uint4*>(to + C::kPBytes) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
        // V rows behind the unit's keys may hold anything, and a weight of zero does not cancel a NaN.
        if (key >= job.n_keys) {
          uint4* row = reinterpret_cast<uint4*>(generic + (sKV - smem_base) + (2 * stage + 1) * C::kTileBytes + tid * HD);
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[buf]));
        if (j > job.j0 && !add_tile(g - 1)) {
          ok = false;
          break;
        }
      }
      if (ok) ok = add_tile(g - 1);
      // The unit's end: sums over lanes here, over warps by everyone.
      float l_me = 0.f, r_me = -INFINITY;              // of row lane (< N)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float l = lsum[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == i) {
          l_me = l;
          r_me = lref[i];
        }
      }
      if (lane < N) {
        sums[n & 1][warp][0][lane] = l_me;
        sums[n & 1][warp][1][lane] = r_me;
      }
      if (ptx::softmax_any(!ok)) break;
      float inv = 0.f;                                 // of row lane
      if (lane < N) {
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float r = sums[n & 1][w][1][lane];
          if (r != -INFINITY) l = fmaf(sums[n & 1][w][0][lane], ptx::ex2_approx(r - ref), l);
        }
        const bool none = l == 0.f;
        inv = none ? 0.f : 1.f / l;
        if (warp == 0 && lane < job.rows) {
          const float lse = none ? -INFINITY : (ref + __log2f(l)) * 0.69314718055994530942f;
          if (job.slot >= 0) {
            p.Lp[static_cast<size_t>(job.slot) * N + lane] = lse;
          } else {
            const int ti = lane / job.heads;
            p.lse[static_cast<long long>(job.head + lane - ti * job.heads) * sh.T_q + job.token + ti] = lse;
          }
        }
      }
      int ti = 0, hi = 0;
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const float o = acc[r] * __shfl_sync(0xffffffffu, inv, r);
        if (r < job.rows && tid < HD) {
          if (job.slot >= 0)
            p.Op[(static_cast<size_t>(job.slot) * N + r) * HD + tid] = o;
          else
            p.o[(job.token + ti) * p.o_t + (job.head + hi) * p.o_h + tid] = __float2bfloat16(o);
        }
        if (++hi == job.heads) {
          hi = 0;
          ++ti;
        }
      }
    }
  } else if (warp == 4) {
    paged_load<HD, C::kStages>(p, &tmK, &tmV, jobs, bar_job_full, bar_job_empty, bar_k_full, bar_v_full, bar_empty,
                               page_scale, sKV, abort_ptr);
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t dq = ptx::desc_of(sQ, 16, C::kAtom, C::kSwizzle);
    constexpr uint32_t idesc_qk = ptx::idesc_e4m3_f32(128, 16, false, false);
    constexpr uint32_t idesc_pv = ptx::idesc_e4m3_f32(128, 16, true, true);
    bool ok = true;
    int g0 = 0;             // tiles of the jobs before
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, kUnitWaits * p.timeout_ns,
                              kRolePagedMma);
      if (!ok) break;
      const int b = jobs[n & 1].b, tiles = jobs[n & 1].j1 - jobs[n & 1].j0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (b < 0) break;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_full), n & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
      // S of tile t + 2 follows O of tile t: its buffer has been read when P of tile t is there.
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
            ptx::mma_f8_warp(tmem_base + C::kColS + (g & 1) * C::kRows, ptx::desc_lo(dk) + 2 * k, ptx::desc_hi(dk),
                             ptx::desc_lo(dq) + part * (C::kQBytes >> 4) + 2 * k, ptx::desc_hi(dq), idesc_qk,
                             part + k > 0 ? 1u : 0u);
        ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full[g & 1]));
        return true;
      };
      for (int t = 0; t < 2 && t < tiles && ok; ++t) ok = qk(t);
      for (int t = 0; t < tiles && ok; ++t) {
        const int g = g0 + t, stage = g % C::kStages, buf = g & 1;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full[buf]), (g >> 1) & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t dv = ptx::desc_of(sKV + (2 * stage + 1) * C::kTileBytes, C::kTileBytes, C::kAtom, C::kSwizzle);
        const uint64_t dp = ptx::desc_of(sP + buf * 2 * C::kPBytes, 128, 2048, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int part = 0; part < 2; ++part)
            ptx::mma_f8_warp(tmem_base + C::kColO + (buf * 4 + k) * C::kRows, ptx::desc_lo(dv) + k * (32 * HD >> 4),
                             ptx::desc_hi(dv), ptx::desc_lo(dp) + part * (C::kPBytes >> 4) + k * 32, ptx::desc_hi(dp),
                             idesc_pv, part > 0 ? 1u : 0u);
        ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[buf]));
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
    if (lane == 0) paged_walk(p, line, jobs, bar_job_full, bar_job_empty, abort_ptr);
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
