// Exact attention of new tokens over a paged cache held in 8 bits (e4m3 with a
// scale for each page and K/V head), for units of few rows: single tokens of a
// batch of answers, a few drafted tokens. sm_103a, tcgen05 (8-bit operands) +
// TMEM + TMA.
//
// 8-bit operands on both sides. K and V go from memory to the tensor core as
// they are stored; no thread converts them. The other operand, a bf16 query row
// or a row of probabilities, enters as the sum of two e4m3 numbers, its first
// four significant bits and the rest to four more (hi, lo), side by side among the
// 16 rows of the products; the reader adds the two halves of S and of O. bf16 has
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
// (relative to the larger one of its warp's pages, of which there are two where pages have
// 16 rows) is added to the exponent, so P carries it. The weight itself is exponentiated once more. O is
// relative to the maximum of score + log2 V scale, the sum of weights to one of the scores, so V
// scales may differ by any factor.
//
// Work: see fa_paged_common.cuh. Rows of a unit are consecutive tokens x the heads of a
// group, row = token * heads + head; N (4 or 8) bounds them. One stream of
// tiles runs through a CTA's units: the next unit's S is computed and its
// first P written before the last O^T of a unit is added and its rows stored.
//
// What bounds it. Long caches: memory (eight answers to 32768 tokens, 8 K/V
// heads of 128: 51 us, 5.4 TB/s, 0.80 of a copy, of which 3 us go by before the first
// tiles are there and 1.5 in the merge). 64 answers of 1 to 8192 tokens: 28.8 us,
// 3.6 TB/s: unit boundaries, which two small CTAs per SM hide in part. Two answers of
// 500 tokens: 9.5 us, latencies alone (a cold instruction cache, the line, the
// table, the first tile, its chain, the merge).
//
// Per CTA (224 threads, two CTAs per SM): warps 0-3 softmax and sums, warp 4
// walks the line and loads pages, warp 5 issues products, warp 6 prepares query rows.
// 128 registers a thread; with N = 8 ptxas spills 20 bytes.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

namespace ptx {
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld8(taddr, r);
  else tmem_ld16(taddr, r);
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
  static constexpr int kThreads = 224;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kStages = HD == 128 ? 3 : 5;    // pairs of tiles
  static constexpr int kTiles = 2 * kStages;
  static constexpr int kTileBytes = 128 * HD;          // K or V
  static constexpr int kCols = 2 * N;                  // columns of S and O^T that are read: hi, lo
  static constexpr int kPBytes = kRows * 128;
  static constexpr int kQBytes = kRows * HD;
  // With d = 64 the M side of V^T P^T is V's 64 columns and 64 lanes that nobody
  // reads, fed from the 8 KB behind the tile: the last one has a pad.
  static constexpr int kPad = HD == 64 ? kTileBytes : 0;
  static constexpr int kSmemBytes = 2 * kPBytes + 2 * kQBytes + kStages * 2 * kTileBytes + kPad + 1024;
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
  constexpr int kJobs = kPagedJobs;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kTiles];    // K and V of a key tile in turn
  __shared__ __align__(8) uint64_t bar_empty[C::kTiles];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_o_full[2];
  __shared__ __align__(8) uint64_t bar_q_full[kJobs];   // (two, and a slow softmax warp could miss a phase)
  __shared__ __align__(8) uint64_t bar_q_empty[2];
  __shared__ __align__(8) uint64_t bar_sums;
  __shared__ __align__(8) uint64_t bar_job_full[kJobs];
  __shared__ __align__(8) uint64_t bar_job_empty[kJobs];
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PagedJob jobs[kJobs];
  __shared__ __align__(16) float page_scale[C::kStages][2][8];   // K, V scales of a tile's pages
  // By unit (modulo 4: written two units ahead of a reader) and row: the scores' scale over the query row's, keys seen.
  __shared__ __align__(16) float row_scale[4][N];
  __shared__ __align__(16) int row_lim[4][N];
  // By tile (modulo 4: a warp may be three tiles behind the first to write), warp and row: the maximum with the V
  // scale - kPagedTop.
  __shared__ __align__(16) float warp_max[4][4][N];
  __shared__ __align__(16) float factor[4][4][N];       // by reading warp: what the four O^T are multiplied by
  __shared__ __align__(16) float corr[4][N];
  __shared__ float sums[4][4][2][N];                    // by unit (modulo 4) and warp: sums of weights, what they are relative to
  __shared__ PagedLine line;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShape& sh = p.s;
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* generic = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
  const uint32_t sP = smem_base, sQ = sP + 2 * C::kPBytes, sKV = sQ + 2 * C::kQBytes;
  static_assert((2 * C::kPBytes) % 1024 == 0 && C::kQBytes % 1024 == 0, "tiles begin on swizzle atoms");

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kTiles; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_p_full[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_o_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_q_empty[t]), 1);
    }
    for (int t = 0; t < kJobs; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_q_full[t]), 32);
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 6);   // warps 0-3, 5 and 6
    }
    ptx::mbar_init(ptx::smem_u32(&bar_sums), 4);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 5) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  // (Rows that hold no query are multiplied, too; their results are not used. Of
  // pages above 16 rows only the first scales are ever written.)
  if (warp == 6) {
    for (int i = lane; i < 2 * C::kQBytes / 16; i += 32)
      reinterpret_cast<uint4*>(generic + (sQ - smem_base))[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = lane; i < C::kStages * 16; i += 32) (&page_scale[0][0][0])[i] = 0.f;
  }
  // The grid before ends; the merge may be scheduled (all CTAs are resident, so it takes no one's place).
  ptx::grid_wait();
  ptx::grid_next();
  if (threadIdx.x == 0) p.split[blockIdx.x].n = 0;
  if (sh.B > kPagedWarpSeqs) paged_line_block<C::kThreads>(p, &line);   // (else the loading warp does)
  ptx::tc_fence_before();
  __syncthreads();
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
    float acc[N];                                  // O^T of the unit, relative to ref
    float ref = kPagedNone;                        // of row lane % N, the same in all warps
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;

    // Adds the four O^T of tile `t` (of this CTA).
    auto add_tile = [&](int t) {
      const int buf = t & 1;
      // (Every warp has written its maxima when the tile's P is complete.)
      if (!wait_warp_or_abort(ptx::smem_u32(&bar_p_full[buf]), (t >> 1) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax))
        return false;
      // Lane l has (warp, row) = l / N, l % N.
      const float m = (&warp_max[t & 3][0][0])[min(lane, 4 * N - 1)];
      float top = m;
#pragma unroll
      for (int o = N; o < 4 * N; o <<= 1) top = ptx::max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool jump = !(top - ref <= kPagedJump);   // (also the first tile with keys, and NaN)
      if (__any_sync(0xffffffffu, jump)) {
        if (lane < N) corr[warp][lane] = jump ? ptx::ex2_approx(ref - top) : 1.f;
        if (jump) ref = top;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] *= corr[warp][i];
      }
      if (lane < 4 * N)
        (&factor[warp][0][0])[lane] = ptx::ex2_approx(m - ref);
      __syncwarp();
      if (!wait_warp_or_abort(ptx::smem_u32(&bar_o_full[buf]), (t >> 1) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax))
        return false;
      ptx::tc_fence_after();
      constexpr int kAtOnce = N == 8 ? 2 : 4;        // (registers)
#pragma unroll
      for (int w0 = 0; w0 < 4; w0 += kAtOnce) {
        uint32_t o[kAtOnce][C::kCols];
#pragma unroll
        for (int w = 0; w < kAtOnce; ++w) ptx::tmem_ld<C::kCols>(tO0 + (buf * 4 + w0 + w) * C::kRows, o[w]);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int w = 0; w < kAtOnce; ++w) {
          ptx::reg_fence<C::kCols>(o[w]);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float sum = __uint_as_float(o[w][i]) + __uint_as_float(o[w][N + i]);
            acc[i] = fmaf(sum, factor[warp][w0 + w][i], acc[i]);
          }
        }
      }
      __syncwarp();                                  // (factor is used again)
      return true;
    };

    // Ends unit `n`, whose tiles have been added.
    auto finish = [&](const PagedJob& job, int n) {
      if (!wait_warp_or_abort(ptx::smem_u32(&bar_sums), n & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax))
        return false;
      float inv = 0.f;                                 // of row lane
      if (lane < N) {
        float l = 0.f, r[4], n_ref = kPagedNone;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          r[w] = sums[n & 3][w][1][lane];
          n_ref = fmaxf(n_ref, r[w]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
          l = fmaf(sums[n & 3][w][0][lane], ptx::ex2_approx(r[w] - n_ref), l);
        const bool none = l == 0.f;
        const float total = n_ref + __log2f(l);
        inv = none ? 0.f : ptx::ex2_approx(ref - total);
        if (warp == 0 && lane < job.rows) {
          const float lse = none ? -INFINITY : total * 0.69314718055994530942f;
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
        acc[r] = 0.f;
      }
      ref = kPagedNone;
      return true;
    };

    bool ok = true;
    int g = 0;                                     // tiles so far
    PagedJob job{}, last{};
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedSoftmax);
      if (!ok) break;
      job = jobs[ring];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      const bool tiles = job.b >= 0;               // (the last job has none, but the unit before is still to be ended)
      if (tiles)
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_full[ring]), (n / kJobs) & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
      if (!ok) break;
      const int all_see = min(job.n_keys, job.lim0);   // keys that every row sees
      float lsum[N], lref[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lsum[i] = 0.f;
        lref[i] = kPagedNone;
      }
      int j = job.j0;
#pragma unroll 1
      do {
       if (tiles) {
        const int stage = g % C::kStages, buf = g & 1;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_full[buf]), (g >> 1) & 1, abort_ptr, p.timeout_ns,
                                kRolePagedSoftmax);
        if (ok)
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_full[2 * stage + 1]), (g / C::kStages) & 1, abort_ptr, p.timeout_ns,
                                  kRolePagedSoftmax);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[C::kCols];
        ptx::tmem_ld<C::kCols>(tS0 + buf * C::kRows, s);
        const int key = j * 128 + tid;
        const float k_sc = page_scale[stage][0][page_slot], v_sc = page_scale[stage][1][page_slot];
        // log2 of the larger V scale of the warp's pages (finite, or NaN), and of the key's relative to that.
        auto log = [](float v) { return ptx::max_nan(ptx::lg2_approx(v), -200.f); };
        float v_top = log(v_sc), v_log = 0.f;
        if (slot0 != slot1) {
          v_log = v_top;
          v_top = log(fmaxf(page_scale[stage][1][slot0], page_scale[stage][1][slot1]));
          v_log -= v_top;
        }
        // (Within 2^60 of each other the maximum of the sums does for the weights' reference, too; beyond, one
        // page's keys may be all that P holds and the other's all the weight, and the scores have a maximum of their own.)
        const bool apart = __any_sync(0xffffffffu, v_log < -60.f);
        ptx::tmem_ld_wait();
        ptx::reg_fence<C::kCols>(s);
        float x[N], m[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
          x[i] = fmaf(__uint_as_float(s[i]) + __uint_as_float(s[N + i]), row_scale[n & 3][i] * k_sc, v_log);
        if ((j + 1) * 128 > all_see) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (key >= row_lim[n & 3][i]) x[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = ptx::max_nan(ptx::warp_max_nan(x[i]) - kPagedTop, kPagedNone);
        if (lane == 0) {
          auto with_v = [&](float mi) { return mi == kPagedNone ? mi : mi + v_top; };
#pragma unroll
          for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4*>(&warp_max[g & 3][warp][i]) =
                make_float4(with_v(m[i]), with_v(m[i + 1]), with_v(m[i + 2]), with_v(m[i + 3]));
        }
        uint32_t hi4[N / 4], lo4[N / 4];
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          float w[4], h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mi = m[i + e];
            w[e] = ptx::ex2_approx(x[i + e] - mi);
            const float score = x[i + e] - v_log, ni = apart ? ptx::warp_max_nan(score) - kPagedTop : mi;
            if (!(ni - lref[i + e] <= kPagedJump)) {
              lsum[i + e] *= ptx::ex2_approx(lref[i + e] - ni);
              lref[i + e] = ni;
            }
            lsum[i + e] += ptx::ex2_approx(score - lref[i + e]);
            h[e] = __uint_as_float(__float_as_uint(w[e]) & 0xfff00000u);
          }
          hi4[i / 4] = to_e4m3x2(h[0], h[1]) | to_e4m3x2(h[2], h[3]) << 16;
          lo4[i / 4] = to_e4m3x2(w[0] - h[0], w[1] - h[1]) | to_e4m3x2(w[2] - h[2], w[3] - h[3]) << 16;
        }
        // [key][16 bytes]: N-major without swizzle
        *reinterpret_cast<uint4*>(generic + buf * C::kPBytes + tid * 16) =
            N == 4 ? make_uint4(hi4[0], lo4[0], 0u, 0u) : make_uint4(hi4[0], hi4[N / 4 - 1], lo4[0], lo4[N / 4 - 1]);
        // V rows behind the unit's keys may hold anything, and a weight of zero does not cancel a NaN.
        if (key >= job.n_keys) {
          uint4* row = reinterpret_cast<uint4*>(generic + (sKV - smem_base) + (2 * stage + 1) * C::kTileBytes + tid * HD);
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[buf]));
       }
        // The tile before, meanwhile: the unit's, or the last of the unit before.
        if (g > 0) {
          ok = add_tile(g - 1);
          if (ok && j == job.j0) ok = finish(last, n - 1);
          if (!ok) break;
        }
        if (tiles) ++g;
      } while (++j < job.j1);
      if (!ok || !tiles) break;
      // The unit's sums of weights over the lanes (the last tile's products run meanwhile).
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lsum[i] += __shfl_xor_sync(0xffffffffu, lsum[i], o);
      }
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          sums[n & 3][warp][0][i] = lsum[i];
          sums[n & 3][warp][1][i] = lref[i];
        }
        ptx::mbar_arrive(ptx::smem_u32(&bar_sums));
      }
      last = job;
    }
  } else if (warp == 4) {
    paged_load<HD, C::kTiles, C::kStages, false>(p, &line, &tmK, &tmV, jobs, bar_job_full, bar_job_empty, bar_full, bar_empty,
                                          page_scale, sKV, abort_ptr);
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    // One stream of tiles over all units: S of tile g + 2 follows O of tile g,
    // whose S has been read when its P is there.
    constexpr uint32_t idesc_qk = ptx::idesc_e4m3_f32(128, 16, false, false);
    constexpr uint32_t idesc_pv = ptx::idesc_e4m3_f32(128, 16, true, true);
    bool ok = true, more = true;
    int n = -1, left = 0, gq = 0;            // unit of the next S, its tiles still to come, that S
    auto qk = [&]() {
      if (left == 0) {
        ++n;
        const int ring = n & (kJobs - 1);
        if (!wait_warp_or_abort(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                                kUnitWaits * p.timeout_ns, kRolePagedMma))
          return false;
        more = jobs[ring].b >= 0;
        left = jobs[ring].j1 - jobs[ring].j0;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
        if (!more) return true;
        if (!wait_warp_or_abort(ptx::smem_u32(&bar_q_full[ring]), (n / kJobs) & 1, abort_ptr, p.timeout_ns, kRolePagedMma))
          return false;
      }
      const int stage = gq % C::kStages;
      if (!wait_warp_or_abort(ptx::smem_u32(&bar_full[2 * stage]), (gq / C::kStages) & 1, abort_ptr, p.timeout_ns,
                              kRolePagedMma))
        return false;
      ptx::tc_fence_after();
      const uint64_t dk = ptx::desc_of(sKV + 2 * stage * C::kTileBytes, 16, C::kAtom, C::kSwizzle);
      const uint64_t dq = ptx::desc_of(sQ + (n & 1) * C::kQBytes, 16, C::kAtom, C::kSwizzle);
#pragma unroll
      for (int k = 0; k < HD / 32; ++k)
        ptx::mma_f8_warp(tmem_base + C::kColS + (gq & 1) * C::kRows, ptx::desc_lo(dk) + 2 * k, ptx::desc_hi(dk),
                         ptx::desc_lo(dq) + 2 * k, ptx::desc_hi(dq), idesc_qk, k > 0 ? 1u : 0u);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full[gq & 1]));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_empty[2 * stage]));
      ++gq;
      if (--left == 0) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[n & 1]));
      return true;
    };
    ok = qk();
    if (ok && more) ok = qk();
    for (int g = 0; ok && g < gq; ++g) {
      const int stage = g % C::kStages, buf = g & 1;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full[buf]), (g >> 1) & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint64_t dv = ptx::desc_of(sKV + (2 * stage + 1) * C::kTileBytes, C::kTileBytes, C::kAtom, C::kSwizzle);
      const uint64_t dp = ptx::desc_of(sP + buf * C::kPBytes, 128, 2048, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ptx::mma_f8_warp(tmem_base + C::kColO + (buf * 4 + k) * C::kRows, ptx::desc_lo(dv) + k * (32 * HD >> 4),
                         ptx::desc_hi(dv), ptx::desc_lo(dp) + k * 32, ptx::desc_hi(dp), idesc_pv, 0u);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[buf]));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_empty[2 * stage + 1]));
      if (more) ok = qk();
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------------ query rows, a unit ahead
    // As hi and lo in the swizzled K-major layout. A row has kLanes lanes, 16 elements each.
    constexpr int kLanes = HD / 16, kPass = 32 / kLanes, kPasses = (N + kPass - 1) / kPass;
    const int part = lane % kLanes;
    for (int n = 0;; ++n) {
      const int ring = n & (kJobs - 1);
      if (!wait_warp_or_abort(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr, kUnitWaits * p.timeout_ns,
                              kRolePagedQuery))
        break;
      const PagedJob job = jobs[ring];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (job.b < 0) break;
      uint4 v[kPasses][2];
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = k * kPass + lane / kLanes;
        v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
        if (r < job.rows) {
          const int ti = r / job.heads, hi = r - ti * job.heads;
          const __nv_bfloat16* src = p.q + (job.token + ti) * p.q_t + (job.head + hi) * p.q_h + 16 * part;
          v[k][0] = *reinterpret_cast<const uint4*>(src);
          v[k][1] = *reinterpret_cast<const uint4*>(src + 8);
        }
      }
      // The unit before the last has read its rows.
      if (!wait_warp_or_abort(ptx::smem_u32(&bar_q_empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedQuery))
        break;
      uint8_t* to = generic + (sQ - smem_base) + (n & 1) * C::kQBytes;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = k * kPass + lane / kLanes;
        float x[16];
        unpack8(v[k][0], x);
        unpack8(v[k][1], x + 8);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (fabsf(x[e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[e]));
          else x[e] = __uint_as_float(0x7fffffffu);
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // 2^up with the largest element in [128, 256)
        const int up = amax > 0.f ? max(-120, min(120, 134 - static_cast<int>(__float_as_uint(amax) >> 23))) : 0;
        const float scale = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        uint32_t hi4[4], lo4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi4[e] = lo4[e] = 0;
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const float a = x[4 * e + 2 * f] * scale, b = x[4 * e + 2 * f + 1] * scale;
            const uint32_t h = to_e4m3x2(a, b);
            const float2 back = from_e4m3x2(h);
            hi4[e] |= h << (16 * f);
            lo4[e] |= to_e4m3x2(a - back.x, b - back.y) << (16 * f);
          }
        }
        if (r < N) {
          auto at = [&](int row) {
            return static_cast<uint32_t>(row) * HD + ((part ^ (HD == 128 ? row & 7 : (row >> 1) & 3)) << 4);
          };
          *reinterpret_cast<uint4*>(to + at(r)) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(to + at(N + r)) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          if (part == 0) {
            row_scale[n & 3][r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            row_lim[n & 3][r] = r >= job.rows ? 0 : min(job.n_keys, sh.causal ? job.lim0 + r / job.heads : job.lim0);
          }
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bar_q_full[ring]));
    }
    __syncwarp();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace fa
