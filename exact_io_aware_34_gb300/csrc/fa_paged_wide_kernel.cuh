// Exact attention of new tokens over a paged 8-bit cache, for units of many
// rows: pieces of prompts. sm_103a, tcgen05 + TMEM + TMA.
//
// With hundreds of query rows per key the tensor core is what bounds the work,
// and fa_paged_kernel's transposed tiles, whose softmax needs a maximum over
// lanes, are in its way. Here a lane has a row, as in fa_varlen_fwd_kernel, and
// both products run in f16: an e4m3 number is exact in f16, a bf16 query row is
// too once a power of two has brought its largest element to [128, 256) (all
// but elements below 2^-25 of that), and P has eleven bits. Four warps convert
// the tiles of K and V from their 8-bit ring into a ring of f16 tiles in the
// tensor core's layout: 2 x 16 K elements for each 128 keys, beside products
// that take 2048 cycles for the unit's 256 rows.
//
// Scales. S times (row's scale x page's K scale) is a score in powers of two;
// log2 of the page's V scale is added to it, so P carries that scale and P V
// needs no other. The maximum that P is written against is that of these sums;
// a page's weights are summed apart and divided by its scale.
// P is written as at most 2^kWideTop times 2^kRescaleLog2 (the maximum moves
// lazily): f16 then resolves weights 2^-31 below the row's largest.
//
// Work: see fa_paged_common.cuh; a unit has up to 256 rows (row = token *
// heads + head), two tiles of 128, each with a softmax warpgroup. The update
// per key block is fa_varlen_fwd_kernel's.
//
// Per CTA (512 threads, one per SM): warps 0-7 softmax and epilogue, warp 8
// walks the line and loads pages, warp 9 issues products, warps 10 and 11 idle,
// warps 12-15 convert query rows and tiles.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

namespace ptx {
// tmem_ld32_max for 16 columns.
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, uint32_t (&r)[16], float& mx) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(mx)
      : "r"(taddr));
}
// Two floats to packed f16x2: `lo` in bits [0,16).
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A float from shared memory, read here (not kept from an earlier read).
__device__ __forceinline__ float lds(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
  return x;
}
// 16 bytes from global to shared memory, asynchronously; and all of this thread's have come.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
}  // namespace ptx

constexpr float kWideTop = 7.f;

template <int HD>
struct PagedWideCfg {
  static constexpr int kRows = 256;
  static constexpr int kThreads = 512;
  static constexpr int kChunks = HD / 64;              // 128-byte swizzle chunks of a row
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTileBytes = kChunks * kChunkBytes;   // f16
  static constexpr int kSlots = HD == 128 ? 3 : 6;     // f16 tiles
  static constexpr int kTiles = HD == 128 ? 3 : 6;     // 8-bit tiles
  static constexpr int kScales = 8;                    // pairs whose scales are held
  static constexpr int kSmemQ = 2 * kTileBytes;
  static constexpr int kSmemBytes = kSmemQ + kSlots * kTileBytes + kTiles * 128 * HD + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;                 // + 128 * tile
  static constexpr uint32_t kColO = 256;               // + HD * tile
  static constexpr int kRegsSoftmax = 184, kRegsOther = 72;
  static_assert(8 * kRegsSoftmax + 8 * kRegsOther <= 16 * 128, "register split exceeds the launch");
  // kind::f16 with f16 operands (format 0).
  static constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(128, 128, false, false) & ~(1u << 7 | 1u << 10);
  static constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, HD, false, true) & ~(1u << 7 | 1u << 10);
};

template <int HD>
__global__ void __launch_bounds__(PagedWideCfg<HD>::kThreads, 1)
    fa_paged_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const PagedParams p) {
  using C = PagedWideCfg<HD>;
  constexpr int kJobs = kPagedJobs;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kTiles];    // 8-bit tiles, K and V of a key tile in turn
  __shared__ __align__(8) uint64_t bar_empty[C::kTiles];
  __shared__ __align__(8) uint64_t bar_slot_full[C::kSlots];
  __shared__ __align__(8) uint64_t bar_slot_empty[C::kSlots];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_o_full[2];
  __shared__ __align__(8) uint64_t bar_q_full;
  __shared__ __align__(8) uint64_t bar_q_empty;
  __shared__ __align__(8) uint64_t bar_job_full[kJobs];
  __shared__ __align__(8) uint64_t bar_job_empty[kJobs];
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PagedJob jobs[kJobs];
  __shared__ __align__(16) float page_scale[C::kScales][4][8];
  __shared__ float row_scale[2][C::kRows];              // by unit (modulo 2)
  __shared__ PagedLine line;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShape& sh = p.s;
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* generic = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
  const uint32_t sQ = smem_base, sSlots = sQ + C::kSmemQ, sTiles = sSlots + C::kSlots * C::kTileBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kTiles; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_empty[s]), 4);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_slot_full[s]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_slot_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_p_full[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_o_full[t]), 1);
    }
    for (int t = 0; t < kJobs; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 13);   // warps 0-7, 9 and 12-15
    }
    ptx::mbar_init(ptx::smem_u32(&bar_q_full), 128);
    ptx::mbar_init(ptx::smem_u32(&bar_q_empty), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  for (int i = threadIdx.x; i < C::kScales * 32; i += C::kThreads) (&page_scale[0][0][0])[i] = 0.f;
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

  if (warp >= 8) ptx::setmaxnreg_dec<C::kRegsOther>();
  if (warp < 8) {
    // ------------------------------------------------------------ softmax + epilogue
    ptx::setmaxnreg_inc<C::kRegsSoftmax>();
    const int t = warp >> 2, quarter = warp & 3, row = t * 128 + quarter * 32 + lane;   // row of the unit
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem_base + lane_addr + C::kColS + 128 * t;
    const uint32_t tO = tmem_base + lane_addr + C::kColO + HD * t;
    bool ok = true;
    int g = 0, pair0 = 0, units = 0;         // key blocks of this tile so far; of the CTA before this unit; this tile's units
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedSoftmax);
      if (!ok) break;
      const PagedJob job = jobs[ring];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (job.b < 0) break;
      const int blocks = job.j1 - job.j0;
      if (t == 1 && job.rows <= 128) {       // no rows in this tile: it is not computed
        pair0 += blocks;
        continue;
      }
      const int ti = row / job.heads;
      const bool live = row < job.rows;
      // Rows that hold no query take the last token's limit, so that they do not mask what the others need not.
      const int seen = sh.causal ? max(0, min(job.n_keys, job.lim0 + min(ti, (job.rows - 1) / job.heads))) : job.n_keys;
      float m_use = -INFINITY, l = 0.f, q_scale = 0.f, v_ref = 0.f, v_unit = 1.f;   // V scale that O is in units of, and its log2
      for (int jj = 0; jj < blocks; ++jj, ++g) {
        const int j = job.j0 + jj, pair = pair0 + jj, itV = 2 * pair + 1;
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_slot_full[itV % C::kSlots]), (itV / C::kSlots) & 1, abort_ptr,
                                p.timeout_ns, kRolePagedSoftmax);
        if (ok)
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_full[t]), g & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
        if (!ok) break;
        ptx::tc_fence_after();
        if (jj == 0) q_scale = row_scale[n & 1][row];
        const int valid = seen - j * 128;
        // Scores past a row's limit become -inf in TMEM, in a short loop (see fa_varlen_fwd_kernel).
        if (!__all_sync(0xffffffffu, valid >= 128)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int v = valid - 32 * c;
            if (__all_sync(0xffffffffu, v >= 32)) continue;
            uint32_t r[32];
            ptx::tmem_ld32(tS + 32 * c, r);
            ptx::tmem_ld_wait();
            ptx::reg_fence32(r);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= v) r[i] = __float_as_uint(-INFINITY);
            ptx::tmem_st32(tS + 32 * c, r);
          }
          ptx::tmem_st_wait();
        }
        const uint32_t scales = ptx::smem_u32(page_scale[pair % C::kScales]);
        if (jj == 0) {
          float top = 0.f;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) top = fmaxf(top, ptx::lds(scales + 32 + 4 * c));
          v_ref = top > 0.f ? ptx::lg2_approx(top) : 0.f;
          v_unit = ptx::ex2_approx(v_ref);
        }
        // Per 16 keys: the factor of S (never zero, so that -inf stays), what is added
        // to it, and 2^- that. (Read again where they are needed: registers.)
        auto factor = [&](int c) {
          return ptx::max_nan(q_scale * ptx::lds(scales + 4 * (16 * c >> sh.page_shift)), 1.17549435e-38f);
        };
        auto offset = [&](int c) {           // (a scale of zero counts as 2^-60 of v_unit)
          return ptx::max_nan(ptx::lds(scales + 64 + 4 * (16 * c >> sh.page_shift)) - v_ref, -60.f);
        };
        // The maximum: keys 64-127 first, so that keys 0-63 are in registers afterwards
        // (all 128 scores and their weights would not fit; the others are read again).
        uint32_t s[4][16];
        float mt = -INFINITY;
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          float mr[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::tmem_ld16_max(tS + 64 * h + 16 * c, s[c], mr[c]);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ptx::reg_fence16(s[c]);
            ptx::reg_fence1(mr[c]);
            mt = fmaxf(mt, fmaf(mr[c], factor(4 * h + c), offset(4 * h + c)));
          }
        }
        float alpha = 1.f;
        bool rescale_o = false;
        if (m_use == -INFINITY) {
          m_use = mt;                        // (nothing but zeros has been added)
        } else {
          const bool need = mt - m_use > kRescaleLog2;
          if (need) {
            alpha = ptx::ex2_approx(m_use - mt);
            m_use = mt;
          }
          rescale_o = need;
        }
        rescale_o = __any_sync(0xffffffffu, rescale_o);
        const float neg_m = m_use == -INFINITY ? 0.f : kWideTop - m_use;
        float sum = 0.f;
        uint32_t pk[32];
        auto exponents = [&](int c) {        // of keys 16 c .., whose scores are in s[c % 4]
          const float a = factor(c), off = offset(c) + neg_m;
          const uint64_t a2 = ptx::f2_pack(a, a), off2 = ptx::f2_pack(off, off);
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float x0, x1;
            ptx::f2_unpack(
                ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[c & 3][i]), __uint_as_float(s[c & 3][i + 1])), a2, off2), x0, x1);
            const float p0 = ptx::ex2_approx(x0), p1 = ptx::ex2_approx(x1);
            acc[(i >> 1) & 1] = ptx::f2_add(acc[(i >> 1) & 1], ptx::f2_pack(p0, p1));
            pk[(c & 3) * 8 + (i >> 1)] = ptx::pack_f16x2(p0, p1);
          }
          float s0, s1;
          ptx::f2_unpack(ptx::f2_add(acc[0], acc[1]), s0, s1);
          sum = fmaf(s0 + s1, fminf(ptx::lds(scales + 96 + 4 * (16 * c >> sh.page_shift)) * v_unit, 1.152921504606847e18f), sum);
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) exponents(c);
        ptx::tmem_st32(tS, pk);
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld16(tS + 64 + 16 * c, s[c]);
        if (rescale_o && jj > 0) {
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            ptx::tmem_ld32(tO + 32 * c, o);
            ptx::tmem_ld_wait();
            ptx::reg_fence32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            ptx::tmem_st32(tO + 32 * c, o);
          }
        }
        ptx::tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::reg_fence16(s[c]);
#pragma unroll
        for (int c = 4; c < 8; ++c) exponents(c);
        l = l * alpha + sum;
        ptx::tmem_st32(tS + 32, pk);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[t]));
      }
      if (!ok) break;
      pair0 += blocks;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_o_full[t]), units++ & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      const bool none = l == 0.f;
      const float inv = none ? 0.f : v_unit / l;
      const float lse = none ? -INFINITY : (m_use - kWideTop + __log2f(l)) * 0.69314718055994530942f;
      const int head = job.head + row - ti * job.heads, token = job.token + ti;
      if (live) {
        if (job.slot >= 0) p.Lp[static_cast<size_t>(job.slot) * C::kRows + row] = lse;
        else p.lse[static_cast<long long>(head) * sh.T_q + token] = lse;
      }
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(tO + 32 * c, o);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(o);
        if (!live) continue;
        if (job.slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.Op + (static_cast<size_t>(job.slot) * C::kRows + row) * HD + 32 * c);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                 __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.o + token * p.o_t + head * p.o_h + 32 * c);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = none ? 0u : ptx::pack_bf16x2(__uint_as_float(o[8 * v + 2 * e]) * inv, __uint_as_float(o[8 * v + 2 * e + 1]) * inv);
            dst[v] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      ptx::tc_fence_before();
    }
  } else if (warp == 8) {
    paged_load<HD, C::kTiles, C::kScales, true>(p, &line, &tmK, &tmV, jobs, bar_job_full, bar_job_empty, bar_full, bar_empty,
                                          page_scale, sTiles, abort_ptr);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    int it0 = 0;                             // tiles (K and V) of the units before
    int g[2] = {0, 0};                       // key blocks of each row tile so far
    auto slot_wait = [&](int it) {
      return wait_warp_or_abort(ptx::smem_u32(&bar_slot_full[it % C::kSlots]), (it / C::kSlots) & 1, abort_ptr,
                                p.timeout_ns, kRolePagedMma);
    };
    const uint32_t idesc_qk = C::kIdescQK | (p.negate ? ptx::kIdescNegateA : 0u);
    auto qk = [&](int t, int it) {
      const uint64_t a = ptx::desc_kmajor_sw128(sQ + t * C::kTileBytes);
      const uint64_t b = ptx::desc_kmajor_sw128(sSlots + (it % C::kSlots) * C::kTileBytes);
      const uint32_t d = tmem_base + C::kColS + 128 * t;
      if constexpr (HD == 128)
        ptx::mma_ss_k128_warp(d, ptx::desc_lo(a), ptx::desc_lo(b), ptx::desc_hi(a), idesc_qk, 0u);
      else
        ptx::mma_ss_k64_warp(d, ptx::desc_lo(a), ptx::desc_lo(b), ptx::desc_hi(a), idesc_qk, 0u);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full[t]));
      ++g[t];
    };
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedMma);
      if (!ok) break;
      const int b = jobs[ring].b, blocks = jobs[ring].j1 - jobs[ring].j0, nt = jobs[ring].rows > 128 ? 2 : 1;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (b < 0) break;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_full), n & 1, abort_ptr, p.timeout_ns, kRolePagedMma) && slot_wait(it0);
      if (!ok) break;
      ptx::tc_fence_after();
      // (Every P of the unit before has been waited for, so S is free; its O is read before this unit's first P.)
      for (int t = 0; t < nt; ++t) qk(t, it0);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_slot_empty[it0 % C::kSlots]));
      if (blocks == 1) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty));
      for (int jj = 0; jj < blocks && ok; ++jj) {
        const int itV = it0 + 2 * jj + 1, itK = itV + 1;
        const bool last = jj + 1 == blocks;
        for (int t = 0; t < nt && ok; ++t) {
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full[t]), (g[t] - 1) & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
          if (ok && t == 0) ok = slot_wait(itV);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t v = ptx::desc_mnmajor_sw128(sSlots + (itV % C::kSlots) * C::kTileBytes, C::kChunkBytes);
          ptx::mma_ts_k128_warp<32>(tmem_base + C::kColO + HD * t, tmem_base + C::kColS + 128 * t, ptx::desc_lo(v),
                                    ptx::desc_hi(v), C::kIdescPV, jj > 0 ? 1u : 0u);
          if (last) {
            ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[t]));
            continue;
          }
          if (t == 0) {
            ok = slot_wait(itK);
            if (!ok) break;
            ptx::tc_fence_after();
          }
          qk(t, itK);
        }
        if (!ok) break;
        ptx::mma_commit_warp(ptx::smem_u32(&bar_slot_empty[itV % C::kSlots]));
        if (!last) {
          ptx::mma_commit_warp(ptx::smem_u32(&bar_slot_empty[itK % C::kSlots]));
          if (jj + 2 == blocks) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty));
        }
      }
      it0 += 2 * blocks;
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ------------------------------------------------------------ conversion to f16
    const int tid = threadIdx.x - 384;
    bool ok = true;
    int it = 0;                              // tiles so far
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedQuery);
      if (!ok) break;
      const PagedJob job = jobs[ring];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (job.b < 0) break;
      // The tiles: a thread has a key's row.
      for (int j = job.j0; j < job.j1 && ok; ++j) {
        const bool clear = j * 128 + tid >= job.n_keys;   // (rows behind the unit's keys may hold anything)
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int tile = it % C::kTiles, slot = it % C::kSlots;
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_full[tile]), (it / C::kTiles) & 1, abort_ptr, p.timeout_ns,
                                  kRolePagedQuery);
          if (!ok) break;
          uint4 v[HD / 16];
          const uint8_t* from = generic + (sTiles - smem_base) + tile * 128 * HD + tid * HD;
#pragma unroll
          for (int i = 0; i < HD / 16; ++i)
            v[i] = *reinterpret_cast<const uint4*>(from + ((i ^ (HD == 128 ? tid & 7 : (tid >> 1) & 3)) << 4));
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_slot_empty[slot]), ((it / C::kSlots) & 1) ^ 1u, abort_ptr,
                                  p.timeout_ns, kRolePagedQuery);
          if (!ok) break;
          uint8_t* to = generic + (sSlots - smem_base) + slot * C::kTileBytes + tid * 128;
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h[2 * e] = e4m3x2_to_f16x2(w[e] & 0xffffu);
              h[2 * e + 1] = e4m3x2_to_f16x2(w[e] >> 16);
            }
            if (clear) {
#pragma unroll
              for (int e = 0; e < 8; ++e) h[e] = 0u;
            }
            uint8_t* chunk = to + (i >> 2) * C::kChunkBytes;
            const int u = 2 * (i & 3);
            *reinterpret_cast<uint4*>(chunk + ((u ^ (tid & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(chunk + (((u + 1) ^ (tid & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_empty[tile]));
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(ptx::smem_u32(&bar_slot_full[slot]));
          if (j > job.j0 || kv > 0) continue;
          // The query rows, behind the unit's first K tile: kLanes lanes a row, 16
          // elements each. They come as bf16 to where they will stand as f16 (all
          // at once: a loop of loads took 15000 cycles and more), and every thread
          // converts what it asked for.
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_empty), (n & 1) ^ 1u, abort_ptr, kUnitWaits * p.timeout_ns,
                                  kRolePagedQuery);
          if (!ok) break;
          constexpr int kLanes = HD / 16, kStep = 128 / kLanes;
          const int part = tid % kLanes, rows = job.rows <= 128 ? 128 : 256, u = 2 * (part & 3);
          // Row r of tile r / 128; 16-byte units 2 part and 2 part + 1, swizzled within their 128-byte chunk.
          auto place = [&](int r) {
            return static_cast<uint32_t>((r >> 7) * C::kTileBytes + (part >> 2) * C::kChunkBytes + (r & 127) * 128);
          };
          int ti = (tid / kLanes) / job.heads, hi = tid / kLanes - ti * job.heads;
#pragma unroll 1
          for (int r = tid / kLanes; r < job.rows; r += kStep) {
            const __nv_bfloat16* src = p.q + (job.token + ti) * p.q_t + (job.head + hi) * p.q_h + 16 * part;
            const uint32_t dst = sQ + place(r);
            ptx::cp_async16(dst + ((u ^ (r & 7)) << 4), src);
            ptx::cp_async16(dst + (((u + 1) ^ (r & 7)) << 4), src + 8);
            for (hi += kStep; hi >= job.heads; hi -= job.heads) ++ti;
          }
          ptx::cp_async_wait();
#pragma unroll 1
          for (int r = tid / kLanes; r < rows; r += kStep) {
            uint8_t* to0 = generic + place(r) + ((u ^ (r & 7)) << 4);
            uint8_t* to1 = generic + place(r) + (((u + 1) ^ (r & 7)) << 4);
            uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
            if (r < job.rows) {
              v0 = *reinterpret_cast<const uint4*>(to0);
              v1 = *reinterpret_cast<const uint4*>(to1);
            }
            float x[16], amax = 0.f;
            unpack8(v0, x);
            unpack8(v1, x + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (fabsf(x[e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[e]));
              else x[e] = __uint_as_float(0x7fffffffu);
            }
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int up = amax > 0.f ? max(-120, min(120, 134 - static_cast<int>(__float_as_uint(amax) >> 23))) : 0;
            const float scale = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = ptx::pack_f16x2(x[2 * e] * scale, x[2 * e + 1] * scale);
            *reinterpret_cast<uint4*>(to0) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(to1) = make_uint4(h[4], h[5], h[6], h[7]);
            if (part == 0) row_scale[n & 1][r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(ptx::smem_u32(&bar_q_full));
        }
      }
    }
    __syncwarp();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace fa
