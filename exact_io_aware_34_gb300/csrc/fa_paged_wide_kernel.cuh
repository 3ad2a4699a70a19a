// Exact attention of new tokens over a paged 8-bit cache, for units of many
// rows: pieces of prompts. sm_103a, tcgen05 + TMEM + TMA.
//
// With hundreds of query rows per key the tensor core is what bounds the work,
// and fa_paged_kernel's transposed tiles, whose softmax needs a maximum over
// lanes, are in its way. Here a lane has a row, as in fa_varlen_fwd_kernel.
// Q K^T takes K as it is stored, and a query row as two e4m3 numbers (see
// fa_paged_kernel.cuh: the cost of one bf16 product). P V runs in f16, in which
// e4m3 numbers are exact and P has eleven bits: four warps convert each V tile
// into the tensor core's layout, 16 K elements for each 128 keys, beside
// products that take 2048 cycles for the unit's 256 rows.
//
// Scales. S times (row's scale x page's K scale) is a score s in powers of two;
// log2 of the page's V scale v is added to it, so P = 2^(s + log2 v - m) carries that
// scale and P V needs no other. m is the maximum of s + log2 v, moved lazily: P is at most
// 2^kWideTop times 2^kRescaleLog2, and f16 resolves what is 2^-31 below the row's largest.
// The sum of weights needs another reference, as V scales may differ by any factor: it is
// sum 2^(s - n), n the maximum of s, moved like m. A page's part of it is its sum of P
// times 2^(m - log2 v - n), which stays at 2^60 where v is so small that f16 holds
// none of its P anyway (these then count as 2^-60 of their weight).
//
// Work: see fa_paged_common.cuh; a unit has up to 256 rows (row = token *
// heads + head), two tiles of 128, each with a softmax warpgroup. The update
// per key block is fa_varlen_fwd_kernel's.
//
// What bounds it: per key tile about 3200 cycles, of which 2048 are products, the
// rest the chain from S to P, which two row tiles hide in part; and about 10000
// cycles at a unit's beginning, mostly its query rows. Pieces of prompts of 1 to
// 1024 tokens on caches to 8192, 32 heads on 8, d = 128: 166 us, 848 TFLOP/s over
// the pairs that are seen (0.43 of the bf16 rate); on pages of 16 or 32 rows, where a tile has
// up to eight scales that are read again where they are needed, 188 us. ptxas
// spills 48 to 88 bytes of the 128 registers a thread. Keys converted to f16 as well
// took 207 us where keys in 8 bits took 188; transposed tiles with 64 rows 704.
//
// Per CTA (512 threads, one per SM): warps 0-7 softmax and epilogue, warp 8
// walks the line and loads pages, warp 9 issues products, warps 10 and 11 idle,
// warps 12-15 convert V tiles.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

namespace ptx {
// tmem_ld32_max for 16 columns, into r[O] .. r[O + 15].
template <int O>
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, uint32_t (&r)[32], float& mx) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=r"(r[O]), "=r"(r[O + 1]), "=r"(r[O + 2]), "=r"(r[O + 3]), "=r"(r[O + 4]), "=r"(r[O + 5]), "=r"(r[O + 6]),
        "=r"(r[O + 7]), "=r"(r[O + 8]), "=r"(r[O + 9]), "=r"(r[O + 10]), "=r"(r[O + 11]), "=r"(r[O + 12]),
        "=r"(r[O + 13]), "=r"(r[O + 14]), "=r"(r[O + 15]), "=f"(mx)
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

// NG: equal parts of a tile whose keys share their pages' scales, 2 for pages of 64
// rows and more, else 8.
template <int HD, int NG>
struct PagedWideCfg {
  static constexpr int kRows = 256;
  static constexpr int kThreads = 512;
  static constexpr int kChunks = HD / 64;              // 128-byte swizzle chunks of a row
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kSlotBytes = kChunks * kChunkBytes;   // a V tile in f16
  static constexpr int kSlots = HD == 128 ? 2 : 4;
  static constexpr int kTileBytes = 128 * HD;          // 8 bits
  static constexpr int kTiles = HD == 128 ? 4 : 8;     // (even: K and V tiles keep their places)
  static constexpr int kScales = 8;                    // pairs whose scales are held
  static constexpr int kSmemQ = 4 * kTileBytes;        // row tile, hi or lo
  static constexpr int kSmemBytes = kSmemQ + kSlots * kSlotBytes + kTiles * kTileBytes + 1024;
  static constexpr uint32_t kSwizzle = HD == 128 ? 2 : 4;
  static constexpr uint32_t kAtom = 8 * HD;            // eight rows of 8 bits
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;                 // + 128 * tile
  static constexpr uint32_t kColO = 256;               // + HD * tile
  static constexpr uint32_t kColP = HD == 64 ? 384 : kColS;  // + 64 or 128 * tile: over S only where there is no other place
  static constexpr uint32_t kStepP = HD == 64 ? 64 : 128;
  static constexpr int kRegsSoftmax = 184, kRegsOther = 72;
  static_assert(8 * kRegsSoftmax + 8 * kRegsOther <= 16 * 128, "register split exceeds the launch");
  // kind::f16 with f16 operands (format 0).
  static constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, HD, false, true) & ~(1u << 7 | 1u << 10);
  static constexpr uint32_t kIdescQK = ptx::idesc_e4m3_f32(128, 128, false, false);
};

template <int HD, int NG>
__global__ void __launch_bounds__(PagedWideCfg<HD, NG>::kThreads, 1)
    fa_paged_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const PagedParams p) {
  using C = PagedWideCfg<HD, NG>;
  constexpr int kJobs = kPagedJobs, kPolls = 8;   // (polls: as in the forward kernel)
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kTiles];    // 8-bit tiles, K and V of a key tile in turn
  __shared__ __align__(8) uint64_t bar_empty[C::kTiles];
  __shared__ __align__(8) uint64_t bar_slot_full[C::kSlots];
  __shared__ __align__(8) uint64_t bar_slot_empty[C::kSlots];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_p_half[2];          // weights of keys 0-63
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_o_full[2];
  __shared__ __align__(8) uint64_t bar_q_full[2];
  __shared__ __align__(8) uint64_t bar_job_full[kJobs];
  __shared__ __align__(8) uint64_t bar_job_empty[kJobs];
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PagedJob jobs[kJobs];
  __shared__ __align__(16) float page_scale[C::kScales][3][8];
  __shared__ float row_scale[C::kRows];
  __shared__ PagedLine line;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShape& sh = p.s;
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* generic = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
  const uint32_t sQ = smem_base, sSlots = sQ + C::kSmemQ, sTiles = sSlots + C::kSlots * C::kSlotBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kTiles; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_empty[s]), s & 1 ? 4 : 1);   // V: the converting warps, K: the products
    }
    for (int s = 0; s < C::kSlots; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_slot_full[s]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_slot_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_q_full[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_p_half[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_p_full[t]), 128);
      ptx::mbar_init(ptx::smem_u32(&bar_o_full[t]), 1);
    }
    for (int t = 0; t < kJobs; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 13);   // warps 0-7, 9 and 12-15
    }
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
  for (int i = threadIdx.x; i < C::kScales * 24; i += C::kThreads) (&page_scale[0][0][0])[i] = 0.f;
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
    const uint32_t tO = tmem_base + lane_addr + C::kColO + HD * t, tP = tmem_base + lane_addr + C::kColP + C::kStepP * t;
    bool ok = true;
    int g = 0, pair0 = 0, units = 0;         // key blocks of this tile so far; of the CTA before this unit; this tile's units
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedSoftmax);
      if (!ok) break;
      const PagedJob job = jobs[ring];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (job.b < 0) break;
      const int blocks = job.j1 - job.j0;
      const int inv_heads = (1 << 20) / job.heads + 1;   // (r * that) >> 20 = r / heads for r < 256
      if (t == 1 && job.rows <= 128) {       // no rows in this tile: it is not computed
        pair0 += blocks;
        continue;
      }
      // The warp's query rows, as hi and lo in the swizzled K-major layout: kLanes
      // lanes a row, 16 elements each. (This tile's products of the unit before
      // have all been waited for.)
      {
        constexpr int kLanes = HD / 16, kPass = 32 / kLanes, kPasses = 32 / kPass;
        const int part = lane % kLanes, r0 = t * 128 + quarter * 32 + lane / kLanes;
        // 16 bytes of hi, and kTileBytes behind them of lo; first they hold the bf16 (all
        // rows are asked for at once, asynchronously, and every lane converts what it asked
        // for; as short loops: unrolled, the code took longer to fetch than to run).
        auto place = [&](int r) {
          return static_cast<uint32_t>(2 * t * C::kTileBytes + (r & 127) * HD +
                                       ((part ^ (HD == 128 ? r & 7 : (r >> 1) & 3)) << 4));
        };
#pragma unroll 1
        for (int k = 0; k < kPasses; ++k) {
          const int r = r0 + k * kPass;
          if (r >= job.rows) break;
          const int ti = (r * inv_heads) >> 20;
          const __nv_bfloat16* src = p.q + (job.token + ti) * p.q_t + (job.head + r - ti * job.heads) * p.q_h + 16 * part;
          ptx::cp_async16(sQ + place(r), src);
          ptx::cp_async16(sQ + place(r) + C::kTileBytes, src + 8);
        }
        ptx::cp_async_wait();
#pragma unroll 1
        for (int k = 0; k < kPasses; ++k) {
          const int r = r0 + k * kPass;
          uint4* to0 = reinterpret_cast<uint4*>(generic + place(r));
          uint4* to1 = reinterpret_cast<uint4*>(generic + place(r) + C::kTileBytes);
          float x[16], amax = 0.f;
          unpack8(r < job.rows ? *to0 : make_uint4(0u, 0u, 0u, 0u), x);
          unpack8(r < job.rows ? *to1 : make_uint4(0u, 0u, 0u, 0u), x + 8);
#pragma unroll
          for (int e = 0; e < 16; ++e) amax = ptx::max_nan(amax, fabsf(x[e]));
          if (!(amax <= 3.402823466e38f)) {
            amax = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (fabsf(x[e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[e]));
              else x[e] = __uint_as_float(0x7fffffffu);
            }
          }
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
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
          *to0 = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *to1 = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          if (part == 0) row_scale[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bar_q_full[t]));
      __syncwarp();
      const float q_scale = row_scale[row];
      __syncwarp();                          // (written again for the next unit)
      const int ti = (row * inv_heads) >> 20;
      const bool live = row < job.rows;
      // Rows that hold no query take the last token's limit, so that they do not mask what the others need not.
      const int seen = sh.causal ? max(0, min(job.n_keys, job.lim0 + min(ti, (job.rows - 1) / job.heads))) : job.n_keys;
      float m_use = -INFINITY, n_use = -INFINITY, l = 0.f;   // what O and l are relative to
      for (int jj = 0; jj < blocks; ++jj, ++g) {
        const int j = job.j0 + jj, pair = pair0 + jj;
        // The scales come with V, so its slot is waited for, too, but behind S: the issuer has then seen every
        // earlier tile in its slot. Before that, the barrier of a warpgroup that skipped units may be
        // two phases behind, which its parity does not tell from done.
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_s_full[t]), g & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
        if (ok)
          ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_slot_full[pair % C::kSlots]), (pair / C::kSlots) & 1, abort_ptr,
                                  p.timeout_ns, kRolePagedSoftmax);
        if (!ok) break;
        ptx::tc_fence_after();
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
        uint32_t s[4][32];
        float mr[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (NG == 2) {
            ptx::tmem_ld32_max(tS + 32 * c, s[c], mr[c]);
          } else {
            ptx::tmem_ld16_max<0>(tS + 32 * c, s[c], mr[2 * c]);
            ptx::tmem_ld16_max<16>(tS + 32 * c + 16, s[c], mr[2 * c + 1]);
          }
        }
        // Per part: the factor of S (never zero, so that -inf stays) and log2 of the V scale (finite, or NaN).
        // Eight parts' are read again where they are needed (registers).
        const int part_shift = NG == 2 ? 6 : 4;
        auto factor = [&](int g) {
          return ptx::max_nan(q_scale * ptx::lds(scales + 4 * ((g << part_shift) >> sh.page_shift)), 1.17549435e-38f);
        };
        auto v_log = [&](int g) { return ptx::lds(scales + 64 + 4 * ((g << part_shift) >> sh.page_shift)); };
        float fa2[2], fb2[2];
        if constexpr (NG == 2) {
#pragma unroll
          for (int g2 = 0; g2 < 2; ++g2) {
            fa2[g2] = factor(g2);
            fb2[g2] = v_log(g2);
          }
        }
        ptx::tmem_ld_wait();
        float mt = -INFINITY, nt = -INFINITY;
        auto top = [&](float mx, float a, float log) {
          nt = fmaxf(nt, mx * a);
          mt = fmaxf(mt, fmaf(mx, a, log));
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ptx::reg_fence32(s[c]);
          ptx::reg_fence1(mr[NG == 2 ? c : 2 * c]);
          if constexpr (NG == 2) {
            top(mr[c], fa2[c >> 1], fb2[c >> 1]);
          } else {
            ptx::reg_fence1(mr[2 * c + 1]);
            top(mr[2 * c], factor(2 * c), v_log(2 * c));
            top(mr[2 * c + 1], factor(2 * c + 1), v_log(2 * c + 1));
          }
        }
        float alpha = 1.f;
        bool rescale_o = false;
        if (m_use == -INFINITY) {
          m_use = mt;                        // (nothing but zeros has been added)
          n_use = nt;
        } else if (fmaxf(mt - m_use, nt - n_use) > kRescaleLog2) {
          const float m_new = fmaxf(m_use, mt), n_new = fmaxf(n_use, nt);
          alpha = ptx::ex2_approx(m_use - m_new);
          l *= ptx::ex2_approx(n_use - n_new);
          m_use = m_new;
          n_use = n_new;
          rescale_o = true;
        }
        rescale_o = __any_sync(0xffffffffu, rescale_o);
        const float neg_m = m_use == -INFINITY ? 0.f : kWideTop - m_use;
        const float neg_n = n_use == -INFINITY ? 0.f : -n_use;
        auto offset = [&](float log) { return ptx::max_nan(log + neg_m, neg_n - 60.f); };
        if constexpr (NG == 2) {
#pragma unroll
          for (int g2 = 0; g2 < 2; ++g2) fb2[g2] = offset(fb2[g2]);
        }
        uint32_t pk[32];
        // Weights of keys 32 c .. 32 c + 31, added to l.
        auto exponents = [&](int c) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float a, off;
            if constexpr (NG == 2) {
              a = fa2[c >> 1];
              off = fb2[c >> 1];
            } else {
              a = factor(2 * c + q);
              off = offset(v_log(2 * c + q));
            }
            const uint64_t a2 = ptx::f2_pack(a, a), off2 = ptx::f2_pack(off, off);
            uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
            for (int i = 16 * q; i < 16 * q + 16; i += 2) {
              float x0, x1;
              ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])), a2, off2),
                             x0, x1);
              const float p0 = ptx::ex2_approx(x0), p1 = ptx::ex2_approx(x1);
              acc[(i >> 1) & 1] = ptx::f2_add(acc[(i >> 1) & 1], ptx::f2_pack(p0, p1));
              pk[(c & 1) * 16 + (i >> 1)] = ptx::pack_f16x2(p0, p1);
            }
            float s0, s1;
            ptx::f2_unpack(ptx::f2_add(acc[0], acc[1]), s0, s1);
            l = fmaf(s0 + s1, ptx::ex2_approx(neg_n - off), l);
          }
        };
        exponents(0);
        exponents(1);
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
        ptx::tmem_st32(tP, pk);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_half[t]));
        exponents(2);
        exponents(3);
        ptx::tmem_st32(tP + 32, pk);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[t]));
      }
      if (!ok) break;
      pair0 += blocks;
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_o_full[t]), units++ & 1, abort_ptr, p.timeout_ns, kRolePagedSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      const bool none = l == 0.f;
      const float total = n_use + __log2f(l);
      const float inv = none ? 0.f : ptx::ex2_approx(m_use - kWideTop - total);
      const float lse = none ? -INFINITY : total * 0.69314718055994530942f;
      const int head = job.head + row - ti * job.heads, token = job.token + ti;
      if (live) {
        if (job.slot >= 0) p.Lp[static_cast<size_t>(job.slot) * C::kRows + row] = lse;
        else p.lse[static_cast<long long>(head) * sh.T_q + token] = lse;
      }
      __syncwarp();                          // (tensor memory is read by whole warps, rows are written by lanes that have one)
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(tO + 32 * c, o);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(o);
        if (live && job.slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.Op + (static_cast<size_t>(job.slot) * C::kRows + row) * HD + 32 * c);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                 __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
        } else if (live) {
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
        __syncwarp();
      }
      ptx::tc_fence_before();
    }
  } else if (warp == 8) {
    paged_load<HD, C::kTiles, C::kScales, true>(p, &line, &tmK, &tmV, jobs, bar_job_full, bar_job_empty, bar_full, bar_empty,
                                          page_scale, sTiles, abort_ptr);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    int pair0 = 0;                           // key tiles of the units before
    int g[2] = {0, 0}, units[2] = {0, 0};    // key tiles and units of each row tile so far
    // S_t = K tile `pair` times the row tile's hi and lo.
    auto k_wait = [&](int pair) {
      const int it = 2 * pair;
      if (!wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_full[it % C::kTiles]), (it / C::kTiles) & 1, abort_ptr, p.timeout_ns,
                              kRolePagedMma))
        return false;
      ptx::tc_fence_after();
      return true;
    };
    const uint32_t idesc_qk = C::kIdescQK | (p.negate ? ptx::kIdescNegateA : 0u);
    auto qk = [&](int t, int pair) {
      const uint64_t a = ptx::desc_of(sQ + 2 * t * C::kTileBytes, 16, C::kAtom, C::kSwizzle);
      const uint64_t b = ptx::desc_of(sTiles + (2 * pair % C::kTiles) * C::kTileBytes, 16, C::kAtom, C::kSwizzle);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < HD / 32; ++k)
          ptx::mma_f8_warp(tmem_base + C::kColS + 128 * t, ptx::desc_lo(a) + part * (C::kTileBytes >> 4) + 2 * k,
                           ptx::desc_hi(a), ptx::desc_lo(b) + 2 * k, ptx::desc_hi(b), idesc_qk, part + k > 0 ? 1u : 0u);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full[t]));
      ++g[t];
    };
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedMma);
      if (!ok) break;
      const int b = jobs[ring].b, blocks = jobs[ring].j1 - jobs[ring].j0, nt = jobs[ring].rows > 128 ? 2 : 1;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (b < 0) break;
      ok = k_wait(pair0);
      // (Every P of the unit before has been waited for, so S is free; its O is read before this unit's first P.)
      for (int t = 0; t < nt && ok; ++t) {
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_q_full[t]), units[t]++ & 1, abort_ptr, p.timeout_ns, kRolePagedMma);
        if (!ok) break;
        ptx::tc_fence_after();
        qk(t, pair0);
      }
      if (!ok) break;
      ptx::mma_commit_warp(ptx::smem_u32(&bar_empty[2 * pair0 % C::kTiles]));
      for (int jj = 0; jj < blocks && ok; ++jj) {
        const int pair = pair0 + jj;
        const bool last = jj + 1 == blocks;
        const uint64_t v = ptx::desc_mnmajor_sw128(sSlots + (pair % C::kSlots) * C::kSlotBytes, C::kChunkBytes);
        for (int t = 0; t < nt && ok; ++t) {
          // P V in two halves: the first runs while the weights of keys 64-127 are still computed.
          const uint32_t d = tmem_base + C::kColO + HD * t, a = tmem_base + C::kColP + C::kStepP * t, par = (g[t] - 1) & 1;
          ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_p_half[t]), par, abort_ptr, p.timeout_ns, kRolePagedMma);
          if (ok && t == 0)
            ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_slot_full[pair % C::kSlots]), (pair / C::kSlots) & 1, abort_ptr,
                                    p.timeout_ns, kRolePagedMma);
          if (!ok) break;
          ptx::tc_fence_after();
          ptx::mma_ts_k64half_warp<0>(d, a, ptx::desc_lo(v), ptx::desc_hi(v), C::kIdescPV, jj > 0 ? 1u : 0u);
          ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_p_full[t]), par, abort_ptr, p.timeout_ns, kRolePagedMma);
          if (!ok) break;
          ptx::tc_fence_after();
          ptx::mma_ts_k64half_warp<1>(d, a, ptx::desc_lo(v), ptx::desc_hi(v), C::kIdescPV, 1u);
          if (last) {
            ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[t]));
          } else {
            // At d = 128 this S is written where the P lies that P V, just issued, reads. Nothing waits for P V in
            // between: products that one thread issues run one after another, as the forward and
            // backward kernels rely on, too (PTX says so of one accumulator and shape; here the kinds differ as well).
            // With a wait for P V the results have the same bits (400 calls of random sizes, ten times each),
            // and the pieces above take 187 us instead of 166.
            if (t == 0) ok = k_wait(pair + 1);
            if (ok) qk(t, pair + 1);
          }
        }
        if (!ok) break;
        ptx::mma_commit_warp(ptx::smem_u32(&bar_slot_empty[pair % C::kSlots]));
        if (!last) ptx::mma_commit_warp(ptx::smem_u32(&bar_empty[2 * (pair + 1) % C::kTiles]));
      }
      pair0 += blocks;
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ------------------------------------------------------------ conversion
    const int tid = threadIdx.x - 384;
    bool ok = true;
    int pair = 0;                            // key tiles so far
    for (int n = 0; ok; ++n) {
      const int ring = n & (kJobs - 1);
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_job_full[ring]), (n / kJobs) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedQuery);
      if (!ok) break;
      const PagedJob job = jobs[ring];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[ring]));
      if (job.b < 0) break;
      // The V tiles: a thread has a key's row.
      for (int j = job.j0; j < job.j1 && ok; ++j, ++pair) {
        const bool clear = j * 128 + tid >= job.n_keys;   // (rows behind the unit's keys may hold anything)
        const int it = 2 * pair + 1, tile = it % C::kTiles, slot = pair % C::kSlots;
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_full[tile]), (it / C::kTiles) & 1, abort_ptr, p.timeout_ns,
                                kRolePagedQuery);
        if (!ok) break;
        uint4 v[HD / 16];
        const uint8_t* from = generic + (sTiles - smem_base) + tile * C::kTileBytes + tid * HD;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
          v[i] = *reinterpret_cast<const uint4*>(from + ((i ^ (HD == 128 ? tid & 7 : (tid >> 1) & 3)) << 4));
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_slot_empty[slot]), ((pair / C::kSlots) & 1) ^ 1u, abort_ptr,
                                p.timeout_ns, kRolePagedQuery);
        if (!ok) break;
        uint8_t* to = generic + (sSlots - smem_base) + slot * C::kSlotBytes + tid * 128;
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
