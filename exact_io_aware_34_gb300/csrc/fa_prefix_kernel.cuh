// Exact attention for a few new tokens of every sequence of a batch, whose
// keys are a prefix that all sequences share and a cache of each sequence's
// own, of its own length: the decode step behind a shared prompt (or, without
// a prefix, of a ragged batch). sm_103a, tcgen05 + TMEM + TMA.
//
// What is computed: softmax attention over the prefix keys and the first
// len_b keys of sequence b's own cache. With the partial results over two
// disjoint key sets merged by the online-softmax rule
//   LSE = ln sum_s e^{LSE_s},  O = sum_s e^{LSE_s - LSE} O_s,
// the two parts are separate problems: against the prefix, the query rows of
// all sequences form one tall tile per K/V head, so its K/V are read once for
// the batch instead of once per sequence; against the own caches each
// sequence has a tile of its group's rows.
//
// Work. A unit is one 128-row query tile and its whole key range: (K/V head,
// tile of sequences) for the prefix, (sequence, K/V head) for the own keys.
// All units' 128-key blocks stand in one line, each unit's behind kUnitCost
// empty places (what a unit costs beside its blocks), and the CTAs (two per SM)
// take equal, contiguous pieces of it. So every CTA has about the same work
// whatever the lengths are, which only the device knows. A piece may hold
// several units' ends and wholes (segments); each segment leaves a float32
// partial result (O normalised by its own l, and LSE) in the workspace, at
// slot (unit + CTA): that number grows by one or two from one segment to the
// next, so no two share a slot, and a unit's segments have consecutive ones.
// prefix_merge_kernel, a programmatic dependent, combines a row's segments.
//
// What bounds it: K and V from memory while caches are long (eight own caches
// of up to 32768 rows, 32 heads on 8, d = 128: 86 us, 0.96 of the measured copy
// rate; a prefix of 32768 rows for 32 answers: 41 us, 0.68). With little to read,
// the latency of a unit's chain (loads, two products, softmax, partial result)
// and of the merge: 64 answers on a prefix of 8192 rows 28.5 us against 10.4 of
// reading, two answers on 500 rows 9.7 us. P is rounded to bf16 for P V, as in
// fa_varlen_fwd_kernel: O is off by 0.0023 of its norm, by 0.0017 with P in float32.
//
// Per CTA (256 threads): warps 0-3 softmax and epilogue, warp 4 TMA producer,
// warp 5 MMA issuer, warp 6 walks the segments one ahead and hands them to
// the others through a two-slot ring, warp 7 clears the V rows past a
// sequence's length (any value may stand there, and a probability of zero does
// not cancel an infinity): such a tile's load completes on a barrier of its
// own, and warp 7 completes the tile's barrier in its place. The block update
// and the masking with -inf are fa_varlen_fwd_kernel's; register split, ring
// and TMEM are fa_decode_kernel's.
#pragma once

#include "fa_decode_kernel.cuh"
#include "fa_varlen_kernel.cuh"

namespace fa {

namespace ptx {

// tma_load_3d for a 4-D map.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2,
                                            int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

}  // namespace ptx

enum : unsigned int { kRolePreProducer = 23, kRolePreMma = 24, kRolePreSoftmax = 25, kRolePreWalk = 26 };

// Places of a unit in the line beside its blocks: a one-block unit takes about
// three times as long as one block of a long one.
constexpr int kUnitCost = 2;

// Sizes that the attention and the merge kernel share.
struct PreShape {
  int B, H, H_kv, G, N_q;
  int n_p;                // prefix keys
  int room;               // rows of a sequence's own cache
  int hp;                 // query heads of a group per tile: min(G, 128 / N_q)
  int ht;                 // tiles per group: ceil(G / hp)
  int bp;                 // sequences per prefix tile: 128 / (hp * N_q) if ht == 1, else 1
  int bt;                 // prefix tiles along the batch: ceil(B / bp)
  int p_blocks;           // 128-key blocks of the prefix
  int p_units;            // prefix units: H_kv * bt * ht, or 0 without a prefix
  int ctas;
};

struct PreParams {
  PreShape s;
  const int* lens;        // [B]
  int2* seg;              // [p_units + own units]: first slot and number of a unit's segments (none for empty units)
  float* Op;              // prefix partials [p_units + ctas][128][d]
  float* Lp;              // [p_units + ctas][128]
  float* Oo;              // own partials [B * H_kv * ht + ctas][hp * N_q][d]
  float* Lo;
  int causal;
  float scale_log2;
  uint32_t idesc_qk;
  unsigned long long timeout_ns;
  int drop_load;
};

struct PreJob {
  int own;                // 0: prefix, 1: own cache, -1: no more segments
  int b0, kvh, h0;        // first sequence, K/V head, first query head within the group
  int j0, j1;             // key blocks
  int n_keys;             // keys of the unit
  int rows;               // rows of the tile that hold queries
  int slot;               // of the partial result, within its array
};

// CTA c of n takes places [line_begin(c), line_begin(c + 1)) of a line of w.
__device__ __forceinline__ int line_begin(int w, int n, int c) {
  const int q = w / n, r = w - q * n;
  return c * q + min(c, r);
}
// The CTA that takes place x.
__device__ __forceinline__ int line_owner(int w, int n, int x) {
  const int q = w / n, r = w - q * n;
  const int split = r * (q + 1);
  return x < split ? x / (q + 1) : r + (x - split) / q;
}

__device__ __forceinline__ int own_len(const PreParams& p, int b) { return max(0, min(p.s.room, p.lens[b])); }
// Places of a unit with `len` keys.
__device__ __forceinline__ int unit_places(int len) { return len > 0 ? kUnitCost + ((len + 127) >> 7) : 0; }

template <int HD>
struct PreCfg {
  static constexpr int kStageBytes = 4 * 2048;      // epilogue: per softmax warp 32 rows x 16 float32 columns
  static constexpr int kSmemBytes = DecCfg<HD>::kSmemBytes + kStageBytes;
  // Two CTAs on an SM, with 1 KB each for the system and 1 KB for the barriers.
  static_assert(2 * (kSmemBytes + 2048) <= 228 * 1024, "two CTAs per SM");
};

template <int HD>
__global__ void __launch_bounds__(DecCfg<HD>::kThreads, DecCfg<HD>::kCtasPerSm)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQp, const __grid_constant__ CUtensorMap tmQo,
                     const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PreParams p) {
  using C = DecCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q_full;
  __shared__ __align__(8) uint64_t bar_q_empty;
  __shared__ __align__(8) uint64_t bar_kv_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_kv_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_s_full;
  __shared__ __align__(8) uint64_t bar_p_full;
  __shared__ __align__(8) uint64_t bar_o_full;
  __shared__ __align__(8) uint64_t bar_job_full[2];
  __shared__ __align__(8) uint64_t bar_job_empty[2];
  __shared__ __align__(8) uint64_t bar_tail[4];   // V tiles with rows to clear have landed
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PreJob jobs[2];
  __shared__ int warp_sum[C::kThreads / 32];
  __shared__ int start_b, start_cum;          // sequence of this CTA's first own place, own places (per unit) before it
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PreShape& sh = p.s;

  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = smem_base;
  const uint32_t sKV = smem_base + C::kTileBytes;
  const uint32_t sStage = sKV + C::kStages * C::kTileBytes;
  uint8_t* kv_generic = smem_raw + (sKV - ptx::smem_u32(smem_raw));

  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&bar_q_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_q_empty), 1);
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_kv_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_kv_empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bar_s_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_p_full), C::kBM);
    ptx::mbar_init(ptx::smem_u32(&bar_o_full), 1);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 7);   // warps 0-5 and 7
    }
    for (int r = 0; r < 4; ++r) ptx::mbar_init(ptx::smem_u32(&bar_tail[r]), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    abort_flag = 0;
    start_b = sh.B;
    start_cum = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 5) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    ptx::prefetch_tmap(&tmQp);
    ptx::prefetch_tmap(&tmQo);
    ptx::prefetch_tmap(&tmKp);
    ptx::prefetch_tmap(&tmVp);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }

  // The line's length: every CTA adds up the own places of all sequences.
  int sum = 0;
  for (int b = threadIdx.x; b < sh.B; b += C::kThreads) sum += unit_places(own_len(p, b));
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  int own_sum = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) own_sum += warp_sum[w];
  const int own_units_per_seq = sh.H_kv * sh.ht;
  const int p_places = sh.p_blocks + kUnitCost;
  const int p_total = sh.p_units * p_places;
  const int total = p_total + own_sum * own_units_per_seq;
  const int x_begin = line_begin(total, sh.ctas, blockIdx.x);
  const int x_end = line_begin(total, sh.ctas, blockIdx.x + 1);
  // Where this CTA's first own place lies. (CTA 0 goes through all lengths and
  // looks for ones that do not fit the cache.)
  const bool check = blockIdx.x == 0;
  if (check || x_end > p_total) {
    const int target = max(0, x_begin - p_total) / own_units_per_seq;   // in places per unit
    int base = 0;
    for (int c0 = 0; c0 < sh.B; c0 += C::kThreads) {
      const int b = c0 + threadIdx.x;
      const int raw_len = b < sh.B ? p.lens[b] : 0;
      const int nu = unit_places(min(sh.room, raw_len));
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
      if (check && (raw_len < 0 || raw_len > sh.room)) {
        if (atomicCAS(&g_status_word, 0u, kStatusBadOffsets) == 0u) {
          g_status_info[0] = kRolePreWalk;
          g_status_info[1] = static_cast<unsigned int>(b);
          g_status_info[2] = g_status_info[3] = 0u;
        }
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
  // (The softmax stands first, as in fa_varlen_fwd_kernel: 1 to 2 % here.)
  if (warp < 4) {
    // ------------------------------------------------------------ softmax + epilogue
    ptx::setmaxnreg_inc<C::kRegsSoftmax>();
    const int row = warp * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem_base + lane_addr + C::kColS;
    const uint32_t tO = tmem_base + lane_addr + C::kColO;
    const float sl2 = p.scale_log2;
    // Row of a tile: (sequence * hp + head) * N_q + new token.
    const int qi = row % sh.N_q;
    const uint32_t stage = sStage + static_cast<uint32_t>(warp) * 2048u;
    bool ok = true;
    int g = 0;
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                              kRolePreSoftmax);
      if (!ok) break;
      const PreJob job = jobs[n & 1];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (job.own < 0) break;
      const int limit = job.own && p.causal ? max(0, job.n_keys - (sh.N_q - 1 - qi)) : job.n_keys;
      const bool active = warp * 32 < job.rows;   // a warp without query rows only keeps the hand-offs going
      float m_use = -INFINITY, l = 0.f, lo = 0.f;
      for (int j = job.j0; j < job.j1; ++j, ++g) {
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_full), g & 1, abort_ptr, p.timeout_ns, kRolePreSoftmax);
        if (!ok) break;
        if (!active) {
          ptx::mbar_arrive(ptx::smem_u32(&bar_p_full));
          continue;
        }
        ptx::tc_fence_after();
        const int valid = limit - j * C::kBN;
        // Scores past a row's limit become -inf in TMEM, in a short loop (see fa_varlen_fwd_kernel).
        if (!__all_sync(0xffffffffu, valid >= C::kBN)) {
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
        uint32_t s[4][32];
        float mr[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld32_max(tS + 32 * c, s[c], mr[c]);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ptx::reg_fence32(s[c]);
          ptx::reg_fence1(mr[c]);
        }
        const float mt = ptx::max3(mr[0], mr[1], fmaxf(mr[2], mr[3]));
        float alpha = 1.f;
        bool rescale_o = false;
        if (j == job.j0) {
          m_use = mt;
        } else {
          const bool need = (mt - m_use) * sl2 > kRescaleLog2;
          rescale_o = __any_sync(0xffffffffu, need);
          if (need) {
            alpha = ptx::ex2_approx((m_use - mt) * sl2);
            m_use = mt;
          }
        }
        const uint64_t sl2x2 = ptx::f2_pack(sl2, sl2);
        const float neg_m = m_use == -INFINITY ? 0.f : -m_use * sl2;
        const uint64_t negmx2 = ptx::f2_pack(neg_m, neg_m);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[2][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            ptx::f2_unpack(
                ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])), sl2x2, negmx2), x0,
                x1);
            const float p0 = ptx::ex2_approx(x0);
            const float p1 = ptx::ex2_approx(x1);
            acc[(i >> 1) & 3] = ptx::f2_add(acc[(i >> 1) & 3], ptx::f2_pack(p0, p1));
            pk[c >> 1][(c & 1) * 16 + (i >> 1)] = ptx::pack_bf16x2(p0, p1);
          }
          if (c == 1) ptx::tmem_st32(tS, pk[0]);
        }
        float sum;
        {
          float a0, a1, b0, b1;
          ptx::f2_unpack(ptx::f2_add(acc[0], acc[1]), a0, a1);
          ptx::f2_unpack(ptx::f2_add(acc[2], acc[3]), b0, b1);
          sum = (a0 + a1) + (b0 + b1);
        }
        // The largest probability enters O's normaliser rounded as P V sees it (see the forward kernel).
        const float pmax = ptx::ex2_approx(fmaf(mt, sl2, neg_m));
        l = l * alpha + sum;
        lo = lo * alpha + (sum + (ptx::round_bf16(pmax) - pmax));
        ptx::tmem_st32(tS + 32, pk[1]);
        if (rescale_o) {
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
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full));
      }
      if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_o_full), n & 1, abort_ptr, p.timeout_ns, kRolePreSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      if (active) {
        const bool none = l == 0.f;            // this row sees none of the segment's keys
        const float inv_l = none ? 0.f : 1.f / lo;
        const int per_slot = job.own ? sh.hp * sh.N_q : C::kBM;
        const size_t at = static_cast<size_t>(job.slot) * per_slot + warp * 32;   // the warp's first row
        float* dst = (job.own ? p.Oo : p.Op) + at * HD;
        const int rows = min(32, job.rows - warp * 32);
        if (lane < rows)
          (job.own ? p.Lo : p.Lp)[at + lane] = none ? -INFINITY : (m_use * sl2 + __log2f(l)) * 0.69314718055994530942f;
        // A few rows are written as they are; more leave through shared memory
        // in 16-column pieces (16-byte units swizzled by row), so that four
        // lanes write 64 bytes of a row.
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          ptx::tmem_ld32(tO + 32 * c, o);
          ptx::tmem_ld_wait();
          ptx::reg_fence32(o);
          if (rows <= 8) {
            if (lane < rows) {
              float4* row_dst = reinterpret_cast<float4*>(dst + static_cast<size_t>(lane) * HD + 32 * c);
#pragma unroll
              for (int v = 0; v < 8; ++v)
                row_dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv_l, __uint_as_float(o[4 * v + 1]) * inv_l,
                                         __uint_as_float(o[4 * v + 2]) * inv_l, __uint_as_float(o[4 * v + 3]) * inv_l);
            }
            continue;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            __syncwarp();       // the piece before has been read
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const uint32_t addr = stage + static_cast<uint32_t>(lane) * 64u + ((v ^ ((lane >> 1) & 3u)) << 4);
              const uint32_t* src = o + 16 * k + 4 * v;
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(__uint_as_float(src[0]) * inv_l),
                           "f"(__uint_as_float(src[1]) * inv_l), "f"(__uint_as_float(src[2]) * inv_l),
                           "f"(__uint_as_float(src[3]) * inv_l)
                           : "memory");
            }
            __syncwarp();
            float4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = 8 * q + (lane >> 2);
              const uint32_t addr = stage + static_cast<uint32_t>(r) * 64u + (((lane ^ (r >> 1)) & 3u) << 4);
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(w[q].x), "=f"(w[q].y), "=f"(w[q].z), "=f"(w[q].w)
                           : "r"(addr)
                           : "memory");
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = 8 * q + (lane >> 2);
              if (r < rows)
                *reinterpret_cast<float4*>(dst + static_cast<size_t>(r) * HD + 32 * c + 16 * k + 4 * (lane & 3)) = w[q];
            }
          }
        }
      }
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_first = ptx::policy_evict_first();
      const uint64_t pol_last = ptx::policy_evict_last();    // prefix tiles are read by every tile of sequences
      const uint32_t q_full = ptx::smem_u32(&bar_q_full);
      int it = 0, q_issued = 0, tails = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        ok = wait_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                           kRolePreProducer);
        if (!ok) break;
        const PreJob job = jobs[n & 1];
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
        if (job.own < 0) break;
        if (n > 0 && !wait_or_abort(ptx::smem_u32(&bar_q_empty), (n - 1) & 1, abort_ptr, p.timeout_ns,
                                    kRolePreProducer)) {
          ok = false;
          break;
        }
        // Rows of the tile beyond the box keep what they held: a row of S and
        // of O depends on its own row of Q alone, and they are not stored.
        const int box_rows = sh.hp * sh.N_q * (job.own ? 1 : sh.bp);
        ptx::mbar_arrive_expect_tx(q_full, C::kChunks * 128 * box_rows);
        for (int c = 0; c < C::kChunks; ++c)
          ptx::tma_load_4d(sQ + c * C::kChunkBytes, job.own ? &tmQo : &tmQp, q_full, c * 64, 0,
                           job.kvh * sh.G + job.h0, job.b0, pol_last);
        q_issued = n + 1;
        const CUtensorMap* maps[2] = {job.own ? &tmK : &tmKp, job.own ? &tmV : &tmVp};
        const uint64_t pol = job.own || sh.bt * sh.ht == 1 ? pol_first : pol_last;
        for (int j = job.j0; j < job.j1 && ok; ++j) {
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = it % C::kStages;
            if (!wait_or_abort(ptx::smem_u32(&bar_kv_empty[slot]), ((it / C::kStages) & 1) ^ 1u, abort_ptr,
                               p.timeout_ns, kRolePreProducer)) {
              ok = false;
              break;
            }
            const int me = it++;
            if (me == p.drop_load) continue;   // test hook: this tile never arrives
            // A V tile with rows past the length: warp 7 completes its barrier.
            const bool tail = kv && job.own && (j + 1) * C::kBN > job.n_keys;
            const uint32_t full = ptx::smem_u32(tail ? &bar_tail[tails++ & 3] : &bar_kv_full[slot]);
            ptx::mbar_arrive_expect_tx(full, C::kTileBytes);
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_4d(sKV + slot * C::kTileBytes + c * C::kChunkBytes, maps[kv], full, c * 64, j * C::kBN,
                               job.kvh, job.own ? job.b0 : 0, pol);
          }
        }
      }
      if (!ok || *abort_ptr) {
        if (q_issued > 0) drain_wait(q_full, (q_issued - 1) & 1, p.timeout_ns);
        for (int r = max(0, tails - 4); r < tails; ++r)
          drain_wait(ptx::smem_u32(&bar_tail[r & 3]), (r >> 2) & 1, p.timeout_ns);
        for (int i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
          if (i != p.drop_load)
            drain_wait(ptx::smem_u32(&bar_kv_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    int it0 = 0, g = 0;       // K/V loads and key blocks of the segments before
    auto kv_wait = [&](int it) {
      return wait_warp_or_abort(ptx::smem_u32(&bar_kv_full[it % C::kStages]), (it / C::kStages) & 1, abort_ptr,
                                p.timeout_ns, kRolePreMma);
    };
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns, kRolePreMma);
      if (!ok) break;
      const int own = jobs[n & 1].own, blocks = jobs[n & 1].j1 - jobs[n & 1].j0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (own < 0) break;
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_full), n & 1, abort_ptr, p.timeout_ns, kRolePreMma);
      // Step jj: P V of block jj - 1 (P sits in the S columns), then Q K^T of block jj.
      for (int jj = 0; jj <= blocks && ok; ++jj) {
        const int itK = it0 + 2 * jj, itV = itK - 1;
        if (jj > 0) {
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full), (g - 1) & 1, abort_ptr, p.timeout_ns, kRolePreMma);
          if (ok) ok = kv_wait(itV);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t b_desc =
              ptx::desc_mnmajor_sw128(sKV + (itV % C::kStages) * C::kTileBytes, C::kChunkBytes);
          ptx::mma_ts_k128_warp<32>(tmem_base + C::kColO, tmem_base + C::kColS, ptx::desc_lo(b_desc),
                                    ptx::desc_hi(b_desc), C::kIdescPV, jj > 1 ? 1u : 0u);
          if (jj == blocks) ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full));
          ptx::mma_commit_warp(ptx::smem_u32(&bar_kv_empty[itV % C::kStages]));
        }
        if (jj < blocks) {
          ok = kv_wait(itK);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t a_desc = ptx::desc_kmajor_sw128(sQ);
          const uint64_t b_desc = ptx::desc_kmajor_sw128(sKV + (itK % C::kStages) * C::kTileBytes);
          if constexpr (HD == 128)
            ptx::mma_ss_k128_warp(tmem_base + C::kColS, ptx::desc_lo(a_desc), ptx::desc_lo(b_desc),
                                  ptx::desc_hi(a_desc), p.idesc_qk, 0u);
          else
            ptx::mma_ss_k64_warp(tmem_base + C::kColS, ptx::desc_lo(a_desc), ptx::desc_lo(b_desc),
                                 ptx::desc_hi(a_desc), p.idesc_qk, 0u);
          ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full));
          ptx::mma_commit_warp(ptx::smem_u32(&bar_kv_empty[itK % C::kStages]));
          if (jj == blocks - 1) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty));
          ++g;
        }
      }
      it0 += 2 * blocks;
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 7) {
    // ------------------------------------------------------------ tails of V tiles
    bool ok = true;
    int it0 = 0, tails = 0;
    for (int n = 0; ok; ++n) {
      ok = wait_idle_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns, kRolePreWalk);
      if (!ok) break;
      const int own = jobs[n & 1].own, blocks = jobs[n & 1].j1 - jobs[n & 1].j0;
      const int have = jobs[n & 1].n_keys - (jobs[n & 1].j1 - 1) * C::kBN;    // keys in the segment's last block
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (own < 0) break;
      it0 += 2 * blocks;
      if (!own || have >= C::kBN) continue;    // (behind the prefix, TMA fills with zeros)
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_tail[tails & 3]), (tails >> 2) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePreWalk);
      if (!ok) break;
      ++tails;
      // Whole 128-byte rows, so the swizzle does not matter.
      const int slot = (it0 - 1) % C::kStages;
      for (int c = 0; c < C::kChunks; ++c)
        for (int i = lane; i < (C::kBN - have) * 8; i += 32)
          reinterpret_cast<uint4*>(kv_generic + slot * C::kTileBytes + c * C::kChunkBytes + have * 128)[i] =
              make_uint4(0u, 0u, 0u, 0u);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_kv_full[slot]));
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------------ segments
    if (lane == 0) {
      int x = x_begin, b = start_b, cum = start_cum;
      for (int n = 0;; ++n) {
        PreJob job;
        job.own = -1;
        int unit = 0, end = 0;       // the unit's number among all, its last place
        while (x < x_end && job.own < 0) {
          int first, len;            // its first place, its keys
          if (x < p_total) {
            unit = x / p_places;
            first = unit * p_places;
            len = sh.n_p;
          } else {
            if (b >= sh.B) break;
            const int y = x - p_total;
            len = own_len(p, b);
            int nu = unit_places(len);
            while (y >= (cum + nu) * own_units_per_seq && b + 1 < sh.B) {   // on to the sequence that holds place y
              cum += nu;
              ++b;
              len = own_len(p, b);
              nu = unit_places(len);
            }
            if (nu == 0) break;
            const int u = min((y - cum * own_units_per_seq) / nu, own_units_per_seq - 1);
            unit = sh.p_units + b * own_units_per_seq + u;
            first = p_total + cum * own_units_per_seq + u * nu;
          }
          const int places = unit_places(len);
          const int from = x - first;
          // A place behind the last unit, or none that holds it (above): lengths that
          // change under the call. What it returns is then undefined, but it ends.
          if (from >= places) break;
          const int to = min(places, from + (x_end - x));
          x += to - from;
          end = first + places - 1;
          job.j0 = max(0, from - kUnitCost);
          job.j1 = max(0, to - kUnitCost);
          if (job.j1 <= job.j0) continue;        // only the places beside its blocks
          job.n_keys = len;
          if (unit < sh.p_units) {
            const int per_head = sh.bt * sh.ht;
            job.own = 0;
            job.kvh = unit / per_head;
            const int t = unit - job.kvh * per_head, tb = t / sh.ht;
            job.b0 = tb * sh.bp;
            job.h0 = (t - tb * sh.ht) * sh.hp;
            job.rows = min(sh.hp, sh.G - job.h0) * sh.N_q * min(sh.bp, sh.B - job.b0);
            job.slot = unit + static_cast<int>(blockIdx.x);
          } else {
            const int u = unit - sh.p_units - b * own_units_per_seq;
            job.own = 1;
            job.b0 = b;
            job.kvh = u / sh.ht;
            job.h0 = (u - job.kvh * sh.ht) * sh.hp;
            job.rows = min(sh.hp, sh.G - job.h0) * sh.N_q;
            job.slot = unit - sh.p_units + static_cast<int>(blockIdx.x);
          }
        }
        if (!wait_or_abort(ptx::smem_u32(&bar_job_empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr,
                           kUnitWaits * p.timeout_ns, kRolePreWalk))
          break;
        jobs[n & 1] = job;
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[n & 1]));
        if (job.own < 0) break;
        // The CTA with a unit's first block notes its segments for the merge.
        if (job.j0 == 0)
          p.seg[unit] = make_int2(job.slot, line_owner(total, sh.ctas, end) - static_cast<int>(blockIdx.x) + 1);
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

// One warp per query row: its segments' partial results over the prefix and
// over the own keys, combined by LSE = m + ln sum_s e^{LSE_s - m},
// O = sum_s e^{LSE_s - LSE} O_s and rounded once to bf16. The lanes read the
// segments' LSE in parallel (32 at a time) and pass the weights by shuffles;
// eight segments' rows are requested before the first is used.
template <int HD>
__global__ void __launch_bounds__(128)
    prefix_merge_kernel(const PreParams p, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE, long long o_sb,
                        long long o_sh, long long o_sn) {
  constexpr int kPer = HD / 32;     // output elements per lane: 4 or 2
  const PreShape& sh = p.s;
  // (Rows fit 32 bits; their threads, 32 each, do not.)
  const unsigned row = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int i = static_cast<int>(row % sh.N_q);
  const unsigned bh = row / sh.N_q;
  const int b = static_cast<int>(bh / sh.H), h = static_cast<int>(bh - static_cast<unsigned>(b) * sh.H);
  const int kvh = h / sh.G, hg = h - kvh * sh.G, t = hg / sh.hp, in_tile = (hg - t * sh.hp) * sh.N_q + i;
  const int per_seq = sh.hp * sh.N_q;
  const int tb = b / sh.bp;
  const int u0 = (kvh * sh.bt + tb) * sh.ht + t, u1 = sh.p_units + (b * sh.H_kv + kvh) * sh.ht + t;
  if (b >= sh.B) return;
  const int len = own_len(p, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // A unit's first slot and number of segments. A CTA that gave up on a wait has
  // not noted the units behind it, and their entries hold anything: the range is
  // clamped to the slots that the unit can have, [u, u + CTAs). (Checked with
  // comparisons instead, two short sequences took 10.2 us, not 9.8.)
  auto segments = [&](int unit, int first_unit) {
    const int2 s = p.seg[unit];
    const int u = unit - first_unit;
    const unsigned before = min(static_cast<unsigned>(s.x - u), static_cast<unsigned>(sh.ctas));
    return make_int2(u + static_cast<int>(before), static_cast<int>(min(static_cast<unsigned>(s.y), sh.ctas - before)));
  };
  // Prefix segments [0, n0), own segments [n0, n): consecutive slots, one row of each.
  int2 s0 = make_int2(0, 0), s1 = make_int2(0, 0);
  if (sh.p_units > 0) s0 = segments(u0, 0);
  if (len > 0) s1 = segments(u1, sh.p_units);
  const int n0 = s0.y, n = s0.y + s1.y;
  const size_t row0 = static_cast<size_t>(s0.x) * 128 + (b - tb * sh.bp) * per_seq + in_tile;
  const size_t row1 = static_cast<size_t>(s1.x) * per_seq + in_tile;
  auto lse_of = [&](int s) {
    return s < n0 ? p.Lp[row0 + static_cast<size_t>(s) * 128] : p.Lo[row1 + static_cast<size_t>(s - n0) * per_seq];
  };
  const float first = lane < n ? lse_of(lane) : -INFINITY;
  float m = first;
  bool any = first != -INFINITY;         // a segment whose keys this row sees (a NaN counts, and comes through)
  for (int s = 32 + lane; s < n; s += 32) {
    const float v = lse_of(s);
    any |= v != -INFINITY;
    m = fmaxf(m, v);
  }
  const bool none = !__any_sync(0xffffffffu, any);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.f;
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  float sum = 0.f;
  if (!none) {
    for (int g0 = 0; g0 < n; g0 += 32) {
      const float mine = g0 == 0 ? first : g0 + lane < n ? lse_of(g0 + lane) : -INFINITY;
      const float w_me = __expf(mine - m);
      sum += w_me;
      for (int k0 = 0; k0 < min(32, n - g0); k0 += 8) {
        float v[8][kPer];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int s = min(g0 + k0 + k, n - 1);       // (past the end: the last again, with weight 0)
          const float* src = (s < n0 ? p.Op + (row0 + static_cast<size_t>(s) * 128) * HD
                                     : p.Oo + (row1 + static_cast<size_t>(s - n0) * per_seq) * HD) + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 f = *reinterpret_cast<const float4*>(src);
            v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
          } else {
            const float2 f = *reinterpret_cast<const float2*>(src);
            v[k][0] = f.x, v[k][1] = f.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float w = __shfl_sync(0xffffffffu, w_me, k0 + k);
          if (g0 + k0 + k < n) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = none ? 0.f : 1.f / sum;
  uint32_t packed[kPer / 2];
#pragma unroll
  for (int e = 0; e < kPer; e += 2) packed[e / 2] = ptx::pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  __nv_bfloat16* dst = O + b * o_sb + h * o_sh + i * o_sn + lane * kPer;
  if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
  else *reinterpret_cast<uint32_t*>(dst) = packed[0];
  if (lane == 0) LSE[row] = none ? -INFINITY : m + __logf(sum);
}

}  // namespace fa
