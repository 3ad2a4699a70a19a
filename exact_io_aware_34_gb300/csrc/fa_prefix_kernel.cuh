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
// All units' 128-key blocks stand in one line, and the CTAs (two per SM) take
// equal, contiguous pieces of it. So every CTA has the same number of blocks
// whatever the lengths are, which only the device knows. A piece may hold
// several units' ends and wholes (segments); each segment leaves a float32
// partial result (O normalised by its own l, and LSE) in the workspace, at
// slot (unit + CTA): that number grows by one or two from one segment to the
// next, so no two share a slot and the merge finds them without a table.
// prefix_merge_kernel, a programmatic dependent, combines a row's segments.
//
// Per CTA (256 threads): warps 0-3 softmax and epilogue, warp 4 TMA producer,
// warp 5 MMA issuer, warp 6 walks the segments one ahead and hands them to
// the others, as in fa_varlen_fwd_kernel. The block update, the masking with
// -inf and the clearing of V rows past a sequence's length are that kernel's;
// register split, ring and TMEM are fa_decode_kernel's.
#pragma once

#include "fa_decode_kernel.cuh"
#include "fa_varlen_kernel.cuh"

namespace fa {

enum : unsigned int { kRolePreProducer = 23, kRolePreMma = 24, kRolePreSoftmax = 25, kRolePreWalk = 26 };

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
  int* cum;               // [B]: own blocks (per unit) of the sequences before b
  long long* total;       // all blocks
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
  int slot;               // of the partial result, within its array
};

// CTA c of n takes blocks [line_begin(c), line_begin(c + 1)) of a line of w.
__device__ __forceinline__ long long line_begin(long long w, int n, int c) {
  const long long q = w / n, r = w - q * n;
  return c * q + (c < r ? c : r);
}
// The CTA that takes block x.
__device__ __forceinline__ int line_owner(long long w, int n, long long x) {
  const long long q = w / n, r = w - q * n;
  const long long split = r * (q + 1);
  return static_cast<int>(x < split ? x / (q + 1) : r + (x - split) / q);
}

__device__ __forceinline__ int own_len(const PreParams& p, int b) { return max(0, min(p.s.room, p.lens[b])); }

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
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) PreJob jobs[2];
  __shared__ long long warp_sum[C::kThreads / 32];
  __shared__ int start_b, start_cum;          // sequence of this CTA's first own block, own blocks before it
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PreShape& sh = p.s;

  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = smem_base;
  const uint32_t sKV = smem_base + C::kTileBytes;
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
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 6);   // producer, issuer, four softmax warps
    }
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

  // The line's length: every CTA adds up the own blocks of all sequences.
  long long sum = 0;
  for (int b = threadIdx.x; b < sh.B; b += C::kThreads) sum += (own_len(p, b) + 127) >> 7;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  long long own_sum = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) own_sum += warp_sum[w];
  const int own_units_per_seq = sh.H_kv * sh.ht;
  const long long p_total = static_cast<long long>(sh.p_units) * sh.p_blocks;
  const long long total = p_total + own_sum * own_units_per_seq;
  const long long x_begin = line_begin(total, sh.ctas, blockIdx.x);
  const long long x_end = line_begin(total, sh.ctas, blockIdx.x + 1);
  // Where this CTA's first own block lies (CTA 0 walks on and notes the sums
  // for the merge, and looks for lengths that do not fit the cache).
  const bool note = blockIdx.x == 0;
  if (note && threadIdx.x == 0) *p.total = total;
  if (note || x_end > p_total) {
    const long long target = (x_begin > p_total ? x_begin - p_total : 0) / own_units_per_seq;   // in blocks per unit
    long long base = 0;
    for (int c0 = 0; c0 < sh.B; c0 += C::kThreads) {
      const int b = c0 + threadIdx.x;
      const int raw_len = b < sh.B ? p.lens[b] : 0;
      const int nb = (max(0, min(sh.room, raw_len)) + 127) >> 7;
      int incl = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      __syncthreads();
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      long long before = base;
      long long chunk = 0;
      for (int w = 0; w < C::kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        chunk += warp_sum[w];
      }
      const long long excl = before + incl - nb;
      if (nb > 0 && excl <= target && target < excl + nb) {
        start_b = b;
        start_cum = static_cast<int>(excl);
      }
      if (note && b < sh.B) {
        p.cum[b] = static_cast<int>(excl);
        if (raw_len < 0 || raw_len > sh.room) {
          if (atomicCAS(&g_status_word, 0u, kStatusBadOffsets) == 0u) {
            g_status_info[0] = kRolePreWalk;
            g_status_info[1] = static_cast<unsigned int>(b);
            g_status_info[2] = g_status_info[3] = 0u;
          }
        }
      }
      base += chunk;
      if (!note && base > target) break;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  volatile int* abort_ptr = &abort_flag;

  if (warp >= 4) ptx::setmaxnreg_dec<C::kRegsControl>();
  if (warp == 6) {
    // ------------------------------------------------------------ segments
    if (lane == 0) {
      long long x = x_begin;
      int b = start_b;
      long long cum = start_cum;
      for (int n = 0;; ++n) {
        PreJob job;
        job.own = -1;
        if (x < x_end) {
          if (x < p_total) {
            const int u = static_cast<int>(x / sh.p_blocks);
            job.own = 0;
            job.j0 = static_cast<int>(x - static_cast<long long>(u) * sh.p_blocks);
            job.j1 = static_cast<int>(min(static_cast<long long>(sh.p_blocks), job.j0 + (x_end - x)));
            const int per_head = sh.bt * sh.ht;
            job.kvh = u / per_head;
            const int t = u - job.kvh * per_head;
            job.b0 = t / sh.ht * sh.bp;
            job.h0 = (t - t / sh.ht * sh.ht) * sh.hp;
            job.n_keys = sh.n_p;
            job.slot = u + static_cast<int>(blockIdx.x);
          } else {
            const long long y = x - p_total;
            int len = own_len(p, b);
            int nb = (len + 127) >> 7;
            while (y >= (cum + nb) * own_units_per_seq && b + 1 < sh.B) {   // on to the sequence that holds block y
              cum += nb;
              ++b;
              len = own_len(p, b);
              nb = (len + 127) >> 7;
            }
            const long long in_seq = y - cum * own_units_per_seq;
            const int u = static_cast<int>(in_seq / nb);
            job.own = 1;
            job.j0 = static_cast<int>(in_seq - static_cast<long long>(u) * nb);
            job.j1 = static_cast<int>(min(static_cast<long long>(nb), job.j0 + (x_end - x)));
            job.b0 = b;
            job.kvh = u / sh.ht;
            job.h0 = (u - job.kvh * sh.ht) * sh.hp;
            job.n_keys = len;
            job.slot = b * own_units_per_seq + u + static_cast<int>(blockIdx.x);
          }
          x += job.j1 - job.j0;
        }
        if (!wait_or_abort(ptx::smem_u32(&bar_job_empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr, p.timeout_ns,
                           kRolePreWalk))
          break;
        jobs[n & 1] = job;
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[n & 1]));
        if (job.own < 0) break;
      }
    }
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_first = ptx::policy_evict_first();
      const uint64_t pol_last = ptx::policy_evict_last();    // prefix tiles are read by every tile of sequences
      const uint32_t q_full = ptx::smem_u32(&bar_q_full);
      int it = 0, q_issued = 0;
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
            const uint32_t full = ptx::smem_u32(&bar_kv_full[slot]);
            ptx::mbar_arrive_expect_tx(full, C::kTileBytes);
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_4d(sKV + slot * C::kTileBytes + c * C::kChunkBytes, maps[kv], full, c * 64, j * C::kBN,
                               job.kvh, job.own ? job.b0 : 0, pol);
          }
        }
      }
      if (!ok || *abort_ptr) {
        if (q_issued > 0) drain_wait(q_full, (q_issued - 1) & 1, p.timeout_ns);
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
  } else if (warp < 4) {
    // ------------------------------------------------------------ softmax + epilogue
    ptx::setmaxnreg_inc<C::kRegsSoftmax>();
    const int row = warp * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem_base + lane_addr + C::kColS;
    const uint32_t tO = tmem_base + lane_addr + C::kColO;
    const float sl2 = p.scale_log2;
    // Row of a tile: (sequence * hp + head) * N_q + new token.
    const int per_seq = sh.hp * sh.N_q;
    const int bi = row / per_seq, hi = (row - bi * per_seq) / sh.N_q, qi = row - bi * per_seq - hi * sh.N_q;
    bool ok = true;
    int it0 = 0, g = 0;
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                              kRolePreSoftmax);
      if (!ok) break;
      const PreJob job = jobs[n & 1];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (job.own < 0) break;
      const int limit = job.own && p.causal ? max(0, job.n_keys - (sh.N_q - 1 - qi)) : job.n_keys;
      const bool live = bi < (job.own ? 1 : min(sh.bp, sh.B - job.b0)) && hi < min(sh.hp, sh.G - job.h0);
      const bool active = __any_sync(0xffffffffu, live);   // a warp without query rows only keeps the hand-offs going
      float m_use = -INFINITY, l = 0.f, lo = 0.f;
      for (int j = job.j0; j < job.j1; ++j, ++g) {
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_full), g & 1, abort_ptr, p.timeout_ns, kRolePreSoftmax);
        if (!ok) break;
        // V rows past the length (any value may stand there) are cleared
        // before P V. Q K^T of this block was issued behind the previous P V,
        // which had waited for its V, so this wait is for the next phase.
        const int have = job.n_keys - j * C::kBN;
        if (have < C::kBN) {
          const int itV = it0 + 2 * (j - job.j0) + 1;
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_kv_full[itV % C::kStages]), (itV / C::kStages) & 1, abort_ptr,
                                  p.timeout_ns, kRolePreSoftmax);
          if (!ok) break;
          uint8_t* v_tile = kv_generic + (itV % C::kStages) * C::kTileBytes;
          for (int c = 0; c < C::kChunks; ++c)
            for (int i = row; i < (C::kBN - have) * 8; i += C::kBM)
              reinterpret_cast<uint4*>(v_tile + c * C::kChunkBytes + have * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
          ptx::fence_proxy_async_smem();
        }
        if (!active) {
          ptx::mbar_arrive(ptx::smem_u32(&bar_p_full));
          continue;
        }
        ptx::tc_fence_after();
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
        const int valid = limit - j * C::kBN;
        float mt;
        if (__all_sync(0xffffffffu, valid >= C::kBN)) {
          mt = ptx::max3(mr[0], mr[1], fmaxf(mr[2], mr[3]));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= valid) s[c][i] = __float_as_uint(-INFINITY);
          float mc[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = k >> 1, bb = (k & 1) * 16;
            mc[k] = fmaxf(__uint_as_float(s[c][bb]), __uint_as_float(s[c][bb + 1]));
#pragma unroll
            for (int i = 2; i < 16; i += 2)
              mc[k] = ptx::max3(mc[k], __uint_as_float(s[c][bb + i]), __uint_as_float(s[c][bb + i + 1]));
          }
          mt = ptx::max3(ptx::max3(mc[0], mc[1], mc[2]), ptx::max3(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7]));
        }
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
      it0 += 2 * (job.j1 - job.j0);
      if (active) {
        const bool none = l == 0.f;            // this row sees none of the segment's keys
        const float inv_l = none ? 0.f : 1.f / lo;
        const int rows = job.own ? per_seq : C::kBM;
        const size_t at = static_cast<size_t>(job.slot) * rows + row;
        float* dst_o = (job.own ? p.Oo : p.Op) + at * HD;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          ptx::tmem_ld32(tO + 32 * c, o);
          ptx::tmem_ld_wait();
          ptx::reg_fence32(o);
          if (!live) continue;
          float4* dst = reinterpret_cast<float4*>(dst_o + 32 * c);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv_l, __uint_as_float(o[4 * v + 1]) * inv_l,
                                 __uint_as_float(o[4 * v + 2]) * inv_l, __uint_as_float(o[4 * v + 3]) * inv_l);
        }
        if (live)
          (job.own ? p.Lo : p.Lp)[at] = none ? -INFINITY : (m_use * sl2 + __log2f(l)) * 0.69314718055994530942f;
      }
    }
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
// segments' LSE in parallel and pass the weights by shuffles.
template <int HD>
__global__ void __launch_bounds__(256)
    prefix_merge_kernel(const PreParams p, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE, long long o_sb,
                        long long o_sh, long long o_sn) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PreShape& sh = p.s;
  const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(sh.B) * sh.H * sh.N_q) return;
  const int i = static_cast<int>(row % sh.N_q);
  const long long bh = row / sh.N_q;
  const int h = static_cast<int>(bh % sh.H), b = static_cast<int>(bh / sh.H);
  const int kvh = h / sh.G, hg = h - kvh * sh.G, t = hg / sh.hp, hi = hg - t * sh.hp;
  const int per_seq = sh.hp * sh.N_q;
  const long long total = *p.total, p_total = static_cast<long long>(sh.p_units) * sh.p_blocks;
  // Prefix segments [0, n0), own segments [n0, n0 + n1): consecutive slots, one row of each.
  int n0 = 0, n1 = 0;
  size_t row0 = 0, row1 = 0;
  if (sh.p_units > 0) {
    const int u = (kvh * sh.bt + b / sh.bp) * sh.ht + t;
    const long long x = static_cast<long long>(u) * sh.p_blocks;
    const int c = line_owner(total, sh.ctas, x);
    n0 = line_owner(total, sh.ctas, x + sh.p_blocks - 1) - c + 1;
    row0 = static_cast<size_t>(u + c) * 128 + (b % sh.bp) * per_seq + hi * sh.N_q + i;
  }
  const int nb = (own_len(p, b) + 127) >> 7;
  if (nb > 0) {
    const int per = sh.H_kv * sh.ht, u = kvh * sh.ht + t;
    const long long x = p_total + static_cast<long long>(p.cum[b]) * per + static_cast<long long>(u) * nb;
    const int c = line_owner(total, sh.ctas, x);
    n1 = line_owner(total, sh.ctas, x + nb - 1) - c + 1;
    row1 = (static_cast<size_t>(b) * per + u + c) * per_seq + hi * sh.N_q + i;
  }
  const int n = n0 + n1;
  auto lse_of = [&](int s) {
    return s < n0 ? p.Lp[row0 + static_cast<size_t>(s) * 128] : p.Lo[row1 + static_cast<size_t>(s - n0) * per_seq];
  };
  float m = -INFINITY;
  bool any = false;                      // a segment whose keys this row sees (a NaN counts, and comes through)
  for (int s = lane; s < n; s += 32) {
    const float v = lse_of(s);
    any |= v != -INFINITY;
    m = fmaxf(m, v);
  }
  const bool none = !__any_sync(0xffffffffu, any);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.f;
  constexpr int kPer = HD / 32;     // output elements per lane: 4 or 2
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  float sum = 0.f;
  if (!none) {
    for (int s0 = 0; s0 < n; s0 += 32) {
      const float w_me = s0 + lane < n ? __expf(lse_of(s0 + lane) - m) : 0.f;
      sum += w_me;
      const int cnt = min(32, n - s0);
#pragma unroll 4
      for (int k = 0; k < cnt; ++k) {
        const float w = __shfl_sync(0xffffffffu, w_me, k);
        const int s = s0 + k;
        const float* src = (s < n0 ? p.Op + (row0 + static_cast<size_t>(s) * 128) * HD
                                   : p.Oo + (row1 + static_cast<size_t>(s - n0) * per_seq) * HD) + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, src[e], acc[e]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = none ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = O + b * o_sb + h * o_sh + i * o_sn + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) LSE[row] = none ? -INFINITY : m + __logf(sum);
}

}  // namespace fa
