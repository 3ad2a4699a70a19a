// Backward of fa_varlen_fwd_kernel: gradients of <dO, O> over packed
// sequences, causal or not, with shared K/V heads, by recomputation from LSE.
// sm_103a, tcgen05 + TMEM + TMA.
//
// Formulas and roles are fa_bwd_kernel's (P = exp(scale S - LSE),
// dV = P^T dO, dS = P (dP - D), dQ = scale dS K, dK = scale dS^T Q; a
// key-block role that owns dK, dV and a query role that owns dQ, 7 products
// per pair of blocks, no atomics, the same bits from run to run). What
// differs:
//   * A query tile is 128 / G tokens x the G heads of a K/V head, as in the
//     forward. The key-block role streams such tiles, so the sum of dK and dV
//     over the group's heads is part of the products' reduction.
//   * Only pairs of blocks with a visible (row, key) are visited: the query
//     role stops at the last key its tile sees, the key-block role starts at
//     the first tile that sees its keys.
//   * The units of both roles are listed by varlen_bwd_plan: those of
//     the key-block role, then those of the query role, the most expensive
//     first in each. A persistent grid takes them by a counter. Within a role
//     the pipeline runs on from unit to unit (rings and barrier phases are
//     never reset): the next unit's fixed tiles are loaded as soon as the last
//     products that read the old ones have completed, and its first products
//     run beside the epilogue. A CTA changes roles once.
//   * Rows of a tile that lie behind a sequence's end belong to the next
//     sequence or to nobody and may hold anything. Scores of invisible pairs
//     become -inf in tensor memory before the exponential (the tensor core
//     forms -S for a negative scale, as in the forward, and scale = 0 runs as
//     2^-126). Where such rows are summed over (Q and dO in the key-block role,
//     K and V in the query role) they are cleared in shared memory: the tile's
//     load completes on a barrier of its own, warp 11 clears the rows and then
//     completes the tile's barrier in its place, so that nobody else knows.
//     (Clearing in the elementwise warps, behind branches that one step in a
//     sequence takes, slowed their every step: 6 % of the call at d = 128, 13 %
//     at 64.) Elsewhere such rows only reach accumulator rows that are not stored.
// What bounds it: the chain of a step (S, exponentials, dP, dS, two products
// that accumulate) through a full TMEM, and at unit boundaries the epilogue's
// stores (3300 to 4700 cycles). Nine documents, 8192 tokens, 32 heads on 8,
// d = 128: 307-310 us, 0.41 of the measured bf16 rate counting five products per
// visible pair (seven are run, on 1.1 times the visible pairs: 196 us of products;
// tensor pipe busy 60 %; 17 changes of unit per CTA and the list are about a
// fifth); 8192 tokens not causal, 32 heads of their own: 2.32-2.36 ms, 0.60; two
// documents of 4096 tokens, 32 heads on 8, d = 64: 483 us, 0.36 (tensor pipe 44 %).
// Rounding: P and dS enter their products as bf16, the type of the operands beside
// them (2^-8 of each at most; gradients off by 0.0024 of their norm, 0.0017 with both
// in float32); everything that is summed is float32, rounded once.
// Two launches: varlen_bwd_prepare_kernel (the plan by one CTA; -LSE log2(e)
// and -D of every tile row by the others), then the products.
#pragma once

#include <type_traits>

#include "fa_bwd_kernel.cuh"
#include "fa_varlen_kernel.cuh"

namespace fa {

enum : unsigned int {
  kRoleVarDqProducer = 17, kRoleVarDqMma = 18, kRoleVarDqSoftmax = 19,
  kRoleVarDkvProducer = 20, kRoleVarDkvMma = 21, kRoleVarDkvSoftmax = 22,
};

struct VarBwdUnit {
  int q0, nq, kv0, nkv;   // the sequence
  int blk;                // key block (dkdv) or query tile
  int tile0;              // place of the sequence's first query tile (bwd_tile0)
  int dkdv;               // role
  int n;                  // key-block role: query tiles to visit (the last n); query role: key blocks (the first n)
};

struct VarBwdPlan {
  int num_units;          // list entries (each stands for H_kv units)
  int num_dkdv;           // of which the first are the key-block role's
  int num_long;           // the query role's first entries, of more than half its most key blocks
  int next;
  int pad[4];
};

struct VarBwdParams {
  __nv_bfloat16 *dQ, *dK, *dV;
  long long dq_st, dq_sh, dk_st, dk_sh, dv_st, dv_sh;
  VarBwdPlan* plan;
  const VarBwdUnit* list;
  const float* nlse2;     // [H_kv][tile_cap][128]: -LSE * log2(e); -inf for rows that do not exist or see nothing
  const float* ndelta;    // the same shape: -D, or 0
  int tile_cap;
  int H_kv, G, tp;
  int group;              // K/V heads whose units are taken together
  int inv_g;              // ceil(65536 / G): r / G = r * inv_g >> 16 for r < 128
  int causal;
  float scale_log2;       // |scale| * log2(e), at least 2^-126
  float scale;
  uint32_t idesc_s;       // instruction descriptor of S and S^T (A negated when scale < 0)
  unsigned long long timeout_ns;
  int drop_load;
};

// ---------------------------------------------------------------- plan
// Query tiles are kept at places that need no sum over the sequences before:
// floor(q0 / tp) + i for the first tile of sequence i leaves room for the tiles
// of all before it, and the last place is below T_q / tp + B.
__device__ __forceinline__ int bwd_tile0(int q0, int i, int tp) { return q0 / tp + i; }

__device__ __forceinline__ VarBwdUnit make_bwd_unit(const SeqSpan& s, int tile0, int local, int key_blocks, int tiles,
                                                    int tp, int causal) {
  VarBwdUnit u;
  u.q0 = s.q0;
  u.nq = s.nq;
  u.kv0 = s.kv0;
  u.nkv = s.nkv;
  u.tile0 = tile0;
  u.dkdv = local < key_blocks;
  const int shift = s.nkv - s.nq;
  if (u.dkdv) {
    u.blk = local;
    const int first = causal ? max(0, u.blk * 128 - shift) / tp : 0;   // first tile with a row that sees the block
    u.n = max(0, tiles - first);
  } else {
    u.blk = local - key_blocks;
    const int last = min(s.nq, (u.blk + 1) * tp) - 1;
    const int see = causal ? min(s.nkv, last + 1 + shift) : s.nkv;
    u.n = max(1, (max(see, 0) + 127) >> 7);
  }
  return u;
}

__device__ __forceinline__ void varlen_bwd_plan(const int* __restrict__ cu_q, const int* __restrict__ cu_kv,
                                                VarBwdPlan* __restrict__ plan, VarBwdUnit* __restrict__ list, int B,
                                                int T_q, int T_kv, int tp, int causal) {
  __shared__ int cum[kPlanThreads + 1];        // units of the chunk before each sequence
  __shared__ SeqSpan span[kPlanThreads];
  __shared__ int hist[2 * kPlanClasses];       // key-block role, query role
  __shared__ int warp_sums[kPlanThreads / 32];
  __shared__ int top;                          // first place of the query role's classes with an entry
  static_assert(2 * kPlanClasses == kPlanThreads, "one class per thread");
  const int tid = threadIdx.x;
  if (!offsets_ok(cu_q, cu_kv, B, T_q, T_kv)) {
    if (tid == 0) plan->num_units = plan->num_dkdv = plan->num_long = plan->next = 0;
    return;
  }
  hist[tid] = 0;
  if (tid == 0) top = 2 * kPlanClasses - 1;
  int total = 0;
  for (int round = 0; round < 2; ++round) {
    for (int c0 = 0; c0 < B; c0 += kPlanThreads) {
      if (round == 0 || B > kPlanThreads) {
        __syncthreads();
        int nt = 0, nk = 0, sum;
        if (c0 + tid < B) {
          span[tid] = seq_span(cu_q, cu_kv, c0 + tid);
          nt = span[tid].nq / tp + (span[tid].nq % tp != 0);
          nk = (span[tid].nkv + 127) / 128;
        }
        const int incl = block_scan(nt + nk, warp_sums, sum);
        cum[tid + 1] = incl;
        if (tid == 0) cum[0] = 0;
        __syncthreads();
      }
      const int chunk = cum[kPlanThreads];
      for (int e = tid; e < chunk; e += kPlanThreads) {
        int lo = 0, hi = kPlanThreads - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (cum[mid] <= e) lo = mid; else hi = mid - 1;
        }
        const SeqSpan s = span[lo];
        const int nt = s.nq / tp + (s.nq % tp != 0), nk = (s.nkv + 127) / 128;
        const VarBwdUnit u = make_bwd_unit(s, bwd_tile0(s.q0, c0 + lo, tp), e - cum[lo], nk, nt, tp, causal);
        // (the place of a class in `hist`: expensive ones first)
        const int cls = (u.dkdv ? 0 : kPlanClasses) + kPlanClasses - 1 - cost_class(max(1, u.n));
        const int at = atomicAdd(&hist[cls], 1);
        if (round == 1) list[at] = u;
      }
      if (round == 0) total += chunk;
    }
    __syncthreads();
    if (round == 0) {
      int sum;
      const int mine = hist[tid];
      if (mine > 0 && tid >= kPlanClasses) atomicMin(&top, tid);
      const int incl = block_scan(mine, warp_sums, sum);
      hist[tid] = incl - mine;
      __syncthreads();
      if (tid == 0) {
        // Units before the query role's first class; its entries before the class an octave below its top.
        plan->num_dkdv = hist[kPlanClasses];
        plan->num_long = (top + 8 < 2 * kPlanClasses ? hist[top + 8] : sum) - hist[kPlanClasses];
      }
      __syncthreads();
    }
  }
  if (tid == 0) {
    plan->num_units = total;
    plan->next = 0;
  }
}

// ---------------------------------------------------------------- plan and rows
// CTA (0, 0) plans. CTA (1 + place, K/V head) writes -LSE log2(e) and -D of the
// 128 rows of a query tile, in the tile's row order; it finds its sequence by
// bisection and checks that one's offsets itself, so that both parts run at
// once (one after the other, as two launches: 326 us instead of 323 at two
// documents of 4096 tokens, 16 heads on 4). HD / 8 lanes read a row in 16-byte pieces, all of a warp's rows requested before the
// first product.
template <int HD>
__global__ void __launch_bounds__(kPlanThreads)
    varlen_bwd_prepare_kernel(const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ dO,
                              const float* __restrict__ LSE, const int* __restrict__ cu_q,
                              const int* __restrict__ cu_kv, VarBwdPlan* __restrict__ plan,
                              VarBwdUnit* __restrict__ list, float* __restrict__ nlse2, float* __restrict__ ndelta,
                              long long o_st, long long o_sh, long long do_st, long long do_sh, int B, int T_q,
                              int T_kv, int tp, int causal, int tile_cap, int G) {
  constexpr int kRowsPerWarp = 128 / (kPlanThreads / 32);
  constexpr int kLanesPerRow = HD / 8;
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kLoads = kRowsPerWarp / kRowsPerLoad;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    if (blockIdx.y == 0) varlen_bwd_plan(cu_q, cu_kv, plan, list, B, T_q, T_kv, tp, causal);
    return;
  }
  const int tile = blockIdx.x - 1, kvh = blockIdx.y;
  int seq = 0;
  for (int hi = B - 1; seq < hi;) {
    const int mid = seq + (hi - seq + 1) / 2;
    if (bwd_tile0(cu_q[mid], mid, tp) <= tile) seq = mid; else hi = mid - 1;
  }
  const int q0 = cu_q[seq], q1 = cu_q[seq + 1];
  const int local = tile - bwd_tile0(q0, seq, tp);
  if (q0 < 0 || q1 > T_q || q1 <= q0) return;      // (bad offsets are the plan's to report)
  if (local < 0 || local > (q1 - q0 - 1) / tp) return;   // no tile at this place
  const int tok0 = q0 + local * tp;
  const int tokens = min(tp, q1 - tok0);           // of this tile
  const int row0 = (threadIdx.x >> 5) * kRowsPerWarp;
  const int lane = threadIdx.x & 31, sub = lane / kLanesPerRow, piece = lane % kLanesPerRow;
  uint4 o4[kLoads], g4[kLoads];
  float lse[kLoads];
  bool live[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = row0 + i * kRowsPerLoad + sub;
    const int x = row / G, h = kvh * G + row - x * G;
    live[i] = x < tokens;
    o4[i] = g4[i] = make_uint4(0u, 0u, 0u, 0u);
    lse[i] = -INFINITY;
    if (live[i]) {
      const long long t = tok0 + x;
      o4[i] = __ldg(reinterpret_cast<const uint4*>(O + t * o_st + h * o_sh + piece * 8));
      g4[i] = __ldg(reinterpret_cast<const uint4*>(dO + t * do_st + h * do_sh + piece * 8));
      if (piece == 0) lse[i] = __ldg(LSE + static_cast<long long>(h) * T_q + t);
    }
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t ow[4] = {o4[i].x, o4[i].y, o4[i].z, o4[i].w};
    const uint32_t gw[4] = {g4[i].x, g4[i].y, g4[i].z, g4[i].w};
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 of = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ow[e]));
      const float2 gf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gw[e]));
      acc = fmaf(of.x, gf.x, acc);
      acc = fmaf(of.y, gf.y, acc);
    }
#pragma unroll
    for (int s = kLanesPerRow / 2; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if (piece == 0) {
      const long long at = (static_cast<long long>(kvh) * tile_cap + tile) * 128 + row0 + i * kRowsPerLoad + sub;
      const bool sees = live[i] && lse[i] != -INFINITY;
      nlse2[at] = sees ? -lse[i] * 1.4426950408889634074f : -INFINITY;
      ndelta[at] = sees ? -acc : 0.f;
    }
  }
}

// ---------------------------------------------------------------- products
struct VarBwdJob {
  VarBwdUnit u;
  int kvh;       // -1: no more units
};

// Shared by both roles' loops: two job slots, handed over by the fetch warp,
// and the barriers that the warp which clears tails takes part in. At most four
// tiles of a kind are in flight, which is what their rings hold.
template <int HD>
struct VarBwdShared {
  VarBwdJob job[2];
  uint64_t full[2], empty[2];   // empty: warps 0-9 and 11
  uint64_t claim;               // the producer nears the end of a unit's loads
  uint64_t q_full[BwdCfg<HD>::kStages], do_full[BwdCfg<HD>::kStages];    // key-block role: Q_i, dO_i (and their vectors)
  uint64_t k_full[DqCfg<HD>::kKSlots], v_full[DqCfg<HD>::kVSlots];       // query role: K_j, V_j
  uint64_t tail[4][4];          // Q, dO, K, V tiles with rows to clear have landed
};

// A barrier of the ten warps that work on units (the fetch warp is not one).
__device__ __forceinline__ void role_sync() { asm volatile("bar.sync 1, 320;" ::: "memory"); }

// role_sync that tells every thread whether `ok` holds in all of them.
__device__ __forceinline__ bool role_sync_and(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 320, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// issue_tile_qk with the caller's instruction descriptor.
template <int HD>
__device__ __forceinline__ void issue_tile_qk_desc(uint32_t d_tmem, uint32_t a_tile, uint32_t b_tile, uint32_t idesc) {
  const uint64_t a_desc = ptx::desc_kmajor_sw128(a_tile), b_desc = ptx::desc_kmajor_sw128(b_tile);
  if constexpr (HD == 128)
    mma_ss_k128_warp64(d_tmem, ptx::desc_lo(a_desc), ptx::desc_lo(b_desc), ptx::desc_hi(a_desc), idesc, 0u);
  else
    mma_ss_k64_warp64(d_tmem, ptx::desc_lo(a_desc), ptx::desc_lo(b_desc), ptx::desc_hi(a_desc), idesc, 0u);
}

// Zeroes rows [from, to) of the 128-row tile at `tile` (generic address),
// whole 128-byte rows, with `threads` threads.
template <int HD>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int to, int tid, int threads) {
  using C = BwdCfg<HD>;
  for (int c = 0; c < C::kChunks; ++c)
    for (int i = tid; i < (to - from) * 8; i += threads)
      reinterpret_cast<uint4*>(tile + c * C::kChunkBytes + from * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Scores of this thread's row outside columns [from, to) of the 64 at `taddr`
// become -inf. A short loop, out of the way of the blocks that do not need it.
__device__ __forceinline__ void mask_columns(uint32_t taddr, int from, int to) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int lo = from - 32 * c, hi = to - 32 * c;
    if (__all_sync(0xffffffffu, lo <= 0 && hi >= 32)) continue;
    uint32_t r[32];
    ptx::tmem_ld32(taddr + 32 * c, r);
    ptx::tmem_ld_wait();
    ptx::reg_fence32(r);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < lo || i >= hi) r[i] = __float_as_uint(-INFINITY);
    ptx::tmem_st32(taddr + 32 * c, r);
  }
  ptx::tmem_st_wait();
}

// This thread's row of HD / 2 accumulator columns, times `mul`, to bf16.
template <int HD>
__device__ __forceinline__ void store_half_row(uint32_t taddr, float mul, __nv_bfloat16* dst, bool store) {
#pragma unroll 1
  for (int c = 0; c < HD / 64; ++c) store_row32(taddr + 32 * c, mul, dst + 32 * c, store);
}

// The query role: units from job n0 on, to the end of the list.
template <int HD>
__device__ __forceinline__ void varlen_dq_loop(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                               const CUtensorMap& tmdO, const VarBwdParams& p, VarBwdShared<HD>& jobs, int n0,
                                               const uint32_t tmem_base, volatile int* abort_ptr) {
  using C = BwdCfg<HD>;
  using D = DqCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q_full, bar_q_empty;      // Q of the unit
  __shared__ __align__(8) uint64_t bar_do_full, bar_do_empty;    // dO of the unit
  __shared__ __align__(8) uint64_t bar_k_empty[D::kKSlots];
  __shared__ __align__(8) uint64_t bar_v_empty[D::kVSlots];
  __shared__ __align__(8) uint64_t bar_st_full;    // S_j complete
  __shared__ __align__(8) uint64_t bar_dpt_full;   // dP_j complete
  __shared__ __align__(8) uint64_t bar_s_free;     // S_j loaded (and K_{j+1} landed)
  __shared__ __align__(8) uint64_t bar_dp_free;
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_acc_full;
  __shared__ __align__(8) uint64_t bar_drain;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = smem_base;
  const uint32_t sdO = smem_base + C::kTileBytes;
  const uint32_t sK = smem_base + 2 * C::kTileBytes;
  const uint32_t sV = sK + D::kKSlots * C::kTileBytes;

  if (threadIdx.x == 0) {
    for (uint64_t* b : {&bar_q_full, &bar_q_empty, &bar_do_full, &bar_do_empty, &bar_st_full, &bar_dpt_full,
                        &bar_acc_full, &bar_drain})
      ptx::mbar_init(ptx::smem_u32(b), 1);
    for (int s = 0; s < D::kKSlots; ++s) ptx::mbar_init(ptx::smem_u32(&bar_k_empty[s]), 1);
    for (int s = 0; s < D::kVSlots; ++s) ptx::mbar_init(ptx::smem_u32(&bar_v_empty[s]), 1);
    for (uint64_t* b : {&bar_s_free, &bar_dp_free, &bar_p_full[0], &bar_p_full[1]})
      ptx::mbar_init(ptx::smem_u32(b), 256);
    ptx::fence_mbar_init();
  }
  role_sync();

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_once = ptx::policy_evict_first();
      const uint64_t pol_shared = ptx::policy_evict_last();
      int it = 0;        // loads of K (even) and V (odd) so far, in the order K_0, V_0, K_1, ...
      int units = 0;
      int issued[2] = {0, 0};    // loads of Q and dO
      int tails[2] = {0, 0};     // K and V tiles with rows to clear
      bool ok = true;
      VarBwdJob job = {};
      auto load = [&](int j) {
        const int g = it >> 1;
        const bool is_v = it & 1;
        const int slots = is_v ? D::kVSlots : D::kKSlots;
        const int slot = g % slots;
        uint64_t* empty = is_v ? bar_v_empty : bar_k_empty;
        uint64_t* full = is_v ? jobs.v_full : jobs.k_full;
        if (!wait_or_abort(ptx::smem_u32(&empty[slot]), ((g / slots) & 1) ^ 1u, abort_ptr, p.timeout_ns,
                           kRoleVarDqProducer))
          return false;
        const int me = it++;
        if (me == p.drop_load) return true;   // test hook: this tile never arrives
        uint32_t fb = ptx::smem_u32(&full[slot]);
        if ((j + 1) * C::kBlk > job.u.nkv) {     // rows behind the end: warp 11 completes `full`
          fb = ptx::smem_u32(&jobs.tail[2 + is_v][tails[is_v] & 3]);
          ++tails[is_v];
        }
        ptx::mbar_arrive_expect_tx(fb, C::kTileBytes);
        const uint32_t dst = (is_v ? sV : sK) + slot * C::kTileBytes;
        for (int c = 0; c < C::kChunks; ++c)
          ptx::tma_load_3d(dst + c * C::kChunkBytes, is_v ? &tmV : &tmK, fb, c * 64, job.u.kv0 + j * C::kBlk, job.kvh,
                           pol_shared);
        return true;
      };
      for (int n = n0; ok; ++n) {
        ok = wait_or_abort(ptx::smem_u32(&jobs.full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                           kRoleVarDqProducer);
        if (!ok) break;
        job = jobs.job[n & 1];
        if (job.kvh < 0) break;
        ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
        const int token = job.u.q0 + job.u.blk * p.tp;
        const uint32_t bytes = C::kChunks * 128 * p.G * p.tp;
        for (int x = 0; x < 2 && ok; ++x) {     // Q, then dO
          uint64_t& empty = x ? bar_do_empty : bar_q_empty;
          const uint32_t full = ptx::smem_u32(x ? &bar_do_full : &bar_q_full);
          if (units > 0)
            ok = wait_or_abort(ptx::smem_u32(&empty), (units - 1) & 1, abort_ptr, p.timeout_ns, kRoleVarDqProducer);
          if (!ok) break;
          ptx::mbar_arrive_expect_tx(full, bytes);
          for (int c = 0; c < C::kChunks; ++c)
            ptx::tma_load_3d((x ? sdO : sQ) + c * C::kChunkBytes, x ? &tmdO : &tmQ, full, c * 64, job.kvh * p.G, token,
                             pol_once);
          issued[x] = units + 1;
          if (x == 0) ok = load(0);
        }
        if (!ok) break;
        ++units;
        const int claim_at = max(0, job.u.n - 2);
        if (claim_at == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.claim));
        ok = load(0);
        for (int j = 1; j < job.u.n && ok; ++j) {
          if (j == claim_at) ptx::mbar_arrive(ptx::smem_u32(&jobs.claim));
          ok = load(j) && load(j);
        }
      }
      if (!ok || *abort_ptr) {
        // Let every copy this thread started land before the CTA exits.
        if (issued[0] > 0) drain_wait(ptx::smem_u32(&bar_q_full), (issued[0] - 1) & 1, p.timeout_ns);
        if (issued[1] > 0) drain_wait(ptx::smem_u32(&bar_do_full), (issued[1] - 1) & 1, p.timeout_ns);
        for (int x = 0; x < 2; ++x)
          for (int r = max(0, tails[x] - 4); r < tails[x]; ++r)
            drain_wait(ptx::smem_u32(&jobs.tail[2 + x][r & 3]), (r >> 2) & 1, p.timeout_ns);
        for (int i = 0; i < it; ++i) {
          const int g = i >> 1;
          const bool is_v = i & 1;
          const int slots = is_v ? D::kVSlots : D::kKSlots;
          const int last = (it - 1 - (is_v ? 1 : 0)) >> 1;
          if (g + slots <= last || i == p.drop_load) continue;
          drain_wait(ptx::smem_u32(&(is_v ? jobs.v_full : jobs.k_full)[g % slots]), (g / slots) & 1, p.timeout_ns);
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    auto k_tile = [&](int g) { return sK + (g % D::kKSlots) * C::kTileBytes; };
    auto v_tile = [&](int g) { return sV + (g % D::kVSlots) * C::kTileBytes; };
    // S_g = Q K^T and dP_g = dO V^T, each committed to its own barrier. A unit's
    // K_0 and V_0 are waited for here; every later K by the elementwise warps
    // before their s_free, V before their dp_free.
    auto issue_s = [&](int g, bool last) {
      ptx::tc_fence_after();
      issue_tile_qk_desc<HD>(tmem_base + D::kColS, sQ, k_tile(g), p.idesc_s);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_st_full));
      if (last) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty));
    };
    auto issue_dp = [&](int g, bool last) {
      ptx::tc_fence_after();
      issue_tile_qk<HD>(tmem_base + D::kColP, sdO, v_tile(g));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_v_empty[g % D::kVSlots]));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_dpt_full));
      if (last) ptx::mma_commit_warp(ptx::smem_u32(&bar_do_empty));
    };
    auto wait = [&](uint64_t* b, int phase) {
      return wait_warp_or_abort(ptx::smem_u32(b), phase & 1, abort_ptr, p.timeout_ns, kRoleVarDqMma);
    };
    bool ok = true;
    int g = 0, units = 0;        // blocks and units so far
    for (int n = n0; ok; ++n) {
      ok = wait(&jobs.full[n & 1], n >> 1);
      if (!ok) break;
      const int kvh = jobs.job[n & 1].kvh, blocks = jobs.job[n & 1].u.n;
      if (kvh < 0) break;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
      ok = wait(&bar_q_full, units) && wait(&jobs.k_full[g % D::kKSlots], g / D::kKSlots);
      if (ok && g > 0) ok = wait(&bar_s_free, g - 1);
      if (!ok) break;
      issue_s(g, blocks == 1);
      ok = wait(&bar_do_full, units) && wait(&jobs.v_full[g % D::kVSlots], g / D::kVSlots);
      if (ok && g > 0) ok = wait(&bar_dp_free, g - 1);
      if (!ok) break;
      issue_dp(g, blocks == 1);
      ++units;
      for (int j = 0; j < blocks; ++j, ++g) {
        if (j + 1 < blocks) {
          // S_{j+1} as soon as S_j has been read; dP_{j+1} once dP_j has.
          ok = wait(&bar_s_free, g);
          if (!ok) break;
          issue_s(g + 1, j + 2 == blocks);
          ok = wait(&bar_dp_free, g);
          if (!ok) break;
          issue_dp(g + 1, j + 2 == blocks);
        }
        ok = wait(&bar_p_full[g & 1], g >> 1);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_tile_acc<HD, 32>(tmem_base + D::kColDQ, tmem_base + D::kColDS + 64u * (g & 1), k_tile(g), j > 0);
        ptx::mma_commit_warp(ptx::smem_u32(&bar_k_empty[g % D::kKSlots]));
      }
      if (ok) ptx::mma_commit_warp(ptx::smem_u32(&bar_acc_full));
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ dS + epilogue
    const int quarter = warp & 3;
    const int half = warp >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t sl2x2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    const uint32_t tS = tmem_base + lane_addr + D::kColS + 64u * half;
    const uint32_t tP = tmem_base + lane_addr + D::kColP + 64u * half;
    const int xr = (row * p.inv_g) >> 16;    // token of this row within a tile
    auto wait = [&](uint64_t* b, int phase) {
      return wait_warp_or_abort(ptx::smem_u32(b), phase & 1, abort_ptr, p.timeout_ns, kRoleVarDqSoftmax);
    };
    bool ok = true;
    int g = 0, units = 0;
    // What the block loop needs of a unit; the next unit's is read while the
    // last product of this one runs.
    int blocks = 0;
    int limit = 0;       // keys this row sees; rows that do not exist take the last token's
    float nl = 0.f, nd = 0.f;
    auto read_job = [&](int n) {
      if (!wait(&jobs.full[n & 1], n >> 1)) return false;
      const VarBwdJob& job = jobs.job[n & 1];
      if (job.kvh < 0) return false;
      const long long vrow = (static_cast<long long>(job.kvh) * p.tile_cap + job.u.tile0 + job.u.blk) * 128 + row;
      nl = p.nlse2[vrow];
      nd = p.ndelta[vrow];
      blocks = job.u.n;
      limit = job.u.nkv;
      if (p.causal) {
        const int tok0 = job.u.blk * p.tp;
        const int last = min(p.tp, job.u.nq - tok0) - 1;
        limit = max(0, min(limit, tok0 + min(xr, last) + 1 + (limit - job.u.nq)));
      }
      return true;
    };
    bool more = read_job(n0);
    for (int n = n0; more; ++n) {
      const uint64_t nlx2 = ptx::f2_pack(nl, nl);
      const uint64_t ndx2 = ptx::f2_pack(nd, nd);
      for (int j = 0; j < blocks; ++j, ++g) {
        ok = wait(&bar_st_full, g);
        if (!ok) break;
        ptx::tc_fence_after();
        const int valid = limit - j * C::kBlk - 64 * half;   // keys of this warp's 64 that this row sees
        if (!__all_sync(0xffffffffu, valid >= 64)) mask_columns(tS, 0, valid);
        uint32_t s[2][32], dp[2][32];
        ptx::tmem_ld32(tS, s[0]);
        ptx::tmem_ld32(tS + 32, s[1]);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(s[0]);
        ptx::reg_fence32(s[1]);
        if (j + 1 < blocks) {
          // K_{j+1} in place before the hand-off that lets S_{j+1} be issued.
          ok = wait(&jobs.k_full[(g + 1) % D::kKSlots], (g + 1) / D::kKSlots);
          if (!ok) break;
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_s_free));

        // P (float32, kept in s) while dP_j is still on the tensor core.
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x0, x1;
            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])),
                                       sl2x2, nlx2),
                           x0, x1);
            s[c][2 * k] = __float_as_uint(ptx::ex2_approx(x0));
            s[c][2 * k + 1] = __float_as_uint(ptx::ex2_approx(x1));
          }
        }
        ok = wait(&bar_dpt_full, g);
        if (!ok) break;
        ptx::tc_fence_after();
        ptx::tmem_ld32(tP, dp[0]);
        ptx::tmem_ld32(tP + 32, dp[1]);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(dp[0]);
        ptx::reg_fence32(dp[1]);
        if (j + 1 < blocks) {
          // V_{j+1} in place before the hand-off that lets dP_{j+1} be issued.
          ok = wait(&jobs.v_full[(g + 1) % D::kVSlots], (g + 1) / D::kVSlots);
          if (!ok) break;
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_dp_free));
        uint32_t pds[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint64_t t =
                ptx::f2_add(ptx::f2_pack(__uint_as_float(dp[c][2 * k]), __uint_as_float(dp[c][2 * k + 1])), ndx2);
            float d0, d1;
            ptx::f2_unpack(
                ptx::f2_mul(ptx::f2_pack(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), t), d0, d1);
            pds[16 * c + k] = ptx::pack_bf16x2(d0, d1);
          }
        }
        ptx::tmem_st32(tmem_base + lane_addr + D::kColDS + 64u * (g & 1) + 32u * half, pds);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[g & 1]));
      }
      if (!ok) break;
      const VarBwdJob& job = jobs.job[n & 1];
      const int tok0 = job.u.blk * p.tp;
      const bool live = row < p.G * p.tp && xr < job.u.nq - tok0;
      __nv_bfloat16* dst = p.dQ + (static_cast<long long>(job.u.q0) + tok0 + xr) * p.dq_st +
                           (job.kvh * p.G + row - xr * p.G) * p.dq_sh + half * (HD / 2);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
      more = read_job(n + 1);
      ok = wait(&bar_acc_full, units++);
      if (!ok) break;
      ptx::tc_fence_after();
      store_half_row<HD>(tmem_base + lane_addr + D::kColDQ + half * (HD / 2), p.scale, dst, live);
    }
  }
  ptx::tc_fence_before();
  role_sync();
  ptx::tc_fence_after();
}

// The key-block role: units from job 0 on, up to the first job of the other
// role, or none (not released). Returns the number of jobs taken, or -1 when a
// role gave up, the same in every thread.
template <int HD>
__device__ __forceinline__ int varlen_dkdv_loop(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                                const CUtensorMap& tmV, const CUtensorMap& tmdO,
                                                const VarBwdParams& p, VarBwdShared<HD>& jobs, const uint32_t tmem_base,
                                                volatile int* abort_ptr) {
  using C = BwdCfg<HD>;
  constexpr uint32_t kColDV = 0;
  constexpr uint32_t kColDK = HD;
  constexpr uint32_t kColR = 2 * HD;    // R0 = kColR, R1 = kColR + 128
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_k_full, bar_k_empty;     // K of the unit
  __shared__ __align__(8) uint64_t bar_v_full, bar_v_empty;     // V of the unit
  __shared__ __align__(8) uint64_t bar_q_empty[C::kStages];     // dK(i) done with Q_i
  __shared__ __align__(8) uint64_t bar_do_empty[C::kStages];    // dV(i) done with dO_i
  __shared__ __align__(8) uint64_t bar_st_full;
  __shared__ __align__(8) uint64_t bar_dpt_full;
  __shared__ __align__(8) uint64_t bar_dp_free;
  __shared__ __align__(8) uint64_t bar_p_full;
  __shared__ __align__(8) uint64_t bar_pt_stored;
  __shared__ __align__(8) uint64_t bar_acc_full;
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ int taken;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int box_rows = p.G * p.tp;
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;
  const uint32_t sK = smem_base;
  const uint32_t sV = smem_base + C::kTileBytes;
  const uint32_t sRing = smem_base + C::kPairBytes;                     // slot s: Q_i, then dO_i
  const uint32_t sVec = sRing + C::kStages * C::kPairBytes;             // slot s: [-lse2 x 128][-D x 128]
  const float* vec = reinterpret_cast<const float*>(smem_raw + (sVec - raw));

  if (threadIdx.x == 0) {
    for (uint64_t* b : {&bar_k_full, &bar_k_empty, &bar_v_full, &bar_v_empty, &bar_st_full, &bar_dpt_full,
                        &bar_acc_full, &bar_drain})
      ptx::mbar_init(ptx::smem_u32(b), 1);
    for (int s = 0; s < C::kStages; ++s)
      for (uint64_t* b : {&bar_q_empty[s], &bar_do_empty[s]}) ptx::mbar_init(ptx::smem_u32(b), 1);
    for (uint64_t* b : {&bar_dp_free, &bar_p_full, &bar_pt_stored}) ptx::mbar_init(ptx::smem_u32(b), 256);
    ptx::fence_mbar_init();
  }
  // Rows of the ring that no load writes are zero.
  if (box_rows < C::kBlk && warp < 8) {
    for (int s = 0; s < 2 * C::kStages; ++s)
      clear_rows<HD>(smem_raw + (sRing - raw) + s * C::kTileBytes, box_rows, C::kBlk, threadIdx.x, 256);
    ptx::fence_proxy_async_smem();
  }
  role_sync();

  bool ok = true;
  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_shared = ptx::policy_evict_last();
      const uint32_t bytes = C::kChunks * 128 * box_rows + C::kBlk * 4;
      int g = 0, units = 0, n = 0;          // query tiles, units, jobs so far
      int issued_k = 0, issued_q = 0, issued_do = 0;
      int tails_q = 0, tails_do = 0;        // Q and dO tiles with rows to clear
      for (; ok; ++n) {
        ok = wait_or_abort(ptx::smem_u32(&jobs.full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                           kRoleVarDkvProducer);
        if (!ok) break;
        const VarBwdJob job = jobs.job[n & 1];
        if (job.kvh < 0 || !job.u.dkdv) break;
        ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
        const int tile_first = (job.u.nq + p.tp - 1) / p.tp - job.u.n;   // first query tile to visit
        const int claim_at = max(0, job.u.n - 2);
        if (job.u.n == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.claim));
        for (int i = 0; i < job.u.n && ok; ++i, ++g) {
          if (i == claim_at) ptx::mbar_arrive(ptx::smem_u32(&jobs.claim));
          const int slot = g % C::kStages;
          const uint32_t par = ((g / C::kStages) & 1) ^ 1u;
          const uint32_t dst = sRing + slot * C::kPairBytes;
          const int token = job.u.q0 + (tile_first + i) * p.tp;
          // Rows behind the end: warp 11 completes the tiles' barriers.
          const bool tail = (tile_first + i + 1) * p.tp > job.u.nq;
          const long long voff =
              (static_cast<long long>(job.kvh) * p.tile_cap + job.u.tile0 + tile_first + i) * C::kBlk;
          if (i == 0) {
            if (units > 0)
              ok = wait_or_abort(ptx::smem_u32(&bar_k_empty), (units - 1) & 1, abort_ptr, p.timeout_ns,
                                 kRoleVarDkvProducer);
            if (!ok) break;
            const uint32_t full = ptx::smem_u32(&bar_k_full);
            ptx::mbar_arrive_expect_tx(full, C::kTileBytes);
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_3d(sK + c * C::kChunkBytes, &tmK, full, c * 64, job.u.kv0 + job.u.blk * C::kBlk, job.kvh,
                               pol_shared);
            issued_k = units + 1;
          }
          if (!wait_or_abort(ptx::smem_u32(&bar_q_empty[slot]), par, abort_ptr, p.timeout_ns, kRoleVarDkvProducer)) {
            ok = false;
            break;
          }
          issued_q = g + 1;
          if (g != p.drop_load) {    // test hook: this step's tiles never arrive
            const uint32_t full = ptx::smem_u32(tail ? &jobs.tail[0][tails_q++ & 3] : &jobs.q_full[slot]);
            ptx::mbar_arrive_expect_tx(full, bytes);
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_3d(dst + c * C::kChunkBytes, &tmQ, full, c * 64, job.kvh * p.G, token, pol_shared);
            ptx::bulk_load_1d(sVec + slot * C::kVecBytes, p.nlse2 + voff, C::kBlk * 4, full, pol_shared);
          }
          if (i == 0) {
            if (units > 0)
              ok = wait_or_abort(ptx::smem_u32(&bar_v_empty), (units - 1) & 1, abort_ptr, p.timeout_ns,
                                 kRoleVarDkvProducer);
            if (!ok) break;
            const uint32_t full = ptx::smem_u32(&bar_v_full);
            ptx::mbar_arrive_expect_tx(full, C::kTileBytes);
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_3d(sV + c * C::kChunkBytes, &tmV, full, c * 64, job.u.kv0 + job.u.blk * C::kBlk, job.kvh,
                               pol_shared);
            ++units;
          }
          if (!wait_or_abort(ptx::smem_u32(&bar_do_empty[slot]), par, abort_ptr, p.timeout_ns, kRoleVarDkvProducer)) {
            ok = false;
            break;
          }
          issued_do = g + 1;
          if (g != p.drop_load) {
            const uint32_t full = ptx::smem_u32(tail ? &jobs.tail[1][tails_do++ & 3] : &jobs.do_full[slot]);
            ptx::mbar_arrive_expect_tx(full, bytes);
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_3d(dst + C::kTileBytes + c * C::kChunkBytes, &tmdO, full, c * 64, job.kvh * p.G, token,
                               pol_shared);
            ptx::bulk_load_1d(sVec + slot * C::kVecBytes + C::kBlk * 4, p.ndelta + voff, C::kBlk * 4, full,
                              pol_shared);
          }
        }
      }
      taken = n;
      if (!ok || *abort_ptr) {
        // Let every copy this thread started land before the CTA exits.
        if (issued_k > 0) drain_wait(ptx::smem_u32(&bar_k_full), (issued_k - 1) & 1, p.timeout_ns);
        if (units > 0) drain_wait(ptx::smem_u32(&bar_v_full), (units - 1) & 1, p.timeout_ns);
        for (int r = max(0, tails_q - 4); r < tails_q; ++r)
          drain_wait(ptx::smem_u32(&jobs.tail[0][r & 3]), (r >> 2) & 1, p.timeout_ns);
        for (int r = max(0, tails_do - 4); r < tails_do; ++r)
          drain_wait(ptx::smem_u32(&jobs.tail[1][r & 3]), (r >> 2) & 1, p.timeout_ns);
        for (int i = issued_q > C::kStages ? issued_q - C::kStages : 0; i < issued_q; ++i)
          if (i != p.drop_load)
            drain_wait(ptx::smem_u32(&jobs.q_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
        for (int i = issued_do > C::kStages ? issued_do - C::kStages : 0; i < issued_do; ++i)
          if (i != p.drop_load)
            drain_wait(ptx::smem_u32(&jobs.do_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (as in bwd_dkdv_cta)
    auto region = [&](int g) { return tmem_base + kColR + 128u * static_cast<uint32_t>(g & 1); };
    auto q_tile = [&](int g) { return sRing + (g % C::kStages) * C::kPairBytes; };
    auto wait = [&](uint64_t* b, int phase) {
      return wait_warp_or_abort(ptx::smem_u32(b), phase & 1, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
    };
    // S_g^T = K Q^T; `last`: the unit's last use of K.
    auto issue_s = [&](int g, bool last) {
      ptx::tc_fence_after();
      issue_tile_qk_desc<HD>(region(g), sK, q_tile(g), p.idesc_s);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_st_full));
      if (last) ptx::mma_commit_warp(ptx::smem_u32(&bar_k_empty));
    };
    // dP_g^T = V dO^T, then, once P^T is in place, dV += P^T dO.
    auto issue_dp_dv = [&](int g, bool first, bool last) {
      ptx::tc_fence_after();
      issue_tile_qk<HD>(region(g + 1), sV, q_tile(g) + C::kTileBytes);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_dpt_full));
      if (last) ptx::mma_commit_warp(ptx::smem_u32(&bar_v_empty));
      if (!wait(&bar_pt_stored, g)) return false;
      ptx::tc_fence_after();
      issue_tile_acc<HD, 64>(tmem_base + kColDV, region(g), q_tile(g) + C::kTileBytes, !first);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_do_empty[g % C::kStages]));
      return true;
    };
    int g = 0, units = 0;
    for (int n = 0; ok; ++n) {
      ok = wait(&jobs.full[n & 1], n >> 1);
      if (!ok) break;
      const int kvh = jobs.job[n & 1].kvh, steps = jobs.job[n & 1].u.n, mine = jobs.job[n & 1].u.dkdv;
      if (kvh < 0 || !mine) break;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
      if (steps == 0) continue;     // no query rows: the elementwise warps store zeros
      ok = wait(&bar_k_full, units) && wait(&jobs.q_full[g % C::kStages], g / C::kStages);
      if (!ok) break;
      issue_s(g, steps == 1);
      ok = wait(&bar_v_full, units) && wait(&jobs.do_full[g % C::kStages], g / C::kStages);
      if (!ok) break;
      ++units;
      ok = issue_dp_dv(g, true, steps == 1);
      for (int i = 0; i < steps && ok; ++i, ++g) {
        // S_{i+1}^T goes in as soon as its region is free (dp_free(i)) and
        // Q_{i+1} has landed, if that happens before p_full(i); otherwise
        // after dK(i). A late Q must not hold back dK(i), whose commit frees
        // the ring slot the next copy needs.
        bool s_issued = false;
        const bool more = i + 1 < steps, last = i + 2 == steps;
        const int s1 = (g + 1) % C::kStages;
        const int in_phase = (g + 1) / C::kStages;
        if (more) {
          ok = wait(&bar_dp_free, g);
          if (!ok) break;
          const uint64_t t0 = ptx::globaltimer_ns();
          while (true) {
            if (__all_sync(0xffffffffu, ptx::mbar_test_wait(ptx::smem_u32(&jobs.q_full[s1]), in_phase & 1))) {
              issue_s(g + 1, last);
              s_issued = true;
              break;
            }
            if (__all_sync(0xffffffffu, ptx::mbar_test_wait(ptx::smem_u32(&bar_p_full), g & 1))) break;
            // Out of time or aborting: the bounded wait below reports it.
            if (__any_sync(0xffffffffu, *abort_ptr != 0) || ptx::globaltimer_ns() - t0 > p.timeout_ns) break;
            __nanosleep(32);
          }
        }
        ok = wait(&bar_p_full, g);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_tile_acc<HD, 64>(tmem_base + kColDK, region(g) + 32, q_tile(g), i > 0);             // dK += dS^T Q_i
        ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[g % C::kStages]));
        if (more) {
          if (!s_issued) {
            ok = wait(&jobs.q_full[s1], in_phase);
            if (!ok) break;
            issue_s(g + 1, last);
          }
          ok = wait(&jobs.do_full[s1], in_phase);
          if (!ok) break;
          ok = issue_dp_dv(g + 1, false, last);
        }
      }
      if (ok) ptx::mma_commit_warp(ptx::smem_u32(&bar_acc_full));
    }
    if (!ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ P, dS + epilogue
    const int quarter = warp & 3;
    const int half = warp >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t sl2x2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    auto wait = [&](uint64_t* b, int phase) {
      return wait_warp_or_abort(ptx::smem_u32(b), phase & 1, abort_ptr, p.timeout_ns, kRoleVarDkvSoftmax);
    };
    int g = 0, units = 0;
    // What the step loop needs of a unit; the next unit's is read while the
    // last product of this one runs.
    int steps = 0;
    int tok0 = 0;        // first token of the step's tile
    int see0 = 0;        // first token of the sequence that sees this key (causal)
    auto read_job = [&](int n) {
      ok = wait(&jobs.full[n & 1], n >> 1);
      const VarBwdJob& job = jobs.job[n & 1];
      if (!ok || job.kvh < 0 || !job.u.dkdv) return false;
      steps = job.u.n;
      tok0 = ((job.u.nq + p.tp - 1) / p.tp - steps) * p.tp;
      see0 = p.causal ? job.u.blk * C::kBlk + row - (job.u.nkv - job.u.nq) : 0;
      return true;
    };
    bool more = read_job(0);
    for (int n = 0; more; ++n) {
      for (int i = 0; i < steps; ++i, ++g, tok0 += p.tp) {
        // Columns x * G + h of this warp's 64 that see this key: from here on.
        const int from = max(0, min(see0 - tok0, p.tp)) * p.G - 64 * half;
        // P^T as soon as S^T(i) is complete (it overlaps the tensor core's dK/dV
        // of the previous block and dP^T of this one), then dS^T once dP^T(i) is.
        ok = wait(&bar_st_full, g);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t tS = tmem_base + lane_addr + kColR + 128u * (g & 1) + 64u * half;
        const uint32_t tP = tmem_base + lane_addr + kColR + 128u * ((g + 1) & 1) + 64u * half;
        if (!__all_sync(0xffffffffu, from <= 0)) mask_columns(tS, from, 64);
        uint32_t s[2][32], dp[2][32];
        ptx::tmem_ld32(tS, s[0]);
        ptx::tmem_ld32(tS + 32, s[1]);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(s[0]);
        ptx::reg_fence32(s[1]);
        // -LSE*log2e and -D of this warp's 64 query columns (broadcast reads).
        const float4* vl = reinterpret_cast<const float4*>(vec + (g % C::kStages) * (C::kVecBytes / 4) + 64 * half);
        const float4* vd = vl + 32;    // + 128 floats
        {
          uint32_t pp[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const float4 l4 = vl[8 * c + v];
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                const int e = 4 * v + 2 * h2;
                const uint64_t nl2 = h2 ? ptx::f2_pack(l4.z, l4.w) : ptx::f2_pack(l4.x, l4.y);
                float x0, x1;
                ptx::f2_unpack(
                    ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), sl2x2, nl2), x0,
                    x1);
                const float p0 = ptx::ex2_approx(x0);
                const float p1 = ptx::ex2_approx(x1);
                s[c][e] = __float_as_uint(p0);
                s[c][e + 1] = __float_as_uint(p1);
                pp[16 * c + 2 * v + h2] = ptx::pack_bf16x2(p0, p1);
              }
            }
          }
          ptx::tmem_st32(tS, pp);
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(ptx::smem_u32(&bar_pt_stored));
        }
        ok = wait(&bar_dpt_full, g);
        if (!ok) break;
        ptx::tc_fence_after();
        ptx::tmem_ld32(tP, dp[0]);
        ptx::tmem_ld32(tP + 32, dp[1]);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(dp[0]);
        ptx::reg_fence32(dp[1]);
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_dp_free));
        uint32_t pds[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const float4 d4 = vd[8 * c + v];
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const int e = 4 * v + 2 * h2;
              const uint64_t nd2 = h2 ? ptx::f2_pack(d4.z, d4.w) : ptx::f2_pack(d4.x, d4.y);
              const uint64_t t =
                  ptx::f2_add(ptx::f2_pack(__uint_as_float(dp[c][e]), __uint_as_float(dp[c][e + 1])), nd2);
              float d0, d1;
              ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), t), d0,
                             d1);
              pds[16 * c + 2 * v + h2] = ptx::pack_bf16x2(d0, d1);
            }
          }
        }
        ptx::tmem_st32(tS + 32, pds);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full));
      }
      if (!ok) break;
      const VarBwdJob& job = jobs.job[n & 1];
      const int key_row = job.u.blk * C::kBlk + row;
      const bool live = key_row < job.u.nkv;
      const long long key = static_cast<long long>(job.u.kv0) + key_row;
      __nv_bfloat16* dv = p.dV + key * p.dv_st + job.kvh * p.dv_sh + half * (HD / 2);
      __nv_bfloat16* dk = p.dK + key * p.dk_st + job.kvh * p.dk_sh + half * (HD / 2);
      const bool any = steps > 0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
      more = read_job(n + 1);
      if (!ok) break;
      if (any) {
        ok = wait(&bar_acc_full, units++);
        if (!ok) break;
        ptx::tc_fence_after();
        store_half_row<HD>(tmem_base + lane_addr + kColDV + half * (HD / 2), 1.f, dv, live);
        store_half_row<HD>(tmem_base + lane_addr + kColDK + half * (HD / 2), p.scale, dk, live);
      } else if (live) {   // a sequence without query rows
        for (int c = 0; c < HD / 16; ++c) {
          reinterpret_cast<uint4*>(dv)[c] = make_uint4(0u, 0u, 0u, 0u);
          reinterpret_cast<uint4*>(dk)[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  }
  ptx::tc_fence_before();
  const bool all_ok = role_sync_and(ok);
  ptx::tc_fence_after();
  return all_ok ? taken : -1;
}

// The warp that clears rows behind a sequence's end: the last Q and dO tiles
// of a key-block unit, the last K and V tiles of a query unit.
template <int HD>
__device__ __forceinline__ void varlen_bwd_tails(const VarBwdParams& p, VarBwdShared<HD>& jobs,
                                                 volatile int* abort_ptr) {
  using C = BwdCfg<HD>;
  using D = DqCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int lane = threadIdx.x & 31;
  int g[2] = {0, 0}, tails[2] = {0, 0};      // steps and tail pairs so far, per role
  for (int n = 0;; ++n) {
    if (!wait_idle_or_abort(ptx::smem_u32(&jobs.full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                            kRoleVarDkvProducer))
      return;
    const int kvh = jobs.job[n & 1].kvh, dkdv = jobs.job[n & 1].u.dkdv, steps = jobs.job[n & 1].u.n;
    const int nq = jobs.job[n & 1].u.nq, nkv = jobs.job[n & 1].u.nkv;
    __syncwarp();
    if (kvh < 0) return;
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&jobs.empty[n & 1]));
    const int r = dkdv ? 0 : 1;
    g[r] += steps;
    // Rows [from, to) of the unit's last streamed pair of tiles.
    const int tiles = (nq + p.tp - 1) / p.tp;
    const int from = dkdv ? (nq - (tiles - 1) * p.tp) * p.G : max(0, nkv - (steps - 1) * C::kBlk);
    const int to = dkdv ? p.G * p.tp : C::kBlk;
    if (steps == 0 || from >= to) continue;
    const int last = g[r] - 1;
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      if (!wait_warp_or_abort(ptx::smem_u32(&jobs.tail[2 * r + x][tails[r] & 3]), (tails[r] >> 2) & 1, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRoleVarDkvProducer))
        return;
      uint8_t* tile;
      uint64_t* full;
      if (dkdv) {
        tile = base + C::kPairBytes + (last % C::kStages) * C::kPairBytes + x * C::kTileBytes;
        full = (x ? jobs.do_full : jobs.q_full) + last % C::kStages;
      } else {
        tile = base + (2 + (x ? D::kKSlots + last % D::kVSlots : last % D::kKSlots)) * C::kTileBytes;
        full = x ? jobs.v_full + last % D::kVSlots : jobs.k_full + last % D::kKSlots;
      }
      clear_rows<HD>(tile, from, to, lane, 32);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(full));
    }
    ++tails[r];
  }
}

// The ten warps of BwdCfg, the fetch warp and the one that clears tails. (All keep
// the 168 registers of the launch: 216 for the elementwise warps, which needs a
// copy of the loops for them alone, was 2 to 5 % slower.)
constexpr int kVarBwdThreads = 384;

template <int HD>
__global__ void __launch_bounds__(kVarBwdThreads, 1)
    fa_varlen_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                         const VarBwdParams p) {
  using C = BwdCfg<HD>;
  __shared__ __align__(16) VarBwdShared<HD> jobs;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int* abort_ptr = &abort_flag;
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(ptx::smem_u32(&jobs.full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&jobs.empty[s]), 11);
    }
    for (uint64_t& b : jobs.q_full) ptx::mbar_init(ptx::smem_u32(&b), 1);
    for (uint64_t& b : jobs.do_full) ptx::mbar_init(ptx::smem_u32(&b), 1);
    for (uint64_t& b : jobs.k_full) ptx::mbar_init(ptx::smem_u32(&b), 1);
    for (uint64_t& b : jobs.v_full) ptx::mbar_init(ptx::smem_u32(&b), 1);
    for (int x = 0; x < 16; ++x) ptx::mbar_init(ptx::smem_u32(&jobs.tail[x >> 2][x & 3]), 1);
    ptx::mbar_init(ptx::smem_u32(&jobs.claim), 1);
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 256) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    ptx::prefetch_tmap(&tmdO);
  }
  // Every thread reads what the launches before wrote (the list, the rows' values).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  // (As one lambda: as plain calls in a branch the compiled loops are 4 % slower.)
  auto work = [&] {
    const int n = varlen_dkdv_loop<HD>(tmQ, tmK, tmV, tmdO, p, jobs, tmem_base, abort_ptr);
    if (n >= 0) varlen_dq_loop<HD>(tmQ, tmK, tmV, tmdO, p, jobs, n, tmem_base, abort_ptr);
  };
  if (warp < 10) {
    work();
  } else if (warp == 10) {
    // ------------------------------------------------------------ unit fetch (converged; lane 0 writes)
    // (A unit is taken when the loads of the one before near their end.)
    {
      const int total = p.plan->num_units * p.H_kv;
      int idx = blockIdx.x;
      for (int n = 0;; ++n) {
        VarBwdJob job;
        job.kvh = -1;
        job.u.dkdv = 0;
        if (idx < total) {
          const int n_k = p.plan->num_dkdv, in_k = n_k * p.H_kv;
          int e;
          if (idx < in_k) {
            place_unit(idx, n_k, p.H_kv, p.group, &e, &job.kvh);       // (the other role evens out its end)
          } else {
            place_unit(idx - in_k, p.plan->num_long, p.H_kv, p.group, &e, &job.kvh);
            e += n_k;
          }
          job.u = p.list[e];
        }
        if (!wait_idle_or_abort(ptx::smem_u32(&jobs.empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr, p.timeout_ns,
                                kRoleVarDqProducer))
          break;
        if (lane == 0) {
          jobs.job[n & 1] = job;
          ptx::mbar_arrive(ptx::smem_u32(&jobs.full[n & 1]));
        }
        __syncwarp();
        if (job.kvh < 0) break;
        if (!wait_idle_or_abort(ptx::smem_u32(&jobs.claim), n & 1, abort_ptr, p.timeout_ns, kRoleVarDqProducer)) break;
        if (lane == 0) idx = static_cast<int>(gridDim.x) + atomicAdd(&p.plan->next, 1);
        idx = __shfl_sync(0xffffffffu, idx, 0);
      }
    }
    __syncwarp();
  } else {
    varlen_bwd_tails<HD>(p, jobs, abort_ptr);
  }
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace fa
