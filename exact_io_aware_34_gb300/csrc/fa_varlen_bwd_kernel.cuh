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
//   * The units of both roles are listed by varlen_bwd_plan_kernel, the
//     most expensive first, and a persistent grid takes them by a counter.
//   * Rows of a tile that lie behind a sequence's end belong to the next
//     sequence or to nobody and may hold anything. In the query role they only
//     reach accumulator rows that are not stored; where they are summed over
//     (Q and dO in the key-block role, K in the query role) they are cleared
//     in shared memory once the products that form S and dP have read them,
//     and their P and dS are zeroed by selection.
// Three launches: the plan; -LSE log2(e) and -D of every tile row
// (varlen_bwd_rows_kernel); the products.
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
  int tile0;              // number of the sequence's first query tile among all sequences'
  int dkdv;               // role
  int n;                  // key-block role: query tiles to visit (the last n); query role: key blocks (the first n)
};

struct VarBwdPlan {
  int num_units;          // list entries (each stands for H_kv units)
  int num_tiles;
  int next;
  int pad[5];
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
  int causal;
  float scale_log2, scale;
  unsigned long long timeout_ns;
  int drop_load;
};

// ---------------------------------------------------------------- plan
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

__global__ void __launch_bounds__(kPlanThreads)
    varlen_bwd_plan_kernel(const int* __restrict__ cu_q, const int* __restrict__ cu_kv, VarBwdPlan* __restrict__ plan,
                           VarBwdUnit* __restrict__ list, int2* __restrict__ tiles, int B, int T_q, int T_kv, int tp,
                           int causal) {
  __shared__ int cum[kPlanThreads + 1];        // units of the chunk before each sequence
  __shared__ int cum_t[kPlanThreads + 1];      // its query tiles
  __shared__ SeqSpan span[kPlanThreads];
  __shared__ int hist[kPlanClasses];
  __shared__ int warp_sums[kPlanThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (!offsets_ok(cu_q, cu_kv, B, T_q, T_kv)) {
    if (tid == 0) plan->num_units = plan->num_tiles = plan->next = 0;
    return;
  }
  if (tid < kPlanClasses) hist[tid] = 0;
  int total = 0, total_tiles = 0;
  for (int round = 0; round < 2; ++round) {
    int tile_base = 0;
    for (int c0 = 0; c0 < B; c0 += kPlanThreads) {
      if (round == 0 || B > kPlanThreads) {
        __syncthreads();
        int nt = 0, nk = 0, sum;
        if (c0 + tid < B) {
          span[tid] = seq_span(cu_q, cu_kv, c0 + tid);
          nt = span[tid].nq / tp + (span[tid].nq % tp != 0);
          nk = (span[tid].nkv + 127) / 128;
        }
        const int incl_t = block_scan(nt, warp_sums, sum);
        cum_t[tid + 1] = incl_t;
        const int incl = block_scan(nt + nk, warp_sums, sum);
        cum[tid + 1] = incl;
        if (tid == 0) cum[0] = cum_t[0] = 0;
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
        const VarBwdUnit u = make_bwd_unit(s, tile_base + cum_t[lo], e - cum[lo], nk, nt, tp, causal);
        const int cls = cost_class(max(1, (u.dkdv ? 4 : 3) * u.n));
        const int at = atomicAdd(&hist[cls], 1);
        if (round == 1) list[at] = u;
        if (round == 0 && !u.dkdv) tiles[u.tile0 + u.blk] = make_int2(s.q0 + u.blk * tp, min(tp, s.nq - u.blk * tp));
      }
      if (round == 0) total += chunk;
      tile_base += cum_t[kPlanThreads];
    }
    total_tiles = tile_base;
    __syncthreads();
    if (round == 0) {
      int sum;
      const int mine = tid < kPlanClasses ? hist[kPlanClasses - 1 - tid] : 0;
      const int incl = block_scan(mine, warp_sums, sum);
      if (tid < kPlanClasses) hist[kPlanClasses - 1 - tid] = incl - mine;
      __syncthreads();
    }
  }
  if (tid == 0) {
    plan->num_units = total;
    plan->num_tiles = total_tiles;
    plan->next = 0;
  }
}

// ---------------------------------------------------------------- rows
// -LSE log2(e) and -D of the 128 rows of every (K/V head, query tile), in the
// tile's row order. One CTA per 64 rows; HD / 8 lanes read a row in 16-byte
// pieces, all of a warp's rows requested before the first product.
template <int HD>
__global__ void __launch_bounds__(256)
    varlen_bwd_rows_kernel(const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ dO,
                           const float* __restrict__ LSE, const VarBwdPlan* plan, const int2* tiles, float* nlse2,
                           float* ndelta, long long o_st, long long o_sh, long long do_st, long long do_sh, int T_q,
                           int tile_cap, int G) {
  constexpr int kRowsPerWarp = 8;
  constexpr int kLanesPerRow = HD / 8;
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kLoads = kRowsPerWarp / kRowsPerLoad;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tile = blockIdx.x >> 1, kvh = blockIdx.y;
  if (tile >= plan->num_tiles) return;
  const int2 tl = tiles[tile];
  const int row0 = (blockIdx.x & 1) * 64 + (threadIdx.x >> 5) * kRowsPerWarp;
  const int lane = threadIdx.x & 31, sub = lane / kLanesPerRow, piece = lane % kLanesPerRow;
  uint4 o4[kLoads], g4[kLoads];
  float lse[kLoads];
  bool live[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = row0 + i * kRowsPerLoad + sub;
    const int x = row / G, h = kvh * G + row - x * G;
    live[i] = x < tl.y;
    o4[i] = g4[i] = make_uint4(0u, 0u, 0u, 0u);
    lse[i] = -INFINITY;
    if (live[i]) {
      const long long t = tl.x + x;
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

// Zeroes rows [from, to) of the 128-row tile at `tile` (generic address),
// whole 128-byte rows, with 256 threads.
template <int HD>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int to, int tid) {
  using C = BwdCfg<HD>;
  for (int c = 0; c < C::kChunks; ++c)
    for (int i = tid; i < (to - from) * 8; i += 256)
      reinterpret_cast<uint4*>(tile + c * C::kChunkBytes + from * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Takes the next unit off the list (one thread).
__device__ __forceinline__ void fetch_job(const VarBwdParams& p, int idx, VarBwdJob* job) {
  job->kvh = -1;
  if (idx < p.plan->num_units * p.H_kv) {
    const int e = idx / p.H_kv;
    job->u = p.list[e];
    job->kvh = idx - e * p.H_kv;
  }
}

// A unit of the query role. Barriers live for the unit: initialised here, and
// every arrival on them has been waited for or made by a thread of this CTA
// before the closing __syncthreads.
template <int HD>
__device__ __forceinline__ bool varlen_dq_unit(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                               const CUtensorMap& tmdO, const VarBwdParams& p, const VarBwdUnit u,
                                               const int kvh, const uint32_t tmem_base, volatile int* abort_ptr,
                                               VarBwdJob* next_job) {
  using C = BwdCfg<HD>;
  using D = DqCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_in_full;
  __shared__ __align__(8) uint64_t bar_k_full[D::kKSlots];
  __shared__ __align__(8) uint64_t bar_k_empty[D::kKSlots];
  __shared__ __align__(8) uint64_t bar_v_full[D::kVSlots];
  __shared__ __align__(8) uint64_t bar_v_empty[D::kVSlots];
  __shared__ __align__(8) uint64_t bar_st_full;
  __shared__ __align__(8) uint64_t bar_dpt_full;
  __shared__ __align__(8) uint64_t bar_s_free;
  __shared__ __align__(8) uint64_t bar_dp_free;
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_acc_full;
  __shared__ __align__(8) uint64_t bar_drain;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n = u.n;
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = smem_base;
  const uint32_t sdO = smem_base + C::kTileBytes;
  const uint32_t sK = smem_base + 2 * C::kTileBytes;
  const uint32_t sV = sK + D::kKSlots * C::kTileBytes;

  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&bar_in_full), 1);
    for (int s = 0; s < D::kKSlots; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_k_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_k_empty[s]), 1);
    }
    for (int s = 0; s < D::kVSlots; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_v_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_v_empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bar_st_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_dpt_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_s_free), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_dp_free), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_p_full[0]), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_p_full[1]), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_acc_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_once = ptx::policy_evict_first();
      const uint64_t pol_shared = ptx::policy_evict_last();
      const uint32_t in_full = ptx::smem_u32(&bar_in_full);
      const int token = u.q0 + u.blk * p.tp;
      ptx::mbar_arrive_expect_tx(in_full, 2 * C::kChunks * 128 * p.G * p.tp);
      for (int c = 0; c < C::kChunks; ++c) {
        ptx::tma_load_3d(sQ + c * C::kChunkBytes, &tmQ, in_full, c * 64, kvh * p.G, token, pol_once);
        ptx::tma_load_3d(sdO + c * C::kChunkBytes, &tmdO, in_full, c * 64, kvh * p.G, token, pol_once);
      }
      int issued = 0;    // loads started, in the order K_0, V_0, K_1, V_1, ...
      bool ok = true;
      for (int it = 0; it < 2 * n && ok; ++it) {
        const int j = it >> 1;
        const bool is_v = it & 1;
        const int slots = is_v ? D::kVSlots : D::kKSlots;
        const int slot = j % slots;
        uint64_t* empty = is_v ? bar_v_empty : bar_k_empty;
        uint64_t* full = is_v ? bar_v_full : bar_k_full;
        if (!wait_or_abort(ptx::smem_u32(&empty[slot]), ((j / slots) & 1) ^ 1u, abort_ptr, p.timeout_ns,
                           kRoleVarDqProducer)) {
          ok = false;
          break;
        }
        issued = it + 1;
        if (it == p.drop_load) continue;   // test hook: this tile never arrives
        const uint32_t fb = ptx::smem_u32(&full[slot]);
        ptx::mbar_arrive_expect_tx(fb, C::kTileBytes);
        const uint32_t dst = (is_v ? sV : sK) + slot * C::kTileBytes;
        for (int c = 0; c < C::kChunks; ++c)
          ptx::tma_load_3d(dst + c * C::kChunkBytes, is_v ? &tmV : &tmK, fb, c * 64, u.kv0 + j * C::kBlk, kvh,
                           pol_shared);
      }
      if (ok) fetch_job(p, static_cast<int>(gridDim.x) + atomicAdd(&p.plan->next, 1), next_job);
      // The issuer's last arrivals on the empty barriers.
      for (int j = max(0, n - D::kKSlots); j < n && ok; ++j)
        ok = wait_or_abort(ptx::smem_u32(&bar_k_empty[j % D::kKSlots]), (j / D::kKSlots) & 1, abort_ptr, p.timeout_ns,
                           kRoleVarDqProducer);
      for (int j = max(0, n - D::kVSlots); j < n && ok; ++j)
        ok = wait_or_abort(ptx::smem_u32(&bar_v_empty[j % D::kVSlots]), (j / D::kVSlots) & 1, abort_ptr, p.timeout_ns,
                           kRoleVarDqProducer);
      if (!ok || *abort_ptr) {
        drain_wait(in_full, 0, p.timeout_ns);
        for (int it = 0; it < issued; ++it) {
          const int j = it >> 1;
          const bool is_v = it & 1;
          const int slots = is_v ? D::kVSlots : D::kKSlots;
          const int last_j = ((issued - 1 - (is_v ? 1 : 0)) >> 1);
          if (j + slots <= last_j || it == p.drop_load) continue;
          drain_wait(ptx::smem_u32(&(is_v ? bar_v_full : bar_k_full)[j % slots]), (j / slots) & 1, p.timeout_ns);
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (as in bwd_dq_cta)
    auto k_tile = [&](int j) { return sK + (j % D::kKSlots) * C::kTileBytes; };
    auto v_tile = [&](int j) { return sV + (j % D::kVSlots) * C::kTileBytes; };
    auto issue_s = [&](int j) {
      ptx::tc_fence_after();
      issue_tile_qk<HD>(tmem_base + D::kColS, sQ, k_tile(j));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_st_full));
    };
    auto issue_dp = [&](int j) {
      ptx::tc_fence_after();
      issue_tile_qk<HD>(tmem_base + D::kColP, sdO, v_tile(j));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_v_empty[j % D::kVSlots]));
      ptx::mma_commit_warp(ptx::smem_u32(&bar_dpt_full));
    };
    bool ok = wait_warp_or_abort(ptx::smem_u32(&bar_in_full), 0, abort_ptr, p.timeout_ns, kRoleVarDqMma);
    if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_k_full[0]), 0, abort_ptr, p.timeout_ns, kRoleVarDqMma);
    if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_v_full[0]), 0, abort_ptr, p.timeout_ns, kRoleVarDqMma);
    if (ok) {
      issue_s(0);
      issue_dp(0);
    }
    for (int j = 0; j < n && ok; ++j) {
      if (j + 1 < n) {
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_s_free), j & 1, abort_ptr, p.timeout_ns, kRoleVarDqMma);
        if (!ok) break;
        issue_s(j + 1);
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_dp_free), j & 1, abort_ptr, p.timeout_ns, kRoleVarDqMma);
        if (!ok) break;
        issue_dp(j + 1);
      }
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full[j & 1]), (j >> 1) & 1, abort_ptr, p.timeout_ns, kRoleVarDqMma);
      if (!ok) break;
      ptx::tc_fence_after();
      issue_tile_acc<HD, 32>(tmem_base + D::kColDQ, tmem_base + D::kColDS + 64u * (j & 1), k_tile(j), j > 0);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_k_empty[j % D::kKSlots]));
    }
    if (ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_acc_full));
    } else {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ dS + epilogue
    const int quarter = warp & 3;
    const int half = warp >> 2;
    const int row = quarter * 32 + lane;
    const int tid = half * 128 + row;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int x = min(row / p.G, p.tp - 1), hq = row - (row / p.G) * p.G;
    const int tok0 = u.blk * p.tp;
    const int live_tok = min(p.tp, u.nq - tok0);
    // Keys this row sees; rows that do not exist take the last token's.
    const int limit =
        p.causal ? max(0, min(u.nkv, tok0 + min(x, live_tok - 1) + 1 + u.nkv - u.nq)) : u.nkv;
    const long long vrow = (static_cast<long long>(kvh) * p.tile_cap + u.tile0 + u.blk) * 128 + row;
    const float nl = p.nlse2[vrow];
    const float nd = p.ndelta[vrow];
    const uint64_t sl2x2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    const uint64_t nlx2 = ptx::f2_pack(nl, nl);
    const uint64_t ndx2 = ptx::f2_pack(nd, nd);
    const uint32_t tS = tmem_base + lane_addr + D::kColS + 64u * half;
    const uint32_t tP = tmem_base + lane_addr + D::kColP + 64u * half;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_st_full), j & 1, abort_ptr, p.timeout_ns, kRoleVarDqSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      uint32_t s[2][32], dp[2][32];
      ptx::tmem_ld32(tS, s[0]);
      ptx::tmem_ld32(tS + 32, s[1]);
      ptx::tmem_ld_wait();
      ptx::reg_fence32(s[0]);
      ptx::reg_fence32(s[1]);
      if (j + 1 < n) {
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_k_full[(j + 1) % D::kKSlots]), ((j + 1) / D::kKSlots) & 1,
                                abort_ptr, p.timeout_ns, kRoleVarDqSoftmax);
        if (!ok) break;
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bar_s_free));

      const int have = u.nkv - j * C::kBlk;    // keys of the sequence in this block
      if (have < C::kBlk) {
        clear_rows<HD>(smem_raw + (sK - raw) + (j % D::kKSlots) * C::kTileBytes, max(have, 0), C::kBlk, tid);
        ptx::fence_proxy_async_smem();
      }
      const int valid = limit - j * C::kBlk - 64 * half;   // keys of this warp's 64 that this row sees
      const bool masked = !__all_sync(0xffffffffu, valid >= 64);
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
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_dpt_full), j & 1, abort_ptr, p.timeout_ns, kRoleVarDqSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      ptx::tmem_ld32(tP, dp[0]);
      ptx::tmem_ld32(tP + 32, dp[1]);
      ptx::tmem_ld_wait();
      ptx::reg_fence32(dp[0]);
      ptx::reg_fence32(dp[1]);
      if (j + 1 < n) {
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_v_full[(j + 1) % D::kVSlots]), ((j + 1) / D::kVSlots) & 1,
                                abort_ptr, p.timeout_ns, kRoleVarDqSoftmax);
        if (!ok) break;
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bar_dp_free));
      uint32_t pds[32];
      auto ds_pass = [&](auto mask) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint64_t t =
                ptx::f2_add(ptx::f2_pack(__uint_as_float(dp[c][2 * k]), __uint_as_float(dp[c][2 * k + 1])), ndx2);
            float d0, d1;
            ptx::f2_unpack(
                ptx::f2_mul(ptx::f2_pack(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), t), d0, d1);
            if (decltype(mask)::value) {
              if (32 * c + 2 * k >= valid) d0 = 0.f;
              if (32 * c + 2 * k + 1 >= valid) d1 = 0.f;
            }
            pds[16 * c + k] = ptx::pack_bf16x2(d0, d1);
          }
        }
      };
      if (masked) ds_pass(std::true_type{});
      else ds_pass(std::false_type{});
      ptx::tmem_st32(tmem_base + lane_addr + D::kColDS + 64u * (j & 1) + 32u * half, pds);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[j & 1]));
    }
    if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_acc_full), 0, abort_ptr, p.timeout_ns, kRoleVarDqSoftmax);
    if (ok) {
      ptx::tc_fence_after();
      const bool live = row < p.G * p.tp && x < live_tok;
      __nv_bfloat16* dst = p.dQ + (static_cast<long long>(u.q0) + tok0 + x) * p.dq_st + (kvh * p.G + hq) * p.dq_sh +
                           half * (HD / 2);
#pragma unroll
      for (int c = 0; c < HD / 64; ++c)
        store_row32(tmem_base + lane_addr + D::kColDQ + half * (HD / 2) + 32 * c, p.scale, dst + 32 * c, live);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (*abort_ptr) return false;
  if (threadIdx.x == 0) {
    ptx::mbar_inval(ptx::smem_u32(&bar_in_full));
    for (int s = 0; s < D::kKSlots; ++s) {
      ptx::mbar_inval(ptx::smem_u32(&bar_k_full[s]));
      ptx::mbar_inval(ptx::smem_u32(&bar_k_empty[s]));
    }
    for (int s = 0; s < D::kVSlots; ++s) {
      ptx::mbar_inval(ptx::smem_u32(&bar_v_full[s]));
      ptx::mbar_inval(ptx::smem_u32(&bar_v_empty[s]));
    }
    for (uint64_t* b : {&bar_st_full, &bar_dpt_full, &bar_s_free, &bar_dp_free, &bar_p_full[0], &bar_p_full[1],
                        &bar_acc_full, &bar_drain})
      ptx::mbar_inval(ptx::smem_u32(b));
  }
  return true;
}

// A unit of the key-block role.
template <int HD>
__device__ __forceinline__ bool varlen_dkdv_unit(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                                 const CUtensorMap& tmV, const CUtensorMap& tmdO,
                                                 const VarBwdParams& p, const VarBwdUnit u, const int kvh,
                                                 const uint32_t tmem_base, volatile int* abort_ptr,
                                                 VarBwdJob* next_job) {
  using C = BwdCfg<HD>;
  constexpr uint32_t kColDV = 0;
  constexpr uint32_t kColDK = HD;
  constexpr uint32_t kColR = 2 * HD;    // R0 = kColR, R1 = kColR + 128
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_kv_full;
  __shared__ __align__(8) uint64_t bar_q_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_q_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_do_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_do_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_st_full;
  __shared__ __align__(8) uint64_t bar_dpt_full;
  __shared__ __align__(8) uint64_t bar_dp_free;
  __shared__ __align__(8) uint64_t bar_p_full;
  __shared__ __align__(8) uint64_t bar_pt_stored;
  __shared__ __align__(8) uint64_t bar_acc_full;
  __shared__ __align__(8) uint64_t bar_drain;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n = u.n;
  const int box_rows = p.G * p.tp;
  const int key0 = u.blk * C::kBlk;                                     // first key, within the sequence
  const int tile_first = (u.nq + p.tp - 1) / p.tp - n;                  // first query tile to visit
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;
  const uint32_t sK = smem_base;
  const uint32_t sV = smem_base + C::kTileBytes;
  const uint32_t sRing = smem_base + C::kPairBytes;                     // slot s: Q_i, then dO_i
  const uint32_t sVec = sRing + C::kStages * C::kPairBytes;             // slot s: [-lse2 x 128][-D x 128]
  const float* vec = reinterpret_cast<const float*>(smem_raw + (sVec - raw));

  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&bar_kv_full), 1);
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_q_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_q_empty[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_do_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_do_empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&bar_st_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_dpt_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_dp_free), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_p_full), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_pt_stored), 256);
    ptx::mbar_init(ptx::smem_u32(&bar_acc_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    ptx::fence_mbar_init();
  }
  // Rows that no load of this unit writes are zero (the memory may hold
  // another role's tiles).
  if (box_rows < C::kBlk && warp < 8) {
    for (int s = 0; s < 2 * C::kStages; ++s)
      clear_rows<HD>(smem_raw + (sRing - raw) + s * C::kTileBytes, box_rows, C::kBlk, threadIdx.x);
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_shared = ptx::policy_evict_last();
      const uint32_t kv_full = ptx::smem_u32(&bar_kv_full);
      ptx::mbar_arrive_expect_tx(kv_full, C::kPairBytes);
      for (int c = 0; c < C::kChunks; ++c) {
        ptx::tma_load_3d(sK + c * C::kChunkBytes, &tmK, kv_full, c * 64, u.kv0 + key0, kvh, pol_shared);
        ptx::tma_load_3d(sV + c * C::kChunkBytes, &tmV, kv_full, c * 64, u.kv0 + key0, kvh, pol_shared);
      }
      int issued_q = 0, issued_do = 0;
      bool ok = true;
      const uint32_t bytes = C::kChunks * 128 * box_rows + C::kBlk * 4;
      for (int i = 0; i < n && ok; ++i) {
        const int slot = i % C::kStages;
        const uint32_t par = ((i / C::kStages) & 1) ^ 1u;
        const uint32_t dst = sRing + slot * C::kPairBytes;
        const int token = u.q0 + (tile_first + i) * p.tp;
        const long long voff = (static_cast<long long>(kvh) * p.tile_cap + u.tile0 + tile_first + i) * C::kBlk;
        if (!wait_or_abort(ptx::smem_u32(&bar_q_empty[slot]), par, abort_ptr, p.timeout_ns, kRoleVarDkvProducer)) {
          ok = false;
          break;
        }
        issued_q = i + 1;
        if (i != p.drop_load) {    // test hook: this step's tiles never arrive
          const uint32_t full = ptx::smem_u32(&bar_q_full[slot]);
          ptx::mbar_arrive_expect_tx(full, bytes);
          for (int c = 0; c < C::kChunks; ++c)
            ptx::tma_load_3d(dst + c * C::kChunkBytes, &tmQ, full, c * 64, kvh * p.G, token, pol_shared);
          ptx::bulk_load_1d(sVec + slot * C::kVecBytes, p.nlse2 + voff, C::kBlk * 4, full, pol_shared);
        }
        if (!wait_or_abort(ptx::smem_u32(&bar_do_empty[slot]), par, abort_ptr, p.timeout_ns, kRoleVarDkvProducer)) {
          ok = false;
          break;
        }
        issued_do = i + 1;
        if (i != p.drop_load) {
          const uint32_t full = ptx::smem_u32(&bar_do_full[slot]);
          ptx::mbar_arrive_expect_tx(full, bytes);
          for (int c = 0; c < C::kChunks; ++c)
            ptx::tma_load_3d(dst + C::kTileBytes + c * C::kChunkBytes, &tmdO, full, c * 64, kvh * p.G, token,
                             pol_shared);
          ptx::bulk_load_1d(sVec + slot * C::kVecBytes + C::kBlk * 4, p.ndelta + voff, C::kBlk * 4, full,
                            pol_shared);
        }
      }
      if (ok) fetch_job(p, static_cast<int>(gridDim.x) + atomicAdd(&p.plan->next, 1), next_job);
      // K and V (nobody else waits for V), and the issuer's last arrivals on the empty barriers.
      if (ok) ok = wait_or_abort(kv_full, 0, abort_ptr, p.timeout_ns, kRoleVarDkvProducer);
      for (int i = max(0, n - C::kStages); i < n && ok; ++i) {
        ok = wait_or_abort(ptx::smem_u32(&bar_q_empty[i % C::kStages]), (i / C::kStages) & 1, abort_ptr, p.timeout_ns,
                           kRoleVarDkvProducer);
        if (ok)
          ok = wait_or_abort(ptx::smem_u32(&bar_do_empty[i % C::kStages]), (i / C::kStages) & 1, abort_ptr,
                             p.timeout_ns, kRoleVarDkvProducer);
      }
      if (!ok || *abort_ptr) {
        drain_wait(kv_full, 0, p.timeout_ns);
        for (int i = issued_q > C::kStages ? issued_q - C::kStages : 0; i < issued_q; ++i)
          if (i != p.drop_load)
            drain_wait(ptx::smem_u32(&bar_q_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
        for (int i = issued_do > C::kStages ? issued_do - C::kStages : 0; i < issued_do; ++i)
          if (i != p.drop_load)
            drain_wait(ptx::smem_u32(&bar_do_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (as in bwd_dkdv_cta)
    auto region = [&](int i) { return tmem_base + kColR + 128u * static_cast<uint32_t>(i & 1); };
    auto q_tile = [&](int i) { return sRing + (i % C::kStages) * C::kPairBytes; };
    bool ok = n > 0;
    if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_kv_full), 0, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
    if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_q_full[0]), 0, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
    if (ok) {
      ptx::tc_fence_after();
      issue_tile_qk<HD>(region(0), sK, q_tile(0));                   // S_0^T = K Q_0^T
      ptx::mma_commit_warp(ptx::smem_u32(&bar_st_full));
    }
    if (ok) ok = wait_warp_or_abort(ptx::smem_u32(&bar_do_full[0]), 0, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
    if (ok) {
      ptx::tc_fence_after();
      issue_tile_qk<HD>(region(1), sV, q_tile(0) + C::kTileBytes);   // dP_0^T = V dO_0^T
      ptx::mma_commit_warp(ptx::smem_u32(&bar_dpt_full));
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_pt_stored), 0, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
      if (ok) {
        ptx::tc_fence_after();
        issue_tile_acc<HD, 64>(tmem_base + kColDV, region(0), q_tile(0) + C::kTileBytes, false);   // dV += P^T dO_0
        ptx::mma_commit_warp(ptx::smem_u32(&bar_do_empty[0]));
      }
    }
    for (int i = 0; i < n && ok; ++i) {
      bool s_issued = false;
      const int s1 = (i + 1) % C::kStages;
      const uint32_t in_par = ((i + 1) / C::kStages) & 1;
      const uint32_t q_full1 = ptx::smem_u32(&bar_q_full[s1]);
      if (i + 1 < n) {
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_dp_free), i & 1, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
        if (!ok) break;
        const uint64_t t0 = ptx::globaltimer_ns();
        while (true) {
          if (__all_sync(0xffffffffu, ptx::mbar_test_wait(q_full1, in_par))) {
            ptx::tc_fence_after();
            issue_tile_qk<HD>(region(i + 1), sK, q_tile(i + 1));      // S_{i+1}^T
            ptx::mma_commit_warp(ptx::smem_u32(&bar_st_full));
            s_issued = true;
            break;
          }
          if (__all_sync(0xffffffffu, ptx::mbar_test_wait(ptx::smem_u32(&bar_p_full), i & 1))) break;
          // Out of time or aborting: the bounded wait below reports it.
          if (__any_sync(0xffffffffu, *abort_ptr != 0) || ptx::globaltimer_ns() - t0 > p.timeout_ns) break;
          __nanosleep(32);
        }
      }
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_p_full), i & 1, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
      if (!ok) break;
      ptx::tc_fence_after();
      issue_tile_acc<HD, 64>(tmem_base + kColDK, region(i) + 32, q_tile(i), i > 0);             // dK += dS^T Q_i
      ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[i % C::kStages]));
      if (i + 1 < n) {
        if (!s_issued) {
          ok = wait_warp_or_abort(q_full1, in_par, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_tile_qk<HD>(region(i + 1), sK, q_tile(i + 1));        // S_{i+1}^T
          ptx::mma_commit_warp(ptx::smem_u32(&bar_st_full));
        }
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_do_full[s1]), in_par, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_tile_qk<HD>(region(i), sV, q_tile(i + 1) + C::kTileBytes);   // dP_{i+1}^T
        ptx::mma_commit_warp(ptx::smem_u32(&bar_dpt_full));
        ok = wait_warp_or_abort(ptx::smem_u32(&bar_pt_stored), (i + 1) & 1, abort_ptr, p.timeout_ns, kRoleVarDkvMma);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_tile_acc<HD, 64>(tmem_base + kColDV, region(i + 1), q_tile(i + 1) + C::kTileBytes, true);   // dV
        ptx::mma_commit_warp(ptx::smem_u32(&bar_do_empty[(i + 1) % C::kStages]));
      }
    }
    if (ok) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_acc_full));
    } else if (n > 0) {
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ P, dS + epilogue
    const int quarter = warp & 3;
    const int half = warp >> 2;
    const int row = quarter * 32 + lane;
    const int tid = half * 128 + row;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t sl2x2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    const int see0 = key0 + row - (u.nkv - u.nq);    // first token of the sequence that sees this key (causal)
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int tok0 = (tile_first + i) * p.tp;
      const int live_tok = min(p.tp, u.nq - tok0);
      const bool ragged = live_tok < p.tp;
      // Columns x * G + g of this warp's 64 that count for this key: [from, to).
      const int from = (p.causal ? max(0, min(see0 - tok0, p.tp)) * p.G : 0) - 64 * half;
      const int to = (ragged ? live_tok * p.G : C::kBlk) - 64 * half;
      const bool masked = !__all_sync(0xffffffffu, from <= 0 && to >= 64);
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_st_full), i & 1, abort_ptr, p.timeout_ns, kRoleVarDkvSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t tS = tmem_base + lane_addr + kColR + 128u * (i & 1) + 64u * half;
      const uint32_t tP = tmem_base + lane_addr + kColR + 128u * ((i + 1) & 1) + 64u * half;
      uint32_t s[2][32], dp[2][32];
      ptx::tmem_ld32(tS, s[0]);
      ptx::tmem_ld32(tS + 32, s[1]);
      ptx::tmem_ld_wait();
      ptx::reg_fence32(s[0]);
      ptx::reg_fence32(s[1]);
      const float4* vl = reinterpret_cast<const float4*>(vec + (i % C::kStages) * (C::kVecBytes / 4) + 64 * half);
      const float4* vd = vl + 32;    // + 128 floats
      {
        uint32_t pp[32];
        auto p_pass = [&](auto mask) {
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
                float p0 = ptx::ex2_approx(x0);
                float p1 = ptx::ex2_approx(x1);
                if (decltype(mask)::value) {
                  const int col = 32 * c + e;
                  if (col < from || col >= to) p0 = 0.f;
                  if (col + 1 < from || col + 1 >= to) p1 = 0.f;
                }
                s[c][e] = __float_as_uint(p0);
                s[c][e + 1] = __float_as_uint(p1);
                pp[16 * c + 2 * v + h2] = ptx::pack_bf16x2(p0, p1);
              }
            }
          }
        };
        if (masked) p_pass(std::true_type{});
        else p_pass(std::false_type{});
        ptx::tmem_st32(tS, pp);
        if (ragged) {
          // Clear the rows behind the sequence's end before dV and dK sum
          // over them; S^T and dP^T have read the tiles by now.
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_dpt_full), i & 1, abort_ptr, p.timeout_ns, kRoleVarDkvSoftmax);
          if (!ok) break;
          uint8_t* slot = smem_raw + (sRing - raw) + (i % C::kStages) * C::kPairBytes;
          clear_rows<HD>(slot, live_tok * p.G, box_rows, tid);
          clear_rows<HD>(slot + C::kTileBytes, live_tok * p.G, box_rows, tid);
          ptx::fence_proxy_async_smem();
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_pt_stored));
      }
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_dpt_full), i & 1, abort_ptr, p.timeout_ns, kRoleVarDkvSoftmax);
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
      auto ds_pass = [&](auto mask) {
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
              if (decltype(mask)::value) {   // dP of a column behind the end may be anything
                if (32 * c + e >= to) d0 = 0.f;
                if (32 * c + e + 1 >= to) d1 = 0.f;
              }
              pds[16 * c + 2 * v + h2] = ptx::pack_bf16x2(d0, d1);
            }
          }
        }
      };
      if (ragged) ds_pass(std::true_type{});
      else ds_pass(std::false_type{});
      ptx::tmem_st32(tS + 32, pds);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bar_p_full));
    }
    if (ok && n > 0)
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_acc_full), 0, abort_ptr, p.timeout_ns, kRoleVarDkvSoftmax);
    if (ok) {
      ptx::tc_fence_after();
      const bool live = key0 + row < u.nkv;
      const long long key = static_cast<long long>(u.kv0) + key0 + row;
      __nv_bfloat16* dv = p.dV + key * p.dv_st + kvh * p.dv_sh + half * (HD / 2);
      __nv_bfloat16* dk = p.dK + key * p.dk_st + kvh * p.dk_sh + half * (HD / 2);
      if (n > 0) {
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          store_row32(tmem_base + lane_addr + kColDV + half * (HD / 2) + 32 * c, 1.f, dv + 32 * c, live);
          store_row32(tmem_base + lane_addr + kColDK + half * (HD / 2) + 32 * c, p.scale, dk + 32 * c, live);
        }
      } else if (live) {   // a sequence without query rows
        for (int c = 0; c < HD / 16; ++c) {
          reinterpret_cast<uint4*>(dv)[c] = make_uint4(0u, 0u, 0u, 0u);
          reinterpret_cast<uint4*>(dk)[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (*abort_ptr) return false;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s)
      for (uint64_t* b : {&bar_q_full[s], &bar_q_empty[s], &bar_do_full[s], &bar_do_empty[s]})
        ptx::mbar_inval(ptx::smem_u32(b));
    for (uint64_t* b : {&bar_kv_full, &bar_st_full, &bar_dpt_full, &bar_dp_free, &bar_p_full, &bar_pt_stored,
                        &bar_acc_full, &bar_drain})
      ptx::mbar_inval(ptx::smem_u32(b));
  }
  return true;
}

template <int HD>
__global__ void __launch_bounds__(BwdCfg<HD>::kThreads, 1)
    fa_varlen_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                         const VarBwdParams p) {
  using C = BwdCfg<HD>;
  __shared__ VarBwdJob jobs[2];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 256) {
    abort_flag = 0;
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    ptx::prefetch_tmap(&tmdO);
  }
  // Every thread reads what the launches before wrote (the list, the rows' values).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 256) fetch_job(p, static_cast<int>(blockIdx.x), &jobs[0]);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const VarBwdUnit u = jobs[k & 1].u;
    const int kvh = jobs[k & 1].kvh;
    if (kvh < 0) break;
    // The producer thread leaves the unit after this one in the other slot.
    if (u.dkdv)
      ok = varlen_dkdv_unit<HD>(tmQ, tmK, tmV, tmdO, p, u, kvh, tmem_base, &abort_flag, &jobs[(k + 1) & 1]);
    else
      ok = varlen_dq_unit<HD>(tmQ, tmK, tmV, tmdO, p, u, kvh, tmem_base, &abort_flag, &jobs[(k + 1) & 1]);
  }
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace fa
