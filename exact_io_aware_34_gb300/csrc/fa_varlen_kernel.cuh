// Exact attention over packed sequences of different lengths, causal or not,
// with shared K/V heads: the prompt (prefill) shape. sm_103a, tcgen05 + TMEM
// + TMA.
//
// B sequences lie one behind the other in Q [T_q, H, d] and K, V
// [T_kv, H_kv, d]; cu_q and cu_kv (device, B + 1 offsets each) say where each
// begins. With n_q and n_kv its lengths, row i of a sequence sees key j of
// the same sequence when j < n_kv and, if causal, j <= i + n_kv - n_q: the
// last row sees every key, as when the first n_kv - n_q keys came from
// earlier calls. The update per key block is the forward kernel's (online
// softmax with a lazily moved maximum); O / l and LSE are unchanged by it. A
// row that sees no key gets O = 0 and LSE = -inf.
//
// Packing. The G = H / H_kv query heads of a K/V head see the same keys, so a
// tile's 128 rows are tp = 128 / G consecutive tokens x G heads (row
// x * G + g; one TMA box {64, G, tp} of Q's [T_q][H][d] view loads them).
// Against 128 tokens of one head, a unit of two tiles then spans 2 tp tokens
// instead of 256: the keys past the diagonal that its blocks compute and mask
// shrink with it, and a short sequence still fills its tiles. K and V are
// read once per group. When G does not divide 128 the last rows of a tile
// stay empty (126 of 128 used for G = 7).
//
// Work. A unit is two tiles of one (sequence, K/V head). Lengths never reach
// the host: a captured call may be replayed with other offsets of the same
// totals. Which of three ways the units are given out depends on sizes alone:
//   * More units than the device holds at once: varlen_plan_kernel lists them,
//     the most key blocks first, and the persistent grid takes them by a
//     counter, so that the short ones fill the end.
//   * Fewer, on at most kSplitKeys keys: CTA i finds unit i by itself; no list.
//   * Fewer, on more keys: the keys are split too (see kSplitCost).
//
// What bounds it: 4 d flops per score on the tensor core against one
// exponential, as in the forward kernel. 8192 tokens, 32 heads on 8, d = 128:
// 310-316 us, 0.90 of the measured bf16 rate in visible scores (tensor pipe busy
// 78 % of the cycles, exponentials 40 %; 101 MB read: Q, K and V once). At d = 64
// 267 us, 0.53: half the products behind the same softmax, no unit above half
// busy. Twelve prompts of 1 to 2047 tokens (8414 in all), d = 128: 89 us, 0.57:
// the 44 key blocks of a CTA take 62 us at the first call's rate (1.12 times as many
// pairs are computed as are visible), the list, the start and seven changes of
// unit the rest.
//
// Masking. Keys past a row's limit get the score -inf before the maximum and
// the exponential. (scale = 0 is run as 2^-126: then -inf stays -inf and a
// finite score counts as 0.) Rows of the V tile past the sequence's end
// belong to the next sequence, or to nobody, and could hold infinities or
// NaN, which a probability of zero does not cancel: they are zeroed in shared
// memory before P V.
//
// Rounding. P enters P V as bf16, because the tensor core takes both operands in
// one type and V is bf16: each probability is off by at most 2^-8 of itself.
// Scores, maxima, sums, O and partial results are float32, and O is rounded once.
// Relative to the float64 result O is off by 0.0020; by 0.0016 with P in float32.
//
// Warp roles: the forward kernel's (warps 0-7 softmax and epilogue of tiles 0
// and 1, warp 8 TMA producer, warp 9 MMA issuer), and warp 10 fetches units
// one ahead and hands them to the others through a two-slot ring.
#pragma once

#include "fa_fwd_kernel.cuh"

namespace fa {

namespace ptx {

// Until all but the latest bulk group have read their shared memory.
__device__ __forceinline__ void bulk_wait_group_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

}  // namespace ptx

enum : unsigned int { kRoleVarProducer = 13, kRoleVarMma = 14, kRoleVarSoftmax = 15, kRoleVarFetch = 16 };

// Words of g_status_word: 1 a wait ran out of time, 2 offsets or lengths in
// device memory that do not describe the caller's buffers.
constexpr unsigned int kStatusBadOffsets = 2;

// Most waits last a step of the pipeline; those of the warps that hand out work
// or clear tails last a whole unit (16.7 million steps, 27 s, at most), and have
// this many times the limit. What stalls a unit stalls a step, so a role with the
// shorter limit ends the wait by the abort flag.
constexpr unsigned long long kUnitWaits = 64;

// Warp-uniform bounded wait of a warp with time to spare: polls twice a
// microsecond, so that it takes no issue slots from the warps beside it.
__device__ __forceinline__ bool wait_idle_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                   unsigned long long timeout_ns, unsigned int role) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!__all_sync(0xffffffffu, ptx::mbar_test_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, *abort_flag != 0 || ptx::globaltimer_ns() - t0 > kUnitWaits * timeout_ns))
      return wait_warp_or_abort(bar, parity, abort_flag, 0, role);   // reports it
    __nanosleep(500);
  }
  return true;
}

struct VarUnit {
  int q_row0;     // first token of the unit in Q / O
  int n_tok;      // tokens of the sequence from there on (may exceed the unit's 2 tp)
  int kv_row0;    // first token of the sequence in K / V
  int n_kv;       // its keys
  int lim0;       // keys the first token sees, before clamping to [0, n_kv] (n_kv when not causal)
  int nb0, nb1;   // key blocks of tiles 0 and 1 (1 <= nb0 <= nb1; a tile that sees nothing masks one block)
  int pad;
};

struct VarPlan {          // head of the workspace; the list follows
  int num_units;          // entries of the list (each stands for H_kv units)
  int num_long;           // its first entries, of more than half the most key blocks
  int next;               // units handed out beyond the grid's first
  int pad[5];
};

// A unit whose keys are split among the pieces first to last of the line, where
// first is the piece that holds its first block (kvh < 0: none begins there).
struct VarCut {
  VarUnit u;
  int kvh, first, last, pad;
};

struct VarParams {
  __nv_bfloat16* O;
  float* LSE;             // [H][T_q]
  const int *cu_q, *cu_kv;
  int B, T_kv;
  VarPlan* plan;          // null: CTA i takes the i-th unit in the sequences' order, without a list
  const VarUnit* list;
  VarCut* cut;            // split keys: one entry per piece; or null
  float *Op, *Lp;         // split keys: partial O [slot][tile][d / 4][128][4] and log2-sum-exp [slot][tile][128]
  long long o_st, o_sh;   // element strides of O (token, head)
  int T_q;
  int H_kv;
  int G;                  // query heads per K/V head
  int group;              // K/V heads whose units are taken together
  int tp;                 // tokens per tile: 128 / G
  int inv_g;              // ceil(65536 / G): r / G = r * inv_g >> 16 for r < 128
  int causal;
  int o_tma;              // 1: G is a power of two, so a warp's 32 rows are a box of O
  float scale_log2;       // |scale| * log2(e), at least 2^-126
  uint32_t idesc_qk;
  unsigned long long timeout_ns;
  int drop_load;
};

// ---------------------------------------------------------------- unit list
// One CTA. Sequences are taken kSeqs at a time: a scan gives each sequence
// its place among the chunk's units, then every thread takes units and finds
// their sequence by bisection, so that one long sequence is spread over the
// threads. Two rounds over the units: count per cost class, then place.
// Classes are eighths of a power of two of the number of key blocks.
constexpr int kPlanThreads = 512;
constexpr int kPlanClasses = 256;

__device__ __forceinline__ int cost_class(int blocks) {
  const int e = 31 - __clz(blocks);
  const int m = e >= 3 ? (blocks >> (e - 3)) & 7 : (blocks << (3 - e)) & 7;
  return min(kPlanClasses - 1, 8 * e + m);
}

struct SeqSpan {
  int q0, nq, kv0, nkv;
};

__device__ __forceinline__ SeqSpan seq_span(const int* cu_q, const int* cu_kv, int i) {
  SeqSpan s;
  s.q0 = cu_q[i];
  s.nq = cu_q[i + 1] - s.q0;
  s.kv0 = cu_kv[i];
  s.nkv = cu_kv[i + 1] - s.kv0;
  return s;
}

// Whether sequence i's offsets do not describe the caller's buffers (they
// start at 0 or later, never decrease and end inside); the device status word
// then says so.
__device__ __forceinline__ bool span_bad(const int* cu_q, const int* cu_kv, int i, int T_q, int T_kv) {
  const int q0 = cu_q[i], q1 = cu_q[i + 1], k0 = cu_kv[i], k1 = cu_kv[i + 1];
  const bool bad = q0 < 0 || q1 < q0 || q1 > T_q || k0 < 0 || k1 < k0 || k1 > T_kv;
  if (bad && atomicCAS(&g_status_word, 0u, kStatusBadOffsets) == 0u) {
    g_status_info[0] = kRoleVarFetch;
    g_status_info[1] = static_cast<unsigned int>(i);
    g_status_info[2] = g_status_info[3] = 0u;
  }
  return bad;
}

// Whether all offsets are good; if not, the call computes nothing. The same
// answer in every thread of the CTA.
__device__ __forceinline__ bool offsets_ok(const int* cu_q, const int* cu_kv, int B, int T_q, int T_kv) {
  bool bad = false;
  for (int i = threadIdx.x; i < B; i += kPlanThreads) bad |= span_bad(cu_q, cu_kv, i, T_q, T_kv);
  return !__syncthreads_or(bad);
}

// Inclusive scan of one int per thread over the CTA; returns the total too.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane < kPlanThreads / 32) warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v += warp_sums[warp - 1];
  total = warp_sums[kPlanThreads / 32 - 1];
  __syncthreads();
  return v;
}

__device__ __forceinline__ VarUnit make_unit(const SeqSpan& s, int u, int tp, int causal) {
  VarUnit r;
  const int x0 = u * 2 * tp;
  r.q_row0 = s.q0 + x0;
  r.n_tok = s.nq - x0;
  r.kv_row0 = s.kv0;
  r.n_kv = s.nkv;
  r.lim0 = causal ? x0 + 1 + (s.nkv - s.nq) : s.nkv;
  const int step = causal ? 1 : 0;
  const int last0 = min(s.nkv, r.lim0 + step * (min(tp, r.n_tok) - 1));
  const int last1 = min(s.nkv, r.lim0 + step * (min(2 * tp, r.n_tok) - 1));
  r.nb0 = max(1, (max(last0, 0) + 127) >> 7);
  r.nb1 = max(1, (max(last1, 0) + 127) >> 7);
  r.pad = 0;
  return r;
}

__global__ void __launch_bounds__(kPlanThreads)
    varlen_plan_kernel(const int* __restrict__ cu_q, const int* __restrict__ cu_kv, VarPlan* __restrict__ plan,
                       VarUnit* __restrict__ list, int B, int T_q, int T_kv, int tp, int causal) {
  __shared__ int cum[kPlanThreads + 1];
  __shared__ SeqSpan span[kPlanThreads];
  __shared__ int hist[kPlanClasses];
  __shared__ int warp_sums[kPlanThreads / 32];
  __shared__ int top;                          // the most expensive class
  // The grid that reads the list may be scheduled now; it waits for this one's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (!offsets_ok(cu_q, cu_kv, B, T_q, T_kv)) {
    if (tid == 0) {
      plan->num_units = 0;
      plan->num_long = 0;
      plan->next = 0;
    }
    return;
  }
  if (tid < kPlanClasses) hist[tid] = 0;
  if (tid == 0) top = 0;
  const int unit_tok = 2 * tp;
  int total = 0;
  for (int round = 0; round < 2; ++round) {
    for (int c0 = 0; c0 < B; c0 += kPlanThreads) {
      int nu = 0, chunk;
      if (round == 0 || B > kPlanThreads) {   // one chunk's spans stay for the second round
        __syncthreads();
        if (c0 + tid < B) {
          span[tid] = seq_span(cu_q, cu_kv, c0 + tid);
          nu = span[tid].nq / unit_tok + (span[tid].nq % unit_tok != 0);
        }
        const int incl = block_scan(nu, warp_sums, chunk);
        cum[tid + 1] = incl;
        if (tid == 0) cum[0] = 0;
        __syncthreads();
      }
      chunk = cum[kPlanThreads];
      for (int e = tid; e < chunk; e += kPlanThreads) {
        int lo = 0, hi = kPlanThreads - 1;    // the last sequence whose first unit is <= e
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (cum[mid] <= e) lo = mid; else hi = mid - 1;
        }
        const VarUnit u = make_unit(span[lo], e - cum[lo], tp, causal);
        if (round == 0) {
          atomicAdd(&hist[cost_class(u.nb1)], 1);
        } else {
          list[atomicAdd(&hist[cost_class(u.nb1)], 1)] = u;
        }
      }
      if (round == 0) total += chunk;
    }
    __syncthreads();
    if (round == 0) {
      // Places: the most expensive class first.
      int sum;
      const int mine = tid < kPlanClasses ? hist[kPlanClasses - 1 - tid] : 0;
      if (mine > 0) atomicMax(&top, kPlanClasses - 1 - tid);
      const int incl = block_scan(mine, warp_sums, sum);
      if (tid < kPlanClasses) hist[kPlanClasses - 1 - tid] = incl - mine;
      // Eight classes are an octave: entries before those of class top - 8 are long.
      if (tid == kPlanClasses - 1 - max(top - 8, 0)) plan->num_long = top >= 8 ? incl - mine : sum;
      __syncthreads();
    }
  }
  if (tid == 0) {
    plan->num_units = total;
    plan->next = 0;
  }
}

// ---------------------------------------------------------------- forward
// The idx-th unit of n list entries x H_kv heads. Of the n_long long entries
// `group` heads are taken at a time, the heads of a group together, so that what
// they stream stays in L2; then the short entries of all heads, which even out
// the end. Within either in the list's order.
__device__ __forceinline__ void place_unit(int idx, int n_long, int H_kv, int group, int* entry, int* kvh) {
  const int in_long = n_long * H_kv;
  if (idx < in_long) {
    const int g = idx / (n_long * group), r = idx - g * n_long * group;
    const int heads = min(group, H_kv - g * group);
    *entry = r / heads;
    *kvh = g * group + r - *entry * heads;
  } else {
    const int r = idx - in_long;
    *entry = r / H_kv;
    *kvh = r - *entry * H_kv;
    *entry += n_long;
  }
}

// What the fetch warp hands to the other roles.
struct VarJob {
  VarUnit u;
  int kvh;        // K/V head; -1: no more units
  int slot;       // place of the partial results; -1: the unit has all its keys, O and LSE are final
};

// The unit of this CTA without a list (one warp): unit blockIdx.x / H_kv of
// the sequences in order, K/V head blockIdx.x % H_kv. For grids that hold every
// unit at once, where no order and no counter is needed: it saves the plan's
// launch, 4 of 10 us for one short prompt.
__device__ __forceinline__ void direct_unit(const VarParams& p, VarJob* job) {
  const int lane = threadIdx.x & 31;
  const int e = static_cast<int>(blockIdx.x) / p.H_kv;
  int base = 0, found = -1, first = 0;
  bool bad = false;
  for (int c0 = 0; c0 < p.B; c0 += 32) {
    const int i = c0 + lane;
    int nu = 0;
    if (i < p.B) {
      bad |= span_bad(p.cu_q, p.cu_kv, i, p.T_q, p.T_kv);
      const int nq = p.cu_q[i + 1] - p.cu_q[i];
      nu = nq > 0 ? (nq - 1) / (2 * p.tp) + 1 : 0;
    }
    int incl = nu;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const unsigned mine = __ballot_sync(0xffffffffu, e >= base + incl - nu && e < base + incl);
    if (mine && found < 0) {
      const int src = __ffs(mine) - 1;
      found = c0 + src;
      first = base + __shfl_sync(0xffffffffu, incl - nu, src);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (__any_sync(0xffffffffu, bad) || found < 0) return;
  job->u = make_unit(seq_span(p.cu_q, p.cu_kv, found), e - first, p.tp, p.causal);
  job->kvh = static_cast<int>(blockIdx.x) - e * p.H_kv;
  job->slot = -1;
}

// Split keys: few units on long caches (a piece of a prompt whose beginning is
// in the cache) would leave most of the device idle. All units lie in one line,
// head after head, each kSplitCost places for its start and end and then one
// place per key (up to its last row's diagonal; with more rows than keys the
// count is too high, see note_cut); CTA c takes the places
// [c P, (c + 1) P), P the line's length over the grid. A unit whose blocks
// fall to several CTAs leaves partial results, which varlen_merge_kernel joins.
// Where the longest unit is at most kSplitGain places longer than P, splitting
// gains less than the merge costs, and CTA i takes unit i whole. Unsplit and
// split (32 heads on 8, d = 128): 64 rows on 16384 keys 167 and 33 us, 512 on
// 32768 356 and 211; where nothing is split after all, finding that out and
// the merge's empty launch make 28 us 31.
constexpr int kSplitCost = 256;   // two key blocks' time
constexpr int kSplitMin = 512;    // least P: four key blocks
constexpr int kSplitGain = 1024;  // eight key blocks
// Calls that could gain by it: units fit the device at once, and a cache this long.
constexpr int kSplitKeys = kSplitMin + kSplitGain;

struct VarLine {
  long long head;       // places of one K/V head's units
  long long piece;      // P
  long long total;      // of all heads
  bool whole, bad;
};

// A sequence's units on the line: nu units, the u-th base + u * step places
// long and beginning at u * base + step * u (u - 1) / 2.
struct LineSeq {
  int nu;
  long long base, step;
  __device__ long long begin(long long u) const { return u * base + step * (u * (u - 1) / 2); }
};

__device__ __forceinline__ LineSeq line_seq(const VarParams& p, const SeqSpan& s) {
  LineSeq r;
  r.nu = s.nq > 0 ? (s.nq - 1) / (2 * p.tp) + 1 : 0;
  r.step = p.causal ? 2 * p.tp : 0;
  r.base = kSplitCost + (p.causal ? max(s.nkv - s.nq, 0) + 2 * p.tp : s.nkv);
  return r;
}

__device__ __forceinline__ VarLine split_line(const VarParams& p, int pieces) {   // one warp
  const int lane = threadIdx.x & 31;
  VarLine l;
  long long sum = 0, most = 0;
  bool bad = false;
  for (int i = lane; i < p.B; i += 32) {
    if (span_bad(p.cu_q, p.cu_kv, i, p.T_q, p.T_kv)) {   // no places: sums of such lengths can pass 2^63
      bad = true;
      continue;
    }
    const LineSeq s = line_seq(p, seq_span(p.cu_q, p.cu_kv, i));
    sum += s.begin(s.nu);
    if (s.nu > 0) most = max(most, s.base + s.step * (s.nu - 1));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  l.head = sum;
  l.total = sum * p.H_kv;
  l.piece = max(static_cast<long long>(kSplitMin), (l.total + pieces - 1) / pieces);
  l.whole = most <= l.piece + kSplitGain;
  l.bad = __any_sync(0xffffffffu, bad);
  return l;
}

// The unit at place x < total of the line (one warp; the same in every lane).
struct LineUnit {
  SeqSpan s;
  int u, kvh;
  long long x0, x1;     // its places
};

__device__ __forceinline__ LineUnit line_find(const VarParams& p, const VarLine& l, long long x) {
  const int lane = threadIdx.x & 31;
  LineUnit r;
  r.kvh = static_cast<int>(x / l.head);
  const long long at = x - r.kvh * l.head;
  long long base = 0, first = 0;
  int found = 0;
  for (int c0 = 0; c0 < p.B; c0 += 32) {
    const int i = c0 + lane;
    long long len = 0;
    if (i < p.B) {
      const LineSeq s = line_seq(p, seq_span(p.cu_q, p.cu_kv, i));
      len = s.begin(s.nu);
    }
    long long incl = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const unsigned mine = __ballot_sync(0xffffffffu, at >= base + incl - len && at < base + incl);
    if (mine) {
      const int src = __ffs(mine) - 1;
      found = c0 + src;
      first = base + __shfl_sync(0xffffffffu, incl - len, src);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  r.s = seq_span(p.cu_q, p.cu_kv, found);
  const LineSeq s = line_seq(p, r.s);
  int lo = 0, hi = s.nu - 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (s.begin(mid) <= at - first) lo = mid; else hi = mid - 1;
  }
  r.u = lo;
  r.x0 = r.kvh * l.head + first + s.begin(lo);
  r.x1 = r.kvh * l.head + first + s.begin(lo + 1);
  return r;
}

// The key blocks [b0, b1) of a unit with nb blocks that CTA c's piece holds,
// and the slot of their partial results. A piece has at most two units in
// part: one that begins before it and one that ends behind it.
struct LinePart {
  int b0, b1, slot;
};

__device__ __forceinline__ LinePart line_part(const VarLine& l, const LineUnit& v, int nb, long long c) {
  auto block = [&](long long y) {
    return static_cast<int>(min(static_cast<long long>(nb), max(0ll, (y - kSplitCost + 64) >> 7)));
  };
  LinePart r;
  r.b0 = c * l.piece <= v.x0 ? 0 : block(c * l.piece - v.x0);
  r.b1 = (c + 1) * l.piece >= v.x1 ? nb : block((c + 1) * l.piece - v.x0);
  r.slot = static_cast<int>(2 * c) + (r.b0 == 0 ? 1 : 0);
  return r;
}

// The unit that begins to be split in piece c, whose end lies inside the line:
// the one across the end, if its first block is in this piece, or the one
// whose start alone lies in the piece before.
__device__ __forceinline__ void note_cut(const VarParams& p, const VarLine& line, int c, VarCut* cut) {
  const LineUnit v = line_find(p, line, (c + 1) * line.piece);
  cut->u = make_unit(v.s, v.u, p.tp, p.causal);
  const LinePart here = line_part(line, v, cut->u.nb1, c);
  if (here.b0 > 0 || here.b1 == 0 || here.b1 == cut->u.nb1) return;
  cut->kvh = v.kvh;
  cut->first = c;
  // The last piece that holds a block of it. A unit's places may go on behind its
  // blocks, for several pieces where a causal sequence has more rows than keys
  // (line_seq counts them as if row i saw the keys up to i).
  int last = static_cast<int>((v.x1 - 1) / line.piece);
  for (; last > c; --last) {
    const LinePart end = line_part(line, v, cut->u.nb1, last);
    if (end.b0 < end.b1) break;
  }
  cut->last = last;
}

template <int HD>
__global__ void __launch_bounds__(FwdCfg<HD>::kThreads, 1)
    fa_varlen_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                         const VarParams p) {
  using C = FwdCfg<HD>;
  constexpr int kPolls = HD == 128 ? 8 : 1;   // as in the forward kernel
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q_full[2];
  __shared__ __align__(8) uint64_t bar_q_empty[2];
  __shared__ __align__(8) uint64_t bar_kv_full[C::kStages];
  __shared__ __align__(8) uint64_t bar_kv_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_p_full[2];
  __shared__ __align__(8) uint64_t bar_p_half[2];
  __shared__ __align__(8) uint64_t bar_o_full[2];
  __shared__ __align__(8) uint64_t bar_job_full[2];
  __shared__ __align__(8) uint64_t bar_job_empty[2];
  __shared__ __align__(8) uint64_t bar_claim;
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(16) VarJob jobs[2];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int box_rows = p.G * p.tp;            // rows of a tile that hold queries

  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = smem_base;
  const uint32_t sKV = smem_base + C::kSmemQ;
  const uint32_t sStage = sKV + C::kSmemKV;
  uint8_t* generic = smem_raw + (smem_base - ptx::smem_u32(smem_raw));

  // Rows of the Q tiles that no query fills stay zero for the kernel's life.
  for (int c = 0; c < C::kQTiles * C::kChunks; ++c)
    for (int i = threadIdx.x; i < (C::kBM - box_rows) * 8; i += C::kThreads)
      reinterpret_cast<uint4*>(generic + c * C::kChunkBytes + box_rows * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bar_kv_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_kv_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_u32(&bar_q_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_q_empty[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_s_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_p_full[t]), C::kBM);
      ptx::mbar_init(ptx::smem_u32(&bar_p_half[t]), C::kBM);
      ptx::mbar_init(ptx::smem_u32(&bar_o_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_full[t]), 1);
      ptx::mbar_init(ptx::smem_u32(&bar_job_empty[t]), 10);   // producer, issuer, eight softmax warps
    }
    ptx::mbar_init(ptx::smem_u32(&bar_claim), 1);
    ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_base_slot), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  volatile int* abort_ptr = &abort_flag;

  if (warp >= 8) ptx::setmaxnreg_dec<C::kRegsControl>();
  // (The softmax stands first: behind the other branches the compiled kernel was
  // 3 to 5 % slower.)
  if (warp < 8) {
    // ------------------------------------------------------------ softmax + epilogue
    ptx::setmaxnreg_inc<C::kRegsSoftmax>();
    const int t = warp >> 2;                 // query tile
    const int quarter = warp & 3;            // TMEM lane quarter
    const int row = quarter * 32 + lane;     // row within the tile: token row / G, head row % G
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem_base + lane_addr + C::kColS + 128 * t;
    const uint32_t tO = tmem_base + lane_addr + C::kColO + HD * t;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int it0 = 0, g = 0;
    for (int n = 0; ok; ++n) {
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                                      kRoleVarSoftmax);
      if (!ok) break;
      // The slot is given back in the epilogue, which reads the rest of it
      // (few values may live through the block loop without spilling).
      const VarJob& job = jobs[n & 1];
      if (job.kvh < 0) break;
      const int nb1 = job.u.nb1, nb = t ? nb1 : job.u.nb0, n_kv = job.u.n_kv;
      const int clear_from = t ? job.u.nb0 : 0;   // first block whose V this tile clears (see below)
      // Keys this row sees. Rows past the sequence's end (never stored) take
      // the last token's, so that they do not mask blocks the others need not.
      const int limit =
          p.causal ? max(0, min(n_kv, job.u.lim0 + min(t * p.tp + min((row * p.inv_g) >> 16, p.tp - 1),
                                                       job.u.n_tok - 1)))
                   : n_kv;
      float m_use = -INFINITY;   // raw-score maximum the exponentials are taken against
      float l = 0.f;             // running sum of exp, relative to m_use (for LSE)
      float lo = 0.f;            // the same with each block's largest term as P V sees it (for O)
      for (int j = 0; j < nb; ++j, ++g) {
        // V_j and K_{j+1} must have landed before this block's hand-off (the
        // issuer does not wait for them); waiting here costs nothing, S_t(j)
        // comes later.
        const int itV = it0 + 2 * j + 1;
        const int have = n_kv - j * C::kBN;    // keys of the sequence in this block
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_kv_full[itV % C::kStages]), (itV / C::kStages) & 1,
                                        abort_ptr, p.timeout_ns, kRoleVarSoftmax);
        if (ok && j + 1 < nb1)
          ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_kv_full[(itV + 1) % C::kStages]),
                                          ((itV + 1) / C::kStages) & 1, abort_ptr, p.timeout_ns, kRoleVarSoftmax);
        if (!ok) break;
        if (have < C::kBN && j >= clear_from) {
          // Whole 128-byte rows, so the swizzle does not matter. Tile 0's P V
          // is issued first, so its warps clear V for both tiles.
          uint8_t* v_tile = generic + C::kSmemQ + (itV % C::kStages) * C::kTileBytes;
          const int first = max(have, 0);
          for (int c = 0; c < C::kChunks; ++c)
            for (int i = row; i < (C::kBN - first) * 8; i += C::kBM)
              reinterpret_cast<uint4*>(v_tile + c * C::kChunkBytes + first * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
          ptx::fence_proxy_async_smem();
        }
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_s_full[t]), g & 1, abort_ptr, p.timeout_ns,
                                        kRoleVarSoftmax);
        if (!ok) break;
        ptx::tc_fence_after();
        const int valid = limit - j * C::kBN;        // keys of this block that this row sees
        // Scores past a row's limit become -inf in TMEM, 32 columns at a time,
        // before the common path reads them. A loop of few instructions: this
        // runs about once per unit, and the unrolled masking of a block in
        // registers spent most of its time fetching instructions.
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
        // The loads also reduce each 32-column piece to its maximum.
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
        // A row sees keys from the first block on or none at all, so after
        // block 0 the maximum is -inf only for a row that sees nothing.
        float alpha = 1.f;
        bool rescale_o = false;
        if (j == 0) {
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
        auto exponents = [&](int c) {
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
        };
        exponents(0);
        exponents(1);
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
        ptx::tmem_st32(tS, pk[0]);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_half[t]));
        exponents(2);
        exponents(3);
        float sum;
        {
          float a0, a1, b0, b1;
          ptx::f2_unpack(ptx::f2_add(acc[0], acc[1]), a0, a1);
          ptx::f2_unpack(ptx::f2_add(acc[2], acc[3]), b0, b1);
          sum = (a0 + a1) + (b0 + b1);
        }
        // P V sees every probability rounded to bf16; the block's largest
        // enters O's normaliser rounded too, so that a row dominated by one
        // key weights it exactly 1 (as in the forward kernel).
        const float pmax = ptx::ex2_approx(fmaf(mt, sl2, neg_m));
        l = l * alpha + sum;
        lo = lo * alpha + (sum + (ptx::round_bf16(pmax) - pmax));
        ptx::tmem_st32(tS + 32, pk[1]);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bar_p_full[t]));
      }
      // A block that only tile 1 visits: its V load is waited for all the same,
      // so that no later wait on its slot meets the phase before.
      for (int j = nb; j < nb1 && ok; ++j) {
        const int itV = it0 + 2 * j + 1;
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_kv_full[itV % C::kStages]), (itV / C::kStages) & 1,
                                        abort_ptr, p.timeout_ns, kRoleVarSoftmax);
      }
      const int xr = (row * p.inv_g) >> 16;             // token of this row within the tile
      const int head = job.kvh * p.G + row - xr * p.G;
      const long long token = static_cast<long long>(job.u.q_row0) + t * p.tp + xr;
      const bool live = row < box_rows && t * p.tp + xr < job.u.n_tok;
      const bool none = limit == 0;
      const float lse2 = m_use * sl2 + __log2f(l);
      const int slot = job.slot;
      if (slot >= 0) {
        if (ok) p.Lp[(slot * 2 + t) * 128 + row] = lo == 0.f ? -INFINITY : lse2;
      } else if (live && ok) {
        p.LSE[static_cast<long long>(head) * p.T_q + token] = none ? -INFINITY : lse2 * 0.69314718055994530942f;
      }
      const float inv_l = slot >= 0 && lo == 0.f ? 0.f : 1.f / lo;
      // The warp's rows as a box of O: first token, last token, first head.
      const int x_first = t * p.tp + ((quarter * 32 * p.inv_g) >> 16);
      const int x_last = t * p.tp + (((quarter * 32 + 31) * p.inv_g) >> 16);
      const int h_first = quarter * 32 - (x_first - t * p.tp) * p.G;
      const bool boxed = p.o_tma && x_last < job.u.n_tok;
      const int box_head = job.kvh * p.G + h_first, box_token = job.u.q_row0 + x_first;
      const uint32_t stage = sStage + static_cast<uint32_t>(warp) * 4096u;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (ok)
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_o_full[t]), n & 1, abort_ptr, p.timeout_ns,
                                        kRoleVarSoftmax);
      if (!ok) break;
      ptx::tc_fence_after();
      it0 += 2 * nb1;
      // O leaves in 32-column pieces through shared memory, where one lane
      // stores them with a tiled TMA store, when the warp's rows are a box of O
      // that lies inside the sequence; else every thread writes its row. Two
      // staging buffers of 32 rows x 64 bytes (64-byte swizzle) per warp.
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(tO + 32 * c, o);
        ptx::tmem_ld_wait();
        ptx::reg_fence32(o);
        if (slot >= 0) {   // a row's next four columns lie 2 KB further, so that a warp writes 512 bytes in one go
          float4* dst = reinterpret_cast<float4*>(p.Op) + (static_cast<size_t>(slot * 2 + t) * (HD / 4) + 8 * c) * 128 + row;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v * 128] = make_float4(__uint_as_float(o[4 * v]) * inv_l, __uint_as_float(o[4 * v + 1]) * inv_l,
                                       __uint_as_float(o[4 * v + 2]) * inv_l, __uint_as_float(o[4 * v + 3]) * inv_l);
          continue;
        }
        uint32_t packed[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          packed[i] = ptx::pack_bf16x2(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l);
        if (none) {
#pragma unroll
          for (int i = 0; i < 16; ++i) packed[i] = 0u;
        }
        if (boxed) {
          if (lane == 0) ptx::bulk_wait_group_read1();   // the buffer's previous store has read it
          __syncwarp();
          const uint32_t buf = stage + static_cast<uint32_t>(c & 1) * 2048u;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint32_t addr = buf + static_cast<uint32_t>(lane) * 64u + ((v ^ ((lane >> 1) & 3u)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(packed[4 * v]),
                         "r"(packed[4 * v + 1]), "r"(packed[4 * v + 2]), "r"(packed[4 * v + 3])
                         : "memory");
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_3d(&tmO, buf, 32 * c, box_head, box_token);
            ptx::bulk_commit_group();
          }
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(p.O + token * p.o_st + head * p.o_sh + 32 * c);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            dst[v] = make_uint4(packed[4 * v], packed[4 * v + 1], packed[4 * v + 2], packed[4 * v + 3]);
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_q = ptx::policy_evict_first();
      const uint64_t pol_kv = ptx::policy_evict_last();
      int it = 0;           // K/V loads so far (the ring position runs on across units)
      int q_issued[2] = {0, 0};
      bool ok = true;
      VarJob job;
      // The next K (even it) or V tile of block j into its ring slot.
      auto load_kv = [&](int j) {
        const int slot = it % C::kStages;
        if (!wait_or_abort<kPolls>(ptx::smem_u32(&bar_kv_empty[slot]), ((it / C::kStages) & 1) ^ 1u, abort_ptr,
                                   p.timeout_ns, kRoleVarProducer))
          return false;
        const int me = it++;
        if (me == p.drop_load) return true;   // test hook: this tile never arrives
        const uint32_t full = ptx::smem_u32(&bar_kv_full[slot]);
        ptx::mbar_arrive_expect_tx(full, C::kTileBytes);
        const void* map = (me & 1) ? static_cast<const void*>(&tmV) : static_cast<const void*>(&tmK);
        for (int c = 0; c < C::kChunks; ++c)
          ptx::tma_load_3d(sKV + slot * C::kTileBytes + c * C::kChunkBytes, map, full, c * 64,
                           job.u.kv_row0 + j * C::kBN, job.kvh, pol_kv);
        return true;
      };
      for (int n = 0; ok; ++n) {
        ok = wait_or_abort<kPolls>(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                                   kRoleVarProducer);
        if (!ok) break;
        job = jobs[n & 1];
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
        if (job.kvh < 0) break;
        // Each Q tile is free once its last Q K^T of the unit before has completed.
        for (int t = 0; t < C::kQTiles && ok; ++t) {
          if (n > 0 && !wait_or_abort<kPolls>(ptx::smem_u32(&bar_q_empty[t]), (n - 1) & 1, abort_ptr, p.timeout_ns,
                                              kRoleVarProducer)) {
            ok = false;
            break;
          }
          const uint32_t q_full = ptx::smem_u32(&bar_q_full[t]);
          ptx::mbar_arrive_expect_tx(q_full, C::kChunks * 128 * box_rows);
          for (int c = 0; c < C::kChunks; ++c)
            ptx::tma_load_3d(sQ + t * C::kTileBytes + c * C::kChunkBytes, &tmQ, q_full, c * 64, job.kvh * p.G,
                             job.u.q_row0 + t * p.tp, pol_q);
          q_issued[t] = n + 1;
          if (t == 0) ok = load_kv(0) && load_kv(0);
        }
        if (job.u.nb1 <= 2) ptx::mbar_arrive(ptx::smem_u32(&bar_claim));
        for (int j = 1; j < job.u.nb1 && ok; ++j) {
          if (job.u.nb1 > 2 && j == job.u.nb1 - 2) ptx::mbar_arrive(ptx::smem_u32(&bar_claim));
          ok = load_kv(j) && load_kv(j);
        }
      }
      if (!ok || *abort_ptr) {
        // Let every copy this thread started land before the CTA exits.
        for (int t = 0; t < 2; ++t)
          if (q_issued[t] > 0) drain_wait(ptx::smem_u32(&bar_q_full[t]), (q_issued[t] - 1) & 1, p.timeout_ns);
        for (int i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
          if (i != p.drop_load)
            drain_wait(ptx::smem_u32(&bar_kv_full[i % C::kStages]), (i / C::kStages) & 1, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    auto issue_pv_half = [&](int t, int it, bool accumulate, int half) {
      const uint64_t b_desc = ptx::desc_mnmajor_sw128(sKV + (it % C::kStages) * C::kTileBytes, C::kChunkBytes);
      const uint32_t d_tmem = tmem_base + C::kColO + HD * t, a_tmem = tmem_base + C::kColS + 128 * t;
      if (half == 0)
        ptx::mma_ts_k64half_warp<0>(d_tmem, a_tmem, ptx::desc_lo(b_desc), ptx::desc_hi(b_desc), C::kIdescPV,
                                    accumulate ? 1u : 0u);
      else
        ptx::mma_ts_k64half_warp<1>(d_tmem, a_tmem, ptx::desc_lo(b_desc), ptx::desc_hi(b_desc), C::kIdescPV, 1u);
    };
    auto issue_qk = [&](int t, int it) {
      const uint64_t a_desc = ptx::desc_kmajor_sw128(sQ + t * C::kTileBytes);
      const uint64_t b_desc = ptx::desc_kmajor_sw128(sKV + (it % C::kStages) * C::kTileBytes);
      const uint32_t d_tmem = tmem_base + C::kColS + 128 * t;
      if constexpr (HD == 128)
        ptx::mma_ss_k128_warp(d_tmem, ptx::desc_lo(a_desc), ptx::desc_lo(b_desc), ptx::desc_hi(a_desc), p.idesc_qk, 0u);
      else
        ptx::mma_ss_k64_warp(d_tmem, ptx::desc_lo(a_desc), ptx::desc_lo(b_desc), ptx::desc_hi(a_desc), p.idesc_qk, 0u);
    };
    bool ok = true;
    int it0 = 0;              // K/V loads of the units before this one
    int g[2] = {0, 0};        // key blocks of each tile so far (phases of s_full, p_half, p_full)
    int was0 = 0, was1 = 0;   // key blocks of the unit before
    // P V of tile t from the V tile of load it, once its probabilities are handed over.
    auto finish_pv = [&](int t, int it, bool accumulate) {
      const uint32_t par = static_cast<uint32_t>(g[t] - 1) & 1u;
      if (!wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_p_half[t]), par, abort_ptr, p.timeout_ns, kRoleVarMma))
        return false;
      ptx::tc_fence_after();
      issue_pv_half(t, it, accumulate, 0);
      if (!wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_p_full[t]), par, abort_ptr, p.timeout_ns, kRoleVarMma))
        return false;
      ptx::tc_fence_after();
      issue_pv_half(t, it, true, 1);
      return true;
    };
    auto start_qk = [&](int t, int it) {
      issue_qk(t, it);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_s_full[t]));
      ++g[t];
    };
    for (int n = 0; ok; ++n) {
      // The last P V of the unit before, whose epilogue then runs beside this
      // unit's first Q K^T.
      if (n > 0 && was0 == was1) {
        ok = finish_pv(0, it0 - 1, was1 > 1);
        if (!ok) break;
        ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[0]));
      }
      if (n > 0) {
        ok = finish_pv(1, it0 - 1, was1 > 1);
        if (!ok) break;
        ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[1]));
        ptx::mma_commit_warp(ptx::smem_u32(&bar_kv_empty[(it0 - 1) % C::kStages]));
      }
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_job_full[n & 1]), (n >> 1) & 1, abort_ptr, p.timeout_ns,
                                      kRoleVarMma);
      if (!ok) break;
      const int kvh = jobs[n & 1].kvh;
      const int nb0 = jobs[n & 1].u.nb0, nb1 = jobs[n & 1].u.nb1;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bar_job_empty[n & 1]));
      if (kvh < 0) break;
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_q_full[0]), n & 1, abort_ptr, p.timeout_ns, kRoleVarMma);
      if (ok)
        ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_kv_full[it0 % C::kStages]), (it0 / C::kStages) & 1,
                                        abort_ptr, p.timeout_ns, kRoleVarMma);
      if (!ok) break;
      ptx::tc_fence_after();
      start_qk(0, it0);
      if (nb0 == 1) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[0]));
      ok = wait_warp_or_abort<kPolls>(ptx::smem_u32(&bar_q_full[1]), n & 1, abort_ptr, p.timeout_ns, kRoleVarMma);
      if (!ok) break;
      ptx::tc_fence_after();
      start_qk(1, it0);
      ptx::mma_commit_warp(ptx::smem_u32(&bar_kv_empty[it0 % C::kStages]));
      if (nb1 == 1) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[1]));
      // Later blocks: K_j and V_{j-1} were waited for by the softmax warps
      // before their first hand-off for block j - 1. Tile 1 visits every block,
      // tile 0 all (nb0 = nb1) or all but the last.
      for (int j = 1; j < nb1 && ok; ++j) {
        const int itK = it0 + 2 * j;
        ok = finish_pv(0, itK - 1, j > 1);
        if (!ok) break;
        if (j < nb0) {
          start_qk(0, itK);
          if (j == nb0 - 1) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[0]));
        } else {
          ptx::mma_commit_warp(ptx::smem_u32(&bar_o_full[0]));
        }
        ok = finish_pv(1, itK - 1, j > 1);
        if (!ok) break;
        ptx::mma_commit_warp(ptx::smem_u32(&bar_kv_empty[(itK - 1) % C::kStages]));
        start_qk(1, itK);
        ptx::mma_commit_warp(ptx::smem_u32(&bar_kv_empty[itK % C::kStages]));
        if (j == nb1 - 1) ptx::mma_commit_warp(ptx::smem_u32(&bar_q_empty[1]));
      }
      it0 += 2 * nb1;
      was0 = nb0;
      was1 = nb1;
    }
    if (!ok) {
      // Wait for every MMA already issued before TMEM is freed.
      ptx::mma_commit_warp(ptx::smem_u32(&bar_drain));
      drain_wait(ptx::smem_u32(&bar_drain), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ unit fetch
    if (p.cut) {
      // Split keys: this CTA's piece of the line, unit by unit.
      const VarLine line = split_line(p, static_cast<int>(gridDim.x));
      long long x = line.bad || line.whole ? line.total : min(line.total, static_cast<long long>(blockIdx.x) * line.piece);
      const long long end = min(line.total, x + line.piece);
      VarJob job;
      job.kvh = -1;
      if (line.whole && !line.bad) direct_unit(p, &job);
      for (int n = 0;;) {
        if (x < end) {
          const LineUnit v = line_find(p, line, x);
          x = v.x1;
          job.u = make_unit(v.s, v.u, p.tp, p.causal);
          const LinePart part = line_part(line, v, job.u.nb1, blockIdx.x);
          if (part.b0 >= part.b1) continue;
          job.kvh = v.kvh;
          job.slot = part.b0 == 0 && part.b1 == job.u.nb1 ? -1 : part.slot;
          job.u.kv_row0 += part.b0 * 128;
          job.u.n_kv -= part.b0 * 128;
          job.u.lim0 -= part.b0 * 128;
          job.u.nb0 = max(1, min(job.u.nb0, part.b1) - part.b0);
          job.u.nb1 = part.b1 - part.b0;
        }
        bool got = true;
        if (lane == 0) {
          got = wait_or_abort(ptx::smem_u32(&bar_job_empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRoleVarFetch);
          if (got) {
            jobs[n & 1] = job;
            ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[n & 1]));
          }
        }
        if (n == 0) {
          // (The first job waits for nothing, so every piece leaves its entry.)
          VarCut cut;
          cut.kvh = -1;
          if (end < line.total) note_cut(p, line, blockIdx.x, &cut);
          if (lane == 0) p.cut[blockIdx.x] = cut;
        }
        if (!__shfl_sync(0xffffffffu, got, 0) || job.kvh < 0) break;
        job.kvh = -1;
        ++n;
      }
    } else if (!p.plan) {
      VarJob job;
      job.kvh = -1;
      direct_unit(p, &job);
      if (lane == 0) {
        jobs[0] = job;
        jobs[1].kvh = -1;
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[0]));
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[1]));
      }
    } else if (lane == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");   // the list is complete and visible
      const int total = p.plan->num_units * p.H_kv;
      int idx = blockIdx.x;
      for (int n = 0;; ++n) {
        VarJob job;
        job.kvh = -1;
        if (idx < total) {
          int e;
          place_unit(idx, p.plan->num_long, p.H_kv, p.group, &e, &job.kvh);
          job.u = p.list[e];
          job.slot = -1;
        }
        if (!wait_or_abort(ptx::smem_u32(&bar_job_empty[n & 1]), ((n >> 1) & 1) ^ 1u, abort_ptr,
                           kUnitWaits * p.timeout_ns, kRoleVarFetch))
          break;
        jobs[n & 1] = job;
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[n & 1]));
        if (job.kvh < 0) break;
        // The next unit is taken when the loads of this one near their end, not
        // at its start: a CTA in a long unit leaves the list to the others.
        if (!wait_or_abort(ptx::smem_u32(&bar_claim), n & 1, abort_ptr, kUnitWaits * p.timeout_ns, kRoleVarFetch)) break;
        idx = static_cast<int>(gridDim.x) + atomicAdd(&p.plan->next, 1);
      }
    }
    __syncwarp();
  }

  // The merge of split keys may be scheduled now; it waits for this grid's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The O stores must have read the staging rows before the CTA's shared
  // memory is released.
  if (warp < 8 && lane == 0) ptx::bulk_wait_group_read0();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// Joins the parts of the unit that begins to be split in piece blockIdx.x:
// LSE = m + log2 sum_s 2^{LSE_s - m}, O = sum_s 2^{LSE_s - LSE} O_s, rounded
// once to bf16. A warp per 32 rows and 16 columns (blockIdx.y: tile, quarter,
// and 64 columns), so that nothing is exchanged; the values of four parts are
// requested before the first is used. What bounds it is the latency of its two
// passes over the parts; the launch gap before it is 2 us of its time.
template <int HD>
__global__ void __launch_bounds__(128) varlen_merge_kernel(const VarParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.y & 1, row = 32 * ((blockIdx.y >> 1) & 3) + lane;
  const int c4 = 16 * (blockIdx.y >> 3) + 4 * warp;       // first column / 4
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const VarCut cut = p.cut[blockIdx.x];
  if (cut.kvh < 0) return;
  const VarUnit u = cut.u;
  const int n = cut.last - cut.first + 1;
  const int xr = (row * p.inv_g) >> 16, x = t * p.tp + xr;
  if (row >= p.G * p.tp || x >= u.n_tok) return;
  // Part s: slot 2 (first + s), the first part's one further.
  auto lse_of = [&](int s) { return p.Lp[static_cast<size_t>((2 * (cut.first + s) + (s == 0)) * 2 + t) * 128 + row]; };
  float m = -INFINITY;
#pragma unroll 8
  for (int s = 0; s < n; ++s) m = fmaxf(m, lse_of(s));     // (a NaN comes through by its weight)
  if (m == -INFINITY) m = 0.f;
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int s0 = 0; s0 < n; s0 += 4) {
    float w[4];
    float4 f[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = min(s0 + k, n - 1);                    // (past the end: the last again, with weight 0)
      w[k] = s0 + k < n ? lse_of(s) : -INFINITY;
      const float4* src = reinterpret_cast<const float4*>(p.Op) +
                          (static_cast<size_t>((2 * (cut.first + s) + (s == 0)) * 2 + t) * (HD / 4) + c4) * 128 + row;
#pragma unroll
      for (int i = 0; i < 4; ++i) f[k][i] = src[i * 128];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // A part of which the row sees nothing adds nothing, not even 0 times a NaN:
      // its O may come from a block that no row of this tile sees.
      if (s0 + k < n && w[k] != -INFINITY) {
        const float e = ptx::ex2_approx(w[k] - m);
        sum += e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i].x = fmaf(e, f[k][i].x, acc[i].x);
          acc[i].y = fmaf(e, f[k][i].y, acc[i].y);
          acc[i].z = fmaf(e, f[k][i].z, acc[i].z);
          acc[i].w = fmaf(e, f[k][i].w, acc[i].w);
        }
      }
    }
  }
  const bool none = (p.causal ? u.lim0 + x : u.n_kv) <= 0 || u.n_kv == 0;     // the row sees no key
  const float inv = none ? 0.f : 1.f / sum;
  const int head = cut.kvh * p.G + row - xr * p.G;
  const long long token = static_cast<long long>(u.q_row0) + x;
  uint4* dst = reinterpret_cast<uint4*>(p.O + token * p.o_st + head * p.o_sh + 4 * c4);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    dst[i] = make_uint4(ptx::pack_bf16x2(acc[2 * i].x * inv, acc[2 * i].y * inv),
                        ptx::pack_bf16x2(acc[2 * i].z * inv, acc[2 * i].w * inv),
                        ptx::pack_bf16x2(acc[2 * i + 1].x * inv, acc[2 * i + 1].y * inv),
                        ptx::pack_bf16x2(acc[2 * i + 1].z * inv, acc[2 * i + 1].w * inv));
  if (c4 == 0)
    p.LSE[static_cast<long long>(head) * p.T_q + token] =
        none ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace fa
