// What the kernels of attention over a paged 8-bit cache share: the line of
// units that equal CTAs cut up, its walk, the loads of pages, and the merge of
// units that several CTAs worked on. See fa_paged_kernel.cuh.
//
// The line. A unit is a tile of query rows of one sequence and K/V head with all
// the keys it sees. All units stand in a line by sequence, head and tile; each takes as
// many places as it has 128-key tiles, and a few for what it costs beside
// them. Every CTA takes an equal piece, whatever the lengths, so one long answer
// among short ones is spread over the device. Causal tiles see ever more keys; their sum is one of floors of
// a line, found in a logarithmic number of steps, so that a piece's first unit is
// found without a list of units or a launch that writes one.
// The merge is launched as a programmatic dependent of the main kernel and costs
// 1.5 us of a call.
#pragma once

#include <climits>

#include "fa_append_kernel.cuh"
#include "fa_decode_kernel.cuh"
#include "fa_prefix_kernel.cuh"

namespace fa {

namespace ptx {

// D[tmem] (+)= A[smem] B[smem]^T, both e4m3, K = 32, from a converged warp whose elected lane issues.
__device__ __forceinline__ void mma_f8_warp(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                            uint32_t b_hi, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 ad, bd;\n\t"
      "setp.ne.b32 p, %6, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 ad, {%1, %2};\n\tmov.b64 bd, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accum)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4: e4m3 operands (format 0), f32 sums.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory matrix descriptor: start, leading and stride byte offsets, swizzle (0 none, 2 128 B, 4 64 B).
__device__ __forceinline__ uint64_t desc_of(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | 1ull << 46 | static_cast<uint64_t>(swizzle) << 61;
}

// 32 lanes x 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Raises the byte count that a barrier's phase waits for, without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Maximum over the warp; NaN if any lane has one.
__device__ __forceinline__ float warp_max_nan(float x) {
  float y;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace ptx

enum : unsigned int { kRolePagedProducer = 30, kRolePagedMma = 31, kRolePagedSoftmax = 32, kRolePagedWalk = 33, kRolePagedQuery = 34 };

// Places of a unit in the line beside its tiles: what it costs beyond them.
// fa_paged_kernel, 1, 2 or 3: 64 answers of 1 to 8192 tokens 31.5, 28.7, 29.1 us; 300 of 16 to 512 49.5, 49.8,
// 51.9; eight long caches 51.7, 51.1, 50.7; 24 drafts at d = 64 17.9, 18.9, 19.5.
constexpr int kPagedCost = 2;
// fa_paged_wide_kernel (its query rows, the first products, its results), 6, 12 or 18: pieces of 1 to 1024 tokens
// on pages of 64 170, 166, 167 us, of 16 190, 188, 190, at d = 64 130, 132, 134; 32 caches
// with 16 new tokens each 95, 102, 108; eight pieces of 512 on 8192 481, 479, 481.
constexpr int kWideCost = 12;
constexpr float kPagedJump = 20.f;   // the reference moves when a tile's maximum is 2^20 above it
constexpr float kPagedNone = -3e38f; // the maximum of no keys (finite, so that differences are)
constexpr float kPagedTop = 8.f;     // a tile's largest weight is written as 2^8 (e4m3 ends at 448)

struct PagedShape {
  int B, H, H_kv, G, T_q;
  int hp, ht, tp;          // heads and tokens of a row tile, head tiles of a group
  int num_pages, page_shift, max_pages;
  int causal, ctas;
  int cost;                // kPagedCost or kWideCost
};

struct PagedSplit {        // a unit that several CTAs share, noted by the one with its beginning
  int n;                   // CTAs, 0: none
  int token, head;         // first row's
  int heads, rows;         // heads per token, rows
  int pad[3];
};

struct PagedParams {
  PagedShape s;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;              // [H, T_q]
  long long q_t, q_h, o_t, o_h;
  const float* k_scale;    // [num_pages, H_kv]
  const float* v_scale;
  const int* table;        // [B, max_pages]
  const int* lens;         // [B]
  const int* cu;           // [B + 1]
  PagedSplit* split;       // [ctas]
  float* Lp;               // [2 * ctas][N]: partial results, slot 2 c: the end of a unit, 2 c + 1: a beginning
  float* Op;               // [2 * ctas][N][d]
  float scale_log2;        // fa_paged_wide_kernel: its size, and whether to negate
  int negate;
  int keep;                // 1: K and V may be read by several CTAs
  unsigned long long timeout_ns;
  int drop_load;
};

struct PagedJob {
  int b, kvh;              // b < 0: no more
  int token, head;         // of row 0 (packed token, query head)
  int heads, rows;         // heads per token, rows that hold queries
  int lim0;                // keys that row 0's token sees; the next token one more (causal)
  int n_keys;              // keys of the unit
  int j0, j1;              // tiles
  int slot;                // of the partial result; -1: none, the unit is whole
};

// sum over i < n of floor((a i + b) / 128): the "floor sum", in as many steps as Euclid's
// algorithm takes for a and 128 (the lattice points under a line, counted by
// swapping axes). a n + b stays below 2^32: it is a number of keys.
__device__ __forceinline__ unsigned floor_sum128(unsigned n, unsigned a, unsigned b) {
  if (n == 0) return 0;
  unsigned sum = static_cast<unsigned>(static_cast<unsigned long long>(n - 1) * n / 2) * (a >> 7) + n * (b >> 7);
  a &= 127u;
  b &= 127u;
  unsigned y = a * n + b, m = a;
  n = y >> 7;
  b = y & 127u;
  a = 128;
#pragma unroll 1
  while (n > 0) {
    const unsigned qa = a / m, qb = b / m;
    sum += static_cast<unsigned>(static_cast<unsigned long long>(n - 1) * n / 2) * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const unsigned was = m;
    m = a;
    a = was;
  }
  return sum;
}

__device__ __noinline__ int paged_div(int a, int b) { return a / b; }

// One sequence as the line sees it, for one K/V head and head tile.
struct PagedSeq {
  int c0, n_q, n_kv;
  int first, groups;       // row tiles [first, groups) see keys
  __device__ __forceinline__ int keys(const PagedShape& s, int i) const {
    return s.causal ? min(n_kv, n_kv - n_q + (i + 1) * s.tp) : n_kv;
  }
  // Places before tile i.
  __device__ __forceinline__ int before(const PagedShape& s, int i) const {
    const int k = i - first;
    if (k <= 0) return 0;
    const int last = (n_kv + 127) >> 7;
    if (!s.causal || (k == groups - first && k == 1)) return k * (s.cost + last);
    const int ramp = i == groups ? k - 1 : k;          // (the last tile may be short)
    return k * s.cost + (i == groups ? last : 0) +
           static_cast<int>(floor_sum128(static_cast<unsigned>(ramp), static_cast<unsigned>(s.tp),
                                         static_cast<unsigned>(n_kv - n_q + (first + 1) * s.tp + 127)));
  }
  __device__ __forceinline__ int places(const PagedShape& s) const { return before(s, groups); }
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  PagedSeq q;
  q.c0 = c0;
  q.n_q = c0 >= 0 && c0 <= c1 && c1 <= p.s.T_q ? c1 - c0 : 0;
  q.n_kv = max(0, min(p.s.max_pages << p.s.page_shift, p.lens[b]));
  // (Code that a decode step does not need is not on its way: a launch meets a cold instruction cache.)
  q.groups = q.n_q > p.s.tp ? paged_div(q.n_q + p.s.tp - 1, p.s.tp) : min(q.n_q, 1);
  q.first = q.n_kv == 0 ? q.groups : 0;
  if (p.s.causal && q.n_kv < q.n_q && q.n_kv > 0) q.first = min(q.groups, paged_div(q.n_q - q.n_kv, p.s.tp));
  return q;
}

__device__ __noinline__ void paged_bad(int b) {
  if (atomicCAS(&g_status_word, 0u, kStatusBadOffsets) == 0u) {
    g_status_info[0] = kRolePagedWalk;
    g_status_info[1] = static_cast<unsigned int>(b);
    g_status_info[2] = g_status_info[3] = 0u;
  }
}

// A CTA's piece of the line, and where it begins.
struct PagedLine {
  int each, rest;          // pieces of each + 1 places for the first `rest` CTAs, of each for the others
  int begin, end;
  int b, cum;              // sequence of the first place; places (per K/V head and head tile) before it
};

// Most sequences whose line one warp adds up by itself.
constexpr int kPagedWarpSeqs = 256;

__device__ __forceinline__ int paged_places(const PagedParams& p, int b) {
  if (b >= p.s.B) return 0;
  if (blockIdx.x == 0) {   // (CTA 0 looks for sequences that do not fit.)
    const int c0 = p.cu[b], c1 = p.cu[b + 1], len = p.lens[b];
    if (c0 < 0 || c0 > c1 || c1 > p.s.T_q || len < 0 || len > p.s.max_pages << p.s.page_shift) paged_bad(b);
  }
  return paged_seq(p, b).places(p.s);
}

__device__ __forceinline__ void paged_cut(PagedLine* l, int seq_sum, int copies, int ctas) {
  const int total = seq_sum * copies, c = static_cast<int>(blockIdx.x);
  l->each = total / ctas;
  l->rest = total - l->each * ctas;
  l->begin = c * l->each + min(c, l->rest);
  l->end = l->begin + l->each + (c < l->rest ? 1 : 0);
}

// The line's length and this CTA's piece, found by one warp (all lanes return
// it): it adds up all sequences' places, then looks for the piece's first.
__device__ __forceinline__ PagedLine paged_line_warp(const PagedParams& p) {
  const int lane = threadIdx.x & 31, copies = p.s.H_kv * p.s.ht;
  const int first = paged_places(p, lane);
  int sum = first;
#pragma unroll 1
  for (int b = lane + 32; b < p.s.B; b += 32) sum += paged_places(p, b);
  PagedLine l;
  paged_cut(&l, __reduce_add_sync(0xffffffffu, sum), copies, p.s.ctas);
  l.b = p.s.B;
  l.cum = 0;
  int base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.s.B; b0 += 32) {
    const int nu = b0 == 0 ? first : paged_seq(p, min(b0 + lane, p.s.B - 1)).places(p.s) * (b0 + lane < p.s.B ? 1 : 0);
    int incl = nu;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const int excl = base + incl - nu;
    const unsigned hit = __ballot_sync(0xffffffffu, nu > 0 && excl * copies <= l.begin && l.begin < (excl + nu) * copies);
    if (hit) {
      const int at = __ffs(hit) - 1;
      l.b = b0 + at;
      l.cum = __shfl_sync(0xffffffffu, excl, at);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return l;
}

// The same by a whole CTA, for more sequences, into *line.
template <int kThreads>
__device__ __noinline__ void paged_line_block(const PagedParams& p, PagedLine* line) {
  __shared__ int warp_sum[kThreads / 32];
  __shared__ int start[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, copies = p.s.H_kv * p.s.ht;
  if (threadIdx.x == 0) start[0] = p.s.B, start[1] = 0;
  int sum = 0;
  for (int b = threadIdx.x; b < p.s.B; b += kThreads) sum += paged_places(p, b);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  int seq_sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) seq_sum += warp_sum[w];
  PagedLine l;
  paged_cut(&l, seq_sum, copies, p.s.ctas);
  if (l.end > l.begin) {
    const int target = l.begin / copies;
    int base = 0;
    for (int b0 = 0; b0 < p.s.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x, nu = paged_places(p, b);
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
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        chunk += warp_sum[w];
      }
      const int excl = before + incl - nu;
      if (nu > 0 && excl <= target && target < excl + nu) start[0] = b, start[1] = excl;
      base += chunk;
      if (base > target) break;
    }
  }
  __syncthreads();
  l.b = start[0];
  l.cum = start[1];
  if (threadIdx.x == 0) *line = l;
}

// Walks a CTA's piece unit by unit; a warp's lanes all hold the same state.
struct PagedWalk {
  PagedLine line;
  PagedSeq q;
  int x, b, u, i, from;    // next place; its sequence, copy, row tile and place within the unit
  bool more;

  __device__ __forceinline__ void begin(const PagedParams& p, const PagedLine& l) {
    const PagedShape& sh = p.s;
    const int copies = sh.H_kv * sh.ht;
    line = l;
    x = l.begin;
    b = l.b;
    u = i = from = 0;
    more = x < l.end && b < sh.B;
    if (!more) return;
    q = paged_seq(p, b);
    const int places = q.places(sh), y = x - l.cum * copies;
    more = places > 0 && y >= 0 && y < places * copies;
    if (!more) return;
    u = y / places;
    from = y - u * places;
    i = q.first;
    int hi = q.groups;                           // before(i) <= from < before(hi): the lanes try 32 places at a time
    if (hi - i > 1) {
      const int lane = threadIdx.x & 31;
      int base = 0;
#pragma unroll 1
      while (hi - i > 1) {
        const int step = (hi - i + 31) >> 5, mid = i + lane * step;
        const int at = mid < hi ? q.before(sh, mid) : INT_MAX;
        const int best = 31 - __clz(__ballot_sync(0xffffffffu, at <= from));
        base = __shfl_sync(0xffffffffu, at, best);
        hi = min(hi, i + (best + 1) * step);
        i += best * step;
      }
      from -= base;
    }
  }

  // The next unit's part in this piece (job.b < 0: none); *end is the unit's last place.
  __device__ __forceinline__ PagedJob next(const PagedParams& p, int* end) {
    const PagedShape& sh = p.s;
    PagedJob job{};
    job.b = -1;
    while (more && x < line.end && job.b < 0) {
      const int keys = q.keys(sh, i), tiles = (keys + 127) >> 7, places = sh.cost + tiles;
      // (Only lengths that change under the call can lead out of the unit. It ends then, with undefined results.)
      if (keys <= 0 || from >= places) {
        more = false;
        break;
      }
      const int to = min(places, from + (line.end - x));
      *end = x - from + places - 1;
      x += to - from;
      job.j0 = max(0, from - sh.cost);
      job.j1 = max(0, to - sh.cost);
      if (job.j1 > job.j0) {
        const int kvh = sh.ht == 1 ? u : u / sh.ht, h0 = (u - kvh * sh.ht) * sh.hp, t0 = i * sh.tp;
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
          if (++u == sh.H_kv * sh.ht) {
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
    return job;
  }

  // The CTA that takes place y.
  __device__ __forceinline__ int owner(int y) const {
    const int split = line.rest * (line.each + 1);
    return y < split ? y / (line.each + 1) : line.rest + (y - split) / line.each;
  }
};

constexpr int kPagedJobs = 4;            // the ring through which units are handed on

// A warp walks its CTA's piece, hands the units on and loads their pages into a
// ring of kTiles tiles, K and V of a key tile in turn. A lane has one page: 32
// entries of the table are read at a time, a batch (or a unit) ahead. The scales
// of a pair of tiles go to page_scale[pair % kScales] (K, V, and with kLogs V's
// logarithm) and count as part of the V tile.
template <int HD, int kTiles, int kScales, bool kLogs>
__device__ __forceinline__ void paged_load(const PagedParams& p, const PagedLine* line, const CUtensorMap* tmK,
                                           const CUtensorMap* tmV, PagedJob* jobs, uint64_t* bar_job_full,
                                           uint64_t* bar_job_empty, uint64_t* bar_full, uint64_t* bar_empty,
                                           float (*page_scale)[kLogs ? 3 : 2][8], uint32_t tiles_at,
                                           volatile int* abort_ptr) {
  constexpr uint32_t kTileBytes = 128 * HD;
  const int lane = threadIdx.x & 31;
  const PagedShape& sh = p.s;
  const uint64_t policy = p.keep ? ptx::policy_evict_last() : ptx::policy_evict_first();
  const int per_tile = 128 >> sh.page_shift, in_page = 1 << sh.page_shift;
  PagedWalk walk;
  walk.begin(p, p.s.B > kPagedWarpSeqs ? *line : paged_line_warp(p));
  auto entry = [&](const PagedJob& job, int e) {
    return job.b >= 0 && e < (job.n_keys + in_page - 1) >> sh.page_shift
               ? p.table[static_cast<long long>(job.b) * sh.max_pages + e] : -1;
  };
  int it = 0, end = 0, end_next = 0;       // tiles so far
  PagedJob job{};
  int id_next = -1;
  bool ok = true;
  // (Unit -1 has no tiles: the first unit is found where the next of any other is.)
#pragma unroll 1
  for (int n = -1;; ++n) {
    if (n >= 0) {
      const int ring = n & (kPagedJobs - 1);
      ok = wait_warp_or_abort(ptx::smem_u32(&bar_job_empty[ring]), ((n / kPagedJobs) & 1) ^ 1u, abort_ptr,
                              kUnitWaits * p.timeout_ns, kRolePagedWalk);
      if (!ok) break;
      if (lane == 0) {
        jobs[ring] = job;
        ptx::mbar_arrive(ptx::smem_u32(&bar_job_full[ring]));
      }
      if (job.b < 0) break;
    }
    PagedJob after{};
    int id = -1, id_after = -1;
    float sk = 0.f, sv = 0.f;
    int j = job.j0;
#pragma unroll 1
    do {
      const int in_batch = (j - job.j0) * per_tile & 31, slot = lane - in_batch;
      const bool mine = n >= 0 && slot >= 0 && slot < per_tile;
      bool drop = false;
      uint32_t full = 0;
      if (n >= 0) {
        if (in_batch == 0) {
          const int e = j * per_tile + lane;
          id = id_next;
          sk = sv = 0.f;
          if (e >= (job.n_keys + in_page - 1) >> sh.page_shift) {
            id = -1;
          } else if (id >= 0 && id < sh.num_pages) {
            sk = p.k_scale[static_cast<long long>(id) * sh.H_kv + job.kvh];
            sv = p.v_scale[static_cast<long long>(id) * sh.H_kv + job.kvh];
          } else {
            paged_bad(job.b);
            id = sh.num_pages;            // outside the tensor: reads as zeros
          }
          id_next = entry(job, e + 32);
        }
        const bool copy = mine && id >= 0;
        const uint32_t bytes = (static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, copy))) << sh.page_shift) * HD;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int tile = it % kTiles;
          ok = wait_warp_or_abort(ptx::smem_u32(&bar_empty[tile]), ((it / kTiles) & 1) ^ 1u, abort_ptr, p.timeout_ns,
                                  kRolePagedProducer);
          if (!ok) break;
          drop = it == p.drop_load;       // test hook
          full = ptx::smem_u32(&bar_full[tile]);
          if (lane == 0 && !drop) {
            if (kv == 0) ptx::mbar_arrive_expect_tx(full, bytes);
            else ptx::mbar_expect_tx(full, bytes);
          }
          __syncwarp();
          if (copy && !drop)
            ptx::tma_load_4d(tiles_at + tile * kTileBytes + (static_cast<uint32_t>(slot * HD) << sh.page_shift),
                             kv == 0 ? tmK : tmV, full, 0, 0, job.kvh, id, policy);
        }
        if (!ok) break;
      }
      if (j == job.j0) {
        // While the first copies are on their way: a beginning is noted for the merge; the next unit and its entries.
        if (n >= 0 && job.slot >= 0 && job.j0 == 0 && lane == 0) {
          PagedSplit s{};
          s.n = walk.owner(end) - static_cast<int>(blockIdx.x) + 1;
          s.token = job.token;
          s.head = job.head;
          s.heads = job.heads;
          s.rows = job.rows;
          p.split[blockIdx.x] = s;
        }
        after = walk.next(p, &end_next);
        id_after = entry(after, after.j0 * per_tile + lane);
      }
      if (n >= 0) {
        // The scales follow; the V tile counts as full when both are there.
        if (mine) {
          page_scale[((it >> 1) - 1) % kScales][0][slot] = sk;
          page_scale[((it >> 1) - 1) % kScales][1][slot] = sv;
          if (kLogs) {
            page_scale[((it >> 1) - 1) % kScales][kLogs ? 2 : 0][slot] = ptx::max_nan(ptx::lg2_approx(sv), -200.f);   // (zero, too)
          }
        }
        __syncwarp();
        if (lane == 0 && !drop) ptx::mbar_arrive(full);
      }
    } while (++j < job.j1);
    if (!ok) break;
    job = after;
    id_next = id_after;
    end = end_next;
  }
  if (__any_sync(0xffffffffu, !ok || *abort_ptr)) {
    for (int i = it > kTiles ? it - kTiles : 0; i < it; ++i)
      if (i != p.drop_load) drain_wait(ptx::smem_u32(&bar_full[i % kTiles]), (i / kTiles) & 1, p.timeout_ns);
  }
  __syncwarp();
}

// Joins the parts of the unit that CTA blockIdx.x began and others went on with:
// one warp per row, LSE = m + ln sum_s e^{LSE_s - m}, O = sum_s e^{LSE_s - LSE} O_s.
// Rows that see no key at all, of which no unit knows, are written here too.
template <int HD, int N>
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedParams p) {
  constexpr int kPer = HD / 32;
  const PagedShape& sh = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  const int warps = 4 * gridDim.y, me = blockIdx.y * 4 + warp;
  ptx::grid_next();
  ptx::grid_wait();
  // Part 0 of a unit is CTA c's beginning, part k the end in CTA c + k. The first
  // parts' LSE and rows are asked for together with the note that says how many there are.
  auto slot = [&](int k, int r) { return static_cast<size_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)) * N + r; };
  constexpr int kEarly = 4;
  const PagedSplit s = p.split[c];
  const int r0 = min(me, N - 1);
  const float lse_early = c + lane < sh.ctas ? p.Lp[slot(lane, r0)] : -INFINITY;
  float early[kEarly][kPer];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const float* src = p.Op + slot(min(k, sh.ctas - 1 - c), r0) * HD + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) early[k][e] = src[e];
  }
  for (int b = c; b < sh.B; b += gridDim.x) {
    const PagedSeq q = paged_seq(p, b);
    const int blind = min(q.n_q, q.first * sh.tp);
    // (Rows are below 2^31; the step behind the last one may not be.)
    for (unsigned r = me; r < static_cast<unsigned>(blind) * sh.H; r += warps) {
      const int t = static_cast<int>(r / sh.H), h = static_cast<int>(r - static_cast<unsigned>(t) * sh.H);
      for (int e = lane; e < HD; e += 32) p.o[(q.c0 + t) * p.o_t + h * p.o_h + e] = __float2bfloat16(0.f);
      if (lane == 0) p.lse[static_cast<long long>(h) * sh.T_q + q.c0 + t] = -INFINITY;
    }
  }
  // (Clamped: lengths that change under the call leave anything here.)
  const int n = min(s.n, sh.ctas - c), rows = min(s.rows, N);
  if (n <= 0 || s.heads <= 0) return;
  for (int r = me; r < rows; r += warps) {
    const int ti = r / s.heads, token = s.token + ti, head = s.head + r - ti * s.heads;
    if (token < 0 || token >= sh.T_q || head < 0 || head >= sh.H) continue;
    const float first = lane >= n ? -INFINITY : r == me ? lse_early : p.Lp[slot(lane, r)];
    float m = first;
    bool any = first != -INFINITY;
    for (int k = lane + 32; k < n; k += 32) {
      const float v = p.Lp[slot(k, r)];
      any |= v != -INFINITY;
      m = fmaxf(m, v);
    }
    const bool none = !__any_sync(0xffffffffu, any);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.f;
    float acc[kPer], sum = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    if (!none) {
      for (int k0 = 0; k0 < n; k0 += 32) {
        const float w_me = k0 + lane >= n ? 0.f : __expf((k0 == 0 ? first : p.Lp[slot(k0 + lane, r)]) - m);
        sum += w_me;
        int k1 = 0;
        if (k0 == 0 && r == me) {
#pragma unroll
          for (int k = 0; k < kEarly; ++k) {
            const float w = __shfl_sync(0xffffffffu, w_me, k);
            if (k < n) {
#pragma unroll
              for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, early[k][e], acc[e]);
            }
          }
          k1 = kEarly;
        }
        for (; k1 < min(32, n - k0); k1 += 4) {
          float v[4][kPer];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* src = p.Op + slot(min(k0 + k1 + k, n - 1), r) * HD + lane * kPer;
            if constexpr (kPer == 4) {
              const float4 f = *reinterpret_cast<const float4*>(src);
              v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
            } else {
              const float2 f = *reinterpret_cast<const float2*>(src);
              v[k][0] = f.x, v[k][1] = f.y;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float w = __shfl_sync(0xffffffffu, w_me, k1 + k);
            if (k0 + k1 + k < n) {
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
    __nv_bfloat16* dst = p.o + token * p.o_t + head * p.o_h + lane * kPer;
    if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
    else *reinterpret_cast<uint32_t*>(dst) = packed[0];
    if (lane == 0) p.lse[static_cast<long long>(head) * sh.T_q + token] = none ? -INFINITY : m + __logf(sum);
  }
}

}  // namespace fa
