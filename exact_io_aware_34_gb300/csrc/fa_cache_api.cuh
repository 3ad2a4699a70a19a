// Entry points for rotary positions and a paged 8-bit cache (declared in
// include/fa.h). Part of fa_api.cu, whose helpers it uses.
#pragma once

namespace {

// device_sm_count, asked once per device.
int cached_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return device_sm_count();
  return sm_count(dev);
}

// 8-bit pages [num_pages, H_kv, page, d] with byte strides (d contiguous).
struct Pages {
  const void* p;
  long long n[3], s[3];           // sizes and strides: page, head, row
  int d;

  long long span() const {
    long long e = d;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * s[i];
    return e;
  }
};

// Strides are positive whole 16-byte units below 2^36; that of a dimension of one entry is never used.
bool make_pages(Pages* c, const void* p, int num_pages, int heads, int page, int d, const fa_page_strides_t* s) {
  *c = Pages{p, {num_pages, heads, page}, {0, 0, 0}, d};
  const long long dense[3] = {static_cast<long long>(heads) * page * d, static_cast<long long>(page) * d, d};
  const long long given[3] = {s ? s->page : 0, s ? s->head : 0, s ? s->row : 0};
  for (int i = 0; i < 3; ++i) {
    c->s[i] = s && c->n[i] > 1 ? given[i] : dense[i];
    if (c->n[i] > 1 && (c->s[i] <= 0 || c->s[i] % 16 != 0 || c->s[i] >= (1LL << 36))) return false;
    if (c->n[i] == 1) c->s[i] = d;
  }
  return reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Dimensions by stride, the largest first.
void by_stride(const Pages& c, int (&order)[3]) {
  order[0] = 0, order[1] = 1, order[2] = 2;
  std::sort(order, order + 3, [&](int a, int b) { return c.s[a] > c.s[b]; });
}

// No two bytes share an address: each dimension, from the smallest stride on, steps over all that lies inside it.
bool pages_distinct(const Pages& c) {
  int order[3];
  by_stride(c, order);
  long long inside = c.d;
  for (int k = 2; k >= 0; --k) {
    const int i = order[k];
    if (c.n[i] == 1) continue;
    if (c.s[i] < inside) return false;
    inside += (c.n[i] - 1) * c.s[i];
  }
  return true;
}

// Whether two caches may share a byte. With equal strides (K and V as parts of
// one buffer) the places decide: some whole steps of each dimension, from the
// largest stride on, would have to bring b within a row's length of a.
bool steps_meet(const Pages& c, const int (&order)[3], int k, long long off) {
  if (k == 3) return off > -c.d && off < c.d;
  const int i = order[k];
  if (c.n[i] == 1) return steps_meet(c, order, k + 1, off);
  long long at = off / c.s[i];
  if (off % c.s[i] < 0) --at;
  for (long long step = at; step <= at + 1; ++step)
    if (step > -c.n[i] && step < c.n[i] && steps_meet(c, order, k + 1, off - step * c.s[i])) return true;
  return false;
}
bool pages_overlap(const Pages& a, const Pages& b) {
  if (!overlaps(a.p, static_cast<size_t>(a.span()), b.p, static_cast<size_t>(b.span()))) return false;
  for (int i = 0; i < 3; ++i)
    if (a.s[i] != b.s[i] || a.n[i] != b.n[i]) return true;
  int order[3];
  by_stride(a, order);
  return steps_meet(a, order, 0, static_cast<long long>(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p)));
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether rows may be written over rows: the same places exactly, or none in common.
bool rows_writable(const Rows& in, const Rows& out) {
  if (in.p == out.p && in.heads == out.heads && (in.T == 1 || in.st == out.st) && (in.heads == 1 || in.sh == out.sh))
    return true;
  return !rows_overlap(in, out);
}

fa::RopeTensor rope_tensor(const Rows& in, const Rows& out) {
  return fa::RopeTensor{static_cast<const __nv_bfloat16*>(in.p),
                        static_cast<__nv_bfloat16*>(const_cast<void*>(out.p)), in.st, in.sh, out.st, out.sh, in.heads};
}

// A CTA's tokens: about 40 KB of rows, as many angles as fit, and no fewer CTAs than four per SM where T allows.
fa::RopeRows rope_rows(const fa::RopeTensor& x, const fa::RopeTensor& y, int T, int d, int rot, int interleaved) {
  const int heads = x.heads + y.heads;
  fa::RopeRows r;
  r.x = x;
  r.y = y;
  r.T = T;
  r.d = d;
  r.rot = rot;
  r.interleaved = interleaved;
  int n = 40960 / (heads * d * 2);
  n = std::min(n, 2 * fa::kRopeAngles / rot);
  n = std::min(n, T / (4 * cached_sm_count()));
  r.tokens = heads > 4096 ? 1 : std::max(1, std::min(n, fa::kRopeMaxTokens));
  r.inv_heads = r.tokens == 1 ? 0u : static_cast<unsigned>(((1ull << 32) + heads - 1) / heads);
  return r;
}

// One launch on `stream`, as a programmatic dependent of what came before (every
// kernel here waits for that on the device before it touches memory).
cudaError_t launch_dependent(const void* kernel, dim3 grid, int threads, int smem, cudaStream_t stream, void** args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

fa_status_t rope_impl(const void* X, void* X_out, int heads, const void* Y, void* Y_out, int heads_y,
                      const int* positions, const double* inv_freq, int T, int d, int rot,
                      const fa_strides_t* strides, int interleaved, int transpose, float factor, cudaStream_t stream) {
  if (!X || !X_out || !positions || !inv_freq || T < 1 || heads < 1 || heads_y < 0 || d < 1 || rot < 1 || rot > d)
    return FA_ERR_INVALID_ARG;
  if (heads > 65535 || heads_y > 65535 || static_cast<long long>(T) * (heads + heads_y) >= (1LL << 31))
    return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (transpose != 0 && transpose != 1) || !std::isfinite(factor))
    return FA_ERR_INVALID_ARG;
  if (heads_y > 0 && (!Y || !Y_out)) return FA_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > 2 * fa::kRopeMaxPairs || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return FA_ERR_INVALID_ARG;
  Rows in[2], out[2];
  const int n = heads_y > 0 ? 2 : 1;
  for (int i = 0; i < n; ++i) {
    const int h = i ? heads_y : heads;
    if (!make_rows(&in[i], i ? Y : X, T, h, d, strides ? strides + 2 * i : nullptr) ||
        !make_rows(&out[i], i ? Y_out : X_out, T, h, d, strides ? strides + 2 * i + 1 : nullptr) ||
        !rows_distinct(out[i]))
      return FA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i) {
    if (rows_overlap(out[i], positions, static_cast<size_t>(T) * 4) ||
        rows_overlap(out[i], inv_freq, static_cast<size_t>(rot) * 4) || !rows_writable(in[i], out[i]))
      return FA_ERR_INVALID_ARG;
    if (n == 2 && rows_overlap(out[i], in[1 - i])) return FA_ERR_INVALID_ARG;
  }
  if (n == 2 && rows_overlap(out[0], out[1])) return FA_ERR_INVALID_ARG;

  fa::RopeParams p;
  p.r = rope_rows(rope_tensor(in[0], out[0]), n == 2 ? rope_tensor(in[1], out[1]) : fa::RopeTensor{}, T, d, rot, interleaved);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.transpose = transpose;
  p.factor = factor;
  void* args[1] = {&p};
  const cudaError_t e = launch_dependent(reinterpret_cast<const void*>(&fa::fa_rope_kernel),
                                         dim3(static_cast<unsigned>((T + p.r.tokens - 1) / p.r.tokens)),
                                         fa::kRopeThreads, 0, stream, args);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

// Sizes that fa_kv_append and fa_fwd_paged accept.
fa_status_t cache_sizes(int B, int H_kv, int T, int d, int num_pages, int page, int max_pages) {
  if (B < 1 || H_kv < 1 || T < 1 || d < 1 || num_pages < 1 || page < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (B > (1 << 20) || H_kv > 65535 || static_cast<long long>(num_pages) * H_kv >= (1LL << 31) ||
      static_cast<long long>(max_pages) * page > kMaxLength || T > kMaxLength)
    return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || (page != 16 && page != 32 && page != 64 && page != 128)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status_t append_impl(const void* K, const void* V, const int* cu_new, void* K_cache, void* V_cache, float* k_scale,
                        float* v_scale, const int* page_table, const int* seq_lens, const void* Q, void* Q_out,
                        const double* inv_freq, const int* positions, int B, int H, int H_kv, int T, int d,
                        int num_pages, int page, int max_pages, int rot, const fa_strides_t* strides,
                        const fa_page_strides_t* cache_strides, int interleaved, float factor, cudaStream_t stream) {
  if (!K || !V || !cu_new || !K_cache || !V_cache || !k_scale || !v_scale || !page_table || !seq_lens)
    return FA_ERR_INVALID_ARG;
  const fa_status_t st = cache_sizes(B, H_kv, T, d, num_pages, page, max_pages);
  if (st != FA_OK) return st;
  if (rot < 0 || rot > d || (rot > 0 && !inv_freq) || (Q && (!Q_out || rot == 0 || H < 1 || H > 65535)))
    return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || !std::isfinite(factor)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * H_kv >= (1LL << 31) || (Q && static_cast<long long>(T) * H >= (1LL << 31)))
    return FA_ERR_INVALID_ARG;
  if (rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  for (const void* a : {static_cast<const void*>(cu_new), static_cast<const void*>(k_scale),
                        static_cast<const void*>(v_scale), static_cast<const void*>(page_table),
                        static_cast<const void*>(seq_lens), static_cast<const void*>(positions)})
    if (!aligned(a, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(inv_freq, 8)) return FA_ERR_INVALID_ARG;
  Rows k, v, q, qo;
  Pages kc, vc;
  if (!make_rows(&k, K, T, H_kv, d, strides) || !make_rows(&v, V, T, H_kv, d, strides ? strides + 1 : nullptr) ||
      !make_pages(&kc, K_cache, num_pages, H_kv, page, d, cache_strides) ||
      !make_pages(&vc, V_cache, num_pages, H_kv, page, d, cache_strides ? cache_strides + 1 : nullptr) ||
      !pages_distinct(kc) || !pages_distinct(vc) || pages_overlap(kc, vc))
    return FA_ERR_INVALID_ARG;
  if (Q && (!make_rows(&q, Q, T, H, d, strides ? strides + 2 : nullptr) ||
            !make_rows(&qo, Q_out, T, H, d, strides ? strides + 3 : nullptr) || !rows_distinct(qo) ||
            !rows_writable(q, qo) || rows_overlap(qo, k) || rows_overlap(qo, v)))
    return FA_ERR_INVALID_ARG;
  // What is written apart from the rows is disjoint from everything else.
  struct Part {
    const void* p;
    size_t n;
  };
  const size_t n_scale = static_cast<size_t>(num_pages) * H_kv * 4;
  const Part written[4] = {{K_cache, static_cast<size_t>(kc.span())}, {V_cache, static_cast<size_t>(vc.span())},
                           {k_scale, n_scale}, {v_scale, n_scale}};
  const Part read[5] = {{cu_new, (static_cast<size_t>(B) + 1) * 4}, {seq_lens, static_cast<size_t>(B) * 4},
                        {page_table, static_cast<size_t>(B) * max_pages * 4},
                        {positions, positions ? static_cast<size_t>(T) * 4 : 0},
                        {inv_freq, inv_freq ? static_cast<size_t>(rot) * 4 : 0}};
  for (int i = 0; i < 4; ++i) {
    for (const Part& r : read)
      if (r.n && overlaps(written[i].p, written[i].n, r.p, r.n)) return FA_ERR_INVALID_ARG;
    for (int j = std::max(2, i + 1); j < 4; ++j)
      if (overlaps(written[i].p, written[i].n, written[j].p, written[j].n)) return FA_ERR_INVALID_ARG;
    if (rows_overlap(k, written[i].p, written[i].n) || rows_overlap(v, written[i].p, written[i].n) ||
        (Q && (rows_overlap(q, written[i].p, written[i].n) || rows_overlap(qo, written[i].p, written[i].n))))
      return FA_ERR_INVALID_ARG;
  }
  for (const Part& r : read)
    if (Q && r.n && rows_overlap(qo, r.p, r.n)) return FA_ERR_INVALID_ARG;

  fa::AppendParams p;
  const Rows* rows[2] = {&k, &v};
  const Pages* pages[2] = {&kc, &vc};
  for (int i = 0; i < 2; ++i) {
    p.kv[i] = static_cast<const __nv_bfloat16*>(rows[i]->p);
    p.in_t[i] = rows[i]->st;
    p.in_h[i] = rows[i]->sh;
    p.cache[i] = static_cast<uint8_t*>(const_cast<void*>(pages[i]->p));
    p.c_page[i] = pages[i]->s[0];
    p.c_head[i] = pages[i]->s[1];
    p.c_row[i] = pages[i]->s[2];
  }
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.cu = cu_new;
  p.table = page_table;
  p.lens = seq_lens;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.q = fa::RopeRows{};
  if (Q) p.q = rope_rows(rope_tensor(q, qo), fa::RopeTensor{}, T, d, rot, interleaved);
  p.B = B;
  p.H_kv = H_kv;
  p.T = T;
  p.d = d;
  p.num_pages = num_pages;
  p.page = page;
  p.max_pages = max_pages;
  p.rot = rot;
  p.interleaved = interleaved;
  p.factor = factor;
  const long long by_page = T / page + 2LL * B;
  p.per_token = T <= by_page;
  p.places = static_cast<int>(std::min<long long>(T, by_page));
  p.warps = p.per_token ? 1 : page / 16;
  p.head_groups = (H_kv * p.warps + 7) / 8;
  p.query_ctas = Q ? (T + p.q.tokens - 1) / p.q.tokens : 0;
  const long long kv_ctas = 2LL * p.places * p.head_groups, ctas = kv_ctas + p.query_ctas;
  if (ctas >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  p.period = p.query_ctas ? static_cast<int>(kv_ctas / p.query_ctas) + 1 : 1;
  const void* kernel = d == 64 ? reinterpret_cast<const void*>(&fa::fa_append_kernel<64>)
                               : reinterpret_cast<const void*>(&fa::fa_append_kernel<128>);
  // The angles of a page's rows; of a query CTA's tokens.
  const int smem = static_cast<int>(sizeof(float2)) * std::max(page * rot / 2, Q ? p.q.tokens * rot / 2 : 0);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  std::call_once(once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(fa::fa_append_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, fa::kAppendMaxSmem);
    if (attr_err[dev] == cudaSuccess)
      attr_err[dev] = cudaFuncSetAttribute(fa::fa_append_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, fa::kAppendMaxSmem);
  });
  if (attr_err[dev] != cudaSuccess) return cuda_fail(attr_err[dev]);
  void* args[1] = {&p};
  e = launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), fa::kAppendThreads, smem, stream, args);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

fa_status_t paged_sizes(int B, int H, int H_kv, int T_q, int d, int num_pages, int page, int max_pages) {
  if (H < 1 || H > 65535) return FA_ERR_INVALID_ARG;
  const fa_status_t st = cache_sizes(B, H_kv, T_q, d, num_pages, page, max_pages);
  if (st == FA_ERR_INVALID_ARG) return st;
  if (H % H_kv != 0 || static_cast<long long>(H) * T_q >= (1LL << 31)) return FA_ERR_INVALID_ARG;
  if (st != FA_OK) return st;
  if (H / H_kv > 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// 4-D map of 8-bit pages; a box is the rows of one page and head.
bool make_page_map(CUtensorMap* m, const Pages& c) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.n[2]),
                        static_cast<cuuint64_t>(c.n[1]), static_cast<cuuint64_t>(c.n[0])};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.s[2]), static_cast<cuuint64_t>(c.s[1]),
                           static_cast<cuuint64_t>(c.s[0])};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(c.d), static_cast<cuuint32_t>(c.n[2]), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(c.p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a unit: 4 or 8 (fa_paged_kernel) while the sequences' new tokens, on
// average, fill no more than a unit of 4 or two of 8, else 256 (fa_paged_wide_kernel).
// Two units read K and V twice, the second time mostly from L2: with 16 rows 24 caches of
// 100 to 8000 keys take 44 us so and 66 in the other kernel, with four tokens of 24 drafts
// at d = 64 19 and 26, four long caches 42 and 48. With 20 rows of 5 heads 37 and 35, with
// 32 rows 62 and 53. (A variant with 16 rows in a unit, and hi and lo as two products,
// took 74 us for the four long caches.) An average says little where rows are unequal: 511 single
// tokens on caches of 300 to 4000 beside 1500 tokens on one, 32 heads on 8, take 973 us in units of 8 and
// 1077 in units of 256 where that one has 4000 keys, 3230 and 1474 where it has 16000; as two calls
// 235 + 115 and 235 + 346. The host knows no sequence's rows, so it cannot tell these from drafts.
int paged_rows(int B, int G, int T_q) {
  const long long rows = static_cast<long long>(T_q) * G;
  return rows <= 4LL * B ? 4 : rows <= 16LL * B ? 8 : 256;
}

fa::PagedShape paged_shape(int B, int H, int H_kv, int T_q, int num_pages, int page, int max_pages, int causal) {
  fa::PagedShape s;
  const int N = paged_rows(B, H / H_kv, T_q);
  s.B = B;
  s.H = H;
  s.H_kv = H_kv;
  s.G = H / H_kv;
  s.T_q = T_q;
  s.hp = std::min(s.G, N);
  s.ht = (s.G + s.hp - 1) / s.hp;
  s.tp = s.ht == 1 ? N / s.hp : 1;
  s.num_pages = num_pages;
  s.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  s.max_pages = max_pages;
  s.causal = causal;
  s.cost = N > 8 ? fa::kWideCost : fa::kPagedCost;
  return s;
}

// Places of the line at most (0: more than can be counted in 32 bits on the device), and the CTAs that share them.
long long paged_places(const fa::PagedShape& s) {
  const double units = (static_cast<double>(s.T_q / s.tp) + s.B) * s.H_kv * s.ht;
  const double places = units * (((static_cast<long long>(s.max_pages) << s.page_shift) + 127) / 128 + s.cost);
  return places < 2147418112.0 ? static_cast<long long>(places) : 0;
}
int paged_ctas(const fa::PagedShape& s, int N) {
  return static_cast<int>(std::min(paged_places(s), (N > 8 ? 1LL : 2LL) * cached_sm_count()));
}

struct PagedLayout {
  size_t Lp, Op, bytes;    // the notes on split units are at the front
};
PagedLayout paged_layout(int ctas, int N, int d) {
  PagedLayout w;
  w.Lp = (static_cast<size_t>(ctas) * sizeof(fa::PagedSplit) + 127) / 128 * 128;
  w.Op = w.Lp + static_cast<size_t>(2 * ctas) * N * 4;
  w.bytes = w.Op + static_cast<size_t>(2 * ctas) * N * d * 4;
  return w;
}

// Per kernel and device: the shared-memory opt-in, and, for a kernel whose
// warpgroups share out registers, whether the built kernel has as many (see the forward launch).
struct PagedKernel {
  const void* main;
  const void* merge;
  int smem, threads, regs;      // regs: needed per thread at launch, 0: any
};

template <int HD, int N, int NG>
const PagedKernel& paged_kernel() {
  if constexpr (N <= 8) {
    using C = fa::PagedCfg<HD, N>;
    static const PagedKernel k{reinterpret_cast<const void*>(&fa::fa_paged_kernel<HD, N>),
                               reinterpret_cast<const void*>(&fa::paged_merge_kernel<HD, N>), C::kSmemBytes, C::kThreads, 0};
    return k;
  } else {
    using C = fa::PagedWideCfg<HD, NG>;
    static_assert(N == C::kRows, "rows of a unit");
    static const PagedKernel k{reinterpret_cast<const void*>(&fa::fa_paged_wide_kernel<HD, NG>),
                               reinterpret_cast<const void*>(&fa::paged_merge_kernel<HD, N>), C::kSmemBytes, C::kThreads,
                               (C::kRegsSoftmax + C::kRegsOther) / 2};
    return k;
  }
}

template <int HD, int N, int NG = 0>
fa_status_t paged_launch(const Pages& kc, const Pages& vc, fa::PagedParams& p, cudaStream_t stream) {
  const PagedKernel& k = paged_kernel<HD, N, NG>();
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  static bool regs_ok[64];
  std::call_once(once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(k.main, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    cudaFuncAttributes fattr;
    if (attr_err[dev] == cudaSuccess) attr_err[dev] = cudaFuncGetAttributes(&fattr, k.main);
    regs_ok[dev] = attr_err[dev] == cudaSuccess && fattr.numRegs >= k.regs;
  });
  if (attr_err[dev] != cudaSuccess) return cuda_fail(attr_err[dev]);
  if (!regs_ok[dev]) return FA_ERR_UNSUPPORTED;
  CUtensorMap mk, mv;
  if (!make_page_map(&mk, kc) || !make_page_map(&mv, vc)) return cuda_fail(cudaErrorInvalidValue);
  void* args[3] = {&mk, &mv, &p};
  e = launch_dependent(k.main, dim3(static_cast<unsigned>(p.s.ctas)), k.threads, k.smem, stream, args);
  if (e != cudaSuccess) return cuda_fail(e);
  void* merge_args[1] = {&p};
  e = launch_dependent(k.merge, dim3(static_cast<unsigned>(p.s.ctas), static_cast<unsigned>((N + 15) / 16)), 128, 0, stream,
                       merge_args);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

template <int HD>
fa_status_t paged_launch_rows(int N, const Pages& kc, const Pages& vc, fa::PagedParams& p, cudaStream_t stream) {
  switch (N) {
    case 4: return paged_launch<HD, 4>(kc, vc, p, stream);
    case 8: return paged_launch<HD, 8>(kc, vc, p, stream);
    default:
      return p.s.page_shift >= 6 ? paged_launch<HD, 256, 2>(kc, vc, p, stream)
                                 : paged_launch<HD, 256, 8>(kc, vc, p, stream);
  }
}

fa_status_t paged_impl(const void* Q, const void* K_cache, const void* V_cache, const float* k_scale,
                       const float* v_scale, const int* page_table, const int* seq_lens, const int* cu_q, void* O,
                       float* LSE, int B, int H, int H_kv, int T_q, int d, int num_pages, int page, int max_pages,
                       const fa_strides_t* strides, const fa_page_strides_t* cache_strides, float scale, int causal,
                       void* workspace, size_t workspace_bytes, int drop_load,
                       unsigned long long timeout_ns, cudaStream_t stream) {
  if (!Q || !K_cache || !V_cache || !k_scale || !v_scale || !page_table || !seq_lens || !cu_q || !O || !LSE)
    return FA_ERR_INVALID_ARG;
  const fa_status_t st = paged_sizes(B, H, H_kv, T_q, d, num_pages, page, max_pages);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  for (const void* a : {static_cast<const void*>(k_scale), static_cast<const void*>(v_scale),
                        static_cast<const void*>(page_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(cu_q), static_cast<const void*>(LSE)})
    if (!aligned(a, 4)) return FA_ERR_INVALID_ARG;
  Rows q, o;
  Pages kc, vc;
  if (!make_rows(&q, Q, T_q, H, d, strides) || !make_rows(&o, O, T_q, H, d, strides ? strides + 1 : nullptr) ||
      !rows_distinct(o) || !make_pages(&kc, K_cache, num_pages, H_kv, page, d, cache_strides) ||
      !make_pages(&vc, V_cache, num_pages, H_kv, page, d, cache_strides ? cache_strides + 1 : nullptr))
    return FA_ERR_INVALID_ARG;
  const size_t n_lse = static_cast<size_t>(H) * T_q * 4, n_scale = static_cast<size_t>(num_pages) * H_kv * 4;
  fa::PagedParams p;
  p.s = paged_shape(B, H, H_kv, T_q, num_pages, page, max_pages, causal);
  if (paged_places(p.s) == 0) return FA_ERR_UNSUPPORTED;
  const int N = paged_rows(B, H / H_kv, T_q);
  p.s.ctas = paged_ctas(p.s, N);
  const PagedLayout w = paged_layout(p.s.ctas, N, d);
  if (!workspace || !aligned(workspace, 128) || workspace_bytes < w.bytes) return FA_ERR_INVALID_ARG;
  auto clash = [&](const void* a, size_t na) { return rows_overlap(o, a, na) || overlaps(LSE, n_lse, a, na) ||
                                                  overlaps(workspace, w.bytes, a, na); };
  if (rows_overlap(o, q) || rows_overlap(q, LSE, n_lse) || rows_overlap(o, LSE, n_lse) ||
      rows_overlap(q, workspace, w.bytes) || rows_overlap(o, workspace, w.bytes) ||
      overlaps(LSE, n_lse, workspace, w.bytes) ||
      clash(K_cache, static_cast<size_t>(kc.span())) || clash(V_cache, static_cast<size_t>(vc.span())) ||
      clash(k_scale, n_scale) || clash(v_scale, n_scale) ||
      clash(page_table, static_cast<size_t>(B) * max_pages * 4) || clash(seq_lens, static_cast<size_t>(B) * 4) ||
      clash(cu_q, (static_cast<size_t>(B) + 1) * 4))
    return FA_ERR_INVALID_ARG;
  p.q = static_cast<const __nv_bfloat16*>(Q);
  p.o = static_cast<__nv_bfloat16*>(O);
  p.lse = LSE;
  p.q_t = q.st;
  p.q_h = q.sh;
  p.o_t = o.st;
  p.o_h = o.sh;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.lens = seq_lens;
  p.cu = cu_q;
  char* ws = static_cast<char*>(workspace);
  p.split = reinterpret_cast<fa::PagedSplit*>(ws);
  p.Lp = reinterpret_cast<float*>(ws + w.Lp);
  p.Op = reinterpret_cast<float*>(ws + w.Op);
  p.scale_log2 = N > 8 ? masked_scale_log2(scale) : static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.negate = scale < 0.f;
  p.keep = p.s.ht > 1 || T_q > static_cast<long long>(B) * p.s.tp;
  p.timeout_ns = timeout_ns;
  p.drop_load = drop_load;
  return d == 64 ? paged_launch_rows<64>(N, kc, vc, p, stream) : paged_launch_rows<128>(N, kc, vc, p, stream);
}

}  // namespace

extern "C" {

fa_status_t fa_rope_frequencies(double* inv_freq, int rot, double base, int ramp, double factor, double low_turns,
                                double high_turns, double original) {
  if (!inv_freq || rot < 2 || rot % 2 != 0 || !(base > 0) || !std::isfinite(base) || !(factor > 0) ||
      !std::isfinite(factor) || ramp < 0 || ramp > 2)
    return FA_ERR_INVALID_ARG;
  if (ramp > 0 && (!(low_turns > 0) || !(high_turns > low_turns) || !std::isfinite(high_turns) || !(original > 0) ||
                   !std::isfinite(original)))
    return FA_ERR_INVALID_ARG;
  for (int j = 0; j < rot / 2; ++j) {
    const double theta = std::pow(base, -2.0 * j / rot);
    double kept = 0.0;             // the share that keeps its frequency
    if (ramp > 0) {
      const double r = original * theta / 6.283185307179586477;
      kept = ramp == 1 ? (r - low_turns) / (high_turns - low_turns)
                       : std::log(r / low_turns) / std::log(high_turns / low_turns);
      kept = std::min(1.0, std::max(0.0, kept));
    }
    inv_freq[j] = theta * (kept + (1.0 - kept) / factor);
  }
  return FA_OK;
}

fa_status_t fa_rope(const void* X, void* X_out, int heads, const void* Y, void* Y_out, int heads_y,
                    const int* positions, const double* inv_freq, int T, int d, int rot, const fa_strides_t* strides,
                    int interleaved, int transpose, float factor, cudaStream_t stream) {
  return rope_impl(X, X_out, heads, Y, Y_out, heads_y, positions, inv_freq, T, d, rot, strides, interleaved, transpose,
                   factor, stream);
}

fa_status_t fa_kv_append(const void* K, const void* V, const int* cu_new, void* K_cache, void* V_cache, float* k_scale,
                         float* v_scale, const int* page_table, const int* seq_lens, const void* Q, void* Q_out,
                         const double* inv_freq, const int* positions, int B, int H, int H_kv, int T, int d,
                         int num_pages, int page_size, int max_pages, int rot, const fa_strides_t* strides,
                         const fa_page_strides_t* cache_strides, int interleaved, float factor, cudaStream_t stream) {
  return append_impl(K, V, cu_new, K_cache, V_cache, k_scale, v_scale, page_table, seq_lens, Q, Q_out, inv_freq,
                     positions, B, H, H_kv, T, d, num_pages, page_size, max_pages, rot, strides, cache_strides,
                     interleaved, factor, stream);
}

size_t fa_fwd_paged_workspace_bytes(int B, int H, int H_kv, int T_q, int d, int num_pages, int page_size,
                                    int max_pages) {
  if (paged_sizes(B, H, H_kv, T_q, d, num_pages, page_size, max_pages) != FA_OK) return 0;
  const fa::PagedShape s = paged_shape(B, H, H_kv, T_q, num_pages, page_size, max_pages, 1);
  const int N = paged_rows(B, H / H_kv, T_q);
  return paged_places(s) ? paged_layout(paged_ctas(s, N), N, d).bytes : 0;
}

fa_status_t fa_fwd_paged(const void* Q, const void* K_cache, const void* V_cache, const float* k_scale,
                         const float* v_scale, const int* page_table, const int* seq_lens, const int* cu_q, void* O,
                         float* LSE, int B, int H, int H_kv, int T_q, int d, int num_pages, int page_size,
                         int max_pages, const fa_strides_t* strides, const fa_page_strides_t* cache_strides,
                         float scale, int causal, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return paged_impl(Q, K_cache, V_cache, k_scale, v_scale, page_table, seq_lens, cu_q, O, LSE, B, H, H_kv, T_q, d,
                    num_pages, page_size, max_pages, strides, cache_strides, scale, causal, workspace, workspace_bytes, -1,
                    kDefaultTimeoutNs, stream);
}

fa_status_t fa_fwd_paged_fault_test(const void* Q, const void* K_cache, const void* V_cache, const float* k_scale,
                                    const float* v_scale, const int* page_table, const int* seq_lens, const int* cu_q,
                                    void* O, float* LSE, int B, int H, int H_kv, int T_q, int d, int num_pages,
                                    int page_size, int max_pages, float scale, int causal, void* workspace,
                                    size_t workspace_bytes, int drop_load, unsigned long long timeout_ns,
                                    cudaStream_t stream) {
  if (timeout_ns == 0) return FA_ERR_INVALID_ARG;
  return paged_impl(Q, K_cache, V_cache, k_scale, v_scale, page_table, seq_lens, cu_q, O, LSE, B, H, H_kv, T_q, d,
                    num_pages, page_size, max_pages, nullptr, nullptr, scale, causal, workspace, workspace_bytes,
                    drop_load < 0 ? -1 : drop_load, timeout_ns, stream);
}

}  // extern "C"
