// Entry points for packed sequences of different lengths (declared in
// include/fa.h): argument checks, descriptors, workspace layout, launches.
// Part of fa_api.cu, whose helpers it uses.
#pragma once

namespace {

// A tensor [T, heads, d] with element strides for T and heads (d contiguous).
struct Rows {
  const void* p;
  int T, heads, d;
  long long st, sh;
  int elem;                       // bytes per element

  // Bytes from the first element to behind the last, and of one token's heads.
  long long row_span() const { return ((heads - 1) * sh + d) * elem; }
  long long span() const { return (T - 1) * st * elem + row_span(); }
};

// Fills strides in (NULL: contiguous [T, heads, d]) and checks what a TMA
// descriptor and 16-byte accesses need: positive strides, whole 16-byte units,
// below 2^40 bytes. The stride of a dimension of one entry is never used.
bool make_rows(Rows* r, const void* p, int T, int heads, int d, const fa_strides_t* s, int elem = 2) {
  *r = Rows{p, T, heads, d, s ? s->token : static_cast<long long>(heads) * d, s ? s->head : d, elem};
  if (T == 1) r->st = static_cast<long long>(heads) * d;
  if (heads == 1) r->sh = d;
  if (T == 1 && heads > 1) r->st = heads * r->sh;
  for (long long v : {r->st, r->sh})
    if (v <= 0 || v * elem % 16 != 0 || v >= (1LL << 39)) return false;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// No two elements of a written tensor share an address.
bool rows_distinct(const Rows& r) {
  const bool heads_in = r.sh >= r.d && r.st >= (r.heads - 1) * r.sh + r.d;
  const bool tokens_in = r.st >= r.d && r.sh >= (r.T - 1) * r.st + r.d;
  return heads_in || tokens_in;
}

// Whether two tensors may share an element. Tensors that are column ranges of
// one wider buffer (equal token strides, each token's heads inside one stride)
// are told apart by their place within the stride; others by their extents.
bool rows_overlap(const Rows& a, const Rows& b) {
  const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (!(x < y + b.span() && y < x + a.span())) return false;
  const long long sa = a.st * a.elem, sb = b.st * b.elem;
  if (sa == sb && a.row_span() <= sa && b.row_span() <= sa) {
    const long long off = ((static_cast<long long>(x - y) % sa) + sa) % sa;   // a's place after b's, modulo the stride
    return !(off >= b.row_span() && sa - off >= a.row_span());
  }
  return true;
}

bool rows_overlap(const Rows& a, const void* b, size_t nb) {
  return overlaps(a.p, static_cast<size_t>(a.span()), b, nb);
}

// bf16 map [d][n1][n2] with element strides s1, s2; box b0 x b1 x b2 with b0 =
// 64 (128-byte swizzle) or 32 (64-byte swizzle).
bool make_map_strided(CUtensorMap* m, const void* base, int d, int n1, long long s1, int n2, long long s2, int b1,
                      int b2, int b0 = 64) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(b0), static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, b0 == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// |scale| * log2(e) for kernels that mask with -inf: never zero, so that a
// masked score stays -inf (a finite score times 2^-126 counts as 0).
float masked_scale_log2(float scale) {
  return std::max(static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634074), 1.17549435e-38f);
}

// Longest T_q, T_kv, N_prefix and N_own: places and blocks behind one are counted
// in 32 bits on the device.
constexpr int kMaxLength = 0x7fff0000;

// Sizes every entry point for packed sequences accepts.
fa_status_t varlen_sizes(int B, int H, int H_kv, int T_q, int T_kv, int d, float scale, int causal) {
  if (B < 1 || H < 1 || H_kv < 1 || T_q < 1 || T_kv < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (B > (1 << 24) || H > 65535 || H % H_kv != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(H) * T_q >= (1LL << 31) || static_cast<long long>(H_kv) * T_kv >= (1LL << 31))
    return FA_ERR_INVALID_ARG;
  if (T_q > kMaxLength || T_kv > kMaxLength) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (H / H_kv > 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// K/V heads whose long units are taken together: as many as stream at most
// 48 MB, of which each of the two halves of L2 (129 MB) keeps a copy. Forward and
// backward of 8192 tokens, 32 K/V heads, not causal: 724 and 2460 us with all
// heads together, 703 and 2320 in groups; 24 MB cost the backward of two
// documents of 4096 tokens 11 % by fewer units to balance.
int head_group(int H_kv, double bytes_per_head) {
  return std::max(1, static_cast<int>(std::min<double>(H_kv, 48e6 / bytes_per_head)));
}

// Units (per K/V head) of the forward list: every sequence rounds up once.
long long varlen_fwd_cap(int B, int H, int H_kv, int T_q) {
  const int tp = 128 / (H / H_kv);
  return T_q / (2 * tp) + static_cast<long long>(B);
}

// Whether all units of all K/V heads can be counted in 32 bits on the device.
bool units_countable(long long units, int H_kv) { return units * H_kv < (1LL << 31) - 65536; }

// Whether the grid holds every unit at once: then there is no list.
bool varlen_fwd_direct(int B, int H, int H_kv, int T_q) {
  return varlen_fwd_cap(B, H, H_kv, T_q) * H_kv <= device_sm_count();
}

// CTAs among which the keys of all units are split, or 0 (see split_line): at
// most one per kSplitMin places of the longest line these sizes allow.
int varlen_fwd_pieces(int B, int H, int H_kv, int T_q, int T_kv, int causal) {
  if (T_kv <= fa::kSplitKeys || !varlen_fwd_direct(B, H, H_kv, T_q)) return 0;
  if (B == 1) {
    // One sequence that fills its buffers, not causal, would be found not to need
    // it: spare the call the finding out and the merge's empty launch (3 of 31 us).
    const int unit_tokens = 2 * (128 / (H / H_kv));
    const double units = (T_q - 1) / unit_tokens + 1;
    auto gains = [&](double first, double longest, int gain) {   // places of its units, growing evenly
      const double line = H_kv * units * (first + longest) / 2;
      return longest > std::max<double>(fa::kSplitMin, line / device_sm_count()) + gain;
    };
    bool split = gains(fa::kSplitCost + static_cast<double>(T_kv), fa::kSplitCost + static_cast<double>(T_kv), fa::kSplitGain);
    // Causal, the longest unit is up to twice the average, but joining the parts of
    // a prompt that nearly fills the device takes as long as twelve blocks. 8 heads
    // on 2, 4096 tokens (2385 places above the average): 47.1 us whole, 45.5 split,
    // with d = 64 41.8 and 34.1; 16 on 4, 2048 and 2300 tokens (1200 and 1250
    // above): 27.4 and 30.4 whole, 36.1 and 40.8 split.
    if (causal && T_q <= T_kv) {
      const double first = fa::kSplitCost + static_cast<double>(T_kv - T_q) + unit_tokens;
      split |= gains(first, first + (units - 1) * unit_tokens, fa::kSplitGain + fa::kSplitGain / 2);
    }
    if (!split) return 0;
  }
  const long long units = varlen_fwd_cap(B, H, H_kv, T_q) * H_kv;
  const double places = static_cast<double>(units) * (fa::kSplitCost + 256.0 + T_kv);
  return static_cast<int>(std::max<double>(units, std::min<double>(device_sm_count(), places / fa::kSplitMin + 1)));
}

size_t varlen_fwd_ws(int B, int H, int H_kv, int T_q, int T_kv, int d, int causal) {
  if (varlen_fwd_direct(B, H, H_kv, T_q))   // per piece two partial results of 256 rows and an entry, or nothing
    return static_cast<size_t>(varlen_fwd_pieces(B, H, H_kv, T_q, T_kv, causal)) *
           (2 * 256 * (d + 1) * sizeof(float) + sizeof(fa::VarCut));
  return sizeof(fa::VarPlan) + static_cast<size_t>(varlen_fwd_cap(B, H, H_kv, T_q)) * sizeof(fa::VarUnit);
}

template <int HD>
fa_status_t varlen_fwd_launch(const Rows& q, const Rows& k, const Rows& v, const Rows& o, float* LSE, const int* cu_q,
                              const int* cu_kv, int B, float scale, int causal, void* ws, int drop_load,
                              unsigned long long timeout_ns, cudaStream_t stream) {
  using C = fa::FwdCfg<HD>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  static bool regs_ok[64];
  std::call_once(once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(fa::fa_varlen_fwd_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmemBytes);
    // The warpgroups' register split must fit the registers the block is
    // launched with (see the forward launch).
    cudaFuncAttributes fattr;
    if (attr_err[dev] == cudaSuccess) attr_err[dev] = cudaFuncGetAttributes(&fattr, fa::fa_varlen_fwd_kernel<HD>);
    regs_ok[dev] = attr_err[dev] == cudaSuccess && 8 * C::kRegsSoftmax + 4 * C::kRegsControl <= 12 * fattr.numRegs;
  });
  if (attr_err[dev] != cudaSuccess) return cuda_fail(attr_err[dev]);
  if (!regs_ok[dev]) return FA_ERR_UNSUPPORTED;

  const int H_kv = k.heads, G = q.heads / k.heads, tp = 128 / G;
  // O's box: a warp's 32 rows, G heads of 32 / G tokens or 32 heads of one.
  const bool o_tma = (G & (G - 1)) == 0;
  CUtensorMap mq, mk, mv, mo;
  if (!make_map_strided(&mq, q.p, HD, q.heads, q.sh, q.T, q.st, G, tp) ||
      !make_map_strided(&mk, k.p, HD, k.T, k.st, k.heads, k.sh, 128, 1) ||
      !make_map_strided(&mv, v.p, HD, v.T, v.st, v.heads, v.sh, 128, 1) ||
      !make_map_strided(&mo, o.p, HD, o.heads, o.sh, o.T, o.st, o_tma ? std::min(G, 32) : 1,
                        o_tma ? std::max(1, 32 / G) : 1, 32))
    return cuda_fail(cudaErrorInvalidValue);

  const long long cap = varlen_fwd_cap(B, q.heads, H_kv, q.T);
  const bool direct = varlen_fwd_direct(B, q.heads, H_kv, q.T);
  const int pieces = varlen_fwd_pieces(B, q.heads, H_kv, q.T, k.T, causal);
  auto* plan = direct ? nullptr : static_cast<fa::VarPlan*>(ws);
  auto* list = reinterpret_cast<fa::VarUnit*>(plan + 1);
  if (!direct) {
    fa::varlen_plan_kernel<<<1, fa::kPlanThreads, 0, stream>>>(cu_q, cu_kv, plan, list, B, q.T, k.T, tp, causal);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e);
  }

  fa::VarParams p;
  p.O = static_cast<__nv_bfloat16*>(const_cast<void*>(o.p));
  p.LSE = LSE;
  p.cu_q = cu_q;
  p.cu_kv = cu_kv;
  p.B = B;
  p.T_kv = k.T;
  p.plan = plan;
  p.list = list;
  p.Op = pieces ? static_cast<float*>(ws) : nullptr;
  p.Lp = pieces ? p.Op + static_cast<size_t>(pieces) * 2 * 256 * HD : nullptr;
  p.cut = pieces ? reinterpret_cast<fa::VarCut*>(p.Lp + static_cast<size_t>(pieces) * 2 * 256) : nullptr;
  p.o_st = o.st;
  p.o_sh = o.sh;
  p.T_q = q.T;
  p.group = head_group(H_kv, 4.0 * HD * k.T);
  p.H_kv = H_kv;
  p.G = G;
  p.tp = tp;
  p.inv_g = (65536 + G - 1) / G;
  p.causal = causal;
  p.o_tma = o_tma ? 1 : 0;
  p.scale_log2 = masked_scale_log2(scale);
  p.idesc_qk = C::kIdescQK | (scale < 0.f ? fa::ptx::kIdescNegateA : 0u);
  p.timeout_ns = timeout_ns;
  p.drop_load = drop_load;
  // Behind a plan, a programmatic dependent launch: the grid sets up while the
  // list is made and waits for it on the device.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pieces ? pieces : std::min<long long>(cap * H_kv, sm_count(dev))));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = direct ? 0 : 1;
  e = cudaLaunchKernelEx(&cfg, fa::fa_varlen_fwd_kernel<HD>, mq, mk, mv, mo, p);
  if (e != cudaSuccess) return cuda_fail(e);
  if (pieces > 1) {   // the merge, as a programmatic dependent too
    cfg.gridDim = dim3(static_cast<unsigned>(pieces - 1), HD / 8);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fa::varlen_merge_kernel<HD>, p);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return FA_OK;
}

fa_status_t varlen_fwd_impl(const void* Q, const void* K, const void* V, void* O, float* LSE, const int* cu_q,
                            const int* cu_kv, int B, int H, int H_kv, int T_q, int T_kv, int d,
                            const fa_strides_t* str, float scale, int causal, void* workspace,
                            size_t workspace_bytes, int drop_load, unsigned long long timeout_ns,
                            cudaStream_t stream) {
  if (!Q || !K || !V || !O || !LSE || !cu_q || !cu_kv) return FA_ERR_INVALID_ARG;
  const fa_status_t st = varlen_sizes(B, H, H_kv, T_q, T_kv, d, scale, causal);
  if (st != FA_OK) return st;
  Rows q, k, v, o;
  if (!make_rows(&q, Q, T_q, H, d, str) || !make_rows(&k, K, T_kv, H_kv, d, str ? str + 1 : nullptr) ||
      !make_rows(&v, V, T_kv, H_kv, d, str ? str + 2 : nullptr) ||
      !make_rows(&o, O, T_q, H, d, str ? str + 3 : nullptr) || !rows_distinct(o))
    return FA_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(LSE), static_cast<const void*>(cu_q), static_cast<const void*>(cu_kv)})
    if (reinterpret_cast<uintptr_t>(ptr) % 4 != 0) return FA_ERR_INVALID_ARG;
  if (!units_countable(varlen_fwd_cap(B, H, H_kv, T_q), H_kv)) return FA_ERR_UNSUPPORTED;
  const size_t need = varlen_fwd_ws(B, H, H_kv, T_q, T_kv, d, causal), n_lse = static_cast<size_t>(H) * T_q * 4;
  const size_t n_cu = (static_cast<size_t>(B) + 1) * 4;
  if (need > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 128 != 0 || workspace_bytes < need))
    return FA_ERR_INVALID_ARG;
  // O, LSE and the workspace are disjoint from every input and each other.
  for (const Rows* in : {&q, &k, &v})
    if (rows_overlap(o, *in) || rows_overlap(*in, LSE, n_lse) || rows_overlap(*in, workspace, need))
      return FA_ERR_INVALID_ARG;
  if (rows_overlap(o, LSE, n_lse) || rows_overlap(o, workspace, need) || overlaps(LSE, n_lse, workspace, need))
    return FA_ERR_INVALID_ARG;
  for (const int* cu : {cu_q, cu_kv})
    if (rows_overlap(o, cu, n_cu) || overlaps(LSE, n_lse, cu, n_cu) || overlaps(workspace, need, cu, n_cu))
      return FA_ERR_INVALID_ARG;
  if (d == 64)
    return varlen_fwd_launch<64>(q, k, v, o, LSE, cu_q, cu_kv, B, scale, causal, workspace, drop_load, timeout_ns,
                                 stream);
  return varlen_fwd_launch<128>(q, k, v, o, LSE, cu_q, cu_kv, B, scale, causal, workspace, drop_load, timeout_ns,
                                stream);
}

// ---------------------------------------------------------------- backward
// Workspace: plan, unit list, then -LSE log2(e) and -D per tile row.
struct VarBwdLayout {
  long long tiles, units;          // upper bounds (per K/V head)
  size_t list, nlse2, ndelta, bytes;
};

VarBwdLayout varlen_bwd_layout(int B, int H, int H_kv, int T_q, int T_kv) {
  const int tp = 128 / (H / H_kv);
  auto up = [](size_t n) { return (n + 127) / 128 * 128; };
  VarBwdLayout w;
  w.tiles = T_q / tp + static_cast<long long>(B);
  w.units = w.tiles + T_kv / 128 + B;
  const size_t rows = static_cast<size_t>(H_kv) * w.tiles * 128 * 4;
  w.list = up(sizeof(fa::VarBwdPlan));
  w.nlse2 = w.list + up(static_cast<size_t>(w.units) * sizeof(fa::VarBwdUnit));
  w.ndelta = w.nlse2 + rows;
  w.bytes = w.ndelta + rows;
  return w;
}

template <int HD>
fa_status_t varlen_bwd_launch(const Rows& q, const Rows& k, const Rows& v, const Rows& o, const Rows& go,
                              const float* LSE, const Rows& dq, const Rows& dk, const Rows& dv, const int* cu_q,
                              const int* cu_kv, int B, float scale, int causal, const VarBwdLayout& w, void* workspace,
                              int drop_load, unsigned long long timeout_ns, cudaStream_t stream) {
  using C = fa::BwdCfg<HD>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  constexpr int kSmem = fa::DqCfg<HD>::kSmemBytes > C::kSmemBytes ? fa::DqCfg<HD>::kSmemBytes : C::kSmemBytes;
  std::call_once(once[dev], [&] {
    attr_err[dev] =
        cudaFuncSetAttribute(fa::fa_varlen_bwd_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (attr_err[dev] != cudaSuccess) return cuda_fail(attr_err[dev]);

  const int H_kv = k.heads, G = q.heads / k.heads, tp = 128 / G;
  CUtensorMap mq, mk, mv, mdo;
  if (!make_map_strided(&mq, q.p, HD, q.heads, q.sh, q.T, q.st, G, tp) ||
      !make_map_strided(&mdo, go.p, HD, go.heads, go.sh, go.T, go.st, G, tp) ||
      !make_map_strided(&mk, k.p, HD, k.T, k.st, k.heads, k.sh, 128, 1) ||
      !make_map_strided(&mv, v.p, HD, v.T, v.st, v.heads, v.sh, 128, 1))
    return cuda_fail(cudaErrorInvalidValue);

  char* ws = static_cast<char*>(workspace);
  auto* plan = reinterpret_cast<fa::VarBwdPlan*>(ws);
  auto* list = reinterpret_cast<fa::VarBwdUnit*>(ws + w.list);
  auto* nlse2 = reinterpret_cast<float*>(ws + w.nlse2);
  auto* ndelta = reinterpret_cast<float*>(ws + w.ndelta);
  fa::varlen_bwd_prepare_kernel<HD>
      <<<dim3(static_cast<unsigned>(1 + w.tiles), static_cast<unsigned>(H_kv)), fa::kPlanThreads, 0, stream>>>(
          static_cast<const __nv_bfloat16*>(o.p), static_cast<const __nv_bfloat16*>(go.p), LSE, cu_q, cu_kv, plan, list,
          nlse2, ndelta, o.st, o.sh, go.st, go.sh, B, q.T, k.T, tp, causal, static_cast<int>(w.tiles), G);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);

  fa::VarBwdParams p;
  p.dQ = static_cast<__nv_bfloat16*>(const_cast<void*>(dq.p));
  p.dK = static_cast<__nv_bfloat16*>(const_cast<void*>(dk.p));
  p.dV = static_cast<__nv_bfloat16*>(const_cast<void*>(dv.p));
  p.dq_st = dq.st;
  p.dq_sh = dq.sh;
  p.dk_st = dk.st;
  p.dk_sh = dk.sh;
  p.dv_st = dv.st;
  p.dv_sh = dv.sh;
  p.plan = plan;
  p.list = list;
  p.nlse2 = nlse2;
  p.ndelta = ndelta;
  p.tile_cap = static_cast<int>(w.tiles);
  p.H_kv = H_kv;
  p.group = head_group(H_kv, 4.0 * HD * (k.T + static_cast<double>(G) * q.T));
  p.G = G;
  p.tp = tp;
  p.inv_g = (65536 + G - 1) / G;
  p.causal = causal;
  p.scale_log2 = masked_scale_log2(scale);
  p.scale = scale;
  p.idesc_s = C::kIdescS | (scale < 0.f ? fa::ptx::kIdescNegateA : 0u);
  p.timeout_ns = timeout_ns;
  p.drop_load = drop_load;
  // A programmatic dependent launch: it sets up beside the last of the launch before.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(w.units * H_kv, sm_count(dev))));
  cfg.blockDim = dim3(fa::kVarBwdThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fa::fa_varlen_bwd_kernel<HD>, mq, mk, mv, mdo, p);
  if (e != cudaSuccess) return cuda_fail(e);
  return FA_OK;
}

fa_status_t varlen_bwd_impl(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                            const float* LSE, void* dQ, void* dK, void* dV, const int* cu_q, const int* cu_kv, int B,
                            int H, int H_kv, int T_q, int T_kv, int d, const fa_strides_t* str, float scale,
                            int causal, void* workspace, size_t workspace_bytes, int drop_load,
                            unsigned long long timeout_ns, cudaStream_t stream) {
  if (!Q || !K || !V || !O || !dO || !LSE || !dQ || !dK || !dV || !cu_q || !cu_kv) return FA_ERR_INVALID_ARG;
  const fa_status_t st = varlen_sizes(B, H, H_kv, T_q, T_kv, d, scale, causal);
  if (st != FA_OK) return st;
  Rows in[5], out[3];   // Q K V O dO, dQ dK dV
  const void* ptr[8] = {Q, K, V, O, dO, dQ, dK, dV};
  const bool keys[8] = {false, true, true, false, false, false, true, true};
  for (int a = 0; a < 8; ++a) {
    Rows* r = a < 5 ? &in[a] : &out[a - 5];
    if (!make_rows(r, ptr[a], keys[a] ? T_kv : T_q, keys[a] ? H_kv : H, d, str ? str + a : nullptr))
      return FA_ERR_INVALID_ARG;
    if (a >= 5 && !rows_distinct(*r)) return FA_ERR_INVALID_ARG;
  }
  for (const void* a : {static_cast<const void*>(LSE), static_cast<const void*>(cu_q), static_cast<const void*>(cu_kv)})
    if (reinterpret_cast<uintptr_t>(a) % 4 != 0) return FA_ERR_INVALID_ARG;
  const VarBwdLayout w = varlen_bwd_layout(B, H, H_kv, T_q, T_kv);
  if (!units_countable(w.units, H_kv)) return FA_ERR_UNSUPPORTED;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 128 != 0 || workspace_bytes < w.bytes)
    return FA_ERR_INVALID_ARG;
  // dQ, dK, dV and the workspace are disjoint from every input and each other.
  const size_t n_lse = static_cast<size_t>(H) * T_q * 4, n_cu = (static_cast<size_t>(B) + 1) * 4;
  for (int a = 0; a < 3; ++a) {
    for (const Rows& r : in)
      if (rows_overlap(out[a], r)) return FA_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (rows_overlap(out[a], out[b])) return FA_ERR_INVALID_ARG;
    if (rows_overlap(out[a], LSE, n_lse) || rows_overlap(out[a], cu_q, n_cu) || rows_overlap(out[a], cu_kv, n_cu) ||
        rows_overlap(out[a], workspace, w.bytes))
      return FA_ERR_INVALID_ARG;
  }
  for (const Rows& r : in)
    if (rows_overlap(r, workspace, w.bytes)) return FA_ERR_INVALID_ARG;
  if (overlaps(workspace, w.bytes, LSE, n_lse) || overlaps(workspace, w.bytes, cu_q, n_cu) ||
      overlaps(workspace, w.bytes, cu_kv, n_cu))
    return FA_ERR_INVALID_ARG;
  if (d == 64)
    return varlen_bwd_launch<64>(in[0], in[1], in[2], in[3], in[4], LSE, out[0], out[1], out[2], cu_q, cu_kv, B, scale,
                                 causal, w, workspace, drop_load, timeout_ns, stream);
  return varlen_bwd_launch<128>(in[0], in[1], in[2], in[3], in[4], LSE, out[0], out[1], out[2], cu_q, cu_kv, B, scale,
                                causal, w, workspace, drop_load, timeout_ns, stream);
}

}  // namespace

extern "C" {

size_t fa_fwd_varlen_workspace_bytes(int B, int H, int H_kv, int T_q, int T_kv, int d) {
  if (varlen_sizes(B, H, H_kv, T_q, T_kv, d, 1.f, 0) != FA_OK) return 0;
  if (!units_countable(varlen_fwd_cap(B, H, H_kv, T_q), H_kv)) return 0;
  return std::max(varlen_fwd_ws(B, H, H_kv, T_q, T_kv, d, 0), varlen_fwd_ws(B, H, H_kv, T_q, T_kv, d, 1));
}

fa_status_t fa_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* LSE, const int* cu_q,
                          const int* cu_kv, int B, int H, int H_kv, int T_q, int T_kv, int d,
                          const fa_strides_t* strides, float scale, int causal, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  return varlen_fwd_impl(Q, K, V, O, LSE, cu_q, cu_kv, B, H, H_kv, T_q, T_kv, d, strides, scale, causal, workspace,
                         workspace_bytes, -1, kDefaultTimeoutNs, stream);
}

fa_status_t fa_fwd_varlen_fault_test(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                     const int* cu_q, const int* cu_kv, int B, int H, int H_kv, int T_q, int T_kv,
                                     int d, float scale, int causal, void* workspace, size_t workspace_bytes,
                                     int drop_load, unsigned long long timeout_ns, cudaStream_t stream) {
  if (timeout_ns == 0) return FA_ERR_INVALID_ARG;
  return varlen_fwd_impl(Q, K, V, O, LSE, cu_q, cu_kv, B, H, H_kv, T_q, T_kv, d, nullptr, scale, causal, workspace, workspace_bytes, drop_load < 0 ? -1 : drop_load, timeout_ns,
                         stream);
}

size_t fa_bwd_varlen_workspace_bytes(int B, int H, int H_kv, int T_q, int T_kv) {
  if (varlen_sizes(B, H, H_kv, T_q, T_kv, 64, 1.f, 0) != FA_OK) return 0;   // (the same for every d)
  const VarBwdLayout w = varlen_bwd_layout(B, H, H_kv, T_q, T_kv);
  return units_countable(w.units, H_kv) ? w.bytes : 0;
}

fa_status_t fa_bwd_varlen(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                          const float* LSE, void* dQ, void* dK, void* dV, const int* cu_q, const int* cu_kv, int B,
                          int H, int H_kv, int T_q, int T_kv, int d, const fa_strides_t* strides, float scale,
                          int causal, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return varlen_bwd_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_q, cu_kv, B, H, H_kv, T_q, T_kv, d, strides, scale,
                         causal, workspace, workspace_bytes, -1, kDefaultTimeoutNs, stream);
}

fa_status_t fa_bwd_varlen_fault_test(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                     const float* LSE, void* dQ, void* dK, void* dV, const int* cu_q,
                                     const int* cu_kv, int B, int H, int H_kv, int T_q, int T_kv, int d, float scale,
                                     int causal, void* workspace, size_t workspace_bytes, int drop_load,
                                     unsigned long long timeout_ns, cudaStream_t stream) {
  if (timeout_ns == 0) return FA_ERR_INVALID_ARG;
  return varlen_bwd_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_q, cu_kv, B, H, H_kv, T_q, T_kv, d, nullptr, scale,
                         causal, workspace, workspace_bytes, drop_load < 0 ? -1 : drop_load, timeout_ns, stream);
}

}  // extern "C"
