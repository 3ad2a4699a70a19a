// Entry points for a batch that shares a prefix (declared in include/fa.h).
// Part of fa_api.cu, whose helpers it uses.
#pragma once

namespace {

// A tensor [B, heads, N, d] with element strides for B, heads and N (d contiguous).
struct Cube {
  const void* p;
  long long n[3], s[3];           // sizes and strides, batch first
  int d;

  long long span() const {        // bytes from the first element to behind the last
    long long e = d;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * s[i];
    return e * 2;
  }
};

// As make_rows, for four dimensions.
bool make_cube(Cube* c, const void* p, int B, int heads, int N, int d, const fa_batch_strides_t* s) {
  *c = Cube{p, {B, heads, N}, {0, 0, 0}, d};
  const long long dense[3] = {static_cast<long long>(heads) * N * d, static_cast<long long>(N) * d, d};
  const long long given[3] = {s ? s->batch : 0, s ? s->head : 0, s ? s->row : 0};
  for (int i = 0; i < 3; ++i) {
    c->s[i] = s && c->n[i] > 1 ? given[i] : dense[i];
    if (c->n[i] > 1 && (c->s[i] <= 0 || c->s[i] % 8 != 0 || c->s[i] >= (1LL << 36))) return false;
    if (c->n[i] == 1) c->s[i] = d;
  }
  return reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// No two elements of a written tensor share an address: taken from the
// smallest stride to the largest, each steps over all that lies inside it.
bool cube_distinct(const Cube& c) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return c.s[a] < c.s[b]; });
  long long inside = c.d;
  for (int i : order) {
    if (c.n[i] == 1) continue;
    if (c.s[i] < inside) return false;
    inside += (c.n[i] - 1) * c.s[i];
  }
  return true;
}

bool make_map4(CUtensorMap* m, const Cube& c, int b_row, int b_head, int b_batch) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.n[2]),
                        static_cast<cuuint64_t>(c.n[1]), static_cast<cuuint64_t>(c.n[0])};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.s[2]) * 2, static_cast<cuuint64_t>(c.s[1]) * 2,
                           static_cast<cuuint64_t>(c.s[0]) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b_row), static_cast<cuuint32_t>(b_head),
                       static_cast<cuuint32_t>(b_batch)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(c.p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Places of the line at most, and whether they can be counted in 32 bits on the device.
long long pre_places(const fa::PreShape& s) {
  return static_cast<long long>(s.p_units) * (s.p_blocks + fa::kUnitCost) +
         static_cast<long long>(s.B) * s.H_kv * s.ht * ((s.room + 127LL) / 128 + fa::kUnitCost);
}
bool places_countable(const fa::PreShape& s) { return pre_places(s) < (1LL << 31) - 65536; }

fa::PreShape pre_shape(int B, int H, int H_kv, int N_q, int n_p, int room) {
  fa::PreShape s;
  s.B = B;
  s.H = H;
  s.H_kv = H_kv;
  s.G = H / H_kv;
  s.N_q = N_q;
  s.n_p = n_p;
  s.room = room;
  s.hp = std::min(s.G, 128 / N_q);
  s.ht = (s.G + s.hp - 1) / s.hp;
  s.bp = s.ht == 1 ? 128 / (s.hp * N_q) : 1;
  s.bt = (B + s.bp - 1) / s.bp;
  s.p_blocks = (n_p + 127) / 128;
  s.p_units = n_p > 0 ? H_kv * s.bt * s.ht : 0;
  s.ctas = static_cast<int>(std::min(pre_places(s), 2LL * device_sm_count()));
  return s;
}

struct PreLayout {
  size_t Op, Lp, Oo, Lo, bytes;   // the units' segments are at the front
};

PreLayout pre_layout(const fa::PreShape& s, int d) {
  auto up = [](size_t n) { return (n + 127) / 128 * 128; };
  const size_t p_rows = s.p_units ? (static_cast<size_t>(s.p_units) + s.ctas) * 128 : 0;
  const size_t o_rows = (static_cast<size_t>(s.B) * s.H_kv * s.ht + s.ctas) * s.hp * s.N_q;
  PreLayout w;
  w.Op = up((static_cast<size_t>(s.p_units) + static_cast<size_t>(s.B) * s.H_kv * s.ht) * sizeof(int2));
  w.Lp = w.Op + p_rows * d * 4;
  w.Oo = w.Lp + up(p_rows * 4);
  w.Lo = w.Oo + o_rows * d * 4;
  w.bytes = w.Lo + up(o_rows * 4);
  return w;
}

// Sizes fa_fwd_prefix accepts.
fa_status_t pre_sizes(int B, int H, int H_kv, int N_q, int n_p, int room, int d) {
  if (B < 1 || H < 1 || H_kv < 1 || N_q < 1 || n_p < 0 || room < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (B > 65535 || H > 65535 || H % H_kv != 0) return FA_ERR_INVALID_ARG;
  const long long lim = 1LL << 31;
  if (static_cast<long long>(B) * H * N_q >= lim || static_cast<long long>(B) * H_kv * room >= lim ||
      static_cast<long long>(H_kv) * n_p >= lim || n_p > kMaxLength || room > kMaxLength)
    return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || N_q > 128 || H / H_kv > 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

template <int HD>
fa_status_t prefix_launch(const Cube& q, const Cube& kp, const Cube& vp, const Cube& k, const Cube& v, const Cube& o,
                          const int* lens, float* LSE, const fa::PreShape& s, float scale, int causal, void* workspace,
                          int drop_load, unsigned long long timeout_ns, cudaStream_t stream) {
  using C = fa::DecCfg<HD>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  static bool regs_ok[64];
  std::call_once(once[dev], [&] {
    attr_err[dev] =
        cudaFuncSetAttribute(fa::fa_prefix_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, fa::PreCfg<HD>::kSmemBytes);
    // The warpgroups' register split must fit the registers the block is
    // launched with (see the forward launch).
    cudaFuncAttributes fattr;
    if (attr_err[dev] == cudaSuccess) attr_err[dev] = cudaFuncGetAttributes(&fattr, fa::fa_prefix_kernel<HD>);
    regs_ok[dev] = attr_err[dev] == cudaSuccess && 4 * C::kRegsSoftmax + 4 * C::kRegsControl <= 8 * fattr.numRegs;
  });
  if (attr_err[dev] != cudaSuccess) return cuda_fail(attr_err[dev]);
  if (!regs_ok[dev]) return FA_ERR_UNSUPPORTED;

  CUtensorMap mqp, mqo, mkp, mvp, mk, mv;
  if (!make_map4(&mqp, q, s.N_q, s.hp, s.bp) || !make_map4(&mqo, q, s.N_q, s.hp, 1) || !make_map4(&mkp, kp, 128, 1, 1) ||
      !make_map4(&mvp, vp, 128, 1, 1) || !make_map4(&mk, k, 128, 1, 1) || !make_map4(&mv, v, 128, 1, 1))
    return cuda_fail(cudaErrorInvalidValue);

  char* ws = static_cast<char*>(workspace);
  const PreLayout w = pre_layout(s, HD);
  fa::PreParams p;
  p.s = s;
  p.lens = lens;
  p.seg = reinterpret_cast<int2*>(ws);
  p.Op = reinterpret_cast<float*>(ws + w.Op);
  p.Lp = reinterpret_cast<float*>(ws + w.Lp);
  p.Oo = reinterpret_cast<float*>(ws + w.Oo);
  p.Lo = reinterpret_cast<float*>(ws + w.Lo);
  p.causal = causal;
  p.scale_log2 = masked_scale_log2(scale);
  p.idesc_qk = C::kIdescQK | (scale < 0.f ? fa::ptx::kIdescNegateA : 0u);
  p.timeout_ns = timeout_ns;
  p.drop_load = drop_load;
  fa::fa_prefix_kernel<HD><<<static_cast<unsigned>(s.ctas), C::kThreads, fa::PreCfg<HD>::kSmemBytes, stream>>>(mqp, mqo, mkp, mvp,
                                                                                                 mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  // The merge as a programmatic dependent launch: it waits on the device.
  const long long rows = static_cast<long long>(s.B) * s.H * s.N_q;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fa::prefix_merge_kernel<HD>, p, static_cast<__nv_bfloat16*>(const_cast<void*>(o.p)),
                         LSE, o.s[0], o.s[1], o.s[2]);
  if (e != cudaSuccess) return cuda_fail(e);
  return FA_OK;
}

fa_status_t prefix_impl(const void* Q, const void* K_prefix, const void* V_prefix, const void* K, const void* V,
                        const int* lens, void* O, float* LSE, int B, int H, int H_kv, int N_q, int n_p, int room, int d,
                        const fa_batch_strides_t* str, float scale, int causal, void* workspace,
                        size_t workspace_bytes, int drop_load, unsigned long long timeout_ns, cudaStream_t stream) {
  if (!Q || !K || !V || !lens || !O || !LSE) return FA_ERR_INVALID_ARG;
  const fa_status_t st = pre_sizes(B, H, H_kv, N_q, n_p, room, d);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (n_p > 0 && (!K_prefix || !V_prefix)) return FA_ERR_INVALID_ARG;
  Cube q, kp, vp, k, v, o;
  if (!make_cube(&q, Q, B, H, N_q, d, str) || !make_cube(&k, K, B, H_kv, room, d, str ? str + 3 : nullptr) ||
      !make_cube(&v, V, B, H_kv, room, d, str ? str + 4 : nullptr) ||
      !make_cube(&o, O, B, H, N_q, d, str ? str + 5 : nullptr) || !cube_distinct(o))
    return FA_ERR_INVALID_ARG;
  if (n_p > 0) {
    if (!make_cube(&kp, K_prefix, 1, H_kv, n_p, d, str ? str + 1 : nullptr) ||
        !make_cube(&vp, V_prefix, 1, H_kv, n_p, d, str ? str + 2 : nullptr))
      return FA_ERR_INVALID_ARG;
  } else {   // no block of the line reads them
    kp = k;
    vp = v;
  }
  for (const void* a : {static_cast<const void*>(LSE), static_cast<const void*>(lens)})
    if (reinterpret_cast<uintptr_t>(a) % 4 != 0) return FA_ERR_INVALID_ARG;
  const fa::PreShape s = pre_shape(B, H, H_kv, N_q, n_p, room);
  if (!places_countable(s)) return FA_ERR_UNSUPPORTED;
  const size_t need = pre_layout(s, d).bytes, n_lse = static_cast<size_t>(B) * H * N_q * 4;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 128 != 0 || workspace_bytes < need)
    return FA_ERR_INVALID_ARG;
  // O, LSE and the workspace are disjoint from every input and each other.
  auto clash = [&](const void* a, size_t na) {
    return overlaps(O, o.span(), a, na) || overlaps(LSE, n_lse, a, na) || overlaps(workspace, need, a, na);
  };
  for (const Cube* in : {&q, &kp, &vp, &k, &v})
    if (clash(in->p, in->span())) return FA_ERR_INVALID_ARG;
  if (clash(lens, static_cast<size_t>(B) * 4) || overlaps(O, o.span(), LSE, n_lse) ||
      overlaps(O, o.span(), workspace, need) || overlaps(LSE, n_lse, workspace, need))
    return FA_ERR_INVALID_ARG;
  if (d == 64)
    return prefix_launch<64>(q, kp, vp, k, v, o, lens, LSE, s, scale, causal, workspace, drop_load, timeout_ns, stream);
  return prefix_launch<128>(q, kp, vp, k, v, o, lens, LSE, s, scale, causal, workspace, drop_load, timeout_ns, stream);
}

}  // namespace

extern "C" {

size_t fa_fwd_prefix_workspace_bytes(int B, int H, int H_kv, int N_q, int N_prefix, int N_own, int d) {
  if (pre_sizes(B, H, H_kv, N_q, N_prefix, N_own, d) != FA_OK) return 0;
  const fa::PreShape s = pre_shape(B, H, H_kv, N_q, N_prefix, N_own);
  return places_countable(s) ? pre_layout(s, d).bytes : 0;
}

fa_status_t fa_fwd_prefix(const void* Q, const void* K_prefix, const void* V_prefix, const void* K, const void* V,
                          const int* seq_lens, void* O, float* LSE, int B, int H, int H_kv, int N_q, int N_prefix,
                          int N_own, int d, const fa_batch_strides_t* strides, float scale, int causal,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return prefix_impl(Q, K_prefix, V_prefix, K, V, seq_lens, O, LSE, B, H, H_kv, N_q, N_prefix, N_own, d, strides,
                     scale, causal, workspace, workspace_bytes, -1, kDefaultTimeoutNs, stream);
}

fa_status_t fa_fwd_prefix_fault_test(const void* Q, const void* K_prefix, const void* V_prefix, const void* K,
                                     const void* V, const int* seq_lens, void* O, float* LSE, int B, int H, int H_kv,
                                     int N_q, int N_prefix, int N_own, int d, float scale, int causal,
                                     void* workspace, size_t workspace_bytes, int drop_load,
                                     unsigned long long timeout_ns, cudaStream_t stream) {
  if (timeout_ns == 0) return FA_ERR_INVALID_ARG;
  return prefix_impl(Q, K_prefix, V_prefix, K, V, seq_lens, O, LSE, B, H, H_kv, N_q, N_prefix, N_own, d, nullptr,
                     scale, causal, workspace, workspace_bytes, drop_load < 0 ? -1 : drop_load, timeout_ns, stream);
}

}  // extern "C"
