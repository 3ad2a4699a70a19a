"""fa_kv_append against the float64 oracle, through the C ABI (needs a GB300).

Tolerances: a value is written as e4m3 of x / scale, off by half a step: 2^-4
of itself, or 2^-10 where it is subnormal. Values that are not rotated are
exact in float32, so their codes have to be the oracle's. A rotated key is off
by 2^-21 (|a| + |b|) before that (see test_gpu_rope). Scales are powers of two:
equal, unless the largest value lies within that error of where they change.
"""
import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_34_gb300 import fa
from tests import parity
from tests.test_gpu_rope import check_rows
from tests.test_gpu_varlen import draw, ok

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(int)


class Cache:
    """Pages with random codes and scales, and a table that gives each sequence pages in random order."""

    def __init__(self, seed, lens, H_kv, page, d, by_token=False, spare=3, extra=2, one_buffer=False):
        g = torch.Generator().manual_seed(seed)
        used = [-(-n // page) for n in lens]
        n = sum(used) + spare
        perm = torch.randperm(n, generator=g).tolist()
        self.table = np.full((len(lens), max(used + [1]) + extra), -1)
        for b, u in enumerate(used):
            self.table[b, :u] = [perm.pop() for _ in range(u)]
        self.page, self.lens, self.n = page, np.asarray(lens), n

        def pages(which):
            c = (torch.randn(n, H_kv, page, d, generator=g) * 60).clamp(-448, 448).to(E4M3).cuda()
            return c.transpose(1, 2).contiguous().transpose(1, 2) if by_token else c

        self.k, self.v = pages(0), pages(1)
        if one_buffer:      # [num_pages, 2, ...]
            both = torch.stack([self.k.view(torch.uint8), self.v.view(torch.uint8)], 1).view(E4M3)
            self.k, self.v = both[:, 0], both[:, 1]
        self.ks, self.vs = (torch.exp2(torch.randint(-9, -5, (n, H_kv), generator=g).float()).cuda() for _ in range(2))

    def device(self):
        return self.k, self.v, self.ks, self.vs, i32(self.table), i32(self.lens)

    def host(self):
        return [parity.to64(x) for x in (self.k, self.ks, self.v, self.vs)]


def check_pages(got, before, x, sizes, cu, cache):
    """got, before: (codes, scale); x: what was to be written, float64; sizes: what its error is 2^-21 of, or None (exact)."""
    codes, scale = got
    want, ws = oracle.append_pages(x, cu, *before, cache.table, cache.lens, cache.page)
    if sizes is None:
        assert np.array_equal(scale, ws)
        assert np.array_equal(codes, want, equal_nan=True)
        return
    raw, _ = oracle.append_pages(x, cu, *before, cache.table, cache.lens, cache.page, exact=True)
    size, unit = oracle.append_pages(sizes, cu, np.zeros_like(want), np.zeros_like(ws), cache.table, cache.lens, cache.page,
                                     exact=True)
    size = size * unit[..., None, None]
    for i, h in zip(*np.nonzero(scale != ws)):      # the largest value within its error of where the scale changes
        least = min(scale[i, h], ws[i, h])
        assert max(scale[i, h], ws[i, h]) == 2 * least
        assert abs(np.abs(raw[i, h]).max() * ws[i, h] / (448 * least) - 1) <= 2.0 ** -18
    f = (ws / scale)[..., None, None]
    tol = np.maximum(2.0 ** -4 * np.abs(raw * f), 2.0 ** -10) + 2.0 ** -21 * size / scale[..., None, None]
    assert (np.abs(codes - raw * f) <= tol * (1 + 2.0 ** -10)).all()


def check(cache, new, H, H_kv, d, rot=0, interleaved=False, seed=0, factor=1.0, base=1e4, positions=None, T_extra=0, **kw):
    cu = offsets(new)
    T = int(cu[-1]) + T_extra
    k, v, q = draw(seed, (max(T, 1), H_kv, d), (max(T, 1), H_kv, d), (max(T, 1), H, d))
    before = cache.host()
    f = fa.fa_rope_frequencies(rot, base, device="cuda") if rot else None
    q_out = torch.full_like(q, 5.0).cuda() if rot else None
    got = fa.fa_kv_append(k.cuda(), v.cuda(), i32(cu), *cache.device(), q=q.cuda(), q_out=q_out, inv_freq=f,
                          interleaved=interleaved, factor=factor, positions=None if positions is None else i32(positions), **kw)
    ok()
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(cache.lens, new)] + [np.zeros(T_extra)]) if positions is None \
        else np.asarray(positions)
    after = cache.host()
    K, V = parity.to64(k), parity.to64(v)
    if rot:
        n = int(cu[-1])
        check_rows(got[:n], q[:n], pos[:n], f, factor, interleaved=interleaved)
        assert (got[n:] == 5.0).all()
        size = np.abs(K)
        h = rot // 2
        a = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
        size[..., a[0]] = size[..., a[1]] = abs(factor) * (size[..., a[0]] + size[..., a[1]])
        size[..., rot:] = 0
        K = oracle.rotate(K, pos, f.cpu().numpy(), interleaved, factor=factor)
        check_pages(after[:2], before[:2], K, size, cu, cache)
    else:
        check_pages(after[:2], before[:2], K, None, cu, cache)
    check_pages(after[2:], before[2:], V, None, cu, cache)


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_prompts_and_tokens(page, d, by_token):
    """Fresh sequences, pieces that begin and end inside pages or at their borders, single tokens, nothing."""
    lens = [1, page, page + 1, 3 * page - 1, 2 * page + 7, 5, 0, 4 * page, 2 * page, page]
    new = [1, page, page + 1, 2 * page, 3, 0, 0, 1, page + 2, page - 1]
    check(Cache(page + d, lens, 2, page, d, by_token), new, 4, 2, d, rot=d, seed=page)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (64, 48), (64, 0)])
def test_rotated_parts(d, rot, interleaved):
    check(Cache(rot, [70, 3, 40], 3, 32, d), [33, 3, 1], 6, 3, d, rot=rot, interleaved=interleaved, factor=1.2, base=5e5)


@pytest.mark.parametrize("B,H,H_kv", [(1, 1, 1), (1, 32, 8), (64, 32, 8), (300, 4, 2)])
def test_decode_steps(B, H, H_kv):
    r = np.random.default_rng(B)
    check(Cache(B, r.integers(1, 500, B), H_kv, 64, 128), [1] * B, H, H_kv, 128, rot=128)


def test_many_steps_equal_what_the_formulas_say():
    """Token after token into the same pages: scales only grow within a page, older rows follow."""
    page, d, H = 16, 64, 2
    cache = Cache(1, [40], H, page, d)
    cache.lens = np.array([0])
    r = np.random.default_rng(2)
    for step in range(40):
        cache.lens = cache.lens + 1
        k, v = (torch.from_numpy(r.standard_normal((1, H, d)) * 2.0 ** r.integers(-12, 6)).to(torch.bfloat16) for _ in range(2))
        before = cache.host()
        fa.fa_kv_append(k.cuda(), v.cuda(), i32([0, 1]), *cache.device())
        ok()
        after = cache.host()
        check_pages(after[:2], before[:2], parity.to64(k), None, [0, 1], cache)
        check_pages(after[2:], before[2:], parity.to64(v), None, [0, 1], cache)


def test_given_positions():
    cache = Cache(9, [20, 33], 2, 16, 64)
    check(cache, [4, 3], 4, 2, 64, rot=64, positions=[1000000, 7, -3, 0, 5, 5, 2 ** 30])


def test_rows_of_no_sequence_are_left_alone():
    check(Cache(10, [20, 33], 2, 16, 64), [4, 3], 4, 2, 64, rot=64, T_extra=5)
    check(Cache(11, [20, 33], 2, 16, 128), [0, 0], 4, 2, 128, rot=64, T_extra=2)


def test_long_prompts():
    """More pages than tokens per CTA, several sequences."""
    check(Cache(12, [3000, 1, 2500], 2, 32, 128), [3000, 1, 1777], 4, 2, 128, rot=128)


def test_one_buffer_for_keys_and_values():
    check(Cache(13, [70, 5], 2, 32, 128, one_buffer=True), [20, 5], 4, 2, 128, rot=128)


@pytest.mark.parametrize("old", [0.3, 0.0, 1e30])
def test_scales_that_other_code_left(old):
    """Not a power of two, zero, far too large."""
    cache = Cache(14, [20, 33], 2, 16, 64)
    cache.ks.fill_(old)
    cache.vs.fill_(old)
    before = cache.host()
    k, v = draw(3, (4, 2, 64), (4, 2, 64))
    cu = [0, 2, 4]
    fa.fa_kv_append(k.cuda(), v.cuda(), i32(cu), *cache.device())
    ok()
    after = cache.host()
    for got, was, x in ((after[:2], before[:2], k), (after[2:], before[2:], v)):
        want, ws = oracle.append_pages(parity.to64(x), cu, *was, cache.table, cache.lens, 16)
        assert np.array_equal(got[1], ws)
        # float32's quotient by another scale may fall on the other side of a tie
        assert (np.abs(got[0] - want) <= np.maximum(2.0 ** -3 * np.abs(want), 2.0 ** -9)).all()
        assert (got[0] != want).mean() < 1e-3


@pytest.mark.parametrize("size", [0.0, 1e-38, 1e-30, 3e38])
def test_smallest_and_largest_values(size):
    cache = Cache(15, [20], 1, 16, 64)
    k = (draw(4, (20, 1, 64))[0].float().clamp(-1, 1) * size).to(torch.bfloat16)
    before = cache.host()
    fa.fa_kv_append(k.cuda(), k.cuda(), i32([0, 20]), *cache.device())
    ok()
    after = cache.host()
    check_pages(after[:2], before[:2], parity.to64(k), None, [0, 20], cache)


def test_values_that_are_not_finite():
    cache = Cache(16, [20, 40], 2, 16, 64)
    k, v = draw(5, (30, 2, 64), (30, 2, 64))
    v[3, 0, 5], v[4, 1, 7], v[29, 1, 0], v[7] = float("inf"), float("-inf"), float("nan"), float("nan")
    before = cache.host()
    fa.fa_kv_append(k.cuda(), v.cuda(), i32([0, 20, 30]), *cache.device())
    ok()
    after = cache.host()
    check_pages(after[2:], before[2:], parity.to64(v), None, [0, 20, 30], cache)
    assert np.isnan(after[2]).any()


def test_strided_inputs_and_in_place_queries():
    T, H, Hk, d = 30, 4, 2, 128
    a, b = Cache(17, [20, 40], Hk, 16, d), Cache(17, [20, 40], Hk, 16, d)
    qkv, = draw(6, (T, H + 2 * Hk, d))
    f = fa.fa_rope_frequencies(d, device="cuda")
    buf, cu = qkv.cuda(), i32([0, 20, 30])
    q, k, v = buf[:, :H], buf[:, H:H + Hk], buf[:, H + Hk:]
    want = fa.fa_kv_append(k.contiguous(), v.contiguous(), cu, *a.device(), q=q.contiguous(), inv_freq=f)
    got = fa.fa_kv_append(k, v, cu, *b.device(), q=q, q_out=q, inv_freq=f)
    ok()
    assert got is q and torch.equal(q, want) and torch.equal(buf[:, H:].cpu(), qkv[:, H:])
    for x, y in zip(a.host(), b.host()):
        assert np.array_equal(x, y, equal_nan=True)


@pytest.mark.parametrize("cu,lens", [([0, 5, 3], [30, 30]), ([0, -1, 3], [30, 30]), ([0, 4, 99], [30, 30]), ([0, 4, 8], [30, 3]),
                                     ([0, 4, 8], [30, 10 ** 6]), ([0, 4, 8], [-5, 30])])
def test_offsets_and_lengths_that_do_not_fit_are_reported(cu, lens):
    cache = Cache(18, [30, 30], 2, 16, 64)
    k, q = draw(7, (8, 2, 64), (8, 4, 64))
    before = cache.host()
    cache.lens = np.array(lens)
    fa.fa_kv_append(k.cuda(), k.cuda(), i32(cu), *cache.device(), q=q.cuda(), inv_freq=fa.fa_rope_frequencies(64, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()
    # a sequence that fits was written, the other was not
    good = [b for b in range(2) if 0 <= cu[b] <= cu[b + 1] <= 8 and cu[b + 1] - cu[b] <= lens[b] <= 64]
    touched = {int(i) for b in good for i in cache.table[b] if i >= 0}
    after = cache.host()
    for x, y in zip(before, after):
        for i in range(cache.n):
            assert i in touched or np.array_equal(x[i], y[i], equal_nan=True)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("cu,lens", [([0, 60, 20, 80], [70, 30, 64]), ([0, 6, 2, 8, 8], [6, 30, 77, 9]), ([0, 300, 10, 310], [300, 1, 301])])
def test_offsets_that_decrease_in_between(cu, lens, page):
    """Rows that two sequences claim: one of them gets each, whole, and nobody else's pages change."""
    cache = Cache(23, lens, 2, page, 64)
    k, = draw(12, (cu[-1], 2, 64))
    before = cache.host()
    for _ in range(5):
        fa.fa_kv_append(k.cuda(), k.cuda(), i32(cu), *cache.device(), q=k.cuda(), inv_freq=fa.fa_rope_frequencies(64, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()
    fit = [b for b in range(len(lens)) if cu[b] <= cu[b + 1]]
    mine = {int(i) for b in fit for i in cache.table[b] if i >= 0}
    for x, y in zip(before, cache.host()):
        for i in set(range(cache.n)) - mine:
            assert np.array_equal(x[i], y[i], equal_nan=True)


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_pages_that_do_not_exist_are_left_out_and_reported(bad):
    cache = Cache(19, [30, 30], 2, 16, 64)
    cache.table[0, 1] = bad
    k, = draw(8, (16, 2, 64))
    before = cache.host()
    fa.fa_kv_append(k.cuda(), k.cuda(), i32([0, 8, 16]), *cache.device())
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()
    after = cache.host()
    i = int(cache.table[0, 0])
    assert np.array_equal(before[0][i], after[0][i])
    j = int(cache.table[1, 1])
    assert not np.array_equal(before[0][j], after[0][j])


def test_side_stream():
    caches = [Cache(24, [400, 90], 2, 32, 128) for _ in range(2)]
    k, v, q = (t.cuda() for t in draw(13, (301, 2, 128), (301, 2, 128), (301, 4, 128)))
    f, cu = fa.fa_rope_frequencies(128, device="cuda"), i32([0, 300, 301])
    side, dev = torch.cuda.Stream(), [c.device() for c in caches]
    torch.cuda.synchronize()
    got = fa.fa_kv_append(k, v, cu, *dev[0], q=q, inv_freq=f, stream=side)
    side.synchronize()
    want = fa.fa_kv_append(k, v, cu, *dev[1], q=q, inv_freq=f)
    ok()
    assert torch.equal(got, want)
    for x, y in zip(*(c.host() for c in caches)):
        assert np.array_equal(x, y, equal_nan=True)


def test_one_page():
    """A cache of a single page and head, of every size."""
    for page in (16, 32, 64, 128):
        for d in (64, 128):
            cache = Cache(25, [page], 1, page, d, spare=0, extra=0)
            check(cache, [page // 2 + 1], 1, 1, d, rot=d)


def test_graph_replay_with_other_lengths():
    """One captured step, replayed for every token of a growing answer."""
    d, page = 64, 16
    cache, plain = Cache(20, [40, 25], 2, page, d), Cache(20, [40, 25], 2, page, d)
    f = fa.fa_rope_frequencies(d, device="cuda")
    k, v, q = (t.cuda() for t in draw(9, (2, 2, d), (2, 2, d), (2, 4, d)))
    cu = i32([0, 1, 2])
    dev = cache.device()
    lens = dev[-1]
    lens.copy_(i32([8, 16]))
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fa.fa_kv_append(k, v, cu, *dev, q=q, q_out=out, inv_freq=f)
    for step in range(9):
        k.mul_(1.5)
        lens += 1
        plain.lens = np.array([9 + step, 17 + step])
        graph.replay()
        want = fa.fa_kv_append(k, v, cu, *plain.device(), q=q, inv_freq=f)
        ok()
        assert torch.equal(out, want)
        for x, y in zip(cache.host(), plain.host()):
            assert np.array_equal(x, y, equal_nan=True)


def test_beyond_32_bit_offsets():
    """Pages more than 2^31 bytes apart."""
    H, page, d = 2, 128, 128
    n = (1 << 31) // (H * page * d) + 40
    cache = Cache(21, [200], H, page, d, spare=0)
    codes = torch.zeros(n, H, page, d, dtype=torch.uint8, device="cuda")
    small, ids = cache, [n - 1, 3]
    for pages in ("k", "v"):
        big = codes.clone().view(E4M3)
        for i in range(2):
            big.view(torch.uint8)[ids[i]] = getattr(small, pages)[int(small.table[0, i])].view(torch.uint8)
        setattr(small, pages + "b", big)
    scale = [torch.ones(n, H, device="cuda") for _ in range(2)]
    for s, t in zip(scale, (small.ks, small.vs)):
        for i in range(2):
            s[ids[i]] = t[int(small.table[0, i])]
    k, v = draw(10, (150, H, d), (150, H, d))
    fa.fa_kv_append(k.cuda(), v.cuda(), i32([0, 150]), small.kb, small.vb, *scale, i32([ids]), i32([200]))
    fa.fa_kv_append(k.cuda(), v.cuda(), i32([0, 150]), *small.device())
    ok()
    for big, s, a, t in ((small.kb, scale[0], small.k, small.ks), (small.vb, scale[1], small.v, small.vs)):
        for i in range(2):
            j = int(small.table[0, i])
            assert torch.equal(big.view(torch.uint8)[ids[i]], a.view(torch.uint8)[j]) and torch.equal(s[ids[i]], t[j])


def test_binding_refusals():
    c = Cache(22, [20], 2, 16, 64)
    k, q = (t.cuda() for t in draw(11, (4, 2, 64), (4, 4, 64)))
    f = fa.fa_rope_frequencies(64, device="cuda")
    kc, vc, ks, vs, table, lens = c.device()
    good = dict(k=k, v=k, cu_new=i32([0, 4]), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=table, seq_lens=lens)
    for bad in (dict(k=k.float()), dict(v=k[:3]), dict(cu_new=i32([4])), dict(cu_new=i32([0, 4]).long()), dict(k_cache=kc.float()),
                dict(v_cache=vc[:, :1]), dict(k_cache=kc[..., :32], v_cache=vc[..., :32]), dict(k_scale=ks.double()),
                dict(v_scale=vs[:1]), dict(page_table=table[0]), dict(page_table=table.long()), dict(seq_lens=i32([1, 2])),
                dict(q=q, q_out=q), dict(q_out=q, inv_freq=f), dict(q=q[:2], inv_freq=f), dict(inv_freq=f.float()),
                dict(positions=i32([0]))):
        with pytest.raises(ValueError):
            fa.fa_kv_append(**{**good, **bad})
    with pytest.raises(fa.FaError):
        fa.fa_kv_append(**{**good, "v_cache": kc})
    assert fa.fa_kv_append(**good, q=q) is q       # nothing to rotate by
    ok()
