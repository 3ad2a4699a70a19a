"""fa_fwd_paged against the float64 oracle, through the C ABI (needs a GB300).

Tolerances, from the arithmetic. With few rows a weight enters P V as two e4m3
numbers: the first four significant bits and the rest to four more, off by at
most 2^-8 of itself, or where it is small by 2^-17 of the largest product of
probability and scale among its 32 keys. With many it enters as f16: off by 2^-12 of
itself, or by 2^-31 of its row's largest. O is rounded once. So |O - ref| <=
2^-8 (A + |ref|) + 2^-17 F, with A = P |V| and F as the oracle returns them, and float32 sums and
exponentials add a few 2^-22 of A. A query element is exact as two e4m3 numbers unless it
is below 2^-9 of its row's largest, and then off by at most 2^-17 of that: a
score is off by that times the sum of |k|, and by d 2^-24 scale |q|.|k| for its
sum; the rest of LSE is float32 steps of values below 32.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_34_gb300 import fa
from tests import parity
from tests.test_gpu_append import Cache, E4M3, i32, offsets
from tests.test_gpu_varlen import check_lse, draw, lse_tol, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def check_o(o, ref, A, F):
    got = parity.to64(o)
    tol = 2.0 ** -8 * (A + np.abs(ref)) + 2.0 ** -17 * F + 1e-5 * A + 1e-30
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


def reference(cache, q, cu, scale, causal):
    k, ks, v, vs = cache.host()
    return oracle.attention_paged(parity.to64(q), k, v, ks, vs, cache.table, cache.lens, cu, scale, causal)


def score_tol(cache, q, scale):
    k, ks, _, _ = cache.host()
    keys = np.abs(k * ks[..., None, None])
    keys = keys[np.isfinite(keys).all(-1)]
    K = torch.from_numpy(keys).float()
    return lse_tol(q, K, scale) + abs(scale) * float(q.float().abs().max()) * 2.0 ** -17 * float(keys.sum(-1).max())


def check(cache, new, H, d, causal=True, scale=None, seed=0, q=None, T_extra=0, **kw):
    cu = offsets(new)
    n = int(cu[-1])
    q = draw(seed, (n + T_extra, H, d))[0] if q is None else q
    scale = 1 / math.sqrt(d) if scale is None else scale
    o, lse = fa.fa_fwd_paged(q.cuda(), *cache.device(), i32(cu), scale=scale, causal=causal, **kw)
    ok()
    O, L, A, F = reference(cache, q, cu, scale, causal)
    check_o(o[:n], O[:n], A[:n], F[:n])
    check_lse(lse[:, :n], L[:, :n], score_tol(cache, q, scale))
    return o, lse


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,H_kv", [(8, 2), (3, 3), (7, 1)])
def test_pages_and_heads(H, H_kv, page, d, by_token):
    """One token per sequence on caches of every kind of length."""
    lens = [1, page - 1, page, page + 1, 127, 128, 129, 0, 500, 257]
    check(Cache(page + H, lens, H_kv, page, d, by_token), [1] * 10, H, d, seed=page + d)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [
    ([3, 1, 0, 8, 2], [300, 1, 70, 8, 2]), ([40], [40]), ([100, 1, 129], [400, 1000, 129]), ([17, 5], [10, 3]),
    ([4, 4, 2], [0, 1, 2]), ([0, 0, 5], [9, 0, 200]),
])
def test_new_tokens(new, lens, d, causal):
    """Drafts, prompts, pieces of them; rows that see nothing; sequences without new tokens or keys."""
    check(Cache(sum(new), lens, 2, 32, d), new, 8, d, causal, seed=sum(lens))


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pieces_of_prompts(page, d, by_token):
    """Long and short pieces beside single tokens; with the last, blocks of unequal scale."""
    new, lens = [200, 1, 33, 128, 7], [900, 300, 33, 140, 2000]
    cache = Cache(page + d, lens, 2, page, d, by_token)
    check(cache, new, 8, d, seed=page)
    g = torch.Generator().manual_seed(page)
    for s in (cache.ks, cache.vs):
        s.mul_(torch.exp2(torch.rand(s.shape, generator=g) * 6 - 5).cuda())
    check(cache, new, 8, d, seed=page, scale=-0.11)


@pytest.mark.parametrize("G,n", [(1, 1), (16, 1), (17, 1), (64, 1), (65, 1), (128, 1), (100, 3), (5, 13), (3, 22), (33, 2), (1, 200)])
def test_heads_per_group(G, n):
    """Groups that fill a tile of rows, do not divide it, or need several."""
    check(Cache(G + n, [260, 17, 0, n], 2, 16, 64), [n, n, n, n], 2 * G, 64, seed=G)


@pytest.mark.parametrize("d", [64, 128])
def test_long_caches(d):
    """Many tiles for every CTA, ragged ends; the same bits from run to run."""
    cache = Cache(31 + d, [10001, 9000, 1, 7003, 10000, 33], 4, 64, d)
    a = check(cache, [1] * 6, 16, d, seed=d)
    q = draw(d, (6, 16, d))[0]
    b = fa.fa_fwd_paged(q.cuda(), *cache.device(), i32(offsets([1] * 6)))
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_sequences():
    lens = np.random.default_rng(3).integers(0, 200, 700)
    check(Cache(32, lens, 2, 16, 64), [1] * 700, 4, 64)


def test_many_sequences_with_pieces():
    """More sequences than one warp adds up, some with a piece of a prompt."""
    r = np.random.default_rng(4)
    lens, new = r.integers(0, 300, 400), np.where(r.random(400) < 0.2, r.integers(0, 90, 400), 1)
    check(Cache(38, lens, 2, 64, 64), new.tolist(), 8, 64)


@pytest.mark.parametrize("new", [1, 5, 16])
def test_one_page(new):
    """A cache of a single page and head, of every size."""
    for page in (16, 32, 64, 128):
        for d in (64, 128):
            check(Cache(39, [page], 1, page, d, spare=0, extra=0), [new], 2, d)


@pytest.mark.parametrize("rows", [1, 40])
def test_offsets_that_decrease_in_between(rows):
    """Rows that two sequences claim get one result or the other's; those of one alone get theirs."""
    lens, n = [900, 30, 500], 4 * rows
    cache = Cache(36, lens, 2, 32, 64)
    q = draw(16, (n, 4, 64))[0].cuda()
    cu = [0, 3 * rows, 2 * rows, n]
    o, lse = fa.fa_fwd_paged(q, *cache.device(), i32(cu))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()
    one = [reference(cache, q, c, 0.125, True) for c in ([0, 3 * rows, 3 * rows, 3 * rows], [2 * rows, 2 * rows, 2 * rows, n])]
    O, L, A, F = one[0]
    check_o(o[:2 * rows], O[:2 * rows], A[:2 * rows], F[:2 * rows])
    O, L, A, F = one[1]
    check_o(o[3 * rows:], O[3 * rows:], A[3 * rows:], F[3 * rows:])


@pytest.mark.parametrize("scale", [0.0, -0.09, 2.0])
def test_scales(scale):
    check(Cache(33, [200, 3, 77], 2, 32, 128), [2, 1, 30], 8, 128, scale=scale)


def test_block_scales_of_every_size():
    """Scales that differ by 2^24 from page to page, not powers of two; queries of very different size."""
    cache = Cache(34, [700, 300], 2, 16, 128)
    g = torch.Generator().manual_seed(1)
    for s in (cache.ks, cache.vs):
        s.copy_(torch.exp2(torch.rand(s.shape, generator=g) * 24 - 26))
    cache.ks.clamp_(max=0.01)
    q = draw(2, (4, 8, 128))[0]
    q[1] *= 2.0 ** -20
    q[2, 3] *= 2.0 ** 6
    check(cache, [3, 1], 8, 128, q=q)


def test_zero_scales():
    """Pages of zeros as other code may write them: codes and scale zero."""
    cache = Cache(35, [200], 2, 32, 64)
    i = int(cache.table[0, 2])
    for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
        c.view(torch.uint8)[i] = 0
        s[i] = 0.0
    o, _ = fa.fa_fwd_paged(draw(3, (1, 4, 64))[0].cuda(), *cache.device(), i32([0, 1]))
    ok()
    q = draw(3, (1, 4, 64))[0]
    cache.vs[i] = 1.0      # (the oracle's F divides by it; the page's values stay zero)
    O, L, A, F = reference(cache, q, [0, 1], 0.125, True)
    F = np.maximum(F, 0)
    check_o(o, O, A, F)


def test_large_scores():
    cache = Cache(36, [400, 390, 5], 2, 32, 128)
    cache.ks[int(cache.table[0, 3])] *= 16
    check(cache, [1, 4, 2], 8, 128, q=draw(4, (7, 8, 128))[0] * 3)


def test_equal_scores():
    """All keys alike: O is the mean of V."""
    cache = Cache(37, [1000, 129], 2, 64, 64)
    cache.k.view(torch.uint8).zero_()
    check(cache, [1, 3], 4, 64)


def test_what_stands_behind_a_length_does_not_matter():
    """NaN codes and scales, and entries of no page, behind every length."""
    cache = Cache(38, [130, 1, 64, 33], 2, 32, 128)
    q = draw(5, (7, 8, 128))[0].cuda()
    cu = i32([0, 1, 2, 6, 7])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    for b, n in enumerate(cache.lens):
        last = int(cache.table[b, (n - 1) // 32])
        if n % 32:
            for c in (cache.k, cache.v):
                c.view(torch.uint8)[last, :, n % 32:] = 0x7f
    used = {int(i) for i in cache.table.flatten() if i >= 0}
    for i in set(range(cache.n)) - used:
        for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
            c.view(torch.uint8)[i] = 0x7f
            s[i] = float("nan")
    cache.table[cache.table < 0] = 2 ** 31 - 1
    got = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_non_finite_values_within_a_length():
    """A NaN key makes the rows that see it NaN; so does a NaN value, in its column; other sequences and heads stay."""
    cache = Cache(39, [200, 150], 2, 32, 64)
    q = draw(6, (2, 4, 64))[0].cuda()
    cu = i32([0, 1, 2])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    cache.k.view(torch.uint8)[int(cache.table[0, 1]), 0, 3, 5] = 0x7f
    cache.v.view(torch.uint8)[int(cache.table[1, 2]), 1, 7, 9] = 0xff
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    assert o[0, :2].isnan().all() and lse[:2, 0].isnan().all()
    assert o[1, 2:, 9].isnan().all()
    o[0, :2], o[1, 2:, 9], lse[:2, 0] = want[0][0, :2], want[0][1, 2:, 9], want[1][:2, 0]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_non_finite_queries_stay_in_their_rows():
    cache = Cache(40, [300, 20], 2, 32, 64)
    q = draw(7, (4, 8, 64))[0].cuda()
    cu = i32([0, 3, 4])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    q[1, 2, 0], q[2, 5, 1] = float("nan"), float("inf")
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    for t, h in ((1, 2), (2, 5)):
        assert o[t, h].isnan().all() and lse[h, t].isnan()
        o[t, h], lse[h, t] = want[0][t, h], want[1][h, t]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_shared_pages():
    """Two sequences whose first pages are the same."""
    cache = Cache(41, [100, 90], 2, 32, 64)
    cache.table[1, :2] = cache.table[0, :2]
    check(cache, [1, 3], 4, 64)


def test_layouts_and_rows_of_no_sequence():
    cache = Cache(42, [130, 77], 2, 32, 128, one_buffer=True)
    q = draw(8, (9, 4, 128))[0].cuda()
    cu = i32([0, 2, 6])
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    wide = torch.full((4, 9, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    out, l2 = wide[:, :, :128].transpose(0, 1), torch.full((4, 9), 5.0, device="cuda")
    fused = torch.cat([q, q], 1)[:, 4:]
    fa.fa_fwd_paged(fused, *cache.device(), cu, o=out, lse=l2)
    ok()
    assert torch.equal(out[:6], o[:6]) and torch.equal(l2[:, :6], lse[:, :6])
    assert (l2[:, 6:] == 5.0).all()
    out[:6] = 7.0
    assert (wide == 7.0).all()
    check(cache, [2, 4], 4, 128, T_extra=3)


def test_agrees_with_the_packed_operator():
    """The same keys as bf16 through fa_fwd_varlen (powers of two as scales: exact in bf16)."""
    lens, new = [300, 77, 128], [40, 77, 1]
    cache = Cache(43, lens, 2, 64, 128)
    k, v = (torch.cat([(c.float() * s[..., None, None])[cache.table[b, :-(-n // 64)]].transpose(1, 2).flatten(0, 1)[:n]
                       for b, n in enumerate(lens)]).to(torch.bfloat16) for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)))
    q = draw(9, (sum(new), 8, 128))[0].cuda()
    o, lse = fa.fa_fwd_paged(q, *cache.device(), i32(offsets(new)))
    o2, lse2 = fa.fa_fwd_varlen(q, k.contiguous(), v.contiguous(), i32(offsets(new)), i32(offsets(lens)))
    ok()
    assert float((lse - lse2).abs().max()) < 1e-4
    assert float((o.float() - o2.float()).norm() / o2.float().norm()) < 2.0 ** -7


@pytest.mark.parametrize("cu,lens", [([0, 5, 3], [30, 30]), ([0, -1, 3], [30, 30]), ([0, 4, 99], [30, 30]),
                                     ([0, 4, 8], [30, 10 ** 6]), ([0, 4, 8], [-5, 30])])
def test_offsets_and_lengths_that_do_not_fit_are_reported(cu, lens):
    cache = Cache(44, [30, 30], 2, 16, 64)
    cache.lens = np.array(lens)
    fa.fa_fwd_paged(draw(10, (8, 4, 64))[0].cuda(), *cache.device(), i32(cu))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_pages_that_do_not_exist_are_reported(bad):
    """The other sequence's results stay."""
    cache = Cache(45, [60, 200], 2, 16, 64)
    q, cu = draw(11, (2, 4, 64))[0].cuda(), i32([0, 1, 2])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    cache.table[0, 1] = bad
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()
    assert torch.equal(o[1], want[0][1]) and torch.equal(lse[:, 1], want[1][:, 1])


def test_graph_replay_with_other_lengths_and_tables():
    cache = Cache(46, [500, 300], 2, 32, 64)
    q = draw(12, (4, 8, 64))[0].cuda()
    dev = cache.device()
    table, lens, cu = dev[4], dev[5], i32([0, 1, 4])
    want = fa.fa_fwd_paged(q, *dev, cu)
    ws = torch.empty(max(1, fa.fa_fwd_paged_workspace_bytes(2, 8, 2, 4, 64, cache.n, 32, table.shape[1])), dtype=torch.uint8,
                     device="cuda")
    o, lse = torch.empty_like(q), torch.empty(8, 4, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_paged(q, *dev, cu, o=o, lse=lse, workspace=ws)
    graph.replay()
    ok()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    cache.lens, cache.table = np.array([3, 290]), cache.table[::-1].copy()
    cache.table[0, 9:], cache.table[1, 10] = -1, cache.table[1, 0]
    lens.copy_(i32(cache.lens))
    table.copy_(i32(cache.table))
    cu.copy_(i32([0, 2, 3]))
    o.fill_(9.0)
    graph.replay()
    ok()
    O, L, A, F = reference(cache, q, [0, 2, 3], 0.125, True)
    check_o(o[:3], O[:3], A[:3], F[:3])
    check_lse(lse[:, :3], L[:, :3], score_tol(cache, q, 0.125))
    assert (o[3] == 9.0).all()


def test_two_streams():
    """Calls that run at the same time, each with its own workspace."""
    caches = [Cache(47 + i, [3000, 700 + i], 2, 32, 128) for i in range(2)]
    q = draw(13, (2, 8, 128))[0].cuda()
    cu = i32([0, 1, 2])
    dev = [c.device() for c in caches]
    want = [fa.fa_fwd_paged(q, *d, cu) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[fa.fa_fwd_paged(q, *d, cu, stream=s) for _ in range(20)] for d, s in zip(dev, streams)]
    ok()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_beyond_32_bit_offsets():
    """Pages more than 2^31 bytes apart."""
    H, page, d = 2, 128, 128
    n = (1 << 31) // (H * page * d) + 40
    cache = Cache(48, [200], H, page, d, spare=0)
    q = draw(14, (1, 4, d))[0].cuda()
    want = fa.fa_fwd_paged(q, *cache.device(), i32([0, 1]))
    ids = [n - 1, 3]
    big = []
    for c in (cache.k, cache.v):
        x = torch.full((n, H, page, d), 0x7f, dtype=torch.uint8, device="cuda")
        for i in range(2):
            x[ids[i]] = c[int(cache.table[0, i])].view(torch.uint8)
        big.append(x.view(E4M3))
    scales = []
    for s in (cache.ks, cache.vs):
        x = torch.full((n, H), float("nan"), device="cuda")
        for i in range(2):
            x[ids[i]] = s[int(cache.table[0, i])]
        scales.append(x)
    got = fa.fa_fwd_paged(q, *big, *scales, i32([ids]), i32([200]), i32([0, 1]))
    ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d,page,interleaved", [(128, 64, False), (64, 16, True)])
def test_answers_token_by_token(d, page, interleaved):
    """Prompts of two users appended and attended, then steps of one token: every step equals attention
    over what the cache holds, and in all it stays near attention over bf16 keys."""
    H, H_kv = 8, 2
    r = np.random.default_rng(d)
    prompts, steps = [37, 150], 20
    cache = Cache(49, [n + steps for n in prompts], H_kv, page, d)
    f = fa.fa_rope_frequencies(d, device="cuda")
    seen_k, seen_v = [[], []], [[], []]
    cache.lens = np.array([0, 0])
    for step in range(steps + 1):
        new = prompts if step == 0 else [1, 1]
        cache.lens = cache.lens + np.array(new)
        cu = offsets(new)
        q, k, v = draw(100 + step, (cu[-1], H, d), (cu[-1], H_kv, d), (cu[-1], H_kv, d))
        turned = fa.fa_kv_append(k.cuda(), v.cuda(), i32(cu), *cache.device(), q=q.cuda(), inv_freq=f, interleaved=interleaved)
        o, lse = fa.fa_fwd_paged(turned, *cache.device(), i32(cu))
        ok()
        O, L, A, F = reference(cache, turned, cu, d ** -0.5, True)
        check_o(o, O, A, F)
        check_lse(lse, L, score_tol(cache, turned, d ** -0.5))
        pos = i32(np.concatenate([np.arange(n - m, n) for n, m in zip(cache.lens, new)]))
        kr = fa.fa_rope(k.cuda(), pos, f, interleaved=interleaved)
        for b in range(2):
            seen_k[b].append(kr[cu[b]:cu[b + 1]])
            seen_v[b].append(v[cu[b]:cu[b + 1]].cuda())
    ks, vs = (torch.cat([torch.cat(s) for s in seen]) for seen in (seen_k, seen_v))
    o2, _ = fa.fa_fwd_varlen(turned, ks, vs, i32(cu), i32(offsets(cache.lens)))
    ok()
    # e4m3 moves keys and values by 2^-4 at most, 2^-5.5 of their norm on average; twice that is allowed
    assert float((o.float() - o2.float()).norm() / o2.float().norm()) < 2 * 2.0 ** -4


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 30]])
@pytest.mark.parametrize("drop", [0, 1, 2, 3, 5])
def test_a_wait_that_runs_out_is_reported(drop, new):
    """A tile load left out: the call ends, says so, and the next one works."""
    cache = Cache(50, [5000, 3000, 700], 2, 64, 128)
    q = draw(15, (sum(new), 8, 128))[0].cuda()
    dev, cu = cache.device(), i32(offsets(new))
    ws = torch.zeros(fa.fa_fwd_paged_workspace_bytes(3, 8, 2, sum(new), 128, cache.n, 64, dev[4].shape[1]), dtype=torch.uint8,
                     device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(8, sum(new), device="cuda")
    assert fa.fa_fwd_paged_fault_test(q, *dev, cu, o, lse, 0.1, True, ws, drop, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    if drop < 2:       # (with few tiles per CTA a third load is never due)
        assert st == fa.FA_ERR_TIMEOUT and 30 <= info[0] <= 34, (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    check(cache, new, 8, 128, q=q.cpu())
