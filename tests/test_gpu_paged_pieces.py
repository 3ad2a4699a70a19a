"""fa_fwd_paged where sequences have many rows (pieces of prompts): the kernel with row tiles of 128, over
the same masks, scales, layouts and calls that test_gpu_paged has for few rows, with its
tolerances (needs a GB300); V scales of any size in both kernels. More than 16 rows (new tokens x heads of a group) per sequence on average
take this kernel; pages of 64 rows and more one form of it, smaller ones the other.
"""
import numpy as np
import pytest
import torch

from exact_io_aware_34_gb300 import fa
from tests.test_gpu_append import Cache, E4M3, i32, offsets
from tests.test_gpu_paged import check, check_o, reference, score_tol
from tests.test_gpu_varlen import check_lse, draw, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def unequal(cache, seed, octaves=6):
    """Scales that differ from page to page, not powers of two."""
    g = torch.Generator().manual_seed(seed)
    for s in (cache.ks, cache.vs):
        s.mul_(torch.exp2(torch.rand(s.shape, generator=g) * octaves - octaves).cuda())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_units_of_one_row_tile_before_units_of_two(page, d):
    """Many units of a CTA that leave its second row tile out, then one that has it: it reads its own pages'
    scales. The same bits from run to run."""
    new, lens = [], []
    for i in range(360):
        new.append(20 if i % 12 < 9 else 64)              # 80 rows, or 256
        lens.append((40, 100, 128)[i % 3] if i % 12 < 9 else (64, 200, 333)[i % 3])
    cache = Cache(page + d, lens, 2, page, d)
    unequal(cache, 1)
    a = check(cache, new, 8, d, seed=3)
    q = draw(3, (sum(new), 8, d))[0].cuda()
    for _ in range(10):
        b = fa.fa_fwd_paged(q, *cache.device(), i32(offsets(new)))
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_end_inside_a_warp(d, G):
    """Units whose last rows hold no query, whole and in parts; what stands between the rows of O stays."""
    new, lens = [17, 31, 33, 50, 64, 95, 100], [300, 31, 4000, 50, 1000, 777, 129]
    cache, n, H = Cache(d + G, lens, 2, 32, d), sum(new), 2 * G
    q = draw(G, (n, H, d))[0]
    o, lse = check(cache, new, H, d, q=q)
    wide, l2 = torch.full((H, n + 2, d + 8), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((H, n + 2), 5.0, device="cuda")
    out = wide[:, :, :d].transpose(0, 1)
    fa.fa_fwd_paged(torch.cat([q, q[:2]]).cuda(), *cache.device(), i32(offsets(new)), o=out, lse=l2)
    ok()
    assert torch.equal(out[:n], o) and torch.equal(l2[:, :n], lse) and (l2[:, n:] == 5.0).all()
    out[:n] = 7.0
    assert (wide == 7.0).all()


def set_page(cache, seq, k, v_scale, codes=True):
    """V scale of page k of a sequence; codes False: zeros, as fa_kv_append writes them with a scale of 2^-100."""
    i = int(cache.table[seq, k])
    cache.vs[i] = v_scale
    if not codes:
        cache.v.view(torch.uint8)[i] = 0


@pytest.mark.parametrize("rows", [1, 2, 40])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("stride", [128, 16])
@pytest.mark.parametrize("first,later,codes", [
    (-100, 51, False), (-100, 28, False), (-100, 119, True), (-135, -6, True), (-135, -6, False), (51, -100, True),
    (118, -140, True), (-60, 40, True),
])
def test_v_scales_of_any_size(first, later, codes, stride, d, page, rows):
    """Whole tiles, or pages in turn, whose V scale is 2^first before and between ones with 2^later (-100: what zeros get, -135: an
    amax of 2^-126 over 448): every weight stays in the sum, whatever its V scale. Units of several tiles,
    most of them whole."""
    lens = [300, 520, 140] * 40
    cache = Cache(page + d, lens, 2, page, d)
    for b, n in enumerate(lens):
        for k in range(-(-n // page)):
            low = (k * page // max(page, stride)) % 2 == 0
            set_page(cache, b, k, 2.0 ** (first if low else later), codes or not low)
    check(cache, [rows] * len(lens), 8, d, seed=rows)


@pytest.mark.parametrize("rows", [1, 2, 40])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("small,large", [(-70, 0), (-100, 20), (-30, 50)])
def test_a_large_v_scale_without_weight(small, large, page, rows):
    """Pages of large values whose keys have no weight (2^-280 of the others') leave small ones as they are, with
    both in one tile, in another order, and in tiles of their own."""
    d, lens = 64, [32 + page, 64 + page, 400] * 40
    cache = Cache(page, lens, 2, page, d)
    q = torch.full((len(lens) * rows, 4, d), 1.0, dtype=torch.bfloat16)
    for b, n in enumerate(lens):
        for k in range(-(-n // page)):
            i, heavy = int(cache.table[b, k]), (k % 3 == 1) if b % 3 < 2 else (k * page // 128 == 1)
            cache.k[i] = torch.full((2, page, d), -4.0 if heavy else 2.0).to(E4M3).cuda()
            cache.ks[i] = 1.0
            set_page(cache, b, k, 2.0 ** (large if heavy else small))
    check(cache, [rows] * len(lens), 4, d, scale=0.5, q=q, causal=False)


PAGES = pytest.mark.parametrize("page", [16, 64])
NEW, LENS = [70, 1, 33, 40], [200, 1, 300, 40]      # 4 x 144 rows with four heads a group


@PAGES
@pytest.mark.parametrize("causal", [True, False])
def test_what_stands_behind_a_length_does_not_matter(page, causal):
    """NaN codes and scales, and entries of no page, behind every length."""
    cache = Cache(page, LENS, 2, page, 128)
    unequal(cache, 5)
    q, cu = draw(5, (sum(NEW), 8, 128))[0].cuda(), i32(offsets(NEW))
    want = fa.fa_fwd_paged(q, *cache.device(), cu, causal=causal)
    for b, n in enumerate(cache.lens):
        last = int(cache.table[b, (n - 1) // page])
        if n % page:
            for c in (cache.k, cache.v):
                c.view(torch.uint8)[last, :, n % page:] = 0x7f
    used = {int(i) for i in cache.table.flatten() if i >= 0}
    for i in set(range(cache.n)) - used:
        for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
            c.view(torch.uint8)[i] = 0x7f
            s[i] = float("nan")
    cache.table[cache.table < 0] = 2 ** 31 - 1
    got = fa.fa_fwd_paged(q, *cache.device(), cu, causal=causal)
    ok()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@PAGES
def test_non_finite_keys_and_values(page):
    """A NaN key makes the rows that see it NaN and no others; a NaN value its column of the rows that see it
    (and perhaps of others of its sequence); other sequences and heads stay."""
    d, new, lens = 64, [60, 50], [300, 170]
    cache = Cache(page, lens, 2, page, d)
    q, cu = draw(6, (110, 8, d))[0].cuda(), i32(offsets(new))
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    at = 270                                            # the first 30 rows do not see it
    cache.k.view(torch.uint8)[int(cache.table[0, at // page]), 0, at % page, 5] = 0x7f
    cache.v.view(torch.uint8)[int(cache.table[1, 100 // page]), 1, 100 % page, 9] = 0xff
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    assert o[30:60, :4].isnan().all() and lse[:4, 30:60].isnan().all()
    assert o[60:, 4:, 9].isnan().all()
    o[30:60, :4], lse[:4, 30:60], o[60:, 4:, 9] = want[0][30:60, :4], want[1][:4, 30:60], want[0][60:, 4:, 9]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@PAGES
def test_non_finite_queries_stay_in_their_rows(page):
    cache = Cache(page, [300, 90], 2, page, 64)
    q, cu = draw(7, (120, 8, 64))[0].cuda(), i32([0, 70, 120])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    bad = ((1, 2, 0, "nan"), (40, 5, 1, "inf"), (100, 7, 63, "-inf"))
    for t, h, c, x in bad:
        q[t, h, c] = float(x)
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    for t, h, _, _ in bad:
        assert o[t, h].isnan().all() and lse[h, t].isnan()
        o[t, h], lse[h, t] = want[0][t, h], want[1][h, t]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@PAGES
def test_block_scales_of_every_size(page):
    """Scales that differ by 2^24 from page to page, queries of very different size."""
    cache = Cache(page, [700, 300], 2, page, 128)
    g = torch.Generator().manual_seed(1)
    for s in (cache.ks, cache.vs):
        s.copy_(torch.exp2(torch.rand(s.shape, generator=g) * 24 - 26))
    cache.ks.clamp_(max=0.01)
    q = draw(2, (90, 8, 128))[0]
    q[1] *= 2.0 ** -20
    q[60, 3] *= 2.0 ** 6
    check(cache, [50, 40], 8, 128, q=q)


@PAGES
@pytest.mark.parametrize("first", [True, False])
def test_zero_scales(page, first):
    """Pages of zeros as other code may write them, codes and scale zero: a sequence's first tile, or one within."""
    cache = Cache(page, [400], 2, page, 64)
    for k in range(128 // page) if first else [200 // page]:
        i = int(cache.table[0, k])
        for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
            c.view(torch.uint8)[i] = 0
            s[i] = 0.0
    q = draw(3, (60, 4, 64))[0]
    o, lse = fa.fa_fwd_paged(q.cuda(), *cache.device(), i32([0, 60]))
    ok()
    cache.vs[cache.vs == 0] = 1.0      # (the oracle's F divides by it; the pages' values stay zero)
    O, L, A, F = reference(cache, q, [0, 60], 0.125, True)
    check_o(o, O, A, F)
    check_lse(lse, L, score_tol(cache, q, 0.125))


@PAGES
def test_large_and_equal_scores(page):
    cache = Cache(page, [400, 390, 50], 2, page, 128)
    cache.ks[int(cache.table[0, 3])] *= 16
    check(cache, [30, 40, 20], 8, 128, q=draw(4, (90, 8, 128))[0] * 3)
    cache.k.view(torch.uint8).zero_()
    check(cache, [30, 40, 20], 8, 128)


@PAGES
def test_parts_of_one_buffer_and_of_a_projection(page):
    cache = Cache(page, [130, 377], 2, page, 128, one_buffer=True)
    q = draw(8, (95, 4, 128))[0].cuda()
    cu = i32([0, 50, 90])
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    out, l2 = torch.full_like(q, 7.0), torch.full((4, 95), 5.0, device="cuda")
    fa.fa_fwd_paged(torch.cat([q, q], 1)[:, 4:], *cache.device(), cu, o=out, lse=l2)
    ok()
    assert torch.equal(out[:90], o[:90]) and torch.equal(l2[:, :90], lse[:, :90])
    assert (out[90:] == 7.0).all() and (l2[:, 90:] == 5.0).all()
    check(cache, [50, 40], 4, 128, T_extra=5)


@PAGES
def test_shared_pages(page):
    cache = Cache(page, [200, 190], 2, page, 64)
    cache.table[1, :128 // page] = cache.table[0, :128 // page]
    check(cache, [20, 60], 8, 64)


@PAGES
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_pages_that_do_not_exist_are_reported(page, bad):
    """The other sequence's results stay."""
    cache = Cache(page, [160, 200], 2, page, 64)
    q, cu = draw(11, (90, 4, 64))[0].cuda(), i32([0, 40, 90])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    ok()
    cache.table[0, 1] = bad
    o, lse = fa.fa_fwd_paged(q, *cache.device(), cu)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()
    assert torch.equal(o[40:], want[0][40:]) and torch.equal(lse[:, 40:], want[1][:, 40:])


@pytest.mark.parametrize("cu,lens", [([0, 50, 30], [60, 60]), ([0, -1, 30], [60, 60]), ([0, 40, 999], [60, 60]),
                                     ([0, 40, 80], [60, 10 ** 6]), ([0, 40, 80], [-5, 60])])
def test_offsets_and_lengths_that_do_not_fit_are_reported(cu, lens):
    cache = Cache(44, [60, 60], 2, 16, 64)
    cache.lens = np.array(lens)
    fa.fa_fwd_paged(draw(10, (80, 4, 64))[0].cuda(), *cache.device(), i32(cu))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status()[0] == fa.FA_ERR_INVALID_ARG
    ok()


@PAGES
def test_graph_replay_with_other_lengths_and_tables(page):
    cache = Cache(page, [500, 300], 2, page, 64)
    q = draw(12, (120, 8, 64))[0].cuda()
    dev = cache.device()
    table, lens, cu = dev[4], dev[5], i32([0, 20, 120])
    want = fa.fa_fwd_paged(q, *dev, cu)
    ws = torch.empty(fa.fa_fwd_paged_workspace_bytes(2, 8, 2, 120, 64, cache.n, page, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    o, lse = torch.empty_like(q), torch.empty(8, 120, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_paged(q, *dev, cu, o=o, lse=lse, workspace=ws)
    graph.replay()
    ok()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    cache.lens, cache.table = np.array([33, 290]), cache.table[::-1].copy()
    cache.table[0, 300 // page + 1:] = -1
    lens.copy_(i32(cache.lens))
    table.copy_(i32(cache.table))
    cu.copy_(i32([0, 60, 110]))           # (27 rows of the first see nothing)
    o.fill_(9.0)
    graph.replay()
    ok()
    O, L, A, F = reference(cache, q, [0, 60, 110], 0.125, True)
    check_o(o[:110], O[:110], A[:110], F[:110])
    check_lse(lse[:, :110], L[:, :110], score_tol(cache, q, 0.125))
    assert (o[110:] == 9.0).all()


@PAGES
def test_two_streams(page):
    """Calls that run at the same time, each with its own workspace."""
    caches = [Cache(47 + i, [3000, 700 + i], 2, page, 128) for i in range(2)]
    q, cu = draw(13, (90, 8, 128))[0].cuda(), i32([0, 70, 90])
    dev = [c.device() for c in caches]
    want = [fa.fa_fwd_paged(q, *d, cu) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[fa.fa_fwd_paged(q, *d, cu, stream=s) for _ in range(20)] for d, s in zip(dev, streams)]
    ok()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_the_same_bits_from_run_to_run(page, d):
    """Many key tiles for every unit, one after the other without a pause: a product that overtook the one before
    it, or a scale read too early, would show as another bit now and then."""
    new, lens = [700, 1, 300, 130], [8000, 5000, 2500, 9001]
    cache = Cache(page + d, lens, 4, page, d)
    unequal(cache, 2, 3)
    q, cu = draw(d, (sum(new), 16, d))[0].cuda(), i32(offsets(new))
    dev = cache.device()
    a = fa.fa_fwd_paged(q, *dev, cu)
    for _ in range(50):
        b = fa.fa_fwd_paged(q, *dev, cu)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ok()


def test_beyond_32_bit_offsets():
    """Pages more than 2^31 bytes apart."""
    H, page, d = 2, 128, 128
    n = (1 << 31) // (H * page * d) + 40
    cache = Cache(48, [200], H, page, d, spare=0)
    q, cu = draw(14, (50, 4, d))[0].cuda(), i32([0, 50])
    want = fa.fa_fwd_paged(q, *cache.device(), cu)
    ids = [n - 1, 3]
    big, scales = [], []
    for c in (cache.k, cache.v):
        x = torch.full((n, H, page, d), 0x7f, dtype=torch.uint8, device="cuda")
        for i in range(2):
            x[ids[i]] = c[int(cache.table[0, i])].view(torch.uint8)
        big.append(x.view(E4M3))
    for s in (cache.ks, cache.vs):
        x = torch.full((n, H), float("nan"), device="cuda")
        for i in range(2):
            x[ids[i]] = s[int(cache.table[0, i])]
        scales.append(x)
    got = fa.fa_fwd_paged(q, *big, *scales, i32([ids]), i32([200]), cu)
    ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("drop", [0, 1, 2, 3, 5, 8, 13])
def test_every_wait_that_runs_out_is_reported(drop, rows):
    """Several units and more loads for each CTA than its ring of tiles holds (10 at most): whichever is left
    out, the call ends and says so, and the next one works."""
    lens, d = [6000, 300] * 24, 64
    cache = Cache(50, lens, 2, 64, d)
    new = [rows] * len(lens)
    q = draw(15, (sum(new), 8, d))[0].cuda()
    dev, cu = cache.device(), i32(offsets(new))
    want = fa.fa_fwd_paged(q, *dev, cu, scale=0.1)
    ok()
    ws = torch.zeros(fa.fa_fwd_paged_workspace_bytes(len(lens), 8, 2, sum(new), d, cache.n, 64, dev[4].shape[1]),
                     dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(8, sum(new), device="cuda")
    assert fa.fa_fwd_paged_fault_test(q, *dev, cu, o, lse, 0.1, True, ws, drop, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_ERR_TIMEOUT and 30 <= info[0] <= 34, (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    got = fa.fa_fwd_paged(q, *dev, cu, scale=0.1)
    ok()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
