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
from tests.test_gpu_paged import check
from tests.test_gpu_varlen import draw, ok

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
