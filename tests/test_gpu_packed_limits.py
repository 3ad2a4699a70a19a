"""Packed and prefix entry points at the edges of what they accept (needs a
GB300): tensors past 2^31 elements, very many sequences, two calls at once,
inputs that are one tensor."""
import numpy as np
import pytest
import torch

from exact_io_aware_34_gb300 import fa
from tests.test_gpu_varlen import draw, offsets, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def test_rows_past_two_to_the_31_elements():
    """The last 500 rows of tensors of 2.25e9 elements: the bits of a call on those rows alone."""
    T, H, d, n = 2_200_000, 8, 128, 500
    cu = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    one = offsets([n]).cuda()
    big, small = [], draw(1, *[(n, H, d)] * 4)
    for x in small:
        t = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda")
        t[:T - n] = float("nan")
        t[T - n:] = x.cuda()
        big.append(t)
    q, k, v, do = (x.cuda() for x in small)
    o, lse = fa.fa_fwd_varlen(q, k, v, one, one)
    o_big, lse_big = fa.fa_fwd_varlen(*big[:3], cu, cu)
    grads = fa.fa_bwd_varlen(q, k, v, o, do, lse, one, one)
    grads_big = fa.fa_bwd_varlen(*big[:3], o_big, big[3], lse_big, cu, cu)
    ok()
    assert torch.equal(o, o_big[T - n:]) and torch.equal(lse, lse_big[:, T - n:])
    for a, b in zip(grads, grads_big):
        assert torch.equal(a, b[T - n:])


def test_caches_past_two_to_the_31_elements():
    """One key that counts near the end of a prefix, another near the end of an own cache, 2.2e9 elements each."""
    H, d, n_p, room = 8, 128, 2_150_000, 1_080_000
    q, = draw(2, (2, H, 1, d))
    k = torch.empty(2, H, room, d, dtype=torch.bfloat16, device="cuda").normal_()
    v = torch.empty_like(k).normal_()
    kp = torch.empty(H, n_p, d, dtype=torch.bfloat16, device="cuda").normal_()
    vp = torch.empty_like(kp).normal_()
    kp[:, n_p - 7] = 40 * q[0, :, 0].sign().cuda()
    k[1, :, room - 9] = 40 * q[1, :, 0].sign().cuda()
    lens = torch.tensor([3, room - 2], dtype=torch.int32, device="cuda")
    o, _ = fa.fa_fwd_prefix(q.cuda(), kp, vp, k, v, lens)
    ok()
    assert torch.equal(o[0, :, 0], vp[:, n_p - 7]) and torch.equal(o[1, :, 0], v[1, :, room - 9])


def test_very_many_sequences():
    """70000 sequences of one token, each of which sees itself: O = V, dV = dO, and no gradient of Q and K."""
    B, H, d = 70000, 2, 64
    q, k, v, do = (x.cuda() for x in draw(3, *[(B, H, d)] * 4))
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    dq, dk, dv = fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu)
    ok()
    s = (q.double() * k.double()).sum(-1) / 8
    assert torch.equal(o, v)
    # a sum of 64 products and the float32 result's own rounding
    assert bool(((lse.T - s).abs() <= 64 * 2.0 ** -24 * (q.double() * k.double()).abs().sum(-1) / 8 + 2.0 ** -22 * 32).all())
    # P = exp(scale S - LSE) is off by what its argument is (below 1e-4), then rounded to bf16
    assert bool(((dv.double() - do.double()).abs() <= (2.0 ** -8 * 2 + 1e-4) * do.double().abs()).all())
    # dP and D are two float32 sums of the same 64 products
    m = 1e-5 * (do.double() * v.double()).abs().sum(-1, keepdim=True) / 8
    assert bool((dq.double().abs() <= m * k.double().abs()).all()) and bool((dk.double().abs() <= m * q.double().abs()).all())


def test_inputs_that_are_one_tensor():
    """K as V, and Q as K and V, give what copies give."""
    x, do = (t.cuda() for t in draw(4, (300, 4, 128), (300, 4, 128)))
    cu = offsets([100, 200]).cuda()
    o, lse = fa.fa_fwd_varlen(x, x, x, cu, cu)
    o2, lse2 = fa.fa_fwd_varlen(x, x.clone(), x.clone(), cu, cu)
    grads = fa.fa_bwd_varlen(x, x, x, o, do, lse, cu, cu)
    grads2 = fa.fa_bwd_varlen(x.clone(), x.clone(), x, o2, do, lse2, cu, cu)
    c, p = (t.cuda() for t in draw(5, (3, 4, 200, 128), (4, 150, 128)))
    lens = torch.tensor([200, 7, 0], dtype=torch.int32, device="cuda")
    y, _ = fa.fa_fwd_prefix(c[:, :, :2], p, p, c, c, lens)
    y2, _ = fa.fa_fwd_prefix(c[:, :, :2].clone(), p, p.clone(), c, c.clone(), lens)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(y, y2)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_calls_on_two_streams_at_once():
    """A training step and a decode step beside each other, over and over: the results of either alone."""
    q, k, v, do = (x.cuda() for x in draw(6, (1500, 8, 128), (1500, 2, 128), (1500, 2, 128), (1500, 8, 128)))
    cu = offsets([700, 1, 799]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    qd, kp, kc = (x.cuda() for x in draw(7, (9, 8, 1, 128), (2, 1000, 128), (9, 2, 500, 128)))
    lens = torch.tensor([500, 3, 0, 77, 128, 129, 400, 1, 250], dtype=torch.int32, device="cuda")
    train = lambda s: fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu, stream=s)  # noqa: E731
    decode = lambda s: fa.fa_fwd_prefix(qd, kp, kp, kc, kc, lens, stream=s)  # noqa: E731
    alone = train(None), decode(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    both = [(train(streams[0]), decode(streams[1]), decode(streams[2])) for _ in range(8)]
    ok()
    for a, b, c in both:
        assert all(torch.equal(x, y) for x, y in zip(a, alone[0]))
        assert all(torch.equal(x, y) for r in (b, c) for x, y in zip(r, alone[1]))


def test_a_non_finite_value_row_reaches_no_further_than_documented():
    """A V row of infinities: rows more than 254 before those that see it, and other sequences, keep their bits."""
    H, d = 4, 128
    for G in (1, 4):
        q, k, v = (x.cuda() for x in draw(8 + G, (1400, H, d), (1400, H // G, d), (1400, H // G, d)))
        cu = offsets([900, 500]).cuda()
        o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
        for row in (300, 511, 640):
            bad = v.clone()
            bad[row] = float("inf")
            o2, lse2 = fa.fa_fwd_varlen(q, k, bad, cu, cu)
            ok()
            assert torch.equal(lse, lse2)
            assert torch.equal(o[:max(0, row - 254)], o2[:max(0, row - 254)]) and torch.equal(o[900:], o2[900:])
            assert not bool(torch.isfinite(o2[row:900].float()).any())


def test_prefix_rows_past_two_to_the_27():
    """134e6 rows: the first and the last sequences have the bits of calls on them alone. (Q's rows overlap: O, its
    partial results and LSE take 52 GB.)"""
    B, H, N_q, d, n = 8200, 128, 128, 64, 6
    assert B * H * N_q > 1 << 27
    x, k, v = (t.cuda() for t in draw(12, ((B + H + N_q) * 64,), (B, 1, 5, d), (B, 1, 5, d)))
    view = lambda b0, b: x[64 * b0:].as_strided((b, H, N_q, d), (64, 64, 64, 1))  # noqa: E731
    lens = torch.arange(B, device="cuda", dtype=torch.int32) % 6
    o = torch.full((B, H, N_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, N_q), 7.0, device="cuda")
    fa.fa_fwd_prefix(view(0, B), None, None, k, v, lens, o=o, lse=lse)
    ok()
    for b0 in (0, B // 2, B - n):
        s = slice(b0, b0 + n)
        o2, lse2 = fa.fa_fwd_prefix(view(b0, n), None, None, k[s], v[s], lens[s].contiguous())
        ok()
        assert torch.equal(o[s], o2) and torch.equal(lse[s], lse2)


def test_a_non_finite_value_row_reaches_no_further_where_keys_are_split():
    """As above, with a part that holds a block of which the unit's first tile sees nothing."""
    for n_q, n_kv in ((390, 2183), (390, 2439), (390, 4231), (600, 2905)):
        q, k, v = (x.cuda() for x in draw(n_kv, (n_q, 4, 128), (n_kv, 4, 128), (n_kv, 4, 128)))
        cq, ck = offsets([n_q]).cuda(), offsets([n_kv]).cuda()
        assert fa.fa_fwd_varlen_workspace_bytes(1, 4, 4, n_q, n_kv, 128) > 0
        o, lse = fa.fa_fwd_varlen(q, k, v, cq, ck)
        for first in (255, 300, 382):     # the first row that sees the bad one
            bad = v.clone()
            bad[n_kv - n_q + first] = float("inf")
            o2, lse2 = fa.fa_fwd_varlen(q, k, bad, cq, ck)
            ok()
            assert torch.equal(lse, lse2)
            assert torch.equal(o[:max(0, first - 254)], o2[:max(0, first - 254)])
            assert not bool(torch.isfinite(o2[first:].float()).any())


def test_scale_of_any_number_type():
    """As the other entry points take it: what float() takes."""
    q, do = (x.cuda() for x in draw(13, (9, 4, 64), (9, 4, 64)))
    c, = (x.cuda() for x in draw(14, (2, 4, 30, 64)))
    cu, lens = offsets([4, 5]).cuda(), torch.tensor([30, 7], dtype=torch.int32, device="cuda")
    for scale in (np.float32(0.25), np.float64(0.25), torch.tensor(0.25), 1):
        o, lse = fa.fa_fwd_varlen(q, q, q, cu, cu, scale=float(scale))
        a = (o, lse) + fa.fa_bwd_varlen(q, q, q, o, do, lse, cu, cu, scale=float(scale)) \
            + fa.fa_fwd_prefix(c[:, :, :1], None, None, c, c, lens, scale=float(scale))
        b = fa.fa_fwd_varlen(q, q, q, cu, cu, scale=scale) + fa.fa_bwd_varlen(q, q, q, o, do, lse, cu, cu, scale=scale) \
            + fa.fa_fwd_prefix(c[:, :, :1], None, None, c, c, lens, scale=scale)
        ok()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
