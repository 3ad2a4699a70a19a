"""fa_fwd_prefix against the float64 oracle, through the C ABI (needs a GB300).

Tolerances: a segment's O is off by at most 2^-8 (A_s + |O_s|) (probabilities
and the normaliser's largest term rounded to bf16, see test_gpu_varlen), the
merge weights these by e^{LSE_s - LSE}, which sums A_s to A and |O_s| to A at
most, and O is rounded once: |O - ref| <= 2^-8 (2 A + |ref|), plus a few 2^-22 A.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_34_gb300 import fa
from tests import parity
from tests.test_gpu_varlen import check_lse, draw, lse_tol, offsets, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def check_o(o, ref, A):
    got = parity.to64(o)
    tol = 2.0 ** -8 * (2 * A + np.abs(ref)) + 1e-5 * A + 1e-30
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


def lens_of(lens):
    return torch.tensor(lens, dtype=torch.int32).cuda()


def make(seed, B, H, H_kv, N_q, n_p, room, d):
    q, kp, vp, k, v = draw(seed, (B, H, N_q, d), (H_kv, n_p, d), (H_kv, n_p, d), (B, H_kv, room, d), (B, H_kv, room, d))
    return q, (kp if n_p else None), (vp if n_p else None), k, v


def check(x, lens, causal=False, scale=None, **kw):
    q, kp, vp, k, v = x
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    dev = [None if t is None else t.cuda() for t in x]
    o, lse = fa.fa_fwd_prefix(*dev, lens_of(lens), scale=scale, causal=causal, **kw)
    ok()
    O, L, A = oracle.attention_prefix(*[None if t is None else parity.to64(t) for t in x], lens, scale, causal)
    check_o(o, O, A)
    keys = torch.cat([k.flatten(), kp.flatten()]) if kp is not None else k.flatten()
    check_lse(lse, L, lse_tol(q, keys, scale))
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,H_kv,N_q", [(8, 2, 1), (4, 4, 3), (7, 1, 1), (6, 2, 5), (32, 1, 8), (4, 1, 128)])
@pytest.mark.parametrize("n_p", [0, 1, 128, 1000])
def test_shapes(n_p, H, H_kv, N_q, d):
    x = make(n_p + H + N_q + d, 5, H, H_kv, N_q, n_p, 300, d)
    check(x, [300, 0, 1, 129, 128], causal=N_q > 1)


@pytest.mark.parametrize("G,N_q", [(1, 1), (16, 1), (128, 1), (100, 1), (128, 3), (5, 37), (3, 128)])
def test_heads_per_group(G, N_q):
    """Groups that fill a tile, do not divide it, or need several."""
    check(make(G + N_q, 3, 2 * G, 2, N_q, 200, 260, 64), [260, 17, 0], causal=True)


@pytest.mark.parametrize("causal", [True, False])
def test_lengths_shorter_than_the_new_tokens(causal):
    """Rows that see nothing (no prefix), or only the prefix."""
    for n_p in (0, 130):
        check(make(5 + n_p, 6, 4, 2, 4, n_p, 140, 128), [0, 1, 3, 4, 130, 140], causal=causal)


def test_many_sequences():
    r = np.random.default_rng(3)
    lens = r.integers(0, 200, 700).tolist()
    check(make(7, 700, 4, 2, 1, 513, 200, 64), lens)


@pytest.mark.parametrize("n_p", [0, 3001])
@pytest.mark.parametrize("d", [64, 128])
def test_several_blocks_and_segments_per_cta(d, n_p):
    """About ten blocks for every CTA, ragged ends inside its piece; the same bits from run to run."""
    x = make(21 + d + n_p, 6, 16, 8, 1, n_p, 10001, d)
    lens = [10001, 9000, 1, 7003, 10000, 33]
    a = check(x, lens)
    dev = [None if t is None else t.cuda() for t in x]
    b = fa.fa_fwd_prefix(*dev, lens_of(lens))
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_long_prefix_and_few_sequences():
    check(make(8, 2, 8, 1, 1, 20001, 64, 128), [5, 64])


def test_no_own_keys_at_all():
    check(make(9, 4, 8, 2, 2, 700, 10, 128), [0] * 4, causal=True)
    check(make(9, 4, 8, 2, 2, 0, 10, 128), [0] * 4, causal=True)


@pytest.mark.parametrize("scale", [0.0, -0.09, 2.0])
def test_scales(scale):
    check(make(10, 3, 8, 2, 2, 300, 200, 128), [200, 3, 77], causal=True, scale=scale)


def test_large_scores():
    q, kp, vp, k, v = make(11, 3, 8, 2, 1, 500, 400, 128)
    kp[:, 77] *= 16
    k[1, :, 300] *= 32
    check((q * 3, kp, vp, k, v), [400, 390, 0])


def test_agrees_with_fa_fwd_kv():
    """Full caches and no prefix: fa_fwd_kv's problem."""
    q, _, _, k, v = make(12, 3, 16, 4, 2, 0, 777, 128)
    o, lse = check((q, None, None, k, v), [777] * 3)
    o2, lse2 = fa.fa_fwd_kv(q.cuda(), k.cuda(), v.cuda())
    ok()
    assert float((o.float() - o2.float()).abs().max()) < 1e-2 and float((lse - lse2).abs().max()) < 1e-4


def test_layouts():
    """Caches stored token by token, a prefix as the first tokens of a packed cache, q and o as [B, N_q, H, d]."""
    q, kp, vp, k, v = (t.cuda() for t in make(13, 4, 8, 2, 3, 300, 200, 128))
    lens = lens_of([200, 1, 0, 130])
    o, lse = fa.fa_fwd_prefix(q, kp, vp, k, v, lens, causal=True)
    flip = lambda t, a, b: t.transpose(a, b).contiguous().transpose(a, b)  # noqa: E731
    wide = torch.full((4, 3, 10, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 1:9, :128].transpose(1, 2)
    o2, lse2 = fa.fa_fwd_prefix(flip(q, 1, 2), flip(kp, 0, 1), flip(vp, 0, 1), flip(k, 1, 2), flip(v, 0, 2), lens,
                                o=out, causal=True)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    out.fill_(7.0)
    assert bool((wide == 7.0).all())


def test_rows_past_a_length_do_not_matter():
    x = [t.cuda() for t in make(14, 4, 8, 2, 2, 129, 300, 128)]
    lens = [0, 5, 130, 300]
    o, lse = fa.fa_fwd_prefix(*x, lens_of(lens))
    for b, n in enumerate(lens):
        x[3][b, :, n:] = float("nan")
        x[4][b, :, n:] = float("inf") if b % 2 else float("nan")
    o2, lse2 = fa.fa_fwd_prefix(*x, lens_of(lens))
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_nan_query_stays_in_its_row():
    x = [t.cuda() for t in make(15, 40, 8, 2, 1, 300, 100, 128)]
    lens = lens_of([50 + b for b in range(40)])
    o, lse = fa.fa_fwd_prefix(*x, lens)
    x[0][7, 3] = float("nan")
    o2, lse2 = fa.fa_fwd_prefix(*x, lens)
    ok()
    assert bool(o2[7, 3].isnan().all()) and bool(lse2[7, 3].isnan().all())
    o2[7, 3], lse2[7, 3] = o[7, 3], lse[7, 3]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_captured_step_replayed_with_grown_lengths():
    q, kp, vp, k, v = (t.cuda() for t in make(16, 6, 8, 2, 1, 400, 500, 128))
    lens = lens_of([1, 100, 499, 3, 128, 0])
    fa.fa_fwd_prefix(q, kp, vp, k, v, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.fa_fwd_prefix(q, kp, vp, k, v, lens)
    s = torch.cuda.Stream()
    for _ in range(3):
        lens += 1
        lens.clamp_(max=500)
        torch.cuda.synchronize()
        g.replay()
        o2, lse2 = fa.fa_fwd_prefix(q, kp, vp, k, v, lens, stream=s)
        ok()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_prompt_then_decode():
    """A run as a server makes it: the shared prompt and each user's own prompt in one packed causal call,
    then decoding steps behind the shared keys, each against attention over the whole sequence."""
    H, Hk, d, n_p, room, scale = 8, 2, 128, 333, 64, 128 ** -0.5
    own = [20, 1, 41]
    B = len(own)
    total = [n_p + n for n in own]
    q, k, v = (t.cuda() for t in draw(17, (sum(total), H, d), (sum(total), Hk, d), (sum(total), Hk, d)))
    cu = offsets(total)
    for b in range(1, B):      # every sequence begins with the same prompt
        k[cu[b]:cu[b] + n_p], v[cu[b]:cu[b] + n_p] = k[:n_p], v[:n_p]
    # prompt: the prefix once, then every user's tokens against prefix and own keys
    ql = [n_p] + own
    kq = torch.cat([q[:n_p]] + [q[cu[b] + n_p:cu[b + 1]] for b in range(B)])
    kk, vv = (torch.cat([t[:n_p]] + [t[cu[b]:cu[b + 1]] for b in range(B)]) for t in (k, v))
    o, lse = fa.fa_fwd_varlen(kq, kk, vv, offsets(ql).cuda(), offsets([n_p] + total).cuda(), scale=scale)
    whole, whole_lse = fa.fa_fwd_varlen(q, k, v, cu.cuda(), cu.cuda(), scale=scale)
    ok()
    at = n_p
    for b in range(B):
        mine, full = slice(at, at + own[b]), slice(int(cu[b]) + n_p, int(cu[b + 1]))
        assert float((o[mine].float() - whole[full].float()).abs().max()) < 2e-2
        assert float((lse[:, mine] - whole_lse[:, full]).abs().max()) < 1e-4
        at += own[b]
    # decode: caches by token, one new token a step
    kp, vp = (t[:n_p].transpose(0, 1) for t in (k, v))
    ck, cv = (torch.full((B, room, Hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b in range(B):
        ck[b, :own[b]], cv[b, :own[b]] = (t[cu[b] + n_p:cu[b + 1]] for t in (k, v))
    lens = lens_of(own)
    for step in range(3):
        nq, nk, nv = (t.cuda() for t in draw(100 + step, (B, H, 1, d), (B, Hk, d), (B, Hk, d)))
        for b in range(B):
            ck[b, own[b] + step], cv[b, own[b] + step] = nk[b], nv[b]
        lens += 1
        o, lse = fa.fa_fwd_prefix(nq, kp, vp, ck.transpose(1, 2), cv.transpose(1, 2), lens, scale=scale, causal=True)
        ok()
        O, L, A = oracle.attention_prefix(*(parity.to64(t) for t in (nq, kp, vp, ck.transpose(1, 2), cv.transpose(1, 2))),
                                          lens.tolist(), scale, True)
        check_o(o, O, A)
        check_lse(lse, L, lse_tol(nq, k, scale))


@pytest.mark.parametrize("drop", [0, 1, 2])
def test_dropped_load_times_out_cleanly(drop):
    x = make(18, 3, 8, 2, 1, 5000, 2000, 128)
    q, kp, vp, k, v = (t.cuda() for t in x)
    lens = lens_of([2000, 100, 0])
    o, lse = torch.zeros_like(q), torch.zeros(3, 8, 1, device="cuda")
    ws = torch.empty(fa.fa_fwd_prefix_workspace_bytes(3, 8, 2, 1, 5000, 2000, 128), dtype=torch.uint8, device="cuda")
    ws.zero_()
    assert fa.fa_fwd_prefix_fault_test(q, kp, vp, k, v, lens, o, lse, 0.1, False, ws, drop, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    if drop < 2:       # with a load or two per CTA a third is never due
        assert st == fa.FA_ERR_TIMEOUT and 23 <= info[0] <= 26, (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    check(x, [2000, 100, 0])


def test_lengths_outside_the_cache_are_clamped_and_reported():
    x = make(19, 3, 4, 2, 1, 100, 50, 64)
    dev = [t.cuda() for t in x]
    o, lse = fa.fa_fwd_prefix(*dev, lens_of([-3, 51, 1 << 30]))
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_ERR_INVALID_ARG and info[0] == 26 and info[1] in (0, 1, 2), (st, info)
    o2, lse2 = check(x, [0, 50, 50])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_binding_refusals():
    q, kp, vp, k, v = (t.cuda() for t in make(20, 3, 4, 2, 1, 10, 20, 64))
    lens = lens_of([1, 2, 3])
    for args in [(q.float(), kp, vp, k, v, lens), (q, kp, None, k, v, lens), (q, kp[:1], vp, k, v, lens),
                 (q, kp, vp, k, v[:, :, :5], lens), (q, kp, vp, k, v, lens.long()), (q, kp, vp, k, v, lens[:2]),
                 (q, kp, vp, k[:2], v[:2], lens), (q, kp, vp, k, v, lens.cpu()), (q[0], kp, vp, k, v, lens),
                 (q, kp[None], vp[None], k, v, lens)]:
        with pytest.raises(ValueError):
            fa.fa_fwd_prefix(*args)
    for kw in [dict(o=q), dict(lse=lens.view(torch.float32).view(3, 1, 1).expand(3, 4, 1).contiguous(), o=k[:, :, :2]),
               dict(workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises((fa.FaError, ValueError)):
            fa.fa_fwd_prefix(q, kp, vp, k, v, lens, **kw)
    big = torch.zeros(1, 1, 129, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.fa_fwd_prefix(big, None, None, big, big.clone(), lens[:1], workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fill", [0x7F, 0xFF, 0x01, None])
@pytest.mark.parametrize("n_p", [0, 300])
def test_dropped_load_in_any_workspace(n_p, fill):
    """Units behind the one whose load is dropped are never noted: what the workspace held there is no address."""
    B, H, H_kv = 300, 16, 8
    x = make(23, B, H, H_kv, 1, n_p, 40, 128)
    dev = [None if t is None else t.cuda() for t in x]
    kp, vp = (torch.empty(H_kv, 0, 128, dtype=torch.bfloat16, device="cuda") if t is None else t for t in dev[1:3])
    lens = lens_of([40] * B)
    o, lse = torch.zeros_like(dev[0]), torch.zeros(B, H, 1, device="cuda")
    ws = torch.empty(fa.fa_fwd_prefix_workspace_bytes(B, H, H_kv, 1, n_p, 40, 128), dtype=torch.uint8, device="cuda")
    if fill is None:
        ws.random_(generator=torch.Generator("cuda").manual_seed(3))
    else:
        ws.fill_(fill)
    args = (dev[0], kp, vp, dev[3], dev[4], lens, o, lse, 0.1, False, ws)
    assert fa.fa_fwd_prefix_fault_test(*args, 0, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_ERR_TIMEOUT and 23 <= info[0] <= 26, (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    check(x, [40] * B)


def test_lengths_that_change_under_the_call():
    """Nobody may count on what such a call returns, but it ends, in time, and harms no other."""
    B, room = 300, 700
    x = make(24, B, 16, 8, 1, 200, room, 64)
    dev = [t.cuda() for t in x]
    g = torch.Generator("cuda").manual_seed(1)
    good = torch.randint(0, room + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    alone = fa.fa_fwd_prefix(*dev, good)
    lens = good.clone()
    calls, writes, other = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    results = []
    for _ in range(200):
        with torch.cuda.stream(writes):
            lens.random_(0, room + 1, generator=g)
            lens[B // 2:] = 0
            lens.fill_(room)
        fa.fa_fwd_prefix(*dev, lens, stream=calls)
        results.append(fa.fa_fwd_prefix(*dev, good, stream=other))
    ok()
    assert all(torch.equal(o, alone[0]) and torch.equal(lse, alone[1]) for o, lse in results)
