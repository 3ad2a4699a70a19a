"""fa_bwd_varlen against the float64 oracle, through the C ABI (needs a GB300).

Tolerances, from the arithmetic: dV sums P rounded to bf16 (each off by at
most 2^-8 of itself) against dO; dQ and dK sum dS rounded the same way, and D
carries O's rounding to bf16 (2^-8 of |dO| |O|). With M the same sums over
absolute values (|dS| counted as P (|dO V^T| + |dO| |O|)):
|dV - ref| <= 2^-8 (M + |ref|), |dQ - ref|, |dK - ref| <= 2^-8 (2 M + |ref|), the last
term being the result's own rounding; float32 adds 1e-4 M at most.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_34_gb300 import fa
from tests import parity
from tests.test_gpu_varlen import LENS, draw, offsets, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def reference(q, k, v, do, cq, ck, scale, causal):
    x = [parity.to64(t) for t in (q, k, v)]
    O, L, _ = oracle.attention_packed(*x, cq, ck, scale, causal)
    grads, mags = oracle.attention_packed_bwd(*x, parity.to64(do), cq, ck, scale, causal)
    return torch.from_numpy(O).to(torch.bfloat16), torch.from_numpy(L).float(), grads, mags


def compare(got, grads, mags, spans):
    for name, g, r, m, n in zip(("dQ", "dK", "dV"), got, grads, mags, spans):
        err, tol = np.abs(parity.to64(g[:n]) - r[:n]), 2.0 ** -8 * ((1 if name == "dV" else 2) * m[:n] + np.abs(r[:n]))
        tol = tol + 1e-4 * m[:n] + 1e-30
        assert np.isfinite(parity.to64(g[:n])).all(), name
        assert (err <= tol).all(), (name, float((err / tol).max()))


def check(q, k, v, do, ql, kl, causal, scale=None, **kw):
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    cq, ck = offsets(ql), offsets(kl)
    o, lse, grads, mags = reference(q, k, v, do, cq.tolist(), ck.tolist(), scale, causal)
    got = fa.fa_bwd_varlen(q.cuda(), k.cuda(), v.cuda(), o.cuda(), do.cuda(), lse.cuda(), cq.cuda(), ck.cuda(),
                           scale=scale, causal=causal, **kw)
    ok()
    compare(got, grads, mags, (int(cq[-1]), int(ck[-1]), int(ck[-1])))
    return got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,H_kv,d", [(4, 1, 128), (8, 2, 64), (2, 2, 128), (7, 1, 64), (3, 1, 128)])
@pytest.mark.parametrize("case", range(len(LENS)))
def test_lengths(case, H, H_kv, d, causal):
    ql, kl = LENS[case]
    kl = kl or ql
    Tk = max(1, sum(kl))
    q, k, v, do = draw(case * 100 + H + d, (sum(ql), H, d), (Tk, H_kv, d), (Tk, H_kv, d), (sum(ql), H, d))
    check(q, k, v, do, ql, kl, causal)


@pytest.mark.parametrize("G", [1, 2, 5, 12, 16, 32, 64, 100, 128])
def test_heads_per_group(G):
    q, k, v, do = draw(G, (150, 2 * G, 64), (400, 2, 64), (400, 2, 64), (150, 2 * G, 64))
    check(q, k, v, do, [3, 140, 7], [200, 141, 59], True)


def test_many_sequences():
    r = np.random.default_rng(6)
    ql = r.integers(0, 4, 1300)
    kl = ql + r.integers(0, 3, 1300)
    ql[700], kl[700] = 500, 700
    T, Tk = int(ql.sum()), int(kl.sum())
    q, k, v, do = draw(9, (T, 2, 64), (Tk, 1, 64), (Tk, 1, 64), (T, 2, 64))
    check(q, k, v, do, ql.tolist(), kl.tolist(), True)


@pytest.mark.parametrize("scale", [0.0, -0.11, 0.7])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(scale, d):
    q, k, v, do = draw(17, (200, 4, d), (350, 2, d), (350, 2, d), (200, 4, d))
    check(q, k, v, do, [150, 50], [200, 150], True, scale=scale)


def test_layouts_give_the_same_bits():
    """Inputs as slices of one buffer, gradients as slices of another, head-major tensors."""
    H, Hk, d, ql = 8, 2, 128, [100, 201, 3]
    T = sum(ql)
    qkv, do = (x.cuda() for x in draw(3, (T, H + 2 * Hk, d), (T, H, d)))
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    cu = offsets(ql).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    a = fa.fa_bwd_varlen(q.contiguous(), k.contiguous(), v.contiguous(), o, do, lse, cu, cu)
    g = torch.full_like(qkv, 9.0)
    b = fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu, dq=g[:, :H], dk=g[:, H:H + Hk], dv=g[:, H + Hk:])
    major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, o, do)]
    outs = [torch.empty(h, T, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1) for h in (H, Hk, Hk)]
    c = fa.fa_bwd_varlen(*major, lse, cu, cu, *outs)
    ok()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_foreign_rows_do_not_matter_and_stay():
    H, Hk, d = 4, 2, 128
    q, k, v, do = draw(21, (300, H, d), (500, Hk, d), (500, Hk, d), (300, H, d))
    cq, ck = (torch.tensor(c, dtype=torch.int32).cuda() for c in ([0, 90, 160], [0, 130, 330]))
    o, lse = (x.cpu() for x in fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cq, ck))
    ref = fa.fa_bwd_varlen(*(x.cuda() for x in (q, k, v, o, do, lse)), cq, ck)
    ok()
    nan = float("nan")
    for first in (True, False):       # everything but one sequence's rows and keys is NaN or infinite
        dirty = [x.clone() for x in (q, k, v, o, do)]
        bad_lse = lse.clone()
        for x, lo, hi in zip(dirty, (90, 130, 130, 90, 90), (160, 330, 330, 160, 160)):
            if first:
                x[lo:] = nan
            else:
                x[:lo], x[hi:] = float("inf"), nan
        bad_lse[:, 160:] = nan
        outs = [torch.full((n, h, d), 5.0, dtype=torch.bfloat16, device="cuda") for n, h in ((300, H), (500, Hk), (500, Hk))]
        fa.fa_bwd_varlen(*(x.cuda() for x in dirty), bad_lse.cuda(), cq, ck, *outs)
        ok()
        for g, r, lo, hi in zip(outs, ref, (90, 130, 130), (160, 330, 330)):
            own = slice(0, lo) if first else slice(lo, hi)
            assert torch.equal(g[own], r[own])
            assert bool((g[hi:] == 5).all())


def test_same_bits_from_run_to_run_and_batch_to_batch():
    q, k, v, do = (x.cuda() for x in draw(31, (700, 8, 128), (700, 2, 128), (700, 2, 128), (700, 8, 128)))
    cu, one = offsets([200, 300, 200]).cuda(), offsets([300]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    a = fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu)
    b = fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu)
    s = slice(200, 500)
    c = fa.fa_bwd_varlen(q[s], k[s], v[s], o[s], do[s], lse[:, s].contiguous(), one, one)
    ok()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x[s], z)


def test_one_sequence_without_mask_is_near_fa_bwd():
    q, k, v, do = draw(35, (400, 4, 128), (400, 4, 128), (400, 4, 128), (400, 4, 128))
    got = check(q, k, v, do, [400], [400], False)
    b = [x.transpose(0, 1)[None].contiguous().cuda() for x in (q, k, v, do)]
    o, lse = fa.fa_fwd(*b[:3])
    ref = fa.fa_bwd(*b[:3], o, b[3], lse)
    ok()
    for g, r in zip(got, ref):
        r = r[0].transpose(0, 1).double()
        assert float((g.double() - r).norm() / r.norm()) < 1e-2


def test_captured_step_replayed_with_other_offsets():
    """Forward and backward in one graph, replayed after the offsets changed, beside eager calls on another stream."""
    q, k, v, do = (x.cuda() for x in draw(33, (600, 4, 64), (600, 2, 64), (600, 2, 64), (600, 4, 64)))
    cu = offsets([100, 250, 250]).cuda()
    fa.fa_bwd_varlen(q, k, v, *fa.fa_fwd_varlen(q, k, v, cu, cu)[:1], do,
                     fa.fa_fwd_varlen(q, k, v, cu, cu)[1], cu, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
        grads = fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu)
    new = offsets([1, 599, 0]).cuda()
    cu.copy_(new)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g.replay()
    o2, lse2 = fa.fa_fwd_varlen(q, k, v, new, new, stream=s)
    ref = fa.fa_bwd_varlen(q, k, v, o2, do, lse2, new, new, stream=s)
    ok()
    for x, y in zip(grads, ref):
        assert torch.equal(x, y)


@pytest.mark.parametrize("drop", [0, 1, 2])
def test_dropped_load_times_out_cleanly(drop):
    q, k, v, do = (x.cuda() for x in draw(51, (500, 4, 128), (500, 2, 128), (500, 2, 128), (500, 4, 128)))
    cu = offsets([500]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    g = [torch.zeros_like(x) for x in (q, k, v)]
    ws = torch.empty(fa.fa_bwd_varlen_workspace_bytes(1, 4, 2, 500, 500), dtype=torch.uint8, device="cuda")
    assert fa.fa_bwd_varlen_fault_test(q, k, v, o, do, lse, cu, cu, *g, 0.1, True, ws, drop, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_ERR_TIMEOUT and 17 <= info[0] <= 22, (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    check(*(x.cpu() for x in (q, k, v, do)), [500], [500], True)


def test_bad_offsets_are_reported_and_write_nothing():
    q, k, v, do = (x.cuda() for x in draw(61, (100, 4, 64), (100, 2, 64), (100, 2, 64), (100, 4, 64)))
    good, bad = offsets([20, 20, 60]).cuda(), torch.tensor([0, 50, 40, 100], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_varlen(q, k, v, good, good)
    g = [torch.full_like(x, 3.0) for x in (q, k, v)]
    for cq, ck in ((bad, good), (good, bad)):
        fa.fa_bwd_varlen(q, k, v, o, do, lse, cq, ck, *g)
        st, info = fa.fa_get_device_status()
        assert st == fa.FA_ERR_INVALID_ARG and info[:2] == [16, 1], (st, info)
    assert all(bool((x == 3).all()) for x in g)


def test_binding_refusals():
    q, k, v, do = (x.cuda() for x in draw(71, (10, 4, 64), (10, 2, 64), (10, 2, 64), (10, 4, 64)))
    cu, lse = offsets([10]).cuda(), torch.zeros(4, 10, device="cuda")
    for args in [(q, k, v, do.float(), do, lse), (q, k, v, do, do[:5], lse), (q, k, v, do, do, lse.t()),
                 (q, k, v[:, :1], do, do, lse)]:
        with pytest.raises(ValueError):
            fa.fa_bwd_varlen(*args, cu, cu)
    for kw in [dict(dq=q), dict(dk=k), dict(dq=torch.empty_like(q), dk=do[:, :2]),
               dict(workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(fa.FaError):
            fa.fa_bwd_varlen(q, k, v, torch.zeros_like(q), do, lse, cu, cu, **kw)


def test_a_unit_may_last_longer_than_the_limit_of_a_wait():
    """One key block of 20001 steps, each wait limited to two milliseconds: the warps that hand out work and clear
    tails wait for the whole unit, and that is no timeout."""
    n, m = 32 * 20_000 + 5, 100
    q, k, v, do = (x.cuda() for x in draw(54, (n, 4, 64), (m, 1, 64), (m, 1, 64), (n, 4, 64)))
    cq, ck = offsets([n]).cuda(), offsets([m]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cq, ck, scale=0.1, causal=False)
    ref = fa.fa_bwd_varlen(q, k, v, o, do, lse, cq, ck, scale=0.1, causal=False)
    ok()
    g = [torch.zeros_like(x) for x in (q, k, v)]
    ws = torch.empty(fa.fa_bwd_varlen_workspace_bytes(1, 4, 1, n, m), dtype=torch.uint8, device="cuda")
    assert fa.fa_bwd_varlen_fault_test(q, k, v, o, do, lse, cq, ck, *g, 0.1, False, ws, -1, 2_000_000) == fa.FA_OK
    ok()
    assert all(torch.equal(x, y) for x, y in zip(g, ref))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,H_kv,d", [(4, 1, 128), (4, 2, 64), (2, 2, 64), (2, 2, 128)])
def test_long_sequences(H, H_kv, d, causal):
    """Units of one to 20 blocks, several for every CTA."""
    ql, kl = [2500, 130, 1, 1200], [2500, 700, 64, 900]
    T, Tk = sum(ql), sum(kl)
    q, k, v, do = draw(60 + H + d, (T, H, d), (Tk, H_kv, d), (Tk, H_kv, d), (T, H, d))
    check(q, k, v, do, ql, kl, causal)


def test_a_last_group_of_fewer_heads():
    """K/V heads taken two at a time, of three: the bits of each head alone."""
    T, d = 20_000, 128
    q, k, v, do = (x.cuda() for x in draw(61, *[(T, 3, d)] * 4))
    cu = offsets([T - 1000, 1000]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    a = fa.fa_bwd_varlen(q, k, v, o, do, lse, cu, cu)
    ok()
    for h in range(3):
        s = slice(h, h + 1)
        b = fa.fa_bwd_varlen(*(x[:, s] for x in (q, k, v, o, do)), lse[s], cu, cu)
        ok()
        assert all(torch.equal(x[:, s], y) for x, y in zip(a, b))
