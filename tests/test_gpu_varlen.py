"""fa_fwd_varlen against the float64 oracle, through the C ABI (needs a GB300).

Tolerances, from the arithmetic: P V sees each probability rounded to bf16
(off by at most 2^-8 of itself) and so is the largest one in O's normaliser;
O is rounded once more. So |O - ref| <= 2^-8 (A + 2 |ref|) with A = P |V|, and
float32 sums and exponentials add a few 2^-22 of A. LSE is float32: a score's
sum of d products is off by at most d 2^-24 scale |q|.|k|, the rest by 2^-22
steps of values below 32. Where keys are split, every part has a normaliser of
its own, whose rounding moves that part's share of O: 2^-8 (2 A + |ref|).
"""
import math

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_34_gb300 import fa
from tests import parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def draw(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(torch.bfloat16) for s in shapes]


def ok():
    torch.cuda.synchronize()
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_OK, (fa.fa_status_string(st), info)


def check_o(o, ref, A, scale_up=1.0, split=False):
    err = np.abs(parity.to64(o) - ref)
    tol = 2.0 ** -8 * (2 * A + np.abs(ref) if split else A + 2 * np.abs(ref)) + 1e-5 * A + 1e-30
    assert np.isfinite(parity.to64(o)).all()
    assert (err <= tol * scale_up).all(), float((err / tol).max())


def lse_tol(q, k, scale):
    """Largest |scale| sum |q||k| of any pair, times d 2^-24, plus the exponentials' share."""
    n = float(q.float().abs().amax() * k.float().abs().amax()) * abs(scale) * q.shape[-1] if q.numel() and k.numel() else 0
    return n * q.shape[-1] * 2.0 ** -24 / 4 + 32 * 2.0 ** -22


def check_lse(lse, ref, tol):
    got = lse.double().cpu().numpy()
    none = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), none)
    assert np.isfinite(got[~none]).all()
    if (~none).any():
        off = float(np.abs(got[~none] - ref[~none]).max())
        assert off <= tol, off


def check(q, k, v, ql, kl, causal, scale=None, split=False, **kw):
    d = q.shape[-1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    cq, ck = offsets(ql), offsets(kl)
    o, lse = fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cq.cuda(), ck.cuda(), scale=scale, causal=causal, **kw)
    ok()
    n = int(cq[-1])
    O, L, A = oracle.attention_packed(*(parity.to64(x) for x in (q, k, v)), cq.tolist(), ck.tolist(), scale, causal)
    check_o(o[:n], O[:n], A[:n], split=split)
    check_lse(lse[:, :n], L[:, :n], lse_tol(q, k, scale))
    return o, lse


LENS = [
    ([1], [1]), ([37], [37]), ([128], [128]), ([129], [129]), ([300, 1, 64, 0, 257], None),
    ([5, 1, 100], [700, 129, 100]),         # later pieces of prompts
    ([10, 200, 3], [4, 0, 128]),            # rows that see nothing, a sequence without keys
    ([0, 0, 7, 0], [3, 0, 260, 0]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,H_kv,d", [(4, 1, 128), (8, 2, 64), (2, 2, 128), (7, 1, 64), (3, 1, 128)])
@pytest.mark.parametrize("empty", [0, 200])
@pytest.mark.parametrize("case", range(len(LENS)))
def test_lengths(case, empty, H, H_kv, d, causal):
    """Without a list of units, and (200 empty sequences behind) with one."""
    ql, kl = LENS[case]
    kl = (kl or ql) + [0] * empty
    ql = ql + [0] * empty
    q, k, v = draw(case * 100 + H + d, (sum(ql), H, d), (max(1, sum(kl)), H_kv, d), (max(1, sum(kl)), H_kv, d))
    check(q, k, v, ql, kl, causal)


@pytest.mark.parametrize("G", [1, 2, 5, 12, 16, 32, 64, 100, 128])
def test_heads_per_group(G):
    q, k, v = draw(G, (150, 2 * G, 64), (400, 2, 64), (400, 2, 64))
    check(q, k, v, [3, 140, 7], [200, 141, 59], True)


@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences(causal):
    """More sequences than the plan's chunk, most of one to three tokens."""
    r = np.random.default_rng(5)
    ql = r.integers(0, 4, 1300)
    kl = ql + r.integers(0, 3, 1300)
    ql[700], kl[700] = 500, 700
    q, k, v = draw(9, (int(ql.sum()), 2, 64), (int(kl.sum()), 1, 64), (int(kl.sum()), 1, 64))
    check(q, k, v, ql.tolist(), kl.tolist(), causal)


@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(scale, d):
    q, k, v = draw(17, (200, 4, d), (350, 2, d), (350, 2, d))
    check(q, k, v, [150, 50], [200, 150], True, scale=scale)


def test_layouts():
    """Slices of one buffer, head-major tensors and outputs inside wider buffers: the same bits."""
    H, Hk, d, ql = 8, 2, 128, [100, 201, 3]
    T = sum(ql)
    qkv, = draw(3, (T, H + 2 * Hk, d))
    qkv = qkv.cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    cu = offsets(ql).cuda()
    o0, l0 = fa.fa_fwd_varlen(q.contiguous(), k.contiguous(), v.contiguous(), cu, cu)
    o1, l1 = fa.fa_fwd_varlen(q, k, v, cu, cu)
    heads = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    wide = torch.full((T, H + 3, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    o2, l2 = fa.fa_fwd_varlen(*heads, cu, cu, o=wide[:, 1:H + 1, :d])
    o3 = torch.empty(H, T, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    fa.fa_fwd_varlen(*heads, cu, cu, o=o3)
    ok()
    for o, l in ((o1, l1), (o2, l2), (o3, l0)):
        assert torch.equal(o, o0) and torch.equal(l, l0)
    wide[:, 1:H + 1, :d] = 7.0
    assert bool((wide == 7.0).all())


def test_foreign_rows_do_not_matter_and_stay():
    """NaN and infinities in other sequences' and nobody's rows; rows behind the last sequence are not written."""
    H, Hk, d = 4, 2, 128
    q, k, v = draw(21, (300, H, d), (500, Hk, d), (500, Hk, d))
    cq, ck = [0, 90, 90 + 70], [0, 130, 130 + 200]
    clean = [x.clone() for x in (q, k, v)]
    for x, y in ((q, float("nan")), (k, float("nan")), (v, float("inf"))):
        x[160 if x is q else 330:] = y
    k[:130], v[:130] = float("nan"), float("-inf")
    cqd, ckd = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cq, ck))
    o = torch.full((300, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, 300), 5.0, device="cuda")
    fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cqd, ckd, o=o, lse=lse)
    ok()
    assert bool((o[160:] == 5).all()) and bool((lse[:, 160:] == 5).all())
    o_ref, l_ref = fa.fa_fwd_varlen(*(x.cuda() for x in clean), cqd, ckd)
    ok()
    assert torch.equal(o[90:160], o_ref[90:160]) and torch.equal(lse[:, 90:160], l_ref[:, 90:160])
    # the first sequence's last block holds the second's keys
    q2, k2, v2 = (x.clone() for x in clean)
    k2[130:], v2[130:] = float("nan"), float("nan")
    o2, l2 = fa.fa_fwd_varlen(q2.cuda(), k2.cuda(), v2.cuda(), cqd, ckd, causal=False)
    o3, l3 = fa.fa_fwd_varlen(*(x.cuda() for x in clean), cqd, ckd, causal=False)
    ok()
    assert torch.equal(o2[:90], o3[:90]) and torch.equal(l2[:, :90], l3[:, :90])


def test_sequence_result_does_not_depend_on_the_batch():
    q, k, v = (x.cuda() for x in draw(31, (700, 8, 128), (700, 2, 128), (700, 2, 128)))
    cu = offsets([200, 300, 200]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    one = offsets([300]).cuda()
    o1, l1 = fa.fa_fwd_varlen(q[200:500], k[200:500], v[200:500], one, one)
    o2, l2 = fa.fa_fwd_varlen(q, k, v, cu, cu)
    ok()
    assert torch.equal(o[200:500], o1) and torch.equal(lse[:, 200:500], l1)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_graph_replayed_with_other_offsets_and_streams():
    q, k, v = (x.cuda() for x in draw(33, (600, 4, 64), (600, 2, 64), (600, 2, 64)))
    cu = offsets([600]).cuda()
    o = torch.empty(600, 4, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 600, device="cuda")
    ws = torch.empty(fa.fa_fwd_varlen_workspace_bytes(3, 4, 2, 600, 600, 64), dtype=torch.uint8, device="cuda")
    cu3 = offsets([100, 250, 250]).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fa.fa_fwd_varlen(q, k, v, cu3, cu3, o=o, lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_fwd_varlen(q, k, v, cu3, cu3, o=o, lse=lse, workspace=ws)
    cu3.copy_(offsets([1, 599, 0]))
    g.replay()
    ref = fa.fa_fwd_varlen(q, k, v, offsets([1, 599, 0]).cuda(), offsets([1, 599, 0]).cuda(), stream=s.cuda_stream)
    ok()
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert cu.shape[0] == 2


LONG = [
    ([1], [5000]), ([100, 17, 0, 64], [4000, 333, 0, 2500]), ([513], [1800]),
    ([70, 1, 33], [20, 6000, 0]),           # rows that see nothing, a sequence without keys
    ([1] * 20 + [40], [5] * 20 + [9000]),   # pieces of many units beside one unit of many pieces
    ([200], [1537]), ([0, 0], [2000, 1]),   # no piece is cut; no rows at all
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,H_kv,d", [(4, 1, 128), (8, 2, 64), (7, 1, 64), (3, 3, 128), (96, 1, 64)])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_split_keys(case, H, H_kv, d, causal):
    """Few rows on long caches: units whose keys are split among CTAs."""
    ql, kl = LONG[case]
    q, k, v = draw(case * 10 + H + d, (max(1, sum(ql)), H, d), (sum(kl), H_kv, d), (sum(kl), H_kv, d))
    o, lse = check(q, k, v, ql, kl, causal, split=True)
    cu = [offsets(x).cuda() for x in (ql, kl)]
    o2, lse2 = fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), *cu, causal=causal)
    n = sum(ql)
    assert torch.equal(o[:n], o2[:n]) and torch.equal(lse[:, :n], lse2[:, :n])


def test_split_keys_layouts_and_foreign_rows():
    """Slices and wider outputs, rows of no sequence, NaN and infinities in other sequences' rows."""
    H, Hk, d, ql, kl = 6, 2, 128, [50, 21], [2900, 1700]
    q, k, v = draw(77, (90, H, d), (5000, Hk, d), (5000, Hk, d))
    k[4600:], v[4600:], q[71:] = float("nan"), float("inf"), float("nan")
    k2, v2 = k.clone(), v.clone()
    k2[:2900], v2[:2900] = float("nan"), float("-inf")
    cq, ck = offsets(ql).cuda(), offsets(kl).cuda()
    o, lse = check(q[:71], k[:4600], v[:4600], ql, kl, True, split=True)
    kv = torch.cat([k2, v2], 1).cuda()
    wide = torch.full((90, H + 3, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    l2 = torch.full((H, 90), 5.0, device="cuda")
    fa.fa_fwd_varlen(q.cuda(), kv[:, :Hk], kv[:, Hk:], cq, ck, o=wide[:, 1:H + 1, :d], lse=l2)
    ok()
    o2 = wide[:71, 1:H + 1, :d].clone()
    check_o(o2[50:], parity.to64(o[50:]), 2 * np.abs(parity.to64(v[2900:4600])).max() + 0 * parity.to64(o[50:]))
    assert bool((l2[:, 71:] == 5).all())
    assert float((l2[:, 50:71] - lse[:, 50:]).abs().max()) <= 2 * lse_tol(q[:71], k[:4600], d ** -0.5)
    wide[:71, 1:H + 1, :d] = 7.0
    assert bool((wide == 7.0).all())


def test_split_keys_scales_and_one_key_that_counts():
    """A key far above the others in one part: the other parts' weights vanish and the row is its V."""
    q, k, v = draw(78, (3, 2, 64), (4000, 1, 64), (4000, 1, 64))
    for scale in (0.0, -0.2, 2.0):
        check(q, k, v, [3], [4000], False, scale=scale, split=True)
    k[2222] = 40 * q[1, 1].sign()
    o, lse = fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), offsets([3]).cuda(), offsets([4000]).cuda(), scale=1.0)
    ok()
    assert torch.equal(o[1, 1].cpu(), v[2222, 0])


def test_split_keys_graph_replayed_with_other_lengths():
    """One captured call: split, whole and empty, each as a call of its own computes it."""
    q, k, v = (x.cuda() for x in draw(79, (64, 4, 64), (6000, 2, 64), (6000, 2, 64)))
    cq, ck = offsets([30, 34]).cuda(), offsets([5000, 1000]).cuda()
    o, lse = torch.empty_like(q), torch.empty(4, 64, device="cuda")
    ws = torch.empty(fa.fa_fwd_varlen_workspace_bytes(2, 4, 2, 64, 6000, 64), dtype=torch.uint8, device="cuda")
    fa.fa_fwd_varlen(q, k, v, cq, ck, o=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_fwd_varlen(q, k, v, cq, ck, o=o, lse=lse, workspace=ws)
    for ql, kl in (([1, 63], [40, 900]), ([64, 0], [5990, 0]), ([2, 62], [3000, 3000]), ([0, 0], [6000, 0])):
        cq.copy_(offsets(ql))
        ck.copy_(offsets(kl))
        ws.fill_(255)
        o.fill_(9)
        g.replay()
        n = sum(ql)
        o2, l2 = fa.fa_fwd_varlen(q, k, v, cq, ck)
        ok()
        assert torch.equal(o[:n], o2[:n]) and torch.equal(lse[:, :n], l2[:, :n])
        assert bool((o[n:] == 9).all())


def test_two_calls_at_once():
    """Two streams, each call with its own workspace: the results of either alone."""
    sets = []
    for seed, ql, kl in ((80, [40, 3], [5000, 900]), (81, [700, 900, 400], [1000, 900, 400])):
        q, k, v = (x.cuda() for x in draw(seed, (sum(ql), 8, 128), (sum(kl), 8, 128), (sum(kl), 8, 128)))
        sets.append((q, k, v, offsets(ql).cuda(), offsets(kl).cuda()))
    alone = [fa.fa_fwd_varlen(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    both = []
    for _ in range(10):
        both += [fa.fa_fwd_varlen(*x, stream=s) for x, s in zip(sets, streams)]
    ok()
    for i, (o, lse) in enumerate(both):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(lse, alone[i % 2][1])


def test_long_prompt_sampled_rows():
    """8192 tokens, 32 heads on 8 (the 8k workload's sizes): rows of every block against the oracle."""
    T, H, Hk, d = 8192, 32, 8, 128
    q, k, v = draw(41, (T, H, d), (T, Hk, d), (T, Hk, d))
    cu = offsets([T]).cuda()
    o, lse = fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cu, cu)
    ok()
    scale = 1 / math.sqrt(d)
    for i in list(range(0, T, 509)) + [T - 1]:
        h = (i * 7) % H
        see = np.ones((1, i + 1), dtype=bool)
        O, L, A, _ = oracle.masked_head(parity.to64(q[i:i + 1, h]), parity.to64(k[:i + 1, h // 4]),
                                        parity.to64(v[:i + 1, h // 4]), scale, see)
        check_o(o[i:i + 1, h], O, A)
        check_lse(lse[h, i:i + 1], L, lse_tol(q, k, scale))


@pytest.mark.parametrize("drop", [0, 1, 3])
def test_dropped_load_times_out_cleanly(drop):
    q, k, v = (x.cuda() for x in draw(51, (300, 4, 128), (300, 2, 128), (300, 2, 128)))
    cu = offsets([300]).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(4, 300, device="cuda")
    ws = torch.empty(fa.fa_fwd_varlen_workspace_bytes(1, 4, 2, 300, 300, 128), dtype=torch.uint8, device="cuda")
    assert fa.fa_fwd_varlen_fault_test(q, k, v, o, lse, cu, cu, 0.1, True, ws, drop, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_ERR_TIMEOUT and info[0] in (13, 14, 15, 16), (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    check(q.cpu(), k.cpu(), v.cpu(), [300], [300], True)


def test_dropped_load_with_split_keys_times_out_cleanly():
    q, k, v = (x.cuda() for x in draw(52, (60, 4, 128), (4000, 2, 128), (4000, 2, 128)))
    cq, ck = offsets([60]).cuda(), offsets([4000]).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(4, 60, device="cuda")
    ws = torch.empty(fa.fa_fwd_varlen_workspace_bytes(1, 4, 2, 60, 4000, 128), dtype=torch.uint8, device="cuda")
    assert fa.fa_fwd_varlen_fault_test(q, k, v, o, lse, cq, ck, 0.1, True, ws, 2, 20_000_000) == fa.FA_OK
    st, info = fa.fa_get_device_status()
    assert st == fa.FA_ERR_TIMEOUT and info[0] in (13, 14, 15, 16), (st, info)
    assert fa.fa_get_device_status()[0] == fa.FA_OK
    check(q.cpu(), k.cpu(), v.cpu(), [60], [4000], True, split=True)


def test_bad_offsets_with_split_keys():
    q, k, v = (x.cuda() for x in draw(62, (100, 4, 64), (3000, 2, 64), (3000, 2, 64)))
    good = offsets([20, 20, 60]).cuda()
    o = torch.full((100, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, 50, 40, 3000], [-1, 20, 40, 100], [0, 20, 40, 3001], [0, 20, 1 << 30, 100]):
        fa.fa_fwd_varlen(q, k, v, good, torch.tensor(bad, dtype=torch.int32, device="cuda"), o=o)
        st, info = fa.fa_get_device_status()
        assert st == fa.FA_ERR_INVALID_ARG and info[0] == 16 and info[1] < 3, (st, info)
    assert bool((o == 3).all())


@pytest.mark.parametrize("empty", [0, 300])
@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [-1, 20, 40, 100], [0, 20, 40, 101], [0, 20, 1 << 30, 100]])
def test_bad_offsets_are_reported_and_write_nothing(bad, empty):
    """The plan's own check of the offsets finds them, lists no work and says so in the status word."""
    q, k, v = (x.cuda() for x in draw(61, (100, 4, 64), (100, 2, 64), (100, 2, 64)))
    good = offsets([20, 20, 60] + [0] * empty).cuda()
    bad = torch.tensor(bad + bad[-1:] * empty, dtype=torch.int32, device="cuda")
    o = torch.full((100, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for cq, ck in ((bad, good), (good, bad), (bad, bad)):
        fa.fa_fwd_varlen(q, k, v, cq, ck, o=o)
        st, info = fa.fa_get_device_status()
        assert st == fa.FA_ERR_INVALID_ARG and info[0] == 16 and info[1] < 3 + empty, (st, info)
    assert bool((o == 3).all())
    assert fa.fa_get_device_status()[0] == fa.FA_OK


def test_binding_refusals():
    q, k, v = (x.cuda() for x in draw(71, (10, 4, 64), (10, 2, 64), (10, 2, 64)))
    cu = offsets([10]).cuda()
    for args in [(q.float(), k, v, cu, cu), (q, k[:5], v, cu, cu), (q, k, v, cu.long(), cu), (q, k, v, cu.cpu(), cu),
                 (q, k, v, cu, offsets([5, 5]).cuda()), (q[..., ::2], k[..., ::2], v[..., ::2], cu, cu),
                 (q[0], k, v, cu, cu)]:
        with pytest.raises(ValueError):
            fa.fa_fwd_varlen(*args)
    for kw in [dict(o=q.float()), dict(lse=torch.empty(10, 4, device="cuda")), dict(workspace=torch.empty(4096))]:
        with pytest.raises(ValueError):
            fa.fa_fwd_varlen(q, k, v, cu, cu, **kw)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_varlen(q, k, v, cu, cu, o=q)
    with pytest.raises(fa.FaError):
        x = torch.zeros(20000, 4, 64, dtype=torch.bfloat16, device="cuda")
        fa.fa_fwd_varlen(x, k, v, offsets([20000]).cuda(), cu, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


MORE_ROWS = [   # query rows, keys, heads, K/V heads, d: sequences with clearly more rows than keys
    ([2200], [1900], 1, 1, 64), ([3000], [2000], 1, 1, 64), ([3000], [2000], 8, 8, 128), ([4500], [2000], 2, 2, 128),
    ([222, 1433], [1856, 270], 8, 2, 64), ([1300, 300, 700], [300, 2100, 0], 6, 2, 128), ([500, 1, 2600], [40, 5000, 1700], 4, 4, 64),
]


@pytest.mark.parametrize("case", range(len(MORE_ROWS)))
def test_split_keys_with_more_rows_than_keys(case):
    """Whatever the workspace held (all ones, NaN, another call's partial results), the first rows see nothing and the
    others what the oracle says."""
    ql, kl, H, H_kv, d = MORE_ROWS[case]
    T, Tk = sum(ql), sum(kl)
    q, k, v, q2, k2 = draw(200 + case, (T, H, d), (Tk, H_kv, d), (Tk, H_kv, d), (T, H, d), (Tk, H_kv, d))
    need = fa.fa_fwd_varlen_workspace_bytes(len(ql), H, H_kv, T, Tk, d)
    ws = torch.empty(max(128, need), dtype=torch.uint8, device="cuda")
    ws.fill_(0x7F)
    a = check(q, k, v, ql, kl, True, split=True, workspace=ws)
    ws.fill_(0xFF)
    b = check(q, k, v, ql, kl, True, split=True, workspace=ws)
    cq, ck = offsets(ql[::-1]).cuda(), offsets(kl[::-1]).cuda()
    fa.fa_fwd_varlen(3 * q2.cuda(), k2.cuda(), v.cuda(), cq, ck, scale=1.0, workspace=ws)
    c = check(q, k, v, ql, kl, True, split=True, workspace=ws)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


@pytest.mark.parametrize("H,H_kv,d", [(8, 2, 128), (8, 8, 64)])
def test_one_causal_prompt_with_few_heads(H, H_kv, d):
    """4096 tokens, whose units nearly fill the device and whose keys are split: rows of every block against the oracle."""
    T = 4096
    q, k, v = draw(43 + d, (T, H, d), (T, H_kv, d), (T, H_kv, d))
    cu = offsets([T]).cuda()
    ws = torch.empty(fa.fa_fwd_varlen_workspace_bytes(1, H, H_kv, T, T, d), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    ws.fill_(0x7F)
    o, lse = fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cu, cu, workspace=ws)
    ok()
    for i in list(range(0, T, 127)) + [T - 1]:
        h = (i * 7) % H
        O, L, A, _ = oracle.masked_head(parity.to64(q[i:i + 1, h]), parity.to64(k[:i + 1, h * H_kv // H]),
                                        parity.to64(v[:i + 1, h * H_kv // H]), d ** -0.5, np.ones((1, i + 1), dtype=bool))
        check_o(o[i:i + 1, h], O, A, split=True)
        check_lse(lse[h, i:i + 1], L, lse_tol(q, k, d ** -0.5))


def test_a_unit_may_last_longer_than_the_limit_of_a_wait():
    """One unit of 3125 key blocks, each wait limited to a millisecond: the warp that hands out work waits for the whole
    unit, and that is no timeout."""
    q, k, v = (x.cuda() for x in draw(53, (64, 4, 64), (400_000, 2, 64), (400_000, 2, 64)))
    cq, ck = (offsets([n] + [0] * 199).cuda() for n in (64, 400_000))     # (too many sequences to split the keys)
    o, lse = torch.zeros_like(q), torch.zeros(4, 64, device="cuda")
    ws = torch.empty(fa.fa_fwd_varlen_workspace_bytes(200, 4, 2, 64, 400_000, 64), dtype=torch.uint8, device="cuda")
    o2, lse2 = fa.fa_fwd_varlen(q, k, v, cq, ck, scale=0.1)
    ok()
    assert fa.fa_fwd_varlen_fault_test(q, k, v, o, lse, cq, ck, 0.1, True, ws, -1, 1_000_000) == fa.FA_OK
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,H_kv", [(16, 4), (4, 4)])
def test_long_prompts_of_64_columns(H, H_kv):
    """Two prompts of some thousand tokens at d = 64: rows of every block against the oracle."""
    lens, d = [6001, 3333], 64
    T = sum(lens)
    q, k, v = draw(44 + H, (T, H, d), (T, H_kv, d), (T, H_kv, d))
    cu = offsets(lens).cuda()
    o, lse = fa.fa_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cu, cu)
    ok()
    for at, n in zip((0, lens[0]), lens):
        for i in list(range(0, n, 127)) + [n - 1]:
            h, r, t = (i * 7) % H, slice(at + i, at + i + 1), slice(at, at + i + 1)
            O, L, A, _ = oracle.masked_head(parity.to64(q[r, h]), parity.to64(k[t, h * H_kv // H]),
                                            parity.to64(v[t, h * H_kv // H]), d ** -0.5, np.ones((1, i + 1), dtype=bool))
            check_o(o[r, h], O, A)
            check_lse(lse[h, r], L, lse_tol(q, k, d ** -0.5))


def test_a_last_group_of_fewer_heads():
    """K/V heads taken two at a time, of three: the bits of each head alone."""
    T, d = 40_000, 128
    q, k, v = (x.cuda() for x in draw(45, (T, 3, d), (T, 3, d), (T, 3, d)))
    cu = offsets([T - 1000, 1000]).cuda()
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu)
    ok()
    for h in range(3):
        s = slice(h, h + 1)
        o1, lse1 = fa.fa_fwd_varlen(q[:, s], k[:, s], v[:, s], cu, cu)
        ok()
        assert torch.equal(o[:, s], o1) and torch.equal(lse[s], lse1)


def test_bad_offsets_whose_places_pass_two_to_the_63():
    """A first sequence of 2^31 - 1 rows whose places on the line of split keys end just below 2^63."""
    q, k, v = (x.cuda() for x in draw(63, (40, 512, 64), (3000, 4, 64), (3000, 4, 64)))
    assert fa.fa_fwd_varlen_workspace_bytes(2, 512, 4, 40, 3000, 64) > 0
    o = torch.full((40, 512, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((512, 40), 3.0, device="cuda")
    top = (1 << 31) - 1
    for bq, bk in (([0, top, 40], [0, 2_143_188_680, 3000]), ([0, top, 40], [0, top - 300, 3000]), ([0, top, 40], [0, top, 3000])):
        for causal in (False, True):
            fa.fa_fwd_varlen(q, k, v, *(torch.tensor(b, dtype=torch.int32, device="cuda") for b in (bq, bk)), o=o, lse=lse,
                             causal=causal)
            st, info = fa.fa_get_device_status()
            assert st == fa.FA_ERR_INVALID_ARG and info[0] == 16 and info[1] < 2, (st, info)
    assert bool((o == 3).all()) and bool((lse == 3).all())
