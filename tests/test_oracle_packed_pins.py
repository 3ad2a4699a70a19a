"""Pins of oracle/packed.py: reductions to the pinned plain oracles, torch
autograd in float64, finite differences, rows that see nothing (CPU only)."""
import numpy as np
import pytest
import torch

import oracle

RNG = np.random.default_rng(11)


def _draw(*shape):
    return RNG.standard_normal(shape)


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


def test_one_sequence_without_mask_is_plain_attention():
    q, k, v = _draw(7, 4, 8), _draw(9, 2, 8), _draw(9, 2, 8)
    O, L, _ = oracle.attention_packed(q, k, v, [0, 7], [0, 9], 0.3, False)
    Or, Lr = oracle.attention_gqa(*(x.transpose(1, 0, 2)[None] for x in (q, k, v)), 0.3)
    assert np.allclose(O.transpose(1, 0, 2), Or[0], atol=1e-14) and np.allclose(L, Lr[0], atol=1e-14)


def _torch_loss(q, k, v, do, cu_q, cu_kv, scale, causal):
    """<dO, O> by torch, sequence by sequence, with an additive mask."""
    total = q.new_zeros(())
    G = q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        r, t = slice(cu_q[b], cu_q[b + 1]), slice(cu_kv[b], cu_kv[b + 1])
        n, m = r.stop - r.start, t.stop - t.start
        first = max(0, n - m) if causal else 0      # rows before this one see nothing
        if n == 0 or m == 0:
            continue
        s = torch.einsum("ihd,jhd->hij", q[r], k[t].repeat_interleave(G, 1)) * scale
        if causal:
            hide = torch.arange(m)[None, :] > torch.arange(n)[:, None] + m - n
            s = s + torch.where(hide, torch.tensor(-1e30, dtype=s.dtype), torch.tensor(0.0, dtype=s.dtype))
        o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v[t].repeat_interleave(G, 1))
        total = total + (o[first:] * do[r][first:]).sum()
    return total


CASES = [([3, 0, 5, 1], [4, 2, 5, 0], True), ([6, 2], [3, 2], True), ([4, 3], [2, 6], False)]


@pytest.mark.parametrize("ql,kl,causal", CASES)
def test_gradients_match_autograd(ql, kl, causal):
    cu_q, cu_kv = _offsets(ql), _offsets(kl)
    q, k, v, do = _draw(cu_q[-1], 4, 8), _draw(cu_kv[-1], 2, 8), _draw(cu_kv[-1], 2, 8), _draw(cu_q[-1], 4, 8)
    grads, _ = oracle.attention_packed_bwd(q, k, v, do, cu_q, cu_kv, 0.4, causal)
    tq, tk, tv = (torch.from_numpy(x).requires_grad_() for x in (q, k, v))
    loss = _torch_loss(tq, tk, tv, torch.from_numpy(do), cu_q, cu_kv, 0.4, causal)
    loss.backward()
    O, _, _ = oracle.attention_packed(q, k, v, cu_q, cu_kv, 0.4, causal)
    assert abs(float(loss.detach()) - (O * do).sum()) < 1e-12
    for g, t in zip(grads, (tq, tk, tv)):
        assert np.allclose(g, t.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_gradients_match_differences(which):
    cu_q, cu_kv = _offsets([3, 2]), _offsets([2, 4])
    x = [_draw(5, 2, 4), _draw(6, 1, 4), _draw(6, 1, 4)]
    do = _draw(5, 2, 4)
    grads, _ = oracle.attention_packed_bwd(*x, do, cu_q, cu_kv, 0.5, True)
    step = _draw(*x[which].shape)
    f = []
    for e in (1e-5, -1e-5):
        y = list(x)
        y[which] = y[which] + e * step
        f.append((oracle.attention_packed(*y, cu_q, cu_kv, 0.5, True)[0] * do).sum())
    assert abs((f[0] - f[1]) / 2e-5 - (grads[which] * step).sum()) < 1e-8


def test_rows_that_see_nothing():
    q, k, v = _draw(5, 1, 4), _draw(2, 1, 4), _draw(2, 1, 4)
    O, L, _ = oracle.attention_packed(q, k, v, [0, 5], [0, 2], 1.0, True)
    assert np.all(O[:3] == 0) and np.all(np.isneginf(L[:, :3])) and np.isfinite(L[:, 3:]).all()
    assert np.allclose(O[3, 0], v[0, 0])
    (dq, _, _), _ = oracle.attention_packed_bwd(q, k, v, _draw(5, 1, 4), [0, 5], [0, 2], 1.0, True)
    assert np.all(dq[:3] == 0)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n_p", [0, 5])
def test_prefix_is_one_sequence_of_prefix_and_own_keys(n_p, causal):
    B, H, Hk, Nq, room, d = 3, 4, 2, 3, 6, 8
    q, k, v = _draw(B, H, Nq, d), _draw(B, Hk, room, d), _draw(B, Hk, room, d)
    kp, vp = _draw(Hk, n_p, d), _draw(Hk, n_p, d)
    lens = [6, 0, 2]
    O, L, _ = oracle.attention_prefix(q, kp if n_p else None, vp if n_p else None, k, v, lens, 0.3, causal)
    for b, n in enumerate(lens):
        if causal and n < Nq:      # the packed rule counts the prefix keys into the causal order
            continue
        kk, vv = (np.concatenate([a, x[b, :, :n]], axis=1).transpose(1, 0, 2) for a, x in ((kp, k), (vp, v)))
        Or, Lr, _ = oracle.attention_packed(q[b].transpose(1, 0, 2), kk, vv, [0, Nq], [0, n_p + n], 0.3, causal)
        assert np.allclose(O[b], Or.transpose(1, 0, 2), atol=1e-13) and np.allclose(L[b], Lr, atol=1e-13)
    if causal and n_p == 0:        # two own keys, three new rows: the first sees nothing
        assert np.all(O[2, :, 0] == 0) and np.all(np.isneginf(L[2, :, 0]))
