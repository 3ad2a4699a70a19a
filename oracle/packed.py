"""Oracle for packed sequences of different lengths and for a shared prefix:
plain, float64, CPU.

TEST INFRASTRUCTURE ONLY (see attention.py). It shares no code with the CUDA
path.

Readings where the pages stop:

* Packed sequences: sequence b owns the query rows [cu_q[b], cu_q[b+1]) of
  Q [T_q, H, d] and the keys [cu_kv[b], cu_kv[b+1]) of K, V [T_kv, H_kv, d].
  Causal: row i of n_q sees the keys j <= i + n_kv - n_q of n_kv, the rule
  under which the last row sees everything. A row that sees nothing has O = 0
  and LSE = -inf and takes part in no gradient.
* Shared prefix: every sequence of the batch sees all prefix keys and the
  first len_b keys of its own cache; causal among its N_q new rows: row i
  sees the own keys j < len_b - (N_q - 1 - i).

Besides O and LSE the forward functions return A = softmax(S) |V|, the scale
of O's rounding error when the probabilities are rounded.
"""
from __future__ import annotations

import numpy as np

__all__ = ["masked_head", "attention_packed", "attention_packed_bwd", "attention_prefix"]


def masked_head(q, k, v, scale: float, see):
    """One head with a visibility matrix: (O, LSE, A, P)."""
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    m0 = np.where(np.isfinite(m), m, 0.0)
    e = np.where(see, np.exp(s - m0[:, None]), 0.0)
    l = e.sum(axis=1)
    p = e / np.where(l > 0, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = m0 + np.log(l)
    return p @ v, lse, p @ np.abs(v), p


def _causal(n_q, n_kv, causal):
    i, j = np.arange(n_q)[:, None], np.arange(n_kv)[None, :]
    return j <= i + n_kv - n_q if causal else np.ones((n_q, n_kv), dtype=bool)


def attention_packed(Q, K, V, cu_q, cu_kv, scale: float, causal: bool):
    """O [T_q, H, d], LSE [H, T_q], A [T_q, H, d]; rows of no sequence are NaN."""
    Q, K, V = (np.asarray(x, dtype=np.float64) for x in (Q, K, V))
    T, H, _ = Q.shape
    G = H // K.shape[1]
    O, A, L = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan), np.full((H, T), np.nan)
    for b in range(len(cu_q) - 1):
        r, t = slice(cu_q[b], cu_q[b + 1]), slice(cu_kv[b], cu_kv[b + 1])
        see = _causal(r.stop - r.start, t.stop - t.start, causal)
        for h in range(H):
            O[r, h], L[h, r], A[r, h], _ = masked_head(Q[r, h], K[t, h // G], V[t, h // G], scale, see)
    return O, L, A


def attention_packed_bwd(Q, K, V, dO, cu_q, cu_kv, scale: float, causal: bool):
    """dQ, dK, dV of <dO, O> (NaN outside the sequences), and for each the
    matching sum of absolute products, the scale of its rounding error."""
    Q, K, V, dO = (np.asarray(x, dtype=np.float64) for x in (Q, K, V, dO))
    H = Q.shape[1]
    G = H // K.shape[1]
    out = [np.full(x.shape, np.nan) for x in (Q, K, V)]
    mag = [np.full(x.shape, np.nan) for x in (Q, K, V)]
    for b in range(len(cu_q) - 1):
        r, t = slice(cu_q[b], cu_q[b + 1]), slice(cu_kv[b], cu_kv[b + 1])
        see = _causal(r.stop - r.start, t.stop - t.start, causal)
        for x in out[1:] + mag[1:]:
            x[t] = 0.0
        for h in range(H):
            q, k, v, do = Q[r, h], K[t, h // G], V[t, h // G], dO[r, h]
            o, _, _, p = masked_head(q, k, v, scale, see)
            dp = do @ v.T
            ds = p * (dp - (do * o).sum(axis=1, keepdims=True))
            # |dS| as it is computed: P and D carry rounded inputs of these sizes
            ads = p * (np.abs(dp) + (np.abs(do) * np.abs(o)).sum(axis=1, keepdims=True))
            out[0][r, h], mag[0][r, h] = scale * (ds @ k), abs(scale) * (ads @ np.abs(k))
            out[1][t, h // G] += scale * (ds.T @ q)
            mag[1][t, h // G] += abs(scale) * (ads.T @ np.abs(q))
            out[2][t, h // G] += p.T @ do
            mag[2][t, h // G] += p.T @ np.abs(do)
    return tuple(out), tuple(mag)


def attention_prefix(Q, K_prefix, V_prefix, K, V, lens, scale: float, causal: bool):
    """Q [B, H, N_q, d]; prefix [H_kv, N_p, d] (or None); own K, V
    [B, H_kv, room, d] of which lens[b] rows exist. O, LSE [B, H, N_q], A."""
    Q, K, V = (np.asarray(x, dtype=np.float64) for x in (Q, K, V))
    B, H, Nq, d = Q.shape
    G = H // K.shape[1]
    if K_prefix is None:
        K_prefix = V_prefix = np.zeros((K.shape[1], 0, d))
    K_prefix, V_prefix = (np.asarray(x, dtype=np.float64) for x in (K_prefix, V_prefix))
    n_p = K_prefix.shape[1]
    O, A, L = np.empty(Q.shape), np.empty(Q.shape), np.empty(Q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        end = n - (Nq - 1) + np.arange(Nq) if causal else np.full(Nq, n)
        see = np.concatenate([np.ones((Nq, n_p), dtype=bool), np.arange(n)[None, :] < end[:, None]], axis=1)
        for h in range(H):
            k = np.concatenate([K_prefix[h // G], K[b, h // G, :n]])
            v = np.concatenate([V_prefix[h // G], V[b, h // G, :n]])
            O[b, h], L[b, h], A[b, h], _ = masked_head(Q[b, h], k, v, scale, see)
    return O, L, A
