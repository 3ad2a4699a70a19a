"""Oracle for rotary positions and a paged 8-bit cache: plain, float64, CPU.

TEST INFRASTRUCTURE ONLY (see attention.py). It shares no code with the CUDA
path.

* Rotation: pair j of a head's first `rot` columns, as the complex number
  a + i b, times factor * e^{i position inv_freq[j]} (its conjugate for the
  transposed rotation).
* A page [H_kv, page, d] of codes and a scale for each head; a value is code *
  scale. Appending: the scale is the smallest power of two (2^-100 at least)
  by which the largest finite value written to the page fits 448, or the
  page's older rows' scale if that is larger; older rows are brought to a
  larger scale by rounding again.
"""
from __future__ import annotations

import numpy as np

from .packed import masked_head

__all__ = ["rotate", "round_e4m3", "least_scale", "append_pages", "attention_paged"]


def rotate(x, positions, inv_freq, interleaved=False, transpose=False, factor=1.0):
    """x [T, heads, d]; positions [T] (integers); inv_freq [rot / 2]."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    a = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    turn = factor * np.exp(1j * np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq))[:, None]
    z = (x[..., a[0]] + 1j * x[..., a[1]]) * (turn.conj() if transpose else turn)
    x[..., a[0]], x[..., a[1]] = z.real, z.imag
    return x


def round_e4m3(y):
    """To the nearest e4m3 value, ties to even; |y| up to 448 (more has no value here), NaN stays."""
    y = np.asarray(y, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(y))), -6.0)
    step = np.exp2(np.where(np.isfinite(e), e, -6.0) - 3.0)
    return np.rint(y / step) * step


def least_scale(amax):
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_pages(x, cu, codes, scale, table, lens, page, exact=False):
    """x [T, H_kv, d] float64, codes [num_pages, H_kv, page, d], scale
    [num_pages, H_kv]: what both hold afterwards (new arrays). With ``exact`` what is
    written is left unrounded."""
    codes, scale = np.array(codes, dtype=np.float64), np.array(scale, dtype=np.float64)
    rnd = (lambda y: y) if exact else round_e4m3
    for b in range(len(cu) - 1):
        n, end = int(cu[b + 1] - cu[b]), int(lens[b])
        for k in range((end - n) // page, -(-end // page) if n else 0):
            p0, p1 = max(end - n, k * page), min(end, (k + 1) * page)
            t0, r0, i = int(cu[b]) + p0 - (end - n), p0 - k * page, int(table[b][k])
            for h in range(x.shape[1]):
                rows = x[t0:t0 + p1 - p0, h]
                fine = np.isfinite(rows)
                s = least_scale(np.abs(rows[fine]).max(initial=0.0))
                if r0:
                    s = max(s, scale[i, h])
                    codes[i, h, :r0] = rnd(codes[i, h, :r0] * (scale[i, h] / s))
                codes[i, h, r0:r0 + p1 - p0] = rnd(np.where(fine, rows, np.nan) / s)
                scale[i, h] = s
    return codes, scale


def attention_paged(Q, k_codes, v_codes, k_scale, v_scale, table, lens, cu_q, scale: float, causal: bool):
    """Q [T, H, d]; O [T, H, d], LSE [H, T], A = P |V| [T, H, d], and F [T, H, d]: a
    row's largest probability times its key's scale, times the sum of all
    |codes|, which a fixed error of every weight is multiplied by. Rows of no
    sequence are NaN."""
    Q = np.asarray(Q, dtype=np.float64)
    T, H, _ = Q.shape
    page = k_codes.shape[2]
    G = H // k_codes.shape[1]
    O, A, F = (np.full(Q.shape, np.nan) for _ in range(3))
    L = np.full((H, T), np.nan)
    for b in range(len(cu_q) - 1):
        r, n = slice(int(cu_q[b]), int(cu_q[b + 1])), int(lens[b])
        n_q = r.stop - r.start
        ids = [int(i) for i in table[b][:-(-n // page)]]
        i, j = np.arange(n_q)[:, None], np.arange(n)[None, :]
        see = j <= i + n - n_q if causal else np.ones((n_q, n), dtype=bool)
        for h in range(H):
            k, v = (np.concatenate([c[i, h // G] * s[i, h // G] for i in ids] or [c[0, 0, :0]])[:n]
                    for c, s in ((k_codes, k_scale), (v_codes, v_scale)))
            O[r, h], L[h, r], A[r, h], p = masked_head(Q[r, h], k, v, scale, see)
            s = np.repeat([v_scale[i, h // G] for i in ids], page)[:n]
            F[r, h] = (p * s).max(axis=1, initial=0.0)[:, None] * np.abs(v / s[:, None]).sum(axis=0)
    return O, L, A, F
