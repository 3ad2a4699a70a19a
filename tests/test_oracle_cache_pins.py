"""Pins of oracle/cache.py: torch's own 8-bit casts, closed forms, brute force, and the pinned packed oracle (CPU only)."""
import numpy as np
import pytest
import torch

import oracle

RNG = np.random.default_rng(17)


def test_rounding_is_torchs_cast():
    y = np.concatenate([RNG.standard_normal(4000) * s for s in (0.001, 0.02, 1.0, 100.0)])
    y = np.clip(y, -448, 448).astype(np.float32)
    edges = np.arange(-2 ** 12, 2 ** 12, dtype=np.float32) * 2.0 ** -11      # subnormals and every tie around them
    for v in (y, edges, edges * 200):
        want = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(oracle.round_e4m3(v), want)


def test_every_code_is_its_own_rounding():
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = v[np.isfinite(v)]
    assert np.array_equal(oracle.round_e4m3(v), v) and v.max() == 448.0


@pytest.mark.parametrize("amax,e", [(0.0, -100), (448.0, 0), (np.nextafter(448.0, 500), 1), (1.0, -8), (0.875, -9),
                                    (3e38, 120), (1e-38, -100)])
def test_least_scale(amax, e):
    assert oracle.least_scale(amax) == 2.0 ** e


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    x, pos = RNG.standard_normal((5, 3, 10)), np.array([0, 1, -7, 10 ** 6, 3])
    f = np.array([1.0, 0.1, 1e-5])
    y = oracle.rotate(x, pos, f, interleaved, factor=1.5)
    assert np.array_equal(y[..., 6:], x[..., 6:]) and np.allclose(y[0, :, :6], 1.5 * x[0, :, :6])
    for t, j in ((2, 1), (3, 0), (4, 2)):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + 3)
        c, s = np.cos(pos[t] * f[j]), np.sin(pos[t] * f[j])
        assert np.allclose(y[t, :, a], 1.5 * (c * x[t, :, a] - s * x[t, :, b]), atol=1e-12)
        assert np.allclose(y[t, :, b], 1.5 * (s * x[t, :, a] + c * x[t, :, b]), atol=1e-12)
    # the transposed rotation is the gradient, and undoes the rotation
    g = RNG.standard_normal(x.shape)
    assert abs((g * y).sum() - (oracle.rotate(g, pos, f, interleaved, True, 1.5) * x).sum()) < 1e-10
    assert np.allclose(oracle.rotate(y, pos, f, interleaved, True, 1 / 1.5), x)


def test_products_of_rotated_rows_depend_on_their_distance():
    q, k, f = RNG.standard_normal((1, 1, 8)), RNG.standard_normal((1, 1, 8)), np.array([1.0, 0.3, 0.02, 0.001])
    dots = [(oracle.rotate(q, [a], f) * oracle.rotate(k, [a - 5], f)).sum() for a in (5, 100, 12345)]
    assert np.allclose(dots, dots[0])


def test_append():
    """Two sequences; the second's first page has older rows, in a scale that suffices for one head only."""
    page, table = 4, [[2, 0], [1, 3]]
    codes, scale = np.full((5, 2, page, 3), 7.0), np.ones((5, 2))
    codes[1, :, :2] = [[[448.0, 0.0625, 2.0 ** -9]]]
    x = RNG.standard_normal((8, 2, 3))
    x[5, 1, 0] = 1000.0            # 2^2 * 448 >= 1000 > 2 * 448
    c, s = oracle.append_pages(x, [0, 5, 8], codes, scale, table, [5, 5], page)
    for i, h, rows, toks in ((2, 0, slice(0, 4), slice(0, 4)), (0, 1, slice(0, 1), slice(4, 5)), (3, 0, slice(0, 1), slice(7, 8))):
        assert s[i, h] == oracle.least_scale(np.abs(x[toks, h]).max())
        assert np.array_equal(c[i, h, rows], oracle.round_e4m3(x[toks, h] / s[i, h]))
    assert s[1, 0] == 1.0 and np.array_equal(c[1, 0, :2], codes[1, 0, :2])
    assert s[1, 1] == 4.0 and np.array_equal(c[1, 1, :2], [[112.0, 2.0 ** -6, 0.0]] * 2)
    assert np.array_equal(c[1, :, 2:], oracle.round_e4m3(x[5:7] / s[1][:, None]).transpose(1, 0, 2))
    assert (c[0, :, 1:] == 7).all() and (c[3, :, 1:] == 7).all() and (c[4] == 7).all() and (s[4] == 1).all()


def test_append_keeps_non_finite_values_apart():
    x = np.array([[[1.0, np.inf, np.nan, -2.0]]])
    c, s = oracle.append_pages(x, [0, 1], np.zeros((1, 1, 4, 4)), np.ones((1, 1)), [[0]], [1], 4)
    assert s[0, 0] == oracle.least_scale(2.0)
    assert np.array_equal(np.isnan(c[0, 0, 0]), [False, True, True, False]) and c[0, 0, 0, 3] == -256.0


@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_is_packed_attention_of_the_gathered_pages(causal):
    page, lens, cu = 4, [9, 0, 4], [0, 3, 4, 8]
    table = [[5, 1, 3], [-1, -1, -1], [2, 77, 77]]
    kc, vc = (oracle.round_e4m3(RNG.standard_normal((6, 2, page, 8)) * 50) for _ in range(2))
    ks, vs = RNG.random((6, 2)) + 0.1, RNG.random((6, 2)) + 0.1
    Q = RNG.standard_normal((8, 6, 8)) / 50
    O, L, A, _ = oracle.attention_paged(Q, kc, vc, ks, vs, table, lens, cu, 0.3, causal)
    k, v = (np.concatenate([(c * s[..., None, None])[i].transpose(1, 0, 2) for i in (5, 1, 3, 2)])
            for c, s in ((kc, ks), (vc, vs)))
    keep = list(range(9)) + list(range(12, 16))
    Or, Lr, Ar = oracle.attention_packed(Q, k[keep], v[keep], cu, [0, 9, 9, 13], 0.3, causal)
    assert np.allclose(O, Or) and np.allclose(L, Lr) and np.allclose(A, Ar)
