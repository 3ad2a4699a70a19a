"""fa_rope against the float64 oracle, through the C ABI (needs a GB300).

Tolerance: the angle's fraction of a turn is cut to 2^-32 and rounded to 24
bits of at most half a turn (2^-24 pi), sincospif is good to about 2^-24 of 1,
the two products and their sum round by 2^-24 each: together below 2^-21
f (|a| + |b|); then one rounding to bf16, 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_34_gb300 import fa
from tests import parity
from tests.test_gpu_varlen import draw, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_34_gb300 import build
    build.build()
    fa.load_library()


def check_rows(got, x, pos, freq, factor=1.0, **kw):
    """got and x [T, heads, d] (torch, CPU or CUDA)."""
    X, f = parity.to64(x), freq.cpu().numpy()
    want = oracle.rotate(X, pos, f, factor=factor, **kw)
    size = np.abs(X)
    half = len(f)
    a = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if kw.get("interleaved") else (slice(0, half), slice(half, 2 * half))
    size[..., a[0]] = size[..., a[1]] = abs(factor) * (size[..., a[0]] + size[..., a[1]])
    err = np.abs(parity.to64(got) - want)
    assert np.array_equal(parity.to64(got)[..., 2 * half:], X[..., 2 * half:])
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size + 1e-38
    assert (err <= tol).all(), float((err / tol).max())


def pos_of(p):
    return torch.as_tensor(p, dtype=torch.int32).cuda()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32), (64, 16), (96, 48), (256, 256), (16, 16), (240, 224)])
def test_layouts_and_parts(d, rot, interleaved, transpose):
    T = 61
    x, y = draw(d + rot, (T, 5, d), (T, 2, d))
    pos = np.arange(T) * 37 + 5
    f = fa.fa_rope_frequencies(rot, device="cuda")
    kw = dict(interleaved=interleaved, transpose=transpose)
    a, b = fa.fa_rope(x.cuda(), pos_of(pos), f, y=y.cuda(), factor=1.1, **kw)
    ok()
    check_rows(a, x, pos, f, 1.1, **kw)
    check_rows(b, y, pos, f, 1.1, **kw)


@pytest.mark.parametrize("T,heads", [(1, 1), (1, 32), (2, 3), (3, 128), (5000, 7), (2433, 40), (9001, 1)])
def test_sizes(T, heads):
    x, = draw(T + heads, (T, heads, 128))
    f = fa.fa_rope_frequencies(128, device="cuda")
    got = fa.fa_rope(x.cuda(), pos_of(np.arange(T)), f)
    ok()
    check_rows(got, x, np.arange(T), f)


def test_far_and_negative_positions():
    """The angle stays exact where float32 products of position and frequency are off by many turns."""
    pos = np.array([0, 1, -1, 10 ** 6 + 3, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321])
    x, = draw(3, (8, 4, 64))
    f = fa.fa_rope_frequencies(64, 5e5, "log_turns", 16.0, 1.0, 32.0, 8192, device="cuda")
    got = fa.fa_rope(x.cuda(), pos_of(pos), f)
    ok()
    check_rows(got, x, pos, f)


def test_frequencies_of_a_turn_and_more_and_of_zero():
    f = torch.tensor([0.0, 2 * np.pi, 7.0, 100.25, 1e-12, 3.0, 6.28, 0.5], dtype=torch.float64).cuda()
    x, = draw(4, (50, 2, 16))
    pos = np.arange(50)
    got = fa.fa_rope(x.cuda(), pos_of(pos), f)
    ok()
    check_rows(got, x, pos, f)


def test_gradient_against_differences():
    """<g, rope(x + h) - rope(x)> = <rope^T(g), h>: the map is linear. Each side is off by
    what its results' roundings to bf16 (2^-8 of each) amount to."""
    g, x, h = draw(5, (33, 4, 64), (33, 4, 64), (33, 4, 64))
    f = fa.fa_rope_frequencies(32, device="cuda")
    pos = pos_of(np.arange(33) + 100)
    r = lambda t, **kw: parity.to64(fa.fa_rope(t.cuda(), pos, f, factor=1.25, **kw))  # noqa: E731
    moved = (x.float() + h.float()).to(torch.bfloat16)
    G, H = parity.to64(g), parity.to64(moved) - parity.to64(x)          # the step that was taken
    a, b, c = r(moved), r(x), r(g, transpose=True)
    ok()
    bound = 2.0 ** -8 * 1.01 * ((np.abs(G) * (np.abs(a) + np.abs(b))).sum() + (np.abs(H) * np.abs(c)).sum())
    assert abs((G * (a - b)).sum() - (c * H).sum()) <= bound
    # and entry by entry against differences of the formula in float64
    e = np.zeros((33, 1, 64))
    X, F, P = parity.to64(x)[:, :1], f.cpu().numpy(), np.arange(33) + 100
    for j in (0, 5, 16, 31, 40):
        e[..., j] = 1.0
        d = oracle.rotate(X + e, P, F, factor=1.25) - oracle.rotate(X - e, P, F, factor=1.25)
        want = (G[:, :1] * d / 2).sum(-1)
        e[..., j] = 0.0
        assert (np.abs(c[:, :1, j] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(G).max()).all()


def test_slices_of_a_projection_and_in_place():
    T, H, Hk, d = 77, 6, 2, 128
    qkv, = draw(6, (T, H + 2 * Hk, d))
    pos, f = np.arange(T) + 9, fa.fa_rope_frequencies(128, device="cuda")
    buf = qkv.cuda()
    q, k = fa.fa_rope(buf[:, :H], pos_of(pos), f, y=buf[:, H:H + Hk])
    ok()
    assert torch.equal(buf.cpu(), qkv)
    check_rows(q, qkv[:, :H], pos, f)
    check_rows(k, qkv[:, H:H + Hk], pos, f)
    fa.fa_rope(buf[:, :H], pos_of(pos), f, y=buf[:, H:H + Hk], out=buf[:, :H], out_y=buf[:, H:H + Hk])
    ok()
    assert torch.equal(buf[:, :H], q) and torch.equal(buf[:, H:H + Hk], k) and torch.equal(buf[:, H + Hk:].cpu(), qkv[:, H + Hk:])
    # head-major storage, into the middle of a wider buffer
    flip = qkv.cuda().transpose(0, 1).contiguous().transpose(0, 1)[:, :H]
    wide = torch.full((T, H + 2, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_rope(flip, pos_of(pos), f, out=wide[:, 1:-1, :d])
    ok()
    assert torch.equal(wide[:, 1:-1, :d], q)
    wide[:, 1:-1, :d] = 3.0
    assert (wide == 3.0).all()


def test_graph_replay_and_side_stream():
    x, = draw(7, (40, 4, 64))
    f, pos = fa.fa_rope_frequencies(64, device="cuda"), pos_of(np.arange(40))
    dx, out = x.cuda(), torch.empty_like(x, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fa.fa_rope(dx, pos, f, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(dx, pos, f, out=out)
    graph.replay()
    ok()
    assert torch.equal(out, got)
    pos += 1000
    graph.replay()
    ok()
    check_rows(out, x, np.arange(40) + 1000, f)


def test_beyond_32_bit_offsets():
    """More than 2^31 elements between the first row and the last."""
    T, heads, d = 70000, 2, 64
    buf = torch.zeros(T, 40000, dtype=torch.bfloat16, device="cuda")
    x = buf[:, 1024:1024 + heads * d].unflatten(1, (heads, d))
    rows, = draw(8, (T, heads, d))
    x.copy_(rows)
    f, pos = fa.fa_rope_frequencies(d, device="cuda"), np.arange(T)
    got = fa.fa_rope(x, pos_of(pos), f)
    ok()
    check_rows(got[-300:], rows[-300:], pos[-300:], f)
    check_rows(got[:300], rows[:300], pos[:300], f)
    fa.fa_rope(x, pos_of(pos), f, out=x)
    ok()
    assert torch.equal(x, got)


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    f, pos = fa.fa_rope_frequencies(64, device="cuda"), pos_of(np.arange(4))
    for bad in (dict(positions=pos[:3]), dict(positions=pos.long()), dict(inv_freq=f.float()), dict(inv_freq=f.cpu()),
                dict(y=x[:3]), dict(out_y=x), dict(out=x[:, :1]), dict(x=x.float()), dict(x=x[..., ::2])):
        with pytest.raises(ValueError):
            fa.fa_rope(**{"x": x, "positions": pos, "inv_freq": f, **bad})
    with pytest.raises(fa.FaError):
        fa.fa_rope(x, pos, f[:4])                 # rot = 8
    with pytest.raises(fa.FaError):
        fa.fa_rope(x[:, :1].expand(4, 2, 64), pos, f)
