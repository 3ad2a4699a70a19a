"""fa_rope, fa_kv_append, fa_fwd_paged: argument checks on the host (CPU only; no address is dereferenced)."""
import math
import os
import subprocess
import sys

import pytest
import torch

from exact_io_aware_34_gb300 import build as fa_build
from exact_io_aware_34_gb300 import fa

A, GAP = 0x7F0000000000, 1 << 32
BAD, NO = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def strides(cls, st, names, dense):
    return None if st is None else (cls * len(names))(*[st.get(n, dense[n]) for n in names])


def rope(lib, st=None, **kw):
    a = {n: A + i * GAP for i, n in enumerate(("X", "XO", "Y", "YO", "pos", "f"))}
    a.update(h=8, hy=2, T=300, d=128, rot=64, il=0, tr=0, factor=1.0)
    a.update(kw)
    dense = {n: (a[h] * a["d"], a["d"]) for n, h in (("X", "h"), ("XO", "h"), ("Y", "hy"), ("YO", "hy"))}
    return lib.fa_rope(a["X"], a["XO"], a["h"], a["Y"], a["YO"], a["hy"], a["pos"], a["f"], a["T"], a["d"], a["rot"],
                       strides(fa.Strides, st, ("X", "XO", "Y", "YO"), dense), a["il"], a["tr"], a["factor"], None)


@pytest.mark.parametrize("kw,expect", [
    *[({n: 0}, BAD) for n in ("X", "XO", "Y", "YO", "pos", "f", "h", "T", "d", "rot")],
    (dict(hy=-1), BAD), (dict(rot=144), BAD), (dict(il=2), BAD), (dict(tr=-1), BAD), (dict(factor=INF), BAD),
    (dict(h=65536), BAD), (dict(T=1 << 29), BAD), (dict(rot=24), NO), (dict(d=72), NO), (dict(d=272), NO),
    (dict(X=A + 8), BAD), (dict(YO=A + 3 * GAP + 4), BAD), (dict(pos=A + 4 * GAP + 2), BAD), (dict(f=A + 5 * GAP + 4), BAD),
    (dict(XO=A + 256), BAD), (dict(XO=A + 2 * GAP), BAD), (dict(YO=A), BAD), (dict(YO=A + GAP), BAD),
    (dict(pos=A + GAP), BAD), (dict(f=A + 3 * GAP), BAD),
    (dict(XO=A, st={"XO": (2048, 128)}), BAD),          # its own input, with other strides
    (dict(st={"X": (1024, 4)}), BAD), (dict(st={"XO": (0, 128)}), BAD), (dict(st={"YO": (128, 128)}), BAD),
])
def test_rope_refusals(lib, kw, expect):
    assert rope(lib, **kw) == expect


@pytest.mark.parametrize("args", [(0, 1e4), (7, 1e4), (64, 0.0), (64, -1.0), (64, INF)])
def test_frequency_refusals(lib, args):
    with pytest.raises(fa.FaError):
        fa.fa_rope_frequencies(*args)
    assert lib.fa_rope_frequencies(None, 64, 1e4, 0, 1.0, 1.0, 2.0, 4096.0) == BAD


@pytest.mark.parametrize("kw", [dict(factor=0.0), dict(factor=INF), dict(scaling="turns", low_turns=0.0),
                                dict(scaling="turns", low_turns=2.0, high_turns=2.0),
                                dict(scaling="log_turns", original=0.0)])
def test_scaling_refusals(lib, kw):
    with pytest.raises(fa.FaError):
        fa.fa_rope_frequencies(64, **{"scaling": "linear", **kw})
    with pytest.raises(ValueError):
        fa.fa_rope_frequencies(64, scaling="other")


def test_frequencies(lib):
    rot, base = 96, 5e5
    plain = [base ** (-2 * j / rot) for j in range(48)]
    assert torch.allclose(fa.fa_rope_frequencies(rot, base), torch.tensor(plain, dtype=torch.float64), rtol=1e-14)
    slow = fa.fa_rope_frequencies(rot, base, "linear", 8.0)
    assert torch.allclose(slow * 8, torch.tensor(plain, dtype=torch.float64), rtol=1e-14)
    for scaling, g in (("turns", lambda r: r), ("log_turns", math.log)):
        got = fa.fa_rope_frequencies(rot, base, scaling, 8.0, 1.5, 20.0, 8192).tolist()
        kinds = set()
        for f, x in zip(plain, got):
            r = 8192 * f / (2 * math.pi)
            w = min(1.0, max(0.0, (g(r) - g(1.5)) / (g(20.0) - g(1.5))))
            assert math.isclose(x, w * f + (1 - w) * f / 8, rel_tol=1e-13)
            kinds.add(0 if w == 0 else 2 if w == 1 else 1)
        assert kinds == {0, 1, 2}


ROWS = ("K", "V", "Q", "QO")


def append(lib, st=None, cst=None, **kw):
    names = ("K", "V", "cu", "KC", "VC", "ks", "vs", "tab", "lens", "Q", "QO", "f", "pos")
    a = {n: A + i * GAP for i, n in enumerate(names)}
    a.update(B=3, H=8, Hk=2, T=50, d=128, n=40, page=32, m=9, rot=128, il=0, factor=1.0)
    a.update(kw)
    dense = {n: (a[h] * a["d"], a["d"]) for n, h in zip(ROWS, ("Hk", "Hk", "H", "H"))}
    pages = (a["Hk"] * a["page"] * a["d"], a["page"] * a["d"], a["d"])
    return lib.fa_kv_append(*[a[n] for n in names], a["B"], a["H"], a["Hk"], a["T"], a["d"], a["n"], a["page"], a["m"],
                            a["rot"], strides(fa.Strides, st, ROWS, dense),
                            strides(fa.PageStrides, cst, ("KC", "VC"), {"KC": pages, "VC": pages}), a["il"], a["factor"], None)


@pytest.mark.parametrize("kw,expect", [
    *[({n: 0}, BAD) for n in ("K", "V", "cu", "KC", "VC", "ks", "vs", "tab", "lens", "QO", "f", "B", "H", "Hk", "T", "d",
                              "n", "page", "m")],
    (dict(rot=0), BAD),                                  # queries, but nothing to rotate by
    (dict(rot=-16), BAD), (dict(rot=144), BAD), (dict(il=2), BAD), (dict(factor=INF), BAD),
    (dict(B=(1 << 20) + 1), BAD), (dict(n=1 << 30), BAD), (dict(m=1 << 27), BAD), (dict(T=1 << 30), BAD),
    (dict(rot=40), NO), (dict(d=96), NO), (dict(page=8), NO), (dict(page=48), NO), (dict(page=256), NO),
    (dict(K=A + 2), BAD), (dict(KC=A + 3 * GAP + 8), BAD), (dict(ks=A + 5 * GAP + 2), BAD), (dict(lens=A + 8 * GAP + 1), BAD),
    (dict(f=A + 11 * GAP + 4), BAD), (dict(pos=A + 12 * GAP + 2), BAD),
    (dict(VC=A + 3 * GAP), BAD), (dict(vs=A + 5 * GAP), BAD), (dict(ks=A + 3 * GAP), BAD), (dict(K=A + 3 * GAP), BAD),
    (dict(tab=A + 5 * GAP), BAD), (dict(QO=A), BAD), (dict(QO=A + 4 * GAP), BAD), (dict(QO=A + 9 * GAP + 256), BAD),
    (dict(pos=A + 10 * GAP), BAD), (dict(cu=A + 4 * GAP), BAD), (dict(f=A + 6 * GAP), BAD),
    (dict(st={"K": (256, 4)}), BAD), (dict(cst={"KC": (8192, 4096, 8)}), BAD), (dict(cst={"VC": (4096, 4096, 128)}), BAD),
    (dict(cst={"KC": (-8192, 4096, 128)}), BAD),
    # parts of one buffer that share a row
    (dict(VC=A + 3 * GAP + 4096, cst={"KC": (16384, 4096, 128), "VC": (16384, 4096, 128)}), BAD),
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == expect


def paged(lib, st=None, cst=None, **kw):
    names = ("Q", "KC", "VC", "ks", "vs", "tab", "lens", "cu", "O", "L")
    a = {n: A + i * GAP for i, n in enumerate(names)}
    a.update(B=3, H=8, Hk=2, T=50, d=128, n=40, page=32, m=9, scale=0.1, causal=1, ws=A + 20 * GAP, wn=1 << 31)
    a.update(kw)
    dense = {n: (a["H"] * a["d"], a["d"]) for n in ("Q", "O")}
    pages = (a["Hk"] * a["page"] * a["d"], a["page"] * a["d"], a["d"])
    return lib.fa_fwd_paged(*[a[n] for n in names], a["B"], a["H"], a["Hk"], a["T"], a["d"], a["n"], a["page"], a["m"],
                            strides(fa.Strides, st, ("Q", "O"), dense),
                            strides(fa.PageStrides, cst, ("KC", "VC"), {"KC": pages, "VC": pages}), a["scale"],
                            a["causal"], a["ws"], a["wn"], None)


PAGED_REFUSALS = [
    *[({n: 0}, BAD) for n in ("Q", "KC", "VC", "ks", "vs", "tab", "lens", "cu", "O", "L", "B", "H", "Hk", "T", "d", "n",
                              "page", "m")],
    (dict(H=7), BAD), (dict(scale=INF), BAD), (dict(causal=2), BAD), (dict(m=1 << 27), BAD), (dict(T=1 << 29), BAD),
    (dict(d=32), NO), (dict(page=20), NO), (dict(H=258), NO),
    (dict(Q=A + 8), BAD), (dict(VC=A + 2 * GAP + 4), BAD), (dict(ks=A + 3 * GAP + 1), BAD), (dict(L=A + 9 * GAP + 2), BAD),
    (dict(O=A), BAD), (dict(O=A + GAP), BAD), (dict(L=A + 2 * GAP), BAD), (dict(L=A + 8 * GAP), BAD), (dict(L=A + 5 * GAP), BAD),
    (dict(O=A + 7 * GAP), BAD), (dict(st={"O": (128, 128)}), BAD), (dict(cst={"KC": (8192, 4096, 24)}), BAD),
    (dict(ws=0), BAD), (dict(ws=A + 20 * GAP + 64), BAD), (dict(wn=1000), BAD), (dict(ws=A), BAD), (dict(ws=A + 2 * GAP), BAD),
    (dict(ws=A + 8 * GAP), BAD), (dict(ws=A + 9 * GAP), BAD), (dict(ws=A + 5 * GAP), BAD),
    # more places than are counted in 32 bits
    (dict(B=1 << 20, T=1 << 20, m=1 << 20, n=9, Hk=1, H=1, page=128), NO),
]


@pytest.mark.parametrize("kw,expect", PAGED_REFUSALS)
def test_paged_refusals(lib, kw, expect):
    assert paged(lib, **kw) == expect


def test_workspace_of_rejected_sizes_is_zero(lib):
    size = fa.fa_fwd_paged_workspace_bytes
    for bad in [(0, 8, 2, 1, 128, 9, 16, 9), (1, 8, 3, 1, 128, 9, 16, 9), (1, 8, 2, 0, 128, 9, 16, 9), (1, 8, 2, 1, 96, 9, 16, 9),
                (1, 8, 2, 1, 128, 9, 20, 9), (1, 258, 2, 1, 128, 9, 16, 9), (1, 8, 2, 1, 128, 0, 16, 9)]:
        assert size(*bad) == 0
    assert size(1 << 20, 1, 1, 1 << 20, 128, 9, 128, 1 << 20) == 0
    need = size(3, 8, 2, 50, 128, 40, 32, 9)
    assert need > 0 and paged(lib, wn=need - 1) == BAD


def test_most_rows(lib):
    """T_q * H up to 2^31 - 2: the merge's row numbers stay below 2^31, with a step of 64 behind the last within 32 bits."""
    size, rows = fa.fa_fwd_paged_workspace_bytes, (1 << 30) - 1
    assert size(1, 2, 1, rows, 64, 9, 16, 9) > 0 and size(1, 2, 1, rows + 1, 64, 9, 16, 9) == 0
    assert 2 * rows - 1 + 64 < 1 << 32


def test_fault_hook_rejects_zero_timeout(lib):
    assert lib.fa_fwd_paged_fault_test(*[A + i * GAP for i in range(10)], 1, 1, 1, 1, 64, 9, 16, 1, 0.1, 0, A + 20 * GAP,
                                       1 << 30, 0, 0, None) == BAD


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pages = torch.zeros(2, 2, 16, 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(2, 2)
    with pytest.raises(ValueError):
        fa.fa_rope(x, i, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        fa.fa_kv_append(x, x, i, pages, pages, s, s, i[None], i)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(x, pages, pages, s, s, i[None], i, i)


def test_imports_with_a_torch_built_without_cuda():
    """Such a build has no torch._C._cuda_* functions."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "from exact_io_aware_34_gb300 import fa\n"
            "x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)\n"
            "try: fa.fa_rope(x, torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))\n"
            "except ValueError: print('refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "refused", out.stderr
