"""fa_fwd_prefix: argument checks on the host (CPU only; no address is dereferenced)."""
import pytest
import torch

from exact_io_aware_34_gb300 import build as fa_build
from exact_io_aware_34_gb300 import fa

A, GAP = 0x7F0000000000, 1 << 32
BAD, NO = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def call(lib, st=None, **kw):
    names = ("Q", "Kp", "Vp", "K", "V", "lens", "O", "L")
    a = {n: A + i * GAP for i, n in enumerate(names)}
    a.update(B=3, H=8, H_kv=2, Nq=2, Np=500, room=300, d=128, scale=0.1, causal=1, ws=A + 20 * GAP, n=1 << 31)
    a.update(kw)
    if st is not None:
        dense = {}
        for n, (h, r) in dict(Q=("H", "Nq"), Kp=("H_kv", "Np"), Vp=("H_kv", "Np"), K=("H_kv", "room"),
                              V=("H_kv", "room"), O=("H", "Nq")).items():
            dense[n] = (a[h] * a[r] * a["d"], a[r] * a["d"], a["d"])
        st = (fa.BatchStrides * 6)(*[st.get(n, dense[n]) for n in ("Q", "Kp", "Vp", "K", "V", "O")])
    return lib.fa_fwd_prefix(*[a[n] for n in names], a["B"], a["H"], a["H_kv"], a["Nq"], a["Np"], a["room"], a["d"],
                             st, a["scale"], a["causal"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,expect", [
    *[({n: 0}, BAD) for n in ("Q", "Kp", "Vp", "K", "V", "lens", "O", "L", "ws", "B", "H", "H_kv", "Nq", "room", "d")],
    (dict(Np=-1), BAD), (dict(H=7), BAD), (dict(B=1 << 16), BAD), (dict(H=1 << 17, H_kv=1 << 17), BAD),
    (dict(room=1 << 30), BAD), (dict(Np=1 << 30), BAD), (dict(causal=2), BAD), (dict(scale=float("inf")), BAD),
    (dict(d=32), NO), (dict(Nq=129), NO), (dict(H=258, H_kv=2), NO),
    (dict(Q=A + 8), BAD), (dict(Kp=A + GAP + 8), BAD), (dict(V=A + 4 * GAP + 2), BAD), (dict(O=A + 6 * GAP + 4), BAD),
    (dict(lens=A + 5 * GAP + 2), BAD), (dict(L=A + 7 * GAP + 1), BAD), (dict(ws=A + 20 * GAP + 16), BAD),
    (dict(n=1000), BAD), (dict(O=A), BAD), (dict(O=A + GAP), BAD), (dict(L=A + 3 * GAP), BAD), (dict(ws=A + 2 * GAP), BAD),
    (dict(ws=A + 6 * GAP), BAD), (dict(L=A + 6 * GAP), BAD), (dict(lens=A + 6 * GAP), BAD),
    (dict(st={"Q": (2048, 256, 4)}), BAD), (dict(st={"K": (-8, 128, 128)}), BAD), (dict(st={"V": (1 << 36, 8, 8)}), BAD),
    (dict(st={"O": (2048, 128, 128)}), BAD),        # two rows of O share memory
    (dict(st={"O": (0, 256, 128)}), BAD),
])
def test_refusals(lib, kw, expect):
    assert call(lib, **kw) == expect


def test_workspace_sizes(lib):
    size = fa.fa_fwd_prefix_workspace_bytes
    assert size(3, 8, 2, 2, 500, 300, 128) > size(3, 8, 2, 2, 0, 300, 128) > 0
    for bad in [(0, 8, 2, 1, 1, 1, 128), (1, 8, 3, 1, 1, 1, 128), (1, 8, 2, 129, 1, 1, 128), (1, 8, 2, 1, -1, 1, 128),
                (1, 8, 2, 1, 1, 0, 128), (1, 8, 2, 1, 1, 1, 96)]:
        assert size(*bad) == 0
    assert call(lib, n=size(3, 8, 2, 2, 500, 300, 128) - 1) == BAD


def test_fault_hook_rejects_zero_timeout(lib):
    assert lib.fa_fwd_prefix_fault_test(*[A + i * GAP for i in range(8)], 1, 1, 1, 1, 8, 8, 128, 0.1, 0, A + 20 * GAP,
                                        1 << 30, 0, 0, None) == BAD


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_fwd_prefix(x, None, None, x, x, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.fa_fwd_prefix(None, None, None, x, x, torch.zeros(1, dtype=torch.int32))


def test_lengths_whose_blocks_are_not_counted_in_32_bits_are_refused(lib):
    size, most = fa.fa_fwd_prefix_workspace_bytes, (1 << 31) - (1 << 16)
    for kw in (dict(Np=most + 1), dict(room=most + 1), dict(Np=(1 << 31) - 1), dict(room=(1 << 31) - 1)):
        kw.update(B=1, H=1, H_kv=1, Nq=1)
        assert call(lib, **kw) == BAD
        assert size(1, 1, 1, 1, kw.get("Np", 1), kw.get("room", 1), 64) == 0
    assert size(1, 1, 1, 1, most, 1, 64) > 0


def test_workspace_of_rejected_sizes_is_zero(lib):
    """More blocks in all than are counted: every sequence has three places of its own per head beside the prefix's."""
    assert fa.fa_fwd_prefix_workspace_bytes(65535, 32768, 32768, 1, 0, 1, 64) == 0
    assert call(lib, B=65535, H=32767, H_kv=32767, Nq=1, Np=0, room=1) == NO
    assert fa.fa_fwd_prefix_workspace_bytes(65535, 32767, 32767, 1, 0, 1, 64) == 0
