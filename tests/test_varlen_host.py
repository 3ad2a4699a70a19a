"""Packed-sequence entry points: argument checks on the host (CPU only). The
addresses are never dereferenced: every call is rejected before any CUDA call."""
import pytest
import torch

from exact_io_aware_34_gb300 import build as fa_build
from exact_io_aware_34_gb300 import fa

A, GAP = 0x7F0000000000, 1 << 30


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def fwd(lib, q_st=None, k_st=None, v_st=None, o_st=None, **kw):
    a = dict(Q=A, K=A + GAP, V=A + 2 * GAP, O=A + 3 * GAP, L=A + 4 * GAP, cq=A + 5 * GAP, ck=A + 6 * GAP, B=2, H=8,
             H_kv=2, Tq=100000, Tk=200, d=128, scale=0.1, causal=1, ws=A + 7 * GAP, n=1 << 20)
    a.update(kw)
    st = None
    if q_st or k_st or v_st or o_st:
        dense = [(a["H"] * a["d"], a["d"]), (a["H_kv"] * a["d"], a["d"])]
        st = (fa.Strides * 4)(q_st or dense[0], k_st or dense[1], v_st or dense[1], o_st or dense[0])
    return lib.fa_fwd_varlen(a["Q"], a["K"], a["V"], a["O"], a["L"], a["cq"], a["ck"], a["B"], a["H"], a["H_kv"],
                             a["Tq"], a["Tk"], a["d"], st, a["scale"], a["causal"], a["ws"], a["n"], None)


BAD, NO = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    *[({n: 0}, BAD) for n in ("Q", "K", "V", "O", "L", "cq", "ck", "ws", "B", "H", "H_kv", "Tq", "Tk", "d")],
    (dict(H=7), BAD), (dict(H=1 << 16, H_kv=1 << 16), BAD), (dict(B=(1 << 24) + 1), BAD),
    (dict(Tq=1 << 28), BAD), (dict(Tk=1 << 30), BAD), (dict(causal=2), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(d=96), NO), (dict(H=258, H_kv=2), NO),
    (dict(Q=A + 8), BAD), (dict(O=A + 3 * GAP + 2), BAD), (dict(L=A + 4 * GAP + 2), BAD),
    (dict(cq=A + 5 * GAP + 1), BAD), (dict(ws=A + 7 * GAP + 64), BAD), (dict(n=100), BAD),
    (dict(O=A), BAD), (dict(O=A + GAP + 256), BAD), (dict(L=A + 2 * GAP), BAD), (dict(ws=A + 3 * GAP), BAD),
    (dict(ws=A + 4 * GAP), BAD), (dict(cq=A + 3 * GAP), BAD), (dict(ck=A + 4 * GAP), BAD), (dict(ck=A + 7 * GAP), BAD),
    (dict(q_st=(1024, 132)), BAD), (dict(q_st=(-1024, 128)), BAD), (dict(k_st=(0, 128)), BAD),
    (dict(v_st=(1 << 39, 128)), BAD), (dict(o_st=(512, 128)), BAD),         # O's rows would share memory
    (dict(o_st=(128, 128 * 99)), BAD),
    # O as columns of the buffer that holds Q, overlapping Q's last head
    (dict(q_st=(2048, 128), o_st=(2048, 128), O=A + 2 * 7 * 128), BAD),
])
def test_forward_refusals(lib, kw, expect):
    assert fwd(lib, **kw) == expect


def bwd(lib, st=None, **kw):
    names = ("Q", "K", "V", "O", "dO", "L", "dQ", "dK", "dV", "cq", "ck")
    a = {n: A + i * GAP for i, n in enumerate(names)}
    a.update(B=2, H=8, H_kv=2, Tq=100, Tk=200, d=128, scale=0.1, causal=1, ws=A + 20 * GAP, n=1 << 24)
    a.update(kw)
    if st is not None:
        dense = [(a["H"] * a["d"], a["d"]), (a["H_kv"] * a["d"], a["d"])]
        st = (fa.Strides * 8)(*[st.get(n, dense[n in ("K", "V", "dK", "dV")])
                                for n in ("Q", "K", "V", "O", "dO", "dQ", "dK", "dV")])
    return lib.fa_bwd_varlen(*[a[n] for n in names], a["B"], a["H"], a["H_kv"], a["Tq"], a["Tk"], a["d"], st,
                             a["scale"], a["causal"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,expect", [
    *[({n: 0}, BAD) for n in ("Q", "K", "V", "O", "dO", "L", "dQ", "dK", "dV", "cq", "ck", "ws", "B", "H", "Tq", "Tk")],
    (dict(H=7), BAD), (dict(d=80), NO), (dict(H=258, H_kv=2), NO), (dict(causal=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(n=1000), BAD), (dict(ws=A + 20 * GAP + 16), BAD),
    (dict(dQ=A), BAD), (dict(dK=A + GAP), BAD), (dict(dV=A + 3 * GAP), BAD), (dict(dK=A + 8 * GAP), BAD),
    (dict(dV=A + 5 * GAP), BAD), (dict(dQ=A + 9 * GAP), BAD), (dict(ws=A + 4 * GAP), BAD), (dict(ws=A + 10 * GAP), BAD),
    (dict(st={"dQ": (512, 128)}), BAD), (dict(st={"dO": (1024, 4)}), BAD),
    # dK and dV as columns of one buffer [200, 4, 128], one head apart: they share a column
    (dict(st={"dK": (512, 128), "dV": (512, 128)}, dK=A + 30 * GAP, dV=A + 30 * GAP + 256), BAD),
])
def test_backward_refusals(lib, kw, expect):
    assert bwd(lib, **kw) == expect


def test_workspace_sizes(lib):
    def need(B=1, H=8, H_kv=2, Tq=99999, Tk=1, d=64):
        return fa.fa_fwd_varlen_workspace_bytes(B, H, H_kv, Tq, Tk, d)

    assert need(Tq=1) == 0 and need(Tq=1, Tk=1536) == 0      # every unit at once, few keys: no list
    assert 0 < need(Tq=1, Tk=1537) < need(Tq=1, Tk=100000) < need(Tq=1, Tk=100000, d=128) < 42e6
    assert need() > 0 and need(Tk=100000) == need()
    assert need(H=32, H_kv=4, Tq=1024, Tk=2048) == 0 < need(B=2, H=32, H_kv=4, Tq=512, Tk=2048)   # one that fills the device
    for bad in [dict(B=0), dict(H_kv=3), dict(H_kv=0), dict(H=258), dict(Tq=0), dict(Tk=0), dict(d=96)]:
        assert need(**bad) == 0
    assert fa.fa_bwd_varlen_workspace_bytes(1, 8, 2, 1, 1) > 0
    for bad in [(0, 8, 2, 1, 1), (1, 8, 3, 1, 1), (1, 258, 2, 1, 1), (1, 8, 2, 0, 1), (1, 8, 2, 1, 0)]:
        assert fa.fa_bwd_varlen_workspace_bytes(*bad) == 0
    assert bwd(lib, n=fa.fa_bwd_varlen_workspace_bytes(2, 8, 2, 100, 200) - 1) == BAD
    assert fwd(lib, n=fa.fa_fwd_varlen_workspace_bytes(2, 8, 2, 100000, 200, 128) - 1) == BAD
    assert fwd(lib, Tq=100, Tk=2000, n=fa.fa_fwd_varlen_workspace_bytes(2, 8, 2, 100, 2000, 128) - 1) == BAD
    assert fwd(lib, Tq=100, Tk=2000, ws=0) == BAD


def test_fault_hook_rejects_zero_timeout(lib):
    assert lib.fa_fwd_varlen_fault_test(A, A + GAP, A + 2 * GAP, A + 3 * GAP, A + 4 * GAP, A + 5 * GAP, A + 6 * GAP, 1,
                                        1, 1, 8, 8, 128, 0.1, 1, A + 7 * GAP, 1 << 20, 0, 0, None) == BAD
    assert lib.fa_bwd_varlen_fault_test(*[A + i * GAP for i in range(11)], 1, 1, 1, 8, 8, 128, 0.1, 1, A + 20 * GAP,
                                        1 << 24, 0, 0, None) == BAD


def test_binding_refuses_cpu_tensors():
    x, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_fwd_varlen(x, x, x, cu, cu)
    with pytest.raises(ValueError):
        fa.fa_fwd_varlen(None, x, x, cu, cu)


def test_a_causal_prompt_that_gains_by_split_keys_has_room_for_them(lib):
    """Units that nearly fill the device: the workspace size covers the causal call, which is split."""
    need = fa.fa_fwd_varlen_workspace_bytes
    for H, H_kv, T, d in ((8, 2, 4096, 128), (8, 8, 4096, 128), (8, 2, 4096, 64)):
        n = need(1, H, H_kv, T, T, d)
        assert 0 < n < 42e6
        assert fwd(lib, B=1, H=H, H_kv=H_kv, Tq=T, Tk=T, d=d, n=n - 1) == BAD
        assert fwd(lib, B=1, H=H, H_kv=H_kv, Tq=T, Tk=T, d=d, ws=0, n=0) == BAD
    for H, H_kv, T in ((16, 4, 2048), (16, 16, 2048), (16, 4, 2300), (32, 4, 1100)):
        assert need(1, H, H_kv, T, T, 128) == 0


LONG = (1 << 31) - (1 << 16)


def test_lengths_whose_blocks_are_not_counted_in_32_bits_are_refused(lib):
    for kw in (dict(Tq=LONG + 1), dict(Tk=LONG + 1), dict(Tq=(1 << 31) - 1), dict(Tk=(1 << 31) - 1)):
        kw.update(B=1, H=1, H_kv=1)
        assert fwd(lib, **kw) == BAD and bwd(lib, **kw) == BAD
        assert fa.fa_fwd_varlen_workspace_bytes(1, 1, 1, kw.get("Tq", 1), kw.get("Tk", 1), 64) == 0
        assert fa.fa_bwd_varlen_workspace_bytes(1, 1, 1, kw.get("Tq", 1), kw.get("Tk", 1)) == 0
    assert fa.fa_fwd_varlen_workspace_bytes(1, 1, 1, LONG, LONG, 64) > 0


def test_workspace_of_rejected_sizes_is_zero(lib):
    fwd_bytes, bwd_bytes = fa.fa_fwd_varlen_workspace_bytes, fa.fa_bwd_varlen_workspace_bytes
    for B, H, H_kv, Tq, Tk in (((1 << 24) + 1, 8, 2, 9, 9), (1, 1 << 16, 1 << 16, 9, 9), (1, 8, 2, 1 << 28, 9),
                               (1, 8, 2, 9, 1 << 30), (1 << 24, 4096, 4096, 9, 9)):
        assert fwd_bytes(B, H, H_kv, Tq, Tk, 64) == 0 and bwd_bytes(B, H, H_kv, Tq, Tk) == 0
    assert fwd(lib, B=1 << 24, H=4096, H_kv=4096, Tq=9, Tk=9) == NO
    assert bwd(lib, B=1 << 24, H=4096, H_kv=4096, Tq=9, Tk=9) == NO
