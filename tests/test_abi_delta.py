"""Host-side refusals of the delta rule's and the q, k norms' C entries: every bad call returns its
status before anything is launched (no device needed)."""
import ctypes as C
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
P = C.c_void_p(1 << 20)                                   # an aligned address; never read on the host


@pytest.fixture(scope="module")
def L():
    from learnable_kv_token_b200 import build
    build.build()
    from learnable_kv_token_b200 import lte
    return lte


def dims(L, **c):
    d = dict(B=2, T=100, H=4, Hk=2, dk=128, dv=64, scale=0.1, dtype=L.LTE_BF16)
    return L.make_gdr_dims(**{**d, **c})


def prefill(L, d, ws_bytes=None, **c):
    a = dict(q=P, k=P, v=P, qs=None, ks=None, vs=None, g=P, beta=P, lens=None, s_in=None, o=P, os=None, s_out=P,
             ws=P)
    a.update(c)
    n = L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_PREFILL) if ws_bytes is None else ws_bytes
    return L._lib.lte_gdr_prefill(C.byref(d), *a.values(), n, None)


def backward(L, d, ws_bytes=None, **c):
    a = dict(q=P, k=P, v=P, qs=None, ks=None, vs=None, g=P, beta=P, lens=None, s_in=None, do=P, dos=None, ds=None,
             dq=P, dk=P, dv=P, dg=P, db=P, ds_in=None, ws=P)
    a.update(c)
    n = L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_BACKWARD) if ws_bytes is None else ws_bytes
    return L._lib.lte_gdr_backward(C.byref(d), *a.values(), n, None)


@pytest.mark.parametrize("bad,status", [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(H=3), INVALID),
                                        (dict(Hk=0), INVALID), (dict(dtype=7), INVALID),
                                        (dict(scale=float("nan")), INVALID), (dict(dk=96), UNSUPPORTED),
                                        (dict(dv=256), UNSUPPORTED), (dict(B=1 << 20, H=1 << 10, Hk=1), UNSUPPORTED)])
def test_dims(L, bad, status):
    d = dims(L, **bad)
    assert L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_PREFILL) == 0
    assert L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_BACKWARD) == 0
    assert prefill(L, d, 1 << 40) == status
    assert backward(L, d, 1 << 40) == status
    if "T" not in bad:
        assert L._lib.lte_gdr_decode_step(C.byref(d), P, P, P, P, P, P, P, None) == status
    null = [None, P, P, P, None, None, None, P, P, None, None, P, None, P, P, 1 << 40, None]
    assert L._lib.lte_gdr_prefill(*null) == INVALID


def test_pointers_strides_and_workspace(L):
    d, odd = dims(L), C.c_void_p((1 << 20) + 8)
    for n in ("q", "k", "v", "g", "beta", "o", "s_out"):
        assert prefill(L, d, **{n: None}) == INVALID, n
    for n in ("q", "k", "v", "o", "s_in", "s_out", "ws"):
        assert prefill(L, d, **{n: odd}) == INVALID, n
    for n in ("q", "k", "v", "g", "beta", "do", "dq", "dk", "dv", "dg", "db"):
        assert backward(L, d, **{n: None}) == INVALID, n
    for n in ("q", "do", "ds", "dq", "ds_in", "ws"):
        assert backward(L, d, **{n: odd}) == INVALID, n
    for s in ((100, 4, 128), (1 << 20, 257, 128), (1 << 20, 512, -128)):     # not whole 16-byte pieces; negative
        st = C.byref(L.lte_strides(*s))
        for n in ("qs", "ks", "vs", "os"):
            assert prefill(L, d, **{n: st}) == INVALID
        assert backward(L, d, dos=st) == INVALID
    need = L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_PREFILL)
    assert need > 0 and prefill(L, d, need - 1) == WORKSPACE and prefill(L, d, ws=None) == WORKSPACE
    need = L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_BACKWARD)
    assert need > 0 and backward(L, d, need - 1) == WORKSPACE and backward(L, d, ws=None) == WORKSPACE
    # fp32 and few tokens run token by token, without a workspace; gradients are bf16 only
    for d in (dims(L, dtype=L.LTE_F32), dims(L, T=15)):
        assert L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_PREFILL) == 0
    d = dims(L, dtype=L.LTE_F32)
    assert L.lte_gdr_workspace_bytes(d, L.LTE_GDR_WS_BACKWARD) == 0 and backward(L, d, 1 << 40) == UNSUPPORTED
    assert L.lte_gdr_workspace_bytes(dims(L), 2) == 0


def test_workspace_grows_with_the_call(L):
    """Long sequences of few heads hold their segments' maps and states besides the records."""
    short, many = (L.lte_gdr_workspace_bytes(dims(L, B=b, T=t), L.LTE_GDR_WS_PREFILL) for b, t in ((1, 6400), (64, 100)))
    assert short > 0 and many > 0
    per_chunk = 3 * 64 * 64 * 2 + 5 * 64 * 4
    assert many == 64 * 4 * 2 * per_chunk                  # enough heads: records only
    assert short > 4 * 100 * per_chunk


def norm(L, **c):
    d = dict(B=2, T=10, Hq=4, Hkv=2, D=128, dtype=L.LTE_BF16, kind=L.LTE_NORM_RMS, eps=1e-6, rot_dim=64,
             interleaved=0, n_pos=10, wq=None, wk=None, table=P)
    d.update(c)
    return L.lte_qk_norm(*d.values())


@pytest.mark.parametrize("bad,status", [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(Hkv=0), INVALID),
                                        (dict(kind=3), INVALID), (dict(eps=0.0), INVALID),
                                        (dict(eps=float("inf")), INVALID), (dict(dtype=5), INVALID),
                                        (dict(rot_dim=24), INVALID), (dict(rot_dim=144), INVALID),
                                        (dict(table=None), INVALID), (dict(table=8), INVALID), (dict(n_pos=0), INVALID),
                                        (dict(n_pos=9), INVALID), (dict(wq=8), INVALID), (dict(D=96), UNSUPPORTED),
                                        (dict(B=1 << 16, T=1 << 14, n_pos=1 << 14), UNSUPPORTED)])
def test_norm(L, bad, status):
    n = norm(L, **bad)
    assert L._lib.lte_qk_norm_rope(C.byref(n), P, P, None, None, None, P, P, None) == status
    assert L._lib.lte_qk_norm_rope_backward(C.byref(n), P, P, None, None, None, P, P, L.LTE_F32, P, P, P, P, P,
                                            1 << 30, None) == status


def test_norm_pointers_and_workspace(L):
    n, odd = norm(L), C.c_void_p((1 << 20) + 4)
    fwd = lambda *a: L._lib.lte_qk_norm_rope(C.byref(n), *a, None)  # noqa: E731
    for i in (0, 1, 5, 6):
        for bad in (None, odd):
            a = [P, P, None, None, None, P, P]
            a[i] = bad
            assert fwd(*a) == INVALID
    assert fwd(P, P, C.byref(L.lte_strides(1 << 20, 260, 128)), None, None, P, P) == INVALID
    bwd = lambda a, m=n: L._lib.lte_qk_norm_rope_backward(C.byref(m), *a, None)  # noqa: E731
    need = L.lte_qk_norm_backward_workspace_bytes(n)
    good = [P, P, None, None, None, P, P, L.LTE_F32, P, P, P, P, P, need]
    for i in (0, 1, 5, 6, 8, 9):
        a = list(good)
        a[i] = None
        assert bwd(a) == INVALID
    assert bwd([*good[:-1], need - 1]) == WORKSPACE and bwd([*good[:-2], None, need]) == WORKSPACE
    f = norm(L, dtype=L.LTE_F32)
    assert bwd([*good[:7], L.LTE_BF16, *good[8:]], f) == INVALID              # fp32 rows, bf16 gradients
    assert bwd(good, norm(L, kind=L.LTE_NORM_NONE)) == INVALID                # a weight gradient without a norm


def test_zero_padding(L):
    one, rows = (C.c_void_p * 9)(*[1 << 20] * 9), (C.c_int64 * 9)(*[64] * 9)
    call = lambda B=2, T=8, lens=P, n=2, x=one, r=rows: L._lib.lte_gdr_zero_padding(B, T, lens, n, x, r, None)  # noqa: E731
    odd = (C.c_void_p * 2)(1 << 20, (1 << 20) + 2)
    for bad in (dict(B=0), dict(T=0), dict(lens=None), dict(n=0), dict(n=9), dict(x=None), dict(r=None), dict(x=odd),
                dict(x=(C.c_void_p * 2)(1 << 20, None)), dict(r=(C.c_int64 * 2)(64, 6)), dict(r=(C.c_int64 * 2)(0, 64))):
        assert call(**bad) == INVALID


def test_withhold(L):
    for bad in ((-1, 0, 10000), (64, 0, 10000), (1, -1, 10000), (1, 0, 999), (1, 0, 1_000_000_001)):
        assert L._lib.lte_gdr_withhold(*bad) == INVALID
    assert L._lib.lte_gdr_withhold(0, 0, 1_000_000_000) == 0


def test_zero_padding_takes_rows_from_the_shape(L, monkeypatch):
    """A tensor of one token per sequence counts as contiguous whatever its token stride, which must not
    become the length of the rows that are set to zero.  (The entry itself is replaced: no device.)"""
    import types

    import torch
    seen = []
    monkeypatch.setattr(L, "_lib", types.SimpleNamespace(
        lte_gdr_zero_padding=lambda B, T, lens, n, x, r, s: seen.append((B, T, n, list(r[:n]))) or 0))
    stream, lens = types.SimpleNamespace(cuda_stream=0), torch.zeros(2, dtype=torch.int32)
    one = torch.zeros(100).as_strided((2, 1, 3, 4), (12, 1000, 4, 1))
    assert one.is_contiguous() and one.stride(1) == 1000
    L.lte_gdr_zero_padding(lens, [one, torch.zeros(2, 1, 5)], stream)
    L.lte_gdr_zero_padding(lens, [torch.zeros(2, 7, 3, dtype=torch.bfloat16), torch.zeros(2, 7)], stream)
    assert seen == [(2, 1, 2, [48, 20]), (2, 7, 2, [6, 4])]
    for bad in ([torch.zeros(2, 7, 3).transpose(0, 1).contiguous().transpose(0, 1)], [torch.zeros(2, 7), torch.zeros(2, 8)]):
        with pytest.raises(ValueError):
            L.lte_gdr_zero_padding(lens, bad, stream)
    for bad in (lens.long(), lens[:1]):
        with pytest.raises(ValueError):
            L.lte_gdr_zero_padding(bad, [torch.zeros(2, 7)], stream)


def test_the_package_names_every_entry(L):
    import learnable_kv_token_b200 as package
    for n in L.EXPORTED:
        if n.startswith(("lte_gdr_", "lte_qk_")):
            assert getattr(package, n) is getattr(L, n), n
