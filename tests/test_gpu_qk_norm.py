"""GPU parity of the q, k norms with rotation (forward, gradients) with the float64 oracle, and their
use in front of the LTE layer and of the delta rule.

Tolerances: fp32 arithmetic rounds a row's sum D times and its result about 8 times, each by at most
2^-24, relative to the row's largest entry: 2^-24 (D + 8) per entry and row; the table adds 2^-24.
bf16 outputs are rounded once: 2^-8 of the entry.  Weight gradients sum the rows' terms in fp32, first
up to n per lane, then over the blocks: errors random in sign, 2^-24 (sqrt(rows) + D) of the terms'
2-norm, which is taken from the oracle's terms."""
import numpy as np
import pytest
import torch

import lte_inputs as LI
from oracle import delta_oracle as DO
from oracle import lte_oracle as O

pytestmark = pytest.mark.gpu
EPS = 1e-6


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


@pytest.fixture(scope="module")
def layer():
    from learnable_kv_token_b200 import layer
    return layer


def close(got, ref, D, dtype, what):
    ref_row = np.abs(ref).max(-1, keepdims=True)
    bound = 2.0 ** -24 * (D + 16) * ref_row + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0) + 1e-37
    err = np.abs(f64(got) - ref)
    assert (err <= bound).all(), f"{what}: {float((err / bound).max()):.3g} of its bound"


def setup(layer, seed, B, T, Hq, Hkv, D, dtype, kind, rot, inter, far, fused, weights=True):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k = (randn(B, T, h, D) * (1 + h) for h in (Hq, Hkv))
    wq, wk = (1 + 0.3 * randn(D) if weights else None for _ in range(2))
    if fused:
        flat = torch.cat([q.reshape(B, T, -1), k.reshape(B, T, -1)], 2).to(dtype).cuda()
        q, k = (x.unflatten(2, (-1, D)) for x in flat.split([Hq * D, Hkv * D], 2))
    else:
        q, k = q.to(dtype).cuda(), k.to(dtype).cuda()
    pos = None
    if far:
        pos = (torch.randint(0, far, (B, 1), generator=g) + torch.arange(T)).int()
    table = layer.rope_table(far + T, rot) if rot else None
    p = layer.QKNorm(kind, EPS, *(None if w is None else w.cuda() for w in (wq, wk)), rot, inter, table)
    ang = DO.rope_angles(np.broadcast_to(np.arange(T), (B, T)) if pos is None else pos.numpy(), rot)
    return q, k, p, None if pos is None else pos.cuda(), ang


CASES = [(2, 7, 4, 2, 64, "rms", 64, False, 0, False), (1, 1, 16, 4, 128, "rms", 128, False, 5000, True),
         (3, 33, 3, 1, 128, "l2", 0, False, 0, False), (1, 130, 4, 4, 64, "l2", 32, True, 0, True),
         (2, 50, 2, 2, 128, "none", 96, False, 100000, False), (1, 9, 1, 1, 64, "rms", 16, True, 70, False),
         (4, 700, 16, 4, 128, "rms", 64, False, 0, True), (1, 5, 1, 7, 64, "none", 0, False, 0, False)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward_and_gradient(layer, c, dtype):
    B, T, Hq, Hkv, D, kind, rot, inter, far, fused = c
    q, k, p, pos, ang = setup(layer, sum(map(int, c[:5])), B, T, Hq, Hkv, D, dtype, kind, rot, inter, far, fused)
    out = layer.qk_norm_rope(q, k, p, positions=pos)
    for x, w, y, n in ((q, p.wq, out[0], "q"), (k, p.wk, out[1], "k")):
        assert y.dtype == dtype and y.is_contiguous()
        close(y, DO.qk_norm(f64(x), f64(w), kind, EPS, ang, rot, inter), D, dtype, n)
    for gt in {torch.float32, dtype}:
        dy = [torch.randn(x.shape, generator=torch.Generator().manual_seed(3)).to(gt).cuda() for x in (q, k)]
        dq, dk, dwq, dwk = layer.qk_norm_rope_backward(q, k, *dy, p, positions=pos)
        again = layer.qk_norm_rope_backward(q, k, *dy, p, positions=pos)
        for x, w, d, dx, dw, n in ((q, p.wq, dy[0], dq, dwq, 0), (k, p.wk, dy[1], dk, dwk, 1)):
            rx, rw = DO.qk_norm_backward(f64(x), f64(w), f64(d), kind, EPS, ang, rot, inter)
            # dx is a difference of two vectors of its row: the bound goes by the larger of them
            if kind != "none":
                m = 1 / D if kind == "rms" else 1.0
                r = 1 / np.sqrt(m * (f64(x) ** 2).sum(-1, keepdims=True) + EPS)
                size = np.abs(r * f64(w) * (DO.rotate(f64(d), -ang, rot, inter) if rot else f64(d))).max(-1, keepdims=True)
            else:
                size = np.abs(rx).max(-1, keepdims=True)
            bound = 2.0 ** -24 * 2 * (D + 16) * size + (2.0 ** -8 * np.abs(rx) if dtype == torch.bfloat16 else 0)
            assert (np.abs(f64(dx) - rx) <= bound + 1e-37).all()
            if kind == "none":
                assert dw is None
                continue
            dn = DO.rotate(f64(d), -ang, rot, inter) if rot else f64(d)
            terms = np.sqrt(((dn * f64(x) * r) ** 2).sum((0, 1, 2)))
            rows = x.shape[0] * x.shape[1] * x.shape[2]
            assert (np.abs(f64(dw) - rw) <= 2.0 ** -24 * (rows ** 0.5 + D + 16) * terms).all()
            assert torch.equal(dw, again[2 + n])


def test_no_weights_and_in_place(layer):
    q, k, p, pos, ang = setup(layer, 8, 2, 40, 4, 2, 128, torch.bfloat16, "l2", 0, False, 0, False, weights=False)
    want = [DO.qk_norm(f64(x), None, "l2", EPS) for x in (q, k)]
    dy = [torch.ones_like(x, dtype=torch.float32) for x in (q, k)]
    assert layer.qk_norm_rope_backward(q, k, *dy, p)[2:] == (None, None)
    layer.qk_norm_rope(q, k, p, q_out=q, k_out=k)
    for x, r in zip((q, k), want):
        close(x, r, 128, torch.bfloat16, "in place")


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kind,rot", [("none", 0), ("none", 32), ("l2", 0)])
def test_the_result_is_the_callers_own(layer, kind, rot, fused):
    """Writing into the result changes neither q nor k, whatever the norm does and however they lie."""
    q, k, p, pos, ang = setup(layer, 13, 2, 9, 2, 1, 64, torch.bfloat16, kind, rot, False, 0, fused)
    before = q.clone(), k.clone()
    out = layer.qk_norm_rope(q, k, p)
    for x, y, b in zip((q, k), out, before):
        if kind == "none" and not rot:
            assert torch.equal(x, y)
        y.fill_(3.0)
        assert torch.equal(x, b)


def test_zero_rows_and_large_values(layer):
    q, k, p, pos, ang = setup(layer, 9, 1, 6, 2, 2, 64, torch.float32, "rms", 64, False, 0, False)
    q[0, 2] = 0
    k[0, 3] *= 1e15
    oq, ok = layer.qk_norm_rope(q, k, p)
    assert (oq[0, 2] == 0).all()
    close(ok, DO.qk_norm(f64(k), f64(p.wk), "rms", EPS, ang, 64, False), 64, torch.float32, "large")


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("eps", [1e-6, 1e-24, 1e-30, 1e-36])
def test_gradients_of_zero_and_tiny_rows(layer, kind, eps):
    """1 / sqrt(eps) to the third power leaves fp32 for eps below 2e-26; the gradient of a row of zeros is
    w dy / sqrt(eps) all the same.  Bounds as in test_forward_and_gradient."""
    q, k, p, pos, ang = setup(layer, 12, 1, 6, 2, 2, 64, torch.float32, kind, 0, False, 0, False)
    p.eps = eps
    q[0, 2] = 0
    k[0, 3] *= 1e-14
    dy = [torch.randn(x.shape, generator=torch.Generator().manual_seed(3)).cuda() for x in (q, k)]
    dq, dk, dwq, dwk = layer.qk_norm_rope_backward(q, k, *dy, p)
    m = 1 / 64 if kind == "rms" else 1.0
    for x, w, d, dx, dw in ((q, p.wq, dy[0], dq, dwq), (k, p.wk, dy[1], dk, dwk)):
        rx, rw = DO.qk_norm_backward(f64(x), f64(w), f64(d), kind, eps)
        r = 1 / np.sqrt(m * (f64(x) ** 2).sum(-1, keepdims=True) + eps)
        size = np.abs(r * f64(w) * f64(d)).max(-1, keepdims=True)
        assert (np.abs(f64(dx) - rx) <= 2.0 ** -24 * 2 * (64 + 16) * size).all()
        terms = np.sqrt(((f64(d) * f64(x) * r) ** 2).sum((0, 1, 2)))
        assert (np.abs(f64(dw) - rw) <= 2.0 ** -24 * (12 ** 0.5 + 64 + 16) * terms).all()


def test_position_outside_the_table(layer):
    """Those rows come out as NaN on the rotated channels, the others as ever; nothing is read out of
    the table."""
    q, k, p, pos, ang = setup(layer, 10, 1, 4, 2, 1, 64, torch.float32, "rms", 32, False, 0, False)
    bad = torch.tensor([[0, 4, -1, 3]], dtype=torch.int32, device="cuda")
    oq, ok = layer.qk_norm_rope(q, k, p, positions=bad)
    for y in (oq, ok):
        assert torch.isnan(y[0, 1:3, :, :32]).all() and torch.isfinite(y[0, 1:3, :, 32:]).all()
        assert torch.isfinite(y[0, [0, 3]]).all()


def test_in_a_graph_and_on_another_stream(layer):
    """Both directions captured, replayed with new rows and positions, beside a call on another stream."""
    g = torch.Generator().manual_seed(9)
    randn = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    xs = [(randn(3, 37, 4, 64), randn(3, 37, 2, 64), randn(3, 37, 4, 64), randn(3, 37, 2, 64),
           torch.randint(0, 64, (3, 37), generator=g, dtype=torch.int32).cuda()) for _ in range(2)]
    w = torch.rand(2, 64, generator=g).cuda() + 0.5
    norm = layer.QKNorm("rms", wq=w[0], wk=w[1], rot_dim=32, table=layer.rope_table(64, 32))

    def both(q, k, dq, dk, pos, **kw):
        return (*layer.qk_norm_rope(q, k, norm, positions=pos, **kw),
                *layer.qk_norm_rope_backward(q, k, dq, dk, norm, positions=pos, **kw))
    want = [both(*x) for x in xs]
    buf = [t.clone() for t in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*buf)
    side = torch.cuda.Stream()
    for t, new in zip(buf, xs[1]):
        t.copy_(new)
    side.wait_stream(torch.cuda.current_stream())
    graph.replay()
    other = both(*xs[0], stream=side)
    torch.cuda.synchronize()
    for a, b in zip((*got, *other), (*want[1], *want[0])):
        assert torch.equal(a, b)


def test_refusals(layer):
    q, k, p, pos, ang = setup(layer, 11, 1, 4, 2, 1, 64, torch.float32, "rms", 32, False, 0, False)
    from dataclasses import replace
    for bad in (replace(p, kind="layer"), replace(p, wq=p.wq.bfloat16()), replace(p, table=None),
                replace(p, rot_dim=16), replace(p, wk=p.wk[:32])):
        with pytest.raises(ValueError):
            layer.qk_norm_rope(q, k, bad)
    with pytest.raises(ValueError):
        layer.qk_norm_rope(q, k.bfloat16(), p)
    with pytest.raises(ValueError):
        layer.qk_norm_rope(q, k, p, positions=torch.zeros(1, 4, device="cuda"))
    with pytest.raises(ValueError):
        layer.qk_norm_rope_backward(q, k, q.half(), k.half(), p)
    for bad in (replace(p, eps=0.0), replace(p, rot_dim=8, table=layer.rope_table(4, 8)),
                replace(p, table=layer.rope_table(3, 32))):              # 4 tokens, 3 positions
        with pytest.raises(layer.L.LteError) as e:
            layer.qk_norm_rope(q, k, bad)
        assert e.value.status == 1


def test_lte_layer_behind_the_norm(layer):
    """prefill and Decoder with a norm equal the same calls on normed, rotated q and k, and the
    gradients chain: the attention's fp32 dq, dk go through the norm's gradient."""
    B, T, steps, Hq, Hkv, D = 2, 96, 4, 8, 2, 128
    g = LI.generator(60)
    q, k, v = (x.cuda() for x in LI.qkv(B, T + steps, Hq, Hkv, D, torch.bfloat16, g, std=1.0))
    cnn = tuple(x.cuda() for x in LI.cnn_weights(Hkv, D, 32, 5, 3, g, 0.1))
    norm = layer.QKNorm("rms", EPS, *((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2)), D, False,
                        layer.rope_table(T + steps, D))
    qn, kn = layer.qk_norm_rope(q, k, norm)
    lp = layer.LayerParams(sink=4, window=32, cap=8, tau=0.5)
    cut = lambda x: x[:, :T].contiguous()  # noqa: E731
    want = layer.prefill(cut(qn), cut(kn), cut(v), lp, cnn=cnn)
    got = layer.prefill(cut(q), cut(k), cut(v), lp, cnn=cnn, norm=norm)
    assert torch.equal(got.o, want.o) and torch.equal(got.k, cut(kn))
    outs = []
    dims = lp.dims(B, T, Hq, Hkv, D, torch.bfloat16)
    for nm, qq, kk, out in ((None, qn, kn, want), (norm, q, k, got)):
        cache = layer.DecodeCache(B, Hkv, D, torch.bfloat16, lp.sink, lp.window, lp.cap)
        cache.init_from_prefill(dims, cut(kn), cut(v), out, T)
        dec = layer.Decoder(dims, cnn, 2, 1, cache, 4, norm=nm)
        for t in range(T, T + steps):
            pos = torch.full((B,), t, dtype=torch.int32, device="cuda") if nm is not None else None
            o, _ = dec.step(qq[:, t].contiguous(), kk[:, t].contiguous(), v[:, t].contiguous(), positions=pos)
            outs.append(o.clone())
    for a, b in zip(outs[:steps], outs[steps:]):
        assert torch.equal(a, b)
    # gradients of sum(do * o) with respect to the projections, against the oracle's chain
    do = LI.normal((B, T, Hq, D), 1.0, torch.bfloat16, g).cuda()
    dq, dk, _ = layer.backward(got.q, got.k, cut(v), got, do, lp)
    dxq, dxk, dwq, dwk = layer.qk_norm_rope_backward(cut(q), cut(k), dq, dk, norm)
    ang = DO.rope_angles(np.broadcast_to(np.arange(T), (B, T)), D)
    masks, scale = got.mask.cpu().numpy(), 1 / D ** 0.5
    o_fw, _, _ = O.prefill(f64(got.q), f64(got.k), f64(cut(v)), masks, 4, 32, 8, scale)
    o_st = torch.from_numpy(o_fw).to(torch.bfloat16).double().numpy()
    rq, rk, _ = O.prefill_backward(f64(got.q), f64(got.k), f64(cut(v)), masks, 4, 32, 8, f64(do), scale, o_out=o_st)
    for x, w, r, dx, dw in ((cut(q), norm.wq, rq, dxq, dwq), (cut(k), norm.wk, rk, dxk, dwk)):
        ex, ew = DO.qk_norm_backward(f64(x), f64(w), r, "rms", EPS, ang, D, False)
        # the attention gradient's own gate (1e-2 of the 2-norm) and one rounding
        assert np.linalg.norm(f64(dx) - ex) <= (1e-2 + 2.0 ** -8) * np.linalg.norm(ex)
        assert np.linalg.norm(f64(dw) - ew) <= 1e-2 * np.linalg.norm(ew) * 3


def test_decoder_with_a_norm_allocates_nothing(layer):
    """A step runs over the decoder's own buffers, with a norm as without."""
    B, T, Hq, Hkv, D = 2, 40, 8, 2, 128
    g = LI.generator(61)
    q, k, v = (x.cuda() for x in LI.qkv(B, T + 3, Hq, Hkv, D, torch.bfloat16, g, std=1.0))
    cnn = tuple(x.cuda() for x in LI.cnn_weights(Hkv, D, 32, 5, 3, g, 0.1))
    norm = layer.QKNorm("rms", EPS, rot_dim=D, table=layer.rope_table(T + 3, D))
    lp = layer.LayerParams(sink=4, window=32, cap=8, tau=0.5)
    cut = lambda x: x[:, :T].contiguous()  # noqa: E731
    out = layer.prefill(cut(q), cut(k), cut(v), lp, cnn=cnn, norm=norm)
    dims = lp.dims(B, T, Hq, Hkv, D, torch.bfloat16)
    cache = layer.DecodeCache(B, Hkv, D, torch.bfloat16, lp.sink, lp.window, lp.cap)
    cache.init_from_prefill(dims, out.k, cut(v), out, T)
    dec = layer.Decoder(dims, cnn, 2, 1, cache, 4, norm=norm)
    args = [[x[:, t].contiguous() for x in (q, k, v)] + [torch.full((B,), t, dtype=torch.int32, device="cuda")]
            for t in range(T, T + 3)]
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    for qt, kt, vt, pos in args:
        dec.step(qt, kt, vt, positions=pos)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
