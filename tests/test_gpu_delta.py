"""GPU parity of the gated delta rule (prompt, step, gradients) with the float64 oracle.

Tolerances, as the 2-norm of the error over the 2-norm of the reference:
 - fp32 arithmetic (fp32 inputs, the step, few tokens): a token rounds every state entry about
   dk + 8 times (the dot product, the update), each by at most 2^-24, independent from token to
   token: 2^-24 (dk + 8) sqrt(T).
 - bf16 prompts, fp32 outputs (states, gate gradients): a product with one or both operands as bf16
   hi + lo pairs is off by at most (2^-8)^2 per split operand; the states pass three such products
   per chunk (S k, T r, u k^T) with five split operands between them, random in sign from entry to
   entry, so by less than their root sum: sqrt(5) 2^-16 = 3.4e-5 at most, and a third of it at the
   rounding's mean size (2^-8 / sqrt(3) per split): 1.2e-5.  The bound taken is 2e-5.  Gradients of
   the gates pass the chain twice, forwards and backwards: 4e-5.
 - bf16 outputs: rounded once (at most 2^-8), behind products that round one operand to bf16 (at
   most 2^-8, independent): sqrt(2) 2^-8; gradients of q and k sum four such terms behind products
   of two rounded operands: sqrt(3) 2^-8."""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as DO

pytestmark = pytest.mark.gpu

STATE_TOL, GATE_TOL = 2e-5, 4e-5
BF16_TOL, GRAD_TOL = 2 ** 0.5 * 2.0 ** -8, 3 ** 0.5 * 2.0 ** -8


def tol32(T, dk):
    return 2.0 ** -24 * (dk + 8) * T ** 0.5


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def rel(got, ref):
    n = np.linalg.norm(ref)
    d = np.linalg.norm(f64(got) - ref)
    return d / n if n else d


@pytest.fixture(scope="module")
def layer():
    from learnable_kv_token_b200 import layer
    return layer


def inputs(seed, B, T, H, Hk, dk, dv, dtype=torch.bfloat16, init=True, lens=None, fused=False):
    """Unit keys; each head has its own pace; on the device.  Rows behind `lens` hold NaN."""
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = randn(B, T, Hk, dk), randn(B, T, Hk, dk), randn(B, T, H, dv)
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    gate = -torch.exp(torch.linspace(-1.2, -8, H)) * torch.nn.functional.softplus(1 + randn(B, T, H))
    beta = torch.sigmoid(randn(B, T, H))
    S0 = 0.3 * randn(B, H, dv, dk) if init else None
    if lens is not None:
        for i, n in enumerate(lens):
            for x in (q, k, v, gate, beta):
                x[i, n:] = float("nan")
        lens = torch.tensor(lens, dtype=torch.int32).cuda()
    q, k, v = (x.to(dtype) for x in (q, k, v))
    if fused:
        flat = torch.cat([x.reshape(B, T, -1) for x in (q, k, v)], 2).cuda()
        q, k, v = (x.unflatten(2, (-1, d)) for x, d in zip(flat.split([Hk * dk, Hk * dk, H * dv], 2), (dk, dk, dv)))
    return dict(q=q.cuda(), k=k.cuda(), v=v.cuda(), g=gate.cuda(), beta=beta.cuda(),
                state=None if S0 is None else S0.cuda(), lens=lens)


def oracle(x, scale=None):
    return DO.delta(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["g"]), f64(x["beta"]), f64(x["state"]),
                    None if x["lens"] is None else x["lens"].cpu().numpy(), scale)


def check_prefill(layer, x, scale=None):
    o, S = layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"], lens=x["lens"],
                               scale=scale)
    torch.cuda.synchronize()
    o_ref, S_ref = oracle(x, scale)
    T, dk = x["q"].shape[1], x["q"].shape[3]
    bf16 = x["q"].dtype == torch.bfloat16
    assert torch.isfinite(o).all() and torch.isfinite(S).all()
    assert rel(S, S_ref) <= max(tol32(T, dk), STATE_TOL if bf16 else 0)
    assert rel(o, o_ref) <= (BF16_TOL if bf16 else tol32(T, dk))
    if x["lens"] is not None:
        for i, n in enumerate(x["lens"].tolist()):
            assert (o[i, n:] == 0).all()
    return o, S


SHAPES = [(2, 1, 2, 2, 64, 64), (1, 5, 4, 1, 128, 128), (2, 17, 4, 2, 64, 128), (1, 63, 2, 2, 128, 64),
          (3, 64, 2, 1, 128, 128), (1, 65, 8, 8, 64, 64), (2, 200, 4, 4, 128, 128), (1, 333, 2, 1, 64, 128)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prefill(layer, dtype, shape):
    check_prefill(layer, inputs(sum(shape), *shape, dtype=dtype, init=shape[1] % 2 == 1))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[0, 1, 130], [64, 130, 63], [129, 0, 65]], ids=str)
def test_prefill_padded_batch(layer, dtype, lens):
    """Rows behind a sequence hold NaN and are not read; a sequence of no tokens keeps its state."""
    x = inputs(9, 3, 130, 4, 2, 128, 128, dtype=dtype, lens=lens, fused=True)
    _, S = check_prefill(layer, x)
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(S[i], x["state"][i])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["same-key", "beta-0", "beta-1", "beta-2", "forget", "forget-all", "no-decay",
                                  "scaled", "zero-key"])
def test_prefill_extreme_gates(layer, dtype, kind):
    x = inputs(21, 2, 150, 4, 2, 128, 128, dtype=dtype)
    scale = None
    if kind == "same-key":                     # every token writes under one key: the chunk's system is dense
        x["k"][:] = x["k"][:, :1].clone()
        x["beta"][:] = 0.9
    elif kind.startswith("beta"):
        x["beta"][:] = float(kind[-1])
        if kind == "beta-2":                   # reflections: the state keeps its size
            x["g"][:] = -0.01
    elif kind == "forget":                     # resets inside a chunk, some of them exact
        x["g"][:, 10::37] = -30.0
        x["g"][:, 70] = float("-inf")
    elif kind == "forget-all":
        x["g"][:] = float("-inf")
    elif kind == "no-decay":
        x["g"][:] = 0.0
    elif kind == "zero-key":
        x["k"][:, ::3] = 0
    else:
        scale = 1.5
    check_prefill(layer, x, scale)


@pytest.mark.parametrize("shape", [(2, 300, 4, 2, 128, 128), (1, 2000, 2, 1, 64, 128), (3, 130, 4, 4, 128, 64)], ids=str)
def test_outputs_are_rounded_once(layer, shape):
    """o is the rounded result almost everywhere.  Where the sum before it is off by d of its row's size (2e-5
    as the states), an entry z of that size comes out as the neighbour with probability 2 d 2^8 / z = c / z, c =
    0.01; over entries with a density of at most 0.8 at any z in (0, 3): 0.8 c (1 + ln(3 / c)) = 0.054.  Twice
    that for rows whose terms are larger than their sum.  (One operand rounded to bf16: over a third differ.)"""
    x = inputs(25, *shape)
    o, _ = layer.delta_prefill(*(x[n] for n in ("q", "k", "v", "g", "beta")), state=x["state"])
    want = torch.from_numpy(oracle(x)[0]).to(torch.bfloat16)
    assert (o.cpu() != want).double().mean() <= 0.108


@pytest.mark.parametrize("init", [False, True])
def test_tokens_of_beta_0_write_nothing(layer, init):
    """As in the step and in the walk by tokens: the state only decays, and stays exactly zero from zero."""
    x = inputs(24, 2, 150, 4, 2, 128, 64, init=init)
    x["beta"][:] = 0.0
    o, S = layer.delta_prefill(*(x[n] for n in ("q", "k", "v", "g", "beta")), state=x["state"])
    if not init:
        assert (o == 0).all() and (S == 0).all()
    else:
        # per chunk the decay's factor, with two units in its last place of the exponential (4 x 2^-24) and its
        # argument's rounding (the states that are not gone by then have |G| < 1: 2^-24), and the product's
        want = f64(x["state"]) * np.exp(f64(x["g"]).sum(1))[..., None, None]
        assert rel(S, want) <= 2.0 ** -24 * 6 * 3


@pytest.mark.parametrize("shape,lens", [((1, 2600, 2, 1, 128, 128), None), ((2, 3000, 1, 1, 64, 128), [2999, 700]),
                                        ((1, 1500, 1, 1, 128, 64), None), ((3, 1100, 1, 1, 64, 64), [0, 1100, 64])],
                         ids=str)
def test_prefill_long_few_heads(layer, shape, lens):
    """Few heads over many chunks: the sequence runs in segments.  The result in place equals the one
    in a new tensor, and slow decay carries the first tokens to the end."""
    x = inputs(40, *shape, lens=lens)
    x["g"].mul_(0.05)
    o, S = check_prefill(layer, x)
    st = x["state"].clone()
    o2, S2 = layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=st, lens=x["lens"], state_out=st)
    assert S2 is st and torch.equal(o, o2) and torch.equal(S, st)


def test_broadcast_and_padded_views(layer):
    """Keys shared by the batch as an expanded view, values in rows wider than they need."""
    x = inputs(41, 3, 100, 2, 2, 64, 128)
    wide = torch.zeros(3, 100, 2, 192, dtype=torch.bfloat16, device="cuda")
    wide[..., 64:] = x["v"]
    y = {**x, "q": x["q"][:1].expand(3, -1, -1, -1), "k": x["k"][:1].expand(3, -1, -1, -1), "v": wide[..., 64:]}
    check_prefill(layer, y)
    check_backward(layer, y)


@pytest.mark.parametrize("lens", [[0, 5, 33], [-7, 99, 32]], ids=str)
def test_zero_padding(layer, lens):
    """Rows behind the lengths (which are clamped) become zero, all else stays: rows of 4, 12, 130 * 4 and
    20 * 2 bytes, so that stretches begin and end anywhere in a group of 16."""
    T, n = 33, torch.tensor(lens, dtype=torch.int32).cuda()
    store = [torch.full((3 * T * w + 9,), 7.0, dtype=t, device="cuda")
             for w, t in ((1, torch.float32), (3, torch.float32), (130, torch.float32), (20, torch.bfloat16))]
    x = [s[4:-5].view(3, T, -1) for s in store]
    layer.L.lte_gdr_zero_padding(n, x)
    for s, t in zip(store, x):
        assert (s[:4] == 7).all() and (s[-5:] == 7).all()
        for b, m in enumerate(min(max(m, 0), T) for m in lens):
            assert (t[b, :m] == 7).all() and (t[b, m:] == 0).all()


def test_prefill_continues(layer):
    """A prompt in three calls, in place on one state, equals the prompt in one call."""
    x = inputs(4, 2, 300, 4, 4, 128, 128)
    o, S = check_prefill(layer, x)
    st, parts = x["state"].clone(), []
    for a, b in ((0, 100), (100, 103), (103, 300)):
        part, _ = layer.delta_prefill(x["q"][:, a:b], x["k"][:, a:b], x["v"][:, a:b],
                                      x["g"][:, a:b].contiguous(), x["beta"][:, a:b].contiguous(), state=st,
                                      state_out=st)
        parts.append(part)
    assert rel(st, f64(S)) <= 2 * STATE_TOL
    assert rel(torch.cat(parts, 1), f64(o)) <= 2 * BF16_TOL


def test_bad_values_stay_in_their_head(layer):
    """A NaN in one head of one sequence reaches that head from its block of 64 tokens on; every other
    head and sequence, and the blocks before, are as without it, forwards and backwards."""
    x = inputs(42, 2, 200, 4, 4, 128, 128)
    names = ("q", "k", "v", "g", "beta")
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    clean = layer.delta_prefill(*(x[n] for n in names), state=x["state"])
    grads = layer.delta_backward(*(x[n] for n in names), do, state=x["state"])
    x["v"][1, 100, 2, 5] = float("nan")
    o, S = layer.delta_prefill(*(x[n] for n in names), state=x["state"])
    bad = layer.delta_backward(*(x[n] for n in names), do, state=x["state"])
    assert torch.isnan(o[1, 100, 2]).any() and torch.isnan(S[1, 2]).any()
    assert torch.equal(o[1, :64, 2], clean[0][1, :64, 2])
    others = [(0, h) for h in range(4)] + [(1, h) for h in (0, 1, 3)]
    for i, h in others:
        assert torch.equal(o[i, :, h], clean[0][i, :, h]) and torch.equal(S[i, h], clean[1][i, h])
        for a, b in zip(bad[:5], grads[:5]):
            assert torch.equal(a[i, :, h], b[i, :, h])
        assert torch.equal(bad[5][i, h], grads[5][i, h])


def test_views_with_odd_strides_of_one(layer):
    """A single token as a view whose unused strides are no multiples of 16 bytes."""
    x = inputs(43, 1, 1, 2, 2, 64, 64)
    wide = torch.zeros(1, 3, 2, 67, dtype=torch.bfloat16, device="cuda")
    odd = wide.as_strided((1, 1, 2, 64), (7, 5, 64, 1))
    odd.copy_(x["q"])
    assert not odd.stride(1) % 8 == 0
    a = layer.delta_prefill(odd, x["k"], x["v"], x["g"], x["beta"], state=x["state"])
    b = layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_repeats(layer):
    x = inputs(5, 3, 190, 4, 2, 64, 128, lens=[190, 3, 100])
    a, b = (layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"], lens=x["lens"])
            for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def check_backward(layer, x, dstate=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    do = torch.randn(x["v"].shape, generator=g).bfloat16().cuda()
    B, T, H, dv = x["v"].shape
    dS = torch.randn(B, H, dv, x["q"].shape[3], generator=g).cuda() * 0.2 if dstate else None
    if x["lens"] is not None:
        for i, n in enumerate(x["lens"].tolist()):
            do[i, n:] = float("nan")
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], do)
    got = layer.delta_backward(*args, state=x["state"], dstate=dS, lens=x["lens"])
    again = layer.delta_backward(*args, state=x["state"], dstate=dS, lens=x["lens"])
    lens = None if x["lens"] is None else x["lens"].cpu().numpy()
    ref = DO.delta_backward(*(f64(t) for t in args), f64(x["state"]), f64(dS), lens)
    for a, b, r, name, tol in zip(got, again, ref, ("dq", "dk", "dv", "dg", "dbeta", "dstate"),
                                  (GRAD_TOL, GRAD_TOL, BF16_TOL, GATE_TOL, GATE_TOL, STATE_TOL)):
        assert torch.equal(a, b), name
        assert torch.isfinite(a).all(), name
        assert rel(a, r) <= tol, f"{name}: {rel(a, r):.3g} > {tol:.3g}"
    if lens is not None:
        for i, n in enumerate(lens):
            assert all((t[i, n:] == 0).all() for t in got[:5])
    return got


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(layer, shape):
    check_backward(layer, inputs(100 + sum(shape), *shape, init=shape[1] % 2 == 1), dstate=shape[0] == 1)


@pytest.mark.parametrize("shape,lens", [((1, 2100, 2, 1, 128, 64), None), ((2, 1601, 1, 1, 64, 128), [1601, 700]),
                                        ((4, 2048, 1, 1, 128, 128), [2048, 0, 1, 1025]),
                                        ((3, 2000, 2, 2, 64, 64), [256, 257, 2000])], ids=str)
def test_backward_long_few_heads(layer, shape, lens):
    """Sequences that are cut into segments, which end in any of them."""
    check_backward(layer, inputs(110 + shape[1], *shape, lens=lens))


@pytest.mark.parametrize("lens", [[0, 1, 130], [64, 130, 63], [129, 0, 65]], ids=str)
def test_backward_padded_batch(layer, lens):
    x = inputs(10, 3, 130, 4, 2, 128, 128, lens=lens, fused=True)
    check_backward(layer, x)


@pytest.mark.parametrize("kind", ["same-key", "beta-0", "beta-1", "forget", "no-decay"])
def test_backward_extreme_gates(layer, kind):
    x = inputs(22, 2, 150, 4, 2, 128, 128)
    if kind == "same-key":
        x["k"][:] = x["k"][:, :1].clone()
        x["beta"][:] = 0.9
    elif kind.startswith("beta"):
        x["beta"][:] = float(kind[-1])
    elif kind == "forget":
        x["g"][:, 10::37] = -30.0
        x["g"][:, 70] = -200.0
    else:
        x["g"][:] = 0.0
    check_backward(layer, x)


@pytest.mark.parametrize("size", [1e-6, 1e-9])
@pytest.mark.parametrize("beta", ["0", "1e-20", "1e-15", "some-0"])
def test_small_gradients_of_small_betas(layer, beta, size):
    """Gradients behind a mean loss are small, and a token that writes nothing has one all the same: they
    scale with dO and dstate, so the bounds are those of gradients of order one."""
    x = inputs(23, 2, 150, 4, 2, 128, 128)
    if beta == "some-0":
        x["beta"][:, ::3] = 0
    else:
        x["beta"][:] = float(beta)
    g = torch.Generator().manual_seed(7)
    do = (torch.randn(x["v"].shape, generator=g) * size).bfloat16().cuda()
    dS = (torch.randn(x["state"].shape, generator=g) * 0.2 * size).cuda()
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], do)
    got = layer.delta_backward(*args, state=x["state"], dstate=dS)
    ref = DO.delta_backward(*(f64(t) for t in args), f64(x["state"]), f64(dS))
    # (dk and dv of tokens that write next to nothing are next to nothing: not held to a share of themselves)
    tols = dict(dq=GRAD_TOL, dk=GRAD_TOL, dv=BF16_TOL, dg=GATE_TOL, dbeta=GATE_TOL, dstate=STATE_TOL)
    for a, r, name in zip(got, ref, tols):
        if beta == "some-0" or name not in ("dk", "dv"):
            assert rel(a, r) <= tols[name], f"{name}: {rel(a, r):.3g} > {tols[name]:.3g}"


@pytest.mark.parametrize("which", ["all", "some"])
def test_no_gradient_of_gates_that_are_shut(layer, which):
    """A gate of e^g = 0 lets nothing pass: its gradient is exactly zero, the others' as ever."""
    x = inputs(26, 2, 150, 4, 2, 128, 64)
    shut = torch.ones_like(x["g"], dtype=torch.bool)
    if which == "some":
        shut = torch.rand(shut.shape, generator=torch.Generator().manual_seed(9)).cuda() < 0.1
        shut[:, :1] = shut[:, 63:66] = True
    x["g"] = torch.where(shut, torch.where(torch.arange(4, device="cuda") % 2 == 0, float("-inf"), -104.0), x["g"])
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    got = layer.delta_backward(*(x[n] for n in ("q", "k", "v", "g", "beta")), do, state=x["state"])
    assert (got[3][shut] == 0).all()
    g = torch.where(shut, float("-inf"), x["g"])               # (in 64 bits e^-104 is not zero)
    ref = DO.delta_backward(*(f64(y) for y in (x["q"], x["k"], x["v"], g, x["beta"], do, x["state"])))
    for a, r, tol in zip(got, ref, (GRAD_TOL, GRAD_TOL, BF16_TOL, GATE_TOL, GATE_TOL, STATE_TOL)):
        assert torch.isfinite(a).all() and rel(a, r) <= tol


def test_backward_by_differences(layer):
    """The gradient of every input along a random direction against a central difference of the
    forward pass, with steps of h = 0.05 of the input's norm along the gradient.
    Slope: 2 h |gradient| |x|, which for v (o is linear in it) is near 0.1 |do| |o|.  Rounding: the n = 8960
    entries of o are off by at most 2^-8 |o_i|, independently in the two losses: sqrt(2) 2^-8 |do| |o| /
    sqrt(n) = 6e-5 |do| |o|, 6e-4 of that slope, and 6e-3 where an input moves the loss a tenth as much.
    Curvature: h^2 / 6 = 4e-4 times a ratio of derivatives of order one.  The gradient itself: 4e-3.
    Together below 2 %; 5 % is allowed."""
    x = inputs(200, 1, 70, 2, 1, 64, 64)
    g = torch.Generator().manual_seed(1)
    do = torch.randn(x["v"].shape, generator=g).bfloat16().cuda()
    names = ("q", "k", "v", "g", "beta", "state")
    got = dict(zip(names, layer.delta_backward(*(x[n] for n in names[:5]), do, state=x["state"])))

    def loss(y):
        o, _ = layer.delta_prefill(*(y[n] for n in names[:5]), state=y["state"])
        return float((o.double() * do.double()).sum())

    for n in names:
        step = got[n].float() / got[n].float().norm() * x[n].float().norm() * 0.05
        up, down = ({**x, n: (x[n].float() + s * step).to(x[n].dtype)} for s in (1, -1))
        real = (up[n].double() - down[n].double())           # the step as rounded to the input's type
        want = float((got[n].double() * real).sum())
        assert abs(loss(up) - loss(down) - want) <= 0.05 * abs(want), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 2, 1, 64, 64), (3, 4, 2, 128, 64), (5, 16, 16, 64, 128), (2, 6, 2, 128, 128)],
                         ids=str)
def test_step(layer, dtype, shape):
    B, H, Hk, dk, dv = shape
    T = 6
    x = inputs(30 + B, B, T, H, Hk, dk, dv, dtype=dtype)
    x["g"][:, 3] = float("-inf")
    o_ref, S_ref = oracle(x)
    st = x["state"].clone()
    for t in range(T):
        o = layer.delta_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), st)
        assert rel(o, o_ref[:, t]) <= (tol32(T, dk) if dtype == torch.float32 else 2.0 ** -8)
    assert rel(st, S_ref) <= tol32(T, dk)


def test_step_in_a_graph(layer):
    """A captured step, replayed with new inputs in its buffers, goes on from the state."""
    B, H, D, T = 4, 8, 128, 5
    x = inputs(77, B, T, H, H, D, D)
    buf = {n: x[n][:, 0].clone() for n in ("q", "k", "v", "g", "beta")}
    st, out = x["state"].clone(), torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.delta_step(*buf.values(), st.clone(), out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.delta_step(*buf.values(), st, out=out)
    o_ref, S_ref = oracle(x)
    for t in range(T):
        for n in buf:
            buf[n].copy_(x[n][:, t])
        graph.replay()
        assert rel(out, o_ref[:, t]) <= 2.0 ** -8
    assert rel(st, S_ref) <= tol32(T, D)


def test_prefill_on_another_stream_and_in_graphs(layer):
    """The workspace belongs to the call: two captured prompts and one on a side stream do not disturb
    one another."""
    xs = [inputs(50 + i, 2, 130 + 70 * i, 4, 4, 128, 128) for i in range(2)]
    want = [layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"]) for x in xs]
    graphs, got = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"]))
        graphs.append(graph)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        x = xs[0]
        o, S = layer.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"], stream=side)
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(S, want[0][1])
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_backward_in_a_graph(layer):
    """A captured gradient pass, replayed with new inputs in its buffers."""
    x, y = inputs(60, 2, 100, 4, 2, 128, 64), inputs(61, 2, 100, 4, 2, 128, 64)
    names = ("q", "k", "v", "g", "beta")
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want = layer.delta_backward(*(y[n] for n in names), do, state=y["state"])
    layer.delta_backward(*(x[n] for n in names), do, state=x["state"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.delta_backward(*(x[n] for n in names), do, state=x["state"])
    for n in (*names, "state"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_segments_in_a_graph_over_their_own_state(layer):
    """A long prompt of few heads, cut into segments, captured with the state updated in its place and
    replayed beside an eager call of the same kind."""
    x = inputs(62, 1, 3000, 2, 2, 128, 128)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want = layer.delta_prefill(*args, state=x["state"])
    st = x["state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = layer.delta_prefill(*args, state=st, state_out=st)
    assert S is st
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        st.copy_(x["state"])
        graph.replay()
        other = layer.delta_prefill(*args, state=x["state"], stream=side)
    torch.cuda.synchronize()
    for a, b in ((o, want[0]), (st, want[1]), (other[0], want[0]), (other[1], want[1])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1500, 4100])
def test_more_heads_than_processors(layer, T):
    """160 states, whose sequences are cut into pieces that hand the state on: as the same sequences
    in two calls of 80, which are not cut, bit by bit; the state in its own place, lengths from none
    to all with the ends of pieces among them."""
    x = inputs(66, 40, T, 4, 2, 64, 64, lens=[T, 0, 1, 64, T // 2, 768, 769, T - 1] * 5)
    names = ("q", "k", "v", "g", "beta")
    st = x["state"].clone()
    o, S = layer.delta_prefill(*(x[n] for n in names), state=st, state_out=st, lens=x["lens"])
    for half in (slice(0, 20), slice(20, 40)):
        o1, S1 = layer.delta_prefill(*(x[n][half] for n in names), state=x["state"][half], lens=x["lens"][half])
        assert torch.equal(o[half], o1) and torch.equal(S[half], S1)


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_more_heads_than_processors(layer, D):
    """The same for the gradients, whose pieces also hand on the state's gradient."""
    T = 1500
    x = inputs(67, 40, T, 4, 2, D, D, lens=[T, 0, 1, 64, T // 2, 512, 513, T - 1] * 5)
    names = ("q", "k", "v", "g", "beta")
    g = torch.Generator().manual_seed(5)
    do, ds = torch.randn(x["v"].shape, generator=g).bfloat16().cuda(), torch.randn(x["state"].shape, generator=g).cuda()
    got = layer.delta_backward(*(x[n] for n in names), do, state=x["state"], dstate=ds, lens=x["lens"])
    for half in (slice(0, 20), slice(20, 40)):
        part = layer.delta_backward(*(x[n][half] for n in names), do[half], state=x["state"][half], dstate=ds[half],
                                    lens=x["lens"][half])
        for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), got, part):
            assert torch.equal(a[half], b), name


def test_gradients_on_two_streams_at_once(layer):
    """Two gradient passes that run side by side give what each gives alone."""
    names = ("q", "k", "v", "g", "beta")
    xs = [inputs(63 + i, 2, 300 + 90 * i, 4, 2, 64, 128, lens=[300, 77]) for i in range(2)]
    dos = [torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(4)).bfloat16().cuda() for x in xs]
    call = lambda x, do, **kw: layer.delta_backward(*(x[n] for n in names), do, state=x["state"], lens=x["lens"], **kw)  # noqa: E731
    want = [call(x, do) for x, do in zip(xs, dos)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [call(x, do, stream=s) for x, do, s in zip(xs, dos, sides)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for i, j in zip(a, b):
            assert torch.equal(i, j)


@pytest.mark.parametrize("shape", [(1, 2000, 2, 1, 64, 64), (40, 1500, 4, 2, 64, 64)], ids=str)
def test_segments_and_pieces_of_gradients_in_a_graph(layer, shape):
    """Captured once, replayed twice with other inputs: the pieces' counters start anew every time."""
    x, y = inputs(68, *shape), inputs(69, *shape)
    names = ("q", "k", "v", "g", "beta")
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    first, want = (layer.delta_backward(*(z[n] for n in names), do, state=z["state"]) for z in (x, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.delta_backward(*(x[n] for n in names), do, state=x["state"])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, first))
    for n in (*names, "state"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits(layer):
    """A sequence whose tensors have over 2^31 elements: its last tokens, and the state, equal those of
    the same tokens in a call of their own behind the state of the others."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    T, tail, H, D = (1 << 20) + 320, 200, 16, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v = randn(1, T, H, D), randn(1, T, H, D), randn(1, T, H, D)
    k /= k.norm(dim=-1, keepdim=True)
    gate = -0.01 * torch.rand(1, T, H, generator=g, device="cuda")
    beta = torch.rand(1, T, H, generator=g, device="cuda")
    assert q.numel() > 1 << 31
    o, S = layer.delta_prefill(q, k, v, gate, beta)
    n = T - tail
    _, S0 = layer.delta_prefill(q[:, :n], k[:, :n], v[:, :n], gate[:, :n], beta[:, :n])
    o1, S1 = layer.delta_prefill(q[:, n:], k[:, n:], v[:, n:], gate[:, n:], beta[:, n:], state=S0)
    assert torch.isfinite(S).all()
    # the chunks of the two calls start at other tokens: equal within the bounds of each
    assert rel(S, f64(S1)) <= 2 * STATE_TOL
    assert rel(o[:, n:], f64(o1)) <= 2 * BF16_TOL


def test_hybrid_layer_together(layer):
    """The linear layer of a hybrid as it is used: unit keys by the L2 norm, the prompt, its gradients
    back through the norm, and decoding that goes on from the prompt's state."""
    B, T, steps, H, Hk, D = 2, 90, 4, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = (randn(B, T + steps, h, D).bfloat16().cuda() for h in (Hk, Hk, H))
    gate, beta = (-0.1 * torch.rand(B, T + steps, H, generator=g)).cuda(), torch.rand(B, T + steps, H, generator=g).cuda()
    norm = layer.QKNorm("l2")
    cut = lambda x: x[:, :T].contiguous()  # noqa: E731
    qn, kn = layer.qk_norm_rope(cut(q), cut(k), norm)
    o, S = layer.delta_prefill(qn, kn, cut(v), cut(gate), cut(beta))
    prompt = S.clone()
    outs = []
    for t in range(T, T + steps):
        qt, kt = layer.qk_norm_rope(q[:, t:t + 1].contiguous(), k[:, t:t + 1].contiguous(), norm)
        outs.append(layer.delta_step(qt[:, 0], kt[:, 0], v[:, t].contiguous(), gate[:, t].contiguous(),
                                     beta[:, t].contiguous(), S))
    # the oracle on the normed q, k as the norm rounds them
    qa, ka = layer.qk_norm_rope(q, k, norm)
    o_ref, S_ref = DO.delta(f64(qa), f64(ka), f64(v), f64(gate), f64(beta))
    assert rel(torch.cat([o, torch.stack(outs, 1)], 1), o_ref) <= BF16_TOL
    assert rel(S, S_ref) <= STATE_TOL
    do = randn(B, T, H, D).bfloat16().cuda()
    dq, dk, *_ = layer.delta_backward(qn, kn, cut(v), cut(gate), cut(beta), do)
    dxq, dxk, dwq, dwk = layer.qk_norm_rope_backward(cut(q), cut(k), dq, dk, norm)
    assert dwq is None and dwk is None and not torch.equal(prompt, S)
    r = DO.delta_backward(f64(qn), f64(kn), f64(cut(v)), f64(gate[:, :T]), f64(beta[:, :T]), f64(do))
    for x, d, got in ((q, r[0], dxq), (k, r[1], dxk)):
        ref, _ = DO.qk_norm_backward(f64(cut(x)), None, d, "l2", 1e-6)
        # the rule's gradient, then one more rounding; the norm takes the part along x away, which
        # leaves the rest's error as it was and the rest smaller: by at most the ratio of the two
        shrink = np.linalg.norm(d / np.linalg.norm(f64(cut(x)), axis=-1, keepdims=True)) / np.linalg.norm(ref)
        assert rel(got, ref) <= GRAD_TOL * max(shrink, 1) + 2.0 ** -8


def test_refusals(layer):
    x = inputs(1, 1, 8, 2, 2, 64, 64)
    call = lambda **c: layer.delta_prefill(**{**{n: x[n] for n in ("q", "k", "v", "g", "beta", "state")}, **c})  # noqa: E731
    bad = [dict(g=x["g"].bfloat16()), dict(beta=x["beta"][:, :4]), dict(k=x["k"][:, :4]), dict(q=x["q"].float()),
           dict(state=x["state"].bfloat16()), dict(lens=torch.tensor([8])), dict(g=x["g"].cpu()),
           dict(q=x["q"].transpose(2, 3).contiguous().transpose(2, 3)), dict(state=x["state"][..., :32])]
    for c in bad:
        with pytest.raises(ValueError):
            call(**c)
    y = inputs(1, 1, 8, 3, 2, 64, 64)                          # 3 value heads, 2 key heads
    with pytest.raises(layer.L.LteError) as e:
        layer.delta_prefill(y["q"], y["k"], y["v"], y["g"], y["beta"])
    assert e.value.status == 1
    z = torch.zeros(1, 8, 2, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(layer.L.LteError) as e:
        layer.delta_prefill(z, z, z, x["g"], x["beta"])
    assert e.value.status == 2
    with pytest.raises(ValueError):
        layer.delta_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["g"][:, 0], x["beta"][:, 0], None or x["g"])
