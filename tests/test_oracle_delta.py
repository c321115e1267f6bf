"""The oracle of the gated delta rule and of the q, k norms against torch autograd, differences and
closed forms (float64, CPU)."""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as DO


def _inputs(seed, B=2, T=9, H=4, Hk=2, dk=6, dv=5):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, T, Hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return (r.standard_normal((B, T, Hk, dk)), k, r.standard_normal((B, T, H, dv)),
            -r.exponential(0.3, (B, T, H)), r.uniform(0, 1, (B, T, H)), r.standard_normal((B, H, dv, dk)))


def _torch_delta(q, k, v, g, b, S0, scale):
    """The matrix form of the recurrence, all heads at once."""
    rep = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    S, out = S0, []
    eye = torch.eye(q.shape[3], dtype=torch.float64)
    for t in range(q.shape[1]):
        kk = k[:, t, :, :, None] * k[:, t, :, None, :]
        bt = b[:, t, :, None, None]
        S = g[:, t].exp()[..., None, None] * S @ (eye - bt * kk) + bt * v[:, t, :, :, None] * k[:, t, :, None, :]
        out.append(scale * (S @ q[:, t, :, :, None])[..., 0])
    return torch.stack(out, 1), S


@pytest.mark.parametrize("seed", [0, 1])
def test_delta_matches_matrix_form_and_autograd(seed):
    x = [torch.tensor(a, requires_grad=True) for a in _inputs(seed)]
    o, S = _torch_delta(*x, 0.7)
    r = np.random.default_rng(seed + 10)
    do, dS = r.standard_normal(o.shape), r.standard_normal(S.shape)
    grads = torch.autograd.grad((o, S), x, (torch.tensor(do), torch.tensor(dS)))
    n = [a.detach().numpy() for a in x]
    o2, S2 = DO.delta(*n[:5], S0=n[5], scale=0.7)
    np.testing.assert_allclose(o2, o.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(S2, S.detach().numpy(), atol=1e-12)
    for a, ref in zip(DO.delta_backward(*n[:5], do, S0=n[5], dST=dS, scale=0.7), grads):
        np.testing.assert_allclose(a, ref.numpy(), atol=1e-11)


def test_delta_backward_by_differences():
    q, k, v, g, b, S0 = _inputs(3, B=1, T=5)
    r = np.random.default_rng(4)
    do, dS = r.standard_normal(v.shape), r.standard_normal(S0.shape)

    def loss(*x):
        o, S = DO.delta(*x[:5], S0=x[5])
        return (do * o).sum() + (dS * S).sum()

    x = [q, k, v, g, b, S0]
    for i, d in enumerate(DO.delta_backward(*x[:5], do, S0=S0, dST=dS)):
        step = r.standard_normal(x[i].shape)
        h = 1e-6
        up, down = (loss(*[a + s * h * step if j == i else a for j, a in enumerate(x)]) for s in (1, -1))
        assert abs((up - down) / (2 * h) - (d * step).sum()) <= 1e-7 * (1 + abs((d * step).sum()))


def test_delta_closed_forms():
    q, k, v, g, b, S0 = _inputs(5)
    # unit keys, b = 1: a key reads back the value just written under it
    o, S = DO.delta(k, k, v, g, np.ones_like(b), scale=1.0)
    np.testing.assert_allclose(o, v, atol=1e-12)
    # b = 0 and no decay: the state stays
    _, S = DO.delta(q, k, v, 0 * g, 0 * b, S0=S0)
    np.testing.assert_allclose(S, S0, atol=0)
    # lengths: a sequence of no tokens keeps its state, the others stop at theirs
    o, S = DO.delta(q, k, v, g, b, S0=S0, lens=[0, 4])
    o4, S4 = DO.delta(q[:, :4], k[:, :4], v[:, :4], g[:, :4], b[:, :4], S0=S0)
    assert (o[0] == 0).all() and (o[1, 4:] == 0).all() and (S[0] == S0[0]).all()
    np.testing.assert_allclose(o[1, :4], o4[1])
    np.testing.assert_allclose(S[1], S4[1])


@pytest.mark.parametrize("kind", ["none", "rms", "l2"])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rotation_and_gradient(kind, inter):
    r = np.random.default_rng(7)
    x, w, dy = r.standard_normal((2, 3, 2, 12)), r.standard_normal(12), r.standard_normal((2, 3, 2, 12))
    rot, ang = 8, DO.rope_angles(np.arange(3) + np.array([[5], [900]]), 8)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = tx
    if kind != "none":
        m = tx.pow(2).mean(-1, keepdim=True) if kind == "rms" else tx.pow(2).sum(-1, keepdim=True)
        n = tx / torch.sqrt(m + 1e-3) * tw
    head = n[..., :rot].unflatten(-1, (4, 2)) if inter else n[..., :rot].unflatten(-1, (2, 4)).transpose(-1, -2)
    z = torch.view_as_complex(head.contiguous()) * torch.polar(torch.ones(2, 3, 1, 4, dtype=torch.float64),
                                                               torch.tensor(ang)[:, :, None])
    y = torch.view_as_real(z)
    y = torch.cat([y.flatten(-2) if inter else y.transpose(-1, -2).flatten(-2), n[..., rot:]], -1)
    np.testing.assert_allclose(DO.qk_norm(x, w, kind, 1e-3, ang, rot, inter), y.detach().numpy(), atol=1e-13)
    y.backward(torch.tensor(dy))
    dx, dw = DO.qk_norm_backward(x, w, dy, kind, 1e-3, ang, rot, inter)
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-12)
    if kind == "none":
        assert dw is None
    else:
        np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)
