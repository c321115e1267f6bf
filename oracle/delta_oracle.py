"""Plain CPU oracle for the gated delta rule and for the query/key norms with rotation.

TEST INFRASTRUCTURE ONLY (same rules as ``oracle/lte_oracle.py``: the GPU library shares no code
with it).  Float64 throughout.

The delta rule follows the state equation of "Sparse Linear Attention: Viewing SWA from the
Perspective of Linear Attention", section "Background: Linear attention", with the value that a key
already holds taken away before the new one is written:

    S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,   o_t = scale S_t q_t,   a_t = e^{g_t}.
"""
from __future__ import annotations

import numpy as np


def delta_recurrent(q, k, v, g, b, S0, scale):
    """One (batch element, value head): q, k [T, dk], v [T, dv], g, b [T], S0 [dv, dk].
    Returns o [T, dv], the states S_0 .. S_T and the errors e_t = v_t - a_t S_{t-1} k_t."""
    S, states, o, err = S0, [S0], np.zeros_like(v), np.zeros_like(v)
    for t in range(len(q)):
        aS = np.exp(g[t]) * S
        err[t] = v[t] - aS @ k[t]
        S = aS + b[t] * np.outer(err[t], k[t])
        o[t] = scale * (S @ q[t])
        states.append(S)
    return o, states, err


def delta_recurrent_backward(q, k, v, g, b, S0, scale, do, dST):
    """Gradients of sum(do * o) + sum(dST * S_T) for one (batch element, value head)."""
    _, states, err = delta_recurrent(q, k, v, g, b, S0, scale)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(b)
    dS = dST
    for t in reversed(range(len(q))):
        a, kt = np.exp(g[t]), k[t]
        dS = dS + scale * np.outer(do[t], q[t])
        dq[t] = scale * states[t + 1].T @ do[t]
        # S_t = aS + b e k^T with e = v - aS k
        y = dS @ kt
        db[t] = y @ err[t]
        de = b[t] * y
        dv[t] = de
        dk[t] = b[t] * dS.T @ err[t] - a * states[t].T @ de
        d_aS = dS - np.outer(de, kt)
        dg[t] = a * np.sum(d_aS * states[t])
        dS = a * d_aS
    return dq, dk, dv, dg, db, dS


def _units(q, k, v, g, b, S0, lens):
    B, T, H, dv = v.shape
    rep = H // q.shape[2]
    for i in range(B):
        n = T if lens is None else int(lens[i])
        for h in range(H):
            s0 = np.zeros((dv, q.shape[3])) if S0 is None else S0[i, h]
            yield i, h, h // rep, n, (q[i, :n, h // rep], k[i, :n, h // rep], v[i, :n, h], g[i, :n, h],
                                      b[i, :n, h], s0)


def delta(q, k, v, g, b, S0=None, lens=None, scale=None):
    """q, k [B,T,Hk,dk], v [B,T,H,dv], g, b [B,T,H], S0 [B,H,dv,dk]; lens [B].  Returns o (zero
    behind a sequence's length) and the final states."""
    scale = q.shape[3] ** -0.5 if scale is None else scale
    o, S = np.zeros(v.shape), np.zeros(v.shape[:1] + v.shape[2:] + q.shape[3:])
    for i, h, _, n, x in _units(q, k, v, g, b, S0, lens):
        ou, states, _ = delta_recurrent(*x, scale)
        o[i, :n, h], S[i, h] = ou, states[-1]
    return o, S


def delta_backward(q, k, v, g, b, do, S0=None, dST=None, lens=None, scale=None):
    """Gradients dq, dk, dv, dg, db, dS0 of sum(do * o) + sum(dST * S_T)."""
    scale = q.shape[3] ** -0.5 if scale is None else scale
    dq, dk, dv, dg, db = (np.zeros(x.shape) for x in (q, k, v, g, b))
    dS0 = np.zeros(v.shape[:1] + v.shape[2:] + q.shape[3:])
    for i, h, hk, n, x in _units(q, k, v, g, b, S0, lens):
        dS = np.zeros_like(x[5]) if dST is None else dST[i, h]
        r = delta_recurrent_backward(*x, scale, do[i, :n, h], dS)
        dq[i, :n, hk] += r[0]
        dk[i, :n, hk] += r[1]
        dv[i, :n, h], dg[i, :n, h], db[i, :n, h], dS0[i, h] = r[2], r[3], r[4], r[5]
    return dq, dk, dv, dg, db, dS0


# ------------------------------------------------------------------------------- norms, rotation
def rope_angles(pos, rot, base=10000.0):
    """[.., rot/2] angles of positions pos."""
    return np.asarray(pos, np.float64)[..., None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(n, ang, rot, interleaved):
    """n [B,T,H,D] with its channel pairs turned by ang [B,T,rot/2]."""
    y = np.array(n, dtype=np.float64)
    ia, ib = _pairs(rot, interleaved)
    c, s = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None]
    y[..., ia] = n[..., ia] * c - n[..., ib] * s
    y[..., ib] = n[..., ib] * c + n[..., ia] * s
    return y


def qk_norm(x, w, kind, eps, ang=None, rot=0, interleaved=False):
    """One of q, k [B,T,H,D]; w [D] or None; kind "none", "rms" or "l2"."""
    if kind != "none":
        ss = (x * x).sum(-1, keepdims=True) / (x.shape[-1] if kind == "rms" else 1)
        x = x / np.sqrt(ss + eps) * (1.0 if w is None else w)
    return rotate(x, ang, rot, interleaved) if rot else np.array(x)


def qk_norm_backward(x, w, dy, kind, eps, ang=None, rot=0, interleaved=False):
    """dx [B,T,H,D] and dw [D] (None for kind "none")."""
    dn = rotate(dy, -ang, rot, interleaved) if rot else dy
    if kind == "none":
        return dn, None
    m = 1.0 / x.shape[-1] if kind == "rms" else 1.0
    r = 1.0 / np.sqrt(m * (x * x).sum(-1, keepdims=True) + eps)
    z = dn if w is None else dn * w
    dx = r * z - m * r ** 3 * x * (z * x).sum(-1, keepdims=True)
    return dx, (dn * x * r).sum((0, 1, 2))
