"""Measured cases of the delta-rule layer and of the query/key norms.

Two groups of operators, each in the forms in which a program meets them:

``norm``, ``norm_grad``   per-head norms of queries and keys with the position rotation in the same
                          pass, and their gradients (those of the norm weights included);
``delta``, ``delta_step``, ``delta_grad``
                          the gated delta rule over a prompt, for one token, and its gradients.

A case is a dict of plain values.  ``run`` computes it with elementary torch operations in 32 bits, or,
where ``own`` is set, through the package's public calls.
"""
from __future__ import annotations

import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 10000.0


# ------------------------------------------------------------------------------------------- cases
def _norm(name, op, B, T, Hq, Hkv, D, dtype="bf16", kind="rms", rot=None, inter=False, far=0, fused=False,
          grad="f32"):
    c = dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, kind=kind, rot=D if rot is None else rot,
             inter=inter, far=far, fused=fused)
    if op == "norm_grad":
        c["grad"] = grad
    return c if name is None else dict(name=name, **c)


def _delta(name, op, B, H, Hk, dk, dv, T=1, dtype="bf16", ragged=False, init=False, fused=False):
    c = dict(op=op, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype)
    if op != "delta_step":
        c.update(ragged=ragged, init=init, fused=fused)
    return c if name is None else dict(name=name, **c)


def listed():
    return [
        # the prompts of the prefill workload: q, k between projection and attention
        _norm("norm-prompt", "norm", 32, 4096, 16, 4, 128),
        # one decode step of the same layer, 32 sequences at their own far positions
        _norm("norm-step", "norm", 32, 1, 16, 4, 128, far=16384, fused=True),
        # training: fp32 gradients from the attention backward, bf16 activations
        _norm("norm-grad", "norm_grad", 8, 4096, 16, 4, 128),
        # a small fp32 layer of odd length, unit-length keys, half of the channels rotated in pairs
        _norm("norm-grad-odd", "norm_grad", 3, 1021, 4, 4, 64, dtype="f32", kind="l2", rot=32, inter=True,
              far=100000),
        # the linear layer of the hybrid over its 4096-token prompts
        _delta("delta-prompt", "delta", 32, 16, 16, 128, 128, T=4096),
        # one long sequence: few heads, a long chain of chunks
        _delta("delta-long", "delta", 1, 16, 16, 128, 128, T=16384),
        # a padded batch that continues from earlier states, shared query/key heads, q, k, v from one projection
        _delta("delta-ragged", "delta", 7, 16, 4, 64, 128, T=1500, ragged=True, init=True, fused=True),
        # a few drafted tokens to verify
        _delta("delta-draft", "delta", 4, 16, 16, 128, 128, T=5, init=True),
        # training on 4096-token sequences
        _delta("delta-grad", "delta_grad", 8, 16, 16, 128, 128, T=4096),
        # training on a padded batch of odd length with an incoming state
        _delta("delta-grad-ragged", "delta_grad", 3, 8, 2, 64, 64, T=777, ragged=True, init=True),
        # one token for each of 32 sequences
        _delta("delta-step", "delta_step", 32, 16, 16, 128, 128),
        # one token of one sequence in fp32, shared query/key heads
        _delta("delta-step-one", "delta_step", 1, 16, 4, 128, 128, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "delta", "delta", "delta_grad", "delta_grad", "delta_step"])
    if op in ("norm", "norm_grad"):
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4])
        Hq = Hkv * rng.choice([1, 2, 4])
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, min(32 if op == "norm" else 8, max(1, (1 << 17) // T)))
        return _norm(None, op, B, T, Hq, Hkv, D, rng.choice(["bf16", "bf16", "f32"]),
                     rng.choice(["rms", "l2", "none"]) if op == "norm" else rng.choice(["rms", "l2"]),
                     rng.choice([0, D // 2, D]), rng.random() < 0.5, rng.choice([0, 0, 1000, 100000]),
                     rng.random() < 0.5, rng.choice(["f32", "same"]))
    Hk = rng.choice([1, 2, 4, 8])
    H = Hk * rng.choice([1, 2, 4]) if Hk < 8 else rng.choice([8, 16])
    dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    if op == "delta_step":
        return _delta(None, op, _log(rng, 1, 32), H, Hk, dk, dv, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "delta":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        T = _log(rng, 1, 16384 if dtype == "bf16" else 2048)
        B = _log(rng, 1, max(1, min(32, ((1 << 21) if dtype == "bf16" else (1 << 18)) // (T * H))))
        return _delta(None, op, B, H, Hk, dk, dv, T, dtype, rng.random() < 0.5, rng.random() < 0.5,
                      rng.random() < 0.5)
    T = _log(rng, 1, 4096)
    B = _log(rng, 1, max(1, min(8, (1 << 19) // (T * H))))
    return _delta(None, op, B, H, Hk, dk, dv, T, "bf16", rng.random() < 0.5, rng.random() < 0.5,
                  rng.random() < 0.5)


def work(c):
    """Each input read once and each output written once; the products of the recurrence itself."""
    e = 2 if c["dtype"] == "bf16" else 4
    n = c["B"] * c["T"]
    if c["op"] in ("norm", "norm_grad"):
        row = n * (c["Hq"] + c["Hkv"]) * c["D"]
        if c["op"] == "norm":
            return {"bytes": 2 * row * e, "flops": 8 * row}
        return {"bytes": row * (2 * e + (4 if c["grad"] == "f32" else e)), "flops": 16 * row}
    qk, v, gates = n * 2 * c["Hk"] * c["dk"], n * c["H"] * c["dv"], 2 * n * c["H"]
    state = c["B"] * c["H"] * c["dk"] * c["dv"]
    cell = n * c["H"] * c["dk"] * c["dv"]
    if c["op"] == "delta_grad":
        # q, k, v, do in, dq, dk, dv out; gates and their gradients; the states' gradients
        return {"bytes": (2 * qk + 3 * v) * e + 8 * gates + 4 * state * (3 if c["init"] else 2), "flops": 16 * cell}
    first = 4 * state if c["op"] == "delta_step" or c["init"] else 0
    return {"bytes": (qk + 2 * v) * e + 4 * gates + first + 4 * state, "flops": 6 * cell}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def rope_table(n, rot):
    """fp32 [n, rot]: cosines of position x frequency, then sines; the angles in 64 bits."""
    f = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _heads(parts, fused):
    """The tensors by themselves, or as neighbouring columns of one projection's output."""
    if not fused:
        return list(parts)
    B, T = parts[0].shape[:2]
    flat = torch.cat([p.reshape(B, T, -1) for p in parts], 2)
    out, at = [], 0
    for p in parts:
        n = p.shape[2] * p.shape[3]
        out.append(flat[:, :, at:at + n].unflatten(2, p.shape[2:]))
        at += n
    return out


def prepare(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    B, T = c["B"], c["T"]
    s = {"case": c}
    if c["op"] in ("norm", "norm_grad"):
        q, k = (_randn(g, B, T, h, c["D"]).mul_(1.0 + h / 16).to(dt) for h in (c["Hq"], c["Hkv"]))
        s["q"], s["k"] = _heads((q, k), c["fused"])
        s["wq"], s["wk"] = (1 + 0.2 * _randn(g, c["D"]) for _ in range(2))
        if c["kind"] == "none":
            s["wq"] = s["wk"] = None
        s["pos"] = None
        if c["far"]:
            start = torch.randint(0, c["far"], (B, 1), generator=g, device="cuda")
            s["pos"] = (start + torch.arange(T, device="cuda")).int()
        s["table"] = rope_table(c["far"] + T, c["rot"]) if c["rot"] else None
        if c["op"] == "norm_grad":
            gt = torch.float32 if c["grad"] == "f32" else dt
            s["dq"], s["dk"] = (_randn(g, B, T, h, c["D"]).to(gt) for h in (c["Hq"], c["Hkv"]))
        return s
    H, Hk, dk, dv = c["H"], c["Hk"], c["dk"], c["dv"]
    # unit-length queries and keys; keys of neighbouring tokens resemble one another, as after a short convolution
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    k = _randn(g, B, T, Hk, dk)
    k = k + 0.5 * torch.roll(k, 1, 1) if T > 1 else k
    q, k, v = (x.to(dt) for x in (unit(_randn(g, B, T, Hk, dk)), unit(k), _randn(g, B, T, H, dv)))
    # each head has a pace of its own, from a few tokens to thousands; now and then a head forgets all at once
    pace = torch.exp(torch.linspace(math.log(0.3), math.log(3e-4), H, device="cuda"))
    gate = -pace * torch.nn.functional.softplus(1 + _randn(g, B, T, H))
    gate = torch.where(torch.rand(B, T, H, generator=g, device="cuda") < 1e-3, -30.0, gate)
    beta = torch.sigmoid(_randn(g, B, T, H))
    s0 = 0.3 * _randn(g, B, H, dv, dk)
    if c["op"] == "delta_step":
        s.update(q=q[:, 0].contiguous(), k=k[:, 0].contiguous(), v=v[:, 0].contiguous(),
                 g=gate[:, 0].contiguous(), beta=beta[:, 0].contiguous(), state=s0)
        return s
    s["q"], s["k"], s["v"] = _heads((q, k, v), c["fused"])
    s.update(g=gate.contiguous(), beta=beta, state=s0 if c["init"] else None, lens=None)
    if c["ragged"]:
        s["lens"] = torch.randint(0, T + 1, (B,), generator=g, device="cuda").int()
        s["lens"][-1] = T
    if c["op"] == "delta_grad":
        s["do"] = _randn(g, B, T, H, dv).to(dt)
        s["dstate"] = 0.1 * _randn(g, B, H, dv, dk) if c["init"] else None
    return s


# --------------------------------------------------------------------------------------- plain forms
def _rotate(n, table, pos, rot, inter, back=False):
    """Rotation of the first `rot` channels of n [B,T,H,D] (the transposed rotation for `back`)."""
    if not rot:
        return n
    T = n.shape[1]
    cs = table[:T][None] if pos is None else table[pos.long()]
    cos, sin = (x[:, :, None] for x in cs.split(rot // 2, -1))
    sin = -sin if back else sin
    x, rest = n[..., :rot], n[..., rot:]
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else x.chunk(2, -1)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
    return torch.cat([y, rest], -1)


def _norm_eps(c):
    return 1e-6


def _norm_plain(x, w, c, s):
    x = x.float()
    if c["kind"] != "none":
        ss = x.square().sum(-1, keepdim=True) * (1 / c["D"] if c["kind"] == "rms" else 1.0)
        x = x * torch.rsqrt(ss + _norm_eps(c)) * w
    return _rotate(x, s["table"], s["pos"], c["rot"], c["inter"])


def _norm_grad_plain(x, w, dy, c, s):
    x, dn = x.float(), _rotate(dy.float(), s["table"], s["pos"], c["rot"], c["inter"], back=True)
    m = 1 / c["D"] if c["kind"] == "rms" else 1.0
    r = torch.rsqrt(x.square().sum(-1, keepdim=True) * m + _norm_eps(c))
    dx = r * w * dn - x * (m * r ** 3) * (dn * w * x).sum(-1, keepdim=True)
    return dx, (dn * x * r).double().sum((0, 1, 2)).float()


def _unit_lower_inverse(m):
    """Inverse of unit lower triangular [..., 64, 64]: the inverses of diagonal blocks, joined in pairs."""
    L = m.shape[-1]
    i = torch.arange(L, device=m.device)
    x = torch.eye(L, device=m.device, dtype=m.dtype).expand_as(m)
    n = 1
    while n < L:
        # the block below the diagonal within each pair of blocks of n rows
        pair = (i[:, None] // (2 * n) == i // (2 * n)) & (i[:, None] // n > i // n)
        x = x - x @ (m * pair) @ x
        n *= 2
    return x


def _delta_plain(q, k, v, g, beta, s0, lens, scale):
    """The gated delta rule in chunks: products within all chunks at once, then the chain of states."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    live = None
    if lens is not None:
        live = torch.arange(T, device=q.device)[None] < lens[:, None]
        k, v = (torch.where(live[..., None, None], x, 0) for x in (k, v))
        g, beta = (torch.where(live[..., None], x, 0) for x in (g, beta))
    pad = -T % CHUNK
    N = (T + pad) // CHUNK

    def chunks(x, heads):  # [B, T, h, d] -> [N, B, H, 64, d]
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).unflatten(1, (N, CHUNK))
        return x.permute(1, 0, 3, 2, 4).repeat_interleave(heads, 2)

    q, k, v = chunks(q, H // Hk), chunks(k, H // Hk), chunks(v, 1)
    G, beta = (chunks(x[..., None], 1) for x in (g, beta))
    G = G.cumsum(-2)
    i = torch.arange(CHUNK, device=q.device)
    low = i[:, None] >= i
    D = torch.where(low, (G - G.mT).masked_fill(~low, 0).exp(), 0)
    t = _unit_lower_inverse(torch.eye(CHUNK, device=q.device) + beta * D * (k @ k.mT) * (i[:, None] > i))
    a = scale * D * (q @ k.mT)
    eG, last = G.exp(), (G[..., -1:, :] - G).exp()
    u0, w = t @ (beta * v), t @ (beta * eG * k)
    qe, kl, el = scale * eG * q, last * k, eG[..., -1:, :]
    S = torch.zeros(B, H, dv, dk, device=q.device) if s0 is None else s0
    out = []
    for c in range(N):  # each chunk starts from the state that the one before it leaves
        u = u0[c] - w[c] @ S.mT
        out.append(qe[c] @ S.mT + a[c] @ u)
        S = el[c] * S + u.mT @ kl[c]
    o = torch.stack(out).permute(1, 0, 3, 2, 4).reshape(B, N * CHUNK, H, dv)[:, :T]
    if live is not None:
        o = torch.where(live[..., None, None], o, 0)
    return o, S


def _scale(c):
    return c["dk"] ** -0.5


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        return {"q": _norm_plain(s["q"], s["wq"], c, s).to(dt), "k": _norm_plain(s["k"], s["wk"], c, s).to(dt)}
    if c["op"] == "norm_grad":
        dq, dwq = _norm_grad_plain(s["q"], s["wq"], s["dq"], c, s)
        dk, dwk = _norm_grad_plain(s["k"], s["wk"], s["dk"], c, s)
        return {"dq": dq.to(dt), "dk": dk.to(dt), "dwq": dwq, "dwk": dwk}
    if c["op"] == "delta_step":
        rep = c["H"] // c["Hk"]
        q, k = (s[n].float().repeat_interleave(rep, 1)[..., None] for n in ("q", "k"))
        S = s["state"] * s["g"].exp()[..., None, None]
        u = s["beta"][..., None, None] * (s["v"].float()[..., None] - S @ k)
        s["state"].copy_(S + u * k.mT)
        return {"o": (_scale(c) * (s["state"] @ q))[..., 0].to(dt), "state": s["state"]}
    if c["op"] == "delta":
        o, S = _delta_plain(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"], s["state"],
                            s["lens"], _scale(c))
        return {"o": o.to(dt), "state": S}
    with torch.enable_grad():
        x = [s[n].float() for n in ("q", "k", "v")] + [s["g"], s["beta"]]
        s0 = torch.zeros(c["B"], c["H"], c["dv"], c["dk"], device="cuda") if s["state"] is None else s["state"]
        x = [t.detach().clone().requires_grad_() for t in x + [s0]]
        o, S = _delta_plain(*x, s["lens"], _scale(c))
        ds = torch.zeros_like(S) if s["dstate"] is None else s["dstate"]
        d = torch.autograd.grad((o, S), x, (s["do"].float(), ds))
    return {"dq": d[0].to(dt), "dk": d[1].to(dt), "dv": d[2].to(dt), "dg": d[3], "dbeta": d[4], "dstate": d[5]}


# ------------------------------------------------------------------------------ the package's calls
def _own(s):
    from learnable_kv_token_b200 import layer
    c = s["case"]
    if c["op"] in ("norm", "norm_grad"):
        p = layer.QKNorm(kind=c["kind"], eps=_norm_eps(c), wq=s["wq"], wk=s["wk"], rot_dim=c["rot"],
                         interleaved=c["inter"], table=s["table"])
        if c["op"] == "norm":
            q, k = layer.qk_norm_rope(s["q"], s["k"], p, positions=s["pos"])
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = layer.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], p, positions=s["pos"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if c["op"] == "delta_step":
        o = layer.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"])
        return {"o": o, "state": s["state"]}
    if c["op"] == "delta":
        o, S = layer.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"], lens=s["lens"])
        return {"o": o, "state": S}
    dq, dk, dv, dg, dbeta, ds0 = layer.delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"],
                                                      state=s["state"], dstate=s["dstate"], lens=s["lens"])
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dstate": ds0}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------- 64-bit definitions
def _exact_norm(x, w, c, s, dy=None):
    """y, or the gradients of x and w, by the definition of norm and rotation in 64 bits."""
    x = x.double()
    D, R = c["D"], c["rot"]
    B, T = x.shape[:2]
    pos = torch.arange(T, device="cuda").expand(B, T) if s["pos"] is None else s["pos"]
    if R:
        # channel pairs as complex numbers, turned by position x frequency
        ang = pos.double()[..., None, None] * ROPE_BASE ** (-2 * torch.arange(R // 2, device="cuda").double() / R)
        turn = torch.polar(torch.ones_like(ang), ang)
        at = torch.arange(R, device="cuda").view(R // 2, 2) if c["inter"] else torch.arange(R, device="cuda").view(2, R // 2).T

    def turned(n, by):
        n = n.clone()
        z = torch.view_as_complex(n[..., at].contiguous()) * by
        n[..., at.reshape(-1)] = torch.view_as_real(z).flatten(-2)
        return n

    if c["kind"] == "none":
        return turned(x, turn) if R else x
    w = w.double()
    h = torch.sqrt(x.pow(2).mean(-1, keepdim=True) + _norm_eps(c)) if c["kind"] == "rms" else torch.sqrt(
        x.pow(2).sum(-1, keepdim=True) + _norm_eps(c))
    if dy is None:
        n = x / h * w
        return turned(n, turn) if R else n
    dn = turned(dy.double(), turn.conj()) if R else dy.double()
    z = x / h
    dz = dn * w
    inner = (dz * z).mean(-1, keepdim=True) if c["kind"] == "rms" else (dz * z).sum(-1, keepdim=True)
    return (dz - z * inner) / h, (dn * z).sum((0, 1, 2))


def _exact_states(S, k, v, a, b, t0, t1):
    """S_{t0-1} .. S_{t1-1} and u of tokens t0 .. t1-1, token by token."""
    states, us = [S], []
    for t in range(t0, t1):
        S = a[:, t, :, None, None] * S
        u = b[:, t, :, None] * (v[:, t] - torch.einsum("bhvk,bhk->bhv", S, k[:, t]))
        S = S + u[..., None] * k[:, t, :, None, :]
        states.append(S)
        us.append(u)
    return states, us


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        return {n: _exact_norm(s[n], s["w" + n], c, s) for n in ("q", "k")}
    if c["op"] == "norm_grad":
        (dq, dwq), (dk, dwk) = (_exact_norm(s[n], s["w" + n], c, s, s["d" + n]) for n in ("q", "k"))
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    B, T, H, Hk, dk, dv = (c[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
    rep, scale = H // Hk, 1 / math.sqrt(dk)
    step = c["op"] == "delta_step"
    tok = (lambda x: x[:, None]) if step else (lambda x: x)
    q, k = (tok(s[n]).double().repeat_interleave(rep, 2) for n in ("q", "k"))
    v, a, b = tok(s["v"]).double(), tok(s["g"]).double().exp(), tok(s["beta"]).double()
    S = torch.zeros(B, H, dv, dk, device="cuda", dtype=torch.float64) if s["state"] is None else s["state"].double()
    lens = None if step else s["lens"]
    live = None if lens is None else (torch.arange(T, device="cuda") < lens[:, None]).double()[..., None]
    if live is not None:  # a token behind its sequence keeps the state and reads nothing
        a, b, q = a * live + (1 - live), b * live, q * live[..., None]
    if c["op"] != "delta_grad":
        o = torch.empty(B, T, H, dv, device="cuda", dtype=torch.float64)
        for t in range(T):
            S = _exact_states(S, k, v, a, b, t, t + 1)[0][1]
            o[:, t] = scale * torch.einsum("bhvk,bhk->bhv", S, q[:, t])
        return {"o": o[:, 0] if step else o, "state": S}
    do = s["do"].double()
    if live is not None:
        do = do * live[..., None]
    dS = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    marks = [S]
    for t0 in range(0, T, 32):
        marks.append(_exact_states(marks[-1], k, v, a, b, t0, min(T, t0 + 32))[0][-1])
    dq, dkk = torch.zeros_like(q), torch.zeros_like(k)
    dvv, dg, db = torch.zeros_like(v), torch.zeros_like(a), torch.zeros_like(b)
    for n in reversed(range(len(marks) - 1)):
        t0, t1 = 32 * n, min(T, 32 * n + 32)
        states, us = _exact_states(marks[n], k, v, a, b, t0, t1)
        for t in reversed(range(t0, t1)):
            St, Sp, u, kt = states[t - t0 + 1], states[t - t0], us[t - t0], k[:, t]
            dS = dS + scale * do[:, t][..., None] * q[:, t, :, None, :]
            dq[:, t] = scale * torch.einsum("bhvk,bhv->bhk", St, do[:, t])
            y = torch.einsum("bhvk,bhk->bhv", dS, kt)
            aS = a[:, t, :, None, None] * Sp
            err = v[:, t] - torch.einsum("bhvk,bhk->bhv", aS, kt)
            f = b[:, t, :, None] * y
            db[:, t] = (y * err).sum(-1)
            dvv[:, t] = f
            dkk[:, t] = torch.einsum("bhvk,bhv->bhk", dS, u) - torch.einsum("bhvk,bhv->bhk", aS, f)
            back = dS - f[..., None] * kt[:, :, None, :]
            dg[:, t] = (back * aS).sum((-2, -1))
            dS = a[:, t, :, None, None] * back
    dq, dkk = (x.unflatten(2, (Hk, rep)).sum(3) for x in (dq, dkk))
    out = {"dq": dq, "dk": dkk, "dv": dvv, "dg": dg, "dbeta": db}
    if live is not None:
        out = {n: x * (live if x.dim() == 3 else live[..., None]) for n, x in out.items()}
    return {**out, "dstate": dS}
