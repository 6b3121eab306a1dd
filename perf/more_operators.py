"""The delta-rule layer's operators that are timed: what is called, on which inputs, and their plain forms.

Five calls of the package, as a program with gated delta-rule layers makes them:

* ``gdr``         the gated delta rule over whole sequences (``ss_gdr_fwd``): per head a state S [K, V],
                  S' = exp(g_t) S_{t-1}, u_t = beta_t (v_t - S'^T k_t), S_t = S' + k_t u_t^T, y_t = scale S_t^T q_t,
                  with q and k divided by their lengths first (or as they are), heads of v sharing heads of k, and
                  reset[b, t] != 0 starting a new document (the state in front of it counts as zero);
* ``gdr_train``   the same and its gradients (``ss_gdr_fwd`` with checkpoints, ``ss_gdr_bwd``);
* ``gdr_step``    the same for one token of each stream (``ss_gdr_step``), the state updated in place;
* ``norm``        the norms behind and before a layer with gate and residual (``ss_gnorm_fwd``):
                  p = y / rms(y) w (over groups of columns), s = residual + scale p silu(gate), n = s / rms(s) w_next;
* ``norm_train``  the same and its gradients (``ss_gnorm_bwd``).

``own`` false computes each in its plain form, with elementary torch operations in 32 bits; true calls the package.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS_QK = 1e-6         # under the root of a key's length
EPS = 1e-5            # under the root of a norm
CHUNK = 64            # tokens that the plain form takes at a time


def _gdr(name, op, B, L, Hk, H, K, V, dtype, **kw):
    return dict(name=name, op=op, B=B, L=L, Hk=Hk, H=H, K=K, V=V, dtype=dtype,
                **{**dict(fused=False, docs=0, state=False, unit=True), **kw})


def listed():
    return [
        # one short prompt of a small model: latency
        _gdr("gdr prompt B1 L64 H4", "gdr", 1, 64, 4, 4, 128, 128, "f32"),
        # a prompt at the training width, inputs as slices of one projection's output, keys shared by two heads
        _gdr("gdr prefill B1 L2048 H40", "gdr", 1, 2048, 20, 40, 128, 128, "bf16", fused=True, state=True),
        # one very long sequence, prefilled in pieces: the state goes in and out
        _gdr("gdr long B1 L131072 H16", "gdr", 1, 131072, 16, 16, 128, 128, "bf16", state=True),
        # a training step's recurrence at the training width
        _gdr("gdr_train B8 L2048 H40", "gdr_train", 8, 2048, 40, 40, 128, 128, "bf16"),
        # several documents packed into ragged rows, odd widths, full precision, states carried over
        _gdr("gdr_train packed B3 L1001 H6", "gdr_train", 3, 1001, 3, 6, 96, 129, "f32", docs=5, state=True),
        # one token of one stream of a small model, and of each of 64 streams of a large one
        _gdr("gdr_step S1 H8", "gdr_step", 1, 1, 8, 8, 64, 64, "bf16"),
        _gdr("gdr_step S64 H64", "gdr_step", 64, 1, 64, 64, 128, 128, "bf16"),
        # the norms between two layers: 64 streams' tokens, and a training batch's
        dict(name="norm M64 K2560", op="norm", M=64, K=2560, group=2560, dtype="bf16", gate=True, residual=True, next=True),
        dict(name="norm M16384 K2560", op="norm", M=16384, K=2560, group=2560, dtype="bf16", gate=True, residual=True, next=True),
        # the norm and gate of each head's output on its way to the projection back
        dict(name="norm heads M16384 K5120", op="norm", M=16384, K=5120, group=128, dtype="bf16", gate=True, residual=False,
             next=False),
        # the norms' training step, at the training width and over ragged rows of odd width in full precision
        dict(name="norm_train M16384 K2560", op="norm_train", M=16384, K=2560, group=2560, dtype="bf16", gate=True, residual=True,
             next=True),
        dict(name="norm_train M3003 K1537", op="norm_train", M=3003, K=1537, group=1537, dtype="f32", gate=True, residual=True,
             next=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdr", "gdr", "gdr_train", "gdr_train", "gdr_step", "norm", "norm_train"])
    dtype = rng.choice(["f32", "bf16"])
    if op.startswith("gdr"):
        K, V = rng.choice([_log(rng, 8, 256), 64, 128]), rng.choice([_log(rng, 8, 256), 64, 128])
        B = _log(rng, 1, 256 if op == "gdr_step" else 8)
        L = 1 if op == "gdr_step" else _log(rng, 1, 131072 if op == "gdr" else 4096)
        most = (1 << 29 if op == "gdr_step" else 1 << 27 if op == "gdr" else 1 << 25) // (B * L * max(K, V))
        if op == "gdr_step":
            most //= min(K, V)
        Hk = _log(rng, 1, max(1, min(32, most)))
        H = Hk * rng.choice([1, 1, 2, 3])
        return _gdr(None, op, B, L, Hk, H, K, V, dtype, fused=rng.random() < 0.4, docs=rng.choice([0, 0, 1, 7]) if L > 1 else 0,
                    state=op == "gdr_step" or rng.random() < 0.5, unit=rng.random() < 0.7)
    M = _log(rng, 1, 16384)
    heads = rng.choice([1, 1, 1, _log(rng, 2, 40)])
    group = _log(rng, 8, max(8, min(8192, (1 << 25) // M) // heads))
    return dict(op=op, M=M, K=heads * group, group=group, dtype=dtype, gate=rng.random() < 0.7, residual=rng.random() < 0.7,
                next=rng.random() < 0.7)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62))
    return g


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}

    def normal(*shape, dtype="f32", scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DT[dtype])

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    op, dt = c["op"], c["dtype"]
    if op.startswith("gdr"):
        B, L, Hk, H, K, V = (c[k] for k in ("B", "L", "Hk", "H", "K", "V"))
        # keys that are used as they are come at a length of about 1
        small = 1.0 if c["unit"] else K ** -0.5
        if c["fused"]:
            p = normal(B, L, 2 * Hk * K + H * V, dtype=dt)
            p[..., Hk * K:2 * Hk * K] *= small
            st["q"], st["k"] = p[..., :Hk * K].view(B, L, Hk, K), p[..., Hk * K:2 * Hk * K].view(B, L, Hk, K)
            st["v"] = p[..., 2 * Hk * K:].view(B, L, H, V)
        else:
            st["q"], st["k"], st["v"] = normal(B, L, Hk, K, dtype=dt), normal(B, L, Hk, K, dtype=dt, scale=small), normal(B, L, H, V, dtype=dt)
        # g = -exp(A_log) softplus(a + bias): rates in [1, 16], steps in [0.001, 0.1] before the input's share
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
        bias = step + torch.log(-torch.expm1(-step))
        st["g"] = -uniform(1.0, 16.0, H) * torch.nn.functional.softplus(normal(B, L, H) + bias)
        st["beta"] = torch.sigmoid(normal(B, L, H))
        st["state"] = normal(B, H, K, V, scale=0.3) if c["state"] or op == "gdr_step" else None
        st["reset"] = None
        if c["docs"]:
            st["reset"] = torch.zeros(B, L, dtype=torch.uint8, device="cuda")
            st["reset"].scatter_(1, torch.randint(0, L, (B, c["docs"]), generator=g, device="cuda"), 1)
        if op == "gdr_step":
            st.update({k: st[k][:, 0] for k in ("q", "k", "v", "g", "beta")})
        if op == "gdr_train":
            st["dy"] = normal(B, L, H, V, dtype=dt)
            st["dstate"] = normal(B, H, K, V, scale=0.3) if c["state"] else None
        return st
    M, K = c["M"], c["K"]
    st["y"] = normal(M, K, dtype=dt)
    st["w"] = 1.0 + normal(c["group"], scale=0.1)
    st["gate"] = normal(M, K, dtype=dt) if c["gate"] else None
    st["residual"] = normal(M, K, dtype=dt, scale=3.0) if c["residual"] else None
    st["scale"] = uniform(0.1, 1.0, K) if c["residual"] else None
    st["w_next"] = 1.0 + normal(K, scale=0.1) if c["next"] else None
    if op == "norm_train":
        st["ds"] = normal(M, K, dtype=dt)
        st["dn"] = normal(M, K, dtype=dt) if c["next"] else None
    return st


def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


# --------------------------------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits (sums of log decays in 64)

def _unit(x, on):
    """x / |x| (or x itself) and 1 / |x|, in 32 bits."""
    x = x.float()
    if not on:
        return x, torch.ones_like(x[..., :1])
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS_QK)
    return x * r, r


def _chunks(x, n):
    """[B, L, H, ...] as [B, H, n, CHUNK, ...], padded with zeros."""
    pad = n * CHUNK - x.shape[1]
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    x = x.view(x.shape[0], n, CHUNK, *x.shape[2:])
    return x.movedim(3, 1).contiguous()


def _tokens(x, L):
    """The other way."""
    x = x.movedim(1, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :L]


def _chunked(st):
    """Everything of the chunks that needs no state."""
    c, f = st["case"], {}
    n, rep = -(-c["L"] // CHUNK), c["H"] // c["Hk"]
    q, f["rq"] = _unit(st["q"], c["unit"])
    k, f["rk"] = _unit(st["k"], c["unit"])
    f["q1"], f["k1"] = q, k
    Q = _chunks(q.repeat_interleave(rep, 2) * c["K"] ** -0.5, n)
    K, V, beta = _chunks(k.repeat_interleave(rep, 2), n), _chunks(st["v"].float(), n), _chunks(st["beta"], n)[..., None]
    g = st["g"].double()
    if st["reset"] is not None:
        g = g.masked_fill((st["reset"] != 0)[..., None], -200.0)          # exp(-200) is 0 in 32 bits
    G = _chunks(g, n).cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, device=G.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(lower == 0, -1e4)).float()
    KK = (K @ K.transpose(-1, -2)) * D * (lower - torch.eye(CHUNK, device=G.device))
    A = beta * KK
    T = torch.eye(CHUNK, device=G.device).expand_as(A).contiguous()          # (1 + A)^-1, row after row
    for i in range(1, CHUNK):
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i]).squeeze(-2)
    f.update(Q=Q, K=K, V=V, beta=beta, D=D, KK=KK, A=A, T=T, P=(Q @ K.transpose(-1, -2)) * D, n=n,
             ga=torch.exp(G).float()[..., None], to_end=torch.exp(G[..., -1:] - G).float()[..., None])
    return f


def _walk(st, f, keep):
    """Outputs and states, chunk after chunk."""
    c = st["case"]
    S = st["state"] if st["state"] is not None else torch.zeros(c["B"], c["H"], c["K"], c["V"], device="cuda")
    out, states, us = [], [], []
    for n in range(f["n"]):
        Q, K, V, T, P, beta, ga, end = (f[k][:, :, n] for k in ("Q", "K", "V", "T", "P", "beta", "ga", "to_end"))
        U = T @ (beta * (V - ga * (K @ S)))
        out.append(ga * (Q @ S) + P @ U)
        if keep:
            states.append(S)
            us.append(U)
        S = ga[:, :, -1:] * S + (end * K).transpose(-1, -2) @ U
    return _tokens(torch.stack(out, 2), c["L"]), S, states, us


def _plain_gdr(st):
    y, S, _, _ = _walk(st, _chunked(st), False)
    out = {"y": y.to(st["v"].dtype)}
    if st["state"] is not None:
        st["state"].copy_(S)
        out["state"] = st["state"]
    return out


def _plain_gdr_train(st):
    c, f = st["case"], _chunked(st)
    y, last, states, us = _walk(st, f, True)
    dO = _chunks(st["dy"].float(), f["n"])
    dS = st["dstate"] if st["dstate"] is not None else torch.zeros_like(last)
    lower = torch.ones(CHUNK, CHUNK, device="cuda").tril()
    strict = lower - torch.eye(CHUNK, device="cuda")
    parts = {k: [None] * f["n"] for k in ("q", "k", "v", "g", "beta")}
    for n in reversed(range(f["n"])):
        Q, K, T, P, A, KK, D, V, beta, ga, end = (f[k][:, :, n] for k in ("Q", "K", "T", "P", "A", "KK", "D", "V", "beta", "ga",
                                                                           "to_end"))
        o, S, U = dO[:, :, n], states[n], us[n]
        Z = T.transpose(-1, -2) @ (P.transpose(-1, -2) @ o + end * (K @ dS))
        dP, dA = (o @ U.transpose(-1, -2)) * lower, -(Z @ U.transpose(-1, -2)) * strict
        qS, kS, kU = ga * (o @ S.transpose(-1, -2)), beta * ga * (Z @ S.transpose(-1, -2)), end * (U @ dS.transpose(-1, -2))
        PD, AD = dP * D, dA * D * beta
        parts["q"][n] = qS + PD @ K
        parts["k"][n] = PD.transpose(-1, -2) @ Q + kU - kS + AD @ K + AD.transpose(-1, -2) @ K
        parts["v"][n] = beta * Z
        parts["beta"][n] = (Z * (V - ga * (K @ S) - KK @ U)).sum(-1)
        # a log decay g_t is in every term that goes from a token in front of t to one from t on
        pair = (dP * P + dA * A) * strict
        before = torch.cat([torch.zeros_like(pair[..., :1]), pair.cumsum(-1)[..., :-1]], -1)
        rows, cols = (Q * qS).sum(-1) - (K * kS).sum(-1), (K * kU).sum(-1)
        parts["g"][n] = (before * lower).sum(-2) + rows.flip(-1).cumsum(-1).flip(-1) + cols.cumsum(-1) - cols \
            + (ga[:, :, -1, 0] * (S * dS).sum((-1, -2)))[..., None]
        dS = ga[:, :, -1:] * dS + (ga * Q).transpose(-1, -2) @ o - (beta * ga * K).transpose(-1, -2) @ Z
    grad = {k: _tokens(torch.stack(v, 2), c["L"]) for k, v in parts.items()}

    def shared(d, x1, r):
        """Heads of v back to the head of k they share, and through the division by the length."""
        d = d.reshape(c["B"], c["L"], c["Hk"], -1, c["K"]).sum(3)
        return (d - x1 * (x1 * d).sum(-1, keepdim=True)) * r if c["unit"] else d

    dg = grad["g"]
    if st["reset"] is not None:
        dg = dg.masked_fill((st["reset"] != 0)[..., None], 0.0)
    io = st["v"].dtype
    out = {"y": y.to(io), "dq": shared(grad["q"] * c["K"] ** -0.5, f["q1"], f["rq"]).to(io), "dk": shared(grad["k"], f["k1"], f["rk"]).to(io),
           "dv": grad["v"].to(io), "dg": dg, "dbeta": grad["beta"], "dstate_init": dS}
    if st["state"] is not None:
        st["state"].copy_(last)
        out["state"] = st["state"]
    return out


def _plain_step(st):
    c, rep = st["case"], st["case"]["H"] // st["case"]["Hk"]
    q, k = (_unit(st[n], c["unit"])[0].repeat_interleave(rep, 1) for n in ("q", "k"))
    S = torch.exp(st["g"])[..., None, None] * st["state"]
    u = st["beta"][..., None] * (st["v"].float() - (S * k[..., None]).sum(-2))
    st["state"].copy_(S + k[..., None] * u[..., None, :])
    y = (st["state"] * q[..., None]).sum(-2) * c["K"] ** -0.5
    return {"y": y.to(st["v"].dtype), "state": st["state"]}


def _norm_parts(st):
    c, f = st["case"], {}
    y = st["y"].float().view(c["M"], -1, c["group"])
    f["ry"] = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    f["yn"] = y * f["ry"]
    p = (f["yn"] * st["w"]).view(c["M"], c["K"])
    f["p"], f["sig"] = p, None
    h = p
    if st["gate"] is not None:
        f["z"] = st["gate"].float()
        f["sig"] = torch.sigmoid(f["z"])
        f["silu"] = f["z"] * f["sig"]
        h = p * f["silu"]
    f["h"] = h
    s = h if st["scale"] is None else h * st["scale"]
    if st["residual"] is not None:
        s = s + st["residual"].float()
    f["s"] = s
    if st["w_next"] is not None:
        f["rs"] = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
        f["sn"] = s * f["rs"]
    return f


def _plain_norm(st):
    f, io = _norm_parts(st), st["y"].dtype
    return {"s": f["s"].to(io), "n": (f["sn"] * st["w_next"]).to(io) if st["w_next"] is not None else None}


def _plain_norm_train(st):
    c, f, io = st["case"], _norm_parts(st), st["y"].dtype
    ds, out = st["ds"].float(), _plain_norm(st)
    if st["dn"] is not None:
        dn = st["dn"].float()
        t = dn * st["w_next"]
        out["dw_next"] = (dn * f["sn"]).sum(0)
        ds = ds + f["rs"] * (t - f["sn"] * (t * f["sn"]).mean(-1, keepdim=True))
    dh = ds
    if st["scale"] is not None:
        out["dscale"] = (ds * f["h"]).sum(0)
        dh = ds * st["scale"]
    dp = dh
    if st["gate"] is not None:
        out["dgate"] = (dh * f["p"] * f["sig"] * (1.0 + f["z"] * (1.0 - f["sig"]))).to(io)
        dp = dh * f["silu"]
    dp = dp.view(c["M"], -1, c["group"])
    out["dw"] = (dp * f["yn"]).sum((0, 1))
    t = dp * st["w"]
    out["dy"] = (f["ry"] * (t - f["yn"] * (t * f["yn"]).mean(-1, keepdim=True))).view(c["M"], c["K"]).to(io)
    if st["residual"] is not None:
        out["dresidual"] = ds.to(io)
    return out


_plain = {"gdr": _plain_gdr, "gdr_train": _plain_gdr_train, "gdr_step": _plain_step, "norm": _plain_norm,
          "norm_train": _plain_norm_train}


# --------------------------------------------------------------------------------------------------
# the package's calls

def _own_gdr(st):
    import selective_state_space_73_amd as ss
    y = ss.ss_gdr_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], state=st["state"], reset=st["reset"],
                      eps=EPS_QK if st["case"]["unit"] else None)
    return {"y": y} if st["state"] is None else {"y": y, "state": st["state"]}


def _own_gdr_train(st):
    import selective_state_space_73_amd as ss
    c, x = st["case"], (st["q"], st["k"], st["v"], st["g"], st["beta"])
    eps = EPS_QK if c["unit"] else None
    ckpt = torch.empty(ss.gdr_ckpt_shape(c["B"], c["L"], c["H"], c["K"], c["V"]), device="cuda")
    y = ss.ss_gdr_fwd(*x, state=st["state"], reset=st["reset"], ckpt=ckpt, eps=eps)
    g = ss.ss_gdr_bwd(*x, ckpt, st["dy"], reset=st["reset"], dstate_final=st["dstate"], eps=eps)
    out = {"y": y, **{k: g[k] for k in ("dq", "dk", "dv", "dg", "dbeta", "dstate_init")}}
    return out if st["state"] is None else {**out, "state": st["state"]}


def _own_step(st):
    import selective_state_space_73_amd as ss
    y = ss.ss_gdr_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], eps=EPS_QK if st["case"]["unit"] else None)
    return {"y": y, "state": st["state"]}


def _own_norm(st):
    import selective_state_space_73_amd as ss
    s, n = ss.ss_gnorm_fwd(st["y"], st["w"], gate=st["gate"], residual=st["residual"], scale=st["scale"], w_next=st["w_next"],
                           eps=EPS)
    return {"s": s, "n": n}


def _own_norm_train(st):
    import selective_state_space_73_amd as ss
    out = _own_norm(st)
    g = ss.ss_gnorm_bwd(st["y"], st["w"], st["ds"], dn=st["dn"], gate=st["gate"], residual=st["residual"], scale=st["scale"],
                        w_next=st["w_next"], eps=EPS)
    return {**out, **{k: v for k, v in g.items() if v is not None}}


_own = {"gdr": _own_gdr, "gdr_train": _own_gdr_train, "gdr_step": _own_step, "norm": _own_norm, "norm_train": _own_norm_train}


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    e = {"f32": 4, "bf16": 2}[c["dtype"]]
    if op.startswith("gdr"):
        n, heads = c["B"] * c["L"], c["B"] * c["H"]
        kv, state = c["K"] * c["V"], 4 * heads * c["K"] * c["V"]
        io = n * e * (2 * c["Hk"] * c["K"] + 2 * c["H"] * c["V"]) + 8 * n * c["H"] + (n if c["docs"] else 0)
        both = state * 2 if c["state"] or op == "gdr_step" else 0
        if op != "gdr_train":
            return {"bytes": io + both, "flops": 7 * n * c["H"] * kv}
        return {"bytes": 2 * io + both + state * (2 if c["state"] else 1), "flops": 24 * n * c["H"] * kv}
    M, K = c["M"], c["K"]
    rows = 2 + sum(bool(c[k]) for k in ("gate", "residual", "next"))
    params = 4 * (c["group"] + (K if c["residual"] else 0) + (K if c["next"] else 0))
    if op == "norm":
        return {"bytes": rows * M * K * e + params, "flops": 14 * M * K}
    # the gradients: of s and n in, of y, gate and residual out
    return {"bytes": 2 * rows * M * K * e + 2 * params, "flops": 50 * M * K}


# --------------------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token

F64 = torch.float64


def _length(x):
    return torch.sqrt((x ** 2).sum(-1, keepdim=True) + EPS_QK)


def _exact_gdr(c, st):
    op, rep = c["op"], c["H"] // c["Hk"]
    B, L, H, K, V = c["B"], c["L"], c["H"], c["K"], c["V"]
    per = 3e-5 + 5 * 8 * B * H * K * V / 2.5e12                        # seconds of a token's step, about
    if L * per * (4 if op == "gdr_train" else 1) > 18:
        return None
    q0, k0, v, g, beta = (st[n].to(F64) if op != "gdr_step" else st[n].to(F64)[:, None] for n in ("q", "k", "v", "g", "beta"))
    lq, lk = (_length(q0), _length(k0)) if c["unit"] else (torch.ones_like(q0[..., :1]), torch.ones_like(k0[..., :1]))
    q = torch.repeat_interleave(q0 / lq, rep, dim=2) / math.sqrt(K)
    k = torch.repeat_interleave(k0 / lk, rep, dim=2)
    a = torch.exp(g)
    if st["reset"] is not None:
        a = torch.where((st["reset"] != 0)[..., None], torch.zeros_like(a), a)
    S = st["state"].to(F64) if st["state"] is not None else torch.zeros(B, H, K, V, dtype=F64, device=v.device)

    def token(S, t):
        """The decayed state, what the value lacks, and the next state."""
        d = S * a[:, t, :, None, None]
        r = v[:, t] - (d * k[:, t, :, :, None]).sum(2)
        return d, r, torch.addcmul(d, k[:, t, :, :, None], (beta[:, t, :, None] * r)[:, :, None, :])

    y = torch.empty(B, L, H, V, dtype=F64, device=v.device)
    seg, starts = max(16, int(math.sqrt(L))), []
    for t in range(L):
        if op == "gdr_train" and t % seg == 0:
            starts.append(S)
        S = token(S, t)[2]
        y[:, t] = (S * q[:, t, :, :, None]).sum(2)
    if op == "gdr_step":
        return {"y": y[:, 0], "state": S}
    out = {"y": y}
    if op == "gdr_train":
        dy = st["dy"].to(F64)
        adj = st["dstate"].to(F64) if st["dstate"] is not None else torch.zeros_like(S)
        dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
        for b in reversed(range(len(starts))):
            states, s = [], starts[b]
            for t in range(b * seg, min(L, b * seg + seg)):
                states.append(s)
                s = token(s, t)[2]
            for t in reversed(range(b * seg, min(L, b * seg + seg))):
                d, r, after = token(states[t - b * seg], t)
                dq[:, t] = (after * dy[:, t, :, None, :]).sum(-1)
                adj = torch.addcmul(adj, q[:, t, :, :, None], dy[:, t, :, None, :])
                du = (adj * k[:, t, :, :, None]).sum(2)
                db[:, t] = (du * r).sum(-1)
                dr = beta[:, t, :, None] * du
                dv[:, t] = dr
                dk[:, t] = (adj * (beta[:, t, :, None] * r)[:, :, None, :]).sum(-1) - (d * dr[:, :, None, :]).sum(-1)
                adj = torch.addcmul(adj, k[:, t, :, :, None], dr[:, :, None, :], value=-1.0)
                dg[:, t] = (adj * d).sum((-1, -2))
                adj = adj * a[:, t, :, None, None]

        def keys(d, x0, ln):
            d = d.unflatten(2, (c["Hk"], rep)).sum(3)
            return (d - x0 * (x0 * d).sum(-1, keepdim=True) / ln ** 2) / ln if c["unit"] else d

        out.update(dq=keys(dq / math.sqrt(K), q0, lq), dk=keys(dk, k0, lk), dv=dv, dg=dg, dbeta=db, dstate_init=adj)
    if st["state"] is not None:
        out["state"] = S
    return out


def exact(case, seed):
    st, c, op = prepare(case, seed), case, case["op"]
    if op.startswith("gdr"):
        return _exact_gdr(c, st)
    G = c["group"]
    y, w = st["y"].to(F64).unflatten(1, (-1, G)), st["w"].to(F64)
    ly = torch.sqrt((y ** 2).sum(-1, keepdim=True) / G + EPS)
    p = (y / ly * w).flatten(1)
    z = st["gate"].to(F64) if st["gate"] is not None else None
    e = torch.exp(-z) if z is not None else None
    act = z / (1.0 + e) if z is not None else torch.ones_like(p)
    alpha = st["scale"].to(F64) if st["scale"] is not None else torch.ones(c["K"], dtype=F64, device=p.device)
    s = alpha * act * p + (st["residual"].to(F64) if st["residual"] is not None else 0.0)
    wn = st["w_next"].to(F64) if st["w_next"] is not None else None
    ls = torch.sqrt((s ** 2).sum(-1, keepdim=True) / c["K"] + EPS)
    out = {"s": s, "n": s / ls * wn if wn is not None else None}
    if op == "norm_train":
        ds = st["ds"].to(F64)
        if wn is not None:
            dn = st["dn"].to(F64)
            out["dw_next"] = (dn * s / ls).sum(0)
            ds = ds + dn * wn / ls - s * (dn * wn * s).sum(-1, keepdim=True) / (c["K"] * ls ** 3)
        if st["scale"] is not None:
            out["dscale"] = (ds * act * p).sum(0)
        if z is not None:
            out["dgate"] = ds * alpha * p * (1.0 + e + z * e) / (1.0 + e) ** 2
        dp = (ds * alpha * act).unflatten(1, (-1, G))
        out["dw"] = (dp * y / ly).sum(1).sum(0)
        out["dy"] = (dp * w / ly - y * (dp * w * y).sum(-1, keepdim=True) / (G * ly ** 3)).flatten(1)
        if st["residual"] is not None:
            out["dresidual"] = ds
    return out
