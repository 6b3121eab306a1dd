"""The operators around the selective scan that are timed: what is called, on which inputs, and their plain forms.

Six calls of the package, as a program with recurrent layers makes them:

* ``glr``    a gated linear recurrence over whole sequences (``ss_glr_fwd``):
             s = sigmoid(r), a = exp(A s), h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, y = h,
             where reset[b, t] != 0 sets a_t = 0 (a new document starts at that token);
* ``train``  the same and its gradients (``ss_glr_fwd`` with checkpoints, ``ss_glr_bwd``);
* ``step``   the same for one token of each stream (``ss_glr_step``), the state updated in place;
* ``norm``   s = x + residual, RMS norm of s, rounded to 8-bit floating point (e4m3) with a scale for each
             block of 128 columns (``ss_norm_q8``);
* ``quant``  the same rounding alone, in blocks of 1 x 128 (activations) or 128 x 128 (weights) (``ss_quant_q8``);
* ``gemm``   the product of two such matrices, Y = X W^T (+ R) (``ss_gemm_q8``).

``own`` false computes each in its plain form, with elementary torch operations in 32 bits; true calls the package.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
QMAX = 448.0          # largest finite e4m3 value
TINY = 2.0 ** -126    # smallest scale
BLK = 128             # columns (and, for weights, rows) that share a scale
CKPT = 64             # tokens between the recurrence's checkpoints


def listed():
    return [
        # one short prompt of a small model: latency
        dict(name="glr prompt B1 L64 D512", op="glr", B=1, L=64, D=512, dtype="f32", fused=False, docs=0, state=False),
        # one very long sequence, prefilled in pieces: the state goes in and out
        dict(name="glr long B1 L131072 D2048", op="glr", B=1, L=131072, D=2048, dtype="bf16", fused=False, docs=0, state=True),
        # a training step's recurrence at the training width, inputs as slices of one projection's output
        dict(name="train B8 L2048 D5120", op="train", B=8, L=2048, D=5120, dtype="bf16", fused=True, docs=0, state=False),
        # several documents packed into ragged rows, odd width, full precision, states carried over
        dict(name="train packed B3 L1001 D1537", op="train", B=3, L=1001, D=1537, dtype="f32", fused=False, docs=5, state=True),
        # one token of each of 64 streams
        dict(name="step S64 D8192", op="step", B=64, D=8192, dtype="bf16"),
        # the norm in front of a layer: 64 streams' tokens, and a training batch's
        dict(name="norm M64 K2560", op="norm", M=64, K=2560, dtype="bf16", residual=True),
        dict(name="norm M16384 K2560", op="norm", M=16384, K=2560, dtype="bf16", residual=True),
        # a mixer's 32-bit output on its way to the projection back, and a weight matrix when it is loaded
        dict(name="quant rows M16384 K5120", op="quant", M=16384, K=5120, dtype="f32", square=False),
        dict(name="quant weights 10240 x 2560", op="quant", M=10240, K=2560, dtype="bf16", square=True),
        # the widening projection: 64 streams' tokens, and a training batch's
        dict(name="gemm M64 N10240 K2560", op="gemm", M=64, N=10240, K=2560, out="bf16", residual=False),
        dict(name="gemm M16384 N10240 K2560", op="gemm", M=16384, N=10240, K=2560, out="bf16", residual=False),
        # a projection back to an odd width with the residual added, over a short ragged prompt
        dict(name="gemm M201 N2561 K5120", op="gemm", M=201, N=2561, K=5120, out="f32", residual=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr", "train", "step", "norm", "quant", "gemm"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("glr", "train"):
        B, L = _log(rng, 1, 8), _log(rng, 1, 131072 if op == "glr" else 8192)
        most = (1 << 26) // (B * L) if op == "glr" else (1 << 25) // (B * L)
        D = _log(rng, 8, max(8, min(8192, most)))
        return dict(op=op, B=B, L=L, D=D, dtype=dtype, fused=rng.random() < 0.4, docs=rng.choice([0, 0, 1, 7]),
                    state=rng.random() < 0.5)
    if op == "step":
        return dict(op=op, B=_log(rng, 1, 256), D=_log(rng, 8, 8192), dtype=dtype)
    if op == "norm":
        M = _log(rng, 1, 16384)
        return dict(op=op, M=M, K=_log(rng, 8, min(8192, (1 << 25) // M)), dtype=dtype, residual=rng.random() < 0.6)
    if op == "quant":
        M = _log(rng, 1, 16384)
        return dict(op=op, M=M, K=_log(rng, 8, min(8192, (1 << 26) // M)), dtype=dtype, square=rng.random() < 0.5)
    # rows of the 8-bit operands start on 16 bytes
    return dict(op="gemm", M=_log(rng, 1, 16384), N=_log(rng, 8, 10240), K=16 * _log(rng, 1, 160),
                out=rng.choice(["f32", "bf16"]), residual=rng.random() < 0.3)


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

    op = c["op"]
    if op in ("glr", "train", "step"):
        B, D, dt = c["B"], c["D"], c["dtype"]
        # exp(A / 8) evenly spread over [0.9, 0.999]: memories of a few tokens to about two thousand
        st["A"] = 8.0 * torch.log(uniform(0.9, 0.999, D))
        if op == "step":
            st.update({k: normal(B, D, dtype=dt) for k in ("x", "r", "i")})
            st["state"] = normal(B, D)
            return st
        L = c["L"]
        if c["fused"]:
            st["x"], st["r"], st["i"] = normal(B, L, 3 * D, dtype=dt).split(D, dim=-1)
        else:
            st.update({k: normal(B, L, D, dtype=dt) for k in ("x", "r", "i")})
        st["state"] = normal(B, D) if c["state"] else None
        st["reset"] = None
        if c["docs"]:
            st["reset"] = torch.zeros(B, L, dtype=torch.uint8, device="cuda")
            at = torch.randint(0, L, (B, c["docs"]), generator=g, device="cuda")
            st["reset"].scatter_(1, at, 1)
        if op == "train":
            st["dy"] = normal(B, L, D, dtype=dt)
            st["dstate"] = normal(B, D) if c["state"] else None
    elif op == "norm":
        st["x"] = normal(c["M"], c["K"], dtype=c["dtype"])
        st["residual"] = normal(c["M"], c["K"], dtype=c["dtype"], scale=3.0) if c["residual"] else None
        st["w"] = 1.0 + normal(c["K"], scale=0.1)
    elif op == "quant":
        st["x"] = normal(c["M"], c["K"], dtype=c["dtype"], scale=0.02 if c["square"] else 1.0)
    else:
        M, N, K = c["M"], c["N"], c["K"]
        st["xq"], st["xs"] = _quant(normal(M, K), False)
        st["wq"], st["ws"] = _quant(normal(N, K, scale=K ** -0.5), True)
        st["residual"] = normal(M, N, dtype=c["out"]) if c["residual"] else None
    return st


def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


# --------------------------------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, in log2(L) steps that each double the reach."""
    s = 1
    while s < b.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _gates(st):
    """sigmoid(r), log a, a, the write coefficient and sigmoid(i), in 32 bits."""
    s, gi = torch.sigmoid(st["r"].float()), torch.sigmoid(st["i"].float())
    la = st["A"] * s
    a, w = torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))
    if st.get("reset") is not None:
        at = (st["reset"] != 0)[..., None]
        a, w = a.masked_fill(at, 0.0), w.masked_fill(at, 1.0)
    return s, la, a, w, gi


def _states(st, a, b):
    """The state before and after every token."""
    h0 = st["state"]
    if h0 is None:
        h0 = torch.zeros_like(b[:, 0])
    b = torch.cat([(b[:, 0] + a[:, 0] * h0)[:, None], b[:, 1:]], 1)
    h = _scan(a, b)
    return torch.cat([h0[:, None], h[:, :-1]], 1), h


def _plain_glr(st):
    _, _, a, w, gi = _gates(st)
    _, h = _states(st, a, w * gi * st["x"].float())
    out = {"y": h.to(st["x"].dtype)}
    if st["state"] is not None:
        st["state"].copy_(h[:, -1])
        out["state"] = st["state"]
    return out


def _plain_train(st):
    x, dy = st["x"].float(), st["dy"].float()
    s, la, a, w, gi = _gates(st)
    before, h = _states(st, a, w * gi * x)
    # the adjoint runs backward in time: g_t = dy_t + a_{t+1} g_{t+1}
    if st["dstate"] is not None:
        dy = torch.cat([dy[:, :-1], (dy[:, -1] + st["dstate"])[:, None]], 1)
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _scan(nxt.flip(1), dy.flip(1)).flip(1)
    # d(log a) through the decay and through the write coefficient (dw/d(log a) = -a^2 / w)
    dla = g * (a * before - torch.where(w > 0, a * a / w, 0.0) * gi * x)
    io = st["x"].dtype
    out = {"y": h.to(io), "dx": (g * w * gi).to(io), "dr": (dla * la * (1.0 - s)).to(io),
           "di": (g * w * x * gi * (1.0 - gi)).to(io), "dA": (dla * s).sum((0, 1), dtype=torch.float64).float(),
           "dstate_init": a[:, 0] * g[:, 0]}
    if st["state"] is not None:
        st["state"].copy_(h[:, -1])
        out["state"] = st["state"]
    return out


def _plain_step(st):
    _, _, a, w, gi = _gates(st)
    st["state"].copy_(a * st["state"] + w * gi * st["x"].float())
    return {"y": st["state"].to(st["x"].dtype), "state": st["state"]}


def _blocks(x, square):
    """x, padded with zeros to whole blocks, as [row block, rows, column block, columns]."""
    M, K = x.shape
    rows = BLK if square else 1
    x = torch.nn.functional.pad(x, (0, -K % BLK, 0, -M % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // BLK, BLK)


def _quant(x, square):
    """e4m3 values and their scales: scale = max |x| / 448 over the block (2^-126 at least)."""
    v = _blocks(x.float(), square)
    scale = (v.abs().amax((1, 3)) / QMAX).clamp_min(TINY)
    q = (v / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(v.shape[0] * v.shape[1], -1)
    return q[:x.shape[0], :x.shape[1]].contiguous(), scale


def _plain_norm(st):
    s = st["x"].float()
    if st["residual"] is not None:
        s = s + st["residual"].float()
    n = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-5) * st["w"]
    q, scale = _quant(n, False)
    return {"q": q, "scale": scale, "sum": s.to(st["x"].dtype) if st["residual"] is not None else None}


def _plain_quant(st):
    q, scale = _quant(st["x"], st["case"]["square"])
    return {"q": q, "scale": scale}


def _values(q, scale, square):
    v = _blocks(q.float(), square) * scale[:, None, :, None]
    return v.view(v.shape[0] * v.shape[1], -1)[:q.shape[0], :q.shape[1]]


def _plain_gemm(st):
    y = _values(st["xq"], st["xs"], False) @ _values(st["wq"], st["ws"], True).t()
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(DT[st["case"]["out"]])


_plain = {"glr": _plain_glr, "train": _plain_train, "step": _plain_step, "norm": _plain_norm, "quant": _plain_quant,
          "gemm": _plain_gemm}


# --------------------------------------------------------------------------------------------------
# the package's calls

def _own_glr(st):
    import selective_state_space_73_amd as ss
    y = ss.ss_glr_fwd(st["x"], st["r"], st["i"], st["A"], state=st["state"], reset=st["reset"])
    return {"y": y} if st["state"] is None else {"y": y, "state": st["state"]}


def _own_train(st):
    import selective_state_space_73_amd as ss
    c = st["case"]
    ckpt = torch.empty(ss.glr_ckpt_shape(c["B"], c["L"], c["D"]), device="cuda")
    y = ss.ss_glr_fwd(st["x"], st["r"], st["i"], st["A"], state=st["state"], reset=st["reset"], ckpt=ckpt)
    g = ss.ss_glr_bwd(st["x"], st["r"], st["i"], st["A"], ckpt, st["dy"], reset=st["reset"], dstate_final=st["dstate"])
    out = {"y": y, **{k: g[k] for k in ("dx", "dr", "di", "dA", "dstate_init")}}
    return out if st["state"] is None else {**out, "state": st["state"]}


def _own_step(st):
    import selective_state_space_73_amd as ss
    y = ss.ss_glr_step(st["x"], st["r"], st["i"], st["A"], st["state"])
    return {"y": y, "state": st["state"]}


def _own_norm(st):
    import selective_state_space_73_amd as ss
    q, scale, s = ss.ss_norm_q8(st["x"], st["w"], residual=st["residual"], eps=1e-5)
    return {"q": q, "scale": scale, "sum": s}


def _own_quant(st):
    import selective_state_space_73_amd as ss
    q, scale = ss.ss_quant_q8(st["x"], square=st["case"]["square"])
    return {"q": q, "scale": scale}


def _own_gemm(st):
    import selective_state_space_73_amd as ss
    return ss.ss_gemm_q8(st["xq"], st["xs"], st["wq"], st["ws"], residual=st["residual"],
                         out_dtype=DT[st["case"]["out"]])


_own = {"glr": _own_glr, "train": _own_train, "step": _own_step, "norm": _own_norm, "quant": _own_quant,
        "gemm": _own_gemm}


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    e = {"f32": 4, "bf16": 2}
    if op == "step":
        n = c["B"] * c["D"]
        return {"bytes": n * (4 * e[c["dtype"]] + 8) + 4 * c["D"], "flops": 20 * n}
    if op in ("glr", "train"):
        n, rows = c["B"] * c["L"] * c["D"], c["B"] * c["D"]
        extra = 4 * c["D"] + (c["B"] * c["L"] if c["docs"] else 0) + (8 * rows if c["state"] else 0)
        if op == "glr":
            return {"bytes": n * 4 * e[c["dtype"]] + extra, "flops": 20 * n}
        return {"bytes": n * 8 * e[c["dtype"]] + extra + 4 * c["D"] + 4 * rows * (2 if c["state"] else 1), "flops": 60 * n}
    if op == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // BLK)
        y = M * N * e[c["out"]] * (2 if c["residual"] else 1)
        return {"bytes": (M + N) * K + 4 * kb * (M + -(-N // BLK)) + y, "flops": 2 * M * N * K}
    M, K, kb = c["M"], c["K"], -(-c["K"] // BLK)
    if op == "norm":
        moved = M * K * (e[c["dtype"]] * (3 if c["residual"] else 1) + 1) + 4 * M * kb + 4 * K
        return {"bytes": moved, "flops": 8 * M * K}
    return {"bytes": M * K * (e[c["dtype"]] + 1) + 4 * kb * (-(-M // BLK) if c["square"] else M), "flops": 4 * M * K}


# --------------------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token and value by value

def _e4m3(v):
    """v rounded to the nearest e4m3 value (4 significant bits, steps of 2^-9 at least), ties to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp_min(-9))
    return (torch.round(v / step) * step).clamp(-QMAX, QMAX)


def _exact_quant(v, square):
    M, K = v.shape
    col = torch.arange(K, device=v.device) // BLK
    row = torch.arange(M, device=v.device) // (BLK if square else 1)
    top = torch.zeros(M, int(col[-1]) + 1, dtype=torch.float64, device=v.device)
    top.scatter_reduce_(1, col.expand(M, K), v.abs(), "amax")
    scale = torch.zeros(int(row[-1]) + 1, top.shape[1], dtype=torch.float64, device=v.device)
    scale.scatter_reduce_(0, row[:, None].expand_as(top), top, "amax")
    scale = torch.maximum(scale / QMAX, torch.full_like(scale, TINY))
    return _e4m3(v / scale[row][:, col]), scale


def exact(case, seed):
    st, c, op = prepare(case, seed), case, case["op"]
    f64 = torch.float64
    if op in ("glr", "train", "step"):
        x, r, i = (st[k].to(f64) if op != "step" else st[k].to(f64)[:, None] for k in ("x", "r", "i"))
        A = st["A"].to(f64)
        B, L, D = x.shape
        s, gi = 1.0 / (1.0 + torch.exp(-r)), 1.0 / (1.0 + torch.exp(-i))
        a = torch.exp(A * s)
        w2 = 1.0 - a * a
        if st.get("reset") is not None:
            keep = (st["reset"] == 0).to(f64)[..., None]
            a, w2 = a * keep, w2 * keep + (1.0 - keep)
        w = torch.sqrt(w2)
        v = gi * x
        h = torch.empty_like(a)
        first = st["state"].to(f64) if st["state"] is not None else torch.zeros(B, D, dtype=f64, device=x.device)
        b, last = w * v, first
        for t in range(L):
            torch.addcmul(b[:, t], a[:, t], last, out=h[:, t])
            last = h[:, t]
        if op == "step":
            return {"y": h[:, 0], "state": h[:, 0]}
        out = {"y": h}
        if op == "train":
            g = st["dy"].to(f64)
            if st["dstate"] is not None:
                g[:, L - 1] += st["dstate"].to(f64)
            for t in range(L - 2, -1, -1):
                g[:, t].addcmul_(a[:, t + 1], g[:, t + 1])
            prev = torch.cat([first[:, None], h[:, :-1]], 1)
            # per token: dh/da = h_{t-1} - (a / w) v, da/ds = A a, da/dA = s a
            da = g * (prev - a / w * v)
            out.update(dx=g * w * gi, di=g * w * x * gi * (1.0 - gi), dr=da * a * A * s * (1.0 - s),
                       dA=(da * a * s).sum(1).sum(0), dstate_init=a[:, 0] * g[:, 0])
        if st["state"] is not None:
            out["state"] = h[:, -1]
        return out
    if op == "norm":
        s = st["x"].to(f64)
        if st["residual"] is not None:
            s = s + st["residual"].to(f64)
        q, scale = _exact_quant(s / torch.sqrt((s ** 2).sum(-1, keepdim=True) / c["K"] + 1e-5) * st["w"].to(f64), False)
        return {"q": q, "scale": scale, "sum": s if st["residual"] is not None else None}
    if op == "quant":
        q, scale = _exact_quant(st["x"].to(f64), c["square"])
        return {"q": q, "scale": scale}
    col = torch.arange(c["K"], device="cuda") // BLK
    row = torch.arange(c["N"], device="cuda") // BLK
    x = st["xq"].to(f64) * st["xs"].to(f64)[:, col]
    y = x @ (st["wq"].to(f64) * st["ws"].to(f64)[row][:, col]).t()
    return y if st["residual"] is None else y + st["residual"].to(f64)
