"""64-bit definitions of the operators around the scan (include/selscan_ops.h), in torch on
the CPU, token by token and value by value.

TEST INFRASTRUCTURE ONLY, like the rest of this package: the HIP library never uses it, and it
shares no code with it.
"""
from __future__ import annotations

import numpy as np
import torch

from . import block as _block
from . import default as _default

F64 = torch.float64


def _gates(x, r, i, A, reset):
    s, g = 1.0 / (1.0 + torch.exp(-r)), 1.0 / (1.0 + torch.exp(-i))
    la = A * s
    a, w = torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))
    if reset is not None:
        on = (reset != 0).unsqueeze(-1)
        a, w = a.masked_fill(on, 0.0), w.masked_fill(on, 1.0)
    return s, g, la, a, w


def glr_fwd(x, r, i, A, state=None, reset=None):
    """(y, final state, checkpoints): h_t = a_t h_{t-1} + w_t sigmoid(i_t) x_t one token after
    the other, the state in front of a reset token not read."""
    x, r, i, A = (t.detach().cpu().to(F64) if not t.requires_grad else t for t in (x, r, i, A))
    B, L, D = x.shape
    reset = None if reset is None else reset.cpu()
    s, g, la, a, w = _gates(x, r, i, A, reset)
    h = torch.zeros(B, D, dtype=F64) if state is None else (state if state.requires_grad else state.cpu().to(F64))
    ys, ck = [], []
    for t in range(L):
        if t % 64 == 0:
            ck.append(h)
        b = w[:, t] * g[:, t] * x[:, t]
        old = a[:, t] * h
        if reset is not None:
            old = torch.where((reset[:, t] != 0)[:, None], torch.zeros_like(old), old)
        h = old + b
        ys.append(h)
    return torch.stack(ys, 1), h, torch.stack(ck, 1)


def glr_bwd(x, r, i, A, dy, state=None, reset=None, dstate_final=None):
    """Gradients by the chain rule in reverse order, and for each the size its terms reach
    (what its rounding errors are measured against): {name: (value, scale)}."""
    x, r, i, A, dy = (t.detach().cpu().to(F64) for t in (x, r, i, A, dy))
    B, L, D = x.shape
    reset = None if reset is None else reset.cpu()
    s, g, la, a, w = _gates(x, r, i, A, reset)
    h0 = torch.zeros(B, D, dtype=F64) if state is None else state.cpu().to(F64)
    y, _, _ = glr_fwd(x, r, i, A, h0, reset)
    before = torch.cat([h0[:, None], y[:, :-1]], 1)
    K = torch.zeros(B, D, dtype=F64) if dstate_final is None else dstate_final.cpu().to(F64)
    G = torch.zeros_like(x)
    for t in range(L - 1, -1, -1):
        G[:, t] = dy[:, t] + K
        K = a[:, t] * G[:, t]
        if reset is not None:
            K = torch.where((reset[:, t] != 0)[:, None], torch.zeros_like(K), K)
    v = g * x
    q = torch.where(w > 0, a * a / w, torch.zeros_like(w))
    dla = G * (a * before - q * v)
    size = G.abs() * (a * before.abs() + q * v.abs())
    if reset is not None:
        on = (reset != 0).unsqueeze(-1)
        dla, size = dla.masked_fill(on, 0.0), size.masked_fill(on, 0.0)
    top = G.abs().amax((0, 1))                                       # per channel

    def pair(val, scale):
        return val, scale

    return {"dx": pair(G * w * g, top), "di": pair(G * w * v * (1 - g), top * v.abs().amax((0, 1))),
            "dr": pair(dla * la * (1 - s), (size * la.abs()).amax((0, 1))),
            "dA": pair((dla * s).sum((0, 1)), (size * s).sum((0, 1))), "dstate_init": pair(K, top)}


def memory(r, A, reset=None):
    """Longest memory among the channels, in tokens: 1 / min(1 - a)."""
    la = A.cpu().to(F64) / (1.0 + torch.exp(-r.detach().cpu().to(F64)))
    return float((1.0 / (-torch.expm1(la)).clamp_min(1e-30)).max())


# ---------------------------------------------------------------------------
# 8-bit floating point with block scales

Q8_MAX, Q8_TINY = 448.0, 2.0 ** -126


def rms_norm(x, w, residual=None, eps=1e-5):
    """(n, s): s = x + residual, n = s / sqrt(mean(s^2) + eps) * w."""
    s = x.cpu().to(F64)
    if residual is not None:
        s = s + residual.cpu().to(F64)
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * w.cpu().to(F64), s


def block_tops(v, square=False):
    """Largest |v| of every block, NaN left out, block by block."""
    v = v.cpu().to(F64).abs()
    M, K = v.shape
    rows = 128 if square else 1
    out = torch.zeros(-(-M // rows), -(-K // 128), dtype=F64)
    for a in range(out.shape[0]):
        for b in range(out.shape[1]):
            blk = v[a * rows:(a + 1) * rows, b * 128:(b + 1) * 128]
            out[a, b] = torch.nan_to_num(blk, nan=0.0, posinf=float("inf")).max()
    return out


def spread(scale, M, K, square=False):
    """A scale per value."""
    row = torch.arange(M) // (128 if square else 1)
    return scale.cpu().to(F64)[row][:, torch.arange(K) // 128]


def values(q, scale, square=False):
    """What q and its scales stand for."""
    return q.cpu().to(torch.float32).to(F64) * spread(scale, q.shape[0], q.shape[1], square)


def half_step(v, scale):
    """Half the distance of neighbouring e4m3 values at v / scale, times scale: 2^-4 of |v| at
    most, 2^-10 scale below the smallest normal value."""
    return torch.maximum(v.abs() * 2.0 ** -4, scale * 2.0 ** -10)


def nearest(v, top):
    """The e4m3 value nearest to 448 v / top (to v 2^126 under the smallest scale), ties to even,
    for v of at most 24 bits and top >= |v| of its block, element by element: 448 v and a midpoint
    times top both fit in 53 bits, so the two sides are compared exactly."""
    v, top = v.cpu().to(F64), top.cpu().to(F64).clamp_min(Q8_MAX * Q8_TINY)
    a = Q8_MAX * v.abs()
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a / top)[1] - 4).clamp_min(-9))
    k = torch.floor(a / top / step)
    k = torch.where(k * step * top > a, k - 1, k)                   # the quotient itself was rounded
    k = torch.where((k + 1) * step * top <= a, k + 1, k)
    mid = (k + 0.5) * step * top
    up = (a > mid) | ((a == mid) & (k % 2 == 1))
    return torch.copysign((k + up.to(F64)) * step, v)


# ---------------------------------------------------------------------------
# the block with 8-bit projections, in pieces that a rounding separates

def block_core(xi, z, W, R, ssm_state, conv_state, zoh=False):
    """From the input projection's two halves [B,L,Di] to the scan's output, as in the block:
    (y [B,L,Di], final ssm_state [B,Di,N], final conv_state [B,Di,3]), numpy float64. W: the
    block's weights as numpy arrays; states as such or None."""
    N = W["A"].shape[1]
    u, cs = _block.conv_silu(xi, W["conv_w"], W["conv_b"], conv_state)
    xp = u @ np.asarray(W["W_x"], np.float64).T
    dr, Bm, Cm = xp[..., :R], xp[..., R:R + N], xp[..., R + N:]
    delta = dr @ np.asarray(W["W_dt"], np.float64).T
    h0 = np.zeros((xi.shape[0], xi.shape[2], N)) if ssm_state is None else ssm_state
    y, hs, _ = _default().conv_scan_fwd(u, delta, W["A"], Bm, Cm, delta_bias=W["dt_bias"], D=W["D"], z=z, ssm_state=h0,
                                             zoh=zoh)
    return y, hs, cs


def rounded_product(y, slack, wq, ws, out_half):
    """(y W^T, how far the 8-bit product of y may be from it), element by element, for y [M,K]
    (64-bit) known to +-slack [M,K] before it is rounded to 8 bits: half a step (taken from the
    true value: slack once more covers the difference) for each value, then fp32 sums of K terms;
    the output's own rounding (out_half) is the caller's."""
    w = values(wq, ws, square=True).abs()
    y = torch.as_tensor(y, dtype=F64)
    per = spread(block_tops(y) / Q8_MAX, *y.shape).clamp_min(Q8_TINY)
    off = half_step(y, per) + 2 * torch.as_tensor(slack, dtype=F64)
    sums = 2.0 ** -15
    return y @ values(wq, ws, square=True).T, off @ w.T + sums * ((y.abs() + off) @ w.T)


# ---------------------------------------------------------------------------
# the gated delta rule

def _unit(x, eps):
    return x if eps is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)


def gdr_fwd(q, k, v, g, beta, state=None, reset=None, scale=None, eps=1e-6):
    """(y, final state), token after token; differentiable where an input asks for it. A log decay of
    -200 or less, and a reset, is a decay of 0: the state in front of it is not read."""
    q, k, v, g, beta = (t if t.requires_grad else t.detach().cpu().to(F64) for t in (q, k, v, g, beta))
    B, L, Hk, K = q.shape
    H, V = v.shape[2:]
    q, k = (_unit(x, eps).repeat_interleave(H // Hk, 2) for x in (q, k))
    scale = K ** -0.5 if scale is None else scale
    S = torch.zeros(B, H, K, V, dtype=F64) if state is None else (state if state.requires_grad else state.cpu().to(F64))
    cut = g <= -200.0
    if reset is not None:
        cut = cut | (reset.cpu() != 0)[..., None]
    ys = []
    for t in range(L):
        gone = cut[:, t, :, None, None]
        a = torch.exp(torch.where(gone, torch.zeros_like(g[:, t, :, None, None]), g[:, t, :, None, None]))
        S = torch.where(gone, torch.zeros_like(S), S * a)
        kt, qt = k[:, t, :, :, None], q[:, t, :, :, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * kt).sum(2))
        S = S + kt * u[:, :, None, :]
        ys.append(scale * (S * qt).sum(2))
    y = torch.stack(ys, 1) if ys else torch.zeros(B, 0, H, V, dtype=F64)
    return y, S


def gdr_bwd(q, k, v, g, beta, dy, state=None, reset=None, dstate_final=None, scale=None, eps=1e-6):
    """Gradients by the chain rule in reverse order, token after token: {name: value}."""
    q0, k0, v, g, beta, dy = (t.detach().cpu().to(F64) for t in (q, k, v, g, beta, dy))
    B, L, Hk, K = q0.shape
    H, V = v.shape[2:]
    rep = H // Hk
    q, k = (_unit(x, eps).repeat_interleave(rep, 2) for x in (q0, k0))
    scale = K ** -0.5 if scale is None else scale
    a = torch.exp(g)
    cut = g <= -200.0
    if reset is not None:
        cut = cut | (reset.cpu() != 0)[..., None]
    S = torch.zeros(B, H, K, V, dtype=F64) if state is None else state.cpu().to(F64)
    before, lack, after = [], [], []
    for t in range(L):
        S = torch.where(cut[:, t, :, None, None], torch.zeros_like(S), S * a[:, t, :, None, None])
        before.append(S)
        lack.append(v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * lack[t])[:, :, None, :]
        after.append(S)
    W = torch.zeros(B, H, K, V, dtype=F64) if dstate_final is None else dstate_final.cpu().to(F64)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for t in range(L - 1, -1, -1):
        kt = k[:, t, :, :, None]
        dq[:, t] = scale * (after[t] * dy[:, t, :, None, :]).sum(-1)
        W = W + scale * q[:, t, :, :, None] * dy[:, t, :, None, :]
        wk = (W * kt).sum(2)
        db[:, t] = (wk * lack[t]).sum(-1)
        dv[:, t] = beta[:, t, :, None] * wk
        dk[:, t] = (W * (beta[:, t, :, None] * lack[t])[:, :, None, :]).sum(-1) - (before[t] * dv[:, t, :, None, :]).sum(-1)
        W = W - kt * dv[:, t, :, None, :]
        dg[:, t] = (before[t] * W).sum((-1, -2))
        W = torch.where(cut[:, t, :, None, None], torch.zeros_like(W), W * a[:, t, :, None, None])

    def keys(d, x):
        d = d.reshape(B, L, Hk, rep, K).sum(3)
        if eps is None:
            return d
        n2 = (x * x).sum(-1, keepdim=True) + eps
        return (d - x * (x * d).sum(-1, keepdim=True) / n2) / torch.sqrt(n2)

    return {"dq": keys(dq, q0), "dk": keys(dk, k0), "dv": dv, "dg": dg, "dbeta": db, "dstate_init": W}


# ---------------------------------------------------------------------------
# the norms around a layer

def gnorm_fwd(y, w, gate=None, residual=None, scale=None, w_next=None, eps=1e-5):
    """(s, n or None), differentiable where an input asks for it."""
    y, w, gate, residual, scale, w_next = (t if t is None or t.requires_grad else t.detach().cpu().to(F64)
                                           for t in (y, w, gate, residual, scale, w_next))
    G = w.numel()
    p = y.reshape(*y.shape[:-1], -1, G)
    p = (p / torch.sqrt((p * p).mean(-1, keepdim=True) + eps) * w).reshape(y.shape)
    h = p if gate is None else p * gate / (1.0 + torch.exp(-gate))
    s = h if scale is None else scale * h
    s = s if residual is None else residual + s
    n = None if w_next is None else s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * w_next
    return s, n


def gnorm_bwd(y, w, ds, dn=None, gate=None, residual=None, scale=None, w_next=None, eps=1e-5):
    """Gradients by hand: {name: (value, what its terms reach)}."""
    y, w, ds, dn, gate, residual, scale, w_next = (None if t is None else t.detach().cpu().to(F64)
                                                   for t in (y, w, ds, dn, gate, residual, scale, w_next))
    G, K = w.numel(), y.shape[-1]
    y = y.reshape(-1, K)
    M = y.shape[0]
    ds = torch.zeros_like(y) if ds is None else ds.reshape(M, K)
    yg = y.reshape(M, -1, G)
    ly = torch.sqrt((yg * yg).mean(-1, keepdim=True) + eps)
    yn = yg / ly
    p = (yn * w).reshape(M, K)
    z = None if gate is None else gate.reshape(M, K)
    sig = None if z is None else 1.0 / (1.0 + torch.exp(-z))
    act = torch.ones_like(p) if z is None else z * sig
    al = torch.ones(K, dtype=F64) if scale is None else scale
    s = al * act * p + (0.0 if residual is None else residual.reshape(M, K))
    out = {}
    if w_next is not None:
        ls = torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
        dn = torch.zeros_like(y) if dn is None else dn.reshape(M, K)
        out["dw_next"] = ((dn * s / ls).sum(0), (dn * s / ls).abs().sum(0))
        t = dn * w_next
        ds = ds + (t - s * (t * s).mean(-1, keepdim=True) / ls ** 2) / ls
    if residual is not None:
        out["dresidual"] = (ds, ds.abs().amax(-1, keepdim=True))
    if scale is not None:
        out["dscale"] = ((ds * act * p).sum(0), (ds * act * p).abs().sum(0))
    dh = ds * al
    if z is not None:
        dz = dh * p * (sig + act * (1.0 - sig))
        out["dgate"] = (dz, (dh * p).abs().amax(-1, keepdim=True))
    dp = (dh * act).reshape(M, -1, G)
    out["dw"] = ((dp * yn).sum((0, 1)), (dp * yn).abs().sum((0, 1)))
    t = dp * w
    dy = (t - yn * (t * yn).mean(-1, keepdim=True)) / ly
    out["dy"] = (dy.reshape(M, K), (t.abs().amax(-1, keepdim=True) / ly).expand_as(t).reshape(M, K))
    return out
