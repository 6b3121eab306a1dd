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
