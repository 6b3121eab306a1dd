"""GPU: the block with 8-bit projections (ss_block_q8_fwd, ss_block_q8_step) and runs of the
operators one behind another, against 64-bit definitions taken from one rounding to the next.

A rounding to 8 bits moves a value by up to 2^-4 of itself, and one that lies near a midpoint
goes either way for a last bit's difference before it. So each stretch between two roundings is
checked by itself: the input projection's result is taken from the same operators called one by
one (each with a test of its own), the definition runs in 64 bits from there to the scan's
output y, and the last product is bounded by half a step per value of y (oracle.ops.
rounded_product). With W_out the identity that bound is one value's half step.

Tolerances of the stretch between (relative, with the rms as the floor): 1e-4 with float32
weights, as for the scan and the block; with bf16 weights an activation enters the matrix cores
as two bf16 terms, off by 2^-16 of each term of delta, B and C: for sums of random signs that is
four times as much of their rms (4 sigma) where the operand itself is up to five times its rms,
three factors: 3 * 4 * 5 * 2^-16 < 1e-3.
"""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import maxrel
from oracle import ops as O

pytestmark = pytest.mark.gpu

ss = pytest.importorskip("selective_state_space_73_amd")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
MID = {"f32": 1e-4, "bf16": 1e-3}
F8 = torch.float8_e4m3fn


def weights(spec, identity=False):
    """(numpy weights, device weights with 8-bit projections)."""
    w = W.gen_block_weights(spec)
    if identity:
        w["W_out"] = np.eye(spec.d_model, spec.d_inner, dtype=np.float32)
    dev = {k: torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda() for k, v in w.items()}
    for k in ("W_in", "W_x", "W_dt", "W_out"):
        dev[k] = dev[k].to(DT[spec.io_dtype])
    return w, ss.block_q8_weights(dev)


def halves(x, g, di):
    """The input projection by single calls: xi, z in float32 on the device."""
    q, s, _ = ss.ss_norm_q8(x, g["norm_w"])
    p = ss.ss_gemm_q8(q, s, g["W_in"], g["S_in"], out_dtype=torch.float32)
    return p[..., :di], p[..., di:]


def check_out(out, x, y, g, io):
    """out against x + e4m3(y) W_out^T, y [B,L,Di] in 64 bits."""
    y = torch.as_tensor(y, dtype=torch.float64).reshape(-1, y.shape[-1])
    rms = y.square().mean().sqrt()
    want, off = O.rounded_product(y, MID[io] * torch.maximum(y.abs(), rms), g["W_out"], g["S_out"], HALF[io])
    want = want + x.double().cpu().reshape(want.shape)
    bound = off + (HALF[io] + 2.0 ** -23) * (want.abs() + off)
    err = (out.double().cpu().reshape(want.shape) - want).abs()
    worst = (err / bound).max().item()
    print(f"out: worst error over bound {worst:.3f}", flush=True)
    assert torch.isfinite(out).all() and worst <= 1.0


def host(t):
    return t.double().cpu().numpy()


CASES = [  # batch, tokens, d_model, expand, d_state, rank, identity W_out
    (1, 1, 16, 1, 4, 1, True), (2, 5, 48, 2, 8, 3, False), (3, 67, 144, 1, 16, 9, True), (2, 130, 256, 2, 16, 16, False),
    (1, 1030, 128, 1, 64, 8, True), (4, 300, 512, 2, 16, 32, False), (1, 4100, 64, 2, 16, 4, False)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,dm,expand,N,R,identity", CASES)
@pytest.mark.parametrize("states", [False, True])
def test_block(B, L, dm, expand, N, R, identity, io, states):
    spec = W.BlockSpec("q8", B, L, dm, expand=expand, d_state=N, dt_rank=R, io_dtype=io, seed=900 + L)
    w, g = weights(spec, identity)
    di = spec.d_inner
    x = torch.from_numpy(W.gen_block_input(spec)).to(DT[io]).cuda()
    st = W.gen_states(B, di, N, seed=spec.seed + 3) if states else None
    h, c = (torch.from_numpy(st[k]).cuda() for k in ("ssm_state", "conv_state")) if states else (None, None)
    xi, z = halves(x, g, di)
    before = torch.cat([c.transpose(1, 2), xi], 1) if states else None
    out = ss.ss_block_q8_fwd(x, g, R, ssm_state=h, conv_state=c)
    y, hr, _ = O.block_core(host(xi), host(z), w, R, *((st["ssm_state"], st["conv_state"]) if states else (None, None)))
    check_out(out, x, y, g, io)
    if states:
        assert torch.equal(c, before[:, -3:].transpose(1, 2))        # the projection's own values
        print(f"state {maxrel(host(h), hr):.2e}", flush=True)
        assert maxrel(host(h), hr) <= MID[io]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_block_zero_order_hold_without_optional_weights_in_place(io):
    spec = W.BlockSpec("q8zoh", 2, 50, 80, expand=2, d_state=16, dt_rank=5, io_dtype=io, seed=950)
    w, g = weights(spec)
    g = {k: v for k, v in g.items() if k not in ("conv_b", "dt_bias", "D")}
    w.update(conv_b=np.zeros(spec.d_inner), dt_bias=np.zeros(spec.d_inner), D=np.zeros(spec.d_inner))
    x = torch.from_numpy(W.gen_block_input(spec)).to(DT[io]).cuda()
    kept = x.clone()
    xi, z = halves(x, g, spec.d_inner)
    y, _, _ = O.block_core(host(xi), host(z), w, 5, None, None, zoh=True)
    out = ss.ss_block_q8_fwd(x, g, 5, zoh=True, out=x)
    assert out is x
    check_out(x, kept, y, g, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("S,dm", [(1, 64), (7, 144), (64, 512), (200, 128)])
def test_block_steps(S, dm, io):
    """Decode from carried states, and the same tokens in one forward call (few enough rows that
    the norm sums a row in one order in both: a value near a midpoint would go either way)."""
    T = 4
    spec = W.BlockSpec("q8step", S, T, dm, expand=2, d_state=16, io_dtype=io, seed=960 + S)
    w, g = weights(spec)
    di, R = spec.d_inner, spec.rank
    x = torch.from_numpy(W.gen_block_input(spec)).to(DT[io]).cuda()
    st = W.gen_states(S, di, 16, seed=961)
    h, c = (torch.from_numpy(st[k]).cuda() for k in ("ssm_state", "conv_state"))
    hf, cf = h.clone(), c.clone()
    hr, cr = st["ssm_state"], st["conv_state"]
    for t in range(T):
        xt = x[:, t].contiguous()
        xi, z = halves(xt, g, di)
        out = ss.ss_block_q8_step(xt, g, R, h, c)
        y, hr, cr = O.block_core(host(xi)[:, None], host(z)[:, None], w, R, hr, cr)
        check_out(out, xt, y, g, io)
        assert np.array_equal(host(c), cr) and maxrel(host(h), hr) <= MID[io]
    ss.ss_block_q8_fwd(x, g, R, ssm_state=hf, conv_state=cf)
    assert maxrel(host(hf), host(h)) <= 2 * MID[io]


def test_block_streams_graph_and_buffers():
    """A captured step replayed between eager work, a call on another stream, given buffers
    with a workspace of exactly the needed size: the same bits each time, nothing behind."""
    spec = W.BlockSpec("q8graph", 3, 200, 144, expand=2, d_state=16, io_dtype="bf16", seed=970)
    _, g = weights(spec)
    R, di = spec.rank, spec.d_inner
    x = torch.from_numpy(W.gen_block_input(spec)).to(torch.bfloat16).cuda()
    xt = x[:, 0].contiguous()
    h0, c0 = torch.randn(3, di, 16).cuda(), torch.randn(3, di, 3).cuda()

    def fresh():
        return h0.clone(), c0.clone()

    h, c = fresh()
    out = ss.ss_block_q8_fwd(x, g, R, ssm_state=h, conv_state=c)
    dims = ss.block_dims(3, 200, 144, di, 16, R, ss.SS_BF16)
    need = ss.ss_block_q8_workspace_bytes(dims)
    big = torch.full((need + 512,), 77, dtype=torch.uint8).cuda()
    room = torch.full((x.numel() + 64,), 3.0, dtype=torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    h1, c1 = fresh()
    side.wait_stream(torch.cuda.current_stream())
    ss.ss_block_q8_fwd(x, g, R, ssm_state=h1, conv_state=c1, out=room[:x.numel()].view(x.shape), workspace=big[:need], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(room[:x.numel()].view(x.shape), out) and (room[x.numel():] == 3).all() and (big[need:] == 77).all()
    assert torch.equal(h, h1) and torch.equal(c, c1)

    h2, c2 = fresh()
    want = []
    for _ in range(4):
        want.append(ss.ss_block_q8_step(xt, g, R, h2, c2))
    h3, c3 = fresh()
    got = torch.empty_like(xt)
    ss.ss_block_q8_step(xt, g, R, *fresh(), out=got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.ss_block_q8_step(xt, g, R, h3, c3, out=got)
    for k in range(4):
        graph.replay()
        assert torch.equal(got, want[k])
        ss.ss_block_q8_fwd(x, g, R)                                  # eager work in between
        torch.cuda.synchronize()
    assert torch.equal(h2, h3) and torch.equal(c2, c3)


def test_block_binding_refusals():
    spec = W.BlockSpec("q8bad", 2, 3, 32, expand=2, d_state=4, dt_rank=2, io_dtype="bf16", seed=980)
    _, g = weights(spec)
    x = torch.zeros(2, 3, 32, dtype=torch.bfloat16).cuda()
    bad = [dict(W_in=g["W_in"].view(torch.uint8)), dict(S_in=g["S_in"].half()), dict(S_out=g["S_out"][:, :0]),
           dict(W_x=g["W_x"].float()), dict(W_out=g["W_out"].cpu()), dict(norm_w=g["norm_w"][:16])]
    for change in bad:
        with pytest.raises((TypeError, ValueError)):
            ss.ss_block_q8_fwd(x, {**g, **change}, 2)
    for call in (lambda: ss.ss_block_q8_fwd(x[:, 0].contiguous(), g, 2), lambda: ss.ss_block_q8_fwd(x.transpose(0, 1), g, 2),
                 lambda: ss.ss_block_q8_fwd(x, g, 2, out=torch.zeros(2, 3, 32).cuda()),
                 lambda: ss.ss_block_q8_fwd(x, g, 2, workspace=torch.zeros(16, dtype=torch.uint8).cuda()),
                 lambda: ss.ss_block_q8_step(x, g, 2, None, None)):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(ss.SelscanError):
        ss.ss_block_q8_step(x[:, 0].contiguous(), g, 2, None, None)


# ---------------------------------------------------------------------------
# the operators one behind another: a layer with the gated recurrence between 8-bit projections

def glr_rel(L, mem):
    return 2.0 ** -18 + 4 * 2.0 ** -24 * min(L, mem)                 # derived with the recurrence's own tests


def layer(x, res, P, h, reset=None, ckpt=None, step=False):
    """s = x + res; n = RMSNorm(s); x, r, i = n W_in^T; y = recurrence; out = s + y W_out^T."""
    D = P["A"].numel()
    q, s, total = ss.ss_norm_q8(x, P["w"], residual=res)
    p = ss.ss_gemm_q8(q, s, P["W_in"], P["S_in"], out_dtype=torch.float32)
    xi, r, i = p.split(D, dim=-1)                                    # views with a row's stride
    if step:
        y = ss.ss_glr_step(xi, r, i, P["A"], h, reset=reset)
    else:
        y = ss.ss_glr_fwd(xi, r, i, P["A"], state=h, reset=reset, ckpt=ckpt)
    yq, ys = ss.ss_quant_q8(y)
    return ss.ss_gemm_q8(yq, ys, P["W_out"], P["S_out"], residual=total, out_dtype=total.dtype), total, (xi, r, i), y


def params(dm, D, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    P = dict(w=(1 + 0.1 * n(dm)).cuda(), A=-torch.exp(torch.rand(D, generator=gen) * 4 - 4).cuda())
    P["W_in"], P["S_in"] = ss.ss_quant_q8((n(3 * D, dm) / dm ** 0.5).to(torch.bfloat16).cuda(), square=True)
    P["W_out"], P["S_out"] = ss.ss_quant_q8((n(dm, D) / D ** 0.5).to(torch.bfloat16).cuda(), square=True)
    return P, gen


def check_layer(out, total, proj, y, h0, h, P, io, reset):
    xi, r, i = proj
    if xi.dim() == 2:
        xi, r, i, y = (t.unsqueeze(1) for t in (xi, r, i, y))
        reset = None if reset is None else reset.unsqueeze(1)
    want, last, _ = O.glr_fwd(xi, r, i, P["A"], h0, reset)
    top = want.abs().max()
    tol = glr_rel(xi.shape[1], O.memory(r, P["A"], reset)) * top
    y = y.double().cpu()
    assert (y - want).abs().max() <= tol + HALF["f32"] * top and (h.double().cpu() - last).abs().max() <= tol + HALF["f32"] * top
    flat = want.reshape(-1, want.shape[-1])
    ref, off = O.rounded_product(flat, torch.full_like(flat, float(tol + HALF["f32"] * top)), P["W_out"], P["S_out"], HALF[io])
    ref = ref + total.double().cpu().reshape(ref.shape)
    err = (out.double().cpu().reshape(ref.shape) - ref).abs()
    worst = (err / (off + (HALF[io] + 2.0 ** -23) * (ref.abs() + off))).max().item()
    print(f"layer: worst error over bound {worst:.3f}", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,dm,D", [(1, 1, 16, 16), (3, 33, 144, 80), (2, 300, 256, 208), (1, 1100, 64, 128)])
def test_recurrent_layer(B, L, dm, D, io):
    P, gen = params(dm, D, 500 + L)
    x, res = (torch.randn(B, L, dm, generator=gen).to(DT[io]).cuda() for _ in range(2))
    reset = (torch.rand(B, L, generator=gen) < 0.02).cuda()
    h0 = torch.randn(B, D, generator=gen).cuda()
    h = h0.clone()
    out, total, proj, y = layer(x, res, P, h, reset)
    assert torch.equal(total, (x.float() + res.float()).to(DT[io]))
    check_layer(out, total, proj, y, h0, h, P, io, reset)
    # the next token of each stream, and two layers one behind the other in a captured graph
    xt, rt = (torch.randn(B, dm, generator=gen).to(DT[io]).cuda() for _ in range(2))
    h1 = h.clone()
    out, total, proj, y = layer(xt, rt, P, h1, step=True)
    check_layer(out, total, proj, y, h, h1, P, io, None)
    h2 = h.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = layer(xt, rt, P, h2, step=True)
        second = layer(first[0], first[1], P, h2, step=True)
    for _ in range(3):
        h2.copy_(h)
        graph.replay()
        h3 = h.clone()
        a = layer(xt, rt, P, h3, step=True)
        b = layer(a[0], a[1], P, h3, step=True)
        assert torch.equal(first[0], a[0]) and torch.equal(second[0], b[0]) and torch.equal(h2, h3)
        torch.cuda.synchronize()
