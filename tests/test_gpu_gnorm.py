"""GPU: the norms around a layer against their 64-bit definition, and the layer that they stand in.

Tolerances, u = 2^-24. A sum over K columns in fp32, 8 of them in a row and then pairwise, is off by at
most (8 + log2 K) u of the sum of squares, a norm by half that; a sigmoid by 4 u and |z| u of its exponent, |z| <= 6 here;
then products. Forward: rel = 2^-24 (16 + log2 K + 8), relative to the terms of a value. Gradients are differences
of two such products (of what the terms reach), sums over M rows of fp32 terms in up to 64 places each, then in 64 bits: 2^-24
(4 (24 + log2 K) + ceil(M / 256)) of the sum of their sizes. Half a step of the I/O type on top.
"""
import math

import pytest
import torch

from oracle import ops as O

pytestmark = pytest.mark.gpu

ss = pytest.importorskip("selective_state_space_73_amd")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
ALL = ("gate", "residual", "scale", "w_next")


def make(M, K, group, io, what, seed=0):
    r = torch.Generator().manual_seed(70 + seed)
    n = lambda *s: torch.randn(*s, generator=r).cuda()  # noqa: E731
    x = dict(y=n(M, K).to(DT[io]), w=1 + 0.1 * n(group))
    more = dict(gate=n(M, K).clamp(-6, 6).to(DT[io]), residual=(3 * n(M, K)).to(DT[io]), scale=torch.rand(K, generator=r).cuda() + 0.1,
                w_next=1 + 0.1 * n(K))
    x.update({k: v if k in what else None for k, v in more.items()})
    return x, n(M, K).to(DT[io]), n(M, K).to(DT[io]) if "w_next" in what else None


def near(got, want, bound):
    got, want = got.detach().double().cpu(), want.double()
    worst = ((got - want).abs() / (bound + 1e-30)).max().item()
    print(f"worst error over bound {worst:.3f}", flush=True)
    assert torch.isfinite(got).all() and worst <= 1.0


def rel(K):
    return 2.0 ** -24 * (24 + math.log2(K) + 1)


def check(x, ds, dn, io):
    M, K = x["y"].shape
    s, n = ss.ss_gnorm_fwd(**x)
    sw, nw = O.gnorm_fwd(**x)
    res = 0.0 if x["residual"] is None else x["residual"].double().cpu().abs()
    near(s, sw, rel(K) * (sw.abs() + 2 * res) + HALF[io] * sw.abs())
    if nw is None:
        assert n is None
    else:
        near(n, nw, rel(K) * (nw.abs() + 2 * nw.abs() * (res + sw.abs()) / sw.abs().clamp_min(1e-9)) + HALF[io] * nw.abs())
    got = ss.ss_gnorm_bwd(ds=ds, dn=dn, **x)
    want = O.gnorm_bwd(ds=ds, dn=dn, **x)
    for k, v in got.items():
        if v is None:
            assert k not in want
            continue
        print(k, end=" ")
        val, size = want[k]
        sums = k in ("dw", "dscale", "dw_next")
        tol = 2.0 ** -24 * (4 * (24 + math.log2(K) + 1) + (math.ceil(M / 256) if sums else 0))
        # the terms of s and of its norm's gradient are up to twice what is left of them
        near(v, val, 4 * tol * size + (2.0 ** -24 if sums else HALF[io]) * val.abs())


SHAPES = [(1, 1, 1), (3, 7, 7), (2, 8, 8), (5, 128, 128), (33, 130, 130), (17, 512, 512), (9, 513, 513), (40, 2560, 2560), (7, 2561, 2561),
          (5, 640, 128), (6, 60, 12), (4, 1536, 3), (3, 8192, 8192), (2, 8193, 8193), (2, 16384, 16384), (2, 16383, 129)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("what", [ALL, (), ("gate",), ("residual",), ("residual", "scale"), ("gate", "w_next"), ("scale", "w_next")])
def test_against_the_definition(shape, io, what):
    x, ds, dn = make(*shape, io, what, seed=sum(shape))
    check(x, ds, dn, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3000, 96, 96), (1100, 2560, 2560), (700, 300, 100), (520, 1537, 1537), (260, 8000, 8000), (4100, 40, 8)])
def test_many_rows(shape, io):
    x, ds, dn = make(*shape, io, ALL, seed=3)
    check(x, ds, dn, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_one_gradient_is_enough(io):
    x, ds, dn = make(20, 200, 200, io, ALL)
    zero = torch.zeros_like(ds)
    for a, b in ((ds, None), (None, dn)):
        got = ss.ss_gnorm_bwd(ds=a, dn=b, **x)
        want = ss.ss_gnorm_bwd(ds=zero if a is None else a, dn=zero if b is None else b, **x)
        assert all(torch.equal(got[k], want[k]) for k in got)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K", [64, 513, 2560, 2561])
@pytest.mark.parametrize("which", ["y", "gate", "residual"])
def test_in_place(which, K, io):
    x, _, _ = make(50, K, K, io, ALL, seed=K)
    s, n = ss.ss_gnorm_fwd(**x)
    at = x[which]
    s2, n2 = ss.ss_gnorm_fwd(**x, s=at)
    assert s2 is at and torch.equal(s, s2) and torch.equal(n, n2)


def test_leading_dimensions_given_outputs_and_alignment():
    x, ds, dn = make(12, 96, 32, "bf16", ALL)
    s, n = ss.ss_gnorm_fwd(**x)
    three = {k: v.view(3, 4, 96) if v is not None and v.dim() == 2 else v for k, v in x.items()}
    out = torch.empty(3, 4, 96, dtype=torch.bfloat16, device="cuda")
    s3, n3 = ss.ss_gnorm_fwd(**three, n=out)
    assert n3 is out and torch.equal(s3.view(12, 96), s) and torch.equal(n3.view(12, 96), n)
    # rows that start anywhere
    big = torch.zeros(12 * 96 + 1, dtype=torch.bfloat16, device="cuda")
    big[1:] = x["y"].reshape(-1)
    odd = {**x, "y": big[1:].view(12, 96)}
    near(ss.ss_gnorm_fwd(**odd)[0], s.double().cpu(), 2 * HALF["bf16"] * s.double().cpu().abs() + 1e-5)
    g, g2 = ss.ss_gnorm_bwd(ds=ds, dn=dn, **x), ss.ss_gnorm_bwd(ds=ds, dn=dn, **odd)
    near(g2["dw"], g["dw"].double().cpu(), 1e-5 * g["dw"].double().cpu().abs().max())
    # nothing around the outputs is touched
    buf = torch.full((12 * 96 + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    ss.ss_gnorm_fwd(**x, s=buf[32:32 + 12 * 96].view(12, 96))
    assert (buf[:32] == 3).all() and (buf[32 + 12 * 96:] == 3).all()


def test_rows_of_zeros_and_bad_rows_stay_to_themselves():
    x, ds, dn = make(9, 300, 300, "f32", ALL)
    s, n = ss.ss_gnorm_fwd(**x)
    for k in ("y", "gate", "residual"):
        x[k][4] = 0
    x["y"][6] = float("nan")
    x["residual"][7, 3] = float("inf")
    s2, n2 = ss.ss_gnorm_fwd(**x)
    keep = [0, 1, 2, 3, 5, 8]
    assert torch.equal(s2[keep], s[keep]) and torch.equal(n2[keep], n[keep])
    assert (s2[4] == 0).all() and (n2[4] == 0).all() and torch.isnan(n2[6]).all() and torch.isinf(s2[7, 3])
    g = ss.ss_gnorm_bwd(ds=ds, dn=dn, **x)
    assert torch.isfinite(g["dy"][keep]).all() and torch.isfinite(g["dresidual"][4]).all()


def test_gates_far_out():
    x, _, _ = make(4, 64, 64, "f32", ("gate",))
    x["gate"][0], x["gate"][1], x["gate"][2] = 100.0, -100.0, 30.0
    s, _ = ss.ss_gnorm_fwd(**x)
    sw, _ = O.gnorm_fwd(**x)
    # |z| u of the exponent
    near(s, sw, (rel(64) + 200 * 2.0 ** -24) * sw.abs() + 1e-37)
    assert torch.isfinite(ss.ss_gnorm_bwd(ds=torch.ones_like(s), **x)["dgate"]).all()


def test_graph_replays_and_streams():
    x, ds, dn = make(700, 640, 128, "bf16", ALL)

    def step():
        return [*ss.ss_gnorm_fwd(**x), *ss.ss_gnorm_bwd(ds=ds, dn=dn, **x).values()]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        x["y"].copy_(torch.randn_like(x["y"]))
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ss.ss_gnorm_bwd(ds=ds, dn=dn, **x, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got.values(), eager[2:]))


def test_binding_refusals():
    x, ds, dn = make(4, 96, 32, "f32", ALL)
    for k, v in (("gate", x["gate"].bfloat16()), ("w", x["w"].double()), ("scale", x["scale"].bfloat16())):
        with pytest.raises(TypeError):
            ss.ss_gnorm_fwd(**{**x, k: v})
    for k, v in (("gate", x["gate"][:2]), ("scale", x["scale"][:5]), ("w_next", x["w"]), ("y", x["y"].t()), ("w", x["w"].view(1, 32))):
        with pytest.raises(ValueError):
            ss.ss_gnorm_fwd(**{**x, k: v})
    with pytest.raises(ss.SelscanError):
        ss.ss_gnorm_fwd(**{**x, "w": torch.ones(7, device="cuda")})
    with pytest.raises(ss.SelscanError):
        ss.ss_gnorm_fwd(**x, eps=0.0)
    with pytest.raises(ValueError):
        ss.ss_gnorm_fwd(**{**x, "w_next": None}, n=ds)
    with pytest.raises(ss.SelscanError):
        ss.ss_gnorm_bwd(ds=None, **x)
    with pytest.raises(ss.SelscanError):
        ss.ss_gnorm_fwd(**x, s=x["y"].view(-1)[:0].new_empty(4, 96), n=x["y"])


def layer(x, P, S, io, Hk, H, K, V):
    """A delta-rule layer as a program runs it: projections, the rule, its heads' norm and gate, the projection back,
    the residual and the next norm."""
    B, L, D = x.shape
    p = x @ P["in"]
    q, k, v, z = p.split([Hk * K, Hk * K, H * V, H * V], dim=-1)
    q, k, v = q.view(B, L, Hk, K), k.view(B, L, Hk, K), v.view(B, L, H, V)
    g = -torch.nn.functional.softplus((x @ P["a"]).float())
    beta = torch.sigmoid((x @ P["b"]).float())
    return p, q, k, v, z.contiguous(), g, beta


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_the_operators_together(io):
    """Forward, one decode step and gradients of a whole layer: each operator's result is checked against its definition on
    the inputs that it had, so that roundings between them do not add up."""
    B, L, D, Hk, H, K, V = 2, 90, 96, 2, 4, 32, 24
    r = torch.Generator().manual_seed(4)
    n = lambda *s: (torch.randn(*s, generator=r) * s[0] ** -0.5).to(DT[io]).cuda()  # noqa: E731
    P = dict(a=n(D, H), b=n(D, H), out=n(H * V, D))
    P["in"] = n(D, 2 * Hk * K + 2 * H * V)
    x = torch.randn(B, L, D, generator=r).to(DT[io]).cuda()
    wh, wp, wn, al = torch.ones(V).cuda(), 1 + 0.1 * torch.randn(D, generator=r).cuda(), 1 + 0.1 * torch.randn(D, generator=r).cuda(), torch.rand(D, generator=r).cuda()
    S = torch.randn(B, H, K, V, generator=r).cuda()
    S0 = S.clone()
    p, q, k, v, z, g, beta = layer(x, P, S, io, Hk, H, K, V)
    ck = torch.empty(ss.gdr_ckpt_shape(B, L, H, K, V), device="cuda")
    y = ss.ss_gdr_fwd(q, k, v, g, beta, state=S, ckpt=ck)
    o, _ = ss.ss_gnorm_fwd(y.view(B, L, H * V), wh, gate=z)
    f = o @ P["out"]
    s, m = ss.ss_gnorm_fwd(f, wp, residual=x, scale=al, w_next=wn)
    yw, Sw = O.gdr_fwd(q, k, v, g, beta, S0)
    tol = 5 * (2 * (K + 192) * 3) ** 0.5 * 2.0 ** -24                     # as for the rule alone
    near(y, yw, tol * yw.abs().max() + HALF[io] * yw.abs())
    near(S, Sw, torch.full_like(Sw, float(tol * max(Sw.abs().max(), S0.abs().max().cpu()))))
    ow, _ = O.gnorm_fwd(y.view(B, L, H * V), wh, gate=z)
    near(o, ow, (rel(V) + 8 * 2.0 ** -24 + HALF[io]) * ow.abs() + 1e-12)
    sw, mw = O.gnorm_fwd(f, wp, None, x, al, wn)
    near(s, sw, rel(D) * (sw.abs() + 2 * x.double().cpu().abs()) + HALF[io] * sw.abs())
    # gradients from the last norm back to the gates
    dm = torch.randn(B, L, D, generator=r).to(DT[io]).cuda()
    back = ss.ss_gnorm_bwd(f, wp, None, dn=dm, residual=x, scale=al, w_next=wn)
    do = back["dy"] @ P["out"].t().contiguous()
    heads = ss.ss_gnorm_bwd(y.view(B, L, H * V), wh, do, gate=z)
    dy = heads["dy"].view(B, L, H, V)
    got = ss.ss_gdr_bwd(q, k, v, g, beta, ck, dy)
    want = O.gdr_bwd(q, k, v, g, beta, dy, S0)
    for name in got:
        near(got[name], want[name], 2 * 5 * (2 * (K + 192 + V) * 3) ** 0.5 * 2.0 ** -24 * want[name].abs().max()
             + (HALF[io] if name in ("dq", "dk", "dv") else 2.0 ** -24) * want[name].abs())
    # one more token of each stream
    x1 = torch.randn(B, 1, D, generator=r).to(DT[io]).cuda()
    _, q, k, v, z, g, beta = layer(x1, P, S, io, Hk, H, K, V)
    Sb = S.clone()
    y1 = ss.ss_gdr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], S)
    yw, Sw = O.gdr_fwd(q, k, v, g, beta, Sb)
    near(y1, yw[:, 0], tol * yw.abs().max() + HALF[io] * yw[:, 0].abs())
    near(S, Sw, torch.full_like(Sw, float(tol * max(Sw.abs().max(), Sb.abs().max().cpu()))))
    o1, _ = ss.ss_gnorm_fwd(y1.view(B, H * V), wh, gate=z[:, 0].contiguous())
    assert o1.shape == (B, H * V) and torch.isfinite(o1).all()
