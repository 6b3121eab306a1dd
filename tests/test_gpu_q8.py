"""GPU: rounding to 8 bits, the norm in front of it and the 8-bit product against their 64-bit
definitions.

Tolerances. A scale is a maximum (exact) over 448, one rounding: 2^-24 of it. q = e4m3(v / s)
with v / s taken as v (1 / s), off by at most 2^-23 of itself (two roundings): the value it
stands for lies within half a step of v, plus 2^-23 |v|. The norm sums K squares, at most 80
on a lane one after the other per 4096 columns and a tree of 6 or 8 above them, halved by the
root, then three products: n is off by at most (K / 4096 + 1) 64 2^-24 of itself, under 2^-15
up to K = 20000. A product's K terms are summed in fp32 in blocks of 128 and then block by
block: under 2 (128 + K / 128) roundings of 2^-24, of the sum of the terms' sizes. With a bf16
output the matrix cores drop, of eight neighbouring terms, what lies below 2^-13 of the
largest: at most 7 2^-13 of it, under 2^-10 of the terms' sizes.
"""
import pytest
import torch

from oracle import ops as O

pytestmark = pytest.mark.gpu

ss = pytest.importorskip("selective_state_space_73_amd")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
F8 = torch.float8_e4m3fn


def rand(*shape, io="f32", seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[io]).cuda()


def check_q(v, q, scale, square=False, rel=2.0 ** -23, top_rel=2.0 ** -24):
    """q and scale against the 64-bit values v they were made from (known to a relative rel)."""
    v = v.cpu().double()
    M, K = v.shape
    want = (O.block_tops(v, square) / O.Q8_MAX).clamp_min(O.Q8_TINY)
    s = scale.cpu().double()
    assert s.shape == want.shape and ((s - want).abs() <= (top_rel + 2.0 ** -30) * want).all()
    assert q.dtype == F8 and q.shape == v.shape
    per = O.spread(scale, M, K, square)
    err = (O.values(q, scale, square) - v).abs()
    bound = O.half_step(v, per) + rel * v.abs()
    print(f"worst error over bound {(err / bound.clamp_min(1e-300)).max():.4f}", flush=True)
    assert (err <= bound).all()


SIZES = [(1, 1), (1, 8), (3, 127), (2, 128), (5, 129), (64, 136), (130, 512), (1030, 520), (1025, 2560), (7, 2048),
         (33, 4104), (1024, 4096), (2, 8200), (3, 20001)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_quant_rows(M, K, io):
    x = rand(M, K, io=io, seed=M + K)
    check_q(x, *ss.ss_quant_q8(x))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (127, 8), (128, 128), (129, 136), (300, 1000), (513, 77)])
def test_quant_squares(M, K, io):
    x = rand(M, K, io=io, seed=M + K, scale=0.02)
    check_q(x, *ss.ss_quant_q8(x, square=True), square=True)


@pytest.mark.parametrize("square", [False, True])
def test_quant_values_that_round_in_known_ways(square):
    """Every e4m3 value, the midpoints between neighbours (ties to even), zeros of both signs,
    the smallest scale, values below the smallest step."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(F8).float()       # 0 .. 448
    x = torch.zeros(3, 384)
    x[0, :127] = codes
    x[0, 128:254] = (codes[:-1] + codes[1:]) / 2
    x[0, 255] = 448.0
    x[0, 256:383] = -codes
    if not square:
        x[1] = x[0] * 2.0 ** -130                                           # the scale stays 2^-126
        x[2, 5] = -0.0
    q, s = ss.ss_quant_q8(x.cuda(), square=square)
    qf = q.float().cpu()
    assert torch.equal(qf[0, :127], codes) and torch.equal(qf[0, 256:383], -codes)
    even = torch.where((torch.arange(126) % 2 == 0), codes[:-1], codes[1:])
    assert torch.equal(qf[0, 128:254], even)
    assert (s[0].cpu() == 1.0).all()
    if not square:
        assert (s[1:].cpu() == 2.0 ** -126).all() and (qf[2] == 0).all()
        assert torch.equal(qf[1], (x[0] / 16).to(F8).float())


def test_quant_non_finite():
    x = rand(3, 256)
    x[0, 3] = float("nan")
    x[1, 130] = float("inf")
    x[2] = float("nan")
    q, s = ss.ss_quant_q8(x)
    qf = q.float().cpu()
    assert torch.isnan(qf[0, 3]) and torch.isfinite(qf[0, :3]).all() and torch.isfinite(qf[0, 4:]).all()
    clean = x[:1].clone()
    clean[0, 3] = 0
    assert torch.equal(s[0], ss.ss_quant_q8(clean)[1][0])
    assert torch.isinf(s[1, 1]) and torch.isnan(O.values(q, s)[1, 128:]).all() and torch.isfinite(qf[1, :128]).all()
    assert torch.isnan(qf[2]).all() and (s[2].cpu() == 2.0 ** -126).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm(M, K, io, res):
    x, w = rand(M, K, io=io, seed=M + K), 1 + rand(K, seed=1, scale=0.1)
    r = rand(M, K, io=io, seed=5, scale=3.0) if res else None
    q, scale, s = ss.ss_norm_q8(x, w, residual=r)
    n, sw = O.rms_norm(x, w, r)
    tol = (K / 4096 + 1) * 64 * 2.0 ** -24
    if res:
        assert s.dtype == x.dtype and ((s.cpu().double() - sw).abs() <= (HALF[io] + 2.0 ** -24) * sw.abs()).all()
    else:
        assert s is None
    check_q(n, q, scale, rel=tol + 2.0 ** -23, top_rel=tol + 2.0 ** -24)


@pytest.mark.parametrize("K", [520, 8200])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_in_place(which, K):
    x, r, w = rand(70, K, io="bf16"), rand(70, K, io="bf16", seed=1), rand(K, seed=2)
    q, scale, s = ss.ss_norm_q8(x, w, residual=r)
    a, b = x.clone(), r.clone()
    got = ss.ss_norm_q8(a, w, residual=b, sum_out=a if which == "x" else b)
    assert got[2] is (a if which == "x" else b)
    assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1], scale) and torch.equal(got[2], s)


def test_norm_zero_row_and_eps():
    x = torch.zeros(4, 300, device="cuda")
    x[1, 7] = 1e-3
    q, scale, _ = ss.ss_norm_q8(x, torch.ones(300, device="cuda"), eps=1.0)
    assert (q.float()[0] == 0).all() and (scale[0].cpu() == 2.0 ** -126).all()
    v = O.values(q, scale)[1, 7]
    assert abs(v - 1e-3) <= 1e-3 * 2.0 ** -4
    n = ss.ss_norm_q8(x, torch.ones(300, device="cuda"), eps=1e-12)
    assert abs(O.values(n[0], n[1])[1, 7] - 300 ** 0.5) <= 300 ** 0.5 * (2.0 ** -4 + 2.0 ** -10)


def test_leading_dimensions_and_alignment():
    x = rand(2, 3, 160, io="bf16")
    q, s = ss.ss_quant_q8(x)
    q2, s2 = ss.ss_quant_q8(x.view(6, 160))
    assert q.shape == (2, 3, 160) and s.shape == (2, 3, 2)
    assert torch.equal(q.view(torch.uint8).view(6, 160), q2.view(torch.uint8)) and torch.equal(s.view(6, 2), s2)
    flat = torch.empty(6 * 160 + 1, dtype=torch.bfloat16, device="cuda")     # rows that start on 2 bytes
    odd = flat[1:].view(6, 160)
    odd.copy_(x.view(6, 160))
    q3, s3 = ss.ss_quant_q8(odd)
    assert torch.equal(q3.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s3, s2)
    w = rand(160, seed=3)
    a, b = ss.ss_norm_q8(odd, w, residual=odd), ss.ss_norm_q8(x.view(6, 160), w, residual=x.view(6, 160))
    assert all(torch.equal(p.view(torch.uint8), o.view(torch.uint8)) for p, o in zip(a, b))


def test_buffers_keep_their_ends():
    x = rand(5, 100)
    q = torch.full((700,), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((20,), 7.0, device="cuda")
    ss.ss_quant_q8(x, q=q[100:600].view(5, 100).view(F8), scale=s[5:10].view(5, 1))
    assert (q[:100] == 7).all() and (q[600:] == 7).all() and (s[:5] == 7).all() and (s[10:] == 7).all()


# ---------------------------------------------------------------------------
# the product

def operands(M, N, K, seed=0):
    xq, xs = ss.ss_quant_q8(rand(M, K, seed=seed))
    wq, ws = ss.ss_quant_q8(rand(N, K, seed=seed + 1, scale=K ** -0.5), square=True)
    return xq, xs, wq, ws


def check_y(y, xq, xs, wq, ws, residual=None, io="bf16"):
    x, w = O.values(xq, xs), O.values(wq, ws, True)
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    K = x.shape[1]
    if residual is not None:
        want, size = want + residual.cpu().double(), size + residual.cpu().double().abs()
    drop = 2.0 ** -10 if io == "bf16" else 0.0
    bound = (drop + 2 * (128 + K / 128) * 2.0 ** -24) * size + HALF[io] * want.abs() * 1.001 + 1e-30
    err = (y.cpu().double() - want).abs()
    print(f"worst error over bound {(err / bound).max():.4f}", flush=True)
    assert (err <= bound).all()


GEMMS = [(1, 1, 16), (1, 33, 128), (2, 129, 144), (15, 64, 112), (16, 200, 2560), (17, 31, 272), (32, 257, 1040),
         (33, 130, 512), (64, 1024, 2560), (65, 36, 640), (201, 261, 1280), (256, 128, 128), (257, 127, 656), (300, 513, 1296),
         (1000, 130, 16), (513, 1025, 384), (1111, 3000, 400)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_product(M, N, K, io):
    ops = operands(M, N, K, seed=M)
    check_y(ss.ss_gemm_q8(*ops, out_dtype=DT[io]), *ops, io=io)
    r = rand(M, N, io=io, seed=9)
    y = ss.ss_gemm_q8(*ops, residual=r, out_dtype=DT[io])
    check_y(y, *ops, residual=r, io=io)
    assert ss.ss_gemm_q8(*ops, residual=r, out=r) is r and torch.equal(r, y)      # in place


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(40, 16500, 272), (64, 16448, 144), (16, 16390, 400), (7, 8200, 1040), (31, 8195, 656), (96, 2570, 528),
                                   (180, 9000, 208), (150, 6001, 16), (2100, 7001, 144), (1300, 2049, 2064)])
def test_product_of_sizes_at_which_tiles_change(M, N, K, io):
    test_product(M, N, K, io)


def test_product_picks_every_element():
    """One value in X and one in W: the output is their product at one place, zero elsewhere,
    for places all over the tiles."""
    M, N, K = 300, 300, 400
    for m, n, k in [(0, 0, 0), (299, 299, 399), (17, 130, 127), (128, 127, 128), (255, 256, 271), (100, 5, 383)]:
        x, w = torch.zeros(M, K, device="cuda"), torch.zeros(N, K, device="cuda")
        x[m, k], w[n, k] = 3.0, -0.5
        for rows in (M, 40):
            xq, xs = ss.ss_quant_q8(x[m // rows * rows:m // rows * rows + rows].contiguous())
            y = ss.ss_gemm_q8(xq, xs, *ss.ss_quant_q8(w, square=True), out_dtype=torch.float32)
            want = torch.zeros_like(y)
            want[m % rows, n] = -1.5
            assert torch.allclose(y, want, rtol=1e-6, atol=0)


def test_product_non_finite_stays_in_its_row():
    xq, xs, wq, ws = operands(70, 140, 256)
    xb = xq.view(torch.uint8).clone()
    xb[3, 7] = 0x7F                                                              # NaN
    y = ss.ss_gemm_q8(xb.view(F8), xs, wq, ws, out_dtype=torch.float32)
    clean = ss.ss_gemm_q8(xq, xs, wq, ws, out_dtype=torch.float32)
    assert torch.isnan(y[3]).all()
    keep = torch.arange(70, device="cuda") != 3
    assert torch.equal(y[keep], clean[keep])


def test_product_rows_do_not_depend_on_their_neighbours():
    """A row's result is the same in a batch of one kernel's size, whatever the other rows hold."""
    xq, xs, wq, ws = operands(300, 260, 640)
    y = ss.ss_gemm_q8(xq, xs, wq, ws)
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(0)).cuda()
    y2 = ss.ss_gemm_q8(xq.view(torch.uint8)[perm].view(F8), xs[perm], wq, ws)
    assert torch.equal(y2, y[perm])


def test_product_streams_graph_and_ends():
    xq, xs, wq, ws = operands(48, 200, 512)
    want = ss.ss_gemm_q8(xq, xs, wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ss.ss_gemm_q8(xq, xs, wq, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    buf = torch.full((48 * 200 + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    ss.ss_gemm_q8(xq, xs, wq, ws, out=buf[32:32 + 48 * 200].view(48, 200))
    assert (buf[:32] == 3).all() and (buf[32 + 48 * 200:] == 3).all()
    x, w = rand(48, 512, io="bf16"), rand(512, seed=4)

    def chain(s):
        q, sc, t = ss.ss_norm_q8(x, w, residual=s)
        y = ss.ss_gemm_q8(q, sc, wq, ws)
        return [y, t, *ss.ss_quant_q8(y)]

    s = rand(48, 512, io="bf16", seed=8)
    chain(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(s)
    for n in range(3):
        x.copy_(rand(48, 512, io="bf16", seed=20 + n))
        eager = chain(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, eager))


# ---------------------------------------------------------------------------
# sizes past 32 bits

def test_rounding_more_rows_than_one_launch_takes():
    M, K = (1 << 22) + 9, 16
    x = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    q, s = ss.ss_quant_q8(x)
    w = rand(K, seed=4)
    nq, ns, t = ss.ss_norm_q8(x, w, residual=x)
    for rows in (slice(0, 40), slice((1 << 22) - 20, M)):
        check_q(x[rows], q[rows], s[rows])
        n, total = O.rms_norm(x[rows], w, x[rows])
        check_q(n, nq[rows], ns[rows], rel=2.0 ** -15 + 2.0 ** -23, top_rel=2.0 ** -15)
        assert torch.equal(t[rows].cpu().double(), total)


def test_product_with_offsets_past_32_bits():
    M, N, K = (1 << 20) + 5, 2064, 16                                   # y: 4.3 GB
    xq, xs, wq, ws = operands(M, N, K, seed=11)
    y = ss.ss_gemm_q8(xq, xs, wq, ws)
    for rows in (slice(0, 70), slice(M - 70, M)):
        check_y(y[rows], xq[rows], xs[rows], wq, ws)
    del y
    M, N, K = 1030, 16, 1 << 22                                         # xq: 4.3 GB
    g = torch.Generator("cuda").manual_seed(12)
    xq = torch.randint(0, 0x78, (M, K), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    wq = torch.randint(0, 0x78, (N, K), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    xs, ws = torch.rand(M, K // 128, device="cuda", generator=g), torch.rand(1, K // 128, device="cuda", generator=g)
    y = ss.ss_gemm_q8(xq, xs, wq, ws, out_dtype=torch.float32)
    check_y(y[-3:], xq[-3:], xs[-3:], wq, ws, io="f32")


def test_empty_tensors_are_refused():
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    q8 = lambda *s: e(*s).to(F8)  # noqa: E731
    for call in (lambda: ss.ss_quant_q8(e(0, 128)), lambda: ss.ss_quant_q8(e(4, 0)), lambda: ss.ss_quant_q8(e(0, 128), square=True),
                 lambda: ss.ss_norm_q8(e(0, 64), e(64)), lambda: ss.ss_gemm_q8(q8(0, 128), e(0, 1), q8(8, 128), e(1, 1)),
                 lambda: ss.ss_gemm_q8(q8(8, 128), e(8, 1), q8(0, 128), e(0, 1)), lambda: ss.ss_gemm_q8(q8(4, 0), e(4, 0), q8(4, 0), e(1, 0)),
                 lambda: ss.ss_glr_fwd(*[e(0, 4, 8)] * 3, e(8)), lambda: ss.ss_glr_fwd(*[e(2, 0, 8)] * 3, e(8)),
                 lambda: ss.ss_glr_fwd(*[e(2, 4, 0)] * 3, e(0)), lambda: ss.ss_glr_step(*[e(0, 8)] * 3, e(8), e(0, 8)),
                 lambda: ss.ss_glr_bwd(*[e(2, 0, 8)] * 3, e(8), e(2, 0, 8), e(2, 0, 8))):
        with pytest.raises((ValueError, ss.SelscanError)):
            call()


def test_calls_in_inference_mode_and_with_gradients_recorded():
    x = rand(40, 256, io="bf16", seed=1)
    q, s = ss.ss_quant_q8(x)
    with torch.inference_mode():
        q1, s1 = ss.ss_quant_q8(x.clone())
    q2, s2 = ss.ss_quant_q8(x.clone().requires_grad_())
    for a, b in ((q1, s1), (q2, s2)):
        assert torch.equal(a.view(torch.uint8), q.view(torch.uint8)) and torch.equal(b, s) and not b.requires_grad
