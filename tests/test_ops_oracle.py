"""CPU: the 64-bit definitions the operators are compared with, against differences and
automatic differentiation."""
import pytest
import torch

from oracle import ops as O

F64 = torch.float64


def _inputs(B, L, D, seed, resets):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    x, r, i, dy = (n(B, L, D) for _ in range(4))
    A = -(torch.rand(D, generator=g, dtype=F64) * 2 + 0.05)
    reset = (torch.rand(B, L, generator=g) < 0.2).to(torch.uint8) if resets else None
    return x, r, i, A, n(B, D), reset, dy, n(B, D)


@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("L", [1, 2, 7, 70])
def test_recurrence_gradients_match_autograd(L, resets):
    x, r, i, A, h0, reset, dy, dh = _inputs(2, L, 3, L, resets)
    leaves = [t.clone().requires_grad_(True) for t in (x, r, i, A, h0)]
    y, h, _ = O.glr_fwd(*leaves[:4], state=leaves[4], reset=reset)
    ((dy * y).sum() + (dh * h).sum()).backward()
    got = O.glr_bwd(x, r, i, A, dy, h0, reset, dh)
    for name, leaf in zip(("dx", "dr", "di", "dA", "dstate_init"), leaves):
        val, scale = got[name]
        # 64 bits: a few hundred roundings of 2^-53, relative to the size of the terms
        assert ((val - leaf.grad).abs() <= 1e-12 * (scale + val.abs() + 1e-3)).all(), name


def test_recurrence_gradients_match_differences():
    x, r, i, A, h0, reset, dy, dh = _inputs(1, 9, 2, 3, True)
    got = O.glr_bwd(x, r, i, A, dy, h0, reset, dh)

    def loss(x, r, i, A, h0):
        y, h, _ = O.glr_fwd(x, r, i, A, h0, reset)
        return float((dy * y).sum() + (dh * h).sum())

    args = [x, r, i, A, h0]
    eps = 1e-5          # central differences: error eps^2 times third derivatives of order 10, rounding 1e-15 / eps
    for name, k in (("dx", 0), ("dr", 1), ("di", 2), ("dA", 3), ("dstate_init", 4)):
        flat = got[name][0].reshape(-1)
        for j in range(flat.numel()):
            up, dn = [t.clone() for t in args], [t.clone() for t in args]
            up[k].reshape(-1)[j] += eps
            dn[k].reshape(-1)[j] -= eps
            num = (loss(*up) - loss(*dn)) / (2 * eps)
            assert abs(num - float(flat[j])) <= 1e-7, (name, j)


def test_recurrence_pieces_and_resets():
    x, r, i, A, h0, _, _, _ = _inputs(1, 130, 4, 5, False)
    y, h, ck = O.glr_fwd(x, r, i, A, h0)
    y1, h1, _ = O.glr_fwd(x[:, :50], r[:, :50], i[:, :50], A, h0)
    y2, h2, _ = O.glr_fwd(x[:, 50:], r[:, 50:], i[:, 50:], A, h1)
    assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(h2, h)
    assert torch.equal(ck[:, 0], h0) and torch.equal(ck[:, 1], y[:, 63]) and torch.equal(ck[:, 2], y[:, 127])
    # a reset is a new sequence from the zero state, whatever came before
    reset = torch.zeros(1, 130, dtype=torch.uint8)
    reset[0, 50] = 1
    bad = x.clone()
    bad[0, 20] = float("nan")
    yr, _, _ = O.glr_fwd(bad, r, i, A, h0, reset)
    s, g = torch.sigmoid(r[:, 50]), torch.sigmoid(i[:, 50])
    assert torch.allclose(yr[:, 50], g * x[:, 50], rtol=1e-14)
    ys, _, _ = O.glr_fwd(x[:, 51:], r[:, 51:], i[:, 51:], A, yr[:, 50])
    assert torch.equal(ys, yr[:, 51:])
    # repeated products stay what the closed form says: constant gates decay geometrically
    c = torch.zeros(1, 6, 1, dtype=F64)
    yc, _, _ = O.glr_fwd(c, c, c, torch.tensor([-0.5], dtype=F64), torch.ones(1, 1, dtype=F64))
    want = torch.exp(-0.25 * torch.arange(1, 7, dtype=F64))
    assert torch.allclose(yc[0, :, 0], want, rtol=1e-14)


# ---------------------------------------------------------------------------
# the block in pieces

@pytest.mark.parametrize("states", [False, True])
def test_block_core_is_the_block_between_its_projections(states):
    import workloads as W
    from oracle import block as ob
    spec = W.BlockSpec("core", 2, 9, 32, d_state=8, dt_rank=3, io_dtype="f32", seed=5)
    w, x, di = W.gen_block_weights(spec), W.gen_block_input(spec), spec.d_inner
    st = W.gen_states(2, di, 8, seed=3)
    st = (st["ssm_state"], st["conv_state"]) if states else (None, None)
    p = ob.rms_norm(x, w["norm_w"]) @ w["W_in"].T.astype("float64")
    y, h, c = O.block_core(p[..., :di], p[..., di:], w, 3, *st)
    out, hr, cr = ob.block_forward(x, w, 3, *st)
    assert abs(x + y @ w["W_out"].T.astype("float64") - out).max() < 1e-12
    assert abs(h - hr).max() < 1e-12 and abs(c - cr).max() < 1e-12


def test_rounded_product_bound_holds_and_is_tight():
    """The bound covers torch's rounding of a disturbed y, and with an identity it is no more
    than a tenth above what values at midpoints reach."""
    g = torch.Generator().manual_seed(4)
    y = torch.randn(6, 256, generator=g).double()
    slack = 1e-5 * torch.ones_like(y)
    for w in (torch.eye(256), torch.randn(40, 256, generator=g)):
        top = (O.block_tops(w, True) / O.Q8_MAX).clamp_min(O.Q8_TINY)
        wq = (w.double() / O.spread(top, *w.shape, square=True)).float().to(torch.float8_e4m3fn)
        want, off = O.rounded_product(y, slack, wq, top, 2.0 ** -24)
        z = y + slack * (2 * torch.rand(y.shape, generator=g).double() - 1)
        s = (O.block_tops(z) / O.Q8_MAX).clamp_min(O.Q8_TINY)
        zq = (z / O.spread(s, *z.shape)).float().to(torch.float8_e4m3fn)
        err = (O.values(zq, s) @ O.values(wq, top, square=True).T - want).abs()
        assert (err <= off).all()
        if w.shape[0] == 256:
            assert (err / off).max() > 0.9
