"""GPU: the gated linear recurrence's gates far out: decays that are small, gates that are nearly
shut or open, write coefficients that underflow.

Tolerances, relative to each element. With u = 2^-24: exp2 of an argument c carries |c| u ln 2 by
the argument's rounding; so for gates of |r| <= q a sigmoid and its complement are off by at most
2 (q + 4) u (argument, exp2, addition, reciprocal, product). A decay exp(A s) is off by
|A s| (4 + the sigmoid's) u. A gradient here is a product of one decay or write coefficient, both
sigmoids, one complement and inputs, 12 roundings, with no sums that cancel. For |A s| <= 20 and
q <= 20 that is under (20 * 56 + 4 * 48 + 12) u < 2^-13.
"""
import pytest
import torch

import test_gpu_glr as ordinary
from oracle import ops as O

pytestmark = pytest.mark.gpu

ss = pytest.importorskip("selective_state_space_73_amd")
REL = 2.0 ** -13


def close(got, want, rel=REL, floor=1e-36):
    got, want = got.detach().double().cpu(), want.double().cpu()
    worst = ((got - want).abs() / (rel * want.abs() + floor)).max().item()
    print(f"worst error over bound {worst:.3g}", flush=True)
    assert torch.isfinite(got).all() and worst <= 1.0


def both(x, r, i, A, h0, dy, dh, reset=None):
    x, r, i, dy = (t.cuda() for t in (x, r, i, dy))
    B, L, D = x.shape
    ck = torch.empty(ss.glr_ckpt_shape(B, L, D), device="cuda")
    h = h0.cuda().clone()
    y = ss.ss_glr_fwd(x, r, i, A.cuda(), state=h, reset=reset, ckpt=ck)
    return y, h, ss.ss_glr_bwd(x, r, i, A.cuda(), ck, dy, reset=reset, dstate_final=dh.cuda())


@pytest.mark.parametrize("L", [1, 2, 5])
@pytest.mark.parametrize("D", [64, 33])
def test_small_decays(L, D):
    """exp(A s) between e^-20 and e^-8, nothing written: a state of a^L, gradients with a factor a."""
    g = torch.Generator().manual_seed(L)
    x = torch.zeros(1, L, D)
    r, i = torch.randn(1, L, D, generator=g), torch.randn(1, L, D, generator=g)
    A = -torch.linspace(8, 20, D) / torch.sigmoid(r[0].max(0).values)
    if L > 2:
        A = A / 3                                                       # a^L stays far from the smallest number
    h0, dh = 1 + torch.rand(1, D, generator=g), 1 + torch.rand(1, D, generator=g)
    dy = torch.zeros(1, L, D)
    y, h, got = both(x, r, i, A, h0, dy, dh)
    yw, hw, _ = O.glr_fwd(x, r, i, A, h0)
    close(y, yw)
    close(h, hw)
    want = O.glr_bwd(x, r, i, A, dy, h0, None, dh)
    for k in ("dr", "dA", "dstate_init"):
        print(k, end=" ")
        close(got[k], want[k][0])
    hs = h0.cuda().clone()
    ys = ss.ss_glr_step(x[:, 0].cuda(), r[:, 0].cuda(), i[:, 0].cuda(), A.cuda(), hs)
    close(ys, yw[:, 0])
    assert torch.equal(ys, hs)


@pytest.mark.parametrize("L", [1, 40])
def test_decays_from_long_memories_to_none(L):
    """exp(A s) from 1 - 2^-20 to e^-20, element by element, over the place where its evaluation changes."""
    D = 2048
    la = -torch.logspace(-6, 1.3, D)
    r = torch.zeros(1, L, D)
    A = 2 * la / L
    x, i = torch.zeros(1, L, D), torch.zeros(1, L, D)
    h0 = torch.ones(1, D)
    y, _, got = both(x, r, i, A, h0, torch.zeros(1, L, D), torch.ones(1, D))
    close(y, O.glr_fwd(x, r, i, A, h0)[0])
    close(got["dstate_init"], O.glr_bwd(x, r, i, A, torch.zeros(1, L, D), h0, None, torch.ones(1, D))["dstate_init"][0])


@pytest.mark.parametrize("L", [3, 130])
def test_write_coefficients_that_underflow(L):
    """1 - a^2 below the smallest normal number: a token that leaves the state as it is, with finite
    gradients, which the other tokens' are not touched by."""
    r = torch.zeros(1, L, 8)
    r[0, 1] = torch.tensor([-83.0, -84.0, -85.0, -86.0, -87.0, -87.3, -87.5, -88.0])
    for a in (-0.1, -0.05, -0.01, -1e-4):
        g = torch.Generator().manual_seed(L)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        x, i, h0, dy, dh = n(1, L, 8), n(1, L, 8), n(1, 8), n(1, L, 8), n(1, 8)
        A = torch.full((8,), a)
        y, h, got = both(x, r, i, A, h0, dy, dh)
        assert torch.isfinite(y).all() and torch.isfinite(h).all()
        want = O.glr_bwd(x, r, i, A, dy, h0, None, dh)
        for k, (val, scale) in want.items():
            print(k, end=" ")
            assert torch.isfinite(got[k]).all()
            # its terms' sizes, as for ordinary gates; what the token itself adds is under 2^-60 of them
            err = (got[k].double().cpu() - val).abs()
            assert (err <= (2.0 ** -13 + 4 * 2.0 ** -24 * L) * scale + 2.0 ** -40).all()


@pytest.mark.parametrize("L", [1, 70])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gradients_of_gates_far_out(L, sign):
    """r or i between 8 and 20: their gradients hold the small factor 1 - sigmoid to its last digits."""
    D = 64
    far = sign * torch.linspace(8, 20, D).expand(1, L, D).contiguous()
    x, zero = torch.zeros(1, L, D), torch.zeros(1, L, D)
    A = -torch.linspace(0.1, 2, D) / L
    if sign < 0:
        A = A * L                                                        # decays near 1
    h0, dh = torch.ones(1, D), torch.ones(1, D)
    _, _, got = both(x, far, zero, A, h0, zero, dh)
    want = O.glr_bwd(x, far, zero, A, zero, h0, None, dh)
    close(got["dr"], want["dr"][0])
    x = 1 + torch.rand(1, L, D, generator=torch.Generator().manual_seed(3))
    dy = torch.ones(1, L, D)
    _, _, got = both(x, zero, far, A - 0.3, h0, dy, dh)
    want = O.glr_bwd(x, zero, far, A - 0.3, dy, h0, None, dh)
    close(got["di"], want["di"][0])
    close(got["dx"], want["dx"][0])


@pytest.mark.parametrize("L", [1, 7, 70, 200])
@pytest.mark.parametrize("D", [6, 5])
def test_a_channel_without_memory(L, D):
    """A = -infinity is a decay of 0: y = sigmoid(i) x, and gradients that end at their token."""
    g = torch.Generator().manual_seed(L)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, r, i, h0, dy, dh = n(2, L, D), n(2, L, D), n(2, L, D), n(2, D), n(2, L, D), n(2, D)
    A = -torch.rand(D, generator=g) - 0.5
    A[2] = -float("inf")
    y, h, got = both(x, r, i, A, h0, dy, dh)
    s = torch.sigmoid(i.double())
    v = s * x.double()
    G = dy.double().clone()
    G[:, -1] += dh.double()
    close(y[..., 2], v[..., 2])
    close(h[:, 2], v[:, -1, 2])
    close(got["dx"][..., 2], (G * s)[..., 2])
    close(got["di"][..., 2], (G * v * (1 - s))[..., 2])
    assert (got["dr"][..., 2] == 0).all() and got["dA"][2] == 0 and (got["dstate_init"][:, 2] == 0).all()
    other = [k for k in range(D) if k != 2]
    fin = A.clone()
    fin[2] = -1.0
    for a, b in zip((y, h, *got.values()), (lambda t: (t[0], t[1], *t[2].values()))(both(x, r, i, fin, h0, dy, dh))):
        assert torch.equal(a[..., other], b[..., other])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(4, 193, 7160), (4, 250, 7171), (3, 513, 4300), (1, 4096, 1790), (1, 4090, 1795)])
def test_backward_on_both_sides_of_the_tile_limit(B, L, D, io):
    """896 tiles of 64 tokens and more (ordinary inputs)."""
    ordinary.test_backward(B, L, D, io, "rare")
