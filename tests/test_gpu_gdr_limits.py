"""GPU: the gated delta rule at the edges of what its calls allow, against its 64-bit definition. Tolerances as in
test_gpu_gdr.py, from which the inputs and the comparisons come."""
import pytest
import torch

from oracle import ops as O

pytestmark = pytest.mark.gpu

ss = pytest.importorskip("selective_state_space_73_amd")
T = pytest.importorskip("test_gpu_gdr")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 64 * 9, 1, 1, 64, 64), (1, 64 * 8 + 1, 1, 3, 100, 70), (2, 1100, 1, 2, 128, 128)])
def test_state_in_and_out_beside_other_work(shape, io):
    """The segments of a sequence run in any order, the last one, which stores the state, before the first one, which
    starts from it, too: other kernels on another stream take places that the first ones wait for."""
    x, S0, dy, dS, _ = T.make(*shape, io, seed=41)
    T.check(x, S0, dy, dS, io)
    want = T.run(x, S0)
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for n in range(8):
        with torch.cuda.stream(side):
            for _ in range(1 + n % 3):
                b = a @ a
        got = T.run(x, S0)
        assert all(torch.equal(s, t) for s, t in zip(got, want))
        torch.cuda.synchronize()
    assert torch.isfinite(b[0, 0])


@pytest.mark.parametrize("K", [2, 8, 100, 128, 256])
def test_what_is_made_in_32_bits_keeps_them(K):
    """States, products with beta, solutions and pairs of tokens of 1 + 2^-8 + 2^-20, each times 1 and next to zeros: every
    product and sum is exact in 32 bits, and the result is 2^-20 above a tie of bf16, so that it rounds up to 1 + 2^-7. With
    fewer than 20 bits of any of them it would be the tie, which goes to 1."""
    up, tie = 1.0 + 2.0 ** -7, 1.0 + 2.0 ** -8 + 2.0 ** -20
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    q, k, v = z(1, 2, 1, K), z(1, 2, 1, K), z(1, 2, 1, 1)
    g, beta = z(1, 2, 1), z(1, 2, 1)

    def call(S=None, dy=None):
        x = (*(t.bfloat16() for t in (q, k, v)), g, beta)
        ck = torch.empty(ss.gdr_ckpt_shape(1, 2, 1, K, 1), device="cuda")
        y = ss.ss_gdr_fwd(*x, scale=1.0, eps=None, state=S, ckpt=ck)
        return y if dy is None else ss.ss_gdr_bwd(*x, ck, dy.bfloat16(), scale=1.0, eps=None)

    # y = S^T q
    q[..., 0] = 1.0
    S = z(1, 1, K, 1)
    S[..., 0, 0] = tie
    assert (call(S).float() == up).all()
    # y_0 = (q . k) beta v
    k[0, 0, 0, 0], v[0, 0, 0, 0], beta[0, 0, 0] = 1.0, 1.0, tie
    assert call()[0, 0, 0, 0].item() == up
    # and its gradients: beta (dy . v) k and beta (dy . v) q
    dy = z(1, 2, 1, 1)
    dy[0, 0] = 1.0
    got = call(dy=dy)
    assert got["dq"][0, 0, 0, 0].item() == up and got["dk"][0, 0, 0, 0].item() == up and got["dv"][0, 0, 0, 0].item() == up
    # x_1 = v_1 - beta_0 (k_1 . k_0) v_0, alone in y_1
    k[0, 1, 0, :2] = 1.0
    q[0, 1, 0, 0], q[0, 1, 0, 1] = 0.0, 1.0
    v[0, 1], beta[0, 0, 0], beta[0, 1, 0] = up, 2.0 ** -8 - 2.0 ** -20, 1.0
    assert call()[0, 1, 0, 0].item() == up
    # -beta_0 (dv_1 . x_0) k_0 in the gradient of k_1
    k[0, 1, 0, 0], beta[0, 0, 0], v[0, 1] = 0.0, tie, 0.0
    dy[0, 0], dy[0, 1] = 0.0, 1.0
    assert call(dy=dy)["dk"][0, 1, 0, 0].item() == -up


@pytest.mark.parametrize("heads", [2, 300])
def test_gradients_of_no_tokens_are_refused(heads):
    x, _, dy, _, _ = T.make(1, 0, 1, heads, 16, 32, "bf16")
    with pytest.raises(ss.SelscanError):
        ss.ss_gdr_bwd(*x, torch.empty(0, device="cuda"), dy)
    assert ss.ss_gdr_fwd(*x).shape == (1, 0, heads, 32)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("beta", [2.5, -0.5])
def test_a_reset_ends_a_segments_memory_whatever_beta_is_behind_it(beta, io):
    """Nine chunks in segments of 4, 4 and 1. The state in front is NaN up to a reset in the middle segment; behind the reset one
    beta is outside [0, 2]. A state grows by at most 1.5 there, and an error with it."""
    x, _, dy, dS, _ = T.make(1, 64 * 9, 1, 2, 64, 48, io, seed=43)
    S0 = torch.full((1, 2, 64, 48), float("nan"), device="cuda")
    at = 64 * 5
    x[4][0, at + 70] = beta
    z = torch.zeros(1, 64 * 9, dtype=torch.uint8, device="cuda")
    z[0, at] = 1
    y, S, ck = T.run(x, S0, reset=z)
    tail = tuple(t[:, at:] for t in x)
    yw, Sw = O.gdr_fwd(*tail)
    T.near(y[:, at:], yw, 1.5 * T.rel(64, 256), io)
    T.near(S, Sw, 1.5 * T.rel(64, 256), "f32")
    assert torch.isnan(y[:, :at]).all()
    got, want = ss.ss_gdr_bwd(*x, ck, dy, reset=z, dstate_final=dS), O.gdr_bwd(*tail, dy[:, at:], None, None, dS)
    for n in ("dq", "dk", "dv", "dbeta"):
        T.near(got[n][:, at:], want[n], 1.5 ** 2 * 2 * T.rel(64, 256, 48), io if n != "dbeta" else "f32")
    # the state's gradient does not depend on the state
    want = O.gdr_bwd(*(t[:, :at] for t in x), dy[:, :at])["dstate_init"]
    T.near(got["dstate_init"], want, 2 * T.rel(64, at, 48), "f32")


def fading(K, V, io, heads=1):
    """Nine chunks, in segments of 4, 4 and 1, each of which brings a state down by 2^-13, and nothing beside it. A power of two
    is the state's own size, so that 2^60 stays within fp32 in products of a state and a gradient."""
    x, S0, dy, dS, _ = T.make(1, 64 * 9, heads, heads, K, V, io, seed=47 + K)
    x[2].zero_()
    x[4].zero_()
    dy.zero_()
    x[3].fill_(-13 / 64 * 0.6931471805599453)
    return x, S0 * 2.0 ** 60, dy, dS * 2.0 ** 60


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (100, 70), (128, 128), (256, 80)])
def test_segments_keep_what_is_left_of_large_states(K, V, io):
    """2^60 down to 2^-57: every result is relative to what is left, with states from the forward and by a copy of a row at
    a later chunk."""
    x, S0, _, _ = fading(K, V, io)
    y, S, _ = T.run(x, S0)
    yw, Sw = O.gdr_fwd(*x, S0)
    for n in range(0, 9):
        at = slice(64 * n + 60, 64 * n + 64)
        T.near(y[:, at], yw[:, at], T.rel(K, 512), io)
    T.near(S, Sw, T.rel(K, 512), "f32")
    # a value in one chunk of a segment, nothing in the next ones, and a short segment behind them
    x[2][:, 200] = 2.0 ** 40
    x[4][:, 200] = 1.0
    y, S, ck = T.run(x, S0)
    yw, Sw = O.gdr_fwd(*x, S0)
    for n in range(4, 9):
        at = slice(64 * n + 60, 64 * n + 64)
        T.near(y[:, at], yw[:, at], T.rel(K, 512), io)
    T.near(S, Sw, T.rel(K, 512), "f32")
    T.near(ck[:-64 * 9 * V].view(9, K, V)[8], O.gdr_fwd(*(t[:, :512] for t in x), S0)[1][0, 0], T.rel(K, 512), "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_nan_stays_however_the_call_is_cut(io):
    """One head of one row runs in segments, of many rows in one: a NaN, which no decay but one of 0 ends, reaches the same
    tokens."""
    x, S0, _, _ = fading(64, 96, io)
    x[2].copy_(torch.randn_like(x[2]))
    x[4].fill_(0.5)
    x[2][0, 10, 0, 3] = float("nan")
    S0[0, 0, 7, 70] = float("inf")
    y, S, _ = T.run(x, S0)
    many = tuple(t.expand(300, *t.shape[1:]).contiguous() for t in x)
    ym, Sm, _ = T.run(many, S0.expand(300, -1, -1, -1))
    bad = torch.zeros(96, dtype=torch.bool, device="cuda")
    bad[3] = bad[70] = True
    for a, b in ((y, S), (ym[:1], Sm[:1])):
        assert (torch.isfinite(a[0, 64:, 0]) == ~bad).all() and (torch.isfinite(b[0, 0]) == ~bad).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (100, 70), (128, 128), (256, 80)])
def test_segments_keep_what_is_left_of_large_gradients(K, V, io):
    """A gradient of the final state of 2^60 that comes down to 2^-57, beside a state of that size in front."""
    x, S0, dy, dS = fading(K, V, io)
    _, _, ck = T.run(x, S0)
    got, want = ss.ss_gdr_bwd(*x, ck, dy, dstate_final=dS), O.gdr_bwd(*x, dy, S0, None, dS)
    for n in ("dg", "dbeta", "dstate_init"):
        assert want[n].abs().max() > 0
        T.near(got[n], want[n], 2 * T.rel(K, 512, V), "f32")
    # and the other way round: a gradient of an output in a late chunk, nothing in front of it
    dy[:, 400] = 2.0 ** 40
    x[4][:, 300:] = 0.5
    x[4][:, 400:] = 0.0
    _, _, ck = T.run(x, S0)
    got, want = ss.ss_gdr_bwd(*x, ck, dy, dstate_final=dS), O.gdr_bwd(*x, dy, S0, None, dS)
    T.near(got["dstate_init"], want["dstate_init"], 2 * T.rel(K, 512, V), "f32")
    for n in range(6):
        at = slice(64 * n, 64 * n + 4)
        T.near(got["dg"][:, at], want["dg"][:, at], 2 * T.rel(K, 512, V), "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_nan_gradients_stay_however_the_call_is_cut(io):
    x, S0, dy, dS = fading(64, 96, io)
    x[4].fill_(0.5)
    dy.copy_(torch.randn_like(dy))
    dS[0, 0, 9, 70] = float("inf")
    dy[0, 500, 0, 3] = float("nan")
    bad = torch.zeros(96, dtype=torch.bool, device="cuda")
    bad[3] = bad[70] = True
    for B in (1, 300):
        many = tuple(t.expand(B, *t.shape[1:]).contiguous() for t in x)
        _, _, ck = T.run(many, S0.expand(B, -1, -1, -1))
        got = ss.ss_gdr_bwd(*many, ck, dy.expand(B, -1, -1, -1).contiguous(), dstate_final=dS.expand(B, -1, -1, -1).contiguous())
        assert (torch.isfinite(got["dv"][0, :448, 0]) == ~bad).all()
        assert (torch.isfinite(got["dstate_init"][0, 0]) == ~bad).all()


def same_finite(got, want, tol, io):
    """Finite in the same places, and there within the tolerance of the largest finite value."""
    got, want = got.double().cpu(), want.double()
    ok = torch.isfinite(want)
    assert (torch.isfinite(got) == ok).all()
    T.near(torch.where(ok, got, 0.0), torch.where(ok, want, 0.0), tol, io)


PLACES = ["v", "inf v", "k", "inf k", "beta", "g", "q", "state", "k in front of a reset", "beta in front of a reset"]


def not_finite(place, x, S0, n):
    """One value of the document [n, n + 50) of x, or of the state."""
    q, k, v, g, beta = x
    if place in ("v", "inf v"):
        v[0, n + 20, 0, 3] = float("nan") if place == "v" else float("-inf")
    elif place in ("k", "inf k"):
        k[0, n + 20, 0, 1] = float("nan") if place == "k" else float("inf")
    elif place == "k in front of a reset":
        k[0, n + 49, 0, 1] = float("nan")
    elif place == "beta in front of a reset":
        beta[0, n + 49, 0] = float("nan")
    elif place == "beta":
        beta[0, n + 20, 0] = float("inf")
    elif place == "g":
        g[0, n + 20, 0] = float("nan")
    elif place == "q":
        q[0, n + 20, 0, 1] = float("nan")
    else:
        S0[0, 0, 5, 2] = float("nan")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("shape,at", [((1, 200, 1, 2, 64, 48), 70), ((1, 200, 2, 2, 100, 33), 0), ((1, 64 * 9, 1, 1, 64, 80), 330),
                                      ((2, 64 * 9, 1, 2, 128, 128), 64 * 8 + 1)])
def test_what_is_not_finite_keeps_to_its_document(shape, at, place, io):
    """Documents of 50 tokens, their first ones anywhere in a chunk, one of them with a value that is not finite: it
    reaches what the formulas say, no token in front of it and none behind the next reset, in one segment and in several."""
    x, S0, _, _, _ = T.make(*shape, io, seed=53)
    z = torch.zeros(shape[0], shape[1], dtype=torch.uint8, device="cuda")
    z[:, at % 50::50] = 1
    if place == "state":
        z[:, :20] = 0
    not_finite(place, x, S0, at)
    y, S, ck = T.run(x, S0, reset=z)
    yw, Sw = O.gdr_fwd(*x, S0, z)
    same_finite(y, yw, T.rel(shape[4], 50), io)
    same_finite(S, Sw, T.rel(shape[4], 50), "f32")
    # the states in front of the chunks
    n = -(-shape[1] // 64)
    states = ck[:shape[0] * shape[3] * n * shape[4] * shape[5]].view(shape[0], shape[3], n, shape[4], shape[5])
    for c in (1, n - 1):
        same_finite(states[:, :, c], O.gdr_fwd(*(t[:, :64 * c] for t in x), S0, z[:, :64 * c])[1], T.rel(shape[4], 50), "f32")


def test_a_state_that_is_reset_may_hold_anything():
    """Nothing of it is looked at, so that starting over costs nothing."""
    x, S0, _, _, _ = T.make(1, 64 * 9, 1, 2, 64, 64, "bf16", seed=59)
    z = torch.zeros(1, 64 * 9, dtype=torch.uint8, device="cuda")
    z[0, 0] = 1
    S0.fill_(float("nan"))
    y, S, _ = T.run(x, S0, reset=z)
    yw, Sw = O.gdr_fwd(*x)
    T.near(y, yw, T.rel(64, 512), "bf16")
    T.near(S, Sw, T.rel(64, 512), "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("place", PLACES + ["dy", "inf dy", "dstate"])
@pytest.mark.parametrize("shape,at,unit", [((1, 200, 1, 2, 64, 48), 70, True), ((1, 200, 2, 2, 100, 33), 0, False),
                                           ((1, 64 * 9, 1, 1, 64, 80), 330, True), ((2, 64 * 9, 1, 2, 128, 128), 64 * 8 + 1, True),
                                           ((1, 100, 1, 1, 200, 20), 31, True)])
def test_gradients_of_what_is_not_finite_keep_to_its_document(shape, at, unit, place, io):
    x, S0, dy, dS, _ = T.make(*shape, io, seed=61)
    K, V, eps = shape[4], shape[5], 1e-6 if unit else None
    if not unit:
        x[1].mul_(K ** -0.5)
    z = torch.zeros(shape[0], shape[1], dtype=torch.uint8, device="cuda")
    z[:, at % 50::50] = 1
    if place == "state":
        z[:, :20] = 0
    if place in ("dy", "inf dy"):
        dy[0, at + 20, 0, 3] = float("nan") if place == "dy" else float("inf")
    elif place == "dstate":
        dS[0, 0, 5, 2] = float("nan")
    else:
        not_finite(place, x, S0, at)
    _, _, ck = T.run(x, S0, reset=z, eps=eps)
    got, want = ss.ss_gdr_bwd(*x, ck, dy, reset=z, dstate_final=dS, eps=eps), O.gdr_bwd(*x, dy, S0, z, dS, None, eps)
    assert any(not torch.isfinite(v).all() for v in want.values()) or place in ("dy", "inf dy", "dstate")
    want["dg"] = want["dg"].masked_fill((z != 0).cpu()[..., None], 0.0)
    for n in T.GRADS:
        print(n, end=" ")
        same_finite(got[n], want[n], 2 * T.rel(K, 64, V), io if n in ("dq", "dk", "dv") else "f32")


@pytest.mark.parametrize("eps", [0.0, -0.0, 1e-60])
def test_an_eps_of_zero_is_refused(eps):
    """It is not None, for which lengths are left alone: sqrt(sum x^2 + 0) has no value for a key of zeros."""
    x, S0, dy, _, _ = T.make(1, 20, 1, 1, 16, 16, "f32")
    _, _, ck = T.run(x)
    with pytest.raises(ValueError):
        ss.ss_gdr_fwd(*x, eps=eps)
    with pytest.raises(ValueError):
        ss.ss_gdr_bwd(*x, ck, dy, eps=eps)
    with pytest.raises(ValueError):
        ss.ss_gdr_step(*(t[:, 0] if t.dim() == 4 else t[:, 0].contiguous() for t in x), S0, eps=eps)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V,odd", [(64, 150, 3), (100, 70, 64), (128, 128, 127)])
def test_one_column_that_runs_again(K, V, odd, io):
    """Columns of a state do not depend on each other: one of 2^60 that nothing is added to, among others of about 1, with a NaN in
    one more. Each is relative to its own size, over the last tokens of every chunk."""
    x, S0, dy, dS, _ = T.make(1, 64 * 11, 1, 2, K, V, io, seed=67 + K)
    x[3].fill_(-13 / 64 * 0.6931471805599453)
    x[2][..., odd] = 0.0
    S0[..., odd] *= 2.0 ** 60
    x[2][0, 30, 1, 5] = float("nan")
    y, S, ck = T.run(x, S0)
    yw, Sw = O.gdr_fwd(*x, S0)
    for n in range(11):
        at = slice(64 * n + 48, 64 * n + 64)
        for h in range(2):
            ok = torch.isfinite(yw[0, at, h]).all(0)
            assert ok.sum() == V - h
            got, want = y[0, at, h].double().cpu()[:, ok], yw[0, at, h][:, ok]
            size = want.abs().amax(0, keepdim=True)
            T.near(got / size, want / size, T.rel(K, 512), io)
    for h in range(2):
        ok = torch.isfinite(Sw[0, h]).all(0)
        assert (torch.isfinite(S[0, h]).all(0).cpu() == ok).all()
        size = Sw[0, h].abs().amax(0)[ok]
        T.near(S[0, h].double().cpu()[:, ok] / size, Sw[0, h][:, ok] / size, T.rel(K, 512), "f32")
