"""CPU: the 64-bit definitions of the gated delta rule and of the norms around a layer, against
automatic differentiation, differences and each other."""
import pytest
import torch

from oracle import ops as O

F64 = torch.float64


def rule(B, L, Hk, H, K, V, seed, resets=False):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r, dtype=F64)  # noqa: E731
    reset = (torch.rand(B, L, generator=r) < 0.2).to(torch.uint8) if resets else None
    return [n(B, L, Hk, K), n(B, L, Hk, K), n(B, L, H, V), -torch.rand(B, L, H, generator=r, dtype=F64), torch.rand(B, L, H, generator=r, dtype=F64)], \
        n(B, H, K, V), reset, n(B, L, H, V), n(B, H, K, V)


@pytest.mark.parametrize("eps", [1e-6, None])
@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("L", [1, 2, 9])
def test_delta_rule_gradients_match_autograd(L, resets, eps):
    x, S0, reset, dy, dS = rule(2, L, 2, 4, 5, 3, L, resets)
    leaves = [t.clone().requires_grad_(True) for t in (*x, S0)]
    y, S = O.gdr_fwd(*leaves[:5], state=leaves[5], reset=reset, eps=eps)
    ((dy * y).sum() + (dS * S).sum()).backward()
    got = O.gdr_bwd(*x, dy, S0, reset, dS, eps=eps)
    for name, leaf in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate_init"), leaves):
        assert torch.allclose(got[name], leaf.grad, rtol=1e-11, atol=1e-11), name


def test_delta_rule_gradients_match_differences():
    x, S0, reset, dy, dS = rule(1, 6, 1, 2, 3, 2, 3, True)
    got = O.gdr_bwd(*x, dy, S0, reset, dS)
    args = [*x, S0]

    def loss(*a):
        y, S = O.gdr_fwd(*a[:5], state=a[5], reset=reset)
        return float((dy * y).sum() + (dS * S).sum())

    eps = 1e-5          # central differences: eps^2 times third derivatives of order 10, rounding 1e-15 / eps
    for j, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dstate_init")):
        flat = got[name].reshape(-1)
        for i in range(flat.numel()):
            up, dn = [t.clone() for t in args], [t.clone() for t in args]
            up[j].reshape(-1)[i] += eps
            dn[j].reshape(-1)[i] -= eps
            assert abs((loss(*up) - loss(*dn)) / (2 * eps) - float(flat[i])) <= 1e-7, (name, i)


def test_delta_rule_is_what_it_says():
    """beta = 1 and no decay: after a token its key reads back its value; orthogonal keys keep theirs;
    pieces equal the whole; a reset is a new sequence."""
    x, S0, _, _, _ = rule(1, 4, 1, 1, 4, 3, 5)
    q, k, v, g, beta = x
    k = torch.eye(4, dtype=F64).view(1, 4, 1, 4)
    y, S = O.gdr_fwd(k, k, v, torch.zeros_like(g), torch.ones_like(beta), scale=1.0, eps=None)
    assert torch.allclose(y, v) and torch.allclose(S[0, 0], v[0, :, 0])
    y, S = O.gdr_fwd(q, x[1], v, g, beta, S0)
    y1, S1 = O.gdr_fwd(q[:, :1], x[1][:, :1], v[:, :1], g[:, :1], beta[:, :1], S0)
    y2, S2 = O.gdr_fwd(q[:, 1:], x[1][:, 1:], v[:, 1:], g[:, 1:], beta[:, 1:], S1)
    assert torch.allclose(torch.cat([y1, y2], 1), y) and torch.allclose(S2, S)
    reset = torch.tensor([[0, 0, 1, 0]], dtype=torch.uint8)
    bad = v.clone()
    bad[:, 0] = float("nan")
    yr, Sr = O.gdr_fwd(q, x[1], bad, g, beta, S0 * float("inf"), reset)
    yn, Sn = O.gdr_fwd(q[:, 2:], x[1][:, 2:], v[:, 2:], torch.cat([g[:, 2:3] * 0 - 1e9, g[:, 3:]], 1), beta[:, 2:])
    assert torch.equal(yr[:, 2:], yn) and torch.equal(Sr, Sn)


@pytest.mark.parametrize("gate,residual,scale,nxt", [(1, 1, 1, 1), (0, 0, 0, 0), (1, 0, 0, 1), (0, 1, 0, 0), (0, 1, 1, 1)])
@pytest.mark.parametrize("group", [12, 4, 1])
def test_norm_gradients_match_autograd(gate, residual, scale, nxt, group):
    r = torch.Generator().manual_seed(group)
    n = lambda *s: torch.randn(*s, generator=r, dtype=F64)  # noqa: E731
    x = dict(y=n(3, 12), w=n(group), gate=n(3, 12) if gate else None, residual=n(3, 12) if residual else None,
             scale=n(12) if scale else None, w_next=n(12) if nxt else None)
    ds, dn = n(3, 12), n(3, 12) if nxt else None
    leaves = {k: t.clone().requires_grad_(True) for k, t in x.items() if t is not None}
    s, m = O.gnorm_fwd(**{**x, **leaves})
    ((ds * s).sum() + (0 if m is None else (dn * m).sum())).backward()
    got = O.gnorm_bwd(ds=ds, dn=dn, **x)
    assert set(got) == {"d" + k for k in leaves}
    for k, leaf in leaves.items():
        assert torch.allclose(got["d" + k][0], leaf.grad, rtol=1e-10, atol=1e-11), k


def test_norm_gradients_match_differences():
    r = torch.Generator().manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=r, dtype=F64)  # noqa: E731
    x = dict(y=n(2, 6), w=n(3), gate=n(2, 6), residual=n(2, 6), scale=n(6), w_next=n(6))
    ds, dn = n(2, 6), n(2, 6)
    got = O.gnorm_bwd(ds=ds, dn=dn, **x)

    def loss(x):
        s, m = O.gnorm_fwd(**x)
        return float((ds * s).sum() + (dn * m).sum())

    eps = 1e-5
    for name, t in x.items():
        flat = got["d" + name][0].reshape(-1)
        for i in range(flat.numel()):
            up, lo = dict(x), dict(x)
            up[name], lo[name] = t.clone(), t.clone()
            up[name].reshape(-1)[i] += eps
            lo[name].reshape(-1)[i] -= eps
            assert abs((loss(up) - loss(lo)) / (2 * eps) - float(flat[i])) <= 1e-7, (name, i)
