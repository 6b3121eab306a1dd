"""CPU: the delta rule's and the norms' C ABI refuses bad arguments on the host before anything reaches
the device. No compute call is made (a forward of no tokens enqueues nothing)."""
import ctypes

import pytest
import torch

import selective_state_space_73_amd as ss

BASE = 1 << 40
GAP = 1 << 38
WS = BASE + 100 * GAP


def last():
    return ss.lib.ss_last_error().decode()


def rdims(**kw):
    d = dict(batch=2, seqlen=200, k_heads=2, heads=4, dk=64, dv=48, io_dtype=ss.SS_F32, scale=0.125, eps=1e-6, reserved=0)
    d.update(kw)
    return ss.ss_gdr_dims(*d.values())


def rargs(**kw):
    v = lambda k, h, d: ss.ss_head_view(BASE + k * GAP, 200 * h * d, h * d, d)  # noqa: E731
    a = dict(q=v(0, 2, 64), k=v(1, 2, 64), v=v(2, 4, 48), g=BASE + 3 * GAP, beta=BASE + 4 * GAP, reset=None, y=BASE + 5 * GAP,
             state=BASE + 6 * GAP, ckpt=BASE + 7 * GAP)
    a.update(kw)
    return ss.ss_gdr_args(*a.values())


def rgrads(**kw):
    a = {n: BASE + (10 + k) * GAP for k, n in enumerate(("dy", "dstate_final", "dq", "dk", "dv", "dg", "dbeta", "dstate_init"))}
    a.update(kw)
    return ss.ss_gdr_grads(*a.values())


def rcall(which, dims=None, args=None, grads=None, ws=WS, ws_bytes=1 << 36):
    dims, args = dims or rdims(), args or rargs()
    if which == "fwd":
        return ss.lib.ss_gdr_fwd(ctypes.byref(dims), ctypes.byref(args), ws, ws_bytes, None)
    if which == "step":
        return ss.lib.ss_gdr_step(ctypes.byref(dims), ctypes.byref(args), None)
    return ss.lib.ss_gdr_bwd(ctypes.byref(dims), ctypes.byref(args), ctypes.byref(grads or rgrads()), ws, ws_bytes, None)


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
@pytest.mark.parametrize("kw,status", [(dict(batch=0), 1), (dict(k_heads=0), 1), (dict(heads=0), 1), (dict(heads=3), 1), (dict(dk=0), 1),
                                       (dict(dv=0), 1), (dict(dk=257), 2), (dict(dv=513), 2), (dict(io_dtype=5), 2), (dict(reserved=1), 1),
                                       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(eps=-1.0), 1),
                                       (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(batch=1 << 31), 1), (dict(batch=1 << 18), 1),
                                       (dict(heads=1 << 17, k_heads=1 << 17), 2)])
def test_rule_bad_dims(which, kw, status):
    assert rcall(which, rdims(**kw)) == status


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("seqlen", [-3, 1 << 31, 1 << 28])
def test_rule_bad_length(which, seqlen):
    assert rcall(which, rdims(seqlen=seqlen)) == 1


def test_rule_of_no_tokens():
    none = ss.ss_head_view(None, 0, 0, 0)
    assert rcall("fwd", rdims(seqlen=0), rargs(q=none, k=none, v=none, y=None), ws=None, ws_bytes=0) == 0
    assert rcall("bwd", rdims(seqlen=0)) == 1 and "seqlen" in last()
    assert ss.ss_gdr_workspace_bytes(rdims(seqlen=0)) == 0 and ss.gdr_ckpt_shape(2, 0, 4, 64, 48) == (0,)


def test_rule_missing_arguments():
    for n in ("q", "k", "v"):
        assert rcall("fwd", args=rargs(**{n: ss.ss_head_view(None, 1, 1, 1)})) == 1 and n in last()
    for n in ("g", "beta", "y"):
        assert rcall("fwd", args=rargs(**{n: None})) == 1 and n in last()
    assert rcall("step", args=rargs(state=None)) == 1 and "state" in last()
    assert rcall("bwd", args=rargs(ckpt=None)) == 1 and "ckpt" in last()
    for n in ("dy", "dq", "dk", "dv", "dg", "dbeta"):
        assert rcall("bwd", grads=rgrads(**{n: None})) == 1 and n in last()
    assert ss.lib.ss_gdr_bwd(ctypes.byref(rdims()), ctypes.byref(rargs()), None, WS, 1 << 36, None) == 1
    assert ss.lib.ss_gdr_fwd(None, ctypes.byref(rargs()), WS, 1 << 36, None) == 1
    assert ss.lib.ss_gdr_fwd(ctypes.byref(rdims()), None, WS, 1 << 36, None) == 1
    assert ss.lib.ss_gdr_step(ctypes.byref(rdims()), None, None) == 1


def test_rule_alignment_strides_overlaps():
    assert rcall("fwd", args=rargs(q=ss.ss_head_view(BASE + 2, 1, 1, 1))) == 1 and "aligned" in last()
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1)):
        assert rcall("fwd", args=rargs(k=ss.ss_head_view(BASE + GAP, *bad))) == 1 and "negative" in last()
    assert rcall("fwd", args=rargs(v=ss.ss_head_view(BASE + 2 * GAP, 1 << 61, 1, 1))) == 1 and "too many" in last()
    for n in ("g", "beta", "state", "ckpt", "y"):
        assert rcall("fwd", args=rargs(**{n: BASE + 30 * GAP + 2})) == 1 and "aligned" in last(), n
    for n in ("dy", "dq", "dk", "dv", "dg", "dbeta", "dstate_final", "dstate_init"):
        assert rcall("bwd", grads=rgrads(**{n: BASE + 30 * GAP + 2})) == 1 and "aligned" in last(), n
    assert rcall("fwd", args=rargs(y=BASE + 64)) == 1 and "y overlaps q" in last()
    assert rcall("fwd", args=rargs(state=BASE + 3 * GAP)) == 1 and "overlaps g" in last()
    assert rcall("fwd", args=rargs(ckpt=BASE + 6 * GAP + 4)) == 1 and "overlaps" in last()
    assert rcall("fwd", args=rargs(reset=BASE + 5 * GAP + 64)) == 1 and "overlaps reset" in last()
    assert rcall("step", args=rargs(state=BASE + 2 * GAP)) == 1 and "overlaps" in last()
    assert rcall("bwd", grads=rgrads(dq=BASE + 10 * GAP)) == 1 and "dq overlaps dy" in last()
    assert rcall("bwd", grads=rgrads(dk=BASE + 12 * GAP)) == 1 and "overlaps" in last()
    assert rcall("bwd", grads=rgrads(dv=WS + 512)) == 1 and "workspace" in last()
    # strides that do not matter are not looked at
    one = rdims(batch=1, k_heads=1, heads=1)
    assert rcall("fwd", one, rargs(q=ss.ss_head_view(BASE, -7, 64, -9)), ws=None) == 3


def test_rule_workspace():
    need = ss.ss_gdr_workspace_bytes(rdims())
    assert need > 0 and rcall("fwd", ws_bytes=need - 1) == 3 and rcall("fwd", ws=None, ws_bytes=need) == 3
    assert rcall("fwd", ws=WS + 8, ws_bytes=need) == 1
    back = ss.ss_gdr_workspace_bytes(rdims(), True)
    assert back > need and rcall("bwd", ws_bytes=back - 1) == 3
    # shared heads of keys need each head's share
    assert back - ss.ss_gdr_workspace_bytes(rdims(k_heads=4), True) == 2 * 2 * 200 * 4 * 64 * 4
    # states before every 64th token, then what each token writes
    assert ss.gdr_ckpt_shape(2, 200, 4, 64, 48) == (2 * 4 * 4 * 64 * 48 + 2 * 200 * 4 * 48,)
    with pytest.raises(ValueError):
        ss.gdr_ckpt_shape(2, 200, 4, 300, 48)


def ndims(**kw):
    d = dict(rows=70, cols=300, group=100, io_dtype=ss.SS_BF16, eps=1e-5)
    d.update(kw)
    return ss.ss_gnorm_dims(*d.values())


def nargs(**kw):
    a = {n: BASE + k * GAP for k, n in enumerate(("y", "w", "gate", "residual", "scale", "w_next", "s", "n"))}
    a.update(kw)
    return ss.ss_gnorm_args(*a.values())


def ngrads(**kw):
    a = {n: BASE + (10 + k) * GAP for k, n in enumerate(("ds", "dn", "dy", "dgate", "dresidual", "dw", "dscale", "dw_next"))}
    a.update(kw)
    return ss.ss_gnorm_grads(*a.values())


def nfwd(dims=None, **kw):
    return ss.lib.ss_gnorm_fwd(ctypes.byref(dims or ndims()), ctypes.byref(nargs(**kw)), None)


def nbwd(dims=None, args=None, ws=WS, ws_bytes=1 << 30, **kw):
    return ss.lib.ss_gnorm_bwd(ctypes.byref(dims or ndims()), ctypes.byref(args or nargs()), ctypes.byref(ngrads(**kw)), ws, ws_bytes, None)


def test_norm_refusals():
    for kw, status in [(dict(rows=0), 1), (dict(cols=0), 1), (dict(group=0), 1), (dict(group=7), 1), (dict(rows=1 << 31), 1),
                       (dict(cols=16385, group=16385), 2), (dict(io_dtype=4), 2), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
                       (dict(eps=float("inf")), 1)]:
        assert nfwd(ndims(**kw)) == status and nbwd(ndims(**kw)) == status, kw
        assert ss.ss_gnorm_workspace_bytes(ndims(**kw)) == 0
    for n in ("y", "w", "s", "n"):
        assert nfwd(**{n: None}) == 1 and n in last(), n
    assert nfwd(w_next=None) == 1 and "without w_next" in last()
    for n in ("y", "gate", "residual", "s", "n"):
        assert nfwd(**{n: BASE + 30 * GAP + 1}) == 1 and "aligned" in last(), n
    for n in ("w", "scale", "w_next"):
        assert nfwd(**{n: BASE + 30 * GAP + 2}) == 1 and "aligned" in last(), n
    for a, b in [("s", "w"), ("n", "y"), ("n", "s"), ("n", "residual"), ("s", "scale")]:
        at = {n: BASE + k * GAP for k, n in enumerate(("y", "w", "gate", "residual", "scale", "w_next", "s", "n"))}
        assert nfwd(**{a: at[b]}) == 1 and "overlaps" in last(), (a, b)
    for b in range(4):                                  # in place: exactly, not shifted
        if b != 1:
            assert nfwd(s=BASE + b * GAP + 64) == 1 and "overlaps" in last()
    assert ss.lib.ss_gnorm_fwd(None, ctypes.byref(nargs()), None) == 1 and ss.lib.ss_gnorm_fwd(ctypes.byref(ndims()), None, None) == 1


def test_norm_backward_refusals():
    assert nbwd(ds=None, dn=None) == 1 and "required" in last()
    assert nbwd(args=nargs(w_next=None, n=None)) == 1 and "without w_next" in last()
    for n in ("dy", "dgate", "dresidual", "dw", "dscale", "dw_next"):
        assert nbwd(**{n: None}) == 1 and n in last(), n
        assert nbwd(**{n: BASE + 30 * GAP + 1}) == 1 and "aligned" in last(), n
    for n, o in (("gate", "dgate"), ("residual", "dresidual"), ("scale", "dscale")):
        assert nbwd(args=nargs(**{n: None})) == 1 and o in last(), n
    assert nbwd(dy=BASE) == 1 and "dy overlaps y" in last()
    assert nbwd(dgate=BASE + 10 * GAP + 64) == 1 and "overlaps ds" in last()
    assert nbwd(dw=WS + 64) == 1 and "workspace" in last()
    need = ss.ss_gnorm_workspace_bytes(ndims())
    assert nbwd(ws_bytes=need - 1) == 3 and nbwd(ws=None) == 3 and nbwd(ws=WS + 4) == 1
    assert ss.lib.ss_gnorm_bwd(ctypes.byref(ndims()), ctypes.byref(nargs()), None, WS, 1 << 30, None) == 1


def test_binding_refuses_host_tensors_and_shapes():
    q, v, g = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2)
    for call in (lambda: ss.ss_gdr_fwd(q, q, v, g, g), lambda: ss.ss_gdr_step(q[0], q[0], v[0], g[0], g[0], v),
                 lambda: ss.ss_gdr_bwd(q, q, v, g, g, v, v), lambda: ss.ss_gnorm_fwd(q, torch.ones(8)),
                 lambda: ss.ss_gnorm_bwd(q, torch.ones(8), q)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ss.ss_gdr_fwd(None, q, v, g, g)
