"""CPU: the operators' C ABI (include/selscan_ops.h) is exported, its structs have the layout the
binding assumes, and every call refuses bad arguments on the host before anything reaches the
device. No compute call is made."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import selective_state_space_73_amd as ss
from selective_state_space_73_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "selscan_ops.h")
BASE = 1 << 40
GAP = 1 << 36


def last():
    return ss.lib.ss_last_error().decode()


def test_header_symbols_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^(?:size_t|ss_status|int)\s+(ss_[a-z0-9_]+)\s*\(", text, flags=re.M))
    assert {"ss_glr_fwd", "ss_glr_bwd", "ss_glr_step", "ss_glr_workspace_bytes", "ss_quant_q8", "ss_norm_q8", "ss_gemm_q8"} <= names
    out = subprocess.run(["nm", "-D", "--defined-only", ss.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert names <= exported


def test_c_compiler_agrees_on_the_structs(tmp_path):
    """Sizes and offsets of every struct as a C compiler lays them out."""
    structs = [s for s in (getattr(ops, n) for n in ops.__all__) if isinstance(s, type) and issubclass(s, ctypes.Structure)]
    assert structs
    lines = []
    for s in structs:
        lines.append(f'printf("{s.__name__} %zu", sizeof({s.__name__}));')
        lines += [f'printf(" %zu", offsetof({s.__name__}, {f[0]}));' for f in s._fields_]
        lines.append('printf("\\n");')
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "selscan_ops.h"\nint main(void){' + "\n".join(lines) + "return 0;}\n")
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.strip().splitlines()
    for s, line in zip(structs, out):
        want = [s.__name__, ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
        assert line.split() == [str(v) for v in want]


# ---------------------------------------------------------------------------
# gated linear recurrence

def gdims(**kw):
    d = dict(batch=2, seqlen=200, d=64, io_dtype=ss.SS_F32, reserved=0)
    d.update(kw)
    return ss.ss_glr_dims(*d.values())


def gargs(**kw):
    v = lambda k: ss.ss_view(BASE + k * GAP, 200 * 64, 64)  # noqa: E731
    a = dict(x=v(0), r=v(1), i=v(2), A=BASE + 3 * GAP, reset=None, y=BASE + 4 * GAP, state=BASE + 5 * GAP, ckpt=BASE + 6 * GAP)
    a.update(kw)
    return ss.ss_glr_args(*a.values())


def ggrads(**kw):
    a = {n: BASE + (10 + k) * GAP for k, n in enumerate(("dy", "dstate_final", "dx", "dr", "di", "dA", "dstate_init"))}
    a.update(kw)
    return ss.ss_glr_grads(*a.values())


WS = BASE + 100 * GAP


def gcall(which, dims=None, args=None, grads=None, ws=WS, ws_bytes=1 << 30):
    dims, args = dims or gdims(), args or gargs()
    if which == "fwd":
        return ss.lib.ss_glr_fwd(ctypes.byref(dims), ctypes.byref(args), ws, ws_bytes, None)
    if which == "step":
        return ss.lib.ss_glr_step(ctypes.byref(dims), ctypes.byref(args), None)
    return ss.lib.ss_glr_bwd(ctypes.byref(dims), ctypes.byref(args), ctypes.byref(grads or ggrads()), ws, ws_bytes, None)


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
@pytest.mark.parametrize("kw,status", [(dict(batch=0), 1), (dict(d=0), 1), (dict(d=(1 << 26) + 1), 1), (dict(io_dtype=5), 2),
                                       (dict(reserved=1), 1), (dict(batch=1 << 31), 1)])
def test_recurrence_bad_dims(which, kw, status):
    assert gcall(which, gdims(**kw)) == status


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("seqlen", [0, -3, 1 << 31])
def test_recurrence_bad_length(which, seqlen):
    assert gcall(which, gdims(seqlen=seqlen)) == 1


def test_recurrence_missing_arguments():
    for n in ("x", "r", "i"):
        assert gcall("fwd", args=gargs(**{n: ss.ss_view(None, 1, 1)})) == 1 and n in last()
    assert gcall("fwd", args=gargs(A=None)) == 1
    assert gcall("fwd", args=gargs(y=None)) == 1
    assert gcall("step", args=gargs(state=None)) == 1 and "state" in last()
    assert gcall("bwd", args=gargs(ckpt=None)) == 1 and "ckpt" in last()
    for n in ("dy", "dx", "dr", "di", "dA"):
        assert gcall("bwd", grads=ggrads(**{n: None})) == 1 and n in last()
    assert ss.lib.ss_glr_bwd(ctypes.byref(gdims()), ctypes.byref(gargs()), None, WS, 1 << 30, None) == 1
    assert ss.lib.ss_glr_fwd(None, ctypes.byref(gargs()), WS, 1 << 30, None) == 1
    assert ss.lib.ss_glr_fwd(ctypes.byref(gdims()), None, WS, 1 << 30, None) == 1


def test_recurrence_alignment_strides_overlaps():
    assert gcall("fwd", args=gargs(x=ss.ss_view(BASE + 2, 200 * 64, 64))) == 1 and "aligned" in last()
    assert gcall("fwd", args=gargs(x=ss.ss_view(BASE, -1, 64))) == 1 and "negative" in last()
    assert gcall("fwd", args=gargs(x=ss.ss_view(BASE, 1 << 61, 64))) == 1 and "too many" in last()
    assert gcall("fwd", args=gargs(A=BASE + 3 * GAP + 2)) == 1
    assert gcall("fwd", args=gargs(y=BASE + 64)) == 1 and "y overlaps x" in last()
    assert gcall("fwd", args=gargs(state=BASE + 4 * GAP + 4)) == 1 and "overlaps" in last()
    assert gcall("fwd", args=gargs(state=BASE + 3 * GAP)) == 1 and "state overlaps A" in last()
    # the batch stride reaches further than the tokens of one row
    assert gcall("fwd", args=gargs(x=ss.ss_view(BASE, 1 << 30, 64), y=BASE + (1 << 32))) == 1
    assert gcall("bwd", grads=ggrads(dx=BASE + 10 * GAP)) == 1 and "dx overlaps dy" in last()
    assert gcall("bwd", grads=ggrads(dr=BASE + 12 * GAP)) == 1 and "overlaps" in last()
    assert gcall("bwd", grads=ggrads(di=WS + 512)) == 1 and "workspace" in last()


def test_recurrence_workspace():
    need = ss.ss_glr_workspace_bytes(gdims())
    assert need > 0 and gcall("fwd", ws_bytes=need - 1) == 3 and gcall("fwd", ws=None, ws_bytes=need) == 3
    assert gcall("fwd", ws=WS + 8, ws_bytes=need) == 1
    assert ss.ss_glr_workspace_bytes(gdims(seqlen=64)) == 0              # one chunk: nothing to hand over
    assert ss.ss_glr_workspace_bytes(gdims(seqlen=0)) == 0
    back = ss.ss_glr_workspace_bytes(gdims(), True)
    assert back > 0 and gcall("bwd", ws_bytes=back - 1) == 3


def test_binding_refuses_host_tensors():
    t = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        ss.ss_glr_fwd(t, t, t, torch.zeros(8))
    with pytest.raises(ValueError):
        ss.ss_glr_fwd(t[0], t[0], t[0], torch.zeros(8))
    with pytest.raises(ValueError):
        ss.ss_glr_step(t[0], t[0], t[0], torch.zeros(8), t[0])


# ---------------------------------------------------------------------------
# 8-bit floating point with block scales

def qdims(**kw):
    d = dict(rows=70, cols=300, io_dtype=ss.SS_BF16, square=0, eps=1e-5, reserved=0)
    d.update(kw)
    return ss.ss_q8_dims(*d.values())


def quant(dims=None, x=BASE, q=BASE + GAP, scale=BASE + 2 * GAP):
    return ss.lib.ss_quant_q8(ctypes.byref(dims or qdims()), x, q, scale, None)


def norm(dims=None, **kw):
    a = dict(x=BASE, residual=BASE + GAP, w=BASE + 2 * GAP, q=BASE + 3 * GAP, scale=BASE + 4 * GAP, sum=BASE + 5 * GAP)
    a.update(kw)
    return ss.lib.ss_norm_q8(ctypes.byref(dims or qdims()), ctypes.byref(ss.ss_norm_q8_args(*a.values())), None)


def test_rounding_refusals():
    for kw, status in [(dict(rows=0), 1), (dict(cols=0), 1), (dict(cols=1 << 31), 1), (dict(rows=1 << 31), 1),
                       (dict(io_dtype=3), 2), (dict(square=2), 1), (dict(reserved=1), 1),
                       (dict(rows=65536 * 128, square=1), 1)]:
        assert quant(qdims(**kw)) == status, kw
    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(x=BASE + 1), dict(scale=BASE + 2 * GAP + 2),
               dict(q=BASE + 16), dict(scale=BASE + GAP + 128)):
        assert quant(**kw) == 1, kw
    assert ss.lib.ss_quant_q8(None, BASE, BASE + GAP, BASE + 2 * GAP, None) == 1


def test_norm_refusals():
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(square=1), dict(rows=0), dict(reserved=3)):
        assert norm(qdims(**kw)) == 1, kw
    for kw in (dict(x=None), dict(w=None), dict(q=None), dict(scale=None), dict(sum=None), dict(residual=None),
               dict(x=BASE + 1), dict(w=BASE + 2 * GAP + 2), dict(q=BASE), dict(scale=BASE + 3 * GAP), dict(sum=BASE + 3 * GAP),
               dict(sum=BASE + 64), dict(sum=BASE + GAP + 64), dict(sum=BASE + 2 * GAP)):
        assert norm(**kw) == 1, kw
    assert ss.lib.ss_norm_q8(ctypes.byref(qdims()), None, None) == 1


def test_product_refusals():
    def call(dims=None, **kw):
        d = dict(m=70, n=130, k=272, y_dtype=ss.SS_BF16, reserved=0)
        d.update(dims or {})
        a = dict(xq=BASE, xs=BASE + GAP, wq=BASE + 2 * GAP, ws=BASE + 3 * GAP, residual=None, y=BASE + 4 * GAP)
        a.update(kw)
        return ss.lib.ss_gemm_q8(ctypes.byref(ss.ss_gemm_q8_dims(*d.values())), ctypes.byref(ss.ss_gemm_q8_args(*a.values())), None)

    for d, status in [(dict(m=0), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(k=264), 2), (dict(k=1 << 31), 1),
                      (dict(m=1 << 31), 1), (dict(y_dtype=2), 2), (dict(reserved=1), 1), (dict(m=(1 << 31) - 1, n=(1 << 31) - 1), 1)]:
        assert call(d) == status, d
    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y=None), dict(xq=BASE + 8), dict(wq=BASE + 2 * GAP + 4),
               dict(y=BASE + 4 * GAP + 8), dict(residual=BASE + 5 * GAP + 2), dict(xs=BASE + GAP + 2), dict(y=BASE),
               dict(y=BASE + 2 * GAP + 32), dict(y=BASE + 3 * GAP), dict(residual=BASE + 4 * GAP + 16)):
        assert call(**kw) == 1, kw


def test_binding_refuses_host_operands():
    t = torch.zeros(4, 128)
    for call in (lambda: ss.ss_quant_q8(t), lambda: ss.ss_norm_q8(t, torch.ones(128)),
                 lambda: ss.ss_gemm_q8(t.to(torch.float8_e4m3fn), t, t.to(torch.float8_e4m3fn), t)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# the block with 8-bit projections

WEIGHTS = ("norm_w", "W_in", "conv_w", "conv_b", "W_x", "W_dt", "dt_bias", "A", "Dskip", "W_out")


def bdims(**kw):
    d = dict(batch=2, seqlen=16, d_model=64, d_inner=128, d_state=16, d_conv=4, dt_rank=4, io_dtype=ss.SS_F32,
             discretization=ss.SS_EULER, norm_eps=1e-5)
    d.update(kw)
    return ss.ss_block_dims(*d.values())


def bcall(dims=None, step=False, ws=WS, ws_bytes=None, weights=True, **kw):
    dims = dims or bdims()
    w = {n: BASE + k * GAP for k, n in enumerate(WEIGHTS)}
    o = dict(S_in=BASE + 20 * GAP, S_out=BASE + 21 * GAP, x=BASE + 22 * GAP, out=BASE + 23 * GAP, h=BASE + 24 * GAP, c=BASE + 25 * GAP)
    for k, v in kw.items():
        (w if k in w else o)[k] = v
    q = ss.ss_block_q8_weights(ss.ss_block_weights(*w.values()), o["S_in"], o["S_out"])
    need = ss.ss_block_q8_workspace_bytes(dims, step) if ws_bytes is None else ws_bytes
    fn = ss.lib.ss_block_q8_step if step else ss.lib.ss_block_q8_fwd
    return fn(ctypes.byref(dims), ctypes.byref(q) if weights else None, o["x"], o["out"], o["h"], o["c"], ws, need, None)


@pytest.mark.parametrize("step", [False, True])
def test_block_refusals(step):
    for kw, status in [(dict(batch=0), 1), (dict(d_model=0), 1), (dict(d_inner=0), 1), (dict(dt_rank=0), 1), (dict(d_model=72), 2),
                       (dict(d_inner=136), 2), (dict(d_state=12), 2), (dict(d_conv=3), 2), (dict(io_dtype=2), 2), (dict(norm_eps=0.0), 1),
                       (dict(norm_eps=float("nan")), 1), (dict(discretization=7), None), (dict(dt_rank=5000), 1),
                       (dict(d_inner=1 << 24), 1), (dict(d_model=1 << 21), 1), (dict(batch=1 << 31), 1)]:
        got = bcall(bdims(**kw), step, ws_bytes=1 << 40)
        assert got == status if status else got != 0, kw
        assert ss.ss_block_q8_workspace_bytes(bdims(**kw), step) == 0, kw
    assert bcall(step=step, weights=False) == 1
    for n in ("norm_w", "W_in", "conv_w", "W_x", "W_dt", "A", "W_out", "S_in", "S_out", "x", "out"):
        assert bcall(step=step, **{n: None}) == 1 and n in last(), n
    for n, at in [("W_in", 8), ("W_x", 8), ("W_dt", 8), ("W_out", 8), ("S_in", 2), ("S_out", 2), ("norm_w", 2), ("conv_w", 2), ("A", 2),
                  ("x", 8), ("out", 8), ("h", 8), ("c", 2), ("conv_b", 2), ("dt_bias", 2), ("Dskip", 2)]:
        assert bcall(step=step, **{n: BASE + 30 * GAP + at}) == 1 and "aligned" in last(), n
    for a, b in [("out", "x"), ("out", "W_in"), ("out", "S_out"), ("h", "x"), ("h", "out"), ("c", "h"), ("c", "A"), ("h", "conv_b")]:
        at = {n: BASE + k * GAP for k, n in enumerate(WEIGHTS)}
        at.update(S_in=BASE + 20 * GAP, S_out=BASE + 21 * GAP, x=BASE + 22 * GAP, out=BASE + 23 * GAP, h=BASE + 24 * GAP)
        assert bcall(step=step, **{a: at[b] - 16}) == 1 and "overlaps" in last(), (a, b)
    need = ss.ss_block_q8_workspace_bytes(bdims(), step)
    assert bcall(step=step, ws_bytes=need - 1) == 3 and bcall(step=step, ws=None) == 3
    assert bcall(step=step, ws=WS + 128) == 1
    assert bcall(step=step, ws=BASE + 22 * GAP) == 1 and "workspace overlaps x" in last()


def test_block_step_needs_states_and_workspace_holds_everything():
    assert bcall(step=True, h=None) == 1 and bcall(step=True, c=None) == 1
    a = lambda v: (v + 255) // 256 * 256  # noqa: E731
    M, dm, di, R, N = 32, 64, 128, 4, 16
    want = a(M * dm) + a(M * 4) + 5 * a(M * di * 4) + a(M * R * 4) + 2 * a(M * N * 4) + a(M * di) + a(M * 4)
    assert ss.ss_block_q8_workspace_bytes(bdims()) == want
    assert ss.ss_block_q8_workspace_bytes(bdims(seqlen=0)) == 0 and ss.ss_block_q8_workspace_bytes(bdims(seqlen=0), True) > 0


def test_block_binding_refuses_host_operands():
    with pytest.raises(ValueError):
        ss.ss_block_q8_fwd(torch.zeros(1, 2, 32), {}, 2)
    with pytest.raises(ValueError):
        ss.block_q8_weights({"W_in": torch.zeros(64, 32), "W_out": torch.zeros(32, 32)})


def test_more_lanes_than_one_launch_holds_are_refused():
    wide = ss.ss_view(BASE, 128, 128)
    views = dict(x=wide, r=ss.ss_view(BASE + 1 * GAP, 0, 0), i=ss.ss_view(BASE + 2 * GAP, 0, 0))
    for which, batch in (("fwd", 1 << 22), ("bwd", 1 << 22), ("step", 1 << 26)):
        assert gcall(which, gdims(batch=batch, seqlen=1, d=2), gargs(**views)) == 1 and "too large" in last(), which
    assert ss.ss_glr_workspace_bytes(gdims(batch=1 << 22, seqlen=1, d=2)) == 0
    assert ss.lib.ss_quant_q8(ctypes.byref(qdims(rows=1, cols=1 << 29, square=1)), BASE, BASE + 64 * GAP, BASE + 99 * GAP, None) == 1
    assert bcall(bdims(batch=65535, seqlen=65), ws_bytes=1 << 60) == 1 and "too large" in last()
