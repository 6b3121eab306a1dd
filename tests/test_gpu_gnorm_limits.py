"""GPU: the norms around a layer at the edges of what their calls allow, against their 64-bit definition. Inputs, tolerances and
comparisons as in test_gpu_gnorm.py."""
import math

import pytest
import torch

from oracle import ops as O

pytestmark = pytest.mark.gpu

ss = pytest.importorskip("selective_state_space_73_amd")
T = pytest.importorskip("test_gpu_gnorm")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 8192, 1), (2, 8150, 1), (3, 8145, 1), (3, 8144, 1), (2, 7681, 1), (2, 8192, 2), (2, 8190, 3), (2, 16384, 1)])
def test_groups_of_a_few_columns_in_wide_rows(shape, io):
    """A group of one column is normed by itself: y / sqrt(y^2 + eps), which is +-1 but for eps, and whose gradient all
    but cancels; the tolerance is relative to the terms that do.

    The bound of dscale has the terms of the gradient of s in it. dscale_c = sum over rows of g h with g = ds + r (t - s m), t = dn w_next,
    r = 1 / rms(s), m = mean(t s) r^2; in fp32 g is off by some roundings of each of its three terms, |ds| + r |t| + r |s m|, however
    far they cancel, and of the M = 2 or 3 products of a column none need be large where g is small in one of them. For one column
    of 16384 in two rows that does happen: |g| is up to a thousand times less than its terms there."""
    x, ds, dn = T.make(*shape, io, T.ALL, seed=sum(shape))
    M, K = x["y"].shape
    s, n = ss.ss_gnorm_fwd(**x)
    sw, nw = O.gnorm_fwd(**x)
    res, half = x["residual"].double().cpu().abs(), T.HALF[io]
    T.near(s, sw, T.rel(K) * (sw.abs() + 2 * res) + half * sw.abs())
    T.near(n, nw, T.rel(K) * (nw.abs() + 2 * nw.abs() * (res + sw.abs()) / sw.abs().clamp_min(1e-9)) + half * nw.abs())
    got, want = ss.ss_gnorm_bwd(ds=ds, dn=dn, **x), O.gnorm_bwd(ds=ds, dn=dn, **x)
    r = 1 / torch.sqrt((sw * sw).mean(-1, keepdim=True) + 1e-5)
    t = dn.double().cpu() * x["w_next"].double().cpu()
    terms = ds.double().cpu().abs() + r * t.abs() + r ** 3 * sw.abs() * (t * sw).mean(-1, keepdim=True).abs()
    h = (sw - x["residual"].double().cpu()) / x["scale"].double().cpu()
    for k, v in got.items():
        print(k, end=" ")
        val, size = want[k]
        sums = k in ("dw", "dscale", "dw_next")
        if k == "dscale":
            size = (terms * h.abs()).sum(0)
        tol = 2.0 ** -24 * (4 * (24 + math.log2(K) + 1) + (math.ceil(M / 256) if sums else 0))
        T.near(v, val, 4 * tol * size + (2.0 ** -24 if sums else half) * val.abs())


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("K,group", [(64, 64), (640, 128), (2560, 2560), (9000, 9000)])
def test_gates_far_out_keep_their_digits(K, group, sign):
    """Gates from 6 to 85, either way: e^-z is as near as near 0, whatever its size, so that silu and its slope are within what a
    sigmoid is allowed near 0 (4 roundings, and as many products), relative to themselves. The slope is sig (1 + z (1 - sig)), whose two
    terms are up to 1 + |z| times sig and do not cancel for |z| >= 6."""
    u = 2.0 ** -24
    x, ds, _ = T.make(5, K, group, "f32", ("gate",), seed=K)
    x["gate"] = (sign * torch.linspace(6, 85, 5 * K).view(5, K)).cuda()
    s, _ = ss.ss_gnorm_fwd(**x)
    sw, _ = O.gnorm_fwd(**x)
    T.near(s, sw, (T.rel(K) + 8 * u) * sw.abs())
    got, want = ss.ss_gnorm_bwd(ds=ds, **x)["dgate"], O.gnorm_bwd(ds=ds, **x)["dgate"][0]
    T.near(got, want, (T.rel(K) + 12 * u) * want.abs())
