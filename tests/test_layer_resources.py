"""The compiler's resource report of the delta rule's and the norms' kernels (kept by build.py): which of them keep
registers in scratch memory. CPU only: reads the report, runs nothing."""
import os
import subprocess

import pytest

from selective_state_space_73_amd import build as B

# (kernel, VGPRs spilled at most). The walks over rows of keys that are not aligned hold an eight of a row in
# registers on its way to LDS; the gradients hold 120 sums and the terms of a state at two workgroups a CU; the
# join's 256 rows of a state are 256 registers by themselves. The norms' gradients in rows of more than 4096
# columns (1024 lanes, 128 registers each) keep the sums over rows of up to sixteen columns a lane.
_BF16, _F32 = "unsigned short", "float"
SPILLS = {f"k_gdr_walk<{_BF16}, 64, true, false, 2>": 43, f"k_gdr_walk<{_BF16}, 128, true, false, 2>": 64,
          f"k_gdr_grads<{_BF16}, 128, true, true, 2>": 2, f"k_gdr_grads<{_BF16}, 128, true, false, 2>": 18,
          f"k_gdr_grads<{_BF16}, 128, false, false, 2>": 9, f"k_gdr_grads<{_F32}, 128, true, true, 2>": 22,
          f"k_gdr_grads<{_F32}, 128, true, false, 2>": 27, f"k_gdr_grads<{_F32}, 128, false, false, 2>": 103,
          f"k_gdr_grads<{_F32}, 256, false, false, 1>": 5, f"k_gdr_join<{_BF16}, 256>": 339, f"k_gdr_join<{_F32}, 256>": 347}
SPILLS.update({f"k_gnorm_bwd<{t}, {vec}, 0, {nv}, {grouped}, 1024, false, 4>": most
               for t, vec, nv, grouped, most in (
                   (_BF16, "true", 1, "true", 10), (_BF16, "false", 1, "true", 18), (_BF16, "false", 1, "false", 16),
                   (_F32, "true", 1, "true", 14), (_F32, "true", 1, "false", 5), (_F32, "false", 1, "true", 18),
                   (_F32, "false", 1, "false", 21), (_BF16, "true", 2, "true", 160), (_BF16, "true", 2, "false", 152),
                   (_BF16, "false", 2, "true", 309), (_BF16, "false", 2, "false", 275), (_F32, "true", 2, "true", 181),
                   (_F32, "true", 2, "false", 170), (_F32, "false", 2, "true", 248), (_F32, "false", 2, "false", 205))})


@pytest.fixture(scope="module")
def report():
    if not os.path.exists(B.RESOURCES):
        pytest.skip("no build report (build() has not run in this tree)")
    raw = B.kernel_resources()
    names = subprocess.run(["c++filt"], input="\n".join(raw), capture_output=True, text=True, check=True).stdout.splitlines()
    return dict(zip((n.replace("void ", "").replace("selscan::", "").split("(")[0] for n in names), raw.values()))


def test_report_covers_the_operators(report):
    for k in ("k_gdr_solve<", "k_gdr_walk<", "k_gdr_ends<", "k_gdr_join<", "k_gdr_walk_back<", "k_gdr_grads<", "k_gdr_keys<", "k_gdr_step<",
              "k_gnorm_fwd<", "k_gnorm_bwd<", "k_gnorm_sum"):
        assert any(n.startswith(k) for n in report), k


def test_only_the_named_kernels_spill(report):
    for n, v in report.items():
        if n.startswith(("k_gdr", "k_gnorm")):
            assert v.get("vgpr_spill", 0) <= SPILLS.get(n, 0), n
            assert n in SPILLS or v.get("scratch", 0) == 0, n
