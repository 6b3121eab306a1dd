"""The compiler's resource report of the operators' kernels (kept by build.py): which of them keep
registers in scratch memory. CPU only: reads the report, runs nothing."""
import os
import subprocess

import pytest

from selective_state_space_73_amd import build as B

# (kernel, VGPRs spilled at most): the recurrence's forward with an odd number of bf16 channels,
# two loads a row and lane; its fp32 backward in runs of 16, at the limit of two waves a SIMD
SPILLS = {"k_glr_scan<unsigned short, false, 16, 16>": 14, "k_glr_scan<unsigned short, false, 16, 8>": 14,
          "k_glr_bwd<float, true, 16, 8, true>": 2, "k_glr_bwd<float, false, 16, 8, true>": 2,
          "k_glr_bwd<float, false, 16, 4, true>": 2}


@pytest.fixture(scope="module")
def report():
    if not os.path.exists(B.RESOURCES):
        pytest.skip("no build report (build() has not run in this tree)")
    raw = B.kernel_resources()
    names = subprocess.run(["c++filt"], input="\n".join(raw), capture_output=True, text=True, check=True).stdout.splitlines()
    return dict(zip((n.replace("void ", "").replace("selscan::", "").split("(")[0] for n in names), raw.values()))


def test_report_covers_the_operators(report):
    for k in ("k_glr_fwd<", "k_glr_scan<", "k_glr_bwd<", "k_glr_step<", "k_glr_da", "k_q8_rows<", "k_q8_square<", "k_gemm_q8<",
              "k_gemm_q8_split<"):
        assert any(n.startswith(k) for n in report), k


def test_only_the_named_kernels_spill(report):
    for n, v in report.items():
        if n.startswith(("k_glr", "k_q8", "k_gemm_q8")):
            assert v.get("vgpr_spill", 0) <= SPILLS.get(n, 0), n
            assert n in SPILLS or v.get("scratch", 0) == 0, n
