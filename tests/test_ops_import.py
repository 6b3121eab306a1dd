"""CPU: the scan and the blocks need libselscan.so alone. The package imports without the operators'
extension, and on a torch without a GPU's functions; the extension's calls say what is missing."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT_EXTENSION = """
import sys
sys.modules["selective_state_space_73_amd._binding"] = None
import torch
import selective_state_space_73_amd as ss
assert ss.ss_version() >= 1
dims = ss.make_dims(1, 64, 32, 16, ss.SS_F32)
assert ss.ss_workspace_bytes(dims) >= 0 and ss.ss_glr_workspace_bytes(ss.ss_glr_dims(1, 200, 64, ss.SS_F32, 0)) > 0
t = torch.zeros(1, 4, 8)
for _ in range(2):
    for call in (lambda: ss.ss_quant_q8(t), lambda: ss.ss_glr_fwd(t, t, t, t[0, 0]), lambda: ss.ss_norm_q8(t, t[0, 0]),
                 lambda: ss.ss_glr_step(t[0], t[0], t[0], t[0, 0], t[0]), lambda: ss.ss_gemm_q8(t, t, t, t),
                 lambda: ss.ss_glr_bwd(t, t, t, t[0, 0], t, t)):
        try:
            call()
        except ImportError as e:
            assert "_binding.so" in str(e)
        else:
            raise AssertionError("no refusal")
print("fine")
"""
WITHOUT_GPU_FUNCTIONS = """
import torch
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
import selective_state_space_73_amd as ss
assert ss.ss_version() >= 1
print("fine")
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]


def test_package_without_the_extension():
    run(WITHOUT_EXTENSION)


def test_package_on_a_torch_without_gpu_functions():
    run(WITHOUT_GPU_FUNCTIONS)
