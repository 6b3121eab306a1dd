"""CPU: sizes that the delta rule's and the norms' C ABI gives, where a wrong one is a race or ends the process."""
import subprocess
import sys

import pytest

import selective_state_space_73_amd as ss


def rdims(**kw):
    d = dict(batch=1, seqlen=64 * 9, k_heads=1, heads=1, dk=64, dv=64, io_dtype=ss.SS_BF16, scale=0.125, eps=1e-6, reserved=0)
    d.update(kw)
    return ss.ss_gdr_dims(*d.values())


def test_segments_have_a_state_in_front_of_every_one():
    """Nine chunks of one head run as segments of 4, 4 and 1. All of them start from the workspace, the first one too: the last
    segment overwrites the caller's state in the same launch. What depends on dv has room for these states at least."""
    for io in (ss.SS_BF16, ss.SS_F32):
        more = ss.ss_gdr_workspace_bytes(rdims(dv=128, io_dtype=io)) - ss.ss_gdr_workspace_bytes(rdims(io_dtype=io))
        assert more >= 3 * 64 * 64 * 4


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(batch=8, heads=40, dk=128, dv=128), dict(batch=4, heads=64, k_heads=2, dv=512)])
def test_no_tokens_need_no_workspace(kw, backward):
    """Whatever the number of heads (in a process of its own: a division by zero ends it)."""
    code = f"import sys; sys.path[:0] = {sys.path!r}; import test_layer_rules as t; " \
           f"print(t.ss.ss_gdr_workspace_bytes(t.rdims(**{dict(kw, seqlen=0)!r}), {backward}))"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["0"], r.stderr[-500:]


@pytest.mark.parametrize("io,forward,backward", [(ss.SS_BF16, 3 * 10 * 256 * 2, 3 * 6 * 512 * 2), (ss.SS_F32, 10 * 256 * 4, 6 * 512 * 4)])
def test_a_chunk_takes_what_it_uses(io, forward, backward):
    """Ten rows of 64 factors, and the inverse: a lower triangle in tiles of 16 x 16, in the backward an upper one in blocks of
    16 x 32, as three bf16 terms or in fp32. (300 heads are one segment.)"""
    def more(back):
        a, b = (ss.ss_gdr_workspace_bytes(rdims(heads=300, k_heads=300, seqlen=64 * n, io_dtype=io, dk=1, dv=1), back) for n in (9, 8))
        return a - b
    assert more(False) == 300 * (2560 + forward)
    # the state's gradient and the flags of a chunk, the gradients of its values
    assert abs(more(True) - 300 * (2560 + backward + 4 + 16 + 64 * 4)) < 1024
