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
