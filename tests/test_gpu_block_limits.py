"""The block operators at the ends of what their documentation says."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import block  # noqa: E402
from test_gpu_block import BF16, F32, check_norm, norm_inputs, randn  # noqa: E402


def test_gave_up_waits_for_every_stream():
    """A stream of torch's does not wait for the default one, nor that for it."""
    x, w = randn((8192, 5120), 1, BF16), randn((5120, 5120), 2, BF16)
    block.linear(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):                                 # some 50 ms
            block.linear(x, w)
        end = torch.cuda.Event()
        end.record()
    assert not end.query()
    assert block.gave_up() == 0
    assert end.query()


def signs(shape, seed, size, dtype):
    return torch.where(randn(shape, seed) < 0, -size, size).to(dtype)


@pytest.mark.parametrize("hidden", [256, 1000, 1437, 7168, 16384])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_the_largest_magnitudes(hidden, dtype):
    """Magnitudes of up to 1e18, whatever the width."""
    for size in (1e17, 0.98e18):
        for kind, post in (("rms", False), ("rms", True), ("layer", False), ("layer", True)):
            a = norm_inputs(6, hidden, dtype, kind, F32, not post, post, 2, kind == "layer")
            a["y"] = signs((6, hidden), 7, size if post else size / 4, dtype)
            if not post:
                a["residual"], a["gate"] = signs((6, hidden), 8, size / 2, dtype), a["gate"].clamp(0.25, 1.0)
            check_norm(a, kind)


def test_norm_of_small_magnitudes():
    """Down to 1e-16 with no eps at all."""
    for hidden in (256, 1437, 16384):
        for kind in ("rms", "layer"):
            check_norm(norm_inputs(6, hidden, F32, kind, F32, False, False, 0, False, std=1e-15), kind, eps=0.0)
            a = norm_inputs(6, hidden, F32, kind, F32, False, False, 0, False)
            a["y"] = signs((6, hidden), 9, 1e-16, F32)
            check_norm(a, kind, eps=0.0)
