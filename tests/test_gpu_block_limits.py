"""The block operators at the ends of what their documentation says."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import block  # noqa: E402
from test_gpu_block import BF16, randn  # noqa: E402


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
