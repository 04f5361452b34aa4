"""The block operators at the ends of what their documentation says."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import block  # noqa: E402
from test_gpu_block import BF16, F32, check_norm, close, host, norm_inputs, randn  # noqa: E402


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


def test_32_bit_gradients_of_products_at_any_magnitude():
    """A 32-bit dz is two bfloat16: 2^-17 of the value, or half of bfloat16's smallest
    step, 2^-134, where that is more.  Seen in what is left of a value without its nearest bfloat16."""
    scale = 2.0 ** 100
    v = torch.tensor([s * 10.0 ** e for e in (-26.3, -30.1, -34.2, -35.4, -36.1, -37.0, -37.4, -38.2, -39.1, -40.3)
                      for s in (1.0, -1.2345678, 1.0 + 2.0 ** -9 + 2.0 ** -20)], dtype=torch.float64).float().cuda()
    dz = torch.zeros((len(v), 8), device="cuda")
    dz[:, 0], dz[:, 1] = v, -v.bfloat16().float()
    w = torch.zeros((8, 16), device="cuda", dtype=BF16)
    w[:2] = scale
    dx = block.linear_backward(dz, torch.zeros((len(v), 16), device="cuda", dtype=BF16), w, dw=False)[0]
    d = host(dz)
    want = np.repeat((d[:, :1] + d[:, 1:2]) * scale, 16, 1)
    slack = np.maximum(2.0 ** -17 * np.abs(d[:, :1]), 2.0 ** -134) * scale
    close("dx", dx, want, np.repeat(slack, 16, 1))


def test_32_bit_gradients_times_an_infinity():
    """No number comes of it, and only where the infinity is."""
    dz, x, w = randn((9, 24), 1, F32), randn((9, 40), 2, BF16), randn((24, 40), 3, BF16)
    dz[4, 7] = 1.0                                           # exactly a bfloat16: its second part is 0
    clean = block.linear_backward(dz, x, w)
    w2, x2 = w.clone(), x.clone()
    w2[7, 5] = float("inf")
    x2[4, 6] = float("inf")
    dx, dw, _ = block.linear_backward(dz, x2, w2)
    assert not dx[:, 5].isfinite().any() and not dw[:, 6].isfinite().any()
    others = [i for i in range(40) if i not in (5, 6)]
    assert torch.equal(dx[:, others], clean[0][:, others]) and torch.equal(dw[:, others], clean[1][:, others])
    assert torch.equal(dx[:, 6], clean[0][:, 6]) and torch.equal(dw[:, 5], clean[1][:, 5])
