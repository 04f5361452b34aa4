"""The products where the plan of a result is more than one kind of tile: tiles done in
one piece, the others in pieces along the sum, which a second kernel adds up and finishes.

Tolerances are test_gpu_block.py's."""
import ctypes as C

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import block, mv  # noqa: E402
from test_gpu_block import BF16, F32, randn  # noqa: E402

# tokens, cols, rows, whether the result has 32 bits: on 152 SMs each is done partly in one piece
MIXED = [(2048, 5120, 5120, False), (2048, 5120, 5120, True), (3000, 4096, 4096, True), (1901, 2403, 5203, False),
         (1901, 2403, 2603, True), (700, 6000, 7777, False)]


def in_pieces(tokens, cols, rows, wide, dtype=2):
    """Bytes of the pieces' sums, by an aligned call's workspace."""
    d = block.LinearDesc(tokens=tokens, cols=cols, rows=rows, x_stride=-(-cols // 8) * 8, w_stride=-(-cols // 8) * 8,
                         residual_stride=rows, dtype=dtype, out_dtype=0 if wide else dtype, bias_dtype=dtype, scale=1.0,
                         x=0x10000, w=0x10000, y=0x10000)
    need = C.c_uint64()
    assert block._library().mv_linear_workspace_bytes(C.byref(d), C.byref(need)) == mv.MV_OK
    return need.value


@pytest.mark.parametrize("tokens,cols,rows,wide", MIXED)
def test_equal_rows_give_equal_rows_in_every_tile(tokens, cols, rows, wide):
    x, w = randn((1, cols), 1, BF16), randn((rows, cols), 2, BF16, cols ** -0.5)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert 0 < in_pieces(tokens, cols, rows, wide) < 4 * tokens * rows
    many = randn((tokens, cols), 3, BF16)
    many[::3] = x
    bias = randn((rows,), 4, F32, 0.1)
    for act in ("none", "gelu", "gelu_tanh", "silu"):
        y, z = block.linear(many, w, bias, act=act, scale=0.5, keep=True, out_dtype=F32 if wide else None)
        assert (z[::3] == z[0]).all(), (act, (z[::3] != z[0]).sum().item())
        assert (y[::3] == y[0]).all(), (act, (y[::3] != y[0]).sum().item())
