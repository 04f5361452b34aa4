"""The products where the plan of a result is more than one kind of tile: tiles done in
one piece, the others in pieces along the sum, which a second kernel adds up and finishes.
Results on any boundary, and longest rows of the third type.

Tolerances are test_gpu_block.py's."""
import ctypes as C

import numpy as np
import pytest

import block_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import block, mv  # noqa: E402
from test_gpu_block import BF16, F16, F32, U, check_norm, close, host, norm_inputs, product_slack, randn  # noqa: E402

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


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,cols,rows,wide", MIXED)
def test_whole_tiles_and_pieces_against_64_bits(tokens, cols, rows, wide, dtype):
    """All columns of rows of every tile of rows, the first and the last among them."""
    out = F32 if wide else dtype
    x, w = randn((tokens, cols), 1, dtype), randn((rows, cols), 2, dtype, cols ** -0.5)
    bias, residual = randn((rows,), 3, F32), randn((tokens, rows), 4, out)
    some = sorted({0, 127, 128, tokens - 1, *range(5, tokens, 131)})
    for act, scale, res, keep in (("gelu", 0.5, residual, True), ("silu", 1.0, None, False), ("gelu_tanh", -2.0, residual, False)):
        got = block.linear(x, w, bias, act=act, residual=res, scale=scale, out_dtype=out, keep=keep)
        y, z = got if keep else (got, None)
        want, wz, m = R.linear(host(x[some]), host(w), host(bias), act, None if res is None else host(res[some]), scale)
        slack = product_slack(m, cols, out)
        close(act, y[some], want, abs(scale) * (1.13 * slack + 2.0 ** -20 * np.maximum(np.abs(wz), 1.0)) + 2 * U * np.abs(want))
        if keep:
            close("z", z[some], wz, slack)


@pytest.mark.parametrize("tokens,cols,rows,grad", [(2048, 5120, 2560, BF16), (1901, 2403, 2603, F32), (2048, 5120, 2560, F32)])
def test_gradients_of_whole_tiles_and_pieces_against_64_bits(tokens, cols, rows, grad):
    dz, x, w = randn((tokens, rows), 1, grad, rows ** -0.5), randn((tokens, cols), 2, BF16), randn((rows, cols), 3, BF16, cols ** -0.5)
    dx, dw, _ = block.linear_backward(dz, x, w)
    parts, k2 = (2.0 ** -17, 2) if grad == F32 else (0.0, 1)
    some = sorted({0, 127, 128, tokens - 1, *range(5, tokens, 131)})
    a, b = host(dz[some]), host(w)
    m = np.abs(a) @ np.abs(b)
    close("dx", dx[some], a @ b, product_slack(m, k2 * rows, BF16) + parts * m)
    some = sorted({0, 127, 128, rows - 1, *range(5, rows, 131)})
    a, b = host(dz[:, some]).T, host(x)
    m = np.abs(a) @ np.abs(b)
    close("dw", dw[some], a @ b, product_slack(m, k2 * tokens, BF16) + parts * m)


@pytest.mark.parametrize("tokens,cols,rows", [(256, 7168, 256), (1901, 2403, 2603), (3, 20480, 512)])
def test_errors_of_32_bit_results_by_their_norm(tokens, cols, rows):
    """Terms of random signs, whose sum is some sqrt(cols) times smaller than its terms'
    magnitudes.  The 32 steps of a run of 512 cut at most 4 U of the sum so far off each, and
    a run's sum so far is no larger, by its norm, than the run's: 128 U of the result's norm, and 16 U after."""
    x, w = randn((tokens, cols), 1, BF16), randn((rows, cols), 2, BF16, cols ** -0.5)
    y = block.linear(x, w, out_dtype=F32)
    want = x.double() @ w.double().t()
    assert (y.double() - want).norm() <= 144 * U * want.norm()


def guarded(shape, dtype, off):
    """A result between guards, ``off`` elements beyond a 16-byte boundary."""
    n = int(np.prod(shape))
    whole = torch.empty(n + 128 + off, device="cuda", dtype=dtype)
    bits = whole.view(torch.int32 if dtype == F32 else torch.int16)
    bits.fill_(0x5A5A)

    def untouched():
        return bool((bits[:64 + off] == 0x5A5A).all() and (bits[64 + off + n:] == 0x5A5A).all())
    return whole[64 + off:64 + off + n].view(shape), untouched


@pytest.mark.parametrize("tokens,cols,rows", [(1, 70, 33), (5, 64, 48), (130, 96, 264), (300, 77, 129), (700, 6000, 1000)])
@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_results_anywhere_and_nothing_beside_them(tokens, cols, rows, off):
    """The C entries take results on any element's boundary: the same as on a 16-byte one."""
    lib, stream = block._library(), torch.cuda.current_stream().cuda_stream
    x, w, dz = randn((tokens, cols), 1, BF16), randn((rows, cols), 2, BF16, cols ** -0.5), randn((tokens, rows), 3, BF16)
    bias = randn((rows,), 4, F32)

    def call(name, pack, args):
        d, need = pack(*args), C.c_uint64()
        assert getattr(lib, name + "_workspace_bytes")(d, C.byref(need)) == mv.MV_OK
        ws = torch.full((need.value + 256,), 255, device="cuda", dtype=torch.uint8)
        assert getattr(lib, name)(d, ws.data_ptr(), need.value, stream) == mv.MV_OK
        assert (ws[need.value:] == 255).all()

    for out in (BF16, F32):
        want = block.linear(x, w, bias, act="silu", keep=True, out_dtype=out)
        (y, yg), (z, zg) = guarded((tokens, rows), out, off), guarded((tokens, rows), BF16, off)
        call("mv_linear", block._linear_desc, (tokens, cols, rows, cols, cols, rows, 2, 0 if out == F32 else 2, 0, 4, 1.0, x.data_ptr(),
                                               w.data_ptr(), bias.data_ptr(), 0, y.data_ptr(), z.data_ptr()))
        assert yg() and zg() and torch.equal(z, want[1])
        # sums are made alike; a row's end may be finished by other instructions for the activation
        assert ((y.double() - want[0].double()).abs() <= 2.0 ** -7 * want[0].double().abs() + 2.0 ** -18).all()
    want = block.linear_backward(dz, x, w, bias=True)
    outs = [guarded(s, BF16, off) for s in ((tokens, cols), (rows, cols), (rows,))]
    call("mv_linear_backward", block._linear_grad_desc, (tokens, cols, rows, cols, cols, rows, 2, 2, dz.data_ptr(), x.data_ptr(),
                                                         w.data_ptr(), *(t.data_ptr() for t, _ in outs)))
    for (got, guard), t in zip(outs, want):
        assert guard() and torch.equal(got, t)


@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_norms_results_anywhere_and_nothing_beside_them(dtype, off):
    lib, stream = block._library(), torch.cuda.current_stream().cuda_stream
    code = {F32: 0, F16: 1, BF16: 2}[dtype]
    for tokens, hidden in ((1, 8), (7, 100), (66, 1437), (9, 5120)):
        y, res, dn = (randn((tokens, hidden), i, dtype) for i in range(3))
        w, post, gate = (randn((hidden,), i, F32, 0.2, 1.0) for i in range(3, 6))
        want, grads = block.norm(y, w, residual=res, post=post, gate=gate), block.norm_backward(dn, y, w, residual=res, post=post, gate=gate)
        d = block._norm_desc(tokens, hidden, 1, hidden, hidden, code, 0, 0, 1.0, 1e-6, y.data_ptr(), res.data_ptr(), w.data_ptr(), 0,
                             post.data_ptr(), 0, gate.data_ptr())
        outs = [guarded((tokens, hidden), dtype, off) for _ in range(2)]
        assert lib.mv_norm(d, *(t.data_ptr() for t, _ in outs), stream) == mv.MV_OK
        back = [guarded((tokens, hidden), dtype, off) for _ in range(2)] + [guarded((hidden,), F32, off) for _ in range(3)]
        (dy, dres, dw, dpost, dgate) = (t.data_ptr() for t, _ in back)
        e = block._norm_grad_desc(hidden, hidden, dn.data_ptr(), 0, dy, dres, dw, 0, dpost, 0, dgate)
        need = C.c_uint64()
        assert lib.mv_norm_backward_workspace_bytes(d, e, C.byref(need)) == mv.MV_OK
        ws = torch.full((need.value + 256,), 255, device="cuda", dtype=torch.uint8)
        assert lib.mv_norm_backward(d, e, ws.data_ptr(), need.value, stream) == mv.MV_OK
        assert (ws[need.value:] == 255).all() and all(g() for _, g in outs + back)
        wants = [*want, grads.dy, grads.dresidual, grads.dweight, grads.dpost, grads.dgate]
        for (got, _), t in zip(outs + back, wants):          # other threads may hold a row: its sums in another order
            eps = torch.finfo(t.dtype).eps
            assert ((got.double() - t.double()).abs() <= eps * t.double().abs() + 2.0 ** -18 * t.double().abs().max()).all()


@pytest.mark.parametrize("hidden", [9000, 12288, 16383, 16384])
def test_norm_longest_rows_of_float16(hidden):
    check_norm(norm_inputs(5, hidden, F16, "layer", F16, True, True, 5, True), "layer", 0.5)
    check_norm(norm_inputs(6, hidden, F16, "rms", F32, True, True, 2, False), "rms")
