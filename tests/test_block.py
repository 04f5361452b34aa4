"""The block operators without a GPU: what the C entry points refuse (all checked
on the host before anything is launched), the Python binding's refusal of host
tensors and of malformed arguments, and the plain 64-bit code against differences."""
import ctypes as C

import numpy as np
import pytest
import torch

import block_reference as R
from experiment_network_simulation_gb300 import block, mv

P = 0x10000          # an aligned address that is only looked at
BIG = 1 << 62        # a workspace of any size


def _calls(cls, base, *rest):
    def d(**kw):
        return C.byref(cls(**{**base, **kw}))
    return d


LINEAR = dict(tokens=4, cols=64, rows=32, x_stride=64, w_stride=64, residual_stride=32, dtype=2, out_dtype=2,
              bias_dtype=2, act=0, scale=1.0, x=P, w=P, bias=None, residual=None, y=P, z=None)


def test_linear_refuses():
    lib = block._library()
    d = _calls(block.LinearDesc, LINEAR)
    need = C.c_uint64(0)
    size = lambda **kw: lib.mv_linear_workspace_bytes(d(**kw), C.byref(need))  # noqa: E731
    assert lib.mv_linear_workspace_bytes(d(), None) == mv.MV_EINVAL
    assert lib.mv_linear_workspace_bytes(None, C.byref(need)) == mv.MV_EINVAL
    for kw in (dict(cols=0), dict(rows=0), dict(dtype=0), dict(dtype=3), dict(out_dtype=1), dict(out_dtype=3),
               dict(bias_dtype=1), dict(act=5), dict(scale=float("inf")), dict(scale=float("nan")), dict(x_stride=63),
               dict(w_stride=63), dict(residual=P, residual_stride=31)):
        assert size(**kw) == mv.MV_EINVAL and need.value == 0, kw
        assert lib.mv_linear(d(**kw), P, BIG, None) == mv.MV_EINVAL, kw
    for kw in (dict(tokens=(1 << 30) + 1), dict(cols=(1 << 30) + 1, x_stride=1 << 31, w_stride=1 << 31),
               dict(rows=(1 << 30) + 1), dict(x_stride=1 << 37), dict(w_stride=1 << 37),
               dict(residual=P, residual_stride=1 << 37), dict(tokens=1 << 30, rows=1 << 30)):
        assert size(**kw) == mv.MV_EOVERFLOW and need.value == 0, kw
    assert size(tokens=0) == mv.MV_OK and need.value == 0
    assert lib.mv_linear(d(tokens=0, x=None, w=None, y=None), None, 0, None) == mv.MV_OK
    run = lambda **kw: lib.mv_linear(d(**kw), P, BIG, None)  # noqa: E731
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=P + 1), dict(w=P + 1), dict(y=P + 1), dict(z=P + 1),
               dict(bias=P + 1), dict(bias=P + 2, bias_dtype=0), dict(residual=P + 1), dict(out_dtype=0, y=P + 2)):
        assert run(**kw) == mv.MV_EINVAL, kw
    # operands on no 16-byte boundary are copied: they need room
    assert size() == mv.MV_OK and need.value == 0
    assert size(x=P + 2) == mv.MV_OK and need.value >= 4 * 64 * 2
    assert lib.mv_linear(d(x=P + 2), None, 0, None) == mv.MV_ENOMEM
    assert lib.mv_linear(d(x=P + 2), P, need.value - 1, None) == mv.MV_ENOMEM
    assert lib.mv_linear(d(x=P + 2), None, need.value, None) == mv.MV_EINVAL
    assert lib.mv_linear(d(x=P + 2), P + 16, need.value, None) == mv.MV_EINVAL


def test_linear_backward_refuses():
    lib = block._library()
    base = dict(tokens=4, cols=64, rows=32, x_stride=64, w_stride=64, dz_stride=32, dtype=2, dz_dtype=2, dz=P, x=P,
                w=P, dx=P, dw=P, dbias=P)
    d = _calls(block.LinearGradDesc, base)
    need = C.c_uint64(0)
    size = lambda **kw: lib.mv_linear_backward_workspace_bytes(d(**kw), C.byref(need))  # noqa: E731
    run = lambda **kw: lib.mv_linear_backward(d(**kw), P, BIG, None)  # noqa: E731
    assert lib.mv_linear_backward_workspace_bytes(d(), None) == mv.MV_EINVAL
    assert lib.mv_linear_backward(None, P, BIG, None) == mv.MV_EINVAL
    for kw in (dict(cols=0), dict(rows=0), dict(dtype=0), dict(dtype=1, dz_dtype=0), dict(dz_dtype=1), dict(x_stride=63),
               dict(w_stride=63), dict(dz_stride=31)):
        assert size(**kw) == mv.MV_EINVAL and need.value == 0 and run(**kw) == mv.MV_EINVAL, kw
    for kw in (dict(tokens=(1 << 30) + 1), dict(rows=(1 << 30) + 1, dz_stride=1 << 31), dict(dz_stride=1 << 37),
               dict(rows=1 << 30, cols=1 << 30, x_stride=1 << 30, w_stride=1 << 30, dz_stride=1 << 30)):
        assert size(**kw) == mv.MV_EOVERFLOW, kw
    for kw in (dict(dz=None), dict(x=None), dict(w=None), dict(dz=P + 1), dict(dz_dtype=0, dz=P + 2), dict(dx=P + 1),
               dict(dw=P + 1), dict(dbias=P + 1)):
        assert run(**kw) == mv.MV_EINVAL, kw
    assert size(dz_dtype=0) == mv.MV_OK and need.value >= 2 * 4 * 32 * 2       # two parts of dz
    assert lib.mv_linear_backward(d(dz_dtype=0), P, need.value - 1, None) == mv.MV_ENOMEM


def test_activation_backward_refuses():
    f = block._library().mv_activation_backward
    base = dict(tokens=4, cols=64, dy_stride=64, z_stride=64, dtype=2, act=2, scale=1.0, dy=P, z=P, dz=P)
    d = _calls(block.ActGradDesc, base)
    assert f(None, None) == mv.MV_EINVAL
    assert f(d(tokens=0, dy=None, z=None, dz=None), None) == mv.MV_OK
    assert f(d(cols=0), None) == mv.MV_OK
    for kw in (dict(dtype=3), dict(act=5), dict(scale=float("nan")), dict(dy=None), dict(z=None), dict(dz=None),
               dict(dy_stride=63), dict(z_stride=63), dict(dy=P + 1), dict(dtype=0, z=P + 2)):
        assert f(d(**kw), None) == mv.MV_EINVAL, kw
    for kw in (dict(tokens=(1 << 31) + 1), dict(dy_stride=1 << 37), dict(z_stride=1 << 37)):
        assert f(d(**kw), None) == mv.MV_EOVERFLOW, kw


NORM = dict(tokens=4, hidden=64, gates=1, y_stride=64, residual_stride=64, dtype=2, param_dtype=0, kind=0, alpha=1.0,
            eps=1e-6, y=P, residual=P, weight=P, bias=None, post=P, post_bias=None, gate=P)


def test_norm_refuses():
    lib = block._library()
    d = _calls(block.NormDesc, NORM)
    run = lambda n=P, r=P, **kw: lib.mv_norm(d(**kw), n, r, None)  # noqa: E731
    assert lib.mv_norm(None, P, P, None) == mv.MV_EINVAL
    assert run(tokens=0, n=None, r=None, y=None, weight=None) == mv.MV_OK
    bad = (dict(hidden=0), dict(dtype=3), dict(param_dtype=1), dict(kind=2), dict(alpha=float("inf")), dict(eps=-1.0),
           dict(eps=float("nan")), dict(gates=0), dict(gates=3), dict(post=None, post_bias=P), dict(y=None),
           dict(weight=None), dict(y_stride=63), dict(residual_stride=63), dict(y=P + 1), dict(residual=P + 1),
           dict(weight=P + 2), dict(gate=P + 2), dict(post=P + 2))
    for kw in bad + (dict(n=None), dict(n=P + 1), dict(r=P + 1)):
        assert run(**kw) == mv.MV_EINVAL, kw
    over = (dict(hidden=16385, y_stride=16385, residual_stride=16385), dict(tokens=(1 << 31) + 1), dict(y_stride=(1 << 31) + 1))
    for kw in over:
        assert run(**kw) == mv.MV_EOVERFLOW, kw
    grads = dict(dn_stride=64, dr_stride=64, dn=P, dr=P, dy=P, dresidual=P, dweight=P, dbias=None, dpost=P, dpost_bias=None,
                 dgate=P)
    g = _calls(block.NormGradDesc, grads)
    need = C.c_uint64(0)
    back = lambda ws=P, n=BIG, g=g(), **kw: lib.mv_norm_backward(d(**kw), g, ws, n, None)  # noqa: E731
    for kw in bad:
        assert back(**kw) == mv.MV_EINVAL, kw
    for kw in over:
        assert back(**kw) == mv.MV_EOVERFLOW, kw
    for kw in (dict(dn=None), dict(dy=None), dict(dweight=None), dict(dresidual=None), dict(dpost=None), dict(dgate=None),
               dict(dbias=P), dict(dpost_bias=P), dict(dn_stride=63), dict(dr_stride=63), dict(dn=P + 1), dict(dy=P + 1),
               dict(dweight=P + 2), dict(dgate=P + 1)):
        assert back(g=g(**kw)) == mv.MV_EINVAL, kw
    assert back(g=g(dn_stride=(1 << 31) + 1)) == mv.MV_EOVERFLOW
    assert lib.mv_norm_backward_workspace_bytes(d(), g(), None) == mv.MV_EINVAL
    assert lib.mv_norm_backward_workspace_bytes(d(), g(), C.byref(need)) == mv.MV_OK and need.value
    assert back(n=need.value - 1) == mv.MV_ENOMEM
    assert back(ws=None) == mv.MV_EINVAL and back(ws=P + 16) == mv.MV_EINVAL


def test_python_refuses():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    for f in (lambda: block.linear(x, x), lambda: block.linear_backward(x, x, x),
              lambda: block.activation_backward(x, x, act="gelu"), lambda: block.norm(x, x[0]),
              lambda: block.norm_backward(x, x, x[0])):
        with pytest.raises(RuntimeError, match="CUDA"):
            f()
    for f in (lambda: block.linear([1], x), lambda: block.norm(None, x), lambda: block.activation_backward(x, 1, act="gelu")):
        with pytest.raises(ValueError):
            f()


def test_workspaces_are_modest():
    """Pieces of tiles take at most a few tiles an SM, whatever the sizes."""
    lib = block._library()
    d = _calls(block.LinearDesc, LINEAR)
    need = C.c_uint64(0)
    for t, k, n in ((1, 20480, 5120), (256, 7168, 256), (2048, 5120, 2560), (100_000, 64, 100_000), (300, 1 << 20, 300)):
        for out in (0, 2):
            assert lib.mv_linear_workspace_bytes(
                d(tokens=t, cols=k, rows=n, x_stride=k, w_stride=k, out_dtype=out), C.byref(need)) == mv.MV_OK
            assert need.value <= 160 << 20, (t, k, n, need.value)


@pytest.mark.parametrize("name", R.ACTS)
def test_reference_slopes(name):
    z = np.linspace(-6, 6, 97) + 0.013
    h = 1e-6
    assert np.allclose((R.act(z + h, name) - R.act(z - h, name)) / (2 * h), R.slope(z, name), atol=1e-8)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("full", [False, True])
def test_reference_norm_gradient(kind, full):
    """Every gradient of the plain code against differences of its results."""
    g = np.random.default_rng(5)
    t, h = 6, 7
    a = dict(y=g.normal(size=(t, h)), weight=g.normal(size=h), residual=g.normal(size=(t, h)))
    if kind == "layer":
        a["bias"] = g.normal(size=h)
    if full:
        a.update(post=g.normal(size=h), gate=g.normal(size=(3, h)))
        if kind == "layer":
            a["post_bias"] = g.normal(size=h)
    dn, dr = g.normal(size=(t, h)), g.normal(size=(t, h))

    def loss(**kw):
        (n, _), (r, _) = R.norm(**{**a, **kw}, alpha=0.5, kind=kind, eps=1e-3)
        return (n * dn).sum() + (r * dr).sum()

    grads = R.norm_backward(dn, **a, dr=dr, alpha=0.5, kind=kind, eps=1e-3)
    assert set(grads) == {"d" + k for k in a}
    for name, v in a.items():
        e = 1e-5
        for at in np.ndindex(v.shape):
            up, down = v.copy(), v.copy()
            up[at] += e
            down[at] -= e
            d = (loss(**{name: up}) - loss(**{name: down})) / (2 * e)
            assert abs(d - grads["d" + name][0][at]) < 1e-7 * (1 + abs(d)), (name, at)
