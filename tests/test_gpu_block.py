"""The block operators on the GPU against plain 64-bit code.

Tolerances, derived before the first run.  U = 2^-24.

Products: the tensor core adds 16 products a step to a sum of 32 bits and cuts off
what is beyond them, 2 U of the magnitude S = sum |x w| at most a step, and as
much again within a step: 4 U S a step over at most 32768 / 16 steps of a chain
(512 / 16 for 32-bit results), and U S for each of the few sums that are added
after.  So (4 K' / 16 + 16) U S, K' the products of a chain.  32-bit dz is held to
2^-17 of each value: 2^-17 S more.
Activations: slope at most 1.13, so 1.13 times z's error; their own exponentials,
reciprocals and erfc to 2^-20 of max(|z|, 1).
A result of 16 bits is rounded once: half a unit in the last place of its value,
eps / 2 relative, or half the smallest subnormal.
Norms: a row's sums of at most 16384 terms are eight or sixteen in a row and then
a tree, so within 32 U; a handful of operations of U each follow, squared sums
under a root and its reciprocal (2 ulp) among them: 64 U of the magnitudes (with
what cancels in a row counted by the reference) for one norm, 128 U through two,
256 U through their gradients.  Sums over T tokens: a run of rows in a row, then
runs and warps in trees: (T_run + 64) U of the magnitudes, T_run at most T.
"""
import numpy as np
import pytest

import block_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import block, moe, mv  # noqa: E402

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: U, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -126, F16: 2.0 ** -25, BF16: 2.0 ** -126}


def host(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def randn(shape, seed, dtype=F32, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mean + std * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def close(name, got, want, slack):
    """Within slack, and half a unit in the last place of the result's type."""
    assert tuple(got.shape) == np.shape(want), (name, got.shape, np.shape(want))
    tol = HALF[got.dtype] * (np.abs(want) + slack) + slack + TINY[got.dtype]
    err = np.abs(host(got) - want)
    worst = np.argmax(err - tol)
    assert (err <= tol).all(), (name, worst, err.flat[worst], tol.flat[worst], want.flat[worst])


def product_slack(m, k, dtype):
    return (4 * min(k, 512 if dtype == F32 else 32768) / 16 + 16) * U * m


def check_linear(x, w, bias=None, act="none", residual=None, scale=1.0, out=None, keep=False):
    got = block.linear(x, w, bias, act=act, residual=residual, scale=scale, out_dtype=out, keep=keep)
    y, z = got if keep else (got, None)
    want, wz, m = R.linear(host(x), host(w), host(bias), act, host(residual), scale)
    slack = product_slack(m, x.shape[1], y.dtype)
    after = abs(scale) * (1.13 * slack + (0 if act == "none" else 2.0 ** -20 * np.maximum(np.abs(wz), 1.0)))
    assert y.dtype == (out or x.dtype) and y.is_contiguous()
    close("y", y, want, after + 2 * U * np.abs(want))
    if keep:
        assert z.dtype == x.dtype
        close("z", z, wz, slack)
    return y


SHAPES = [  # tokens, cols, rows: one token, few, tiles' edges and one beyond, odd, whole tiles
    (1, 8, 8), (1, 1, 1), (1, 20480, 33), (2, 64, 128), (7, 100, 60), (16, 72, 129), (17, 640, 256), (33, 513, 257),
    (64, 128, 1000), (65, 1437, 101), (127, 63, 127), (128, 64, 64), (129, 65, 65), (255, 320, 384), (257, 257, 255),
    (300, 1000, 777), (1000, 64, 520), (513, 2048, 1024), (2048, 192, 2560),
    (1000, 64, 1), (300, 7, 3), (5, 3, 300), (64, 512, 20480), (200, 136, 30000)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_shapes(shape, dtype):
    t, k, n = shape
    x, w = randn((t, k), 1, dtype), randn((n, k), 2, dtype, k ** -0.5)
    check_linear(x, w)
    check_linear(x, w, out=F32)
    check_linear(x, w, randn((n,), 3, dtype), "gelu_tanh", randn((t, n), 4, dtype), 0.5, keep=True)
    check_linear(x, w, randn((n,), 5, F32), "silu", randn((t, n), 6, F32), out=F32, keep=True)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("shape", [(3, 64, 40), (130, 96, 264)])
def test_linear_activations(shape, act):
    t, k, n = shape
    x, w = randn((t, k), 1, BF16, 3.0), randn((n, k), 2, BF16, k ** -0.5)
    for out in (None, F32):
        for keep in (False, True):
            check_linear(x, w, None, act, None, 1.0, out, keep)
            check_linear(x, w, randn((n,), 3, BF16), act, randn((t, n), 4, out or BF16), -2.5, out, keep)


@pytest.mark.parametrize("tokens,cols,rows", [(70, 70000, 40), (2, 40000, 256), (300, 33000, 300)])
def test_linear_long_sums(tokens, cols, rows):
    """Positive terms: what is cut off does not cancel."""
    x, w = randn((tokens, cols), 1, BF16).abs(), randn((rows, cols), 2, BF16, 1 / cols).abs()
    check_linear(x, w, out=F32)
    check_linear(x, w)


def test_linear_strides_and_alignment():
    t, k, n = 70, 96, 72
    base = randn((t, 3 * k + 5), 1, BF16)
    wide = randn((n, 2 * k + 8), 2, BF16, 0.1)
    res = randn((t, n + 3), 3, BF16)
    for x in (base[:, :k], base[:, 1:k + 1], base[:, 8:k + 8], base[::2][:, :k].contiguous()):
        r = res[:len(x), :n] if len(x) == t else None
        check_linear(x, wide[:, 8:k + 8], None, "relu", r)
        check_linear(x, wide[:, 3:k + 3], None, "none", res[:len(x), 3:], 0.5)
    dz = randn((t, 2 * n + 1), 4, BF16)
    check_backward(dz[:, :n], base[:, 1:k + 1], wide[:, 8:k + 8])
    check_backward(dz[:, n:2 * n], base[:, :k], wide[:, 1:k + 1])


def check_backward(dz, x, w):
    dx, dw, db = block.linear_backward(dz, x, w, bias=True)
    a, b, c = host(dz), host(x), host(w)
    parts = 2.0 ** -17 if dz.dtype == F32 else 0.0
    k2 = 2 if dz.dtype == F32 else 1
    mx, mw = np.abs(a) @ np.abs(c), np.abs(a).T @ np.abs(b)
    close("dx", dx, a @ c, product_slack(mx, k2 * a.shape[1], BF16) + parts * mx)
    close("dw", dw, a.T @ b, product_slack(mw, k2 * a.shape[0], BF16) + parts * mw)
    close("dbias", db, a.sum(0), (len(a) + 64) * U * np.abs(a).sum(0))


@pytest.mark.parametrize("dtype,grad", [(F16, F16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_backward_shapes(shape, dtype, grad):
    t, k, n = shape
    check_backward(randn((t, n), 1, grad, n ** -0.5), randn((t, k), 2, dtype), randn((n, k), 3, dtype, k ** -0.5))


def test_linear_backward_long_sums():
    check_backward(randn((70000, 40), 1, BF16, 1e-3).abs(), randn((70000, 72), 2, BF16).abs(), randn((40, 72), 3, BF16))


def test_linear_backward_parts_and_extremes():
    """What is not asked for is not there; 32-bit gradients of any magnitude."""
    dz, x, w = randn((9, 24), 1, F32), randn((9, 40), 2, BF16), randn((24, 40), 3, BF16)
    full = block.linear_backward(dz, x, w, bias=True)
    for dx, dw, bias in [(True, False, False), (False, True, False), (False, False, True), (False, False, False)]:
        got = block.linear_backward(dz, x, w, dx=dx, dw=dw, bias=bias)
        for want, have, asked in zip(full, got, (dx, dw, bias)):
            assert torch.equal(have, want) if asked else have is None
    one = torch.eye(24, 40, device="cuda").to(BF16)
    for v in (3.4028e38, -3.4e38, 1e-30, 6.0e-8, 1.0 + 2.0 ** -12):
        d = torch.full((5, 24), v, device="cuda")
        got = block.linear_backward(d, x[:5], one, dw=False)[0]
        want = np.zeros((5, 40))
        want[:, :24] = v
        top = 2.0 ** 128 * (1 - 2.0 ** -9)                   # from here on bfloat16 rounds to infinity
        if abs(v) < top:
            close("dx", got, want, 2.0 ** -17 * np.abs(want))
        else:
            assert (got[:, :24] == (np.inf if v > 0 else -np.inf)).all()


def test_beyond_two_to_the_31():
    """Offsets that 32 bits do not hold: results of more than 2^32 bytes and 2^31 elements."""
    t, n = 70001, 32768
    x, w = randn((t, 64), 1, BF16), randn((n, 64), 2, BF16)
    y, z = block.linear(x, w, act="relu", keep=True)
    g = block.activation_backward(y, z, act="relu", scale=2.0)
    rows = [0, 1, 65535, 65536, 70000]
    want = host(x[rows]) @ host(w).T
    m = np.abs(host(x[rows])) @ np.abs(host(w)).T
    close("z", z[rows], want, product_slack(m, 64, BF16))
    assert torch.equal(y[rows], z[rows].clamp_min(0)) and torch.equal(g[rows], 2 * y[rows])
    del z, g
    dx = block.linear_backward(y, x, w, dw=False)[0]
    a, b = host(y[rows]), host(w)
    close("dx", dx[rows], a @ b, product_slack(np.abs(a) @ np.abs(b), n, BF16))
    h = 4096
    s = y.view(-1)[:t * n // h * h].view(-1, h)              # 560008 rows
    p = randn((h,), 3, F32)
    nn, r = block.norm(s, p, residual=s)
    rows = [0, 524288, len(s) - 1]
    close("n", nn[rows], R.norm(host(s[rows]), host(p), residual=host(s[rows]))[0][0], 2.0 ** -16)
    dy = block.norm_backward(nn, s, p, dr=r, residual=s).dy
    want = R.norm_backward(host(nn[rows]), host(s[rows]), host(p), dr=host(r[rows]), residual=host(s[rows]))["dy"]
    close("dy", dy[rows], want[0], 256 * U * want[1])


def test_linear_zero_sizes():
    x, w = randn((5, 16), 1, BF16), randn((8, 16), 2, BF16)
    assert block.linear(x[:0], w).shape == (0, 8)
    y, z = block.linear(x, w[:0], keep=True)
    assert y.shape == z.shape == (5, 0)
    dx, dw, db = block.linear_backward(x[:0, :8], x[:0], w, bias=True)
    assert dx.shape == (0, 16) and dw.shape == (8, 16) and not dw.any() and not db.any()
    dx, dw, db = block.linear_backward(x[:, :0], x, w[:0], bias=True)
    assert dx.shape == (5, 16) and not dx.any() and dw.shape == (0, 16) and db.shape == (0,)
    assert block.activation_backward(x[:0], x[:0], act="gelu").shape == (0, 16)
    n, r = block.norm(x[:0], w[0])
    assert n.shape == r.shape == (0, 16)
    g = block.norm_backward(x[:0], x[:0], w[0], residual=x[:0], post=w[0], gate=w[:2])
    assert g.dy.shape == g.dresidual.shape == (0, 16) and g.dgate.shape == (2, 16)
    assert not g.dweight.any() and not g.dpost.any() and not g.dgate.any() and g.dbias is None


@pytest.mark.parametrize("tokens", [3, 200])
def test_linear_infinities_stay_in_their_row_and_column(tokens):
    """A value that is not finite touches its token's row, or its output's column, alone."""
    k, n = 100, 77
    x, w = randn((tokens, k), 1, BF16), randn((n, k), 2, BF16)
    clean = block.linear(x, w)
    x2, w2 = x.clone(), w.clone()
    x2[1, 5] = float("nan")
    w2[7, 9] = float("inf")
    y = block.linear(x2, w2)
    rows, cols = [i for i in range(tokens) if i != 1], [i for i in range(n) if i != 7]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert y[1].isnan().all() and not y[:, 7].isfinite().any()
    dz = randn((tokens, n), 3, BF16)
    dz2 = dz.clone()
    dz2[2, 4] = float("inf")
    dx, dw, db = block.linear_backward(dz2, x, w, bias=True)
    cx, cw, cb = block.linear_backward(dz, x, w, bias=True)
    rows, cols = [i for i in range(tokens) if i != 2], [i for i in range(n) if i != 4]
    assert torch.equal(dx[rows], cx[rows]) and torch.equal(dw[cols], cw[cols]) and torch.equal(db[cols], cb[cols])
    assert not dx[2].isfinite().any() and not dw[4].isfinite().any() and db[4].isinf()


def test_linear_equal_rows_give_equal_rows():
    """A token's result does not depend on its place, nor on the tokens beside it."""
    x, w = randn((1, 777), 1, BF16), randn((500, 777), 2, BF16)
    for t in (2, 20, 100, 300, 700):
        many = randn((t, 777), 3, BF16)
        many[::3] = x
        y = block.linear(many, w, out_dtype=F32)
        assert (y[::3] == y[0]).all()
        other = randn((t, 777), 4, BF16)
        other[::3] = x
        assert torch.equal(block.linear(other, w, out_dtype=F32)[::3], y[::3])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("act", R.ACTS)
def test_activation_backward(act, dtype):
    for shape, pad in [((1, 1), 0), ((3, 7), 0), ((5, 64), 0), ((33, 1000), 0), ((7, 40), 8), ((6, 33), 3)]:
        z, dy = randn((shape[0], shape[1] + pad), 1, dtype, 2.0)[:, :shape[1]], randn(shape, 2, dtype)
        got = block.activation_backward(dy, z, act=act, scale=0.5)
        want = 0.5 * host(dy) * R.slope(host(z), act)
        # the slope's terms, of at most 1.13 and |z| exp(-z^2 / 2), to 2^-20
        close(act, got, want, 2.0 ** -20 * 1.5 * np.abs(0.5 * host(dy)))
        assert got.is_contiguous() and got.dtype == dtype


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_activations_at_their_ends(dtype):
    """Infinities are the limits, NaN stays, small values keep their relative precision."""
    z = torch.tensor([[float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e4, -1e4, 6e4, -6e4]], device="cuda").to(dtype)
    one = torch.ones_like(z)
    eye = torch.eye(9, 16, device="cuda").to(dtype)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        d = host(block.activation_backward(one, z, act=act))[0]
        assert d[0] == 1 and d[1] == 0 and np.isnan(d[2]) and d[5] == d[7] == 1 and d[6] == d[8] == 0, (act, d)
        assert d[3] == d[4] == (0 if act == "relu" else 0.5)
        if dtype == F32:
            continue
        # one column of w is 1: y = act(z), token by token
        y = host(block.linear(eye[:9, :9].contiguous() * 0 + z[0].nan_to_num(0, 0, 0)[:, None] * eye[:9, :9],
                              torch.ones((1, 9), device="cuda").to(dtype), act=act))[:, 0]
        assert y[3] == 0 and y[5] == host(z)[0, 5] and abs(y[6]) == 0, (act, y)
    big = torch.tensor([[float("inf")], [-float("inf")], [float("nan")]], device="cuda").to(dtype)
    if dtype != F32:
        for act in ("relu", "gelu", "gelu_tanh", "silu"):
            y = host(block.linear(big, torch.ones((1, 1), device="cuda").to(dtype), act=act))[:, 0]
            assert y[0] == np.inf and y[1] == 0 and np.isnan(y[2]), (act, y)


def norm_inputs(tokens, hidden, dtype, kind, params, residual, post, gates, biases, seed=0, std=1.0, mean=0.0):
    a = dict(y=randn((tokens, hidden), seed, dtype, 0.7 * std, mean), weight=randn((hidden,), seed + 1, params, 0.2, 1.0))
    if residual:
        a["residual"] = randn((tokens, hidden), seed + 2, dtype, 2.0 * std)
    if biases:
        a["bias"] = randn((hidden,), seed + 3, params)
    if post:
        a["post"] = randn((hidden,), seed + 4, params, 0.2, 1.0)
        if biases:
            a["post_bias"] = randn((hidden,), seed + 5, params)
    if gates:
        a["gate"] = randn((gates, hidden), seed + 6, params, 0.3, 0.5)
    return a


def check_norm(a, kind, alpha=1.0, eps=1e-6, with_dr=True):
    own = {k: v for k, v in a.items() if k not in ("y", "weight", "bias")}
    n, r = block.norm(a["y"], a["weight"], a.get("bias"), **own, alpha=alpha, kind=kind, eps=eps)
    plain = {k: host(v) for k, v in a.items()}
    (wn, mn), (wr, mr) = R.norm(**plain, alpha=alpha, kind=kind, eps=eps)
    if set(a) <= {"y", "weight", "bias"}:
        assert r is a["y"]
    close("r", r, wr, 64 * U * mr)
    close("n", n, wn, 128 * U * mn)
    dn = randn(a["y"].shape, 90, a["y"].dtype, 0.3)
    dr = randn(a["y"].shape, 91, a["y"].dtype, 0.3) if with_dr else None
    got = block.norm_backward(dn, a["y"], a["weight"], a.get("bias"), dr=dr, **own, alpha=alpha, kind=kind, eps=eps)
    want = R.norm_backward(host(dn), **plain, dr=host(dr), alpha=alpha, kind=kind, eps=eps)
    tokens = len(dn)
    for name in got._fields:
        g = getattr(got, name)
        if name not in want:
            assert g is None, name
            continue
        w, m = want[name]
        by_token = name in ("dy", "dresidual")
        assert g.dtype == (a["y"].dtype if by_token else a["weight"].dtype) and g.is_contiguous()
        close(name, g, w, (256 if by_token else 256 + tokens + 64) * U * m)
    return n, r, got


WIDTHS = [1, 2, 7, 8, 24, 31, 32, 64, 100, 256, 257, 511, 512, 520, 1000, 1437, 2048, 4104, 5120, 5128, 7168, 7169, 7176, 8192]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_norm_widths(hidden, dtype):
    for i, (kind, params, residual, post, gates, tokens) in enumerate([
            ("rms", F32, True, False, 0, 5), ("layer", dtype, True, True, 3, 9), ("rms", dtype, False, True, 1, 11),
            ("layer", F32, False, False, 7, 7), ("layer", F32, True, False, 0, 1)]):
        if hidden < 8 and kind == "layer":
            residual = True                                  # two values have nothing but a sign after the first norm
        a = norm_inputs(tokens, hidden, dtype, kind, params, residual, post, gates, kind == "layer", seed=10 * i)
        check_norm(a, kind, alpha=0.5 if i % 2 else 1.0, eps=1e-3, with_dr=i != 1)


@pytest.mark.parametrize("hidden", [9000, 12288, 16383, 16384])
def test_norm_longest_rows(hidden):
    for dtype in (F32, BF16):
        check_norm(norm_inputs(5, hidden, dtype, "layer", F32, True, True, 5, True), "layer", 0.5)
        check_norm(norm_inputs(6, hidden, dtype, "rms", F32, True, True, 2, False), "rms")


@pytest.mark.parametrize("tokens,gates", [(1, 1), (2, 2), (3, 1), (600, 1), (600, 600), (600, 4), (605, 5), (1300, 26), (2500, 500), (2002, 1001), (4000, 8), (3999, 3), (6000, 40), (9001, 1)])
def test_norm_gates(tokens, gates):
    """Runs of tokens that share a gate, across blocks and within, of odd and even lengths."""
    check_norm(norm_inputs(tokens, 72, F32, "layer", F32, True, True, gates, True), "layer", 0.5)
    check_norm(norm_inputs(tokens, 40, BF16, "rms", BF16, True, False, gates, False), "rms")


def test_norm_every_combination():
    for kind in ("rms", "layer"):
        for residual in (False, True):
            for post in (False, True):
                for gates in (0, 1, 4):
                    for biases in (False, True):
                        a = norm_inputs(12, 96, F32, kind, F32, residual, post, gates, biases)
                        check_norm(a, kind, alpha=0.25, with_dr=gates != 1)


def test_norm_far_mean_and_large_values():
    """A mean far from 0 costs the deviation nothing; large and small magnitudes."""
    check_norm(norm_inputs(20, 512, F32, "layer", F32, False, False, 0, True, mean=300.0), "layer")
    check_norm(norm_inputs(20, 512, F32, "layer", F32, False, True, 1, True, mean=300.0), "layer")
    check_norm(norm_inputs(20, 512, F32, "rms", F32, True, True, 1, False, std=1e12), "rms")
    check_norm(norm_inputs(20, 512, F32, "layer", F32, True, False, 0, True, std=1e-12), "layer", eps=1e-30)
    n, r = block.norm(torch.zeros((3, 64), device="cuda"), torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    assert (n == 1).all()                                    # nothing over eps


def test_norm_what_is_not_finite_stays_in_its_row():
    a = norm_inputs(9, 256, BF16, "layer", F32, True, True, 3, True)
    own = {k: v for k, v in a.items() if k not in ("y", "weight", "bias")}
    dn, dr = randn((9, 256), 1, BF16), randn((9, 256), 2, BF16)

    def run(y):
        n, r = block.norm(y, a["weight"], a["bias"], **own, kind="layer")
        return (n, r), block.norm_backward(dn, y, a["weight"], a["bias"], dr=dr, **own, kind="layer")

    (n, r), g = run(a["y"])
    y = a["y"].clone()
    y[3, 17] = float("nan")                                  # the first row of the second gate
    (n2, r2), g2 = run(y)
    rest = [i for i in range(9) if i != 3]
    assert torch.equal(n[rest], n2[rest]) and torch.equal(r[rest], r2[rest]) and n2[3].isnan().all()
    assert torch.equal(g.dy[rest], g2.dy[rest]) and torch.equal(g.dresidual[rest], g2.dresidual[rest])
    assert torch.equal(g.dgate[[0, 2]], g2.dgate[[0, 2]]) and g2.dgate[1].isnan().all()


def test_norm_strides_and_alignment():
    for dtype, hidden in ((BF16, 64), (F32, 64), (F16, 63)):
        a = norm_inputs(10, hidden, dtype, "rms", F32, True, True, 2, False)
        for pad, off in ((8, 0), (8, 8), (3, 1), (1, 0)):
            b = dict(a)
            for k in ("y", "residual"):
                wide = randn((10, hidden + pad + off), 5, dtype)
                wide[:, off:off + hidden] = a[k]
                b[k] = wide[:, off:off + hidden]
            n, r, g = check_norm(b, "rms")
        off_by = torch.empty(hidden + 1, device="cuda")[1:].copy_(a["weight"])      # parameters on no 16-byte boundary
        check_norm({**a, "weight": off_by}, "rms")
    y = randn((8, 64), 1, BF16)
    g = torch.ones(64, device="cuda")
    one = block.norm_backward(y, y, g, gate=g)
    assert one.dgate.shape == (64,) and block.norm_backward(y, y, g, gate=g[None]).dgate.shape == (1, 64)


def layer_run(x, s):
    """A dense branch between two norms, forward and backward, and a router's product."""
    n, r = block.norm(x, s["w1"], residual=s["stream"], gate=s["gate"], post=s["post"])
    h, z = block.linear(n, s["up"], s["b"], act="gelu_tanh", keep=True)
    y = block.linear(h, s["down"])
    logits = block.linear(n, s["router"], out_dtype=F32)
    ids, weights = moe.route(logits, 2, scores="sigmoid")
    # backward: the sum of all results
    dw = torch.ones_like(weights)
    dlogits = moe.route_backward(logits, ids, dw, scores="sigmoid")
    dn, drouter, _ = block.linear_backward(dlogits, n, s["router"])
    dh, ddown, _ = block.linear_backward(torch.ones_like(y), h, s["down"])
    dz = block.activation_backward(dh, z, act="gelu_tanh")
    dn2, dup, db = block.linear_backward(dz, n, s["up"], bias=True)
    grads = block.norm_backward(dn2 + dn, x, s["w1"], dr=torch.ones_like(r), residual=s["stream"], gate=s["gate"], post=s["post"])
    return [n, r, z, y, logits, ids, weights, drouter, ddown, dup, db, *[g for g in grads if g is not None]]


def layer_state(tokens, hidden, inner, experts, seed=0):
    s = dict(w1=randn((hidden,), seed, F32, 0.1, 1.0), stream=randn((tokens, hidden), seed + 1, BF16, 2.0),
             gate=randn((hidden,), seed + 2, F32, 0.1, 0.5), post=randn((hidden,), seed + 3, F32, 0.1, 1.0),
             up=randn((inner, hidden), seed + 4, BF16, hidden ** -0.5), b=randn((inner,), seed + 5, BF16, 0.1),
             down=randn((hidden, inner), seed + 6, BF16, inner ** -0.5), router=randn((experts, hidden), seed + 7, BF16, hidden ** -0.5))
    return randn((tokens, hidden), seed + 8, BF16), s


@pytest.mark.parametrize("tokens,hidden,inner,experts", [(1, 256, 512, 16), (37, 200, 333, 60), (300, 512, 1024, 64)])
def test_a_layer_forward_and_backward(tokens, hidden, inner, experts):
    """All of them together against 64-bit differentiation.  Every tensor between is rounded
    to bfloat16, 2^-9 of its norm or so, and at most ten of them lie on a path."""
    x, s = layer_state(tokens, hidden, inner, experts)
    got = layer_run(x, s)
    d = {k: v.double().requires_grad_(True) for k, v in {**s, "x": x}.items()}

    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    r = d["stream"] + d["gate"] * rms(d["x"], d["post"])
    n = rms(r, d["w1"])
    z = n @ d["up"].t() + d["b"]
    h = torch.nn.functional.gelu(z, approximate="tanh")
    y = h @ d["down"].t()
    logits = n @ d["router"].t()
    ids = got[5].long()                                      # the choice is compared in test_gpu_moe.py
    score = torch.sigmoid(logits).gather(1, ids)
    weights = score / score.sum(1, keepdim=True)
    # the branch's own gradient, the router's and the stream's
    (y.sum() + r.sum() + weights.sum()).backward()
    want = [n, r, z, y, logits, None, weights, d["router"].grad, d["down"].grad, d["up"].grad, d["b"].grad,
            d["x"].grad, d["stream"].grad, d["w1"].grad, d["post"].grad, d["gate"].grad]
    assert len(got) == len(want)
    scale = max(d["router"].grad.norm().item(), 1e-3)
    for i, (a, b) in enumerate(zip(got, want)):
        if b is None:
            continue
        if i == 7:            # renormalised weights add up to one: their gradient is what cancels
            assert (a.double() - b).norm() <= 2.0 ** -6 * max(scale, n.norm().item() * 2.0 ** -9)
        else:
            assert (a.double() - b).norm() <= 10 * 2.0 ** -9 * 2 * b.norm() + 1e-6, i


def test_captured_and_replayed_with_an_eager_graph_alive():
    """Forward and backward in a CUDA graph: replays equal eager calls, new inputs give new results."""
    x, s = layer_state(70, 264, 1000, 32)
    eager = layer_run(x, s)
    leaf = x.float().requires_grad_(True)                    # an autograd graph of the same values stays alive
    alive = (leaf * leaf).sum()
    static, side = x.clone(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_run(static, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer_run(static, s)
    for seed in (None, 77):
        fresh = x if seed is None else randn(x.shape, seed, BF16)
        static.copy_(fresh)
        graph.replay()
        want = eager if seed is None else layer_run(fresh, s)
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), i
    alive.backward()
    assert torch.equal(leaf.grad, 2 * leaf.detach())


def test_two_streams_at_once():
    """Calls under way on two streams, with more work than one fills, do not meet."""
    states = [layer_state(300, 1024, 4096, 64, seed=100 * i) for i in range(2)]
    want = [layer_run(*st) for st in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(6):
        for i, st in enumerate(states):
            with torch.cuda.stream(streams[i]):
                got[i] = layer_run(*st)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert block.gave_up() == 0


def test_on_another_stream_than_the_current_one():
    x, w = randn((40, 256), 1, BF16), randn((136, 256), 2, BF16)
    g = randn((256,), 3, F32)
    side = torch.cuda.Stream()
    want = (block.linear(x, w), *block.norm(x, g, residual=x), block.activation_backward(x, x, act="silu"),
            *block.linear_backward(x[:, :136], x, w, bias=True),
            *[v for v in block.norm_backward(x, x, g, residual=x) if v is not None])
    torch.cuda.synchronize()
    got = (block.linear(x, w, stream=side), *block.norm(x, g, residual=x, stream=side),
           block.activation_backward(x, x, act="silu", stream=side),
           *block.linear_backward(x[:, :136], x, w, bias=True, stream=side),
           *[v for v in block.norm_backward(x, x, g, residual=x, stream=side) if v is not None])
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_bits_on_every_run():
    x, w = randn((1777, 1437), 1, F16), randn((1001, 1437), 2, F16)
    dz = randn((1777, 1001), 3, F16)
    a = norm_inputs(1777, 1437, F16, "layer", F32, True, True, 1, True)
    own = {k: v for k, v in a.items() if k not in ("y", "weight", "bias")}

    def run():
        return [block.linear(x, w, act="gelu"), block.linear(x[:5], w, out_dtype=F32), *block.linear_backward(dz, x, w, bias=True),
                *block.norm(a["y"], a["weight"], a["bias"], **own, kind="layer"),
                *block.norm_backward(x, a["y"], a["weight"], a["bias"], **own, kind="layer")]

    first = run()
    for _ in range(4):
        assert all(torch.equal(p, q) for p, q in zip(first, run()))


def test_refusals():
    x, w = randn((4, 16), 1, BF16), randn((8, 16), 2, BF16)
    v = torch.ones(16, device="cuda")
    for f in (lambda: block.linear(x, w.half()), lambda: block.linear(x.float(), w.float()), lambda: block.linear(x, w[:, :8]),
              lambda: block.linear(x, w, v), lambda: block.linear(x, w, act="swish"), lambda: block.linear(x[:, :0], w[:, :0]),
              lambda: block.linear(x, w, out_dtype=F16), lambda: block.linear(x, w, residual=x),
              lambda: block.linear(x, w, residual=x[:, :8], out_dtype=F32), lambda: block.linear(x, w, scale=float("nan")),
              lambda: block.linear(x.t(), w), lambda: block.linear(x[0], w), lambda: block.linear(x, w, scale=1e39),
              lambda: block.linear_backward(x, x, w), lambda: block.linear_backward(x[:, :8].float(), x.half(), w.half()),
              lambda: block.linear_backward(x[:, :8], x.float(), w), lambda: block.activation_backward(x, x.half(), act="gelu"),
              lambda: block.activation_backward(x, x, act="tanh"), lambda: block.activation_backward(x[:2], x, act="gelu"),
              lambda: block.norm(x, v.half()), lambda: block.norm(x, v[:8]), lambda: block.norm(x, v, kind="batch"),
              lambda: block.norm(x, v, post_bias=v), lambda: block.norm(x, v, gate=torch.ones((3, 16), device="cuda")),
              lambda: block.norm(x, v, gate=torch.ones((0, 16), device="cuda")), lambda: block.norm(x, v, eps=-1.0),
              lambda: block.norm(x, v, alpha=float("inf")), lambda: block.norm(x, v, residual=x.float()),
              lambda: block.norm(x, v, post=v.bfloat16()), lambda: block.norm(x[:, :0], v[:0]),
              lambda: block.norm(randn((1, 16385), 1), torch.ones(16385, device="cuda")),
              lambda: block.norm_backward(x[:2], x, v), lambda: block.norm_backward(x, x, v, dr=x.float())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(RuntimeError):
        block.linear(x, w.cpu())
    assert mv.MV_OK == 0
