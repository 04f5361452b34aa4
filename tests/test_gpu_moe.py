"""The routed-expert operators on the GPU against plain 64-bit code.

Tolerances.  Float32 results: a weight is a ratio of scores, each the end of
an exponential (2 ulp), a division and a sum of at most 1024 positive terms in
a tree (11 levels), and the exponent x - m is rounded at |x - m| 2^-24 and
scaled to base two at as much again: relative 2^-24 (64 + 4 range), range the
spread of a row's logits.  Sixteen-bit results add half a unit in the last
place.  Choices are compared where they are decided by more than 2^-18 (the
scores' error is below 2^-20): rows with a closer call are not in the inputs;
exact ties are.
"""
import numpy as np
import pytest

import moe_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import moe, mv  # noqa: E402

U = 2.0 ** -24
HALF_ULP = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def spread(x):
    f = x[np.isfinite(x)]
    return float(f.max() - f.min()) if f.size else 0.0


def check_route(logits, topk, bias=None, **kw):
    """Route `logits` and compare with the plain code where it is decided."""
    ids, w = moe.route(logits, topk, bias=bias, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert ids.shape == w.shape == (logits.shape[0], topk)
    x = host(logits)
    want, ww, gaps = R.route(x, topk, bias=None if bias is None else host(bias), **kw)
    sure = gaps > 2.0 ** -18
    assert 2 * sure.sum() >= len(gaps)
    ids, w = ids.cpu().numpy(), host(w)
    assert np.array_equal(ids[sure], want[sure])
    tol = U * (64 + 4 * spread(x))
    # scores below the normal range of 32 bits round absolutely
    err = np.abs(w[sure] - ww[sure])
    assert (err <= tol * np.abs(ww[sure]) + 2.0 ** -126).all(), err.max()
    for row in ids:                                  # distinct, empty slots last
        got = row[row >= 0]
        assert len(set(got)) == len(got) and (row[len(got):] == -1).all()
    return ids, w


def randn(shape, seed, dtype=F32, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (spread * torch.randn(shape, generator=g, device="cuda")).to(dtype)


SHAPES = [  # tokens, experts, topk, groups, top_groups
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 8, 2, 1, 1), (33, 7, 3, 1, 1), (65, 60, 4, 1, 1),
    (17, 64, 6, 1, 1), (9, 65, 8, 1, 1), (40, 128, 8, 1, 1), (31, 129, 9, 1, 1),
    (300, 256, 8, 1, 1), (257, 256, 8, 8, 4), (19, 160, 6, 8, 3), (23, 60, 5, 6, 2),
    (11, 96, 4, 3, 1), (8, 257, 32, 1, 1), (6, 512, 10, 16, 5), (5, 1000, 17, 1, 1),
    (4, 1024, 32, 32, 32), (13, 32, 32, 1, 1), (12, 32, 4, 32, 7), (7, 33, 11, 11, 5)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_route_shapes(shape, dtype):
    T, E, k, G, tg = shape
    for n, (scores, with_bias, rule, renorm) in enumerate([
            ("softmax", False, "max", True), ("softmax", False, "max", False),
            ("sigmoid", True, "top2", True), ("sigmoid", False, "top2", False),
            ("sigmoid", True, "max", False), ("softmax", True, "top2", True),
            ("softmax", True, "max", False)]):
        x = randn((T, E), 100 * n + E, dtype, 2.0)
        b = randn((E,), n + 7, F32, 0.1) if with_bias else None
        check_route(x, k, b, scores=scores, groups=G, top_groups=tg, group_rule=rule,
                    renorm=renorm, scale=1.0 if n % 2 else 2.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(scores, dtype):
    """Equal logits (-0 and 0 among them), equal groups, equal biased scores."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-2, 3, (200, 96), generator=g, device="cuda").to(dtype) * 0.5
    x = torch.where((x == 0) & (torch.rand((200, 96), generator=g, device="cuda") < 0.5), -x, x)
    x[:20] = 0.25
    for k, G, tg, rule in [(8, 1, 1, "max"), (6, 8, 3, "max"), (6, 8, 3, "top2"), (12, 3, 2, "top2")]:
        check_route(x, k, scores=scores, groups=G, top_groups=tg, group_rule=rule)
    same = torch.full((96,), 0.125, device="cuda")
    check_route(x, 8, same, scores=scores, groups=8, top_groups=2)
    ids, _ = moe.route(x[:1], 5, scores=scores, bias=same)
    assert ids.tolist() == [[0, 1, 2, 3, 4]]


@pytest.mark.parametrize("E", [40, 256, 300])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_closed_experts_and_empty_rows(dtype, E):
    x = randn((64, E), 5, dtype)
    x[0] = -np.inf                                   # nothing left
    x[1] = float("nan")
    x[2] = -np.inf; x[2, E - 1] = 0.5                # one left
    x[3, ::2] = -np.inf
    x[4, 1::3] = float("nan")
    x[5, :E - 3] = -np.inf                           # fewer than topk
    x[6] = torch.finfo(dtype).min                    # the type's lowest value is open, and ties
    x[7, :] = torch.finfo(dtype).min; x[7, 9] = 1.0
    b = randn((E,), 6, F32, 0.1)
    b[3], b[5] = -np.inf, float("nan")
    for scores, renorm in [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]:
        for bias, G, tg, rule in [(None, 1, 1, "max"), (b, 1, 1, "max"), (None, 4, 2, "max"),
                                  (b, 4, 2, "top2"), (None, 4, 2, "top2")]:
            ids, w = moe.route(x, 6, scores=scores, bias=bias, groups=G, top_groups=tg,
                               group_rule=rule, renorm=renorm)
            want, ww, gaps = R.route(host(x), 6, scores, None if bias is None else host(bias), G,
                                     tg, rule, renorm)
            sure = gaps > 2.0 ** -18
            # rows 6 and 7 have a spread of the type's whole range: choices are still exact
            assert np.array_equal(ids.cpu().numpy()[sure], want[sure])
            rows = sure & (np.arange(64) != 7)
            assert np.allclose(host(w)[rows], ww[rows], rtol=U * 128, atol=2.0 ** -126)
            assert (ids[0] == -1).all() and (ids[1] == -1).all() and (w[:2] == 0).all()
            if bias is not None:
                assert not ((ids == 3) | (ids == 5)).any()


@pytest.mark.parametrize("renorm", [True, False])
def test_infinite_logits_take_the_whole_softmax(renorm):
    x = randn((4, 48), 8)
    x[0, 11] = np.inf
    x[1, 5] = x[1, 40] = np.inf
    x[2, :] = np.inf
    for bias in (None, randn((48,), 9, F32, 0.01)):
        ids, w = moe.route(x, 4, bias=bias, renorm=renorm)
        want, ww, _ = R.route(host(x), 4, bias=None if bias is None else host(bias), renorm=renorm)
        assert np.array_equal(ids.cpu().numpy()[0, :1], want[0, :1])
        if bias is None:
            assert np.array_equal(ids.cpu().numpy(), want)
            assert np.allclose(host(w), ww, rtol=U * 128)
        assert np.isfinite(host(w)).all()


def test_route_rows_apart_and_offset():
    """Rows of a wider array, at odd offsets, of every type; one row; none."""
    for dtype in (F32, F16, BF16):
        wide = randn((50, 300), 12, dtype)
        for a, n in [(1, 256), (0, 256), (3, 64), (7, 61), (2, 130)]:
            x = wide[:, a:a + n]
            ids, w = moe.route(x, 5, scores="sigmoid", renorm=False)
            ids2, w2 = moe.route(x.contiguous(), 5, scores="sigmoid", renorm=False)
            assert torch.equal(ids, ids2) and torch.equal(w, w2)
            check_route(x, 5)
            dx = moe.route_backward(x, ids, w, renorm=False)
            assert dx.is_contiguous()
            assert torch.equal(dx, moe.route_backward(x.contiguous(), ids, w, renorm=False))
        ids, w = moe.route(wide[:0], 5)
        assert ids.shape == w.shape == (0, 5)
        assert moe.route_backward(wide[:0], ids, w).shape == (0, 300)


def test_route_many_rows_equal_each_alone():
    """A long batch gives every row what it gets alone, run after run."""
    for E, G, tg, scores, rule, dtype in [(256, 8, 4, "sigmoid", "top2", F32), (60, 1, 1, "softmax", "max", BF16),
                                          (384, 1, 1, "sigmoid", "max", F16)]:
        x = randn((20_011, E), 20, dtype)
        b = randn((E,), 21, F32, 0.05) if scores == "sigmoid" else None
        kw = dict(scores=scores, bias=b, groups=G, top_groups=tg, group_rule=rule, renorm=scores == "sigmoid")
        ids, w = moe.route(x, 8, **kw)
        again, w_again = moe.route(x, 8, **kw)
        assert torch.equal(ids, again) and torch.equal(w, w_again)
        for t in (0, 1, 7_777, 20_010):
            i1, w1 = moe.route(x[t:t + 1], 8, **kw)
            assert torch.equal(ids[t:t + 1], i1) and torch.equal(w[t:t + 1], w1)
        d = randn((20_011, 8), 22)
        dx = moe.route_backward(x, ids, d, scores=scores, renorm=kw["renorm"])
        assert torch.equal(dx, moe.route_backward(x, ids, d, scores=scores, renorm=kw["renorm"]))
        assert torch.equal(dx[7_777:7_778], moe.route_backward(
            x[7_777:7_778], ids[7_777:7_778], d[7_777:7_778], scores=scores, renorm=kw["renorm"]))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("E,k,G,tg", [(256, 8, 8, 4), (256, 8, 1, 1), (60, 4, 1, 1), (160, 6, 8, 3), (96, 1, 3, 1),
                                      (250, 7, 5, 5), (33, 8, 11, 5), (8, 2, 1, 1), (64, 8, 32, 9), (224, 5, 7, 2), (512, 8, 1, 1), (32, 3, 1, 1), (288, 5, 1, 1),
                                      (1024, 8, 1, 1)])
def test_long_batches_choose_as_short_ones(E, k, G, tg, dtype):
    """Long and short batches are worked by different kernels: ids and weights
    are the same bits, in ordinary rows, rows of ties, closed, infinite and
    not-a-number logits, near and far biases."""
    T = 9_001
    x = randn((T, E), E + k, dtype, 1.5)
    g = torch.Generator(device="cuda").manual_seed(E)
    kind = torch.randint(0, 24, (T,), generator=g, device="cuda")
    hole = torch.rand((T, E), generator=g, device="cuda") < 0.6
    x[kind == 1] = 0.5                                         # ties
    x[kind == 2] = (x[kind == 2] * 2).round() / 2              # many ties, -0 among them
    x[(kind == 3)[:, None] & hole] = -np.inf
    x[kind == 4] = -np.inf
    x[(kind == 5)[:, None] & hole] = float("nan")
    x[(kind == 6)[:, None] & hole] = np.inf
    x[(kind == 7)[:, None] & hole] = torch.finfo(dtype).min
    x[kind == 8] = torch.finfo(dtype).max
    x[kind == 9] *= 30
    x[kind == 10] -= 200
    u = torch.rand((E,), generator=g, device="cuda")
    shut = u.clone()
    shut[::3], shut[1] = -np.inf, float("nan")
    for scores, rule, renorm, bias in [
            ("softmax", "max", True, None), ("softmax", "max", False, None), ("sigmoid", "max", False, None),
            ("sigmoid", "top2", True, 0.1 * u), ("sigmoid", "max", True, 50 * u), ("sigmoid", "top2", False, 1000 + u),
            ("sigmoid", "top2", True, None), ("sigmoid", "max", True, shut), ("softmax", "top2", False, 0.01 * u),
            ("softmax", "max", True, shut), ("sigmoid", "max", True, -3e5 * u)]:
        kw = dict(scores=scores, group_rule=rule, renorm=renorm, bias=bias, groups=G, top_groups=tg)
        ids, w = moe.route(x, k, **kw)
        parts = [moe.route(x[a:a + 1500], k, **kw) for a in range(0, T, 1500)]
        assert torch.equal(ids, torch.cat([p[0] for p in parts]))
        assert torch.equal(w, torch.cat([p[1] for p in parts]))
        assert torch.isfinite(w).all()
        some = torch.arange(0, T, 97, device="cuda")
        want, _, gaps = R.route(host(x[some]), k, scores, None if bias is None else host(bias), G, tg, rule, renorm)
        sure = gaps > 2.0 ** -18 * max(1.0, 0.0 if bias is None else float(bias[bias.isfinite()].abs().max()) / 8)
        got = ids[some].cpu().numpy()
        ordinary = kind[some].cpu().numpy() > 10
        assert np.array_equal(got[sure & ordinary], want[sure & ordinary])


def test_close_calls_are_decided_by_32_bit_scores():
    """Orders closer than any shortcut could tell: float32 logits one unit
    apart, and biased scores rebuilt with torch's own exp and division."""
    base = torch.linspace(0.4, 0.6, 64, device="cuda").repeat(32, 1)
    step = torch.arange(64, device="cuda")[torch.randperm(64, device="cuda")]
    x = torch.full((32, 64), 0.75, device="cuda")
    x = (x.view(torch.int32) + step.int()).view(torch.float32)        # 64 neighbouring floats
    ids, _ = moe.route(x, 10)
    want = x.sort(dim=1, descending=True, stable=True).indices[:, :10]
    assert torch.equal(ids.long(), want)
    b = (0.5 - 1.0 / (1.0 + torch.exp(-base[0]))).contiguous()        # makes the sums nearly equal
    v = 1.0 / (1.0 + torch.exp(-base)) + b
    ids, _ = moe.route(base, 10, scores="sigmoid", bias=b)
    assert torch.equal(ids.long(), v.sort(dim=1, descending=True, stable=True).indices[:, :10])


@pytest.mark.parametrize("k", [5, 12])
@pytest.mark.parametrize("E,G,tg", [(48, 1, 1), (256, 8, 3), (90, 5, 2), (700, 1, 1)])
def test_biases_of_any_range(E, G, tg, k):
    """Narrow, wide, far-off and infinite biases: the choice is that of the
    32-bit sums, rebuilt with torch's own exp, division and stable sort."""
    x = randn((150, E), E, F32, 3.0)
    x[:5] = 0.25
    g = torch.Generator(device="cuda").manual_seed(E + k)
    u = torch.rand((E,), generator=g, device="cuda")
    odd = u.clone()
    odd[3], odd[7], odd[11] = np.inf, np.inf, -np.inf
    for b in (0.01 * u, u - 0.5, 8 * u, -300 * u, 40.0 + u, 3e4 + u, 1e7 + u, 1e9 * u, odd, 0 * u):
        s = 1.0 / (1.0 + torch.exp(-x))
        v = (s + b).masked_fill(b == -np.inf, -np.inf)
        if G > 1:
            two = v.view(150, G, -1).sort(dim=2, descending=True).values[:, :, :2]
            best = two[:, :, 0] + two[:, :, 1].masked_fill(two[:, :, 1] == -np.inf, 0.0)
            keep = best.sort(dim=1, descending=True, stable=True).indices[:, :tg]
            stays = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
            v = v.view(150, G, -1).masked_fill(~stays[:, :, None], -np.inf).view(150, E)
        want = v.sort(dim=1, descending=True, stable=True).indices[:, :k]
        ids, w = moe.route(x, k, scores="sigmoid", bias=b.contiguous(), groups=G, top_groups=tg,
                           group_rule="top2", renorm=False)
        assert torch.equal(ids.long(), want)
        assert torch.allclose(w, s.gather(1, want), rtol=64 * U, atol=0)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False),
                                           ("sigmoid", True), ("sigmoid", False)])
def test_backward_is_the_formula(scores, renorm, dtype):
    for T, E, k in [(1, 1, 1), (3, 8, 2), (33, 60, 4), (70, 160, 6), (29, 256, 8), (5, 513, 11),
                    (4, 1024, 32)]:
        x = randn((T, E), E + k, dtype, 2.0)
        if E > 8:
            x[0, 3:5] = -np.inf
        ids, w = moe.route(x, k, scores=scores, renorm=renorm, scale=2.5)
        g = randn((T, k), E)
        if T > 2:
            ids[1, -1] = -1                          # an empty slot
            ids[2] = -1                              # a token that went nowhere
        dx = moe.route_backward(x, ids, g, scores=scores, renorm=renorm, scale=2.5)
        assert dx.dtype == dtype and dx.shape == (T, E)
        want = R.route_backward(host(x), ids.cpu().numpy(), host(g), scores, renorm, 2.5)
        # a difference of terms as large as scale |g| times the score (or weight)
        terms = 2.5 * np.abs(host(g)).max(1, keepdims=True)
        tol = U * (128 + 4 * spread(host(x))) * terms * (2 if renorm else 1)
        err = np.abs(host(dx) - want)
        assert (err <= tol + HALF_ULP[dtype] * np.abs(want) + 2.0 ** -25).all()
        if renorm or scores == "sigmoid":            # nothing but the choices has a gradient
            chosen = np.zeros((T, E + 1), bool)
            np.put_along_axis(chosen, np.where(ids.cpu().numpy() < 0, E, ids.cpu().numpy()), True, 1)
            assert (host(dx)[~chosen[:, :E]] == 0).all()


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False),
                                           ("sigmoid", True), ("sigmoid", False)])
def test_backward_against_differences(scores, renorm):
    """Central differences of the 64-bit weights at step h: error h^2 f''' / 6,
    below 1e-8 here, far under the 32-bit gradient's."""
    x = randn((6, 20), 2, F32, 1.5)
    ids, _ = moe.route(x, 5, scores=scores, renorm=renorm)
    g = randn((6, 5), 3)
    dx = host(moe.route_backward(x, ids, g, scores=scores, renorm=renorm, scale=1.5))
    xs, picks, gs, h = host(x), ids.cpu().numpy(), host(g), 1e-4
    for t in range(6):
        for e in range(20):
            up, down = xs[t].copy(), xs[t].copy()
            up[e] += h
            down[e] -= h
            d = (R.weights_of(up, picks[t], scores, renorm, 1.5)
                 - R.weights_of(down, picks[t], scores, renorm, 1.5)) / (2 * h)
            assert abs((d * gs[t]).sum() - dx[t, e]) <= 1e-5


def test_backward_where_a_row_is_closed():
    x = randn((5, 40), 4)
    x[0], x[1] = -np.inf, float("nan")
    x[2, 7] = np.inf
    ids, _ = moe.route(x, 4, renorm=False)
    g = randn((5, 4), 5)
    dx = moe.route_backward(x, ids, g, renorm=False)
    assert torch.isfinite(dx).all() and (dx[:2] == 0).all() and (dx[2] == 0).all()
    for scores in ("softmax", "sigmoid"):
        ids, _ = moe.route(x, 4, scores=scores)
        assert torch.isfinite(moe.route_backward(x, ids, g, scores=scores)).all()


# --------------------------------------------------------------------------
def check_exchange(ids, place, ranks, **kw):
    load, sent = moe.exchange(ids, place, ranks, **kw)
    assert load.dtype == sent.dtype == torch.int32
    starts = kw.pop("starts", None)
    want = R.exchange(ids.cpu().numpy() if ids.dim() == 3 else ids[None].cpu().numpy(),
                      place.cpu().numpy(), ranks,
                      starts=None if starts is None else starts.tolist(), **kw)
    lead = () if ids.dim() == 2 else (ids.shape[0],)
    assert load.shape == (*lead, len(place)) and sent.shape[-1] == ranks
    assert np.array_equal(load.cpu().numpy().reshape(want[0].shape), want[0])
    assert np.array_equal(sent.cpu().numpy().reshape(want[1].shape), want[1])


def picks(shape, experts, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, experts + 2, shape, generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("once", [True, False])
@pytest.mark.parametrize("B,T,k,E,ranks,sources", [
    (1, 1, 1, 1, 1, 1), (1, 12, 8, 16, 4, 4), (3, 60, 3, 60, 7, 5), (2, 64, 8, 256, 512, 64),
    (1, 37, 32, 1024, 9, 37), (5, 0, 2, 8, 3, 3), (2, 30, 5, 40, 8192, 2), (1, 3000, 6, 31, 3, 1),
    (4, 9, 1, 5, 2, 9)])
def test_exchange_counts(B, T, k, E, ranks, sources, once):
    """Ids and places beyond both ends are left out."""
    ids = picks((B, T, k), E, T + E)
    place = torch.randint(-1, ranks + 1, (E,), device="cuda", dtype=torch.int32,
                          generator=torch.Generator(device="cuda").manual_seed(E))
    check_exchange(ids, place, ranks, sources=sources, once=once)


@pytest.mark.parametrize("once", [True, False])
def test_exchange_uneven_sources(once):
    ids = picks((3, 500, 4), 24, 1)
    place = (torch.arange(24, device="cuda") % 10).int()
    for cuts in ([0, 0, 1, 1, 250, 499, 500, 500], [0, 500], [0, 0, 0, 500, 500]):
        check_exchange(ids, place, 10, starts=torch.tensor(cuts, device="cuda"), once=once)
    one = ids[1].contiguous()
    check_exchange(one, place, 10, starts=torch.tensor([0, 3, 500], device="cuda"), once=once)


@pytest.mark.parametrize("once", [True, False])
def test_exchange_all_to_one_and_long(once):
    """Every slot on one expert; more tokens on one source than a block's first pass."""
    ids = torch.full((1, 4096, 3), 5, device="cuda", dtype=torch.int32)
    place = torch.zeros(8, device="cuda", dtype=torch.int32)
    check_exchange(ids, place, 2, sources=2, once=once)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, 64, (1, 200_000, 4), generator=g, device="cuda", dtype=torch.int32)
    place = (torch.arange(64, device="cuda") // 4).int()
    for starts in (None, torch.tensor([0, 10, 199_000, 200_000], device="cuda")):
        n = 2 if starts is None else 3
        load, sent = moe.exchange(ids, place, 16, sources=n, starts=starts, once=once)
        assert torch.equal(load[0].long(), torch.bincount(ids.view(-1).long(), minlength=64))
        to = place[ids[0].long()].long()
        hit = torch.nn.functional.one_hot(to, 16).sum(1)
        hit = hit.clamp(max=1) if once else hit
        edge = [0, 100_000, 200_000] if starts is None else starts.tolist()
        for s in range(n):
            assert torch.equal(sent[0, s].long(), hit[edge[s]:edge[s + 1]].sum(0))


# --------------------------------------------------------------------------
def layer(E, H, I, group, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nib = lambda *d: torch.randint(0, 256, d, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    sc = lambda n, *d: ((0.5 + torch.rand(d, generator=g, device="cuda")) / (4 * n ** 0.5)).to(dtype)  # noqa: E731
    return (nib(E, 2 * I, H // 2), sc(H, E, 2 * I, H // group), nib(E, H, I // 2),
            sc(I, E, H, I // group))


def check_experts(x, ids, w, mats, group):
    """Rounding h to the type of x costs half a unit of every product W2 h,
    rounding y half a unit of y; sums in 32 bits of H and I terms cost
    (H + I) 2^-24 of the magnitudes summed, which the first bound's other half
    takes in.  Over all values the roundings are independent: together within
    two half units in the 2-norm."""
    y = moe.experts(x, ids, w, *mats)
    assert y.dtype == x.dtype and y.shape == x.shape and y.is_contiguous()
    h = [host(m) if m.is_floating_point() else m.cpu().numpy() for m in mats]
    want, size = R.experts(host(x), ids.cpu().numpy(), host(w), *h, group)
    half = HALF_ULP[x.dtype]
    err = np.abs(host(y) - want)
    assert (err <= half * np.abs(want) + 2 * half * size + 2.0 ** -23).all()
    if np.linalg.norm(want) > 0:
        assert np.linalg.norm(err) <= 2 * half * np.linalg.norm(want)
    return y


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,k,E,H,I,group", [
    (1, 1, 1, 32, 32, 32), (1, 8, 16, 256, 128, 128), (2, 2, 3, 64, 192, 64), (7, 4, 33, 288, 96, 32),
    (9, 2, 2, 128, 384, 128), (17, 3, 5, 640, 64, 64), (40, 8, 8, 96, 160, 32), (150, 4, 6, 256, 256, 64),
    (3, 32, 40, 1152, 384, 128), (1, 1, 2, 4096, 32, 32), (5, 1, 1, 32, 1056, 32)])
def test_experts_shapes(T, k, E, H, I, group, dtype):
    mats = layer(E, H, I, group, dtype, T + H)
    x = randn((T, H), T + 1, dtype)
    g = torch.Generator(device="cuda").manual_seed(T)
    order = torch.rand((T, max(E, k)), generator=g, device="cuda").argsort(1)[:, :k].int()
    ids = torch.where(order < E, order, -1)
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    check_experts(x, ids, w, mats, group)


def test_experts_skew_and_absence():
    """All tokens on one expert; on none; ids beyond both ends; a weight of 0;
    the same expert in two slots."""
    E, H, I, group = 6, 256, 128, 64
    mats = layer(E, H, I, group, BF16, 1)
    x = randn((70, H), 2, BF16)
    w = torch.rand((70, 3), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    ids = torch.full((70, 3), -1, device="cuda", dtype=torch.int32)
    assert (check_experts(x, ids, w, mats, group) == 0).all()
    ids[:, 1] = 4
    check_experts(x, ids, w, mats, group)
    ids[:, 0], ids[:35, 2], ids[35:, 2] = 6, 1 << 30, -(1 << 31)
    check_experts(x, ids, w, mats, group)
    ids[:, 0] = 4
    check_experts(x, ids, w, mats, group)
    w[:] = 0
    assert (check_experts(x, ids, w, mats, group) == 0).all()


def test_experts_extreme_nibbles_and_gates():
    """Every byte value, gates far into both tails, scales of both signs."""
    E, H, I, group = 2, 512, 64, 32
    w13, s13, w2, s2 = layer(E, H, I, group, F16, 1)
    w13.view(-1)[:256] = torch.arange(256, device="cuda", dtype=torch.uint8)
    w13[1] = 0                                        # every weight -8
    w2[0] = 255                                       # every weight 7
    s13[0, :8] *= -1
    x = randn((6, H), 2, F16)
    ids = torch.tensor([[0], [1]] * 3, device="cuda", dtype=torch.int32)
    check_experts(x, ids, torch.ones((6, 1), device="cuda"), (w13, s13, w2, s2), group)
    x[:] = 0
    assert (check_experts(x, ids, torch.ones((6, 1), device="cuda"), (w13, s13, w2, s2), group) == 0).all()


def test_experts_rows_of_any_magnitude():
    """bfloat16 rows far above and below half's range, alone and side by side, a
    row that spans both, and one of zeros: each row to the precision of its own
    size (two half units in the 2-norm; the spanning row's small entries are
    below the 32-bit sums' resolution of its large ones)."""
    E, H, I, group = 2, 256, 64, 64
    mats = layer(E, H, I, group, BF16, 8)
    x = randn((7, H), 9, BF16)
    powers = [0, 30, -40, 50, -20, 0, 0]
    x = (x.float() * torch.tensor([2.0 ** p for p in powers], device="cuda")[:, None]).to(BF16)
    x[5] *= torch.where(torch.arange(H, device="cuda") % 3 == 0, 2.0 ** 24, 2.0 ** -12).to(BF16)
    x[6] = 0
    ids = torch.tensor([[0, 1]] * 7, device="cuda", dtype=torch.int32)
    w = torch.full((7, 2), 0.5, device="cuda")
    y = moe.experts(x, ids, w, *mats)
    h = [host(m) if m.is_floating_point() else m.cpu().numpy() for m in mats]
    want, _ = R.experts(host(x), ids.cpu().numpy(), host(w), *h, group)
    for t in range(6):
        assert np.linalg.norm(host(y)[t] - want[t]) <= 2 * HALF_ULP[BF16] * np.linalg.norm(want[t]), t
    assert (y[6] == 0).all()


def test_experts_rows_apart_repeat_and_absent_experts_unread():
    E, H, I, group = 5, 320, 96, 32
    mats = layer(E, H, I, group, BF16, 4)
    wide = randn((12, 400), 5, BF16)
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.rand((12, E), generator=g, device="cuda").argsort(1)[:, :2].int()
    w = torch.rand((12, 2), generator=g, device="cuda")
    x = wide[:, 16:16 + H]
    y = check_experts(x, ids, w, mats, group)
    assert torch.equal(y, moe.experts(x.contiguous(), ids, w, *mats))
    # a token alone gets what it gets in the batch; experts nobody chose may hold anything
    for t in (0, 5, 11):
        m = [a.clone() for a in mats]
        away = [e for e in range(E) if e not in ids[t].tolist()]
        m[1][away] = float("nan")
        m[3][away] = float("inf")
        assert torch.equal(moe.experts(x[t:t + 1].contiguous(), ids[t:t + 1], w[t:t + 1], *m), y[t:t + 1])
    # a NaN in one token's row stays there
    bad = x.contiguous()
    bad[3, 7] = float("nan")
    z = moe.experts(bad, ids, w, *mats)
    keep = [t for t in range(12) if t != 3]
    assert torch.isnan(z[3]).all() and torch.equal(z[keep], y[keep])


def test_no_tokens_and_other_streams():
    E, H, I, group = 3, 64, 64, 64
    mats = layer(E, H, I, group, BF16, 4)
    none = moe.experts(torch.empty((0, H), device="cuda", dtype=BF16),
                       torch.empty((0, 2), device="cuda", dtype=torch.int32),
                       torch.empty((0, 2), device="cuda"), *mats)
    assert none.shape == (0, H)
    x = randn((4000, 256), 1)
    want = moe.route(x, 8, scores="sigmoid")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.route(x, 8, scores="sigmoid", stream=side)
    place = (torch.arange(256, device="cuda") // 4).int()
    side.wait_stream(torch.cuda.current_stream())
    load, sent = moe.exchange(got[0], place, 64, sources=40, stream=side)
    dx = moe.route_backward(x, got[0], got[1], scores="sigmoid", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    l2, s2 = moe.exchange(want[0], place, 64, sources=40)
    assert torch.equal(load, l2) and torch.equal(sent, s2)
    assert torch.equal(dx, moe.route_backward(x, want[0], want[1], scores="sigmoid"))


def test_calls_can_be_captured():
    """A graph of route, exchange and experts replays on new inputs."""
    E, H, I, group = 8, 128, 64, 32
    mats = layer(E, H, I, group, BF16, 9)
    logits, x = randn((6, E), 1), randn((6, H), 2, BF16)
    place = (torch.arange(E, device="cuda") // 4).int()

    def step():
        ids, w = moe.route(logits, 2)
        return (*moe.exchange(ids, place, 2, sources=3), moe.experts(x, ids, w, *mats),
                moe.route_backward(logits, ids, w))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    logits.copy_(randn((6, E), 11))
    x.copy_(randn((6, H), 12, BF16))
    graph.replay()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


# --------------------------------------------------------------------------
def refuses(f, *a, **kw):
    with pytest.raises((ValueError, mv.MVError)):
        f(*a, **kw)


def test_refusals():
    x = randn((4, 12), 1)
    for kw in (dict(topk=0), dict(topk=13), dict(topk=2, groups=5), dict(topk=2, groups=0),
               dict(topk=2, groups=3, top_groups=4), dict(topk=5, groups=3, top_groups=1),
               dict(topk=2, scores="tanh"), dict(topk=2, group_rule="sum"),
               dict(topk=2, scale=float("nan")), dict(topk=2, bias=torch.zeros(11, device="cuda")),
               dict(topk=2, bias=torch.zeros(12, device="cuda", dtype=F16)),
               dict(topk=2, bias=torch.zeros(24, device="cuda")[::2])):
        refuses(moe.route, x, **kw)
    refuses(moe.route, x.double(), 2)
    refuses(moe.route, x.t(), 2)
    refuses(moe.route, x[:1].expand(4, 12), 2)
    refuses(moe.route, randn((2, 1025), 1), 2)
    ids, w = moe.route(x, 3)
    refuses(moe.route_backward, x, ids.long(), w)
    refuses(moe.route_backward, x, ids[:3], w)
    refuses(moe.route_backward, x, ids, w.half())
    refuses(moe.route_backward, x, ids, w, scores="none")
    place = torch.zeros(12, device="cuda", dtype=torch.int32)
    refuses(moe.exchange, ids, place, 0)
    refuses(moe.exchange, ids, place, 8193, sources=1)
    refuses(moe.exchange, ids, place, 3)             # 4 tokens over 3 sources
    refuses(moe.exchange, ids, place.long(), 2)
    refuses(moe.exchange, ids, place, 2, starts=torch.tensor([0, 4], device="cuda").int())
    refuses(moe.exchange, ids, place, 2, sources=2, starts=torch.tensor([0, 4], device="cuda"))
    refuses(moe.exchange, ids, place, 2, starts=torch.tensor([0], device="cuda"))
    mats = layer(3, 64, 64, 32, BF16, 1)
    y = randn((4, 64), 1, BF16)
    pick, w2 = ids[:, :2].contiguous() % 3, w[:, :2].contiguous()
    moe.experts(y, pick, w2, *mats)
    refuses(moe.experts, y.half(), pick, w2, *mats)
    refuses(moe.experts, y.float(), pick, w2, *mats)
    refuses(moe.experts, y[:, :32], pick, w2, *mats)
    refuses(moe.experts, y, pick[:3], w2, *mats)
    refuses(moe.experts, y, pick, w2.half(), *mats)
    refuses(moe.experts, y, pick, w2, mats[0][:2].contiguous(), *mats[1:])
    refuses(moe.experts, y, pick, w2, *mats[:3], mats[3][:, :, :1].contiguous())
    refuses(moe.experts, y, pick, w2, mats[0], mats[1].repeat(1, 1, 2), *mats[2:])   # group 16
    odd = randn((4, 67), 1, BF16)
    refuses(moe.experts, odd[:, :64], pick, w2, *mats)           # rows 67 apart
    refuses(moe.experts, randn((4, 72), 1, BF16)[:, 1:65], pick, w2, *mats)   # base off by 2 bytes
