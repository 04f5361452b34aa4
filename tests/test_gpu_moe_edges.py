"""The routed-expert operators where they can go wrong: extremes of value, size
and shape, against plain 64-bit code."""
import numpy as np
import pytest

import moe_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import moe, moe_layer  # noqa: E402
from test_gpu_moe import BF16, F16, F32, HALF_ULP, U, host, layer, randn, spread  # noqa: E402


# ---- experts ---------------------------------------------------------------
def experts_of(x, ids, w, mats, group):
    """(result, 64-bit result, magnitudes summed) of one call."""
    y = moe.experts(x, ids, w, *mats)
    h = [host(m) if m.is_floating_point() else m.cpu().numpy() for m in mats]
    return (y, *R.experts(host(x), ids.cpu().numpy(), host(w), *h, group))


def one_slot(T, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    return ids, torch.rand((T, k), generator=g, device="cuda") + 0.1


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,E,k,H,I,group", [(5, 3, 1, 256, 256, 128), (12, 1, 1, 64, 320, 64),
                                             (24, 1, 1, 128, 256, 32), (60, 6, 2, 128, 128, 32)])
def test_experts_round_once(T, E, k, H, I, group, dtype):
    """Nothing but the result is rounded to the type: the inner activations are
    held to 2^-18 or so of their value, which leaves the sum off by less than
    2^-18 of a result's usual magnitude, 2^-8 of a float16 unit there.  Where
    terms cancel, a result 2^-j as large (2^-j as likely) has units 2^-j as
    large: all in all a few times 2^-8 of the results land on the other side of
    a rounding boundary; one in twenty is allowed.  (An inner rounding to the
    type turns over a third of them.)"""
    mats = layer(E, H, I, group, dtype, T + H)
    x = randn((T, H), T + 1, dtype)
    ids, w = one_slot(T, E, k, T)
    y, want, size = experts_of(x, ids, w, mats, group)
    once = torch.from_numpy(want).to(dtype)
    assert (y.cpu() == once).float().mean() >= 0.95
    # H and I additions that each may lose 2^-23 of what is summed; inner sums are 8 to 16 times their result
    bound = HALF_ULP[dtype] * np.abs(want) + (2.0 ** -17 + (16 * H + I) * 2.0 ** -23) * size
    assert (np.abs(host(y) - want) <= bound).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_experts_inner_activations_of_any_magnitude(dtype):
    """Inner activations far beyond float16's range, and far below it, whose
    products are well inside."""
    E, H, I, group = 2, 128, 128, 64
    w13, s13, w2, s2 = layer(E, H, I, group, dtype, 31)
    ids = torch.tensor([[0, 1]] * 9, device="cuda", dtype=torch.int32)
    w = torch.full((9, 2), 0.5, device="cuda")
    for up, down in ((2.0 ** 8, 2.0 ** -7), (2.0 ** -9, 2.0 ** 8)):
        x = (randn((9, H), 32) * up).to(dtype)
        y, want, size = experts_of(x, ids, w, (w13, s13, w2, (s2.float() * down).to(dtype)), group)
        bound = HALF_ULP[dtype] * np.abs(want) + (2.0 ** -17 + (16 * H + I) * 2.0 ** -23) * size + 2.0 ** -25
        assert (np.abs(host(y) - want) <= bound).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H,I,group", [(4480, 2176, 128), (2240, 2112, 64), (1120, 1568, 32)])
def test_experts_over_many_steps(H, I, group, dtype):
    """Rows of many steps, chunks and scale epochs with an odd tail, for one, two
    and three tiles of pairs an expert; a token in a large batch gets the bits
    it gets alone.  Error as check_experts in test_gpu_moe derives it."""
    E = 2
    mats = layer(E, H, I, group, dtype, H)
    x = randn((31, H), H + 1, dtype)
    for n in (1, 13, 24, 31):                        # tiles: 1; 2; 3; 3 and 1
        ids = torch.tensor([[t % 16 and 0 or 1] for t in range(n)], device="cuda", dtype=torch.int32)
        if n == 24:
            ids[:] = 0
        w = torch.ones((n, 1), device="cuda")
        y = moe.experts(x[:n], ids, w, *mats)
        if n == 31:
            h = [host(m) if m.is_floating_point() else m.cpu().numpy() for m in mats]
            want, size = R.experts(host(x), ids.cpu().numpy(), host(w), *h, group)
            half, err = HALF_ULP[dtype], np.abs(host(y) - want)
            assert (err <= half * np.abs(want) + 2 * half * size + 2.0 ** -23).all()
            assert np.linalg.norm(err) <= 2 * half * np.linalg.norm(want)
        for t in sorted({0, 5 % n, n - 1}):
            alone = moe.experts(x[t:t + 1], ids[t:t + 1], w[t:t + 1], *mats)
            assert torch.equal(alone, y[t:t + 1]), (n, t)


# ---- exchange --------------------------------------------------------------
def check_counts(ids, place, ranks, once, starts=None, sources=None):
    kw = dict(starts=None if starts is None else torch.tensor(starts, device="cuda"), sources=sources, once=once)
    load, sent = moe.exchange(ids, place, ranks, **kw)
    want = R.exchange(ids.cpu().numpy(), place.cpu().numpy(), ranks, sources=sources, starts=starts, once=once)
    assert np.array_equal(load.cpu().numpy(), want[0])
    assert np.array_equal(sent.cpu().numpy(), want[1])


def random_ids(shape, experts, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, experts + 1, shape, generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("once", [True, False])
@pytest.mark.parametrize("B,T,k", [(1, 40, 4), (3, 40, 4), (1, 9000, 4), (40, 300, 3), (300, 40, 5)])
def test_exchange_of_tokens_that_no_source_holds(B, T, k, once):
    """Starts that leave tokens out before the first source and behind the last:
    they count nowhere, however large the call."""
    ids = random_ids((B, T, k), 24, T)
    place = (torch.arange(24, device="cuda") % 6).int()
    for starts in ([3, 11, 11, 20, T - 7], [0, T - 1], [5, 5, 6, T], [T, T], [0, 0]):
        check_counts(ids, place, 6, once, starts=starts)


@pytest.mark.parametrize("once", [True, False])
@pytest.mark.parametrize("B,S,T,k,E,ranks", [(700, 37, 74, 3, 20, 10), (2, 2000, 4000, 5, 33, 7),
                                             (40, 32, 64, 8, 1024, 8192), (1, 1300, 2600, 32, 40, 9),
                                             (1300, 1, 3, 1, 5, 2)])
def test_exchange_of_many_sources(B, S, T, k, E, ranks, once):
    """Eight sources an SM and more: runs of sources that span batches, one warp
    a block where counts are large, ids a token that do not divide a warp."""
    ids = random_ids((B, T, k), E, S)
    place = torch.randint(-1, ranks + 1, (E,), device="cuda", dtype=torch.int32,
                          generator=torch.Generator(device="cuda").manual_seed(E))
    check_counts(ids, place, ranks, once, sources=S)


@pytest.mark.parametrize("once", [True, False])
def test_exchange_of_many_uneven_sources(once):
    g = np.random.default_rng(3)
    T = 9000
    cuts = np.sort(np.concatenate([g.integers(0, 40, 900), g.integers(6000, T + 1, 800)]))      # a long one amid short and empty ones
    starts = [0, *cuts.tolist(), T]
    ids = random_ids((2, T, 6), 50, 4)
    place = (torch.arange(50, device="cuda") // 4).int()
    check_counts(ids, place, 13, once, starts=starts)
    check_counts(ids, place, 13, once, starts=[7, *[max(7, c) for c in cuts.tolist()]])


# ---- route -----------------------------------------------------------------
# experts, groups: with more than eight slots no lane layout of a warp holds them
UNEVEN = [(960, 3), (960, 5), (960, 6), (960, 10), (960, 12), (720, 5), (720, 9), (720, 10), (720, 18), (720, 20),
          (561, 17), (1020, 17), (1023, 3), (1023, 31), (1023, 11)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("E,G", UNEVEN)
def test_route_many_slots_of_uneven_groups(E, G, dtype):
    x = randn((5, E), E + G, dtype, 2.0)
    x[3, ::3] = -np.inf
    x[4] = 0.5
    b = randn((E,), G, F32, 0.1)
    for scores, bias, rule, renorm in [("softmax", None, "max", True), ("softmax", b, "max", False),
                                       ("sigmoid", b, "top2", True), ("sigmoid", None, "top2", False)]:
        for tg, k in ((G, 9), (max(2, G // 2), 32)):
            k = min(k, tg * (E // G))
            kw = dict(scores=scores, groups=G, top_groups=tg, group_rule=rule, renorm=renorm)
            ids, w = moe.route(x, k, bias=bias, **kw)
            want, ww, gaps = R.route(host(x), k, bias=None if bias is None else host(bias), **kw)
            sure = gaps > 2.0 ** -18
            assert 2 * sure.sum() >= 5
            assert np.array_equal(ids.cpu().numpy()[sure], want[sure])
            tol = U * (64 + 4 * spread(host(x)))
            assert (np.abs(host(w) - ww) <= tol * np.abs(ww) + 2.0 ** -126)[sure].all()


def test_every_documented_size_is_taken():
    """Every way to part up to 1024 experts into groups, with 9 and 32 slots:
    the ids are those of the logits' own stable order."""
    for G in range(2, 33):
        for E in range(G, 1025, G):
            if E % (7 * G) and E + G <= 1024:        # a seventh of them, and the largest
                continue
            x = randn((2, E), E)
            for k in {min(9, E), min(32, E)}:
                ids, _ = moe.route(x, k, groups=G, top_groups=G)
                assert torch.equal(ids.long(), x.sort(dim=1, descending=True, stable=True).indices[:, :k]), (E, G, k)


def test_a_bias_closes_the_choice_not_the_score():
    """The bias is no part of the score: an expert that it closes is never
    chosen, and keeps its share of the softmax."""
    for T in (7, 3000):
        x = randn((T, 64), 3, F32, 2.0)
        b = torch.zeros(64, device="cuda")
        b[5], b[9] = -np.inf, float("nan")
        for k in (4, 12):
            ids, w = moe.route(x, k, bias=b, renorm=False)
            p = torch.softmax(x.double(), dim=1)
            v = p.float()
            v[:, [5, 9]] = -1.0
            want = v.sort(dim=1, descending=True, stable=True).indices[:, :k]
            assert (ids.long() == want).all(1).float().mean() > 0.99       # 32-bit scores differ in the last place
            assert not ((ids == 5) | (ids == 9)).any()
            assert torch.allclose(w.double(), p.gather(1, ids.long()), rtol=U * (64 + 4 * spread(host(x))), atol=0)
        x[:, 9] = np.inf                                  # all of the softmax, and not to be chosen
        ids, w = moe.route(x, 4, bias=b, renorm=False)
        assert (w == 0).all() and not (ids == 9).any()


CLOSE = [(1024, 8, 1, 1, "softmax", 0.0, 3e-4), (512, 6, 8, 3, "softmax", 0.0, 1e-3), (256, 8, 8, 4, "sigmoid", -8.0, 1e-3),
         (300, 10, 1, 1, "sigmoid", -9.0, 1e-4), (192, 5, 1, 1, "sigmoid", 12.0, 1e-5)]


@pytest.mark.parametrize("T", [40, 2500])
@pytest.mark.parametrize("E,k,G,tg,scores,shift,spread_of_bias", CLOSE)
def test_choices_of_scores_that_nearly_meet(E, k, G, tg, scores, shift, spread_of_bias, T):
    """Small or saturated scores, whose order turns on a few units of 2^-22: the
    choice is within the 32-bit scores' error (2^-20 of the greatest, at most 1)
    of the best, and the weights are those of the experts chosen."""
    x = randn((T, E), E + k, F32, 1.0) + shift
    b = randn((E,), k, F32, spread_of_bias)
    ids, w = moe.route(x, k, scores=scores, bias=b, groups=G, top_groups=tg, group_rule="top2", renorm=False)
    at = ids.long()
    assert (at >= 0).all() and (at.sort(dim=1).values.diff(dim=1) > 0).all()
    s = torch.softmax(x.double(), dim=1) if scores == "softmax" else torch.sigmoid(x.double())
    assert torch.allclose(w.double(), s.gather(1, at), rtol=U * (64 + 4 * spread(host(x))), atol=0)
    v = s + b.double()
    err = 2.0 ** -20
    if G > 1:
        two = v.view(T, G, -1).topk(2, dim=2).values.sum(2)
        used = torch.zeros_like(two, dtype=torch.bool).scatter_(1, at // (E // G), True)
        assert (used.sum(1) <= tg).all()
        least = two.topk(tg, dim=1).values[:, -1:]                        # no group used that is clearly worse
        assert (two >= least - 2 * err)[used].all()
        sure = (least[:, 0] - two.topk(tg + 1, dim=1).values[:, -1]) > 2 * err
        keep = torch.zeros_like(two, dtype=torch.bool).scatter_(1, two.topk(tg, dim=1).indices, True)
        v = v.view(T, G, -1).masked_fill(~keep[:, :, None], -np.inf).view(T, E)[sure]
        at = at[sure]
        assert len(at) > 0
    got = v.gather(1, at)
    assert (got - v.topk(k, dim=1).values).abs().max() <= err             # slot by slot


DEEP = [(7, 20, 4, 1, 1), (2600, 64, 4, 1, 1), (2600, 32, 6, 4, 2), (9, 300, 5, 1, 1), (11, 48, 12, 1, 1), (9, 48, 12, 4, 2)]


@pytest.mark.parametrize("T,E,k,G,tg", DEEP)
def test_sigmoid_of_very_negative_logits(T, E, k, G, tg):
    """Scores down to nothing in 32 bits: renormalised weights depend on their
    ratio alone.  Short and long batches, a few and many slots, exact ties."""
    for shift in (-16.0, -19.0, -60.0, -88.0, -95.0, -200.0, -600.0):
        x = (randn((T, E), E, F32, 2.0) + shift)[:T]
        x[1] = shift                                                      # ties
        x[2, 3] = 1.0                                                     # one that is not small
        x[3, ::2] = -np.inf
        kw = dict(scores="sigmoid", groups=G, top_groups=tg)
        ids, w = moe.route(x, k, **kw)
        some = np.unique(np.r_[0:min(T, 9), T - 1, np.arange(0, T, 199)])
        want, ww, gaps = R.route(host(x)[some], k, **kw)
        sure = gaps > 0                                                   # logits in order: exact
        assert sure.all() and np.array_equal(ids.cpu().numpy()[some], want)
        # row 2 spreads over the whole shift: what is far below its greatest rounds absolutely
        tol = U * (64 + 4 * 20) * np.abs(ww) + 2.0 ** -100
        assert (np.abs(host(w)[some] - ww) <= tol).all(), shift
        g = randn((T, k), 5)
        dx = host(moe.route_backward(x, ids, g, scores="sigmoid"))
        assert np.isfinite(dx).all(), shift
        dd = R.route_backward(host(x)[some], want, host(g)[some], "sigmoid", True, 1.0)
        terms = np.abs(host(g)[some]).max(1, keepdims=True)
        assert (np.abs(dx[some] - dd) <= U * 256 * terms).all(), shift


# ---- route_backward --------------------------------------------------------
@pytest.mark.parametrize("E,k", [(11, 11), (40, 11), (200, 11)])
def test_sigmoid_gradient_in_both_tails(E, k):
    """To relative precision: a score and its complement are each an exponential
    (2 units), a sum and a division, and three products follow."""
    tail = torch.tensor([-80.0, -30.0, -20.0, -10.0, -5.0, 0.0, 5.0, 10.0, 15.0, 20.0, 80.0], device="cuda")
    x = torch.full((3, E), -90.0, device="cuda")
    x[:, E - 11:] = tail
    ids = torch.arange(E - 11, E, device="cuda", dtype=torch.int32).repeat(3, 1).contiguous()
    g = randn((3, k), 8).abs() + 0.5
    s = 1.0 / (1.0 + torch.exp(-tail.double()))
    c = 1.0 / (1.0 + torch.exp(tail.double()))
    dx = moe.route_backward(x, ids, g, scores="sigmoid", renorm=False, scale=2.5)[:, E - 11:].double()
    want = 2.5 * g.double() * s * c
    assert ((dx - want).abs() <= 16 * U * want.abs()).all()
    dx = moe.route_backward(x, ids, g, scores="sigmoid", renorm=True, scale=2.5)[:, E - 11:].double()
    w = s / s.sum()
    dot = (g.double() * w).sum(1, keepdim=True)
    want = 2.5 * w * (g.double() - dot) * c
    # the sums over eleven slots and the difference of g and its mean lose to their own size
    assert ((dx - want).abs() <= 32 * U * 2.5 * w * c * (g.double() + dot) + 2.0 ** -126).all()


# ---- arguments and timing --------------------------------------------------
def test_scale_beyond_32_bits_is_refused():
    x = randn((4, 12), 1)
    ids, w = moe.route(x, 3, scale=3.0e38)
    for scale in (1e39, -1e300, float("inf")):
        with pytest.raises(ValueError):
            moe.route(x, 3, scale=scale)
        with pytest.raises(ValueError):
            moe.route_backward(x, ids, w, scale=scale)


def test_expert_times_leave_the_host_out(monkeypatch):
    """A host that is slow to enqueue (2 ms here) does not lengthen the device's time."""
    import time
    small = moe_layer.Layer(servers=2, gpus=1, tokens=3, experts=8, topk=2, hidden=256, inner=64, group=32)
    ids, w = moe.route(moe_layer.logits(small, 1), 2)
    own = moe.experts

    def slow(*a, **kw):
        time.sleep(0.002)
        return own(*a, **kw)

    monkeypatch.setattr(moe, "experts", slow)
    assert 0 < max(moe_layer.expert_ns(small, ids, w)) < 1_000_000
