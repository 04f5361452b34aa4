"""Routed-expert operators without a GPU: what the C entry points refuse (all
checked on the host before anything is launched), the Python binding's
refusal of host tensors, and the plain 64-bit code against hand values."""
import ctypes as C

import numpy as np
import pytest
import torch

import moe_reference as R
from experiment_network_simulation_gb300 import moe, mv

P = 0x10000          # an aligned address that is only looked at


def route_desc(**kw):
    f = dict(tokens=4, row_stride=16, experts=16, topk=2, groups=4, top_groups=2, dtype=0,
             scores=0, group_rule=0, renorm=1, scale=1.0, logits=P, bias=None, ids=P, weights=P)
    return moe.RouteDesc(**{**f, **kw})


def test_route_refuses():
    f = moe._library().mv_route
    assert f(None, None) == mv.MV_EINVAL
    assert f(C.byref(route_desc(tokens=0, logits=None, ids=None, weights=None)), None) == mv.MV_OK
    for kw in (dict(experts=0), dict(topk=0), dict(topk=17), dict(topk=9), dict(groups=0),
               dict(groups=3), dict(groups=33, experts=33), dict(top_groups=0), dict(top_groups=5),
               dict(dtype=3), dict(scores=2), dict(group_rule=2), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(logits=None), dict(ids=None), dict(weights=None),
               dict(row_stride=15), dict(logits=P + 2), dict(bias=P + 1), dict(ids=P + 2),
               dict(weights=P + 1), dict(dtype=1, logits=P + 1)):
        assert f(C.byref(route_desc(**kw)), None) == mv.MV_EINVAL, kw
    for kw in (dict(experts=1028, row_stride=1028), dict(experts=256, row_stride=256, topk=33),
               dict(tokens=1 << 41), dict(row_stride=1 << 32)):
        assert f(C.byref(route_desc(**kw)), None) == mv.MV_EOVERFLOW, kw


def test_route_backward_refuses():
    f = moe._library().mv_route_backward
    base = dict(tokens=4, row_stride=16, experts=16, topk=2, dtype=1, scores=1, renorm=0, scale=1.0,
                logits=P, ids=P, dweights=P, dlogits=P)
    d = lambda **kw: C.byref(moe.RouteGradDesc(**{**base, **kw}))  # noqa: E731
    assert f(None, None) == mv.MV_EINVAL
    assert f(d(tokens=0, logits=None), None) == mv.MV_OK
    for kw in (dict(experts=0), dict(topk=0), dict(topk=17), dict(dtype=9), dict(scores=2),
               dict(scale=float("nan")), dict(logits=None), dict(ids=None), dict(dweights=None),
               dict(dlogits=None), dict(row_stride=3), dict(dlogits=P + 1), dict(ids=P + 1)):
        assert f(d(**kw), None) == mv.MV_EINVAL, kw
    assert f(d(experts=1025, row_stride=1025), None) == mv.MV_EOVERFLOW
    assert f(d(experts=64, row_stride=64, topk=33), None) == mv.MV_EOVERFLOW


def test_exchange_refuses():
    f = moe._library().mv_exchange
    base = dict(batches=2, tokens=12, topk=2, experts=8, sources=4, ranks=4, once=1, ids=P, place=P,
                starts=None, load=P, sent=P)
    d = lambda **kw: C.byref(moe.ExchangeDesc(**{**base, **kw}))  # noqa: E731
    assert f(None, None) == mv.MV_EINVAL
    assert f(d(batches=0, ids=None), None) == mv.MV_OK
    for kw in (dict(experts=0), dict(topk=0), dict(sources=0), dict(ranks=0), dict(sources=5),
               dict(ids=None), dict(place=None), dict(load=None), dict(sent=None), dict(ids=P + 1),
               dict(starts=P + 4), dict(sent=P + 2)):
        assert f(d(**kw), None) == mv.MV_EINVAL, kw
    for kw in (dict(experts=1025), dict(topk=33), dict(ranks=8193), dict(tokens=1 << 31),
               dict(tokens=1 << 30), dict(sources=(1 << 24) + 4), dict(batches=(1 << 24) + 1),
               dict(batches=1 << 24, sources=1 << 24, tokens=1 << 24)):
        assert f(d(**kw), None) == mv.MV_EOVERFLOW, kw


def test_experts_refuse():
    lib = moe._library()
    base = dict(tokens=4, row_stride=128, topk=2, experts=8, hidden=128, inner=64, group=64, dtype=2,
                x=P, ids=P, weights=P, w13=P, s13=P, w2=P, s2=P, y=P)
    d = lambda **kw: C.byref(moe.ExpertsDesc(**{**base, **kw}))  # noqa: E731
    need = C.c_uint64(0)
    size = lambda **kw: lib.mv_experts_workspace_bytes(d(**kw), C.byref(need))  # noqa: E731
    assert size() == mv.MV_OK and need.value > 0 and need.value % 256 == 0
    assert lib.mv_experts_workspace_bytes(d(), None) == mv.MV_EINVAL
    assert lib.mv_experts_workspace_bytes(None, C.byref(need)) == mv.MV_EINVAL
    for kw in (dict(experts=0), dict(topk=0), dict(dtype=0), dict(dtype=3), dict(group=16),
               dict(group=48), dict(hidden=0), dict(inner=0), dict(hidden=96), dict(inner=96)):
        assert size(**kw) == mv.MV_EINVAL and need.value == 0, kw
    for kw in (dict(experts=1025), dict(topk=33), dict(hidden=1 << 21), dict(inner=1 << 21),
               dict(tokens=(1 << 24) + 1), dict(row_stride=1 << 32)):
        assert size(**kw) == mv.MV_EOVERFLOW, kw
    assert size() == mv.MV_OK
    run = lambda ws=P, n=need.value, **kw: lib.mv_experts(d(**kw), ws, n, None)  # noqa: E731
    assert run(tokens=0, x=None, ws=None, n=0) == mv.MV_OK
    assert run(n=need.value - 1) == mv.MV_ENOMEM
    for kw in (dict(ws=None), dict(ws=P + 16), dict(x=None), dict(ids=None), dict(weights=None),
               dict(w13=None), dict(s13=None), dict(w2=None), dict(s2=None), dict(y=None),
               dict(row_stride=64), dict(row_stride=129), dict(x=P + 2), dict(w13=P + 8),
               dict(y=P + 8), dict(ids=P + 2)):
        assert run(**kw) == mv.MV_EINVAL, kw


def test_host_tensors_are_refused():
    x = torch.zeros((4, 8))
    with pytest.raises(RuntimeError, match="no CPU fallback"):
        moe.route(x, 2)
    with pytest.raises(ValueError):
        moe.route([[0.0]], 1)
    with pytest.raises(RuntimeError):
        moe.exchange(torch.zeros((4, 2), dtype=torch.int32), torch.zeros(8, dtype=torch.int32), 2)


def test_reference_route_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [8.0, 8.0, 1.0, 1.0]]))
    ids, w, _ = R.route(x, 2)
    assert ids.tolist() == [[2, 1], [0, 1]] and np.allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]])
    ids, w, _ = R.route(x, 2, renorm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5], [16 / 18, 16 / 18]])
    # a bias moves the choice, not the weight
    ids, w, _ = R.route(x[:1], 2, bias=[1.0, 0, 0, 0], renorm=False)
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[1 / 8, 1 / 2]])
    # groups {1, 2} and {4, 1}: by their best the second stays, row 2 the first
    ids, _, _ = R.route(x, 2, groups=2, top_groups=1)
    assert ids.tolist() == [[2, 3], [0, 1]]
    y = np.log(np.array([[3.0, 3.0, 4.0, 1.0]]))
    assert R.route(y, 2, groups=2, top_groups=1)[0].tolist() == [[2, 3]]
    assert R.route(y, 2, groups=2, top_groups=1, group_rule="top2")[0].tolist() == [[0, 1]]
    x[0, 1:] = -np.inf
    ids, w, _ = R.route(x[:1], 3, scores="sigmoid")
    assert ids.tolist() == [[0, -1, -1]] and w.tolist() == [[1.0, 0.0, 0.0]]


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False),
                                           ("sigmoid", True), ("sigmoid", False)])
def test_reference_gradient_by_differences(scores, renorm):
    rng = np.random.default_rng(1)
    x, g = rng.normal(size=(3, 9)), rng.normal(size=(3, 4))
    ids = R.route(x, 4, scores)[0]
    dx = R.route_backward(x, ids, g, scores, renorm, 2.5)
    for t in range(3):
        for e in range(9):
            d = np.zeros(9)
            d[e] = 1e-5
            num = (R.weights_of(x[t] + d, ids[t], scores, renorm, 2.5)
                   - R.weights_of(x[t] - d, ids[t], scores, renorm, 2.5)) / 2e-5
            assert abs((num * g[t]).sum() - dx[t, e]) < 1e-8


def test_reference_exchange_and_experts_by_hand():
    ids = np.array([[[0, 1], [2, 0]], [[1, 1], [-1, 3]]], np.int32)
    load, sent = R.exchange(ids, np.array([0, 0, 1]), 2, once=True)
    assert load.tolist() == [[2, 1, 1], [0, 2, 0]]
    assert sent.tolist() == [[[1, 0], [1, 1]], [[1, 0], [0, 0]]]
    assert R.exchange(ids, np.array([0, 0, 1]), 2, once=False)[1].tolist() == [
        [[2, 0], [1, 1]], [[2, 0], [0, 0]]]
    w = R.unpack(np.array([[0x90, 0x7F]], np.uint8), np.array([[0.5, 2.0]]), 2)
    assert w.tolist() == [[-4.0, 0.5, 14.0, -2.0]]
