"""A decode step of a mixture-of-experts layer, router to simulated exchange:
the operators' traffic is the simulator's input, and the simulation of it
equals the oracle's."""
import numpy as np
import pytest

import moe_reference as R
from experiment_network_simulation_gb300 import inputs as I
from oracle import oracle as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import moe, moe_layer, mv  # noqa: E402
from test_gpu_parity import assert_same  # noqa: E402

SMALL = moe_layer.Layer(servers=4, gpus=4, tokens=3, experts=32, topk=4, hidden=256, inner=64, group=32)


def test_traffic_of_the_router_simulates_like_the_oracle():
    x = moe_layer.logits(SMALL, 1)
    exps = []
    for kw in ({}, dict(groups=4, top_groups=2, group_rule="top2")):
        ids, w = moe.route(x, SMALL.topk, scores="sigmoid", **kw)
        byte, load = moe_layer.traffic(SMALL, ids)
        place = SMALL.place().cpu().numpy()
        want = R.exchange(ids.cpu().numpy()[None], place, SMALL.ranks)
        assert np.array_equal(byte, want[1][0].astype(np.int64) * 512)
        assert np.array_equal(load.cpu().numpy(), want[0][0])
        if kw:                                       # a token's copies go to two servers at most
            servers = ids.cpu().numpy() // 8
            assert max(len(set(row)) for row in servers) <= 2
        exps.append(moe_layer.experiment(SMALL, byte, [2000 + 100 * r for r in range(SMALL.ranks)]))
    packed = I.Batch(exps).pack()
    got = mv.simulate(packed)
    assert (got["status"] == mv.EXP_DONE).all()
    assert_same(got, O.run(packed))


def test_balance_evens_the_load():
    x = moe_layer.logits(SMALL, 2)
    bias = torch.zeros(32, device="cuda")
    free = moe_layer.traffic(SMALL, moe.route(x, 4, scores="sigmoid")[0])[1].float()
    for _ in range(60):
        ids, _ = moe.route(x, 4, scores="sigmoid", bias=bias)
        bias = moe_layer.balance(bias, moe_layer.traffic(SMALL, ids)[1], 0.02)
    even = moe_layer.traffic(SMALL, moe.route(x, 4, scores="sigmoid", bias=bias)[0])[1].float()
    assert free.sum() == even.sum() == 16 * 3 * 4
    assert even.std() < 0.6 * free.std() and even.max() < free.max()


def test_compare_runs_every_router():
    rows = moe_layer.compare(SMALL, rounds=5)
    assert len(rows) == 4 and all(r["done"] and r["step_us"] > 0 and r["busiest_ns"] > 0 for r in rows)
    with pytest.raises(ValueError):
        moe_layer.Layer(experts=100)
