"""Blocks of a decode step in a row: norm, residual and gate, the router's product and
choice, the experts, as the command that simulates a decode step has them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from experiment_network_simulation_gb300 import moe_layer as L  # noqa: E402

LAYER = L.Layer(servers=2, gpus=2, tokens=3, experts=16, topk=4, hidden=512, inner=256, group=64)


def plain_choose(d, y, stream):
    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    d = {k: v.double() for k, v in d.items()}
    r = stream.double() + d["gate"] * rms(y.double(), d["post"])
    return rms(r, d["weight"]), r, d


@pytest.mark.parametrize("tokens", [1, 12, 300])
def test_choose_against_64_bits(tokens):
    """n and the stream are rounded once, the logits come from the rounded n; a choice is
    compared where the scores it is between differ by more than 2^-14 (logits to 2^-15)."""
    d = L.dense(LAYER, seed=3)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    y, stream = (torch.randn((tokens, LAYER.hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    n, r, ids, weights = L.choose(LAYER, d, y, stream)
    wn, wr, e = plain_choose(d, y, stream)
    for got, want in ((n, wn), (r, wr)):
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16).all()
    score = torch.sigmoid(n.double() @ e["router"].t() + e["bias"])
    best = score.sort(dim=1, descending=True)
    gap = (best.values[:, :LAYER.topk] - best.values[:, 1:LAYER.topk + 1]).amin(1)
    sure = gap > 2.0 ** -14
    assert 2 * sure.sum() >= tokens
    assert torch.equal(ids[sure].long(), best.indices[sure, :LAYER.topk])
    chosen = score.gather(1, ids.long())
    assert ((weights.double() - chosen / chosen.sum(1, keepdim=True)).abs() <= 2.0 ** -14).all()


def test_blocks_in_a_row_and_in_a_graph():
    """Four blocks: a captured step replays to the eager result, and the stream goes on."""
    mats = L.random_experts(LAYER, LAYER.experts)
    ds = [L.dense(LAYER, seed=s) for s in range(4)]

    def run(y, stream):
        for d in ds:
            y, stream = L.block_step(LAYER, d, mats, y, stream)
        return y, stream

    g = torch.Generator(device="cuda").manual_seed(1)
    x, start = (torch.randn((5, LAYER.hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = run(x, start)
    assert want[0].isfinite().all() and want[1].isfinite().all() and not torch.equal(want[1], start)
    static = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(static, start)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(static, start)
    for _ in range(3):
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_dense_ns():
    assert 0 < L.dense_ns(LAYER, repeats=3) < 10_000_000
