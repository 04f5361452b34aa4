"""One decode step of a mixture-of-experts layer, from the router's logits to
the simulated exchange.

The pplx MoE page times dispatch and combine for a given routing; how the
router spreads the tokens decides both the traffic and which rank's experts
work longest.  Here the parts are run together: the router picks experts for
every rank's tokens (:func:`.moe.route`), their placement gives the bytes
from rank to rank (:func:`.moe.exchange`), each rank's experts do their work on
what the rank receives (:func:`.moe.experts`, timed on the device), and the
simulator steps dispatch, that work, and combine over a fabric
(:func:`.inputs.moe_workload`).  Routers are compared on the same logits:
free choice, choice within few groups (a group's experts share a server, so a
token's copies go to fewer servers), and a balance bias that :func:`balance`
moves from step to step.  Before the router stand the norm, the residual and the
router's product of the block (:func:`choose`, :func:`block_step`); their time, the
same for every router, is measured (:func:`dense_ns`) and is no part of the simulated
step, which begins with the dispatch.

    python -m experiment_network_simulation_gb300.moe_layer
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import inputs as I
from . import block, moe, mv


@dataclass
class Layer:
    """A layer over servers x gpus ranks, experts spread evenly over them."""
    servers: int = 8
    gpus: int = 8
    tokens: int = 4              # a rank's, in this step
    experts: int = 256
    topk: int = 8
    hidden: int = 7168
    inner: int = 2048
    group: int = 128             # columns a weight scale stands for

    def __post_init__(self):
        if self.experts % self.ranks:
            raise ValueError(f"{self.experts} experts do not spread evenly over {self.ranks} ranks")

    @property
    def ranks(self) -> int:
        return self.servers * self.gpus

    def place(self, device="cuda") -> torch.Tensor:
        """The rank of every expert: equal consecutive shares."""
        return (torch.arange(self.experts, device=device) * self.ranks // self.experts).int()


def logits(layer: Layer, seed: int = 0, zipf: float = 1.2, device="cuda") -> torch.Tensor:
    """Synthetic router logits of every rank's tokens: the log-popularity of a
    Zipf law over a seeded order of the experts, halved, plus a normal part."""
    g = torch.Generator(device=device).manual_seed(seed)
    order = torch.randperm(layer.experts, generator=g, device=device).float()
    x = torch.randn((layer.ranks * layer.tokens, layer.experts), generator=g, device=device)
    return x - 0.5 * zipf * torch.log(order + 1.0)


def balance(bias: torch.Tensor, load: torch.Tensor, step: float) -> torch.Tensor:
    """The bias after one step of balancing: up by ``step`` for experts below the
    mean load, down for those above."""
    load = load.float()
    return bias + step * torch.sign(load.mean() - load)


def traffic(layer: Layer, ids: torch.Tensor) -> tuple[np.ndarray, torch.Tensor]:
    """(bytes from rank to rank, load of every expert): 16-bit activations, one
    copy of a token to every rank that holds an expert of its."""
    load, sent = moe.exchange(ids, layer.place(ids.device), layer.ranks)
    return sent.cpu().numpy().astype(np.int64) * (2 * layer.hidden), load


def random_experts(layer: Layer, n: int, seed: int = 0, device="cuda") -> tuple:
    """Random weights of ``n`` experts, as :func:`.moe.experts` takes them."""
    g = torch.Generator(device=device).manual_seed(seed)
    h, i, c = layer.hidden, layer.inner, layer.group

    def q(*shape):
        return torch.randint(0, 256, shape, generator=g, device=device, dtype=torch.uint8)

    def s(k, *shape):
        return ((0.5 + torch.rand(shape, generator=g, device=device)) / (5 * k ** 0.5)).bfloat16()

    return q(n, 2 * i, h // 2), s(h, n, 2 * i, h // c), q(n, h, i // 2), s(i, n, h, i // c)


def expert_ns(layer: Layer, ids: torch.Tensor, weights: torch.Tensor, repeats: int = 5) -> list[int]:
    """Every rank's experts' work on the tokens it receives, in ns: the median
    of ``repeats`` device timings, L2 rewritten before each.  One set of random
    weights stands for every rank's.  A timing counts only if all of it was
    enqueued before the device came to it: else the device waited for the host,
    and L2 is rewritten more often the next time."""
    per = layer.experts // layer.ranks
    mats = random_experts(layer, per, device=ids.device)
    x = torch.randn((ids.shape[0], layer.hidden), device=ids.device).bfloat16()
    timer = _Timer(ids.device, repeats)
    out = []
    for r in range(layer.ranks):
        here = (ids >= r * per) & (ids < (r + 1) * per)
        rows = here.any(1).nonzero().flatten()
        if not rows.numel():
            out.append(0)
            continue
        local = torch.where(here, ids - r * per, -1)[rows].int().contiguous()
        mine, w = x[rows].contiguous(), weights[rows].contiguous()
        out.append(timer(lambda: moe.experts(mine, local, w, *mats)))
    return out


class _Timer:
    """Device time of a call in ns, as :func:`expert_ns` describes it."""

    def __init__(self, device, repeats: int):
        self.flush = torch.empty(1 << 28, dtype=torch.uint8, device=device)
        self.repeats, self.fills = repeats, 1

    def __call__(self, call) -> int:
        times = []
        while len(times) < self.repeats + 2:
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            for _ in range(self.fills):
                self.flush.zero_()
            a.record()
            call()
            b.record()
            late = a.query()
            b.synchronize()
            if not late:
                times.append(a.elapsed_time(b))
            elif self.fills < 1 << 12:
                self.fills *= 2
            else:
                raise RuntimeError("the host takes too long to enqueue the work")
        return int(1e6 * sorted(times[2:])[self.repeats // 2])


def dense(layer: Layer, seed: int = 0, device="cuda") -> dict:
    """Random weights of what a block does before its experts: the norm of the last
    branch, that branch's gate, the norm before this one, the router's matrix and bias."""
    g = torch.Generator(device=device).manual_seed(seed)

    def near(mean, *shape):
        return mean + 0.1 * torch.randn(shape, generator=g, device=device)

    return dict(post=near(1.0, layer.hidden), gate=near(0.5, layer.hidden), weight=near(1.0, layer.hidden),
                router=(torch.randn((layer.experts, layer.hidden), generator=g, device=device) * layer.hidden ** -0.5).bfloat16(),
                bias=near(0.0, layer.experts))


def choose(layer: Layer, d: dict, y: torch.Tensor, stream: torch.Tensor, **kw) -> tuple:
    """A block up to its dispatch, [tokens, hidden] bfloat16: the last branch's output
    ``y`` joins the ``stream``, which is normed and routed: (n, stream, ids, weights)."""
    n, stream = block.norm(y, d["weight"], residual=stream, post=d["post"], gate=d["gate"])
    logits = block.linear(n, d["router"], d["bias"], out_dtype=torch.float32)
    return (n, stream, *moe.route(logits, layer.topk, scores="sigmoid", **kw))


def block_step(layer: Layer, d: dict, mats: tuple, y: torch.Tensor, stream: torch.Tensor, **kw) -> tuple:
    """A block's decode step on one device that has all the experts: (y, stream) of the next."""
    n, stream, ids, weights = choose(layer, d, y, stream, **kw)
    return moe.experts(n, ids, weights, *mats), stream


def dense_ns(layer: Layer, repeats: int = 5, device="cuda") -> int:
    """What a rank's tokens take up to their dispatch, in ns (:func:`choose`)."""
    d = dense(layer, device=device)
    y, stream = (torch.randn((layer.tokens, layer.hidden), device=device).bfloat16() for _ in range(2))
    return _Timer(y.device, repeats)(lambda: choose(layer, d, y, stream))


def experiment(layer: Layer, byte: np.ndarray, compute_ns, gbps: int = 400, pkt: int = 4096) -> I.Experiment:
    """Dispatch, the experts' work and combine on a rail-optimised fabric."""
    tick = I.tick_ps(pkt, gbps)
    topo = I.rail_optimized(layer.servers, layer.gpus, layer.servers, max(1, layer.servers // 2),
                            I.delay_ticks(1_000_000, tick))
    work = I.moe_workload(byte, layer.gpus, max(1, -(-10_000_000 // tick)), compute_ns=compute_ns)
    return I.Experiment(topo, work, I.RING, 4, 512 * I.KIB, pkt, 64, tick)


def compare(layer: Layer, seed: int = 0, rounds: int = 40, step: float = 0.02) -> list[dict]:
    """Simulated step times of four routers on the same logits."""
    x = logits(layer, seed)
    limited = dict(groups=layer.servers, top_groups=max(1, layer.servers // 2), group_rule="top2")
    bias = torch.zeros(layer.experts, device=x.device)
    for _ in range(rounds):
        ids, _ = moe.route(x, layer.topk, scores="sigmoid", bias=bias)
        bias = balance(bias, traffic(layer, ids)[1], step)
    rows, exps = [], []
    for name, kw in [("free", {}), ("half of the servers", limited), ("balanced", dict(bias=bias)),
                     ("balanced, half of the servers", dict(bias=bias, **limited))]:
        ids, weights = moe.route(x, layer.topk, scores="sigmoid", **kw)
        byte, load = traffic(layer, ids)
        ns = expert_ns(layer, ids, weights)
        exps.append(experiment(layer, byte, ns))
        rows.append(dict(router=name, copies=int(byte.sum() // (2 * layer.hidden)),
                         busiest_load=float(load.max() / load.float().mean()), busiest_ns=max(ns),
                         tick_ps=exps[-1].tick_ps))
    res = mv.simulate(I.Batch(exps, "moe-decode-step").pack())
    for row, status, end in zip(rows, res["status"], res["end_tick"]):
        row["done"] = int(status) == mv.EXP_DONE
        row["step_us"] = (int(end) + 1) * row.pop("tick_ps") / 1e6
    return rows


if __name__ == "__main__":
    print(f"norm, logits and choice of a rank's tokens before dispatch: {dense_ns(Layer()) / 1e3:.1f} us")
    for row in compare(Layer()):
        print(f"{row['router']:32s} {row['copies']:6d} copies, busiest expert {row['busiest_load']:4.1f} x "
              f"the mean, experts' work {row['busiest_ns'] / 1e3:6.1f} us at most, step {row['step_us']:8.1f} us")
