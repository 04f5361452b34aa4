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
moves from step to step.

    python -m experiment_network_simulation_gb300.moe_layer
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import inputs as I
from . import moe, mv


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
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=ids.device)
    out, fills = [], 1
    for r in range(layer.ranks):
        here = (ids >= r * per) & (ids < (r + 1) * per)
        rows = here.any(1).nonzero().flatten()
        if not rows.numel():
            out.append(0)
            continue
        local = torch.where(here, ids - r * per, -1)[rows].int().contiguous()
        mine, w = x[rows].contiguous(), weights[rows].contiguous()
        times = []
        while len(times) < repeats + 2:
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            for _ in range(fills):
                flush.zero_()
            a.record()
            moe.experts(mine, local, w, *mats)
            b.record()
            late = a.query()
            b.synchronize()
            if not late:
                times.append(a.elapsed_time(b))
            elif fills < 1 << 12:
                fills *= 2
            else:
                raise RuntimeError("the host takes too long to enqueue the experts' work")
        out.append(int(1e6 * sorted(times[2:])[repeats // 2]))
    return out


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
    for row in compare(Layer()):
        print(f"{row['router']:32s} {row['copies']:6d} copies, busiest expert {row['busiest_load']:4.1f} x "
              f"the mean, experts' work {row['busiest_ns'] / 1e3:6.1f} us at most, step {row['step_us']:8.1f} us")
