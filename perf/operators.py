"""The routed-expert operators as they are measured: inputs, plain forms and the framework's calls.

Four operators of a mixture-of-experts layer: ``route`` (scores, groups,
top-k, weights), ``route_backward`` (its gradient), ``exchange`` (how many
tokens every rank sends to every other, what the simulator's all-to-all takes)
and ``experts`` (the SwiGLU products of the chosen experts, 4-bit weights with
group scales).  ``run`` computes them with elementary torch operations, or,
where ``own`` is true, with the framework's calls on the same inputs.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def _route(tokens, experts, topk, dtype, scores, bias=False, groups=1, top_groups=1,
           rule="max", renorm=True, scale=1.0, pad=0, **kw):
    return dict(op="route", tokens=tokens, experts=experts, topk=topk, dtype=dtype, scores=scores,
                bias=bias, groups=groups, top_groups=top_groups, rule=rule, renorm=renorm,
                scale=scale, pad=pad, **kw)


def _backward(tokens, experts, topk, dtype, scores, renorm, scale=1.0, **kw):
    return dict(op="backward", tokens=tokens, experts=experts, topk=topk, dtype=dtype,
                scores=scores, renorm=renorm, scale=scale, **kw)


def _exchange(batch, ranks, tokens, experts, topk, once, ragged=False, **kw):
    return dict(op="exchange", batch=batch, ranks=ranks, tokens=tokens, experts=experts,
                topk=topk, once=once, ragged=ragged, **kw)


def _experts(tokens, topk, experts, total, hidden, inner, group, dtype, **kw):
    return dict(op="experts", tokens=tokens, topk=topk, experts=experts, total=total,
                hidden=hidden, inner=inner, group=group, dtype=dtype, **kw)


def listed():
    return [
        # one token of a decode step: launch and latency only
        _route(1, 256, 8, "f32", "sigmoid", bias=True, groups=8, top_groups=4, rule="top2",
               scale=2.5, name="route 1x256 sigmoid groups"),
        # a prefill batch through a small layer, odd sizes, with padding rows that route nowhere
        _route(4099, 60, 4, "bf16", "softmax", renorm=False, pad=77, name="route 4099x60 softmax"),
        # one experiment of the MoE workload: 512 ranks x 128 tokens, balanced by a bias
        _route(65536, 256, 8, "f32", "sigmoid", bias=True, groups=8, top_groups=4, rule="top2",
               scale=2.5, name="route 65536x256 sigmoid groups"),
        # sixteen experiments' tokens at once, plain softmax routing
        _route(1 << 20, 256, 8, "bf16", "softmax", name="route 1048576x256 softmax"),
        # a training step's micro-batch: the dense gradient, and the one of the chosen alone
        _backward(65536, 256, 8, "f32", "softmax", False, name="backward 65536x256 softmax"),
        _backward(8191, 160, 6, "bf16", "sigmoid", True, scale=2.5,
                  name="backward 8191x160 sigmoid"),
        # a decode step over 64 ranks with uneven batches, some of them empty
        _exchange(1, 64, 64 * 37, 256, 8, True, ragged=True, name="exchange 64 ranks ragged"),
        # the MoE workload's traffic for 64 router seeds
        _exchange(64, 512, 512 * 128, 256, 8, False, name="exchange 64x512 ranks"),
        # one token through its eight experts
        _experts(1, 8, 64, 64, 7168, 2048, 128, "bf16", name="experts 1 token"),
        # a few tokens, small layer, the finest scales, odd counts
        _experts(7, 4, 33, 33, 2880, 1440, 32, "f16", name="experts 7 tokens group 32"),
        # a decode batch on a rank that holds 32 of 256 experts
        _experts(64, 8, 32, 256, 7168, 2048, 128, "bf16", name="experts 64 tokens 32 of 256"),
        # a larger batch over a layer of many narrow experts: about twenty tokens each
        _experts(200, 6, 60, 60, 2048, 1408, 64, "bf16", name="experts 200 tokens narrow"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """An odd number of groups: the last tile is not a whole one."""
    return 2 * rng.randint(lo // 2, (hi - 1) // 2) + 1


def draw(rng):
    op = rng.choice(["route", "route", "backward", "exchange", "experts", "experts"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "route":
        tokens = _log(rng, 1, 250_000)
        topk = rng.randint(1, 10)
        scores = rng.choice(["softmax", "sigmoid"])
        scale = rng.choice([1.0, 2.5])
        if rng.random() < 0.5:
            groups = rng.choice([2, 4, 8])
            experts = groups * rng.randint(4, 32)
            tg = rng.randint(1, groups)
            topk = min(topk, tg * (experts // groups))
            bias = scores == "sigmoid" and rng.random() < 0.7
            return _route(tokens, experts, topk, dtype, scores, bias=bias, groups=groups,
                          top_groups=tg, rule="top2" if bias else "max",
                          renorm=rng.random() < 0.7, scale=scale, pad=rng.choice([0, tokens // 9]))
        experts = _log(rng, topk, 512)
        bias = scores == "sigmoid" and rng.random() < 0.5
        return _route(tokens, experts, topk, dtype, scores, bias=bias,
                      renorm=rng.random() < 0.7, scale=scale, pad=rng.choice([0, tokens // 9]))
    if op == "backward":
        experts = _log(rng, 8, 512)
        topk = rng.randint(1, min(10, experts))
        return _backward(_log(rng, 1, 32768), experts, topk, dtype,
                         rng.choice(["softmax", "sigmoid"]),
                         topk > 1 and rng.random() < 0.5,      # one choice: always the whole weight
                         scale=rng.choice([1.0, 2.5]))
    if op == "exchange":
        ranks = _log(rng, 2, 512)
        experts = _log(rng, 16, 256)
        return _exchange(_log(rng, 1, 32), ranks, ranks * _log(rng, 1, 128), experts,
                         rng.randint(1, 8), rng.random() < 0.5, ragged=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    experts, tokens = rng.randint(4, 36), _log(rng, 1, 64)
    topk = rng.randint(1, min(8, experts))
    elsewhere = tokens * topk >= 32 and rng.random() < 0.33
    return _experts(tokens, topk, experts, experts * (4 if elsewhere else 1),
                    group * _odd(rng, 4, 5120 // group), group * _odd(rng, 2, 2048 // group),
                    group, rng.choice(["bf16", "f16"]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _popularity(experts, g):
    """Log-popularity of the experts: Zipf(1.2) over a seeded order."""
    order = torch.randperm(experts, generator=g, device="cuda").float()
    return -1.2 * torch.log(order + 1.0)


def _gumbel(shape, g):
    u = torch.rand(shape, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7)
    return u.log_().neg_().log_().neg_()


def _logits(c, g):
    """Router logits: half the log-popularity, plus what the token adds."""
    x = torch.randn((c["tokens"], c["experts"]), generator=g, device="cuda")
    x += 0.5 * _popularity(c["experts"], g)
    if c.get("pad"):
        x[c["tokens"] - c["pad"]:] = -math.inf
    return x.to(DTYPES[c["dtype"]])


def _choices(tokens, topk, experts, pop, g):
    """[tokens, topk] distinct experts by Gumbel top-k."""
    out = torch.empty((tokens, topk), dtype=torch.int32, device="cuda")
    for a in range(0, tokens, 1 << 20):
        n = min(1 << 20, tokens - a)
        out[a:a + n] = (_gumbel((n, experts), g) + pop).topk(topk, dim=1).indices
    return out


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "route":
        s["logits"] = _logits(c, g)
        s["bias"] = 0.05 * torch.randn(c["experts"], generator=g, device="cuda") if c["bias"] else None
    elif c["op"] == "backward":
        s["logits"] = _logits(c, g)
        s["ids"] = s["logits"].float().topk(c["topk"], dim=1).indices.int()
        s["dweights"] = torch.randn((c["tokens"], c["topk"]), generator=g, device="cuda")
    elif c["op"] == "exchange":
        b, t, r = c["batch"], c["tokens"], c["ranks"]
        topk = min(c["topk"], c["experts"])
        s["ids"] = _choices(b * t, topk, c["experts"], _popularity(c["experts"], g), g).view(b, t, topk)
        s["place"] = (torch.arange(c["experts"], device="cuda") * r // c["experts"]).int()
        s["starts"] = None
        if c["ragged"]:      # uneven batches a rank, some of them empty
            cuts = torch.randint(0, t + 1, (r - 1,), generator=g, device="cuda").sort().values
            s["starts"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), t)])
    else:
        e, h, i, n = c["experts"], c["hidden"], c["inner"], c["group"]
        dt = DTYPES[c["dtype"]]
        ids = _choices(c["tokens"], c["topk"], c["total"], 0.0, g)
        s["ids"] = torch.where(ids < e, ids, -1)         # experts of other ranks are not here
        w = torch.rand((c["tokens"], c["topk"]), generator=g, device="cuda") + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["x"] = torch.randn((c["tokens"], h), generator=g, device="cuda").to(dt)
        nib = lambda *d: torch.randint(0, 256, d, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
        sc = lambda k, *d: ((0.5 + torch.rand(d, generator=g, device="cuda")) / (5 * math.sqrt(k))).to(dt)  # noqa: E731
        s["w13"], s["s13"] = nib(e, 2 * i, h // 2), sc(h, e, 2 * i, h // n)
        s["w2"], s["s2"] = nib(e, h, i // 2), sc(i, e, h, i // n)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c)


def _plain_route(s, c):
    x, b, k = s["logits"].float(), s["bias"], c["topk"]
    T, E = x.shape
    closed = (x == -math.inf) | x.isnan()
    x = x.masked_fill(closed, -math.inf)
    if c["scores"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        m = x.amax(1, keepdim=True)
        score = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
        score = score / score.sum(1, keepdim=True)
    # without a bias the score's order is the logit's
    v = x if b is None and c["rule"] == "max" else score if b is None else score + b
    v = v.masked_fill(closed, -math.inf)
    if c["groups"] > 1:
        gv = v.view(T, c["groups"], -1)
        if c["rule"] == "max":
            best = gv.amax(2)
        else:
            two = gv.sort(dim=2, descending=True).values[:, :, :2]
            best = two[:, :, 0] + two[:, :, 1].masked_fill(two[:, :, 1] == -math.inf, 0.0)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stays = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        v = gv.masked_fill(~stays[:, :, None], -math.inf).view(T, E)
    v, ids = v.sort(dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    none = v == -math.inf
    if c["renorm"] and c["scores"] == "softmax":
        y = x.gather(1, ids).masked_fill(none, -math.inf)
        m = y.amax(1, keepdim=True)
        w = torch.exp(y - m.masked_fill(m == -math.inf, 0.0))
    else:
        w = score.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / total.masked_fill(total == 0, 1.0)
    return ids.masked_fill(none, -1).int(), w * c["scale"]


def _plain_backward(s, c):
    x, g, ids = s["logits"].float(), s["dweights"], s["ids"].long()
    if c["scores"] == "softmax" and not c["renorm"]:
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        dot = (g * p.gather(1, ids)).sum(1, keepdim=True)
        dx = p * (torch.zeros_like(p).scatter_(1, ids, g) - dot) * c["scale"]
        return dx.to(s["logits"].dtype)
    y = x.gather(1, ids)
    if c["scores"] == "softmax":
        w = torch.exp(y - y.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        d = w * (g - (g * w).sum(1, keepdim=True)) * c["scale"]
    else:
        sg = 1.0 / (1.0 + torch.exp(-y))
        d = g
        if c["renorm"]:
            total = sg.sum(1, keepdim=True)
            d = (g - (g * sg).sum(1, keepdim=True) / total) / total
        d = d * sg * (1.0 - sg) * c["scale"]
    return torch.zeros_like(x).scatter_(1, ids, d).to(s["logits"].dtype)


def _plain_exchange(s, c):
    ids, place, R = s["ids"].long(), s["place"].long(), c["ranks"]
    B, T, k = ids.shape
    E = place.numel()
    batch = torch.arange(B, device="cuda")[:, None, None]
    load = torch.bincount((batch * E + ids).view(-1), minlength=B * E).view(B, E)
    token = torch.arange(T, device="cuda")
    if s["starts"] is None:
        src = token // (T // R)
    else:
        src = torch.searchsorted(s["starts"][1:], token, right=True)
    dst = place[ids]
    cell = (batch * R + src[None, :, None]) * R + dst
    if c["once"]:            # a token goes to a rank once, however many of its experts live there
        same = dst[:, :, :, None] == dst[:, :, None, :]
        first = ~(same & torch.ones(k, k, dtype=torch.bool, device="cuda").tril(-1)).any(3)
        cell = torch.where(first, cell, B * R * R)
    sent = torch.bincount(cell.view(-1), minlength=B * R * R + 1)[:B * R * R].view(B, R, R)
    return load.int(), sent.int()


def _unpack(q, scale):
    """(q - 8) * scale of packed 4-bit rows; the low half of a byte comes first."""
    w = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float().sub_(8.0)
    return w.view(*scale.shape, -1).mul_(scale.float()[..., None]).view(w.shape)


def _plain_experts(s, c):
    x, ids, I = s["x"].float(), s["ids"].long(), c["inner"]
    seen, at = torch.unique(torch.cat([ids.new_full((1,), -1), ids.view(-1)]), return_inverse=True)
    seen, at = seen[1:], at[1:].view_as(ids)                     # at: 0 for no expert of this rank
    z = x @ _unpack(s["w13"][seen], s["s13"][seen]).transpose(1, 2)   # these experts, every token
    h = z[:, :, :I] / (1.0 + torch.exp(-z[:, :, :I])) * z[:, :, I:]
    o = h @ _unpack(s["w2"][seen], s["s2"][seen]).transpose(1, 2)
    w = torch.zeros((x.shape[0], seen.numel() + 1), device="cuda")
    w.scatter_add_(1, at, s["weights"])
    return (o * w[:, 1:].t()[:, :, None]).sum(0).to(s["x"].dtype)


_plain = {"route": _plain_route, "backward": _plain_backward, "exchange": _plain_exchange,
          "experts": _plain_experts}


def _own_route(s, c):
    from experiment_network_simulation_gb300 import moe
    return moe.route(s["logits"], c["topk"], scores=c["scores"], bias=s["bias"],
                     groups=c["groups"], top_groups=c["top_groups"], group_rule=c["rule"],
                     renorm=c["renorm"], scale=c["scale"])


def _own_backward(s, c):
    from experiment_network_simulation_gb300 import moe
    return moe.route_backward(s["logits"], s["ids"], s["dweights"], scores=c["scores"],
                              renorm=c["renorm"], scale=c["scale"])


def _own_exchange(s, c):
    from experiment_network_simulation_gb300 import moe
    return moe.exchange(s["ids"], s["place"], c["ranks"], starts=s["starts"], once=c["once"])


def _own_experts(s, c):
    from experiment_network_simulation_gb300 import moe
    return moe.experts(s["x"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"])


_own = {"route": _own_route, "backward": _own_backward, "exchange": _own_exchange,
        "experts": _own_experts}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(c):
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["topk"]
        return {"bytes": t * e * SIZE[c["dtype"]] + 4 * e * c["bias"] + 8 * t * k,
                "flops": 6.0 * t * e}
    if c["op"] == "backward":
        t, e, k, b = c["tokens"], c["experts"], c["topk"], SIZE[c["dtype"]]
        dense = c["scores"] == "softmax" and not c["renorm"]
        return {"bytes": t * e * b + 8 * t * k + (t * e if dense else t * k) * b,
                "flops": (8.0 * t * e) if dense else 12.0 * t * k}
    if c["op"] == "exchange":
        b, t, r, e = c["batch"], c["tokens"], c["ranks"], c["experts"]
        k = min(c["topk"], e)
        return {"bytes": 4 * (b * t * k + b * e + b * r * r + e), "flops": 2.0 * b * t * k}
    t, k, h, i = c["tokens"], c["topk"], c["hidden"], c["inner"]
    visited = c["experts"] * (1.0 - (1.0 - k / c["total"]) ** t)     # expected, uniform choices
    each = 3 * h * i / 2 + 3 * h * i / c["group"] * 2
    here = t * k * c["experts"] / c["total"]
    return {"bytes": visited * each + 4 * t * h + 8 * t * k, "flops": 6.0 * here * h * i}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return _exact[c["op"]](s, c)


def _exact_route(s, c):
    parts = []
    for x in s["logits"].double().split(1 << 17):
        n, E = x.shape
        is_open = x > -math.inf
        if c["scores"] == "sigmoid":
            score = torch.sigmoid(x)
        else:
            score = torch.softmax(torch.where(is_open.any(1, keepdim=True), x, 0.0), dim=1)
        if s["bias"] is not None:
            v = score + s["bias"].double()
        else:
            v = score if c["rule"] == "top2" else x
        v = torch.where(is_open, v, -math.inf)
        if c["groups"] > 1:
            size = E // c["groups"]
            gv = v.reshape(n, c["groups"], size)
            first = gv.max(2).values
            if c["rule"] == "top2" and size > 1:
                second = gv.topk(2, dim=2).values[:, :, 1]
                first = first + torch.where(second > -math.inf, second, 0.0)
            # a group stays if fewer than top_groups come before it
            idx = torch.arange(c["groups"], device=x.device)
            before = (first[:, None, :] > first[:, :, None]) | (
                (first[:, None, :] == first[:, :, None]) & (idx[None, :] < idx[:, None]))
            stays = before.sum(2) < c["top_groups"]
            v = torch.where(stays.repeat_interleave(size, dim=1), v, -math.inf)
        order = torch.argsort(-v, dim=1, stable=True)[:, :c["topk"]]
        chosen = torch.gather(v, 1, order) > -math.inf
        if c["renorm"] and c["scores"] == "softmax":
            y = torch.where(chosen, torch.gather(x, 1, order), -math.inf)
            w = torch.softmax(torch.where(chosen.any(1, keepdim=True), y, 0.0), dim=1)
        else:
            w = torch.gather(score, 1, order)
            if c["renorm"]:
                w = w / torch.where(chosen, w, 0.0).sum(1, keepdim=True).clamp_min(1e-300)
        parts.append((torch.where(chosen, order, -1), torch.where(chosen, w, 0.0) * c["scale"]))
    return torch.cat([p[0] for p in parts]).int(), torch.cat([p[1] for p in parts])


def _exact_backward(s, c):
    """The Jacobian of the weights, written as weight = scale * f(chosen scores)."""
    out = []
    for x, ids, g in zip(s["logits"].double().split(1 << 16), s["ids"].long().split(1 << 16),
                         s["dweights"].double().split(1 << 16)):
        x = x.requires_grad_(True)
        sc = torch.sigmoid(x) if c["scores"] == "sigmoid" else torch.softmax(x, dim=1)
        w = torch.gather(sc, 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        out.append(torch.autograd.grad((w * c["scale"] * g).sum(), x)[0])
    return torch.cat(out)


def _exact_exchange(s, c):
    ids, place = s["ids"].cpu().numpy(), s["place"].cpu().numpy()
    B, T, k = ids.shape
    if B * T * k > 4_000_000:
        return None
    R, E = c["ranks"], c["experts"]
    starts = (np.arange(R + 1) * (T // R) if s["starts"] is None else s["starts"].cpu().numpy())
    load, sent = np.zeros((B, E), np.int32), np.zeros((B, R, R), np.int32)
    for b in range(B):
        load[b] = np.bincount(ids[b].ravel(), minlength=E)
        for r in range(R):
            rows = place[ids[b, starts[r]:starts[r + 1]]]
            for row in rows:
                d, n = np.unique(row, return_counts=True)
                sent[b, r, d] += 1 if c["once"] else n.astype(np.int32)
    return load, sent


def _exact_experts(s, c):
    x, ids, wt = s["x"].double(), s["ids"], s["weights"].double()
    y = torch.zeros_like(x)
    n, I = c["group"], c["inner"]

    def matrix(q, scale):
        w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
        w[:, 0::2] = (q % 16).double() - 8
        w[:, 1::2] = (q // 16).double() - 8
        return w * scale.double().repeat_interleave(n, dim=1)

    for e in range(c["experts"]):
        at = (ids == e).nonzero()
        if at.numel():
            t, j = at[:, 0], at[:, 1]
            z = x[t] @ matrix(s["w13"][e], s["s13"][e]).t()
            h = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
            y.index_add_(0, t, wt[t, j][:, None] * (h @ matrix(s["w2"][e], s["s2"][e]).t()))
    return y


_exact = {"route": _exact_route, "backward": _exact_backward, "exchange": _exact_exchange,
          "experts": _exact_experts}
