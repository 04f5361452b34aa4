"""The block operators as they are measured: inputs, plain forms and the framework's calls.

The dense side of a transformer block, next to the routed experts: ``linear``
(a matrix product with bias, activation and residual in its epilogue: the
router's logits, a dense layer), ``linear_backward`` and
``activation_backward`` (its gradients), ``norm`` (the norms after one branch
and before the next, with the branch's gate and the residual between them) and
``norm_backward``.  ``run`` computes them with elementary torch operations, or,
where ``own`` is true, with the framework's calls on the same inputs.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def _linear(tokens, cols, rows, dtype, act="none", bias=False, residual=False, scale=1.0,
            out=None, keep=False, **kw):
    return dict(op="linear", tokens=tokens, cols=cols, rows=rows, dtype=dtype, act=act, bias=bias,
                residual=residual, scale=scale, out=out or dtype, keep=keep, **kw)


def _linear_backward(tokens, cols, rows, dtype, grad=None, bias=False, **kw):
    return dict(op="linear_backward", tokens=tokens, cols=cols, rows=rows, dtype=dtype,
                grad=grad or dtype, bias=bias, **kw)


def _act(tokens, cols, dtype, act, scale=1.0, **kw):
    return dict(op="activation_backward", tokens=tokens, cols=cols, dtype=dtype, act=act,
                scale=scale, **kw)


def _norm(op, tokens, hidden, dtype, kind, params="f32", residual=True, alpha=1.0, post=False,
          gates=0, biases=False, **kw):
    """gates: rows of the gate (0: none, 1: one for all, else equal runs of tokens share one)."""
    return dict(op=op, tokens=tokens, hidden=hidden, dtype=dtype, kind=kind, params=params,
                residual=residual, alpha=alpha, post=post, gates=gates, biases=biases, **kw)


def listed():
    return [
        # one token of a decode step through a GPT-13B layer's second dense matrix, whole
        _linear(1, 20480, 5120, "bf16", bias=True, residual=True, name="linear 1 token 20480 to 5120"),
        # a decode step's tokens of 64 ranks before the router: logits in 32 bits
        _linear(256, 7168, 256, "bf16", out="f32", name="linear 256 tokens to 256 logits"),
        # odd sizes throughout: rows that no 16-byte copy is aligned to
        _linear(1777, 1437, 1001, "f16", act="silu", bias=True, residual=True, scale=0.5,
                name="linear 1777 x 1437 to 1001"),
        # four micro-batches through a GPT-13B layer's first dense matrix, the pre-activations kept
        # for the backward pass
        _linear(8192, 5120, 20480, "bf16", act="gelu_tanh", bias=True, keep=True,
                name="linear 8192 x 5120 to 20480 gelu"),
        # the backward pass of one micro-batch through one of its eight tensor-parallel parts
        _linear_backward(2048, 5120, 2560, "bf16", bias=True, name="linear_backward 2048 x 5120 x 2560"),
        # the router's: gradients of the logits in 32 bits, for a whole experiment's tokens
        _linear_backward(65536, 7168, 256, "bf16", grad="f32", name="linear_backward 65536 x 7168 x 256"),
        # between the two dense matrices: a small part, and the four micro-batches' whole layer
        _act(2048, 2560, "f16", "gelu", scale=0.5, name="activation_backward 2048 x 2560"),
        _act(8192, 20480, "bf16", "gelu_tanh", name="activation_backward 8192 x 20480"),
        # one token of a decode step, norms on both sides of a branch
        _norm("norm", 1, 7168, "bf16", "rms", post=True, gates=1, name="norm 1 x 7168"),
        # a prefill of 16 prompts, each with its own gate
        _norm("norm", 16384, 5120, "bf16", "layer", params="bf16", gates=16, biases=True,
              name="norm 16384 x 5120 layer"),
        # the training step of a narrow layer of odd width, and of a wide one
        _norm("norm_backward", 4099, 1437, "f32", "layer", biases=True, alpha=0.5,
              name="norm_backward 4099 x 1437 layer"),
        _norm("norm_backward", 16384, 7168, "bf16", "rms", post=True, gates=1,
              name="norm_backward 16384 x 7168"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over its logarithm: mostly whole eights, as layers have, some odd."""
    n = _log(rng, lo, hi)
    return n | 1 if rng.random() < 0.25 else max(8, n // 8 * 8)


_MOST = 8192 * 5120 * 20480


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "activation_backward", "norm",
                     "norm_backward"])
    half = rng.choice(["bf16", "f16"])
    any_type = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("linear", "linear_backward"):
        cols, rows = _size(rng, 64, 16384), _size(rng, 32, 16384)
        most = _MOST // (cols * rows) // (1 if op == "linear" else 2)
        tokens = _log(rng, 1, max(1, min(65536, most)))
        if op == "linear":
            act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
            return _linear(tokens, cols, rows, half, act=act, bias=rng.random() < 0.5,
                           residual=rng.random() < 0.5, scale=rng.choice([1.0, 0.5]),
                           out="f32" if rng.random() < 0.25 else half,
                           keep=act != "none" and rng.random() < 0.5)
        return _linear_backward(tokens, cols, rows, half, bias=rng.random() < 0.5,
                                grad="f32" if half == "bf16" and rng.random() < 0.3 else half)
    if op == "activation_backward":
        return _act(_log(rng, 1, 8192), _size(rng, 32, 20480), any_type,
                    rng.choice(["relu", "gelu", "gelu_tanh", "silu"]), scale=rng.choice([1.0, 0.5]))
    kind = rng.choice(["rms", "layer"])
    gates = rng.choice([0, 1, rng.randint(2, 32)])
    tokens = _log(rng, 1, 16384)
    if gates > 1:
        tokens = max(1, tokens // gates) * gates
    return _norm(op, tokens, _size(rng, 32, 7168), any_type, kind,
                 params=rng.choice(["f32", any_type]), residual=rng.random() < 0.8,
                 alpha=rng.choice([1.0, 0.5]), post=rng.random() < 0.5, gates=gates,
                 biases=kind == "layer")


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    dt = DTYPES[c["dtype"]]

    def randn(*shape, std=1.0, mean=0.0, dtype=dt):
        x = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g)
        return (x + mean if mean else x).to(dtype)

    if c["op"] == "linear":
        t, k, n = c["tokens"], c["cols"], c["rows"]
        s["x"], s["w"] = randn(t, k), randn(n, k, std=k ** -0.5)
        s["bias"] = randn(n, std=0.1) if c["bias"] else None
        s["residual"] = randn(t, n, std=2.0, dtype=DTYPES[c["out"]]) if c["residual"] else None
    elif c["op"] == "linear_backward":
        t, k, n = c["tokens"], c["cols"], c["rows"]
        s["x"], s["w"] = randn(t, k), randn(n, k, std=k ** -0.5)
        s["dz"] = randn(t, n, std=n ** -0.5, dtype=DTYPES[c["grad"]])
    elif c["op"] == "activation_backward":
        s["dy"], s["z"] = randn(c["tokens"], c["cols"], std=0.05), randn(c["tokens"], c["cols"], std=1.5)
    else:
        t, h, pt = c["tokens"], c["hidden"], DTYPES[c["params"]]
        s["y"] = randn(t, h, std=0.7, mean=0.1)
        s["residual"] = randn(t, h, std=2.0) if c["residual"] else None
        s["weight"] = randn(h, std=0.1, mean=1.0, dtype=pt)
        s["bias"] = randn(h, std=0.1, dtype=pt) if c["biases"] else None
        s["post"] = randn(h, std=0.1, mean=1.0, dtype=pt) if c["post"] else None
        s["post_bias"] = randn(h, std=0.1, dtype=pt) if c["post"] and c["biases"] else None
        s["gate"] = randn(c["gates"], h, std=0.3, mean=0.5, dtype=pt) if c["gates"] else None
        if c["op"] == "norm_backward":
            s["dn"], s["dr"] = randn(t, h, std=0.05), randn(t, h, std=0.05)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c)


_EPS = 1e-6
_TANH = math.sqrt(2.0 / math.pi)


def _plain_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_TANH * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_linear(s, c):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _plain_act(z, c["act"])
    if c["scale"] != 1.0:
        y = y * c["scale"]
    if s["residual"] is not None:
        y = s["residual"].float() + y
    y = y.to(DTYPES[c["out"]])
    return (y, z.to(s["x"].dtype)) if c["keep"] else y


def _plain_linear_backward(s, c):
    dz, dt = s["dz"].float(), s["x"].dtype
    dx, dw = dz @ s["w"].float(), dz.t() @ s["x"].float()
    return dx.to(dt), dw.to(dt), dz.sum(0).to(dt) if c["bias"] else None


def _plain_activation_backward(s, c):
    z = s["z"].float()
    if c["act"] == "relu":
        d = (z > 0.0).float()
    elif c["act"] == "gelu":
        d = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    elif c["act"] == "gelu_tanh":
        t = torch.tanh(_TANH * (z + 0.044715 * z * z * z))
        d = 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _TANH * (1.0 + 3.0 * 0.044715 * z * z)
    else:
        q = 1.0 / (1.0 + torch.exp(-z))
        d = q * (1.0 + z * (1.0 - q))
    return (s["dy"].float() * d * c["scale"]).to(s["z"].dtype)


def _plain_normed(x, kind):
    """(x without its mean over its deviation, one over that deviation)."""
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    inv = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS)
    return x * inv, inv


def _plain_branch(s, c):
    """The normed branch, the branch before its gate, the gate of every row, the stream."""
    y, yn, inv, gate = s["y"].float(), None, None, None
    u = y
    if s["post"] is not None:
        yn, inv = _plain_normed(y, c["kind"])
        u = yn * s["post"].float()
        if s["post_bias"] is not None:
            u = u + s["post_bias"].float()
    r = u
    if s["gate"] is not None:
        gate = s["gate"].float().repeat_interleave(c["tokens"] // c["gates"], dim=0)
        r = r * gate
    if s["residual"] is not None:
        r = c["alpha"] * s["residual"].float() + r
    return yn, inv, u, gate, r


def _plain_norm(s, c):
    r = _plain_branch(s, c)[-1]
    n = _plain_normed(r, c["kind"])[0] * s["weight"].float()
    if s["bias"] is not None:
        n = n + s["bias"].float()
    return n.to(s["y"].dtype), r.to(s["y"].dtype)


def _plain_norm_grad(dn, xn, inv, kind):
    d = dn - xn * (dn * xn).mean(1, keepdim=True)
    if kind == "layer":
        d = d - dn.mean(1, keepdim=True)
    return d * inv


def _plain_norm_backward(s, c):
    dt, pt = s["y"].dtype, s["weight"].dtype
    yn, yinv, u, gate, r = _plain_branch(s, c)
    rn, rinv = _plain_normed(r, c["kind"])
    dn = s["dn"].float()
    out = dict(dweight=(dn * rn).sum(0).to(pt))
    if s["bias"] is not None:
        out["dbias"] = dn.sum(0).to(pt)
    d = s["dr"].float() + _plain_norm_grad(dn * s["weight"].float(), rn, rinv, c["kind"])
    if s["residual"] is not None:
        out["dresidual"] = (c["alpha"] * d).to(dt)
    if gate is not None:
        out["dgate"] = (d * u).view(c["gates"], -1, c["hidden"]).sum(1).to(pt)
        d = d * gate
    if s["post"] is not None:
        out["dpost"] = (d * yn).sum(0).to(pt)
        if s["post_bias"] is not None:
            out["dpost_bias"] = d.sum(0).to(pt)
        d = _plain_norm_grad(d * s["post"].float(), yn, yinv, c["kind"])
    out["dy"] = d.to(dt)
    return _grads(out)


_NAMES = ("dy", "dresidual", "dweight", "dbias", "dpost", "dpost_bias", "dgate")


def _grads(d):
    return tuple(d.get(n) for n in _NAMES)


_plain = {"linear": _plain_linear, "linear_backward": _plain_linear_backward,
          "activation_backward": _plain_activation_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward}


def _own_linear(s, c):
    from experiment_network_simulation_gb300 import block
    return block.linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"],
                        scale=c["scale"], out_dtype=DTYPES[c["out"]], keep=c["keep"])


def _own_linear_backward(s, c):
    from experiment_network_simulation_gb300 import block
    return block.linear_backward(s["dz"], s["x"], s["w"], bias=c["bias"])


def _own_activation_backward(s, c):
    from experiment_network_simulation_gb300 import block
    return block.activation_backward(s["dy"], s["z"], act=c["act"], scale=c["scale"])


def _own_norm(s, c):
    from experiment_network_simulation_gb300 import block
    return block.norm(s["y"], s["weight"], s["bias"], residual=s["residual"], alpha=c["alpha"],
                      post=s["post"], post_bias=s["post_bias"], gate=s["gate"], kind=c["kind"],
                      eps=_EPS)


def _own_norm_backward(s, c):
    from experiment_network_simulation_gb300 import block
    return tuple(block.norm_backward(
        s["dn"], s["y"], s["weight"], s["bias"], dr=s["dr"], residual=s["residual"],
        alpha=c["alpha"], post=s["post"], post_bias=s["post_bias"], gate=s["gate"],
        kind=c["kind"], eps=_EPS))


_own = {"linear": _own_linear, "linear_backward": _own_linear_backward,
        "activation_backward": _own_activation_backward, "norm": _own_norm,
        "norm_backward": _own_norm_backward}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(c):
    b = SIZE[c["dtype"]]
    if c["op"] == "linear":
        t, k, n, o = c["tokens"], c["cols"], c["rows"], SIZE[c["out"]]
        return {"bytes": b * (t * k + n * k + n * c["bias"] + t * n * c["keep"]) + o * t * n * (1 + c["residual"]),
                "flops": 2.0 * t * k * n}
    if c["op"] == "linear_backward":
        t, k, n = c["tokens"], c["cols"], c["rows"]
        return {"bytes": 2 * b * (t * k + n * k) + b * n * c["bias"] + SIZE[c["grad"]] * t * n,
                "flops": 4.0 * t * k * n}
    if c["op"] == "activation_backward":
        return {"bytes": 3 * b * c["tokens"] * c["cols"], "flops": 20.0 * c["tokens"] * c["cols"]}
    t, h, p = c["tokens"], c["hidden"], SIZE[c["params"]]
    params = h * (1 + c["biases"] + c["post"] * (1 + c["biases"]) + c["gates"]) * p
    if c["op"] == "norm":
        return {"bytes": t * h * b * (3 + c["residual"]) + params, "flops": 12.0 * t * h}
    return {"bytes": t * h * b * (4 + 2 * c["residual"]) + 2 * params, "flops": 30.0 * t * h}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(c, seed):
    return _exact[c["op"]](prepare(c, seed), c)


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    # (1 + tanh v) / 2 is the logistic function of 2 v
    return z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))


def _exact_linear(s, c):
    x, w = s["x"].double(), s["w"].double()
    ys, zs = [], []
    for a in range(0, c["rows"], 4096):
        z = torch.einsum("tk,nk->tn", x, w[a:a + 4096])
        if s["bias"] is not None:
            z += s["bias"][a:a + 4096].double()
        y = c["scale"] * _exact_act(z, c["act"])
        if s["residual"] is not None:
            y += s["residual"][:, a:a + 4096].double()
        ys.append(y)
        zs.append(z if c["keep"] else None)
    y = torch.cat(ys, 1)
    return (y, torch.cat(zs, 1)) if c["keep"] else y


def _exact_linear_backward(s, c):
    x, w, dz = s["x"].double(), s["w"].double(), s["dz"].double()
    dw = torch.zeros_like(w)
    dx = []
    for a in range(0, c["tokens"], 8192):
        d = dz[a:a + 8192]
        dx.append(torch.einsum("tn,nk->tk", d, w))
        dw += torch.einsum("tn,tk->nk", d, x[a:a + 8192])
    return torch.cat(dx), dw, torch.einsum("tn->n", dz) if c["bias"] else None


def _exact_activation_backward(s, c):
    out = []
    for dy, z in zip(s["dy"].split(2048), s["z"].split(2048)):
        z = z.double().requires_grad_(True)
        out.append(torch.autograd.grad(_exact_act(z, c["act"]), z, dy.double() * c["scale"])[0])
    return torch.cat(out)


def _exact_norm_rows(s, c, at, leaf):
    """Normed stream and stream of the tokens ``at``; ``leaf`` gives an input in 64 bits."""
    def normed(x, w, b):
        if c["kind"] == "layer":
            x = x - x.sum(1, keepdim=True) / c["hidden"]
        x = x * torch.rsqrt(x.square().sum(1, keepdim=True) / c["hidden"] + _EPS) * w
        return x if b is None else x + b

    r = leaf("y")
    if c["post"]:
        r = normed(r, leaf("post"), leaf("post_bias"))
    if c["gates"]:
        r = r * leaf("gate")[torch.arange(at.start, at.stop, device="cuda") // (c["tokens"] // c["gates"])]
    if c["residual"]:
        r = r + c["alpha"] * leaf("residual")
    return normed(r, leaf("weight"), leaf("bias")), r


_BY_TOKEN = ("y", "residual", "dn", "dr")


def _exact_norm(s, c):
    n, r = [], []
    for a in range(0, c["tokens"], 4096):
        at = slice(a, min(a + 4096, c["tokens"]))

        def leaf(name):
            t = s[name]
            return None if t is None else (t[at] if name in _BY_TOKEN else t).double()

        one = _exact_norm_rows(s, c, at, leaf)
        n.append(one[0])
        r.append(one[1])
    return torch.cat(n), torch.cat(r)


def _exact_norm_backward(s, c):
    """By differentiating the forward formula."""
    names = ("y", "residual", "weight", "bias", "post", "post_bias", "gate")
    total = {n: [] if n in _BY_TOKEN else 0.0 for n in names if s[n] is not None}
    for a in range(0, c["tokens"], 4096):
        at = slice(a, min(a + 4096, c["tokens"]))
        leaves = {n: (s[n][at] if n in _BY_TOKEN else s[n]).double().requires_grad_(True) for n in total}
        n, r = _exact_norm_rows(s, c, at, leaves.get)
        loss = (n * s["dn"][at].double()).sum() + (r * s["dr"][at].double()).sum()
        for name, d in zip(leaves, torch.autograd.grad(loss, list(leaves.values()))):
            if name in _BY_TOKEN:
                total[name].append(d)
            else:
                total[name] = total[name] + d
    return _grads({"d" + n: torch.cat(d) if n in _BY_TOKEN else d for n, d in total.items()})


_exact = {"linear": _exact_linear, "linear_backward": _exact_linear_backward,
          "activation_backward": _exact_activation_backward, "norm": _exact_norm,
          "norm_backward": _exact_norm_backward}
