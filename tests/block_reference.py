"""The block operators in plain 64-bit numpy: results, and beside each the sum of the
magnitudes it is made of, which rounding errors are relative to."""
import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erf = np.vectorize(math.erf, otypes=[np.float64])
_C = math.sqrt(2.0 / math.pi)


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * 0.5 * (1.0 + np.tanh(0.5 * z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        q = 0.5 * (1.0 + np.tanh(0.5 * z))
        return q * (1.0 + z * (1.0 - q))
    return np.ones_like(z)


def linear(x, w, bias=None, act_name="none", residual=None, scale=1.0):
    """(y, z, magnitude of z's sum)."""
    z, m = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, m = z + bias, m + np.abs(bias)
    y = scale * act(z, act_name)
    return (y if residual is None else residual + y), z, m


def _normed(x, kind, eps):
    """(N(x), mean, 1 / deviation), by rows."""
    mean = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(x), 1))
    inv = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    return (x - mean) * inv, mean, inv


def _gates(gate, tokens):
    return np.repeat(gate, tokens // len(gate), axis=0)


def norm(y, weight, bias=None, residual=None, alpha=1.0, post=None, post_bias=None, gate=None,
         kind="rms", eps=1e-6):
    """((n, magnitude), (r, magnitude)); gate [gates, hidden]."""
    u, m = y, np.abs(y)
    if post is not None:
        yn, mean, inv = _normed(y, kind, eps)
        u, m = yn * post, (np.abs(y) + np.abs(y).mean(1, keepdims=True)) * inv * np.abs(post)
        if post_bias is not None:
            u, m = u + post_bias, m + np.abs(post_bias)
    if gate is not None:
        g = _gates(gate, len(y))
        u, m = u * g, m * np.abs(g)
    if residual is not None:
        u, m = alpha * residual + u, np.abs(alpha * residual) + m
    rn, mean, inv = _normed(u, kind, eps)
    spread = 1.0 + np.sqrt((m * m).mean(1, keepdims=True)) * inv     # what cancels in r weighs more in N(r)
    n, mn = rn * weight, (m + m.mean(1, keepdims=True)) * inv * spread * np.abs(weight)
    if bias is not None:
        n, mn = n + bias, mn + np.abs(bias)
    return (n, mn), (u, m)


def _norm_grad(g, m, xn, inv, kind, spread):
    """Gradient through N, and its magnitude."""
    d = g - xn * (g * xn).mean(1, keepdims=True)
    a = np.abs(xn) + 1.0
    m = m + a * ((m * a).mean(1, keepdims=True))
    if kind == "layer":
        d = d - g.mean(1, keepdims=True)
    return d * inv, m * inv * spread


def norm_backward(dn, y, weight, bias=None, dr=None, residual=None, alpha=1.0, post=None,
                  post_bias=None, gate=None, kind="rms", eps=1e-6):
    """{name: (gradient, magnitude)} of the arguments that are there."""
    out = {}
    u, mu = y, np.abs(y)
    yspread = 1.0
    if post is not None:
        yn, mean, yinv = _normed(y, kind, eps)
        yspread = 1.0 + np.sqrt((y * y).mean(1, keepdims=True)) * yinv
        u, mu = yn * post, (np.abs(y) + np.abs(y).mean(1, keepdims=True)) * yinv * np.abs(post)
        if post_bias is not None:
            u, mu = u + post_bias, mu + np.abs(post_bias)
    r, m = u, mu
    if gate is not None:
        g = _gates(gate, len(y))
        r, m = r * g, m * np.abs(g)
    if residual is not None:
        r, m = alpha * residual + r, np.abs(alpha * residual) + m
    rn, mean, inv = _normed(r, kind, eps)
    spread = 1.0 + np.sqrt((m * m).mean(1, keepdims=True)) * inv
    mrn = (m + m.mean(1, keepdims=True)) * inv * spread
    out["dweight"] = (dn * rn).sum(0), (np.abs(dn) * mrn).sum(0)
    if bias is not None:
        out["dbias"] = dn.sum(0), np.abs(dn).sum(0)
    G, mG = _norm_grad(dn * weight, np.abs(dn * weight), rn, inv, kind, spread)
    if dr is not None:
        G, mG = G + dr, mG + np.abs(dr)
    if residual is not None:
        out["dresidual"] = alpha * G, abs(alpha) * mG
    if gate is not None:
        shape = (len(gate), -1, y.shape[1])
        out["dgate"] = (G * u).reshape(shape).sum(1), (mG * mu).reshape(shape).sum(1)
        G, mG = G * g, mG * np.abs(g)
    if post is not None:
        out["dpost"] = (G * yn).sum(0), (mG * (np.abs(yn) + 1.0) * yspread).sum(0)
        if post_bias is not None:
            out["dpost_bias"] = G.sum(0), mG.sum(0)
        G, mG = _norm_grad(G * post, mG * np.abs(post), yn, yinv, kind, yspread)
    out["dy"] = G, mG
    return out
