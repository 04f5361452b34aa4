"""Plain 64-bit implementations of the routed-expert operators, from their
definitions, one row or one expert at a time (numpy, CPU)."""
import numpy as np


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, np.float64)))


def softmax_open(x, opened):
    """Softmax over the open entries; an infinite logit takes the whole."""
    p = np.zeros(len(x))
    if opened.any():
        m = x[opened].max()
        p[opened] = (x[opened] == m).astype(float) if np.isinf(m) else np.exp(x[opened] - m)
        p /= p.sum()
    return p


def route(logits, topk, scores="softmax", bias=None, groups=1, top_groups=1, group_rule="max",
          renorm=True, scale=1.0):
    """(ids, weights, gaps): gaps[t] is the smallest difference of order values
    (of groups, too) that a decision of row t was made on, ties apart."""
    x_all = np.asarray(logits, np.float64)
    T, E = x_all.shape
    ids, weights = np.full((T, topk), -1, np.int32), np.zeros((T, topk))
    gaps = np.full(T, np.inf)
    two = groups > 1 and group_rule == "top2"
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    for t in range(T):
        x = x_all[t]
        has = ~np.isnan(x) & (x != -np.inf)
        opened = has & ~np.isnan(b) & (b != -np.inf)
        s = softmax_open(x, has) if scores == "softmax" else np.where(has, sigmoid(np.where(has, x, 0)), 0)
        v = x if bias is None and not two else s + b
        left = [e for e in range(E) if opened[e]]
        if groups > 1:
            size = E // groups
            value = {}
            for g in range(groups):
                best = sorted((v[e] for e in left if e // size == g), reverse=True)
                if best:
                    value[g] = sum(best[:2]) if two else best[0]
            order = sorted(value, key=lambda g: (-value[g], g))
            if len(order) > top_groups:
                a, c = value[order[top_groups - 1]], value[order[top_groups]]
                d = 0.0 if a == c else a - c
                gaps[t] = min(gaps[t], d if d > 0 else np.inf)
            left = [e for e in left if e // size in order[:top_groups]]
        order = sorted(left, key=lambda e: (-v[e], e))
        for a, c in zip(order[:topk], order[1:]):
            d = 0.0 if v[a] == v[c] else v[a] - v[c]
            gaps[t] = min(gaps[t], d if d > 0 else np.inf)
        order = order[:topk]
        ids[t, :len(order)] = order
        if renorm and scores == "softmax":
            w = softmax_open(x[order], np.ones(len(order), bool))
        else:
            w = s[order]
            if renorm and w.sum() > 0:
                w = w / w.sum()
        weights[t, :len(order)] = scale * w
    return ids, weights, gaps


def weights_of(x, ids, scores, renorm, scale):
    """One row's weights at fixed choices (for differences)."""
    has = ~np.isnan(x) & (x != -np.inf)
    s = softmax_open(x, has) if scores == "softmax" else np.where(has, sigmoid(np.where(has, x, 0)), 0)
    w = np.array([s[i] if i >= 0 else 0.0 for i in ids])
    return scale * (w / w.sum() if renorm and w.sum() > 0 else w)


def route_backward(logits, ids, dweights, scores="softmax", renorm=True, scale=1.0):
    """The gradient by the chain rule over the full Jacobian of every row."""
    x_all = np.asarray(logits, np.float64)
    out = np.zeros_like(x_all)
    for t, x in enumerate(x_all):
        slot = [j for j, i in enumerate(ids[t]) if 0 <= i < len(x)]
        pick = [int(ids[t][j]) for j in slot]
        if not pick:
            continue
        g = np.asarray(dweights[t], np.float64)[slot]
        has = ~np.isnan(x) & (x != -np.inf)
        s = softmax_open(x, has) if scores == "softmax" else np.where(has, sigmoid(np.where(has, x, 0)), 0)
        if renorm:
            total = s[pick].sum()
            if total == 0:
                continue
            ds = (g - (g * s[pick]).sum() / total) / total
        else:
            ds = g
        full = np.zeros(len(x))
        full[pick] = ds
        if scores == "softmax":
            out[t] = scale * s * (full - (full * s).sum())
        else:
            out[t] = scale * full * s * (1 - s)
    return out


def exchange(ids, place, ranks, sources=None, starts=None, once=True):
    B, T, k = ids.shape
    E = len(place)
    S = len(starts) - 1 if starts is not None else (sources or ranks)
    if starts is None:
        starts = [s * (T // S) for s in range(S + 1)]
    load, sent = np.zeros((B, E), np.int32), np.zeros((B, S, ranks), np.int32)
    for b in range(B):
        for s in range(S):
            for t in range(starts[s], starts[s + 1]):
                to = []
                for e in ids[b, t]:
                    if 0 <= e < E:
                        load[b, e] += 1
                        if 0 <= place[e] < ranks:
                            to.append(int(place[e]))
                for d in (set(to) if once else to):
                    sent[b, s, d] += 1
    return load, sent


def unpack(q, scale, group):
    """[rows, cols / 2] bytes, [rows, cols / group] scales -> [rows, cols]."""
    q = np.asarray(q)
    w = np.empty((q.shape[0], 2 * q.shape[1]))
    w[:, 0::2], w[:, 1::2] = q & 15, q >> 4
    return (w - 8) * np.repeat(np.asarray(scale, np.float64), group, axis=1)


def experts(x, ids, weights, w13, s13, w2, s2, group):
    """(y, size): size is the sum of the magnitudes that each y is a sum of."""
    x = np.asarray(x, np.float64)
    T, H = x.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    y, size = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        at = np.argwhere(np.asarray(ids) == e)
        if not len(at):
            continue
        up, down = unpack(w13[e], s13[e], group), unpack(w2[e], s2[e], group)
        for t, j in at:
            z = up @ x[t]
            h = z[:I] * sigmoid(z[:I]) * z[I:]
            w = float(weights[t, j])
            y[t] += w * (down @ h)
            size[t] += abs(w) * (np.abs(down) @ np.abs(h))
    return y, size
