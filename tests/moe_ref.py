"""Definitions in 64 bits of what lies between the products of an expert layer
(routing, the experts' rows, dispatch, combine), for the tests; token by token in
numpy, no code shared with the kernels."""
import numpy as np

F32_MAX = float(np.finfo(np.float32).max)
ALIGN = 128


def scores(x, sigmoid):
    """x [G] in 64 bits -> (s, available)."""
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), F32_MAX)
    on = x > -np.inf
    s = np.zeros(len(x))
    if sigmoid:
        s[on] = 1.0 / (1.0 + np.exp(np.minimum(-x[on], 700.0)))
    elif on.any():
        e = np.exp(x[on] - x[on].max())
        s[on] = e / e.sum()
    return s, on


def route(logits, bias, k, sigmoid, groups=1, top_groups=1, best=1, renorm=True, scale=1.0):
    """(experts [T, k], weights [T, k]) of numpy logits [T, G]."""
    T, G = logits.shape
    experts, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        s, on = scores(logits[t].astype(np.float64), sigmoid)
        # both scores rise with the logit, beyond where 64 bits tell them apart: where all
        # biases are equal the logits order them (but sums of two, which order the groups)
        x = np.minimum(logits[t].astype(np.float64), F32_MAX)
        even = bias is None or (bias == bias[0]).all()
        c = s + (0.0 if bias is None else bias.astype(np.float64))
        if even and (top_groups == groups or best == 1):
            c = x.copy()
        c[~on] = -np.inf
        if top_groups < groups:
            g = c.reshape(groups, -1)
            value = []
            for row in g:
                r = sorted((v for v in row if v > -np.inf), reverse=True)[:best]
                value.append(sum(r) if r else -np.inf)
            stay = sorted(range(groups), key=lambda i: (-value[i], i))[:top_groups]
            g = (x if even else c).reshape(groups, -1)
            c = np.concatenate([g[i] if i in stay else np.full(len(g[i]), -np.inf) for i in range(groups)])
            c[~on] = -np.inf
        order = [e for e in sorted(range(G), key=lambda i: (-c[i], i)) if c[e] > -np.inf][:k]
        w = s[order]
        if renorm and len(order):
            # (a softmax over the sum of some of its values is the softmax of these
            # logits, also where the values are below what 64 bits hold)
            w = w / (w.sum() + 1e-20) if sigmoid else scores(logits[t][order].astype(np.float64), False)[0]
        experts[t, :len(order)] = order
        weights[t, :len(order)] = scale * w
    return experts, weights


def route_backward(logits, experts, dw, sigmoid, renorm, scale):
    """(d_logits [T, G], the same sums over magnitudes) in 64 bits."""
    T, G = logits.shape
    out, mag = np.zeros((T, G)), np.zeros((T, G))
    for t in range(T):
        s, _ = scores(logits[t].astype(np.float64), sigmoid)
        on = [j for j, e in enumerate(experts[t]) if e >= 0]
        e = experts[t][on]
        d = scale * dw[t][on].astype(np.float64)
        if renorm and not sigmoid:   # (of the softmax of the chosen logits alone)
            p, _ = scores(logits[t][e].astype(np.float64), False)
            np.add.at(out[t], e, p * (d - (d * p).sum()))
            np.add.at(mag[t], e, p * (np.abs(d) + (np.abs(d) * p).sum()))
            continue
        w = s[e]
        a = np.abs(d)
        if renorm:
            total = w.sum() + 1e-20
            a = (a + (a * w / total).sum()) / total
            d = (d - (d * w / total).sum()) / total
        ds, da = np.zeros(G), np.zeros(G)
        np.add.at(ds, e, d)
        np.add.at(da, e, a)
        if sigmoid:
            x = np.minimum(np.where(np.isnan(logits[t]), -np.inf, logits[t].astype(np.float64)), F32_MAX)
            slope = s / (1.0 + np.exp(np.minimum(x, 700)))
            out[t], mag[t] = ds * slope, da * slope
        else:
            out[t] = s * (ds - (ds * s).sum())
            mag[t] = s * (da + (da * s).sum())
    return out, mag


def rows(experts, G, layout, room=0):
    """(sizes, rows, m_indices) of the choices' rows."""
    T, k = experts.shape
    n = np.zeros(G, np.int64)
    place = np.full((T, k), -1, np.int64)
    for t in range(T):
        for j in range(k):
            e = experts[t, j]
            if 0 <= e < G:
                place[t, j] = n[e]
                n[e] += 1
    padded = (n + ALIGN - 1) // ALIGN * ALIGN if layout == "contiguous" else n
    first = np.concatenate([[0], np.cumsum(padded)[:-1]])
    out = np.full((T, k), -1, np.int32)
    m = np.full(room, -1, np.int32)
    for t in range(T):
        for j in range(k):
            e, p = experts[t, j], place[t, j]
            if p < 0:
                continue
            r = p if layout == "masked" else first[e] + p
            if layout != "ragged" and r >= room:
                continue
            out[t, j] = e * room + r if layout == "masked" else r
            if layout == "contiguous":
                m[r] = e
    sizes = np.minimum(n, room) if layout == "masked" else n
    return sizes.astype(np.int32), out, m


def combine(Y, rows_, weights, R):
    """(out, the same sum over magnitudes) in 64 bits."""
    T, k = rows_.shape
    K = Y.shape[1]
    out = np.zeros((T, K)) if R is None else R.astype(np.float64).copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if rows_[t, j] >= 0:
                y = Y[rows_[t, j]].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
                out[t] += y
                mag[t] += np.abs(y)
    return out, mag
