"""Plain 64-bit forms of the routing, dispatch, combine and fused-epilogue
operators, loops over tokens and slots included, written from their definitions
in include/fp4.h.  Test infrastructure: shares nothing with the kernels."""
import math

import numpy as np

NONE, RELU, SILU, GELU, GELU_TANH = range(5)
ACTS = {"none": NONE, "relu": RELU, "silu": SILU, "gelu": GELU, "gelu_tanh": GELU_TANH}

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(x, a):
    if a == RELU:
        return np.maximum(x, 0.0)
    if a == SILU:
        return x * sigmoid(x)
    if a == GELU:
        return 0.5 * x * _erfc(-x / math.sqrt(2.0))
    if a == GELU_TANH:
        return 0.5 * x * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    return x.copy()


def act_grad(x, a):
    if a == RELU:
        return (x > 0).astype(np.float64)
    if a == SILU:
        s = sigmoid(x)
        return s + x * s * (1.0 - s)
    if a == GELU:
        return 0.5 * _erfc(-x / math.sqrt(2.0)) + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if a == GELU_TANH:
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    return np.ones_like(x)


def epilogue(z, a, gated, residual=None):
    d = act(z[..., 0::2], a) * z[..., 1::2] if gated else act(z, a)
    return d if residual is None else d + residual


def epilogue_grad(dD, z, a, gated):
    if not gated:
        return dD * act_grad(z, a)
    g, u = z[..., 0::2], z[..., 1::2]
    dz = np.empty_like(z)
    dz[..., 0::2] = dD * u * act_grad(g, a)
    dz[..., 1::2] = dD * act(g, a)
    return dz


# ---------------------------------------------------------------- routing ----
def scores(logits, sigmoid_scores):
    """float64 scores of [T, E] logits, and the masked entries."""
    l = logits.astype(np.float64)
    dead = np.isnan(l) | (l == -np.inf)
    l = np.where(l == np.inf, float(np.finfo(np.float32).max), l)
    if sigmoid_scores:
        return np.where(dead, 0.0, sigmoid(np.where(dead, 0.0, l))), dead
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        live = ~dead[t]
        if live.any():
            e = np.exp(l[t, live] - l[t, live].max())
            s[t, live] = e / e.sum()
    return s, dead


def route(logits, k, sigmoid_scores, bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    T, E = logits.shape
    s, dead = scores(logits, sigmoid_scores)
    if bias is not None:
        v = s + bias.astype(np.float64)
    elif groups > 1 and group_top == 2:
        v = s
    else:
        v = np.where(dead, -np.inf, logits.astype(np.float64))
    v = np.where(dead | np.isnan(v), -np.inf, v)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        left = list(range(E))
        if groups > 1:
            size = E // groups
            gs = []
            for g in range(groups):
                m = sorted((v[t, e] for e in range(g * size, (g + 1) * size) if v[t, e] > -np.inf), reverse=True)
                gs.append(sum(m[:group_top]) if m else -np.inf)
            best = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            left = [e for e in left if e // size in best]
        left = [e for e in sorted(left, key=lambda e: (-v[t, e], e)) if v[t, e] > -np.inf][:k]
        ids[t, :len(left)] = left
        p = s[t, left]
        if renorm:
            p = p / p.sum() if p.sum() > 0 else 0 * p
        w[t, :len(left)] = scale * p
    return ids, w, v


def route_weights(logits, ids, sigmoid_scores, renorm, scale):
    """The weights of given ids as a function of the logits (for differences)."""
    s, _ = scores(logits, sigmoid_scores)
    T, k = ids.shape
    w = np.zeros((T, k))
    for t in range(T):
        live = ids[t] >= 0
        p = s[t, ids[t, live]]
        if renorm and p.sum() > 0:
            p = p / p.sum()
        w[t, live] = scale * p
    return w


def route_grad(dw, logits, ids, sigmoid_scores, renorm, scale):
    """d logits by the chain rule, one Jacobian per token."""
    T, E = logits.shape
    s, dead = scores(logits, sigmoid_scores)
    out = np.zeros((T, E))
    for t in range(T):
        live = [j for j in range(ids.shape[1]) if ids[t, j] >= 0]
        sel = [int(ids[t, j]) for j in live]
        if not sel:
            continue
        g = scale * dw[t, live].astype(np.float64)      # gradient of the (renormalized) scores
        p = s[t, sel]
        if renorm:
            S = p.sum()
            g = (g - (g * p).sum() / S) / S if S > 0 else 0 * g
        ds = np.zeros(E)
        ds[sel] = g
        if sigmoid_scores:
            out[t] = ds * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        out[t, dead[t]] = 0.0
    return out


# ------------------------------------------------------- dispatch, combine ----
def sort_slots(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    row_slots = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    slot_rows = np.full(T * k, -1, np.int32)
    slot_rows[row_slots] = np.arange(len(row_slots))
    full = np.full(T * k, -1, np.int32)
    full[:len(row_slots)] = row_slots
    return offsets, slot_rows.reshape(T, k), full


def combine(rows, weights, slot_rows, residual=None):
    T, k = weights.shape
    y = np.zeros((T, rows.shape[1])) if residual is None else residual.astype(np.float64).copy()
    for t in range(T):
        for j in range(k):
            if slot_rows[t, j] >= 0:
                y[t] += float(weights[t, j]) * rows[slot_rows[t, j]].astype(np.float64)
    return y


def combine_grad(dy, rows, weights, slot_rows):
    T, k = weights.shape
    d_rows = np.zeros(rows.shape)
    d_w = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = slot_rows[t, j]
            if r >= 0:
                d_rows[r] = float(weights[t, j]) * dy[t].astype(np.float64)
                d_w[t, j] = (dy[t].astype(np.float64) * rows[r].astype(np.float64)).sum()
    return d_rows, d_w
