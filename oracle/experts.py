"""Plain, slow, fp64 reference of the calls around a layer of experts: the
root-mean-square norm, the choice of experts, the rows' order by expert, and
their gradients.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see the package docstring).

Written from the formulas in include/mhc.h; tests/test_oracle_experts_pins.py
checks the gradients against differences.  Inputs and outputs are numpy float64
unless said.  The 8-bit format is mhc_backward's ckpt_encode / ckpt_decode.
"""

import numpy as np

LARGEST = float(np.finfo(np.float32).max)


def rmsnorm(s, weight=None, eps=1e-5):
    """(y, rstd) of the rows s [B, C]."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    y = s * rstd[:, None]
    return (y if weight is None else y * np.asarray(weight, np.float64)), rstd


def rmsnorm_bwd(s, weight, rstd, dy, dsum=None):
    """(dx, dweight) with rstd as given."""
    s, rstd, dy = (np.asarray(t, np.float64) for t in (s, rstd, dy))
    n = s * rstd[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, np.sum(dy * n, axis=0)


def clean(logits):
    """Logits as they count: NaN as minus infinity, plus infinity as fp32's largest number."""
    x = np.asarray(logits, np.float64)
    return np.minimum(np.where(np.isnan(x), -np.inf, x), LARGEST)


def _softmax(x):
    """Of one row's values; zeros where there is none but minus infinity."""
    if not np.any(x > -np.inf):
        return np.zeros_like(x)
    e = np.where(x > -np.inf, np.exp(x - np.max(x)), 0.0)
    return e / np.sum(e)


def _log_sigmoid(x):
    return np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def _best(values, count):
    """The indexes of the `count` largest, in descending order, the lowest first
    of equal ones; those that are minus infinity are left out."""
    order = sorted(range(len(values)), key=lambda i: (-values[i], i))
    return [i for i in order[:count] if values[i] > -np.inf]


def weights_of(x, ids, softmax, renorm, scale):
    """One row's weights for chosen ids (-1: none) from its cleaned logits x."""
    there = [i for i, e in enumerate(ids) if 0 <= e < len(x)]
    w = np.zeros(len(ids))
    if there:
        chosen = x[[ids[i] for i in there]]
        if renorm:
            w[there] = _softmax(chosen if softmax else np.where(chosen > -np.inf, _log_sigmoid(chosen), -np.inf))
        else:
            w[there] = _softmax(x)[[ids[i] for i in there]] if softmax else sigmoid(chosen)
    return scale * w


def route(logits, k, bias=None, groups=1, top_groups=1, softmax=False, renorm=True, scale=1.0):
    """(ids int [B, k], weights [B, k]).  Without a bias the order is that of the logits."""
    logits = clean(logits)
    B, E = logits.shape
    ids, weights = np.full((B, k), -1, np.int64), np.zeros((B, k))
    for b in range(B):
        x = logits[b]
        choice = x
        if bias is not None:
            choice = (_softmax(x) if softmax else sigmoid(x)) + np.asarray(bias, np.float64)
        choice = np.where((x > -np.inf) & ~np.isnan(choice), choice, -np.inf)
        if top_groups < groups:
            each = choice.reshape(groups, -1)
            rank = []
            for g in each:
                two = sorted(g, reverse=True)[:2]
                rank.append(two[0] + two[1] if bias is not None and len(two) > 1 and two[1] > -np.inf else two[0])
            kept = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            choice = np.concatenate([each[g] if g in kept else np.full(E // groups, -np.inf) for g in range(groups)])
        at = _best(choice, k)
        ids[b, :len(at)] = at
        weights[b] = weights_of(x, ids[b], softmax, renorm, scale)
    return ids, weights


def route_bwd(logits, ids, dweights, softmax=False, renorm=True, scale=1.0):
    """dlogits [B, E]."""
    logits = clean(logits)
    out = np.zeros_like(logits)
    for b, x in enumerate(logits):
        at = [int(e) for e in ids[b]]
        dw = np.array([scale * float(d) if 0 <= e < len(x) else 0.0 for e, d in zip(at, dweights[b])])
        w = weights_of(x, at, softmax, renorm, 1.0)
        if softmax and not renorm:
            p = _softmax(x)
            out[b] = -p * np.sum(w * dw)
        g = w * (dw - np.sum(w * dw)) if renorm else w * dw
        for e, d in zip(at, g):
            if 0 <= e < len(x) and x[e] > -np.inf:
                out[b, e] += d if softmax else d * sigmoid(-x[e])
    return out


def order(ids, E):
    """(slots int [B, k], offsets int [E + 1])."""
    ids = np.asarray(ids)
    slots = np.full(ids.size, -1, np.int64)
    offsets, at = np.zeros(E + 1, np.int64), 0
    for e in range(E):
        mine = np.flatnonzero(ids.reshape(-1) == e)
        slots[mine] = at + np.arange(len(mine))
        at += len(mine)
        offsets[e + 1] = at
    return slots.reshape(ids.shape), offsets


def combine(Y, slots, weights=None, shared=None):
    """out [B, C] and the sum of its terms' magnitudes."""
    Y = np.asarray(Y, np.float64)
    out = np.zeros((slots.shape[0], Y.shape[1])) if shared is None else np.array(shared, np.float64)
    size = np.abs(out)
    for b, row in enumerate(slots):
        for j, s in enumerate(row):
            if 0 <= s < len(Y):
                term = (1.0 if weights is None else float(weights[b, j])) * Y[s]
                out[b] += term
                size[b] += np.abs(term)
    return out, size


def combine_bwd(Y, slots, weights, dout):
    """(dY with NaN where no slot points, dweights, the magnitudes of its terms)."""
    Y, dout = np.asarray(Y, np.float64), np.asarray(dout, np.float64)
    dY = np.full(Y.shape, np.nan)
    dw, size = np.zeros(slots.shape), np.zeros(slots.shape)
    for b, row in enumerate(slots):
        for j, s in enumerate(row):
            if 0 <= s < len(Y):
                dY[s] = float(weights[b, j]) * dout[b]
                dw[b, j] = np.sum(dout[b] * Y[s])
                size[b, j] = np.sum(np.abs(dout[b] * Y[s]))
    return dY, dw, size
