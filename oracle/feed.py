"""Float64 reference of the feed-forward layer's operators, dense or of
experts: the router and its gradient, the order by expert, the way into it and
back, and the linear product with bias, activation and residual.  Test
infrastructure only."""

import math

import numpy as np

GATED = ("swiglu", "geglu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


# ---------------------------------------------------------------- router


def scores(logits, score="softmax"):
    """Each expert's score, row by row; a row of -inf scores 0 everywhere, a softmax' row
    with a NaN or +inf is NaN everywhere."""
    v = np.asarray(logits, np.float64)
    if score == "sigmoid":
        return _sigmoid(v)
    out = np.zeros_like(v)
    for t, row in enumerate(v):
        top = row.max()
        if top != -np.inf:
            with np.errstate(invalid="ignore"):
                e = np.exp(row - top)
            out[t] = e / e.sum()
    return out


def route(logits, k, score="softmax", renormalize=False, scale=1.0):
    """(index, weight, score_sum) by choosing one expert after another."""
    v = np.asarray(logits, np.float64)
    s = scores(v, score)
    index = np.full((len(v), k), -1, np.int32)
    weight = np.zeros((len(v), k))
    for t in range(len(v)):
        left = np.where(np.isnan(v[t]), -np.finfo(np.float32).max, v[t])
        for j in range(k):
            e = int(np.argmax(left))  # the first of equal ones
            if left[e] == -np.inf:
                break
            index[t, j], weight[t, j], left[e] = e, s[t, e], -np.inf
        if renormalize and weight[t].sum() != 0:
            weight[t, index[t] >= 0] /= weight[t].sum()
    return index, scale * weight, s.sum(0)


def route_grad(logits, index, dweight=None, dscore_sum=None, score="softmax", renormalize=False,
               scale=1.0):
    """Gradient of sum dweight*weight + sum dscore_sum*score_sum, the choice held."""
    v = np.asarray(logits, np.float64)
    s = scores(v, score)
    g = np.zeros_like(v)    # with respect to the scores
    out = np.zeros_like(v)  # with respect to the logits, of renormalised weights
    if dscore_sum is not None:
        g += np.asarray(dscore_sum, np.float64)
    if dweight is not None:
        for t in range(len(v)):
            js = [j for j, e in enumerate(index[t]) if 0 <= e < v.shape[1]]
            es = [index[t, j] for j in js]
            d = scale * np.asarray(dweight, np.float64)[t, js]
            if renormalize and js:
                # weights scale q, q the chosen scores' shares: dq_i / dlog s_j = q_i ([i = j] - q_j)
                q = s[t, es] / s[t, es].sum()
                slope = _sigmoid(-v[t, es]) if score == "sigmoid" else 1.0  # dlog s / dl, up to
                np.add.at(out[t], es, q * (d - (q * d).sum()) * slope)      # what all share
            else:
                np.add.at(g[t], es, d)
    if score == "sigmoid":
        return out + g * s * _sigmoid(-v)
    return out + s * (g - (s * g).sum(1, keepdims=True))


# ---------------------------------------------------------------- order


def sort(index, experts):
    """(offsets, token, slot) of the pairs (token, choice) by expert."""
    index = np.asarray(index)
    tokens, k = index.shape
    slot = np.full((tokens, k), -1, np.int32)
    token = np.full(tokens * k, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    row = 0
    for e in range(experts):
        for t, j in zip(*np.nonzero(index == e)):
            token[row], slot[t, j] = t, row
            row += 1
        offsets[e + 1] = row
    return offsets, token, slot


def gather(x, token):
    x, token = np.asarray(x), np.asarray(token)
    ok = (token >= 0) & (token < len(x))
    return np.where(ok[:, None], x[np.where(ok, token, 0)], 0)


def combine(y, slot, weight=None, residual=None):
    y = np.asarray(y, np.float64)
    out = np.zeros((len(slot), y.shape[1])) if residual is None else np.array(residual, np.float64)
    for t, row in enumerate(slot):
        for j, r in enumerate(row):
            if 0 <= r < len(y):
                out[t] += (1.0 if weight is None else float(weight[t, j])) * y[r]
    return out


def combine_grad(dout, y, slot, weight):
    """(dy, dweight); rows in no slot are zero."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    dy, dweight = np.zeros_like(y), np.zeros(slot.shape)
    for t, row in enumerate(slot):
        for j, r in enumerate(row):
            if 0 <= r < len(y):
                dy[r] += (1.0 if weight is None else float(weight[t, j])) * dout[t]
                dweight[t, j] = dout[t] @ y[r]
    return dy, dweight


# ---------------------------------------------------------------- product


def bend(v, act):
    """f(v) and f'(v), f silu (silu, swiglu) or gelu (gelu, geglu)."""
    v = np.asarray(v, np.float64)
    if act in ("silu", "swiglu"):
        g = _sigmoid(v)
        return v * g, g * (1.0 + v * _sigmoid(-v))
    phi = 0.5 * _erfc(-v / math.sqrt(2.0))
    return v * phi, phi + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def activate(pre, act):
    if act is None:
        return np.asarray(pre, np.float64)
    if act in GATED:
        gate, up = np.split(np.asarray(pre, np.float64), 2, axis=-1)
        return bend(gate, act)[0] * up
    return bend(pre, act)[0]


def activate_grad(dout, pre, act):
    dout = np.asarray(dout, np.float64)
    if act is None:
        return dout
    if act in GATED:
        gate, up = np.split(np.asarray(pre, np.float64), 2, axis=-1)
        f, slope = bend(gate, act)
        return np.concatenate([dout * up * slope, dout * f], -1)
    return dout * bend(pre, act)[1]


def _parts(rows, offsets):
    return [(0, rows)] if offsets is None else list(zip(offsets, offsets[1:]))


def product(x, w, bias=None, act=None, residual=None, offsets=None):
    """(out, pre) of rows x; w [n, k], or [experts, n, k] with offsets.  Rows past
    the last expert's are zero."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    if offsets is None:
        w, bias = w[None], None if bias is None else np.asarray(bias)[None]
    pre = np.zeros((len(x), w.shape[1]))
    for e, (a, b) in enumerate(_parts(len(x), offsets)):
        pre[a:b] = x[a:b] @ w[e].T
        if bias is not None:
            pre[a:b] += np.asarray(bias[e], np.float64)
    out = activate(pre, act)
    return (out if residual is None else out + np.asarray(residual, np.float64)), pre


def product_grad(dpre, x, w, offsets=None):
    """dx, dw, dbias from the gradient before the activation."""
    dpre, x, w = (np.asarray(v, np.float64) for v in (dpre, x, w))
    ws = w[None] if offsets is None else w
    dx, dw, dbias = np.zeros_like(x), np.zeros_like(ws), np.zeros(ws.shape[:2])
    for e, (a, b) in enumerate(_parts(len(x), offsets)):
        dx[a:b] = dpre[a:b] @ ws[e]
        dw[e] = dpre[a:b].T @ x[a:b]
        dbias[e] = dpre[a:b].sum(0)
    return (dx, dw[0], dbias[0]) if offsets is None else (dx, dw, dbias)
