"""Float64 reference of the residual layer's operators: the gated linear
recurrence and its gradients, the root-mean-square norm, the 8-bit block
format and its linear product.  Test infrastructure only."""

import numpy as np

FP8_GROUP = 128
FP8_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gated_scan(x, r, i, log_decay, reset=None, h0=None):
    """(out, last state) of h_t = a_t h_{t-1} + beta_t iota_t x_t, step by step."""
    x, r, i, lam = (np.asarray(v, np.float64) for v in (x, r, i, log_decay))
    bsz, length, dim = x.shape
    h = np.zeros((bsz, dim)) if h0 is None else np.array(h0, np.float64)
    out = np.empty_like(x)
    for t in range(length):
        log_a = lam * _sigmoid(r[:, t])
        new = np.exp(log_a) * h + np.sqrt(-np.expm1(2 * log_a)) * _sigmoid(i[:, t]) * x[:, t]
        if reset is not None:
            new = np.where(np.asarray(reset)[:, t, None] != 0, _sigmoid(i[:, t]) * x[:, t], new)
        h = out[:, t] = new
    return out, h.copy()


def gated_scan_grad(x, r, i, log_decay, dout, reset=None, h0=None, dlast=None):
    """Gradients of sum dout*out + sum dlast*last with respect to every input."""
    x, r, i, lam, dout = (np.asarray(v, np.float64) for v in (x, r, i, log_decay, dout))
    bsz, length, dim = x.shape
    out, _ = gated_scan(x, r, i, lam, reset, h0)
    start = np.zeros((bsz, dim)) if h0 is None else np.asarray(h0, np.float64)
    carry = np.zeros((bsz, dim)) if dlast is None else np.array(dlast, np.float64)
    dx, dr, di = (np.empty_like(x) for _ in range(3))
    dlam = np.zeros(dim)
    for t in range(length - 1, -1, -1):
        rho, iota = _sigmoid(r[:, t]), _sigmoid(i[:, t])
        a, beta2 = np.exp(lam * rho), -np.expm1(2 * lam * rho)
        beta = np.sqrt(beta2)
        before = start if t == 0 else out[:, t - 1]
        g = dout[:, t] + carry
        inv = np.divide(1.0, beta, out=np.zeros_like(beta), where=beta > 0)
        dlog_a = a * g * before - a * a * inv * g * iota * x[:, t]
        carry = a * g
        if reset is not None:
            cut = np.asarray(reset)[:, t, None] != 0
            beta, dlog_a, carry = (np.where(cut, v, w) for v, w in
                                   ((1.0, beta), (0.0, dlog_a), (0.0, carry)))
        dx[:, t] = g * beta * iota
        di[:, t] = g * beta * x[:, t] * iota * (1 - iota)
        dr[:, t] = dlog_a * lam * rho * (1 - rho)
        dlam += (dlog_a * rho).sum(0)
    return dict(dx=dx, dr=dr, di=di, dlog_decay=dlam, dh0=carry)


def rms_norm(x, weight, residual=None, eps=1e-5):
    """(y, s)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    return s / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps) * np.asarray(weight, np.float64), s


def rms_norm_grad(dy, s, weight, eps=1e-5, dres=None):
    dy, s, weight = (np.asarray(v, np.float64) for v in (dy, s, weight))
    rms = np.sqrt(np.mean(s * s, -1, keepdims=True) + eps)
    n = s / rms
    ds = (dy * weight - n * np.mean(n * dy * weight, -1, keepdims=True)) / rms
    if dres is not None:
        ds = ds + np.asarray(dres, np.float64)
    return dict(ds=ds, dweight=(dy * n).reshape(-1, s.shape[-1]).sum(0))


def e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even."""
    v = np.asarray(v, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.round(v / step) * step


def quantize(y, tile_rows=1):
    """(values, scale): one scale for every tile_rows x 128 values of y [M, K];
    scale [ceil(K / 128), M] for rows, [ceil(M / 128), ceil(K / 128)] for tiles."""
    y = np.asarray(y, np.float64)
    m, k = y.shape
    q = np.empty_like(y)
    scale = np.empty((-(-m // tile_rows), -(-k // FP8_GROUP)))
    for a in range(scale.shape[0]):
        for g in range(scale.shape[1]):
            at = np.s_[a * tile_rows:(a + 1) * tile_rows, g * FP8_GROUP:(g + 1) * FP8_GROUP]
            m = max(np.max(np.abs(y[at])), AMAX_FLOOR)
            scale[a, g] = m / FP8_MAX
            # not y / scale: the rounded scale would move a quotient off its tie
            q[at] = e4m3(FP8_MAX * y[at] / m)
    return q, (scale.T if tile_rows == 1 else scale)


def linear(xq, x_scale, wq, w_scale, bias=None):
    """(out, sum of the terms' magnitudes) of the block-scaled product."""
    xq, x_scale, wq, w_scale = (np.asarray(v, np.float64) for v in (xq, x_scale, wq, w_scale))
    k, n = xq.shape[1], wq.shape[0]
    x = xq * np.repeat(x_scale.T, FP8_GROUP, 1)[:, :k]
    w = wq * np.repeat(np.repeat(w_scale, FP8_GROUP, 0)[:n], FP8_GROUP, 1)[:, :k]
    b = 0.0 if bias is None else np.asarray(bias, np.float64)
    return x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)
