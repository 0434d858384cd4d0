"""PyTorch-facing binding of the feed-forward layer's operators, dense or of
experts: the router, the order of its tokens by expert and the way back, and the
linear product with bias, activation and residual, each with its gradient.

As in ``layer``: argument marshalling only.  Scratch comes from torch's caching
allocator on the current stream, so the calls can be captured into a graph.

A layer of experts, in order: expert_route_fwd, expert_sort, expert_linear_fwd
(token=token: it reads the tokens' rows itself), a second expert_linear_fwd,
expert_combine_fwd with the weights.
"""

from ctypes import byref

import torch

from . import _lib
from .api import _DTYPES, _raise
from .layer import _act, _check, _like, _on, _ptr, _row_stride, _stream, _work

_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "swiglu": 3, "geglu": 4}
_GATED = 3  # activations from this one on take two halves


def _route_args(logits, k, score, renormalize):
    code = _act(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    _check(logits, "logits", logits.dtype, logits.shape, logits.device)
    tokens, experts = logits.shape
    return _lib.RouteDims(tokens, experts, k, _SCORES[score], int(bool(renormalize)), code)


def expert_route_fwd(logits, k, score="softmax", renormalize=False, scale=1.0,
                     return_score_sum=False):
    """Router of a layer of experts on the GPU: the k experts with the largest
    logits of every token and their weights.

    logits: [tokens, experts] (float32 or bfloat16).  A token's scores are the
    softmax of its logits or the sigmoid of each; a weight is scale times the
    chosen expert's score, divided by the chosen scores' sum with renormalize.
    Returns index [tokens, k] int32 (largest logit first, equal ones by number;
    an expert whose logit is -inf is not chosen, and an entry left without one is
    -1 with weight 0), weight [tokens, k] float32 and, with return_score_sum,
    score_sum [experts] float32, every expert's scores summed over the tokens.
    A NaN counts as the lowest finite logit in the choice.  Under a softmax it makes
    its row's weights NaN, chosen or not (so does +inf); under a sigmoid it does where
    it is chosen, its own weight or with renormalize the row's.  At most 1024 experts and 16 choices.
    """
    dims = _route_args(logits, k, score, renormalize)
    dev, shape = logits.device, (logits.shape[0], k)
    lib = _lib.load()
    with _on(dev):
        nbytes = lib.expert_route_work_bytes(byref(dims))
        work = _work(nbytes if return_score_sum or nbytes < 0 else 0, dev)
        index = torch.empty(shape, dtype=torch.int32, device=dev)
        weight = torch.empty(shape, dtype=torch.float32, device=dev)
        total = None
        if return_score_sum:
            total = torch.empty(logits.shape[1], dtype=torch.float32, device=dev)
        rc = lib.expert_route_fwd(_ptr(logits), scale, _ptr(index), _ptr(weight), _ptr(total),
                                  _ptr(work), byref(dims), _stream(dev))
    _raise(rc)
    return (index, weight, total) if return_score_sum else (index, weight)


def expert_route_bwd(logits, index, dweight, score="softmax", renormalize=False, scale=1.0,
                     dscore_sum=None):
    """Backward of expert_route_fwd on the GPU, with the choice held: dlogits, in
    logits' type and shape, from dweight [tokens, k] and dscore_sum [experts]
    (float32; either may be None).  index: what the forward returned (an entry
    outside the experts takes no part).  With renormalize the weights are shares of
    the entries that do: where choices are dropped behind the router, give the index
    without them to expert_sort only, and the forward's own here, with the dweight
    of expert_combine_bwd, which is 0 for them."""
    if index is None:
        raise ValueError("index is required")
    if dweight is None and dscore_sum is None:
        raise ValueError("dweight or dscore_sum is required")
    if index.dim() != 2:
        raise ValueError("index must be [tokens, k]")
    k = index.shape[1]
    dims = _route_args(logits, k, score, renormalize)
    dev, shape = logits.device, (logits.shape[0], k)
    _check(index, "index", torch.int32, shape, dev)
    _check(dweight, "dweight", torch.float32, shape, dev)
    _check(dscore_sum, "dscore_sum", torch.float32, (logits.shape[1],), dev)
    dlogits = _like(logits)
    with _on(dev):
        rc = _lib.load().expert_route_bwd(_ptr(logits), scale, _ptr(index), _ptr(dweight),
                                          _ptr(dscore_sum), _ptr(dlogits), byref(dims),
                                          _stream(dev))
    _raise(rc)
    return dlogits


def _gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU, not on {t.device}")


def expert_sort(index, experts):
    """The order of the tokens by expert, on the GPU: rows offsets[e] ..
    offsets[e + 1] - 1 are expert e's, in the order of (token, choice).

    index: [tokens, k] int32; an entry outside 0 .. experts - 1 (a choice that
    was dropped; expert_route_bwd takes the index with it) has no row.  Returns
    int32 offsets [experts + 1], token [tokens * k] (every row's token; -1 past
    offsets[experts]) and slot [tokens, k] (every choice's row; -1 for one without).
    """
    _gpu(index, "index")
    if index.dim() != 2:
        raise ValueError("index must be [tokens, k]")
    shape, dev = index.shape, index.device
    _check(index, "index", torch.int32, shape, dev)
    tokens, k = shape
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.expert_sort_work_bytes(tokens, k, experts), dev)
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
        token = torch.empty(tokens * k, dtype=torch.int32, device=dev)
        slot = torch.empty_like(index)
        rc = lib.expert_sort(_ptr(index), tokens, k, experts, _ptr(offsets), _ptr(token),
                             _ptr(slot), _ptr(work), _stream(dev))
    _raise(rc)
    return offsets, token, slot


def expert_gather(x, token, out=None):
    """Tokens into the experts' order on the GPU: out[r] = x[token[r]], zeros
    where token[r] is none of x's rows.  x: [tokens, dim]; token: [rows] int32.
    The gradient is expert_combine_fwd(dout, slot)."""
    code = _act(x, "x")
    if x.dim() != 2 or token.dim() != 1:
        raise ValueError("x must be [tokens, dim] and token [rows]")
    dev, dtype = x.device, x.dtype
    rows, (tokens, dim) = token.shape[0], x.shape
    _check(x, "x", dtype, x.shape, dev)
    _check(token, "token", torch.int32, (rows,), dev)
    if out is None:
        out = torch.empty((rows, dim), dtype=dtype, device=dev)
    else:
        _check(out, "out", dtype, (rows, dim), dev)
    dims = _lib.OrderDims(tokens, rows, dim, 1, code, code)
    with _on(dev):
        rc = _lib.load().expert_gather(_ptr(x), _ptr(token), _ptr(out), byref(dims), _stream(dev))
    _raise(rc)
    return out


def _slots(slot, weight, dev):
    if slot is None or slot.dim() != 2:
        raise ValueError("slot must be [tokens, k]")
    _check(slot, "slot", torch.int32, slot.shape, dev)
    _check(weight, "weight", torch.float32, slot.shape, dev)


def expert_combine_fwd(y, slot, weight=None, residual=None, out=None):
    """The experts' rows back to their tokens on the GPU: out[t] = residual[t] +
    sum_j weight[t, j] y[slot[t, j]], summed in float32.

    y: [rows, dim] (float32 or bfloat16); slot: [tokens, k] int32, one outside
    the rows adds nothing; weight: [tokens, k] float32 (None: ones); residual:
    [tokens, dim], float32 or bfloat16 (its own choice), which is then out's type
    (y's without).  out may be residual itself, to add in place.
    """
    code = _act(y, "y")
    if y.dim() != 2:
        raise ValueError("y must be [rows, dim]")
    dev = y.device
    rows, dim = y.shape
    _check(y, "y", y.dtype, y.shape, dev)
    _slots(slot, weight, dev)
    tokens, k = slot.shape
    rcode, rtype = code, y.dtype
    if residual is not None:
        rcode, rtype = _act(residual, "residual"), residual.dtype
        _check(residual, "residual", rtype, (tokens, dim), dev)
    if out is None:
        out = torch.empty((tokens, dim), dtype=rtype, device=dev)
    else:
        _check(out, "out", rtype, (tokens, dim), dev)
    dims = _lib.OrderDims(tokens, rows, dim, k, code, rcode)
    with _on(dev):
        rc = _lib.load().expert_combine_fwd(_ptr(y), _ptr(slot), _ptr(weight), _ptr(residual),
                                            _ptr(out), byref(dims), _stream(dev))
    _raise(rc)
    return out


def expert_combine_bwd(dout, y, slot, weight, dy=None):
    """Backward of expert_combine_fwd on the GPU (residual's gradient is dout).

    dout: [tokens, dim], the gradient of out; y, slot, weight as in the forward.
    Returns a dict: dy [rows, dim] in y's type (a row that no slot names is left
    as it is: give dy to choose what) and, where weight is not None, dweight
    [tokens, k] float32.  A row may be in one slot only.
    """
    code, rcode = _act(y, "y"), _act(dout, "dout")
    if y.dim() != 2:
        raise ValueError("y must be [rows, dim]")
    dev = y.device
    rows, dim = y.shape
    _check(y, "y", y.dtype, y.shape, dev)
    _slots(slot, weight, dev)
    tokens, k = slot.shape
    _check(dout, "dout", dout.dtype, (tokens, dim), dev)
    if dy is None:
        dy = _like(y)
    else:
        _check(dy, "dy", y.dtype, y.shape, dev)
    g = dict(dy=dy)
    if weight is not None:
        g["dweight"] = torch.empty_like(weight)
    dims = _lib.OrderDims(tokens, rows, dim, k, code, rcode)
    with _on(dev):
        rc = _lib.load().expert_combine_bwd(_ptr(dout), _ptr(y), _ptr(slot), _ptr(weight),
                                            _ptr(dy), _ptr(g.get("dweight")), byref(dims),
                                            _stream(dev))
    _raise(rc)
    return g


def _product_args(x, w, offsets, token, activation, out_code):
    """dims, device, shape of the rows' leading dimensions, nw."""
    code = _act(x, "x")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"unsupported activation {activation!r}")
    act = _ACTIVATIONS[activation]
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    dev, dtype, shape = x.device, x.dtype, x.shape
    experts = 0
    if offsets is None:
        if len(shape) < 2 or w.dim() != 2:
            raise ValueError("x must be [..., k] and w [n, k]")
        nw, k = w.shape
    else:
        if len(shape) != 2 or w.dim() != 3:
            raise ValueError("x must be [rows, k] and w [experts, n, k]")
        experts, nw, k = w.shape
        if experts == 0:
            raise ValueError("w must hold an expert")
        _check(offsets, "offsets", torch.int32, (experts + 1,), dev)
    if shape[-1] != k:
        raise ValueError(f"x has {shape[-1]} columns, w {k}")
    _check(w, "w", dtype, w.shape, dev)
    ld = _row_stride(x, "x", dtype, shape, dev)
    x_rows = x.numel() // k if k else 0
    if token is None:
        rows, lead = x_rows, shape[:-1]
    else:
        if token.dim() != 1:
            raise ValueError("token must be [rows]")
        rows = token.shape[0]
        lead = (rows,)
        _check(token, "token", torch.int32, lead, dev)
    n = nw
    if act >= _GATED:
        if nw % 2:
            raise ValueError("a gated activation needs two halves of w's rows")
        n = nw // 2
    if k % 8:
        raise ValueError("the columns of x and w must be a multiple of 8")
    return (_lib.ProductDims(rows, n, k, x_rows, ld, experts, act, code,
                             code if out_code is None else out_code), dev, lead, nw)


def _linear_fwd(x, w, offsets, token, bias, activation, residual, return_pre, out_dtype, out):
    if out_dtype is None:
        out_dtype = x.dtype if residual is None else residual.dtype
    if out_dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {out_dtype}")
    dims, dev, lead, nw = _product_args(x, w, offsets, token, activation, _DTYPES[out_dtype])
    shape = tuple(lead) + (dims.n,)
    _check(bias, "bias", torch.float32, w.shape[:-1], dev)
    _check(residual, "residual", out_dtype, shape, dev)
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.linear_fwd_work_bytes(byref(dims)), dev)
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=dev)
        else:
            _check(out, "out", out_dtype, shape, dev)
        pre = torch.empty(tuple(lead) + (nw,), dtype=x.dtype, device=dev) if return_pre else None
        rc = lib.linear_fwd(_ptr(x), _ptr(token), _ptr(w), _ptr(offsets), _ptr(bias),
                            _ptr(residual), _ptr(out), _ptr(pre), _ptr(work), byref(dims),
                            _stream(dev))
    _raise(rc)
    return (out, pre) if return_pre else out


def _linear_bwd(dout, x, w, offsets, token, activation, pre, need_dx, need_dw, bias, dx):
    ocode = _act(dout, "dout")
    dims, dev, lead, nw = _product_args(x, w, offsets, token, activation, ocode)
    lead = tuple(lead)
    _check(dout, "dout", dout.dtype, lead + (dims.n,), dev)
    if (pre is None) != (dims.activation == 0):
        raise ValueError("pre is given exactly with an activation")
    _check(pre, "pre", x.dtype, lead + (nw,), dev)
    wants = (_lib.SSM_WANT_DX * bool(need_dx) | _lib.SSM_WANT_DW * bool(need_dw)
             | _lib.SSM_WANT_DBIAS * bool(bias))
    if not wants:
        raise ValueError("no gradient is asked for")
    g = {}
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.linear_bwd_work_bytes(byref(dims), wants), dev)
        if need_dx:
            shape = lead + (dims.k,)
            if dx is None:
                dx = torch.empty(shape, dtype=x.dtype, device=dev)
            else:
                _check(dx, "dx", x.dtype, shape, dev)
            g["dx"] = dx
        if need_dw:
            g["dw"] = torch.empty_like(w)
        if bias:
            g["dbias"] = torch.empty(w.shape[:-1], dtype=torch.float32, device=dev)
        rc = lib.linear_bwd(_ptr(dout), _ptr(x), _ptr(token), _ptr(w), _ptr(offsets), _ptr(pre),
                            _ptr(g.get("dx")), _ptr(g.get("dw")), _ptr(g.get("dbias")),
                            _ptr(work), byref(dims), _stream(dev))
    _raise(rc)
    return g


def linear_fwd(x, w, bias=None, activation=None, residual=None, return_pre=False,
               out_dtype=None, out=None):
    """Linear layer with bias, activation and residual on the GPU, in one pass:
    out = act(x w^T + bias) + residual, summed in float32 and rounded once.

    x: [..., k] (float32 or bfloat16; contiguous, or column slices of one
    projection's output); w: [n, k] in x's type; bias: [n] float32; activation:
    None, "silu", "gelu" (by the normal distribution function), or, of w's first
    and second half of rows, "swiglu" (silu(first) * second) and "geglu"; residual:
    [..., n] (n / 2 with those two) of out's type, which is out_dtype, residual's
    or else x's.  out may be residual itself, to add in place.  Returns out, or
    (out, pre) with return_pre: the values before the activation, in x's type, as
    linear_bwd takes them.  k must be a multiple of 8, the tensors 16-byte aligned.
    """
    return _linear_fwd(x, w, None, None, bias, activation, residual, return_pre, out_dtype, out)


def linear_bwd(dout, x, w, activation=None, pre=None, need_dx=True, need_dw=True, bias=False):
    """Backward of linear_fwd on the GPU (residual's gradient is dout).

    dout: the gradient of out, in out's type; x, w, activation as in the forward;
    pre: what it returned with return_pre, given exactly with an activation.
    Returns a dict of those asked for: dx [..., k] and dw [n, k] in x's type and,
    with bias (a truth value), dbias [n] float32.  With an activation, or a dout of
    another type, the gradient before the activation is rounded to x's type in front
    of the two products (dbias is summed before that).
    """
    return _linear_bwd(dout, x, w, None, None, activation, pre, need_dx, need_dw, bias, None)


def _need_offsets(offsets):
    if offsets is None:
        raise ValueError("offsets is required")


def expert_linear_fwd(x, w, offsets, token=None, bias=None, activation=None, return_pre=False,
                      out_dtype=None, out=None):
    """linear_fwd over the rows of each expert on the GPU: rows offsets[e] ..
    offsets[e + 1] - 1 take w[e] and bias[e].

    w: [experts, n, k]; offsets: [experts + 1] int32 and token: [rows] int32 as
    expert_sort returns them.  With token row r of the product is x's row
    token[r] (zeros where that is none), so the tokens need no copy in the
    experts' order; without, x holds the rows in order.  bias: [experts, n]
    float32.  Returns out [rows, n], or (out, pre); rows ahead of offsets[0] (of a run
    of the order's experts, w[a:b] with offsets[a:b + 1]) and from offsets[experts] on
    are left as they are (give out to choose what).
    """
    _need_offsets(offsets)
    return _linear_fwd(x, w, offsets, token, bias, activation, None, return_pre, out_dtype, out)


def expert_linear_bwd(dout, x, w, offsets, token=None, activation=None, pre=None, need_dx=True,
                      need_dw=True, bias=False, dx=None):
    """Backward of expert_linear_fwd on the GPU.

    dout: [rows, n], the gradient of out; the rest as in the forward and in
    linear_bwd.  Returns a dict of those asked for: dx [rows, k], the gradient of
    every row in the experts' order (with token, expert_combine_fwd(dx, slot) sums
    it by token; rows of no expert are left as they are), dw
    [experts, n, k] in x's type and, with bias, dbias [experts, n] float32, zeros
    for an expert without rows.
    """
    _need_offsets(offsets)
    return _linear_bwd(dout, x, w, offsets, token, activation, pre, need_dx, need_dw, bias, dx)
