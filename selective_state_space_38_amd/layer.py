"""PyTorch-facing binding of the residual layer's operators: the gated linear
recurrence, the root-mean-square norm with the residual's addition and an
8-bit output, and the linear product of 8-bit operands with block scales.

As in ``api``: argument marshalling only.  Scratch comes from torch's caching
allocator on the current stream, so the calls can be captured into a graph.
"""

import contextlib
from ctypes import byref

import torch

from . import _lib
from . import api
from .api import _DTYPES, _raise

FP8 = torch.float8_e4m3fn
FP8_GROUP = 128

# The calls for a few tokens last some microseconds, most of them here: the
# checks below take the common case in one condition, and the device is entered
# only where it is not the current one (entering it and torch's stream object
# cost 1.3 and 1.9 us, these two 0.4 together).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_NO_CONTEXT = contextlib.nullcontext()


def _on(device):
    if device.index == _current_device():
        return _NO_CONTEXT
    return torch.cuda.device(device)


def _stream(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype, shape, device):
    if t is None or (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape
                     and t.device == device and t.is_contiguous()):
        return
    api._check(t, name, dtype, shape, device)


def _act(t, name):
    """dtype code of an activation tensor on a GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU, not on {t.device}")
    return _DTYPES[t.dtype]


def _row_stride(t, name, dtype, shape, device):
    """Elements between consecutive rows of t, whose last dimension is
    contiguous and whose other dimensions step evenly (a contiguous tensor, or
    column slices of one)."""
    dim = shape[-1]
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device:
        if t.is_contiguous():
            return dim
        s = t.stride()  # the usual slices: 1.2 us less for three than the checks below
        if len(s) == 3:
            if s[2] == 1 and s[1] >= dim and shape[1] > 1 and s[0] == s[1] * shape[1]:
                return s[1]
        elif len(s) == 2 and s[1] == 1 and s[0] >= dim and shape[0] > 1:
            return s[0]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return dim
    strides = t.stride()
    if dim > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    ld, rows = None, 1
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size != 1:
            if ld is None:
                ld = stride
            if stride != ld * rows:
                raise ValueError(f"the rows of {name} must be evenly spaced")
        rows *= size
    if ld is None:
        return dim
    if ld < dim:
        raise ValueError(f"the rows of {name} overlap")
    return ld


def _like(x):
    """A contiguous tensor of x's type and shape (torch.empty costs 0.5 us more)."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _work(nbytes, device):
    _raise(nbytes if nbytes < 0 else 0)
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _gated_args(x, r, i, log_decay, shape):
    code = _act(x, "x")
    dev, dtype, dim = x.device, x.dtype, shape[-1]
    if log_decay is None:
        raise ValueError("log_decay is required")
    _check(log_decay, "log_decay", torch.float32, (dim,), dev)
    return _lib.GatedDims(shape[0], shape[1] if len(shape) == 3 else 1, dim,
                          _row_stride(x, "x", dtype, shape, dev),
                          _row_stride(r, "r", dtype, shape, dev),
                          _row_stride(i, "i", dtype, shape, dev), code), dev


def _check_reset(reset, shape, dev):
    if reset is not None and reset.dtype != torch.uint8:
        _check(reset, "reset", torch.bool, shape, dev)
    else:
        _check(reset, "reset", torch.uint8, shape, dev)


def _check_ckpt(ckpt, dims, dev):
    if ckpt is None:
        return
    if ckpt.dtype != torch.float32 or ckpt.device != dev or not ckpt.is_contiguous():
        raise ValueError("ckpt must be a contiguous float32 tensor on the same device")
    if ckpt.numel() * 4 < _lib.load().gated_ckpt_bytes(byref(dims)):
        raise ValueError("ckpt is too small (use gated_ckpt_buffer)")


def gated_ckpt_buffer(x):
    """A float32 device buffer for the gated recurrence's training pair (the
    state before every 16th step) of activations x [batch, L, dim]."""
    bsz, L, dim = x.shape
    dims = _lib.GatedDims(bsz, L, dim, dim, dim, dim, _act(x, "x"))
    nbytes = _lib.load().gated_ckpt_bytes(byref(dims))
    _raise(nbytes if nbytes < 0 else 0)
    return torch.empty(nbytes // 4, dtype=torch.float32, device=x.device)


def gated_scan_fwd(x, r, i, log_decay, reset=None, h0=None, return_last_state=False, out=None,
                   last_state=None, ckpt=None):
    """Gated linear recurrence over a sequence on the GPU.

    With a = exp(log_decay * sigmoid(r)): h_t = a_t h_{t-1} +
    sqrt(1 - a_t^2) sigmoid(i_t) x_t, per channel; returns out = h (x's dtype)
    and, with return_last_state, the float32 state after the last step.

    x, r, i: [batch, L, dim] (float32 or bfloat16, all the same; contiguous,
    or column slices of one projection's output); log_decay: [dim] float32,
    <= 0; reset: [batch, L] bool or uint8, true where a document starts (the
    state before is dropped, r is not used and the input is taken with weight
    sigmoid(i));
    h0: [batch, dim] float32.  ckpt: a buffer from gated_ckpt_buffer() that
    keeps what gated_scan_bwd starts from.
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, dim]")
    shape = x.shape
    dims, dev = _gated_args(x, r, i, log_decay, shape)
    bsz, L, dim = shape
    _check_reset(reset, (bsz, L), dev)
    _check(h0, "h0", torch.float32, (bsz, dim), dev)
    _check_ckpt(ckpt, dims, dev)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", x.dtype, shape, dev)
    if return_last_state and last_state is None:
        last_state = (torch.empty((bsz, dim), dtype=torch.float32, device=dev) if h0 is None
                      else torch.empty_like(h0))
    _check(last_state, "last_state", torch.float32, (bsz, dim), dev)
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.gated_scan_work_bytes(byref(dims)), dev)
        rc = lib.gated_scan_fwd(_ptr(x), _ptr(r), _ptr(i), _ptr(log_decay), _ptr(reset),
                                _ptr(h0), _ptr(out), _ptr(last_state), _ptr(ckpt), _ptr(work),
                                byref(dims), _stream(dev))
    _raise(rc)
    return (out, last_state) if return_last_state else out


def gated_scan_bwd(x, r, i, log_decay, dout, reset=None, h0=None, dlast=None, ckpt=None):
    """Backward of gated_scan_fwd on the GPU.

    Inputs as in the forward, plus dout [batch, L, dim], the gradient of the
    output, and dlast [batch, dim] float32 (optional), the gradient of the
    last state.  Returns a dict: dx, dr, di [batch, L, dim] in x's dtype,
    dlog_decay [dim] and, where h0 is given, dh0 [batch, dim] in float32.
    ckpt: the buffer the forward filled on the same inputs (without it the
    call runs the forward's recurrence itself).
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, dim]")
    shape = x.shape
    dims, dev = _gated_args(x, r, i, log_decay, shape)
    bsz, L, dim = shape
    _check_reset(reset, (bsz, L), dev)
    _check(h0, "h0", torch.float32, (bsz, dim), dev)
    if dout is None:
        raise ValueError("dout is required")
    _check(dout, "dout", x.dtype, shape, dev)
    _check(dlast, "dlast", torch.float32, (bsz, dim), dev)
    _check_ckpt(ckpt, dims, dev)
    g = {k: _like(x) for k in ("dx", "dr", "di")}
    g["dlog_decay"] = torch.empty_like(log_decay)
    if h0 is not None:
        g["dh0"] = torch.empty_like(h0)
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.gated_scan_bwd_work_bytes(byref(dims), int(ckpt is not None)),
                     dev)
        rc = lib.gated_scan_bwd(_ptr(x), _ptr(r), _ptr(i), _ptr(log_decay), _ptr(reset),
                                _ptr(h0), _ptr(dout), _ptr(dlast), _ptr(ckpt), _ptr(g["dx"]),
                                _ptr(g["dr"]), _ptr(g["di"]), _ptr(g["dlog_decay"]),
                                _ptr(g.get("dh0")), _ptr(work), byref(dims),
                                _stream(dev))
    _raise(rc)
    return g


def gated_state_update(state, x, r, i, log_decay, out=None):
    """One step of the gated recurrence on the GPU, updating ``state``
    ([batch, dim] float32) in place.  x, r, i: [batch, dim].  Returns out
    [batch, dim] in x's dtype."""
    if x.dim() != 2:
        raise ValueError("x must be [batch, dim]")
    shape = x.shape
    dims, dev = _gated_args(x, r, i, log_decay, shape)
    if state is None:
        raise ValueError("state is required")
    _check(state, "state", torch.float32, shape, dev)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", x.dtype, shape, dev)
    with _on(dev):
        rc = _lib.load().gated_state_update(_ptr(state), _ptr(x), _ptr(r), _ptr(i),
                                            _ptr(log_decay), _ptr(out), byref(dims),
                                            _stream(dev))
    _raise(rc)
    return out


def _rows(x, name):
    code = _act(x, name)
    if x.dim() < 2:
        raise ValueError(f"{name} must be [..., dim]")
    dim = x.shape[-1]
    return code, x.numel() // dim if dim else 0, dim


def _norm_args(x, weight, residual, residual_out):
    code, rows, dim = _rows(x, "x")
    dev, shape = x.device, x.shape
    _check(x, "x", x.dtype, shape, dev)
    if weight is None:
        raise ValueError("weight is required")
    _check(weight, "weight", torch.float32, (dim,), dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs residual")
        return _lib.NormDims(rows, dim, code, code), dev, None
    rcode = _act(residual, "residual")
    _check(residual, "residual", residual.dtype, shape, dev)
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    else:
        _check(residual_out, "residual_out", residual.dtype, shape, dev)
    return _lib.NormDims(rows, dim, code, rcode), dev, residual_out


def rms_norm_fwd(x, weight, residual=None, eps=1e-5, out=None, residual_out=None):
    """Root-mean-square norm on the GPU, with the residual's addition in front:
    s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight.

    x: [..., dim] (float32 or bfloat16); weight: [dim] float32; residual:
    [..., dim], float32 or bfloat16 (its own choice).  Returns y (x's dtype)
    or, where residual is given, (y, s) with s in residual's dtype;
    residual_out may be residual itself, to add in place.
    """
    dims, dev, residual_out = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", x.dtype, x.shape, dev)
    with _on(dev):
        rc = _lib.load().rms_norm_fwd(_ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(out),
                                      _ptr(residual_out), byref(dims), _stream(dev))
    _raise(rc)
    return out if residual is None else (out, residual_out)


def _fp8_outputs(x, rows, dim, dev):
    q = torch.empty_like(x, dtype=FP8)
    scale = torch.empty((-(-dim // FP8_GROUP), rows), dtype=torch.float32, device=dev)
    return q, scale


def rms_norm_fp8(x, weight, residual=None, eps=1e-5, residual_out=None):
    """rms_norm_fwd with its output in 8 bits: returns (q, scale) or, where
    residual is given, (q, scale, s).  q: x's shape, float8_e4m3fn; scale:
    [ceil(dim / 128), rows] float32, y ~ q * scale for every 128 values of a
    row (rows are x's leading dimensions, flattened).  dim must be a multiple
    of 16."""
    dims, dev, residual_out = _norm_args(x, weight, residual, residual_out)
    q, scale = _fp8_outputs(x, dims.rows, dims.dim, dev)
    with _on(dev):
        rc = _lib.load().rms_norm_fp8(_ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(q),
                                      _ptr(scale), _ptr(residual_out), byref(dims),
                                      _stream(dev))
    _raise(rc)
    return (q, scale) if residual is None else (q, scale, residual_out)


def fp8_quantize(x):
    """x [..., dim] (float32 or bfloat16) in 8 bits with a scale for every 128
    values of a row: (q, scale) as rms_norm_fp8 returns them."""
    code, rows, dim = _rows(x, "x")
    _check(x, "x", x.dtype, x.shape, x.device)
    dims = _lib.NormDims(rows, dim, code, code)
    q, scale = _fp8_outputs(x, rows, dim, x.device)
    with _on(x.device):
        rc = _lib.load().fp8_quantize(_ptr(x), _ptr(q), _ptr(scale), byref(dims),
                                      _stream(x.device))
    _raise(rc)
    return q, scale


def rms_norm_bwd(dy, s, weight, eps=1e-5, dres=None):
    """Backward of rms_norm_fwd on the GPU.  dy: [..., dim], the gradient of y;
    s: the normalised sum (the s that rms_norm_fwd returned, or x where there
    was no residual); dres (optional, s's dtype): the gradient that reaches s
    on the residual's own way.  Returns a dict: ds (s's dtype), the gradient of
    both x and residual, and dweight [dim] float32."""
    code, rows, dim = _rows(dy, "dy")
    dev, shape = dy.device, dy.shape
    scode = _act(s, "s")
    _check(dy, "dy", dy.dtype, shape, dev)
    _check(s, "s", s.dtype, shape, dev)
    if weight is None:
        raise ValueError("weight is required")
    _check(weight, "weight", torch.float32, (dim,), dev)
    _check(dres, "dres", s.dtype, shape, dev)
    dims = _lib.NormDims(rows, dim, code, scode)
    g = dict(ds=torch.empty_like(s), dweight=torch.empty_like(weight))
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.rms_norm_bwd_work_bytes(byref(dims)), dev)
        rc = lib.rms_norm_bwd(_ptr(dy), _ptr(s), _ptr(weight), eps, _ptr(dres), _ptr(g["ds"]),
                              _ptr(g["dweight"]), _ptr(work), byref(dims), _stream(dev))
    _raise(rc)
    return g


def fp8_quantize_weight(w):
    """A linear layer's weight [n, k] (float32 or bfloat16) in 8 bits:
    (wq [n, k] float8_e4m3fn, w_scale [ceil(n / 128), ceil(k / 128)] float32),
    one scale for every tile of 128 x 128.  Any k is converted; fp8_linear takes
    multiples of 16 (pad the inputs with zeros)."""
    code = _act(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [n, k]")
    n, k = w.shape
    _check(w, "w", w.dtype, (n, k), w.device)
    q = torch.empty((n, k), dtype=FP8, device=w.device)
    scale = torch.empty((-(-n // FP8_GROUP), -(-k // FP8_GROUP)), dtype=torch.float32,
                        device=w.device)
    with _on(w.device):
        rc = _lib.load().fp8_quantize_weight(_ptr(w), code, n, k, _ptr(q), _ptr(scale),
                                             _stream(w.device))
    _raise(rc)
    return q, scale


def fp8_linear(xq, x_scale, wq, w_scale, bias=None, out_dtype=torch.bfloat16, out=None):
    """Linear layer on 8-bit operands on the GPU.

    xq [..., k] float8_e4m3fn with x_scale [ceil(k / 128), rows] (from
    rms_norm_fp8 or fp8_quantize); wq [n, k], w_scale (from
    fp8_quantize_weight); bias: [n] float32.  k must be a multiple of 16.
    Returns out [..., n] in out_dtype (float32 or bfloat16).

    float32 outputs, and bfloat16 ones of up to 32 rows, are summed in float32.
    bfloat16 outputs of more rows are summed by the 8-bit matrix instruction,
    128 inputs at a time, which cuts the products of every 8 inputs at 2^-13 of
    the largest: below the output's own rounding unless the terms cancel.  Where
    that matters, ask for float32 (half the rate) and convert.
    """
    if not isinstance(xq, torch.Tensor) or not isinstance(wq, torch.Tensor):
        raise TypeError("xq and wq must be torch.Tensors")
    if xq.device.type != "cuda":
        raise ValueError(f"xq must be on the GPU, not on {xq.device}")
    if xq.dim() < 2 or wq.dim() != 2:
        raise ValueError("xq must be [..., k] and wq [n, k]")
    if out_dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {out_dtype}")
    if x_scale is None or w_scale is None:
        raise ValueError("x_scale and w_scale are required")
    dev = xq.device
    n, k = wq.shape
    lead = tuple(xq.shape[:-1])
    rows = xq.numel() // k if k else 0
    groups = -(-k // FP8_GROUP)
    _check(xq, "xq", FP8, lead + (k,), dev)
    _check(wq, "wq", FP8, (n, k), dev)
    _check(x_scale, "x_scale", torch.float32, (groups, rows), dev)
    _check(w_scale, "w_scale", torch.float32, (-(-n // FP8_GROUP), groups), dev)
    _check(bias, "bias", torch.float32, (n,), dev)
    if out is None:
        out = torch.empty(lead + (n,), dtype=out_dtype, device=dev)
    else:
        _check(out, "out", out_dtype, lead + (n,), dev)
    dims = _lib.LinearDims(rows, n, k, _DTYPES[out_dtype])
    lib = _lib.load()
    with _on(dev):
        work = _work(lib.fp8_linear_work_bytes(byref(dims)), dev)
        rc = lib.fp8_linear(_ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias),
                            _ptr(out), _ptr(work), byref(dims), _stream(dev))
    _raise(rc)
    return out
