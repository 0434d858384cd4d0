"""The norm with the residual's addition, the 8-bit block format and its linear
product on the GPU against their float64 reference.

Tolerances, on the largest magnitude of the compared array unless said.  Norm,
float32: 1e-5 (a sum of at most 16384 squares in float32, pairwise over lanes:
below 30 roundings of 2^-24 in a row, and four more operations); bfloat16
outputs 4e-3 (their rounding).  dweight sums over rows in float32: 1e-5 per
row count's root is far inside 1e-4.  8-bit values: the scale to 1e-5, the
value to half a step of e4m3, max(|y| / 16, scale * 2^-10), and 1e-4 of |y| for
the float32 arithmetic that decides a tie.  Linear: a float32 sum of k products
of 8-bit values and of k / 128 scaled partial sums errs by at most
(k + 8) 2^-23 of the terms' summed magnitude, whatever the order and whether a
partial sum is rounded or cut.  bfloat16 outputs: 2^-8 of themselves on top, and
2^-11 of the terms' summed magnitude, since the 8-bit matrix instruction adds in
a window of that many bits below its largest product (measured: 2^-11.5 of it).
"""

import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 1e-5, torch.bfloat16: 4e-3}
DTYPES = [torch.float32, torch.bfloat16]


def ref(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, tol, name=""):
    got = ref(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    scale, err = np.max(np.abs(want)), np.max(np.abs(got - want))
    assert err <= tol * scale, f"{name}: {err:.3e} of {scale:.3e}"


def rand(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to("cuda", dtype)


def check_quantized(q, scale, y):
    """q, scale (GPU) of y (float64 [M, K])."""
    want_q, want_scale = layer.quantize(y)
    got_scale, got_q = ref(scale), ref(q.float())
    np.testing.assert_allclose(got_scale, want_scale, rtol=1e-5)
    by = np.repeat(got_scale.T, layer.FP8_GROUP, 1)[:, :y.shape[1]]
    bound = np.maximum(np.abs(y) / 16, by * 2.0 ** -10) + 1e-4 * np.abs(y)
    assert (np.abs(got_q * by - y) <= bound).all()
    assert np.max(np.abs(got_q)) <= layer.FP8_MAX
    # the same code but for values that float32 puts on the other side of a tie
    assert np.mean(got_q != want_q) <= 1e-3 + 1.0 / y.size


NORM_SHAPES = [(1, 16), (3, 128), (5, 144), (2, 768), (7, 1536), (33, 2560), (4, 4112), (3, 5120),
               (2, 8192), (2, 16384), (1030, 256)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [None] + DTYPES)
@pytest.mark.parametrize("rows,dim", NORM_SHAPES + [(3, 1), (4, 17), (5, 1001), (2, 16383)])
def test_norm(rows, dim, residual, dtype):
    from selective_state_space_38_amd import rms_norm_fwd
    x, w = rand(rows, dim, dtype=dtype), 1 + rand(dim, seed=1, scale=0.2)
    res = None if residual is None else rand(rows, dim, dtype=residual, seed=2, scale=3.0)
    y, s = layer.rms_norm(ref(x), ref(w), ref(res))
    got = rms_norm_fwd(x, w, residual=res)
    if res is None:
        close(got, y, TOL[dtype], "y")
        return
    close(got[0], y, TOL[dtype], "y")
    close(got[1], s, TOL[residual], "s")
    # added in place
    own = res.clone()
    again = rms_norm_fwd(x, w, residual=own, residual_out=own)
    assert again[1] is own and torch.equal(own, got[1]) and torch.equal(again[0], got[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [None] + DTYPES)
@pytest.mark.parametrize("rows,dim", NORM_SHAPES)
def test_norm_fp8(rows, dim, residual, dtype):
    from selective_state_space_38_amd import rms_norm_fp8
    x, w = rand(rows, dim, dtype=dtype), 1 + rand(dim, seed=1, scale=0.2)
    res = None if residual is None else rand(rows, dim, dtype=residual, seed=2, scale=3.0)
    y, s = layer.rms_norm(ref(x), ref(w), ref(res))
    got = rms_norm_fp8(x, w, residual=res)
    assert got[0].dtype == torch.float8_e4m3fn and got[1].shape == (-(-dim // 128), rows)
    check_quantized(got[0], got[1], y)
    if res is not None:
        close(got[2], s, TOL[residual], "s")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim", NORM_SHAPES)
def test_quantize(rows, dim, dtype):
    from selective_state_space_38_amd import fp8_quantize
    x = rand(rows, dim, dtype=dtype)
    x[0] = 0.0                   # a row of zeros
    x[-1, :16] *= 2.0 ** -90     # values far below the others of their group
    if rows > 2:
        x[1] *= 2.0 ** 100
        x[2] *= 2.0 ** -110      # below the format's smallest scale
    q, scale = fp8_quantize(x)
    check_quantized(q, scale, ref(x))
    assert not q[0].float().any()


def test_quantize_non_finite_values_stay_in_their_group():
    from selective_state_space_38_amd import fp8_quantize, rms_norm_fwd
    x = rand(3, 512)
    x[1, 200] = float("nan")
    q, scale = fp8_quantize(x)
    clean = x.clone()
    clean[1, 200] = 0.0
    cq, cscale = fp8_quantize(clean)
    q, cq = q.float(), cq.float()
    assert torch.isnan(q[1, 200])
    for rows, cols in ((slice(0, 1), slice(None)), (slice(2, 3), slice(None)),
                       (slice(1, 2), slice(0, 128)), (slice(1, 2), slice(256, 512))):
        assert torch.equal(q[rows, cols], cq[rows, cols])
    y = rms_norm_fwd(x, torch.ones(512, device="cuda"))
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


def test_norm_of_zeros():
    from selective_state_space_38_amd import rms_norm_bwd, rms_norm_fp8, rms_norm_fwd
    x, w = torch.zeros(4, 256, device="cuda"), torch.ones(256, device="cuda")
    assert not rms_norm_fwd(x, w).any()
    q, scale = rms_norm_fp8(x, w)
    assert not q.float().any() and torch.isfinite(scale).all() and (scale > 0).all()
    g = rms_norm_bwd(torch.ones_like(x), x, w)
    assert torch.isfinite(g["ds"]).all() and not g["dweight"].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("stream", DTYPES)
@pytest.mark.parametrize("rows,dim", NORM_SHAPES + [(3, 1), (4, 17), (5, 1001), (2, 16383)])
def test_norm_backward(rows, dim, stream, dtype):
    from selective_state_space_38_amd import rms_norm_bwd
    dy, s = rand(rows, dim, dtype=dtype), rand(rows, dim, dtype=stream, seed=1, scale=3.0)
    w = 1 + rand(dim, seed=2, scale=0.2)
    for dres in (None, rand(rows, dim, dtype=stream, seed=3)):
        g = rms_norm_bwd(dy, s, w, dres=dres)
        want = layer.rms_norm_grad(ref(dy), ref(s), ref(w), dres=ref(dres))
        close(g["ds"], want["ds"], max(TOL[stream], 1e-5), "ds")
        close(g["dweight"], want["dweight"], 1e-4, "dweight")
        again = rms_norm_bwd(dy, s, w, dres=dres)
        assert all(torch.equal(g[k], again[k]) for k in g)


def test_norm_gradient_against_differences():
    # step 1e-2: third-derivative error about 1e-4, rounding 1e-6 / 1e-2
    from selective_state_space_38_amd import rms_norm_bwd, rms_norm_fwd
    x, dy, w = rand(6, 300), rand(6, 300, seed=1), 1 + rand(300, seed=2, scale=0.2)
    g = rms_norm_bwd(dy, x, w)
    for way, key in ((rand(6, 300, seed=3), "ds"), (rand(300, seed=4), "dweight")):
        def value(eps):
            y = rms_norm_fwd(x + eps * way, w) if key == "ds" else rms_norm_fwd(x, w + eps * way)
            return float((y.double() * dy.double()).sum())
        want = (value(1e-2) - value(-1e-2)) / 2e-2
        got = float((g[key].double() * way.double()).sum())
        assert abs(got - want) <= 3e-3 * max(abs(want), float((g[key] * way).norm()))


def linear_inputs(m, n, k, seed=0):
    xq, xs = layer.quantize(np.random.default_rng(seed).standard_normal((m, k)))
    wq, ws = layer.quantize(np.random.default_rng(seed + 1).standard_normal((n, k)) / k ** 0.5, 128)
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).float().cuda()  # noqa: E731
    return (dev(xq).to(torch.float8_e4m3fn), dev(xs), dev(wq).to(torch.float8_e4m3fn), dev(ws))


def check_linear(args, bias, dtype, out):
    want, size = layer.linear(ref(args[0].float()), ref(args[1]), ref(args[2].float()),
                              ref(args[3]), ref(bias))
    k = args[0].shape[1]
    bound = (k + 8) * 2.0 ** -23 * size
    if dtype == torch.bfloat16:
        bound = bound + np.abs(want) * 2.0 ** -8 + size * 2.0 ** -11
    err = np.abs(ref(out) - want)
    assert out.dtype == dtype and err.shape == want.shape
    assert (err <= bound).all(), float(np.max(err / np.maximum(bound, 1e-30)))


LINEAR = [(1, 16, 16), (1, 1, 32), (1, 768, 256), (2, 130, 144), (7, 257, 128), (8, 5120, 2560),
          (16, 48, 1536), (17, 1536, 768), (31, 100, 2576), (33, 129, 400), (64, 512, 640),
          (65, 384, 1024), (100, 1000, 112), (128, 128, 128), (129, 127, 272), (250, 640, 512),
          (333, 1536, 768), (513, 260, 1040), (1025, 1030, 384), (2048, 768, 1536)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(m, n, k, dtype):
    from selective_state_space_38_amd import fp8_linear
    args = linear_inputs(m, n, k, seed=m)
    for bias in (None, rand(n, seed=5)):
        out = fp8_linear(*args, bias=bias, out_dtype=dtype)
        check_linear(args, bias, dtype, out)
        assert torch.equal(out, fp8_linear(*args, bias=bias, out_dtype=dtype))


def test_linear_large_against_float64_on_the_gpu():
    from selective_state_space_38_amd import fp8_linear, fp8_quantize, fp8_quantize_weight
    m, n, k = 4099, 2570, 2560
    x, w = rand(m, k), rand(n, k, seed=1, scale=k ** -0.5)
    xq, xs = fp8_quantize(x)
    wq, ws = fp8_quantize_weight(w)
    xd = xq.double() * xs.double().t().repeat_interleave(128, 1)[:, :k]
    wd = wq.double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    want = xd @ wd.t().contiguous()
    out = fp8_linear(xq, xs, wq, ws, out_dtype=torch.float32).double()
    # rounding errors of both signs: within the root of their count
    assert float((out - want).norm() / want.norm()) <= k ** 0.5 * 2.0 ** -23
    # and what the format itself costs: two 8-bit roundings of up to 2^-4
    full = x.double() @ w.double().t().contiguous()
    assert float((want - full).norm() / full.norm()) < 0.06


def test_linear_rows_do_not_touch_each_other():
    from selective_state_space_38_amd import fp8_linear
    args = linear_inputs(40, 200, 256)
    clean = fp8_linear(*args, out_dtype=torch.float32)
    xq = args[0].clone()
    xq.view(torch.uint8)[13, 7] = 0x7f  # NaN
    out = fp8_linear(xq, *args[1:], out_dtype=torch.float32)
    assert torch.isnan(out[13]).all()
    rest = [r for r in range(40) if r != 13]
    assert torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (130, 200), (768, 48), (257, 1537)])
def test_quantize_weight(n, k, dtype):
    from selective_state_space_38_amd import fp8_quantize_weight
    w = rand(n, k, dtype=dtype)
    q, scale = fp8_quantize_weight(w)
    want_q, want_scale = layer.quantize(ref(w), 128)
    np.testing.assert_allclose(ref(scale), want_scale, rtol=1e-6)
    assert np.mean(ref(q.float()) != want_q) <= 1e-3 + 1.0 / want_q.size


def test_streams_and_graph():
    from selective_state_space_38_amd import (fp8_linear, fp8_quantize_weight, rms_norm_bwd,
                                              rms_norm_fp8)
    x, res, norm_w = rand(200, 1024, dtype=torch.bfloat16), rand(200, 1024, seed=1), \
        1 + rand(1024, seed=2, scale=0.1)
    wq, ws = fp8_quantize_weight(rand(384, 1024, seed=3, scale=0.03))

    def call():
        q, scale, s = rms_norm_fp8(x, norm_w, residual=res)
        out = fp8_linear(q, scale, wq, ws)
        return (out, s, *rms_norm_bwd(x, s, norm_w).values())

    want = call()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = call()
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for k in range(4):
        x.copy_(rand(200, 1024, dtype=torch.bfloat16, seed=10 + k))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_offsets_past_32_bits():
    from selective_state_space_38_amd import fp8_linear, rms_norm_fp8, rms_norm_fwd
    rows, dim = 140000, 16384
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(dim, device="cuda")
    y = rms_norm_fwd(x, w)
    assert torch.equal(y[-5:], rms_norm_fwd(x[-5:].contiguous(), w))
    q, scale = rms_norm_fp8(x, w)
    q5, s5 = rms_norm_fp8(x[-5:].contiguous(), w)
    assert torch.equal(q[-5:].view(torch.uint8), q5.view(torch.uint8))
    assert torch.equal(scale[:, -5:], s5)
    del x, y, q
    m, n, k = 600000, 4096, 32
    args = linear_inputs(64, n, k)
    xq = args[0].view(torch.uint8).repeat(m // 64, 1).view(torch.float8_e4m3fn)
    xs = args[1].repeat(1, m // 64)
    out = fp8_linear(xq, xs, *args[2:])
    small = fp8_linear(xq[:640].contiguous(), xs[:, :640].contiguous(), *args[2:])
    assert torch.equal(out[-640:], small)


def test_refusals():
    from selective_state_space_38_amd import (fp8_linear, fp8_quantize, fp8_quantize_weight,
                                              rms_norm_bwd, rms_norm_fp8, rms_norm_fwd)
    x, w = rand(4, 64), torch.ones(64, device="cuda")
    for f in (rms_norm_fwd, rms_norm_fp8):
        with pytest.raises(ValueError):
            f(x.half(), w)
        with pytest.raises(ValueError):
            f(x, w[:32])
        with pytest.raises(ValueError):
            f(x, w.bfloat16())
        with pytest.raises(ValueError):
            f(x.t(), w)
        with pytest.raises(ValueError):
            f(x, w, residual=rand(4, 32))
        with pytest.raises(ValueError):
            f(x, w, residual_out=x)
        with pytest.raises(RuntimeError):
            f(x, w, eps=0.0)
        with pytest.raises(RuntimeError):
            f(x, w, eps=float("nan"))
        with pytest.raises(RuntimeError):
            f(x[:0], w)
    with pytest.raises(RuntimeError):
        rms_norm_fwd(rand(1, 16385), torch.ones(16385, device="cuda"))
    with pytest.raises(RuntimeError):  # 8-bit rows are moved 16 values at a time
        fp8_quantize(rand(4, 24))
    with pytest.raises(RuntimeError):  # not 16-byte aligned
        fp8_quantize(rand(65)[1:].view(4, 16))
    with pytest.raises(ValueError):
        rms_norm_bwd(x, rand(4, 32), w)
    with pytest.raises(ValueError):
        rms_norm_bwd(x, x, w, dres=x.bfloat16())
    with pytest.raises(ValueError):
        fp8_quantize_weight(x[0])
    args = linear_inputs(4, 16, 64)
    with pytest.raises(ValueError):
        fp8_linear(args[0].float(), *args[1:])
    with pytest.raises(ValueError):
        fp8_linear(args[0], args[1].t().contiguous(), *args[2:])
    with pytest.raises(ValueError):
        fp8_linear(*args, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fp8_linear(*args, bias=torch.zeros(4, device="cuda"))
    with pytest.raises(RuntimeError):
        fp8_linear(*linear_inputs(4, 16, 24))
    with pytest.raises(RuntimeError):
        fp8_linear(args[0][:0], args[1][:, :0].contiguous(), *args[2:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [1, 2, 3])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (5, 130, 144), (65, 264, 400), (130, 72, 128),
                                   (257, 300, 1296), (300, 520, 272), (513, 257, 2064)])
def test_linear_tiles(m, n, k, shape, dtype, monkeypatch):
    """Every tile shape, whole and with the inputs split into parts."""
    from selective_state_space_38_amd import fp8_linear
    args, bias = linear_inputs(m, n, k, seed=m), rand(n, seed=5)
    monkeypatch.setenv("SSM_FORCE_LINEAR_SHAPE", str(shape))
    for parts in (1, 2, 3, 7):
        monkeypatch.setenv("SSM_FORCE_LINEAR_PARTS", str(parts))
        for b in (None, bias):
            check_linear(args, b, dtype, fp8_linear(*args, bias=b, out_dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_output_alignment(dtype):
    # an output that starts one element into its buffer, for every path
    from selective_state_space_38_amd import fp8_linear
    for m, n, k in ((3, 64, 256), (70, 128, 256), (1100, 1536, 128), (300, 64, 2048)):
        args = linear_inputs(m, n, k)
        buf = torch.full((m * n + 2,), 7.0, dtype=dtype, device="cuda")
        out = buf[1:-1].view(m, n)
        fp8_linear(*args, out_dtype=dtype, out=out)
        assert torch.equal(out, fp8_linear(*args, out_dtype=dtype))
        assert float(buf[0]) == float(buf[-1]) == 7.0
