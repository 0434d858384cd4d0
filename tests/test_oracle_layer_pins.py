"""The residual layer's float64 reference against independent facts: closed
forms and central differences (CPU)."""

import numpy as np
import pytest

from oracle import layer

RNG = np.random.default_rng


def _inputs(seed, bsz=2, length=7, dim=5):
    g = RNG(seed)
    x, r, i, dout = (g.standard_normal((bsz, length, dim)) for _ in range(4))
    lam = -np.exp(g.uniform(np.log(0.005), np.log(4.0), dim))
    reset = np.zeros((bsz, length), bool)
    reset[0, 3] = reset[1, 0] = True
    return dict(x=x, r=r, i=i, lam=lam, dout=dout, reset=reset, h0=g.standard_normal((bsz, dim)),
                dlast=g.standard_normal((bsz, dim)))


def test_recurrence_closed_form():
    v = _inputs(0)
    out, last = layer.gated_scan(v["x"], v["r"], v["i"], v["lam"], None, v["h0"])
    sig = lambda t: 1 / (1 + np.exp(-t))  # noqa: E731
    a = np.exp(v["lam"] * sig(v["r"]))
    b = np.sqrt(1 - a * a) * sig(v["i"]) * v["x"]
    for t in range(out.shape[1]):
        want = np.prod(a[:, :t + 1], 1) * v["h0"]
        for s in range(t + 1):
            want = want + np.prod(a[:, s + 1:t + 1], 1) * b[:, s]
        np.testing.assert_allclose(out[:, t], want, rtol=1e-12)
    np.testing.assert_array_equal(last, out[:, -1])


def test_recurrence_keeps_a_constant_variance():
    # beta^2 = 1 - a^2: white input of variance s^2 gives a state of variance s^2
    g = RNG(1)
    length, dim = 400, 4000
    x = g.standard_normal((1, length, dim))
    one = np.full((1, length, dim), 50.0)  # both gates open
    out, _ = layer.gated_scan(x, one, one, np.full(dim, -0.05))
    assert abs(np.var(out[:, -1]) - 1.0) < 0.1


def test_reset_starts_anew():
    v = _inputs(2)
    out, _ = layer.gated_scan(v["x"], v["r"], v["i"], v["lam"], v["reset"], v["h0"])
    sig_i = 1 / (1 + np.exp(-v["i"]))
    np.testing.assert_allclose(out[0, 3], sig_i[0, 3] * v["x"][0, 3], rtol=1e-13)
    # after the reset: as a sequence of its own from that state
    rest, _ = layer.gated_scan(v["x"][:1, 4:], v["r"][:1, 4:], v["i"][:1, 4:], v["lam"], None,
                               out[:1, 3])
    np.testing.assert_allclose(out[:1, 4:], rest, rtol=1e-13)


def _difference(f, a, eps=1e-6):
    g = np.empty_like(a)
    flat, gf = a.reshape(-1), g.reshape(-1)
    for j in range(flat.size):
        keep = flat[j]
        flat[j] = keep + eps
        hi = f()
        flat[j] = keep - eps
        lo = f()
        flat[j] = keep
        gf[j] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("with_reset", [False, True])
def test_recurrence_gradient_against_differences(with_reset):
    v = _inputs(3, length=5, dim=3)
    reset = v["reset"] if with_reset else None

    def value():
        out, last = layer.gated_scan(v["x"], v["r"], v["i"], v["lam"], reset, v["h0"])
        return np.sum(v["dout"] * out) + np.sum(v["dlast"] * last)

    g = layer.gated_scan_grad(v["x"], v["r"], v["i"], v["lam"], v["dout"], reset, v["h0"],
                              v["dlast"])
    for name, key in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlog_decay"),
                      ("h0", "dh0")):
        np.testing.assert_allclose(g[key], _difference(value, v[name]), rtol=1e-5, atol=1e-7)


def test_norm_gradient_against_differences():
    g = RNG(4)
    x, res, dy, dres = (g.standard_normal((3, 6)) for _ in range(4))
    w = g.standard_normal(6)

    def value():
        y, s = layer.rms_norm(x, w, res, 1e-3)
        return np.sum(dy * y) + np.sum(dres * s)

    grad = layer.rms_norm_grad(dy, x + res, w, 1e-3, dres)
    np.testing.assert_allclose(grad["ds"], _difference(value, x), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(grad["ds"], _difference(value, res), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(grad["dweight"], _difference(value, w), rtol=1e-6, atol=1e-8)


def test_norm_has_unit_mean_square():
    y, _ = layer.rms_norm(RNG(5).standard_normal((4, 50)) * 7, np.ones(50), None, 1e-12)
    np.testing.assert_allclose(np.mean(y * y, -1), 1.0, rtol=1e-9)


def test_e4m3_against_the_list_of_its_values():
    # sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities, 0x7f is NaN
    codes = np.arange(0x7f)
    exp, man = codes >> 3, codes & 7
    values = np.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * 2.0 ** (exp - 7.0))
    assert values[-1] == layer.FP8_MAX
    np.testing.assert_array_equal(layer.e4m3(values), values)
    np.testing.assert_array_equal(layer.e4m3(-values), -values)
    v = np.abs(RNG(6).standard_normal(20000)) * np.exp2(RNG(7).uniform(-12, 7, 20000))
    v = np.minimum(v, 448.0)
    nearest = np.abs(values[None] - v[:, None]).min(1)
    np.testing.assert_allclose(np.abs(layer.e4m3(v) - v), nearest, rtol=1e-12, atol=1e-18)
    # ties go to the even mantissa
    np.testing.assert_array_equal(layer.e4m3([(values[8] + values[9]) / 2,
                                              (values[9] + values[10]) / 2]),
                                  [values[8], values[10]])


def test_linear_against_loops():
    g = RNG(8)
    m, n, k = 3, 130, 144
    xq, xs = layer.quantize(g.standard_normal((m, k)))
    wq, ws = layer.quantize(g.standard_normal((n, k)), 128)
    bias = g.standard_normal(n)
    out, _ = layer.linear(xq, xs, wq, ws, bias)
    for a, b in ((0, 0), (1, 127), (2, 128), (0, 129)):
        want = bias[b] + sum(xq[a, c] * xs[c // 128, a] * wq[b, c] * ws[b // 128, c // 128]
                             for c in range(k))
        assert abs(out[a, b] - want) < 1e-12 * max(1.0, abs(want))
