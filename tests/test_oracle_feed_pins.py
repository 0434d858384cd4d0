"""The feed-forward layer's float64 reference against independent facts: closed
forms, library routines and central differences (CPU)."""

import numpy as np
import pytest
import torch

from oracle import feed
from test_oracle_layer_pins import _difference

RNG = np.random.default_rng


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_against_library(score):
    v = RNG(0).standard_normal((5, 9)) * 3
    t = torch.from_numpy(v)
    want = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    np.testing.assert_allclose(feed.scores(v, score), want.numpy(), rtol=1e-13)


def test_route_chooses_the_largest():
    v = RNG(1).standard_normal((20, 12))
    v[3, 4] = v[3, 9] = v[3].max() + 1   # equal: the lower number first
    v[5, :] = -np.inf
    v[6, 2:] = -np.inf
    index, weight, total = feed.route(v, 3, renormalize=True, scale=2.0)
    top = np.argsort(-v, axis=1, kind="stable")[:, :3]
    whole = [t for t in range(20) if t not in (5, 6)]
    np.testing.assert_array_equal(index[whole], top[whole])
    assert index[3, 0] == 4 and index[3, 1] == 9
    assert (index[5] == -1).all() and (weight[5] == 0).all() and index[6, 2] == -1
    np.testing.assert_allclose(np.delete(weight.sum(1), 5), 2.0, rtol=1e-13)
    np.testing.assert_allclose(total.sum(), 19.0, rtol=1e-13)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(score, renormalize):
    g = RNG(2)
    v, dw, ds = g.standard_normal((4, 6)), g.standard_normal((4, 3)), g.standard_normal(6)
    index, _, _ = feed.route(v, 3)

    def value():
        s = feed.scores(v, score)
        w = np.take_along_axis(s, index, 1)
        if renormalize:
            w = w / w.sum(1, keepdims=True)
        return 1.7 * np.sum(dw * w) + np.sum(ds * s.sum(0))

    got = feed.route_grad(v, index, dw, ds, score, renormalize, 1.7)
    np.testing.assert_allclose(got, _difference(value, v), rtol=1e-6, atol=1e-8)


def test_order_is_a_stable_sort():
    index = RNG(3).integers(-1, 5, (40, 3)).astype(np.int32)
    offsets, token, slot = feed.sort(index, 5)
    flat = index.reshape(-1)
    pairs = np.argsort(np.where(flat < 0, 5, flat), kind="stable")[:(flat >= 0).sum()]
    np.testing.assert_array_equal(token[:len(pairs)], pairs // 3)
    assert (token[len(pairs):] == -1).all() and offsets[-1] == len(pairs)
    np.testing.assert_array_equal(slot.reshape(-1)[pairs], np.arange(len(pairs)))
    np.testing.assert_array_equal(np.diff(offsets), np.bincount(flat[flat >= 0], minlength=5))


def test_into_the_order_and_back():
    g = RNG(4)
    x, w = g.standard_normal((10, 4)), g.random((10, 2))
    index = g.integers(0, 3, (10, 2)).astype(np.int32)
    _, token, slot = feed.sort(index, 3)
    xs = feed.gather(x, token)
    np.testing.assert_allclose(feed.combine(xs, slot, w, x), x * (1 + w.sum(1, keepdims=True)))


def test_combine_gradient_against_differences():
    g = RNG(5)
    y, w, dout = g.standard_normal((6, 3)), g.random((4, 2)), g.standard_normal((4, 3))
    slot = np.array([[0, 5], [1, -1], [3, 2], [9, 4]], np.int32)  # two without a row
    dy, dweight = feed.combine_grad(dout, y, slot, w)
    value = lambda: np.sum(dout * feed.combine(y, slot, w))  # noqa: E731
    np.testing.assert_allclose(dy, _difference(value, y), rtol=1e-7, atol=1e-9)
    np.testing.assert_allclose(dweight, _difference(value, w), rtol=1e-7, atol=1e-9)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu", "geglu"])
def test_activations_against_library(act):
    v = np.concatenate([np.linspace(-9, 9, 300), [0.0]])
    t = torch.from_numpy(v)
    if act in feed.GATED:
        pre = np.concatenate([v, v[::-1]])
        f = torch.nn.functional.silu if act == "swiglu" else torch.nn.functional.gelu
        want = f(t) * torch.from_numpy(v[::-1].copy())
    else:
        pre = v
        want = {None: lambda u: u, "silu": torch.nn.functional.silu,
                "gelu": torch.nn.functional.gelu}[act](t)
    np.testing.assert_allclose(feed.activate(pre, act), want.numpy(), rtol=1e-9, atol=1e-14)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("experts", [0, 3])
def test_product_gradient_against_differences(act, experts):
    g = RNG(6)
    n = 4 if act in feed.GATED else 2
    x, dout = g.standard_normal((5, 3)), g.standard_normal((5, 2))
    offsets = [0, 2, 2, 5] if experts else None  # one without rows
    lead = (3,) if experts else ()
    w, bias = g.standard_normal((*lead, n, 3)), g.standard_normal((*lead, n))
    _, pre = feed.product(x, w, bias, act, offsets=offsets)
    got = feed.product_grad(feed.activate_grad(dout, pre, act), x, w, offsets)
    value = lambda: np.sum(dout * feed.product(x, w, bias, act, offsets=offsets)[0])  # noqa: E731
    for name, a, v in zip(("dx", "dw", "dbias"), got, (x, w, bias)):
        np.testing.assert_allclose(a, _difference(value, v), rtol=1e-6, atol=1e-8, err_msg=name)
