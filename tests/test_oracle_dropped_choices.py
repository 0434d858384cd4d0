"""The router's gradient where choices are dropped behind it: a kept weight is still a
share of all the choices, so the gradient needs the forward's index, not the one without
the dropped choices.  The reference against central differences."""

import numpy as np
import pytest

from oracle import feed


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_takes_the_index_with_them(renormalize, score):
    g = np.random.default_rng(0)
    v, k = g.standard_normal((7, 6)), 3
    index, _, _ = feed.route(v, k, score, renormalize)
    kept = g.random(index.shape) < 0.6
    dw = np.where(kept, g.standard_normal(index.shape), 0.0)  # 0 for a choice without a row

    def value(v):  # the choice held
        s = feed.scores(v, score)
        w = np.take_along_axis(s, index, 1)
        return (dw * (w / w.sum(1, keepdims=True) if renormalize else w)).sum()

    want, step = np.zeros_like(v), 1e-5
    for at in np.ndindex(v.shape):
        d = np.zeros_like(v)
        d[at] = step
        want[at] = (value(v + d) - value(v - d)) / (2 * step)
    # differences: third derivatives of a few times step^2, and 2^-52 / step of rounding
    np.testing.assert_allclose(feed.route_grad(v, index, dw, None, score, renormalize), want, atol=1e-8)
    masked = feed.route_grad(v, np.where(kept, index, -1), dw, None, score, renormalize)
    assert np.allclose(masked, want, atol=1e-8) != renormalize  # shares of the kept ones are other weights


def test_one_of_two_dropped():
    # two equal scores, one kept with dweight 1/2: w = s0 / (s0 + s1), dw/dl0 = 1/4
    v = np.array([[0.0, 0.0, -5.0, -5.0]])
    got = feed.route_grad(v, np.array([[0, 1]]), np.array([[0.5, 0.0]]), renormalize=True)
    np.testing.assert_allclose(got, [[0.125, -0.125, 0, 0]], atol=1e-15)
