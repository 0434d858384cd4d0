"""The router's float64 reference on logits that are not finite, against torch."""

import numpy as np
import pytest
import torch

from oracle import feed

NAN, INF = float("nan"), float("inf")
ROWS = np.array([[0.5, 2.0, -1.0, NAN], [0.5, NAN, 1.0, 0.0], [INF, 0.0, 1.0, 2.0], [0.3, NAN, -INF, -INF]])


@pytest.mark.parametrize("renormalize", [False, True])
def test_a_softmax_with_a_value_that_is_not_finite(renormalize):
    np.testing.assert_array_equal(feed.scores(ROWS), torch.softmax(torch.from_numpy(ROWS), 1).numpy())
    index, weight, total = feed.route(ROWS, 3, renormalize=renormalize)
    assert index.tolist() == [[1, 0, 2], [2, 0, 3], [0, 3, 2], [0, 1, -1]]
    np.testing.assert_array_equal(np.isnan(weight), index >= 0)
    assert weight[3, 2] == 0 and np.isnan(total).all()
    assert np.isnan(feed.route_grad(ROWS, index, np.ones((4, 3)), renormalize=renormalize)).all()


def test_a_sigmoid_keeps_them_apart():
    index, weight, total = feed.route(ROWS, 3, "sigmoid", renormalize=True)
    s = torch.sigmoid(torch.from_numpy(ROWS)).numpy()
    for t in (0, 1, 2):   # the NaN is not chosen
        np.testing.assert_allclose(weight[t], s[t, index[t]] / s[t, index[t]].sum(), rtol=1e-14)
    assert np.isnan(weight[3, :2]).all() and weight[3, 2] == 0
    np.testing.assert_array_equal(np.isnan(total), [False, True, False, True])
