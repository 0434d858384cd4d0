"""The router, forward and backward, on rows with a logit that is not finite, against
its float64 reference: a weight is a score over the chosen scores' sum, and a softmax
with a NaN or +inf has no score that is a number, whichever experts are chosen.

Tolerances.  A score is within rel = (2 |a| + E + 20) 2^-24 of itself, |a| <= 64 the
exponent's argument; a renormalised weight takes two scores' errors.  A gradient is a
sum of at most two products of a share, at most 1, and scale |dweight|: four scores'
errors and 2 E half steps of their summed magnitude, and its type's own half step.
"""

import numpy as np
import pytest
import torch

from oracle import feed

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def ref(t):
    return t.double().cpu().numpy()


def bad_rows(experts, dtype):
    """(logits, the same without what is not finite); row 0 and the last stay clean."""
    v = torch.randn(9, experts, generator=torch.Generator().manual_seed(experts))
    clean = v.clone()
    v[1, v[1].argmin()] = NAN                # is not among the largest
    v[2, v[2].argmax()] = NAN                # would have been
    v[3, 3] = INF
    v[4] = -INF
    v[5] = NAN
    v[6, 2:] = -INF                          # fewer finite ones than choices, and a NaN
    v[6, 1] = NAN
    v[7, 4], v[7, 5] = INF, NAN
    return v.to("cuda", dtype), clean.to("cuda", dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts", [7, 20, 128, 300, 1000])
def test_weights_and_gradient(experts, renormalize, score, dtype):
    from selective_state_space_38_amd import expert_route_bwd, expert_route_fwd
    k, opts = 4, dict(score=score, renormalize=renormalize, scale=1.5)
    logits, clean = bad_rows(experts, dtype)
    index, weight, total = expert_route_fwd(logits, k, return_score_sum=True, **opts)
    want_index, want, want_total = feed.route(ref(logits), k, score, renormalize, 1.5)
    np.testing.assert_array_equal(index.cpu().numpy(), want_index)
    rel = (2 * 64 + experts + 20) * 2.0 ** -24
    np.testing.assert_allclose(ref(weight), want, rtol=2 * rel, atol=0)  # NaN where it is NaN
    np.testing.assert_array_equal(np.isnan(ref(total)), np.isnan(want_total))
    if score == "softmax":  # whatever is chosen
        assert weight[[1, 2, 3, 5, 7]].isnan().all()
    else:
        assert torch.isfinite(weight[[1, 3]]).all()
    again = expert_route_fwd(logits, k, **opts)
    np.testing.assert_array_equal(ref(again[1]), ref(weight))

    dw = torch.randn(9, k, generator=torch.Generator().manual_seed(1)).cuda()
    got = expert_route_bwd(logits, index, dw, **opts)
    want = feed.route_grad(ref(logits), want_index, ref(dw), None, score, renormalize, 1.5)
    size = 2 * 1.5 * np.abs(ref(dw)).max(1, keepdims=True)
    bound = (4 * rel + 2 * experts * 2.0 ** -24) * size + HALF_STEP[dtype] * np.abs(want)
    np.testing.assert_array_equal(np.isnan(ref(got)), np.isnan(want))
    here = ~np.isnan(want)
    assert (np.abs(ref(got) - want) <= bound)[here].all()
    if score == "softmax":  # a row has both weights and gradients that are numbers, or neither
        assert torch.equal(got.isnan().any(1), weight.isnan().any(1))
    other = expert_route_fwd(clean, k, **opts)
    for t in (0, 8):
        assert torch.equal(index[t], other[0][t]) and torch.equal(weight[t], other[1][t])
        assert torch.equal(got[t], expert_route_bwd(clean, other[0], dw, **opts)[t])
