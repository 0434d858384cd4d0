"""The router and the order by expert on the GPU against their float64
reference.

Tolerances.  Scores are exp2 of a float32 argument a = (l - top) log2 e over a
sum: a is off by at most 2 half steps of |a| (the difference and the product),
2^-23 |a|, which is as much of exp2(a) times ln 2; exp2, the division and the
product with it and scale add 6 half steps and two units of the instruction,
and the sum of E terms, all positive, E + 6 half steps.  So a score is within
(2 |a| + E + 20) 2^-24 of itself, with |a| <= 1.45 * the row's spread, here
below 64.  Gradients are sums of such products: the same share of the terms'
summed magnitude, with 2 E more half steps for the sums over a row.  bfloat16
outputs: 2^-8 of themselves on top.
"""

import numpy as np
import pytest
import torch

from oracle import feed

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
SHAPES = [(1, 1, 1), (1, 2, 2), (5, 7, 3), (64, 16, 2), (33, 17, 16), (100, 32, 1), (17, 60, 4),
          (130, 64, 8), (1000, 65, 6), (257, 128, 8), (31, 200, 5), (19, 256, 16), (9, 257, 4),
          (7, 512, 8), (5, 1000, 3), (3, 1024, 16), (16400, 8, 2)]


def logits_of(tokens, experts, dtype, seed=0, masked=False):
    g = torch.Generator().manual_seed(seed)
    v = 2.0 * torch.randn(tokens, experts, generator=g)
    if masked:
        v[torch.rand(tokens, experts, generator=g) < 0.3] = -float("inf")
        v[torch.rand(tokens, generator=g) < 0.2] = -float("inf")
    return v.to("cuda", dtype)


def ref(t):
    return t.double().cpu().numpy()


def rel_of(v, experts):
    finite = np.where(np.isfinite(v), v, np.nan)
    spread = max(1.0, np.nanmax(finite, initial=0) - np.nanmin(finite, initial=0))
    assert 1.45 * spread < 64
    return (2 * 64 + experts + 20) * 2.0 ** -24


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("tokens,experts,k", SHAPES)
def test_route(tokens, experts, k, masked, renormalize, score, dtype):
    from selective_state_space_38_amd import expert_route_bwd, expert_route_fwd
    logits = logits_of(tokens, experts, dtype, masked=masked)
    v = ref(logits)
    opts = dict(score=score, renormalize=renormalize, scale=1.5)
    want_index, want_weight, want_total = feed.route(v, k, score, renormalize, 1.5)
    index, weight, total = expert_route_fwd(logits, k, return_score_sum=True, **opts)
    assert index.dtype == torch.int32 and weight.dtype == total.dtype == torch.float32
    np.testing.assert_array_equal(index.cpu().numpy(), want_index)
    rel = rel_of(v, experts)
    # a renormalised weight: two scores' errors, and the chosen ones' sum
    assert (np.abs(ref(weight) - want_weight) <= 2 * rel * want_weight).all()
    assert (np.abs(ref(total) - want_total) <= (rel + tokens * 2.0 ** -24) * want_total).all()
    again = expert_route_fwd(logits, k, **opts)
    assert torch.equal(again[0], index) and torch.equal(again[1], weight)

    g = torch.Generator().manual_seed(1)
    dw, ds = torch.randn(tokens, k, generator=g).cuda(), torch.randn(experts, generator=g).cuda()
    s = feed.scores(v, score)
    for d1, d2 in ((dw, ds), (dw, None), (None, ds)):
        got = expert_route_bwd(logits, index, d1, dscore_sum=d2, **opts)
        assert got.dtype == dtype and got.shape == logits.shape
        a, b = (None if d is None else ref(d) for d in (d1, d2))
        want = feed.route_grad(v, want_index, a, b, score, renormalize, 1.5)
        # the terms' summed magnitude: every g_e is at most the largest |scale dw| (twice
        # that over the chosen sum) and |dscore_sum|
        size = s * 0
        if b is not None:
            size = size + s * (np.abs(b) + (s * np.abs(b)).sum(1, keepdims=True))
        if a is not None:
            big = 1.5 * np.abs(a).max(1, keepdims=True)
            if renormalize:
                q = np.zeros_like(s)
                for t in range(tokens):
                    es = [e for e in want_index[t] if e >= 0]
                    if es:
                        q[t, es] = s[t, es] / s[t, es].sum()
                size = size + 2 * big * q
            else:
                chosen = np.zeros_like(s)
                for j in range(k):
                    at = want_index[:, j]
                    chosen[np.arange(tokens)[at >= 0], at[at >= 0]] = 1
                size = size + big * s * (chosen + (s * chosen).sum(1, keepdims=True))
        bound = (4 * rel + 2 * experts * 2.0 ** -24) * size + HALF_STEP[dtype] * np.abs(want)
        assert (np.abs(ref(got) - want) <= bound + 1e-37).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_logits_go_by_number(dtype):
    from selective_state_space_38_amd import expert_route_fwd
    for experts in (3, 40, 130, 700):
        logits = torch.zeros(5, experts, dtype=dtype, device="cuda")
        logits[1, experts // 2] = 1.0
        logits[2, :] = -2.0
        index, weight = expert_route_fwd(logits, 3)
        want, w, _ = feed.route(ref(logits), 3)
        np.testing.assert_array_equal(index.cpu().numpy(), want)
        np.testing.assert_allclose(ref(weight), w, rtol=1e-5)


def test_values_that_are_not_finite():
    from selective_state_space_38_amd import expert_route_bwd, expert_route_fwd
    logits = torch.randn(6, 20, generator=torch.Generator().manual_seed(2)).cuda()
    clean = logits.clone()
    logits[1, 3] = float("nan")
    logits[2, 4] = float("inf")
    logits[3] = -float("inf")
    logits[4] = float("nan")
    for score in ("softmax", "sigmoid"):
        index, weight = expert_route_fwd(logits, 4, score=score)
        got, w = index.cpu(), weight.cpu()
        assert ((got >= -1) & (got < 20)).all()
        for t in range(6):  # an expert is chosen once
            chosen = got[t][got[t] >= 0]
            assert len(set(chosen.tolist())) == len(chosen)
        other = expert_route_fwd(clean, 4, score=score)
        for t in (0, 5):  # other tokens are not touched
            assert torch.equal(index[t], other[0][t]) and torch.equal(weight[t], other[1][t])
        assert (got[3] == -1).all() and (w[3] == 0).all()
        assert w[4].isnan().all()
        assert got[2, 0] == 4 and (score == "sigmoid" or w[2].isnan().all())
        if score == "softmax":
            assert w[1].isnan().all()
        g = expert_route_bwd(logits, index, torch.ones_like(weight), score=score)
        assert (g[3] == 0).all() and torch.equal(
            g[0], expert_route_bwd(clean, other[0], torch.ones_like(weight), score=score)[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", [7, 128, 200, 1000])
def test_choice_over_every_bit_pattern(experts, dtype):
    # both zeros are equal, a NaN of either sign is the lowest finite value, -inf is not chosen
    from selective_state_space_38_amd import expert_route_fwd
    tokens, k = 700, 6
    bits = np.random.default_rng(experts).integers(0, 1 << 16, (tokens, experts)).astype(np.uint32)
    few = np.array([0x0000, 0x8000, 0x7f80, 0xff80, 0x7fc0, 0xffc0, 0x7f81, 0xff7f, 0x7f7f, 0x0001,
                    0x8001], np.uint32)
    bits[::2] = few[np.random.default_rng(1).integers(0, len(few), (tokens // 2, experts))]
    values = (bits << 16).view(np.float32)
    logits = torch.from_numpy(values).cuda().to(dtype)
    low = float(torch.finfo(dtype).min)
    want = ref(logits)
    want = np.where(np.isnan(want), low, want)
    index, weight = expert_route_fwd(logits, k)
    order = np.argsort(-want, axis=1, kind="stable")[:, :k]
    none = np.take_along_axis(want, order, 1) == -np.inf
    np.testing.assert_array_equal(index.cpu().numpy(), np.where(none, -1, order))
    assert (ref(weight)[none] == 0).all()


def test_far_logits_keep_their_shares():
    # sigmoids that all but vanish: the chosen ones' shares are still those of exp(l)
    from selective_state_space_38_amd import expert_route_bwd, expert_route_fwd
    logits = torch.tensor([[-200.0, -201.0, -300.0, -202.0]], device="cuda")
    index, weight = expert_route_fwd(logits, 3, score="sigmoid", renormalize=True)
    e = np.exp(-np.arange(3.0))
    assert index.tolist() == [[0, 1, 3]]
    np.testing.assert_allclose(ref(weight)[0], e / e.sum(), rtol=1e-4)
    dw = torch.tensor([[1.0, -1.0, 2.0]], device="cuda")
    q = e / e.sum()
    g = expert_route_bwd(logits, index, dw, score="sigmoid", renormalize=True)
    want = q * (np.array([1.0, -1.0, 2.0]) - (q * [1.0, -1.0, 2.0]).sum())
    np.testing.assert_allclose(ref(g)[0, [0, 1, 3]], want, rtol=1e-4)


def test_index_outside_the_experts_takes_no_part():
    from selective_state_space_38_amd import expert_route_bwd
    logits = logits_of(4, 10, torch.float32)
    index = torch.tensor([[0, 3], [-1, 2], [10, 5], [7, 7]], dtype=torch.int32, device="cuda")
    dw = torch.randn(4, 2, generator=torch.Generator().manual_seed(3)).cuda()
    for renormalize in (False, True):
        got = expert_route_bwd(logits, index, dw, renormalize=renormalize)
        rows = [0, 1, 2] if renormalize else [0, 1, 2, 3]  # (twice the same: no weight the forward gives)
        want = feed.route_grad(ref(logits), index.cpu().numpy(), ref(dw), None, "softmax", renormalize)
        np.testing.assert_allclose(ref(got)[rows], want[rows], atol=1e-6)


SORTS = [(1, 1, 1), (3, 2, 4), (1, 16, 1024), (100, 1, 3), (512, 2, 64), (513, 2, 7), (1024, 4, 60),
         (1025, 4, 1024), (5000, 8, 128), (40000, 3, 1), (37001, 8, 5), (32768, 16, 1023)]


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("tokens,k,experts", SORTS)
def test_sort(tokens, k, experts, dropped):
    from selective_state_space_38_amd import expert_sort
    g = np.random.default_rng(tokens + k)
    # uneven, and the same expert twice for a token
    index = np.minimum(g.integers(0, experts, (tokens, k)), g.integers(0, experts, (tokens, k)))
    index = index.astype(np.int32)
    if dropped:
        index[g.random((tokens, k)) < 0.3] = -1
        index[g.random((tokens, k)) < 0.05] = experts
        index[g.random((tokens, k)) < 0.05] = 2 ** 31 - 1
    offsets, token, slot = (t.cpu().numpy() for t in expert_sort(torch.from_numpy(index).cuda(), experts))
    flat = index.reshape(-1)
    ok = (flat >= 0) & (flat < experts)
    order = np.argsort(np.where(ok, flat, experts), kind="stable")
    rows = ok.sum()
    np.testing.assert_array_equal(offsets, np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=experts))]))
    np.testing.assert_array_equal(token[:rows], order[:rows] // k)
    assert (token[rows:] == -1).all()
    want = np.full(tokens * k, -1, np.int32)
    want[order[:rows]] = np.arange(rows)
    np.testing.assert_array_equal(slot.reshape(-1), want)
    if tokens * k <= 2048:
        for a, b in zip((offsets, token, slot), feed.sort(np.where(ok.reshape(index.shape), index, -1), experts)):
            np.testing.assert_array_equal(a, b)


def test_refusals():
    from selective_state_space_38_amd import expert_route_bwd, expert_route_fwd, expert_sort
    logits = logits_of(4, 8, torch.float32)
    index, weight = expert_route_fwd(logits, 2)
    for bad in (logits.cpu(), logits.half(), logits[0], logits.t()):
        with pytest.raises(ValueError):
            expert_route_fwd(bad, 2)
    with pytest.raises(ValueError):
        expert_route_fwd(logits, 2, score="tanh")
    for k in (0, 9, 17):
        with pytest.raises(RuntimeError):
            expert_route_fwd(logits, k)
    with pytest.raises(RuntimeError):
        expert_route_fwd(torch.zeros(2, 1025, device="cuda"), 2)
    with pytest.raises(ValueError):
        expert_route_bwd(logits, None, weight)
    with pytest.raises(ValueError):
        expert_route_bwd(logits, index, None)
    with pytest.raises(ValueError):
        expert_route_bwd(logits, index.long(), weight)
    with pytest.raises(ValueError):
        expert_route_bwd(logits, index, weight[:2])
    for bad in (index.long(), index.cpu(), index[0], index.t()):
        with pytest.raises(ValueError):
            expert_sort(bad, 8)
    for experts in (0, 1025):
        with pytest.raises(RuntimeError):
            expert_sort(index, experts)
