"""The 8-bit product's tiles of 128 outputs by 256 tokens, forced at sizes that
cut them and by the rule's own choice.  Inputs and tolerances are those of
test_norm_linear_gpu."""

import pytest
import torch

import test_norm_linear_gpu as base

pytestmark = pytest.mark.gpu


def product(m, n, k):
    from selective_state_space_38_amd import fp8_linear
    args = base.linear_inputs(m, n, k, seed=m + n + k)
    bias = base.rand(n, seed=3)
    return args, bias, fp8_linear(*args, bias=bias, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("parts", [1, 3])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (5, 130, 144), (65, 264, 400), (130, 72, 128),
                                   (257, 129, 272), (512, 385, 384), (300, 256, 1040),
                                   (256, 128, 640), (1000, 1031, 256)])
def test_tall_tiles(m, n, k, parts, monkeypatch):
    monkeypatch.setenv("SSM_FORCE_LINEAR_SHAPE", "4")
    monkeypatch.setenv("SSM_FORCE_LINEAR_PARTS", str(parts))
    args, bias, out = product(m, n, k)
    base.check_linear(args, bias, torch.bfloat16, out)


@pytest.mark.parametrize("m,n,k", [(4224, 4352, 272), (5000, 5001, 144)])
def test_chosen_tall_tiles(m, n, k):
    # more tiles of 256 x 256 than CUs, a last round that is not full
    args, bias, out = product(m, n, k)
    base.check_linear(args, bias, torch.bfloat16, out)


def test_tall_tiles_repeat(monkeypatch):
    # the same bits from every call, whatever workgroups share a CU
    monkeypatch.setenv("SSM_FORCE_LINEAR_SHAPE", "4")
    out = product(2048, 1280, 1040)[2]
    for _ in range(5):
        assert torch.equal(product(2048, 1280, 1040)[2], out)


@pytest.mark.parametrize("dtype", base.DTYPES)
@pytest.mark.parametrize("n,k", [(300, 1004), (129, 36), (16, 7), (1000, 520)])
def test_weights(n, k, dtype):
    base.test_quantize_weight(n, k, dtype)


def test_weights_of_extreme_tiles():
    # a tile of zeros, one far above the others and one below the smallest scale
    import numpy as np

    from oracle import layer
    from selective_state_space_38_amd import fp8_quantize_weight
    w = base.rand(256, 256)
    w[:128, :128] = 0.0
    w[:128, 128:] *= 2.0 ** 100
    w[128:, :128] *= 2.0 ** -120
    q, scale = fp8_quantize_weight(w)
    want_q, want_scale = layer.quantize(base.ref(w), 128)
    np.testing.assert_allclose(base.ref(scale), want_scale, rtol=1e-6)
    assert not q[:128, :128].float().any()
    assert np.mean(base.ref(q.float()) != want_q) <= 1e-3
