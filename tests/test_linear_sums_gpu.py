"""The 8-bit product's sums where one input dominates a block, as a language
model's few large activations do, and where terms cancel.

Tolerances.  Summed in float32 (float32 outputs, and up to 32 rows): (k + 8)
2^-23 of the terms' summed magnitude, as in test_norm_linear_gpu.  bfloat16
outputs: 2^-8 of themselves on top (half a unit of 8 significant bits).  bfloat16
outputs of more rows: the matrix instruction cuts seven of every 8 products to a multiple of
2^(E - 13), E the largest sum of a pair's exponents among the 8 (an exponent is
at least -6, that of a subnormal value), so each 8 lose less than 7 2^(E - 13).
"""

import numpy as np
import pytest
import torch

import test_norm_linear_gpu as base
from oracle import layer

pytestmark = pytest.mark.gpu


def on_gpu(v, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(v)).float().cuda().to(dtype)


def cut(xq, x_scale, wq, w_scale):
    """Largest sum of what the 8-bit instruction cuts off each output's terms."""
    exp = lambda v: np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))  # noqa: E731
    ex, ew = exp(xq), exp(wq)
    lost = np.zeros((xq.shape[0], wq.shape[0]))
    for g in range(0, xq.shape[1], 8):
        most = np.max([ex[:, None, j] + ew[None, :, j] for j in range(g, g + 8)], 0)
        scale = x_scale[g // 128][:, None] * np.repeat(w_scale[:, g // 128], 128)[:wq.shape[0]]
        lost += 7 * np.exp2(most - 13) * scale
    return lost


def dominated(m, n, k, ratio, mean, seed=0):
    """A row's block of 128 holds one value `ratio` times the others."""
    g = np.random.default_rng(seed)
    x, w = g.standard_normal((m, k)) + mean, g.standard_normal((n, k))
    x[:, 5::128] *= ratio
    if mean:
        w = np.abs(w)
    return layer.quantize(x) + layer.quantize(w, 128)


def check(values, dtype, float32_sums):
    from selective_state_space_38_amd import fp8_linear
    xq, xs, wq, ws = values
    want, size = layer.linear(xq, xs, wq, ws)
    out = fp8_linear(on_gpu(xq, torch.float8_e4m3fn), on_gpu(xs),
                     on_gpu(wq, torch.float8_e4m3fn), on_gpu(ws), out_dtype=dtype)
    bound = (xq.shape[1] + 8) * 2.0 ** -23 * size
    if not float32_sums:
        bound = bound + cut(*values)
    if dtype == torch.bfloat16:
        bound = bound + (np.abs(want) + bound) * 2.0 ** -8
    err = np.abs(base.ref(out) - want)
    assert (err <= bound).all(), float(np.max(err / bound))


RATIOS = [(1, 0.0), (30, 0.0), (1000, 0.0), (1000, 1.0)]


@pytest.mark.parametrize("ratio,mean", RATIOS)
@pytest.mark.parametrize("dtype", base.DTYPES)
@pytest.mark.parametrize("m", [1, 9, 16, 17, 32])
def test_few_rows(m, dtype, ratio, mean):
    check(dominated(m, 129, 528, ratio, mean, seed=m), dtype, True)


@pytest.mark.parametrize("ratio,mean", RATIOS)
@pytest.mark.parametrize("shape", [1, 2])
def test_float32_tiles(shape, ratio, mean, monkeypatch):
    monkeypatch.setenv("SSM_FORCE_LINEAR_SHAPE", str(shape))
    check(dominated(133, 260, 528, ratio, mean), torch.float32, True)


@pytest.mark.parametrize("ratio,mean", RATIOS)
@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("shape", [1, 2, 3, 4])
def test_bfloat16_tiles(shape, parts, ratio, mean, monkeypatch):
    monkeypatch.setenv("SSM_FORCE_LINEAR_SHAPE", str(shape))
    monkeypatch.setenv("SSM_FORCE_LINEAR_PARTS", str(parts))
    check(dominated(133, 260, 528, ratio, mean), torch.bfloat16, False)


@pytest.mark.parametrize("dtype", base.DTYPES)
@pytest.mark.parametrize("m", [1, 16, 32, 33, 300])
def test_small_terms_beside_one_that_cancels(m, dtype):
    # 2^16 and seven times 7.5 in 8 inputs, -2^16 in the next block: 52.5 is
    # left, each 7.5 below 2^(16 - 13)
    from selective_state_space_38_amd import fp8_linear
    x, w = np.zeros((m, 256)), np.zeros((80, 256))
    x[:, :8], w[:, :8] = 1.875, 4.0
    x[:, [3, 130]], w[:, 3], w[:, 130] = 256.0, 256.0, -256.0
    out = base.ref(fp8_linear(on_gpu(x, torch.float8_e4m3fn), on_gpu(np.ones((2, m))),
                              on_gpu(w, torch.float8_e4m3fn), on_gpu(np.ones((1, 2))),
                              out_dtype=dtype))
    if dtype == torch.float32 or m <= 32:
        assert (out == 52.5).all()
    else:
        assert (np.abs(out - 52.5) <= 7 * 2.0 ** (16 - 13)).all()
