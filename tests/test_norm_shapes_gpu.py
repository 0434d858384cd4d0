"""The norm's and the quantization's rows in each of their launch shapes.
Inputs and tolerances are those of test_norm_linear_gpu."""

import pytest
import torch

import test_norm_linear_gpu as base

pytestmark = pytest.mark.gpu

DTYPES = base.DTYPES
# rows that share a wave and leave its last places empty, one wave's longest,
# the first of four waves' (each direction's)
SHAPES = [(70, 64), (17, 80), (131, 208), (259, 240), (3, 512), (5, 528), (2, 2576), (3, 3584),
          (2, 3600), (1, 4096)]
ODD = [(33, 8), (67, 63), (9, 65), (1, 100), (21, 251), (2, 509), (3, 2561), (2, 3585), (1, 4095)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [None, torch.float32])
@pytest.mark.parametrize("rows,dim", SHAPES + ODD)
def test_norm(rows, dim, residual, dtype):
    base.test_norm(rows, dim, residual, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_fp8(rows, dim, dtype):
    base.test_norm_fp8(rows, dim, torch.float32, dtype)
    base.test_quantize(rows, dim, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("stream", DTYPES)
@pytest.mark.parametrize("rows,dim", SHAPES + ODD + [(1500, 24), (20000, 70)])
def test_norm_bwd(rows, dim, stream, dtype):
    base.test_norm_backward(rows, dim, stream, dtype)


@pytest.mark.parametrize("dim", [64, 144, 1024, 4096])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_rows_keep_their_values(dim, bad):
    # rows share a wave and a workgroup, not their sums
    from selective_state_space_38_amd import fp8_quantize, rms_norm_bwd, rms_norm_fp8, rms_norm_fwd
    x = base.rand(23, dim)
    w, dy = 1 + base.rand(dim, seed=1, scale=0.2), base.rand(23, dim, seed=2)
    spoilt = x.clone()
    spoilt[6, 5] = bad
    rest = [k for k in range(23) if k != 6]

    def outputs(t):
        q, scale = rms_norm_fp8(t, w)
        q0, scale0 = fp8_quantize(t)
        return [rms_norm_fwd(t, w), rms_norm_bwd(dy, t, w)["ds"], q.float(), scale.t(), q0.float(),
                scale0.t()]

    for got, want in zip(outputs(spoilt), outputs(x)):
        assert torch.equal(got[rest], want[rest])
