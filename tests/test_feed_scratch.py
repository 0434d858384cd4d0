"""Scratch of the linear product's gradient, by what is asked for (host only)."""

import ctypes

import pytest

from selective_state_space_38_amd import _lib

DX, DW, DBIAS = _lib.SSM_WANT_DX, _lib.SSM_WANT_DW, _lib.SSM_WANT_DBIAS


def work(wants, rows=16384, n=5120, k=2560, experts=0, activation=0, dtype=1, out_dtype=1):
    d = _lib.ProductDims(rows, n, k, rows, k, experts, activation, dtype, out_dtype)
    return _lib.load().linear_bwd_work_bytes(ctypes.byref(d), wants)


@pytest.mark.parametrize("activation,width", [(0, 1), (1, 1), (2, 1), (3, 2), (4, 2)])
def test_bias_alone_takes_its_partial_sums(activation, width):
    # a float32 sum a column of every 128 rows (32 below 2^25 outputs); nothing for the products
    for types in (dict(), dict(out_dtype=0), dict(dtype=0, out_dtype=0)):
        assert work(DBIAS, activation=activation, **types) == 128 * 5120 * width * 4
        assert work(DBIAS, rows=2047, n=771, activation=activation, **types) == \
            -(-64 * 771 * width * 4 // 16) * 16
        assert work(DBIAS, experts=16, activation=activation, **types) == (128 + 16) * 5120 * width * 4


@pytest.mark.parametrize("wants", [DX, DW, DX | DW, DX | DW | DBIAS])
def test_products_take_the_gradient_before_the_activation(wants):
    base = work(wants)
    for activation, width, size, types in ((1, 1, 2, dict()), (3, 2, 2, dict()), (0, 1, 2, dict(out_dtype=0)),
                                           (2, 1, 4, dict(dtype=0))):
        assert work(wants, activation=activation, **types) >= 16384 * 5120 * width * size
    assert base < 16384 * 5120 * 2      # dout serves as it is
