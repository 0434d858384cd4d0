"""Host-only checks of the feed-forward layer's entry points: bad arguments are
rejected before the GPU is touched, and scratch queries answer on the host."""

import ctypes

import pytest

from selective_state_space_38_amd import _lib

SSM_OK, SSM_EINVAL, SSM_EDTYPE, SSM_EALIGN = 0, -1, -2, -3

# fake, never dereferenced device addresses (validation fails first)
P = [ctypes.c_void_p(0x100000 + 0x1000 * i) for i in range(20)]
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)
EIGHT = ctypes.c_void_p(0x100008)
NAN = float("nan")


def _dims(cls, base, kw):
    v = dict(base, **kw)
    return cls(*(v[f] for f, _ in cls._fields_))


def _route(**kw):
    return _dims(_lib.RouteDims, dict(tokens=5, experts=8, topk=2, score=0, renormalize=0, dtype=0), kw)


def _order(**kw):
    return _dims(_lib.OrderDims, dict(tokens=5, rows=10, dim=7, topk=2, dtype=0, residual_dtype=0), kw)


def _product(**kw):
    return _dims(_lib.ProductDims, dict(rows=10, n=16, k=24, x_rows=10, ld_x=24, experts=0,
                                        activation=0, dtype=1, out_dtype=1), kw)


def _call(name, base, d, tail, kw):
    v = dict(base, **kw)
    return getattr(_lib.load(), name)(*v.values(), *((ctypes.byref(d),) if d is not None else ()),
                                      *tail, None)


def _route_fwd(d, **kw):
    return _call("expert_route_fwd", dict(logits=P[0], scale=1.0, index=P[1], weight=P[2],
                                          total=P[3], work=P[4]), d, (), kw)


def _route_bwd(d, **kw):
    return _call("expert_route_bwd", dict(logits=P[0], scale=1.0, index=P[1], dweight=P[2],
                                          dtotal=P[3], dlogits=P[4]), d, (), kw)


@pytest.mark.parametrize("kw", [
    dict(tokens=0), dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(topk=0),
    dict(topk=9), dict(topk=17, experts=64), dict(score=2), dict(score=-1),
    dict(tokens=1 << 30, topk=2), dict(tokens=(1 << 25) + 1, topk=1)])
def test_route_dims(kw):
    d = _route(**kw)
    assert _route_fwd(d) == _route_bwd(d) == SSM_EINVAL
    assert _lib.load().expert_route_work_bytes(ctypes.byref(d)) == SSM_EINVAL


def test_route_arguments():
    d = _route()
    lib = _lib.load()
    assert lib.expert_route_work_bytes(ctypes.byref(d)) > 0
    assert lib.expert_route_work_bytes(None) == SSM_EINVAL
    assert _route_fwd(_route(dtype=2)) == _route_bwd(_route(dtype=-1)) == SSM_EDTYPE
    for key in ("logits", "index", "weight", "work"):
        assert _route_fwd(d, **{key: None}) == SSM_EINVAL, key
    for key in ("logits", "index", "weight", "total"):
        assert _route_fwd(d, **{key: HALF}) == SSM_EALIGN, key
    assert _route_fwd(d, work=EIGHT) == _route_fwd(_route(dtype=1), logits=ODD) == SSM_EALIGN
    assert _route_fwd(d, weight=P[1]) == _route_fwd(d, index=P[0]) == SSM_EINVAL
    for key in ("logits", "index", "dlogits"):
        assert _route_bwd(d, **{key: None}) == SSM_EINVAL, key
    assert _route_bwd(d, dweight=None, dtotal=None) == SSM_EINVAL
    assert _route_bwd(d, dlogits=P[0]) == SSM_EINVAL
    assert _route_bwd(d, dlogits=HALF) == SSM_EALIGN


def test_sort_arguments():
    lib = _lib.load()

    def sort(index=P[0], tokens=5, topk=2, experts=8, offsets=P[1], token=P[2], slot=P[3],
             work=P[4]):
        return lib.expert_sort(index, tokens, topk, experts, offsets, token, slot, work, None)

    for kw in (dict(tokens=0), dict(topk=0), dict(topk=17), dict(experts=0), dict(experts=1025),
               dict(tokens=1 << 30)):
        assert sort(**kw) == SSM_EINVAL, kw
    for key in ("index", "offsets", "token", "slot"):
        assert sort(**{key: None}) == SSM_EINVAL, key
        assert sort(**{key: HALF}) == SSM_EALIGN, key
    assert sort(slot=P[0]) == sort(token=P[1]) == SSM_EINVAL
    assert sort(tokens=100000, work=None) == SSM_EINVAL
    assert lib.expert_sort_work_bytes(5, 2, 8) == 0          # one workgroup
    assert lib.expert_sort_work_bytes(100000, 2, 8) > 0
    assert lib.expert_sort_work_bytes(0, 2, 8) == SSM_EINVAL


def test_order_arguments():
    def gather(d, **kw):
        return _call("expert_gather", dict(x=P[0], token=P[1], xs=P[2]), d, (), kw)

    def fwd(d, **kw):
        return _call("expert_combine_fwd", dict(y=P[0], slot=P[1], weight=P[2], residual=P[3],
                                                out=P[4]), d, (), kw)

    def bwd(d, **kw):
        return _call("expert_combine_bwd", dict(dout=P[0], y=P[1], slot=P[2], weight=P[3], dy=P[4],
                                                dweight=P[5]), d, (), kw)

    for f in (gather, fwd, bwd):
        for kw in (dict(tokens=0), dict(rows=0), dict(dim=0), dict(topk=0), dict(topk=17),
                   dict(rows=(1 << 30) + 1), dict(rows=(1 << 25) + 1), dict(tokens=(1 << 25) + 1),
                   dict(dim=(1 << 24) + 1)):
            assert f(_order(**kw)) == SSM_EINVAL, kw
        assert f(_order(dtype=4)) == f(_order(residual_dtype=4)) == SSM_EDTYPE
    d = _order()
    for key in ("x", "token", "xs"):
        assert gather(d, **{key: None}) == SSM_EINVAL
        assert gather(d, **{key: HALF}) == SSM_EALIGN
    assert gather(d, xs=P[0]) == SSM_EINVAL
    for key in ("y", "slot", "out"):
        assert fwd(d, **{key: None}) == SSM_EINVAL
    for key in ("y", "slot", "weight", "residual", "out"):
        assert fwd(d, **{key: HALF}) == SSM_EALIGN
    assert fwd(d, out=P[0]) == fwd(d, out=P[2]) == SSM_EINVAL
    for key in ("dout", "slot", "dy", "y", "weight"):
        assert bwd(d, **{key: None}) == SSM_EINVAL, key
    assert bwd(d, dy=P[1]) == bwd(d, dweight=P[3]) == bwd(d, dy=P[5]) == SSM_EINVAL
    assert bwd(d, dweight=HALF) == bwd(d, dy=HALF) == SSM_EALIGN


def _fwd(d, **kw):
    return _call("linear_fwd", dict(x=P[0], token=None, w=P[1], offsets=None, bias=P[2],
                                    residual=P[3], out=P[4], pre=P[5], work=P[6]), d, (), kw)


def _bwd(d, **kw):
    return _call("linear_bwd", dict(dout=P[0], x=P[1], token=None, w=P[2], offsets=None, pre=None,
                                    dx=P[4], dw=P[5], dbias=P[6], work=P[7]), d, (), kw)


@pytest.mark.parametrize("kw", [
    dict(rows=0), dict(n=0), dict(k=0), dict(k=20), dict(x_rows=0), dict(ld_x=16),
    dict(ld_x=28), dict(experts=-1), dict(experts=1025), dict(activation=5), dict(activation=-1),
    dict(rows=(1 << 30) + 8, x_rows=(1 << 30) + 8), dict(n=(1 << 20) + 8),
    dict(k=(1 << 20) + 8, ld_x=(1 << 20) + 8), dict(rows=1 << 30, x_rows=1 << 30, n=1 << 20),
    dict(rows=1 << 30, x_rows=1 << 30), dict(experts=1024, n=1 << 18, k=1 << 18, ld_x=1 << 18),
    dict(x_rows=9)])
def test_product_dims(kw):
    d = _product(**kw)
    assert _fwd(d) == _bwd(d) == SSM_EINVAL
    if "x_rows" not in kw or kw["x_rows"] != 9:  # (that one the calls alone can tell)
        assert _lib.load().linear_fwd_work_bytes(ctypes.byref(d)) == SSM_EINVAL
        assert _lib.load().linear_bwd_work_bytes(ctypes.byref(d), 7) == SSM_EINVAL


def test_product_arguments():
    d = _product()
    assert _fwd(_product(dtype=2)) == _bwd(_product(out_dtype=2)) == SSM_EDTYPE
    for key in ("x", "w", "out"):
        assert _fwd(d, **{key: None}) == SSM_EINVAL, key
    for key in ("x", "w", "bias", "residual", "out", "pre", "work"):
        assert _fwd(d, **{key: EIGHT}) == SSM_EALIGN, key
    assert _fwd(d, offsets=P[8]) == _fwd(_product(experts=3)) == SSM_EINVAL
    assert _fwd(d, token=P[8]) == SSM_EINVAL                  # without experts
    assert _fwd(_product(experts=3), offsets=HALF) == SSM_EALIGN
    assert _fwd(_product(experts=3, x_rows=4), offsets=P[8], token=HALF) == SSM_EALIGN
    assert _fwd(d, out=P[0]) == _fwd(d, pre=P[4]) == _fwd(d, pre=P[1]) == SSM_EINVAL
    for key in ("dout", "x", "w"):
        assert _bwd(d, **{key: None}) == SSM_EINVAL, key
    for key in ("dout", "x", "w", "dx", "dw", "work"):
        assert _bwd(d, **{key: EIGHT}) == SSM_EALIGN, key
    assert _bwd(d, dbias=HALF) == SSM_EALIGN
    assert _bwd(d, dx=None, dw=None, dbias=None) == SSM_EINVAL
    assert _bwd(d, pre=P[8]) == _bwd(_product(activation=1)) == SSM_EINVAL
    assert _bwd(d, dx=P[0]) == _bwd(d, dw=P[4]) == SSM_EINVAL
    assert _bwd(d, work=None) == SSM_EINVAL                   # dbias sums need it
    lib = _lib.load()
    assert lib.linear_bwd_work_bytes(ctypes.byref(d), 0) == SSM_EINVAL
    assert lib.linear_bwd_work_bytes(ctypes.byref(d), 8) == SSM_EINVAL
    with_act = lib.linear_bwd_work_bytes(ctypes.byref(_product(activation=3)), 7)
    assert with_act >= lib.linear_bwd_work_bytes(ctypes.byref(d), 7) + 10 * 32 * 2
