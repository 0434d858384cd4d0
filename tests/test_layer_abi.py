"""Host-only checks of the residual layer's entry points: bad arguments are
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


def _gated(**kw):
    v = dict(batch=2, seqlen=64, dim=100, ld_x=100, ld_r=100, ld_i=100, dtype=0)
    v.update(kw)
    return _lib.GatedDims(*(v[f] for f, _ in _lib.GatedDims._fields_))


def _fwd(d, **kw):
    v = dict(x=P[0], r=P[1], i=P[2], lam=P[3], reset=None, h0=None, out=P[4], last=None, ckpt=None,
             work=P[5])
    v.update(kw)
    return _lib.load().gated_scan_fwd(*v.values(), None if d is None else ctypes.byref(d), None)


def _bwd(d, **kw):
    v = dict(x=P[0], r=P[1], i=P[2], lam=P[3], reset=None, h0=None, dout=P[4], dlast=None,
             ckpt=P[5], dx=P[6], dr=P[7], di=P[8], dlam=P[9], dh0=None, work=P[10])
    v.update(kw)
    return _lib.load().gated_scan_bwd(*v.values(), ctypes.byref(d), None)


def _step(d, **kw):
    v = dict(state=P[0], x=P[1], r=P[2], i=P[3], lam=P[4], out=P[5])
    v.update(kw)
    return _lib.load().gated_state_update(*v.values(), ctypes.byref(d), None)


@pytest.mark.parametrize("field,value", [
    ("batch", 0), ("seqlen", 0), ("dim", 0), ("batch", -1), ("dim", (1 << 24) + 1),
    ("seqlen", 1 << 31), ("batch", 1 << 25), ("ld_x", 99), ("ld_r", 0), ("ld_i", -100),
    ("ld_x", 1 << 27)])
def test_gated_dims(field, value):
    d = _gated(**{field: value})
    assert _fwd(d) == _bwd(d) == SSM_EINVAL
    lib = _lib.load()
    assert lib.gated_scan_work_bytes(ctypes.byref(d)) == SSM_EINVAL
    assert lib.gated_ckpt_bytes(ctypes.byref(d)) == SSM_EINVAL
    assert lib.gated_scan_bwd_work_bytes(ctypes.byref(d), 0) == SSM_EINVAL


def test_gated_arguments():
    d = _gated()
    assert _fwd(None) == SSM_EINVAL
    assert _fwd(_gated(dtype=2)) == SSM_EDTYPE
    for key in ("x", "r", "i", "lam", "out"):
        assert _fwd(d, **{key: None}) == SSM_EINVAL, key
    for key in ("x", "r", "i", "lam", "dout", "dx", "dr", "di", "dlam", "work"):
        assert _bwd(d, **{key: None}) == SSM_EINVAL, key
    for key in ("x", "r", "i", "lam", "out"):
        assert _fwd(d, **{key: HALF}) == SSM_EALIGN, key
    # two bytes are enough for a bfloat16 slice, one is not
    assert _fwd(_gated(dtype=1), x=ODD) == SSM_EALIGN
    assert _fwd(d, ckpt=EIGHT) == SSM_EALIGN
    assert _bwd(d, work=EIGHT) == SSM_EALIGN
    assert _fwd(d, out=P[0]) == SSM_EINVAL
    assert _fwd(d, last=P[4]) == SSM_EINVAL
    assert _fwd(d, ckpt=P[4]) == SSM_EINVAL
    assert _bwd(d, dx=P[4]) == SSM_EINVAL
    assert _bwd(d, dr=P[6]) == SSM_EINVAL
    assert _step(d) == SSM_EINVAL  # more than one step
    one = _gated(seqlen=1)
    for key in ("state", "x", "r", "i", "lam", "out"):
        assert _step(one, **{key: None}) == SSM_EINVAL, key
    assert _step(one, out=P[0]) == SSM_EINVAL
    assert _step(one, state=P[1]) == SSM_EINVAL


def test_gated_scratch_sizes():
    lib = _lib.load()
    d = _gated(seqlen=33)
    assert lib.gated_ckpt_bytes(ctypes.byref(d)) == 2 * 3 * 100 * 4
    assert lib.gated_scan_work_bytes(ctypes.byref(_gated(seqlen=1))) == 0
    with_ckpt = lib.gated_scan_bwd_work_bytes(ctypes.byref(d), 1)
    assert with_ckpt > 0
    assert lib.gated_scan_bwd_work_bytes(ctypes.byref(d), 0) >= with_ckpt + 2 * 3 * 100 * 4


def _norm(rows=4, dim=64, dtype=0, residual=0):
    return _lib.NormDims(rows, dim, dtype, residual)


def test_norm_arguments():
    lib = _lib.load()

    def fwd(d, x=P[0], res=None, w=P[1], eps=1e-5, y=P[2], out=None):
        return lib.rms_norm_fwd(x, res, w, eps, y, out, ctypes.byref(d), None)

    def fp8(d, x=P[0], res=None, w=P[1], eps=1e-5, q=P[2], scale=P[3], out=None):
        return lib.rms_norm_fp8(x, res, w, eps, q, scale, out, ctypes.byref(d), None)

    def bwd(d, dy=P[0], s=P[1], w=P[2], eps=1e-5, dres=None, ds=P[3], dw=P[4], work=P[5]):
        return lib.rms_norm_bwd(dy, s, w, eps, dres, ds, dw, work, ctypes.byref(d), None)

    for f in (fwd, fp8, bwd):
        for bad in (_norm(rows=0), _norm(dim=0), _norm(dim=16385), _norm(rows=1 << 31)):
            assert f(bad) == SSM_EINVAL
        assert f(_norm(dtype=3)) == f(_norm(residual=-1)) == SSM_EDTYPE
        for eps in (0.0, -1.0, float("nan")):
            assert f(_norm(), eps=eps) == SSM_EINVAL
        assert f(_norm(), w=None) == SSM_EINVAL
    for f in (fwd, fp8):
        assert f(_norm(), x=None) == SSM_EINVAL
        assert f(_norm(), res=P[6]) == SSM_EINVAL       # residual without residual_out
        assert f(_norm(), out=P[6]) == SSM_EINVAL
        assert f(_norm(), x=ODD) == SSM_EALIGN
    assert fwd(_norm(), y=None) == fwd(_norm(), y=P[0]) == SSM_EINVAL
    assert fwd(_norm(), res=P[6], out=P[2]) == SSM_EINVAL
    assert fp8(_norm(), q=None) == fp8(_norm(), scale=None) == SSM_EINVAL
    assert fp8(_norm(dim=72)) == SSM_EINVAL             # not whole runs of 16 values
    assert fp8(_norm(), x=EIGHT) == fp8(_norm(), q=EIGHT) == fp8(_norm(), w=EIGHT) == SSM_EALIGN
    assert lib.fp8_quantize(P[0], P[1], P[2], ctypes.byref(_norm(dim=24)), None) == SSM_EINVAL
    assert lib.fp8_quantize(P[0], P[1], P[2], None, None) == SSM_EINVAL
    for key in ("dy", "s", "ds", "dw", "work"):
        assert bwd(_norm(), **{key: None}) == SSM_EINVAL, key
    assert bwd(_norm(), ds=P[1]) == bwd(_norm(), dw=P[3]) == SSM_EINVAL
    assert bwd(_norm(), work=EIGHT) == SSM_EALIGN
    assert lib.rms_norm_bwd_work_bytes(ctypes.byref(_norm())) > 0


def test_linear_arguments():
    lib = _lib.load()

    def linear(m=4, n=64, k=256, dtype=0, x=P[0], xs=P[1], w=P[2], ws=P[3], bias=None, out=P[4],
               work=P[5]):
        d = _lib.LinearDims(m, n, k, dtype)
        return lib.fp8_linear(x, xs, w, ws, bias, out, work, ctypes.byref(d), None)

    for kw in (dict(m=0), dict(n=0), dict(k=0), dict(k=24), dict(m=(1 << 30) + 1),
               dict(n=(1 << 24) + 1), dict(k=(1 << 20) + 16), dict(m=1 << 30, n=1 << 24)):
        assert linear(**kw) == SSM_EINVAL, kw
    assert linear(dtype=2) == SSM_EDTYPE
    for key in ("x", "xs", "w", "ws", "out"):
        assert linear(**{key: None}) == SSM_EINVAL, key
    assert linear(x=EIGHT) == linear(w=EIGHT) == linear(xs=HALF) == linear(out=HALF) == SSM_EALIGN
    assert linear(out=P[0]) == SSM_EINVAL
    d = _lib.LinearDims(4, 64, 24, 0)
    assert lib.fp8_linear_work_bytes(ctypes.byref(d)) == SSM_EINVAL
    for args in ((None, 0, 4, 4, P[1], P[2]), (P[0], 0, 0, 4, P[1], P[2]),
                 (P[0], 0, 4, 0, P[1], P[2]), (P[0], 0, 4, 4, P[0], P[2]),
                 (P[0], 0, 4, 4, P[1], P[1])):
        assert lib.fp8_quantize_weight(*args, None) == SSM_EINVAL
    assert lib.fp8_quantize_weight(P[0], 5, 4, 4, P[1], P[2], None) == SSM_EDTYPE
    assert lib.fp8_quantize_weight(HALF, 0, 4, 4, P[1], P[2], None) == SSM_EALIGN
