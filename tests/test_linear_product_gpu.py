"""The linear product with bias, activation and residual on the GPU, dense and
over experts' rows, and its gradient, against their float64 reference.

Tolerances.  A float32 sum of K products and a bias errs by at most (K + 8) 2^-23
of the terms' summed magnitude, whatever its order and whether a partial sum is
rounded or cut.  The activations' slopes are at most 1.13, so that much of it
passes into out; their own error is at most (v^2 + 16) 2^-22 of themselves (the
exponential's argument is off by 2^-23 of itself, v or v^2 / 2; a dozen more
roundings, and the instructions' last bits).  Outputs add half a step of their
type.  In the gradient dpre, with the same relative error, is rounded to the
activations' type in front of the products: the reference rounds as well, and
where the two may fall on different sides of a tie the difference counts.
"""

import numpy as np
import pytest
import torch

from oracle import feed

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
ACTS = [None, "silu", "gelu", "swiglu", "geglu"]
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# rows, n, k: one row, the few-row kernel's limits, edges of tiles and blocks, long sums
DENSE = [(1, 8, 8), (1, 264, 1000), (7, 16, 24), (16, 40, 64), (17, 64, 72), (32, 136, 200),
         (33, 64, 64), (64, 72, 136), (65, 128, 128), (130, 200, 264), (257, 264, 72), (300, 136, 520)]


def rand(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to("cuda", dtype)


def ref(t):
    return None if t is None else t.double().cpu().numpy()


def widths(n, act):
    return 2 * n if act in feed.GATED else n


def check_fwd(x, w, bias, act, res, got, pre, offsets=None):
    """x, w, ...: float64 arrays; got, pre: GPU tensors."""
    k = x.shape[1]
    out, want_pre = feed.product(x, w, bias, act, res, offsets)
    _, size = feed.product(np.abs(x), np.abs(w), None if bias is None else np.abs(bias), None, None,
                           offsets)
    err = (k + 8) * 2.0 ** -23 * size
    if pre is not None:
        half = HALF_STEP[pre.dtype]
        assert (np.abs(ref(pre) - want_pre) <= err + half * (np.abs(want_pre) + err)).all()
    if act in feed.GATED:
        gate, up = np.split(want_pre, 2, -1)
        e1, e2 = np.split(err, 2, -1)
        f = np.abs(feed.bend(gate, act)[0])
        far = 1.13 * e1 * (np.abs(up) + e2) + f * e2 + f * np.abs(up) * (gate ** 2 + 16) * 2.0 ** -22
    elif act is not None:
        far = 1.13 * err + np.abs(feed.bend(want_pre, act)[0]) * (want_pre ** 2 + 16) * 2.0 ** -22
    else:
        far = err
    if res is not None:
        far = far + 2.0 ** -24 * np.abs(out)
    bound = far + HALF_STEP[got.dtype] * (np.abs(out) + far) + 1e-37
    diff = np.abs(ref(got) - out)
    assert (diff <= bound).all(), f"{(diff / bound).max():.3g} of the bound"


def choose(name, monkeypatch):
    """Which kernel runs: what the sizes choose, or one of them."""
    if name == "planned":
        return name
    both, _, rest = name.rpartition("both ")
    side, _, parts = rest.partition(" in ")
    monkeypatch.setenv("SSM_FORCE_PRODUCT_SHAPE", str(["rows", "64", "128", "256"].index(side)))
    monkeypatch.setenv("SSM_FORCE_PRODUCT_PAIR", str(int("both" in name)))
    if parts:
        monkeypatch.setenv("SSM_FORCE_PRODUCT_PARTS", parts)
    return name


SHAPES = ["planned", "rows", "64", "64 in 3", "128", "128 in 2", "256"]


@pytest.fixture(params=SHAPES)
def shape(request, monkeypatch):
    return choose(request.param, monkeypatch)


# ("both": dx and dw by one launch, dw in so many parts)
@pytest.fixture(params=[s for s in SHAPES if s != "rows"] +
                ["both 64", "both 64 in 3", "both 128", "both 128 in 2", "both 256"])
def back_shape(request, monkeypatch):
    return choose(request.param, monkeypatch)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n,k", DENSE)
def test_linear(rows, n, k, act, dtype, shape):
    from selective_state_space_38_amd import linear_fwd
    nw = widths(n, act)
    x, w = rand(rows, k, dtype=dtype), rand(nw, k, dtype=dtype, seed=1, scale=k ** -0.5)
    bias = rand(nw, seed=2)
    out, pre = linear_fwd(x, w, bias=bias, activation=act, return_pre=True)
    assert out.dtype == pre.dtype == dtype and out.shape == (rows, n) and pre.shape == (rows, nw)
    check_fwd(ref(x), ref(w), ref(bias), act, None, out, pre)
    assert torch.equal(linear_fwd(x, w, bias=bias, activation=act), out)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    for res in (rand(rows, n, dtype=dtype, seed=3, scale=3.0), rand(rows, n, dtype=other, seed=3)):
        got = linear_fwd(x, w, activation=act, residual=res)
        assert got.dtype == res.dtype
        check_fwd(ref(x), ref(w), None, act, ref(res), got, None)
        own = res.clone()  # in place
        assert linear_fwd(x, w, activation=act, residual=own, out=own) is own
        assert torch.equal(own, got)


def test_column_slices_and_leading_dimensions():
    from selective_state_space_38_amd import linear_bwd, linear_fwd
    for dtype in DTYPES:
        wide = rand(3, 50, 96, dtype=dtype)
        x = wide[..., 32:72]
        w = rand(24, 40, dtype=dtype, seed=1)
        got = linear_fwd(x, w, activation="silu")
        assert got.shape == (3, 50, 24)
        assert torch.equal(got, linear_fwd(x.contiguous(), w, activation="silu"))
        dout = rand(3, 50, 24, dtype=dtype, seed=2)
        a = linear_bwd(dout, x, w, bias=True)
        b = linear_bwd(dout, x.contiguous(), w, bias=True)
        assert a["dx"].shape == (3, 50, 40) and all(torch.equal(a[key], b[key]) for key in b)


def experts_of(counts, rows, k, dtype, seed=0, spare=0):
    """x by token, offsets and token for the given rows of each expert."""
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    g = np.random.default_rng(seed)
    token = g.integers(0, rows, offsets[-1] + spare).astype(np.int32)
    x = rand(rows, k, dtype=dtype, seed=seed)
    return x, torch.from_numpy(offsets).cuda(), torch.from_numpy(token).cuda()


COUNTS = [[1], [0, 1, 0], [3, 0, 17, 1], [33, 64, 0, 0, 65, 2], [0, 0, 300], [130, 1, 129, 128, 0],
          [1] * 70 + [0] * 5 + [4], [5] * 130]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_expert_linear(counts, act, dtype, shape):
    from selective_state_space_38_amd import expert_linear_fwd
    n, k, rows = (72 if len(counts) % 2 else 75), 136, 50
    nw = widths(n, act)
    x, offsets, token = experts_of(counts, rows, k, dtype, spare=9)
    w = rand(len(counts), nw, k, dtype=dtype, seed=1, scale=k ** -0.5)
    bias = rand(len(counts), nw, seed=2)
    token[0] = rows              # no token: a row of zeros
    xs = feed.gather(ref(x), token.cpu().numpy())
    ends, all_rows = offsets.tolist(), len(token)
    kept = rand(all_rows, n, dtype=dtype, seed=5)
    own = kept.clone()
    out, pre = expert_linear_fwd(x, w, offsets, token=token, bias=bias, activation=act,
                                 return_pre=True, out=own)
    assert out is own and pre.shape == (all_rows, nw)
    used = ends[-1]
    check_fwd(xs[:used], ref(w), ref(bias), act, None, out[:used], pre[:used], ends)
    assert torch.equal(out[used:], kept[used:])      # behind the last expert's: as they were
    # rows in order already, no bias, another output type
    xt = torch.from_numpy(xs).to("cuda", dtype)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    got = expert_linear_fwd(xt, w, offsets, activation=act, out_dtype=other)
    check_fwd(xs[:used], ref(w), None, act, None, got[:used], None, ends)


# ---------------------------------------------------------------- gradient


def rounded(v, dtype):
    return torch.from_numpy(v).to(dtype).double().numpy()


def check_bwd(got, dout, x, w, pre, act, dtype, exact_dpre, bias, offsets=None):
    """got: the GPU's dict; the rest float64 arrays.  exact_dpre: dout serves as it is."""
    dpre = feed.activate_grad(dout, pre, act)
    if act is None:
        rel, slack = np.zeros_like(dpre), np.zeros_like(dpre)
    else:
        # a derivative is a sum of two terms: its error goes by their size, not its own
        v = np.concatenate([np.split(pre, 2, -1)[0]] * 2, -1) if act in feed.GATED else pre
        up = np.split(pre, 2, -1)[1] if act in feed.GATED else 1.0
        g = np.abs(dout) * np.abs(up)
        size = np.concatenate([1.13 * g, np.abs(dout) * np.abs(np.split(v, 2, -1)[0])], -1) \
            if act in feed.GATED else 1.13 * g
        rel = (v ** 2 + 32) * 2.0 ** -22
        slack = rel * size
    r = dpre if exact_dpre else rounded(dpre, dtype)
    if exact_dpre:
        far = slack
    else:
        far = np.maximum(np.abs(rounded(dpre + slack, dtype) - r), np.abs(r - rounded(dpre - slack, dtype)))
    half = HALF_STEP[dtype]
    dx, dw, _ = feed.product_grad(r, x, w, offsets)
    adx, adw, adb = feed.product_grad(np.abs(dpre), np.abs(x), np.abs(w), offsets)
    fdx, fdw, fdb = feed.product_grad(far, np.abs(x), np.abs(w), offsets)
    _, _, db = feed.product_grad(dpre, x, w, offsets)
    _, _, sdb = feed.product_grad(slack, x, w, offsets)
    for name, want, size, more, terms, h in (
            ("dx", dx, adx, fdx, w.shape[-2], half), ("dw", dw, adw, fdw, len(x), half),
            ("dbias", db, adb, sdb, len(x), 2.0 ** -24)):
        if name not in got:
            assert name == "dbias" and not bias
            continue
        err = (terms + 8) * 2.0 ** -23 * size + 1.01 * more
        bound = err + h * (np.abs(want) + err) + 1e-37
        diff = np.abs(ref(got[name]) - want)
        assert (diff <= bound).all(), f"{name}: {np.nanmax(diff / bound):.3g} of the bound"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n,k", DENSE)
def test_linear_gradient(rows, n, k, act, dtype, back_shape):
    from selective_state_space_38_amd import linear_bwd
    nw = widths(n, act)
    x, w = rand(rows, k, dtype=dtype), rand(nw, k, dtype=dtype, seed=1)
    pre = None if act is None else rand(rows, nw, dtype=dtype, seed=2, scale=2.0)
    dout = rand(rows, n, dtype=dtype, seed=3)
    g = linear_bwd(dout, x, w, activation=act, pre=pre, bias=True)
    assert g["dx"].dtype == g["dw"].dtype == dtype and g["dbias"].dtype == torch.float32
    check_bwd(g, ref(dout), ref(x), ref(w), ref(pre), act, dtype, act is None, True)
    # each alone
    for key, kw in (("dx", dict(need_dw=False)), ("dw", dict(need_dx=False)),
                    ("dbias", dict(need_dx=False, need_dw=False, bias=True))):
        one = linear_bwd(dout, x, w, activation=act, pre=pre, **kw)
        assert set(one) == {key}
        if "both" not in back_shape:  # (the parts of a sum may differ)
            assert torch.equal(one[key], g[key])
    # the other type's dout
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    dout = rand(rows, n, dtype=other, seed=3)
    g = linear_bwd(dout, x, w, activation=act, pre=pre, bias=True)
    check_bwd(g, ref(dout), ref(x), ref(w), ref(pre), act, dtype, dtype == torch.float32 and act is None, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", [None, "silu", "geglu"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_expert_linear_gradient(counts, act, dtype, back_shape):
    from selective_state_space_38_amd import expert_linear_bwd
    n, k, rows = (72 if len(counts) % 2 else 75), 136, 50
    nw = widths(n, act)
    x, offsets, token = experts_of(counts, rows, k, dtype, spare=9)
    token[0] = -1
    w = rand(len(counts), nw, k, dtype=dtype, seed=1)
    all_rows, ends = len(token), offsets.tolist()
    used = ends[-1]
    pre = None if act is None else rand(all_rows, nw, dtype=dtype, seed=2, scale=2.0)
    dout = rand(all_rows, n, dtype=dtype, seed=3)
    kept = rand(all_rows, k, dtype=dtype, seed=4)
    if pre is not None:
        pre[used:] = float("nan")
    dout[used:] = float("nan")   # rows behind the last expert's take no part
    g = expert_linear_bwd(dout, x, w, offsets, token=token, activation=act, pre=pre, bias=True,
                          dx=kept.clone())
    xs = feed.gather(ref(x), token.cpu().numpy())[:used]
    assert torch.equal(g["dx"][used:], kept[used:])
    g["dx"] = g["dx"][:used]
    check_bwd(g, ref(dout)[:used], xs, ref(w), None if pre is None else ref(pre)[:used], act, dtype,
              act is None, True, ends)
    for e, c in enumerate(counts):
        if c == 0:
            assert not g["dw"][e].any() and not g["dbias"][e].any()
    in_order = expert_linear_bwd(dout, torch.from_numpy(np.concatenate([xs, np.zeros((9, k))])).to("cuda", dtype),
                                 w, offsets, activation=act, pre=pre)
    assert torch.equal(in_order["dw"], g["dw"]) and torch.equal(in_order["dx"][:used], g["dx"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_row_that_is_not_finite_stays_its_own(dtype, shape, monkeypatch):
    from selective_state_space_38_amd import expert_linear_bwd, expert_linear_fwd
    counts, n, k = [5, 40, 3, 70], 72, 136
    x, offsets, token = experts_of(counts, 118, k, dtype)
    token = torch.arange(118, dtype=torch.int32, device="cuda")
    w = rand(4, n, k, dtype=dtype, seed=1)
    clean = expert_linear_fwd(x, w, offsets, token=token)
    bad = x.clone()
    bad[44] = float("nan")      # the last row of expert 1
    bad[45, 3] = float("inf")   # the first of expert 2
    got = expert_linear_fwd(bad, w, offsets, token=token)
    rest = [r for r in range(118) if r not in (44, 45)]
    assert got[44].isnan().all() and torch.equal(got[rest], clean[rest])
    if shape == "rows":
        monkeypatch.delenv("SSM_FORCE_PRODUCT_SHAPE")
        monkeypatch.setenv("SSM_FORCE_PRODUCT_PAIR", "1")
    dout = rand(118, n, dtype=dtype, seed=2)
    a = expert_linear_bwd(dout, x, w, offsets, token=token, bias=True)
    b = expert_linear_bwd(dout, bad, w, offsets, token=token, bias=True)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dbias"], b["dbias"])
    assert torch.equal(a["dw"][[0, 3]], b["dw"][[0, 3]])
    assert b["dw"][1].isnan().all() and not torch.isfinite(b["dw"][2][:, 3]).any()
    bad = dout.clone()
    bad[44] = float("nan")
    b = expert_linear_bwd(bad, x, w, offsets, token=token, bias=True)
    assert torch.equal(a["dx"][rest], b["dx"][rest]) and torch.equal(a["dw"][[0, 2, 3]], b["dw"][[0, 2, 3]])
    assert torch.equal(a["dbias"][[0, 2, 3]], b["dbias"][[0, 2, 3]]) and b["dbias"][1].isnan().all()


def test_offsets_outside_the_rows_stay_inside(shape, monkeypatch):
    # what the host cannot check: nothing outside the given arrays is touched
    from selective_state_space_38_amd import expert_linear_bwd, expert_linear_fwd
    n, k, rows = 24, 40, 37
    x, w = rand(rows, k), rand(3, n, k, seed=1)
    guard = rand(rows + 64, n, seed=2)
    for ends in ([0, 50, 60, 70], [-9, 5, 3, 37], [40, 41, 42, 43], [0, 2 ** 31 - 1, -2 ** 31, 5]):
        offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
        whole = guard.clone()
        expert_linear_fwd(x, w, offsets, out=whole[:rows])
        assert torch.equal(whole[rows:], guard[rows:])
        for both in "01":
            monkeypatch.setenv("SSM_FORCE_PRODUCT_PAIR", both)
            expert_linear_bwd(whole[:rows], x, w, offsets, bias=True)
    torch.cuda.synchronize()


def test_refusals():
    from selective_state_space_38_amd import (expert_linear_bwd, expert_linear_fwd, linear_bwd,
                                              linear_fwd)
    x, w = rand(10, 24), rand(16, 24)
    for bad in (x.cpu(), x.half(), x[:, :16], x[0], rand(10, 48)[:, ::2], x.bfloat16()):
        with pytest.raises(ValueError):
            linear_fwd(bad, w)
    for kw in (dict(w=rand(16, 20)), dict(x=rand(10, 20), w=rand(16, 20)), dict(w=w.t()), dict(activation="tanh"),
               dict(activation="swiglu", w=rand(25, 24)), dict(bias=rand(15)), dict(bias=rand(16).double()),
               dict(residual=rand(10, 15)), dict(out_dtype=torch.float16), dict(out=rand(9, 16)),
               dict(residual=rand(10, 16), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            linear_fwd(**{**dict(x=x, w=w), **kw})
    with pytest.raises(RuntimeError):                          # not 16-byte aligned
        linear_fwd(rand(10 * 24 + 1)[1:].view(10, 24), w)
    with pytest.raises(RuntimeError):                          # rows 36 values apart
        linear_fwd(rand(10, 36)[:, :24], w)
    with pytest.raises(RuntimeError):                          # an output that is an input
        linear_fwd(rand(16, 16), (v := rand(16, 16)), out=v)
    with pytest.raises(RuntimeError):
        linear_fwd(rand(0, 24), w)
    dout = rand(10, 16)
    for kw in (dict(dout=rand(10, 15)), dict(dout=dout.half()), dict(pre=dout), dict(activation="silu"),
               dict(need_dx=False, need_dw=False), dict(activation="silu", pre=rand(9, 16))):
        with pytest.raises(ValueError):
            linear_bwd(**{**dict(dout=dout, x=x, w=w), **kw})
    we, offsets = rand(3, 16, 24), torch.tensor([0, 2, 4, 10], dtype=torch.int32, device="cuda")
    token = torch.zeros(10, dtype=torch.int32, device="cuda")
    for kw in (dict(offsets=None), dict(offsets=offsets[:3]), dict(offsets=offsets.long()),
               dict(token=token.long()), dict(token=token.view(2, 5)), dict(w=w), dict(x=rand(2, 5, 24)),
               dict(w=rand(0, 16, 24))):
        with pytest.raises(ValueError):
            expert_linear_fwd(**{**dict(x=x, w=we, offsets=offsets), **kw})
    with pytest.raises(ValueError):
        expert_linear_bwd(dout, x, we, None)
    with pytest.raises(ValueError):
        expert_linear_bwd(dout, x, we, offsets, dx=rand(9, 24))
