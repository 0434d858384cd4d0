"""The linear product and its gradient on the GPU at sizes with many tiles, strips and parts,
every row and column in use, against float64.

Without an activation: operands are whole numbers of -2 .. 2, so that each sum, of at most
70000 products of size 4, is a whole number below 2^24 that float32 holds whatever the
order: outputs equal the float64 product's, rounded once.  No tolerance.

With one: a float32 sum of K products and a bias errs by at most (K + 8) 2^-23 of the terms'
summed magnitude.  A slope or value of the activation is within (v^2 + 32) 2^-22 of its
terms' size (1.13 at most for a slope); dpre, rounded to the activations' type in front of
the products, errs by its half step more, and so do the outputs.
"""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def whole(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)


def rand(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def force(monkeypatch, shape=None, pair=None, parts=None):
    for name, v in (("SHAPE", shape), ("PAIR", pair), ("PARTS", parts)):
        if v is not None:
            monkeypatch.setenv(f"SSM_FORCE_PRODUCT_{name}", str(v))


# rows, n, k: more tiles than CUs, many strips of row tiles, a long sum over the rows
LARGE = [(4100, 5128, 2568), (1031, 2568, 1288), (70000, 264, 136), (2047, 768, 1536), (300, 9000, 1032)]
# (shape, one launch, parts): as the sizes choose, or 64, 128 and 256 to a side
PLANS = [(None, None, None), (1, 1, 3), (1, 0, 5), (2, 1, 2), (2, 0, None), (3, 1, None), (3, 0, None)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("rows,n,k", LARGE)
def test_whole_numbers(rows, n, k, plan, dtype, monkeypatch):
    from selective_state_space_38_amd import linear_bwd, linear_fwd
    force(monkeypatch, *plan)
    x, w = whole(rows, k, dtype=dtype, seed=0), whole(n, k, dtype=dtype, seed=1)
    bias, res = whole(n, dtype=torch.float32, seed=2), whole(rows, n, dtype=torch.float32, seed=3)
    want = x.double() @ w.double().t().contiguous() + bias.double()
    assert torch.equal(linear_fwd(x, w, bias=bias), want.to(dtype))
    assert torch.equal(linear_fwd(x, w, bias=bias, residual=res), (want + res).float())
    dout = whole(rows, n, dtype=dtype, seed=4)
    g = linear_bwd(dout, x, w, bias=True)
    assert torch.equal(g["dx"], (dout.double() @ w.double()).to(dtype))
    assert torch.equal(g["dw"], (dout.double().t().contiguous() @ x.double()).to(dtype))
    assert torch.equal(g["dbias"], dout.double().sum(0).float())


# rows of each expert: many tiles of some, none of others, nearly all of one, a few each, all of one
COUNTS = [[700, 0, 33, 1300, 1, 0, 146, 512, 129, 0, 640], [5, 3000, 0, 9] + [17] * 20, [40] * 64,
          [0] * 40 + [512] + [0] * 23]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("plan", PLANS + [(0, None, None)], ids=str)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_whole_numbers_of_experts(counts, plan, dtype, monkeypatch):
    from selective_state_space_38_amd import expert_linear_bwd, expert_linear_fwd
    force(monkeypatch, *plan)
    n, k, tokens, spare = 392, 520, 900, 70
    ends = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(ends.astype(np.int32)).cuda()
    rows, used = int(ends[-1]) + spare, int(ends[-1])
    g = torch.Generator(device="cuda").manual_seed(7)
    token = torch.randint(0, tokens, (rows,), generator=g, device="cuda", dtype=torch.int32)
    token[used // 2] = -1
    x, w = whole(tokens, k, dtype=dtype, seed=0), whole(len(counts), n, k, dtype=dtype, seed=1)
    bias, dout = whole(len(counts), n, dtype=torch.float32, seed=2), whole(rows, n, dtype=dtype, seed=3)
    xs = torch.where((token >= 0)[:, None], x[token.clamp_min(0).long()], 0).double()
    kept = rand(rows, n, dtype=dtype, seed=5)
    out = expert_linear_fwd(x, w, offsets, token=token, bias=bias, out=kept.clone())
    kept_dx = rand(rows, k, dtype=dtype, seed=6)
    got = expert_linear_bwd(dout, x, w, offsets, token=token, bias=True, dx=kept_dx.clone())
    assert torch.equal(out[used:], kept[used:]) and torch.equal(got["dx"][used:], kept_dx[used:])
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        d = dout[a:b].double()
        want = xs[a:b] @ w[e].double().t().contiguous() + bias[e].double()
        assert torch.equal(out[a:b], want.to(dtype)), e
        assert torch.equal(got["dx"][a:b], (d @ w[e].double()).to(dtype)), e
        assert torch.equal(got["dw"][e], (d.t().contiguous() @ xs[a:b]).to(dtype)), e
        assert torch.equal(got["dbias"][e], d.sum(0).float()), e


# ---------------------------------------------------------------- with an activation


def bent(v, act):
    """f(v) and f'(v) in float64."""
    if act in ("silu", "swiglu"):
        s = torch.sigmoid(v)
        return v * s, s * (1.0 + v * torch.sigmoid(-v))
    phi = 0.5 * torch.erfc(-v / math.sqrt(2.0))
    return v * phi, phi + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def inside(got, want, bound, name):
    worst = ((got.double() - want).abs() / bound).max().item()
    assert worst <= 1, f"{name}: {worst:.3g} of the bound"  # (a NaN fails too)


def check_gradient(got, dout, x, w, pre, act, dtype, name=""):
    """got: the GPU's dict; x, w, pre, dout: float64."""
    gated = act in ("swiglu", "geglu")
    v, up = pre.chunk(2, 1) if gated else (pre, None)
    f, slope = bent(v, act)
    rel = (v * v + 32) * 2.0 ** -22
    g = dout.abs() * (up.abs() if gated else 1.0)
    dpre, far = dout * slope * (up if gated else 1.0), 1.13 * g * rel
    if gated:
        dpre, far = torch.cat([dpre, dout * f], 1), torch.cat([far, (dout * v).abs() * rel], 1)
    half = HALF_STEP[dtype]
    # dpre in front of the products: its own error, and its rounding's
    apart = far + half * (dpre.abs() + far)
    adx, adw = dpre.abs() @ w.abs(), dpre.abs().t().contiguous() @ x.abs()
    for key, want, size, more, terms, h in (
            ("dx", dpre @ w, adx, apart @ w.abs(), w.shape[0], half),
            ("dw", dpre.t().contiguous() @ x, adw, apart.t().contiguous() @ x.abs(), len(x), half),
            ("dbias", dpre.sum(0), dpre.abs().sum(0), far.sum(0), len(x), 2.0 ** -24)):
        if key in got:
            err = (terms + 8) * 2.0 ** -23 * size + 1.01 * more
            inside(got[key], want, err + h * (want.abs() + err) + 1e-37, name + key)


# 47 partial sums of the bias, three a strand; over 2^25 outputs, where a partial sum takes 128 rows
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("rows,n,k", [(1500, 520, 264), (8200, 4104, 16)])
def test_gradient(rows, n, k, pair, act, dtype, monkeypatch):
    from selective_state_space_38_amd import linear_bwd
    force(monkeypatch, pair=pair)
    nw = 2 * n if act in ("swiglu", "geglu") else n
    x, w = rand(rows, k, dtype=dtype), rand(nw, k, dtype=dtype, seed=1)
    pre, dout = rand(rows, nw, dtype=dtype, seed=2, scale=2.0), rand(rows, n, dtype=dtype, seed=3)
    got = linear_bwd(dout, x, w, activation=act, pre=pre, bias=True)
    check_gradient(got, dout.double(), x.double(), w.double(), pre.double(), act, dtype)
    alone = linear_bwd(dout, x, w, activation=act, pre=pre, need_dx=False, need_dw=False, bias=True)
    assert torch.equal(alone["dbias"], got["dbias"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("counts,n,k", [([700, 0, 33, 1300, 1], 264, 136), ([2500, 0, 5700, 3, 129], 4104, 16)],
                         ids=["32 rows", "128 rows"])
def test_gradient_of_experts(counts, n, k, pair, act, dtype, monkeypatch):
    from selective_state_space_38_amd import expert_linear_bwd
    force(monkeypatch, pair=pair)
    nw = 2 * n if act == "swiglu" else n
    ends = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(ends.astype(np.int32)).cuda()
    rows = int(ends[-1])
    assert (rows * n >= 1 << 25) == (n > 264)
    x, w = rand(rows, k, dtype=dtype), rand(len(counts), nw, k, dtype=dtype, seed=1)
    pre, dout = rand(rows, nw, dtype=dtype, seed=2, scale=2.0), rand(rows, n, dtype=dtype, seed=3)
    got = expert_linear_bwd(dout, x, w, offsets, activation=act, pre=pre, bias=True)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a == b:
            assert not got["dw"][e].any() and not got["dbias"][e].any()
            continue
        mine = dict(dx=got["dx"][a:b], dw=got["dw"][e], dbias=got["dbias"][e])
        check_gradient(mine, dout[a:b].double(), x[a:b].double(), w[e].double(), pre[a:b].double(), act,
                       dtype, f"expert {e}: ")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "geglu"])
@pytest.mark.parametrize("rows,n,k", [(4100, 2568, 1288), (16500, 520, 264)])
def test_forward(rows, n, k, act, dtype):
    from selective_state_space_38_amd import linear_fwd
    nw = 2 * n if act == "geglu" else n
    x, w, bias = rand(rows, k, dtype=dtype), rand(nw, k, dtype=dtype, seed=1, scale=k ** -0.5), rand(nw, seed=2)
    out, pre = linear_fwd(x, w, bias=bias, activation=act, return_pre=True)
    want = x.double() @ w.double().t().contiguous() + bias.double()
    size = x.double().abs() @ w.double().abs().t().contiguous() + bias.double().abs()
    err, half = (k + 8) * 2.0 ** -23 * size, HALF_STEP[dtype]
    inside(pre, want, err + half * (want.abs() + err), "pre")
    (v, up), (e1, e2) = (want.chunk(2, 1), err.chunk(2, 1)) if act == "geglu" else ((want, None), (err, None))
    f = bent(v, act)[0]
    far = 1.13 * e1 + f.abs() * (v * v + 16) * 2.0 ** -22
    if act == "geglu":
        far, f = far * (up.abs() + e2) + f.abs() * e2, f * up
    inside(out, f, far + half * (f.abs() + far) + 1e-37, "out")
