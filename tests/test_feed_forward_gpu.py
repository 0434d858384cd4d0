"""The feed-forward layer's operators together, as a layer calls them: a layer of
experts forward and backward against torch in float64, on other streams, from
captured graphs and through the example.

Tolerances of the float32 layer, on the largest magnitude of the compared array:
each product is a float32 sum of at most 264 terms, off by at most 272 2^-23 =
3.3e-5 of its terms' summed magnitude; the forward is two of them and a sum of k
rows, the backward four, so 4 stages of 3.3e-5 and what the other operators' few
roundings add stay below 2e-4 of the terms' magnitude, which here is at most 5 times
the largest result: 1e-3.
"""

import pathlib
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent / "examples"))

TOL = 1e-3


def rand(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to("cuda", dtype)


def close(got, want, tol=TOL, name=""):
    got, want = got.double(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    err, size = (got - want).abs().max().item(), want.abs().max().item()
    assert err <= tol * size, f"{name}: {err:.3e} of {size:.3e}"


def layer_of(tokens, dim, hidden, experts, dtype=torch.float32):
    return dict(x=rand(tokens, dim, dtype=dtype), wr=rand(experts, dim, dtype=dtype, seed=1, scale=dim ** -0.5),
                w1=rand(experts, 2 * hidden, dim, dtype=dtype, seed=2, scale=dim ** -0.5),
                b1=rand(experts, 2 * hidden, seed=3, scale=0.1),
                w2=rand(experts, dim, hidden, dtype=dtype, seed=4, scale=hidden ** -0.5),
                dout=rand(tokens, dim, dtype=dtype, seed=5), dtotal=rand(experts, seed=6, scale=0.1))


def run(v, k, capacity=None):
    """Forward and backward of a layer of experts; capacity: most rows an expert takes."""
    import selective_state_space_38_amd as ssm
    experts = len(v["w1"])
    logits = ssm.linear_fwd(v["x"], v["wr"])
    index, weight, total = ssm.expert_route_fwd(logits, k, renormalize=True, return_score_sum=True)
    if capacity is not None:  # choices past an expert's capacity are dropped
        hot = torch.nn.functional.one_hot(index.long().flatten(), experts)
        place = (hot.cumsum(0) * hot).sum(1).view_as(index)
        index = torch.where(place <= capacity, index, -1)
    offsets, token, slot = ssm.expert_sort(index, experts)
    h, pre = ssm.expert_linear_fwd(v["x"], v["w1"], offsets, token=token, bias=v["b1"],
                                   activation="swiglu", return_pre=True)
    y = ssm.expert_linear_fwd(h, v["w2"], offsets)
    out = ssm.expert_combine_fwd(y, slot, weight, residual=v["x"])
    g = ssm.expert_combine_bwd(v["dout"], y, slot, weight)
    dweight = g["dweight"]
    g2 = ssm.expert_linear_bwd(g["dy"], h, v["w2"], offsets)
    g1 = ssm.expert_linear_bwd(g2["dx"], v["x"], v["w1"], offsets, token=token, activation="swiglu",
                               pre=pre, bias=True)
    dlogits = ssm.expert_route_bwd(logits, index, dweight, renormalize=True, dscore_sum=v["dtotal"])
    gr = ssm.linear_bwd(dlogits, v["x"], v["wr"])
    dx = ssm.expert_combine_fwd(g1["dx"], slot, residual=v["dout"]) + gr["dx"]
    return dict(index=index, out=out, dx=dx, dwr=gr["dw"], dw1=g1["dw"], db1=g1["dbias"], dw2=g2["dw"])


def reference(v, index):
    """The same in float64 by autograd, choice by choice."""
    t = {k: a.double().cpu().requires_grad_() for k, a in v.items()}
    index = index.cpu()
    p = torch.softmax(t["x"] @ t["wr"].t(), 1)
    chosen = [p.gather(1, index[:, j:j + 1].clamp_min(0).long())[:, 0] for j in range(index.shape[1])]
    kept = [index[:, j] >= 0 for j in range(index.shape[1])]
    return t, p, chosen, kept


@pytest.mark.parametrize("tokens,dim,hidden,experts,k", [
    (1, 8, 8, 2, 1), (3, 40, 24, 5, 2), (70, 264, 136, 6, 3), (600, 64, 128, 16, 4), (33, 128, 264, 40, 8)])
def test_layer_of_experts(tokens, dim, hidden, experts, k):
    v = layer_of(tokens, dim, hidden, experts)
    got = run(v, k)
    t, p, chosen, _ = reference(v, got["index"])
    total = sum(chosen)
    out = t["x"]
    for j in range(k):
        e = got["index"][:, j].cpu().long()
        pre = torch.bmm(t["w1"][e], t["x"].unsqueeze(2)).squeeze(2) + t["b1"][e]
        gate, up = pre.chunk(2, 1)
        y = torch.bmm(t["w2"][e], (torch.nn.functional.silu(gate) * up).unsqueeze(2)).squeeze(2)
        out = out + (chosen[j] / total).unsqueeze(1) * y
    value = (out * t["dout"].detach()).sum() + (p.sum(0) * t["dtotal"].detach()).sum()
    names = ("x", "wr", "w1", "b1", "w2")
    grads = torch.autograd.grad(value, [t[n] for n in names])
    close(got["out"].cpu(), out.detach(), name="out")
    for n, g in zip(names, grads):
        if k == experts == 1 and n == "wr":
            continue
        close(got["d" + n].cpu(), g, name="d" + n)


def test_dropped_choices():
    # experts take 20 rows each: what is past that adds nothing and gets no gradient
    v = layer_of(200, 64, 40, 4)
    got = run(v, 2, capacity=20)
    index = got["index"]
    counts = torch.bincount(index[index >= 0].flatten().cpu(), minlength=4)
    assert (counts <= 20).all() and (index < 0).any(1).all(0).item() is False
    gone = (index < 0).all(1)
    assert gone.any()
    assert torch.equal(got["out"][gone], v["x"][gone])
    for key in ("dw1", "dw2", "dx", "dwr"):
        assert torch.isfinite(got[key]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_other_streams_at_once(dtype):
    v = [layer_of(n, 128, 72, 8, dtype=dtype) for n in (300, 7)]
    want = [run(a, 2) for a in v]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in v]
    for _ in range(3):
        got = []
        for a, s in zip(v, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run(a, 2))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for key in b:
                assert torch.equal(a[key], b[key]), key


@pytest.mark.parametrize("tokens", [4, 500])
def test_forward_and_backward_from_two_graphs(tokens):
    v = layer_of(tokens, 136, 64, 8, dtype=torch.bfloat16)
    kept = {k: a.clone() for k, a in v.items()}
    other = {k: rand(*a.shape, dtype=a.dtype, seed=20 + i, scale=float(a.float().std()))
             for i, (k, a) in enumerate(v.items())}
    want = [run(kept, 2), run(other, 2)]
    run(v, 2)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(v, 2)
        graphs.append((g, out))
    for which in (0, 1, 1, 0):
        for key, a in v.items():
            a.copy_((kept, other)[which][key])
        for g, out in graphs:
            for t in out.values():
                t.fill_(-7)
            g.replay()
        run(kept, 2)                                    # eager work in between
        torch.cuda.synchronize()
        for g, out in graphs:
            for key, t in want[which].items():
                assert torch.equal(out[key], t), key


def test_results_do_not_depend_on_timing():
    v = layer_of(3000, 264, 136, 12, dtype=torch.bfloat16)
    want = run(v, 3)
    for _ in range(5):
        got = run(v, 3)
        for key in want:
            assert torch.equal(got[key], want[key]), key


def test_products_past_32_bits_of_bytes():
    # rows that start more than 2^32 bytes into x and out
    import selective_state_space_38_amd as ssm
    rows, k, n = (1 << 20) + 300, 2056, 16
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    last = rand(5, k, dtype=torch.bfloat16)
    x[-5:] = last
    w = rand(n, k, dtype=torch.bfloat16, seed=1)
    out = ssm.linear_fwd(x, w)
    assert torch.equal(out[-5:], ssm.linear_fwd(last, w)) or \
        (out[-5:].double() - last.double() @ w.double().t()).abs().max() <= 2.0 ** -7 * out[-5:].abs().max()
    assert not out[:1000].any()
    dout = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    dout[-5:] = rand(5, n, dtype=torch.bfloat16, seed=2)
    g = ssm.linear_bwd(dout, x, w, bias=True)
    close(g["dw"], dout[-5:].double().t() @ last.double(), tol=2.0 ** -7)
    close(g["dx"][-5:], dout[-5:].double() @ w.double(), tol=2.0 ** -7)
    close(g["dbias"], dout[-5:].double().sum(0), tol=1e-5)


def loss_in_double(layers, tokens, target, rate=1e-2):
    stream, balance = tokens.double(), 0.0

    def swiglu(v):
        gate, up = v.chunk(2, -1)
        return torch.nn.functional.silu(gate) * up

    for layer in layers:
        u = stream * torch.rsqrt(stream.square().mean(1, keepdim=True) + 1e-5) * layer.norm.double()
        w1, w2 = layer.w1.double(), layer.w2.double()
        if not hasattr(layer, "wr"):
            stream = stream + swiglu(u @ w1.t()) @ w2.t()
            continue
        p = torch.softmax(u @ layer.wr.double().t(), 1)
        chosen, index = p.topk(layer.k, 1)
        share = torch.bincount(index.flatten(), minlength=layer.experts) / index.numel()
        balance = balance + layer.experts * (share * p.sum(0)).sum() / len(u)
        weight = chosen / chosen.sum(1, keepdim=True)
        for j in range(layer.k):
            h = swiglu(torch.bmm(w1[index[:, j]], u.unsqueeze(2)).squeeze(2))
            stream = stream + weight[:, j:j + 1] * torch.bmm(w2[index[:, j]], h.unsqueeze(2)).squeeze(2)
    return (stream - target.double()).square().mean() + rate * balance


def test_example_runs_and_its_gradients():
    import expert_layer as ex
    layers = [ex.Dense(64, 48, 0, dtype=torch.float32), ex.Experts(64, 40, 6, 2, 1, dtype=torch.float32)]
    tokens = rand(50, 64)
    target = rand(50, 64, seed=1)
    out = ex.forward(layers, tokens)
    assert out.shape == (50, 64) and torch.isfinite(out).all()
    params = [p.requires_grad_() for layer in layers for p in layer.params()]
    loss = ex.loss_of(layers, tokens, target)
    grads = torch.autograd.grad(loss, params)
    # against float64 autograd with the same choice (a difference along the router's
    # gradient, which is small, would change the choice); the tolerance: two layers' stages
    want = torch.autograd.grad(loss_in_double(layers, tokens, target), params)
    for p, g, w in zip(params, grads, want):
        close(g, w, 2 * TOL, str(tuple(p.shape)))
    for p in params:
        p.requires_grad_(False)
    few = tokens[:4].clone()
    want = ex.forward(layers, few)
    graph, got = ex.capture(layers, few)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    before = [p.clone() for layer in layers for p in layer.params()]
    assert len(ex.train(layers, tokens, target, 2)) == 2
    after = [p for layer in layers for p in layer.params()]
    assert all(not torch.equal(a, b) for a, b in zip(before, after))
