"""The operators together: the example's layers, in pieces and as a whole.

Tolerance: two ways to one state differ by float32 roundings, which move an
8-bit value by at most one of its steps where it lies between two; were all
moved, the difference would be a step, 2^-3 of a value; on the norm over all
values, 2^-4 is that with one value in four moved.
"""

import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def stack(dim, inner, count=2):
    from residual_layer import Layer
    return [Layer(dim, inner, k).serve() for k in range(count)]


@pytest.mark.parametrize("dim,inner", [(256, 384), (208, 144)])
@pytest.mark.parametrize("batch,length", [(1, 40), (3, 200)])
def test_decode_continues_prefill(dim, inner, batch, length):
    from residual_layer import decode, prefill
    layers = stack(dim, inner)
    g = torch.Generator().manual_seed(length)
    tokens = torch.randn(batch, length + 8, dim, generator=g).bfloat16().cuda()
    whole, last = prefill(layers, tokens)
    first, states = prefill(layers, tokens[:, :length].contiguous())
    assert off(first, whole[:, :length]) <= 2 ** -4
    for t in range(length, length + 8):
        got = decode(layers, tokens[:, t].contiguous(), states)
        assert off(got, whole[:, t]) <= 2 ** -4
    for got, want in zip(states, last):
        assert off(got, want) <= 2 ** -4


def test_packed_documents_are_apart():
    from residual_layer import prefill
    layers = stack(256, 384)
    g = torch.Generator().manual_seed(3)
    tokens = torch.randn(1, 300, 256, generator=g).bfloat16().cuda()
    cuts = [0, 1, 130, 300]
    reset = torch.zeros(1, 300, dtype=torch.bool, device="cuda")
    reset[:, cuts[:-1]] = True
    whole, last = prefill(layers, tokens, reset)
    for a, b in zip(cuts, cuts[1:]):
        one, states = prefill(layers, tokens[:, a:b].contiguous(), reset[:, a:b].contiguous())
        assert off(whole[:, a:b], one) <= 2 ** -4
    for got, want in zip(last, states):
        assert off(got, want) <= 2 ** -4


def test_decode_from_a_graph():
    from residual_layer import capture, decode, prefill
    layers = stack(256, 384)
    g = torch.Generator().manual_seed(6)
    tokens = torch.randn(3, 30, 256, generator=g).bfloat16().cuda()
    _, states = prefill(layers, tokens[:, :20].contiguous())
    eager = [s.clone() for s in states]
    token = tokens[:, 20].contiguous()
    graph, out = capture(layers, token, states)
    for got, want in zip(states, eager):
        assert torch.equal(got, want)
    for t in range(20, 30):
        want = decode(layers, tokens[:, t].contiguous(), eager)
        token.copy_(tokens[:, t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for a, b in zip(states, eager):
            assert torch.equal(a, b)


def test_training_lowers_the_loss():
    from residual_layer import Layer, train
    layers = [Layer(128, 192, k) for k in range(2)]
    g = torch.Generator().manual_seed(4)
    tokens = torch.randn(2, 96, 128, generator=g).bfloat16().cuda()
    reset = torch.zeros(2, 96, dtype=torch.bool, device="cuda")
    reset[:, 50] = True
    losses = train(layers, tokens, tokens.float().cumsum(1) * 0.1, reset, 10)
    assert losses[-1] < losses[0]


def test_command():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "residual_layer.py"),
                          "--layers", "2", "--dim", "256", "--inner", "384", "--batch", "2",
                          "--seqlen", "256", "--steps", "4", "--train-steps", "2"],
                         capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    assert "prefill" in out.stdout and "decode" in out.stdout
