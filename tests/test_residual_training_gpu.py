"""The example's training step reaches every parameter of every layer."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def test_every_parameter_moves():
    from residual_layer import Layer, train
    names = ("norm", "w_in", "b_in", "w_out", "log_decay")
    layers = [Layer(128, 192, k) for k in range(3)]
    before = [[getattr(layer, n).clone() for n in names] for layer in layers]
    g = torch.Generator().manual_seed(4)
    tokens = torch.randn(2, 96, 128, generator=g).bfloat16().cuda()
    reset = torch.zeros(2, 96, dtype=torch.bool, device="cuda")
    reset[:, 50] = True
    losses = train(layers, tokens, tokens.float().cumsum(1) * 0.1, reset, 4)
    assert losses[-1] < losses[0]
    for k, layer in enumerate(layers):
        for name, was in zip(names, before[k]):
            now = getattr(layer, name)
            assert torch.isfinite(now).all()
            # all of a bias's columns, x, r and i, as of the others
            share = float((now != was).float().mean())
            assert share > 0.9, (k, name, share)
