"""A carry wait of the gated recurrence that hits its bound ends and is
reported.  A bound of no repeated poll makes every wait give up that is not
satisfied at once; with a thousand workgroups of a few steps in one chain, started
together, some are not.  Inputs are those of test_gated_scan_gpu."""

import pytest
import torch

from test_gated_scan_gpu import backward, forward, make

pytestmark = pytest.mark.gpu


def run(call, monkeypatch):
    """call() with a bound of no repeated poll, and the report of it."""
    from selective_state_space_38_amd import check_device_errors
    monkeypatch.setenv("SSM_FORCE_GATED_WAVES", "2")
    want = call()
    check_device_errors()  # none timed out
    monkeypatch.setenv("SSM_TEST_SPIN_LIMIT", "0")
    call()
    monkeypatch.delenv("SSM_TEST_SPIN_LIMIT")
    with pytest.raises(RuntimeError, match="SSM_ETIMEOUT"):
        check_device_errors()
    check_device_errors()  # reported once
    again = call()
    check_device_errors()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_forward(monkeypatch):
    s = make(1, 1 << 15, 64, torch.float32)
    run(lambda: forward(s), monkeypatch)


def test_backward(monkeypatch):
    from selective_state_space_38_amd import gated_ckpt_buffer
    s = make(1, 1 << 15, 64, torch.float32)
    ckpt = gated_ckpt_buffer(s["x"])
    forward(s, ckpt=ckpt)
    run(lambda: tuple(backward(s, ckpt).values()), monkeypatch)
