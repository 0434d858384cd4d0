"""A gate that is not a number, in one channel of one sequence: what depends on
it is not a number, everything else is what it is without it, bit for bit.
Inputs are those of test_gated_scan_gpu."""

import pytest
import torch

from test_gated_scan_gpu import DTYPES, backward, forward, make

pytestmark = pytest.mark.gpu

ROW, CHANNEL = 1, 5
CASES = [(2, 40, 66, 39, None), (2, 40, 66, 10, [25]), (2, 600, 66, 300, [120, 450]),
         (3, 2500, 70, 2499, None), (2, 2500, 70, 700, [100, 2000]), (2, 2500, 70, 50, [300]),
         (260, 3, 130, 1, None), (260, 3, 130, 2, [1])]


def spoilt(s, key, at):
    t = s[key].clone()
    t[ROW, at, CHANNEL] = float("nan")
    return {**s, key: t}


def check(got, want, nan_steps, name):
    """got is not a number at ROW, CHANNEL and the steps given, and want elsewhere."""
    bad = torch.zeros_like(want, dtype=torch.bool)
    bad[ROW, nan_steps, CHANNEL] = True
    assert torch.isnan(got[bad]).all(), name
    assert torch.equal(got[~bad], want[~bad]), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bsz,length,dim,at,resets", CASES)
def test_decay_gate(bsz, length, dim, at, resets, dtype):
    s = make(bsz, length, dim, dtype, resets=resets, seed=at)
    bad = spoilt(s, "r", at)
    out, last = forward(s)
    got, got_last = forward(bad)
    begin = max([t for t in resets or [] if t <= at], default=0)      # of the document
    end = min([t for t in resets or [] if t > at], default=length)
    check(got, out, slice(at, end), "out")
    check(got_last[:, None], last[:, None], slice(0, 1 if end == length else 0), "last")
    g, want = backward(bad), backward(s)
    check(g["dx"], want["dx"], slice(begin, at + 1), "dx")
    check(g["di"], want["di"], slice(begin, at + 1), "di")
    # the decay's gradient needs the state before a step, too
    first = begin + 1 if begin in (resets or []) else begin
    check(g["dr"], want["dr"], slice(first, end), "dr")
    check(g["dh0"][:, None], want["dh0"][:, None], slice(0, 0 if first > begin else 1), "dh0")
    rest = [c for c in range(dim) if c != CHANNEL]
    assert torch.isnan(g["dlog_decay"][CHANNEL])
    assert torch.equal(g["dlog_decay"][rest], want["dlog_decay"][rest])


@pytest.mark.parametrize("dtype", DTYPES)
def test_decay_rate(dtype):
    s = make(2, 300, 66, dtype, resets=[100])
    bad = {**s, "log_decay": s["log_decay"].clone()}
    bad["log_decay"][CHANNEL] = float("nan")
    g, want = backward(bad), backward(s)
    rest = [c for c in range(66) if c != CHANNEL]
    for k in want:
        assert torch.equal(g[k][..., rest], want[k][..., rest]), k
    # at a reset the input's weight does not depend on the rate
    kept = torch.zeros(2, 300, dtype=torch.bool, device="cuda") | s["reset"]
    for k in ("dx", "di"):
        assert torch.isnan(g[k][..., CHANNEL][~kept]).all(), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_step(dtype):
    from selective_state_space_38_amd import gated_state_update
    s = make(2, 1, 66, dtype)
    one = {k: s[k][:, 0].contiguous() for k in ("x", "r", "i")}
    want_state, state = s["h0"].clone(), s["h0"].clone()
    want = gated_state_update(want_state, one["x"], one["r"], one["i"], s["log_decay"])
    one["r"][ROW, CHANNEL] = float("nan")
    out = gated_state_update(state, one["x"], one["r"], one["i"], s["log_decay"])
    check(out[:, None], want[:, None], slice(0, 1), "out")
    check(state[:, None], want_state[:, None], slice(0, 1), "state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bsz,length,dim,at", [(2, 40, 66, 0), (2, 40, 66, 39), (2, 600, 66, 128),
                                               (2, 2500, 70, 1000), (260, 3, 130, 1)])
def test_decay_gate_at_a_reset(bsz, length, dim, at, dtype):
    # a document's first step does not use its decay gate: nothing changes
    s = make(bsz, length, dim, dtype, resets=[0, at], seed=at)
    bad = spoilt(s, "r", at)
    for got, want in zip(forward(bad), forward(s)):
        assert torch.equal(got, want)
    got, want = backward(bad), backward(s)
    for k in want:
        assert torch.equal(got[k], want[k]), k
