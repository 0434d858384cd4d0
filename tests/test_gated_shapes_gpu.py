"""The gated recurrence in each of its launch shapes: workgroups of few and of
many waves, two channels per lane at odd channel counts.  Inputs and tolerances
are those of test_gated_scan_gpu."""

import pytest
import torch

from test_gated_scan_gpu import DTYPES, check_backward, check_forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [31, 33, 257, 600])
@pytest.mark.parametrize("waves", [2, 4, 16])
def test_waves(waves, length, dtype, monkeypatch):
    monkeypatch.setenv("SSM_FORCE_GATED_WAVES", str(waves))
    s = make(3, length, 66, dtype, resets=[0, 17, 256], fused=True, seed=waves)
    check_forward(s)
    check_backward(s)
    check_backward(make(2, length, 65, dtype, seed=waves), ckpt=False)


@pytest.mark.parametrize("bsz,length,dim", [(3, 8192, 129), (3, 8200, 131), (1, 11000, 259),
                                            (40, 300, 255), (130, 40, 257), (260, 1, 127)])
def test_pairs_of_channels(bsz, length, dim):
    # bfloat16 with enough work for every compute unit at two channels a lane;
    # the last lane's pair overlaps its neighbour's where dim is odd
    s = make(bsz, length, dim, torch.bfloat16, resets=[0, 33, 4096], fused=True, seed=dim)
    check_forward(s)
    check_backward(s)


@pytest.mark.parametrize("dtype", DTYPES)
def test_unaligned_slices(dtype):
    # columns that start and step at odd elements
    from selective_state_space_38_amd import gated_scan_fwd, gated_state_update
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(2, 150, 3 * 67 + 2, generator=g).to("cuda", dtype)
    x, r, i = (wide[..., 1 + 67 * k:68 + 67 * k] for k in range(3))
    lam = -torch.rand(67, generator=g).cuda()
    want = gated_scan_fwd(x.contiguous(), r.contiguous(), i.contiguous(), lam)
    assert torch.equal(gated_scan_fwd(x, r, i, lam), want)
    state, other = torch.zeros(2, 67, device="cuda"), torch.zeros(2, 67, device="cuda")
    one = [t[:, 0] for t in (x, r, i)]
    got = gated_state_update(state, *one, lam)
    assert torch.equal(got, gated_state_update(other, *(t.contiguous() for t in one), lam))
    assert torch.equal(state, other)
