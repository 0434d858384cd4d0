"""A run of an order's experts on the GPU: their matrices with that run of the offsets, which
then does not begin at 0.  Its rows are those of the call for all experts, the others are left
as they are.

Operands are whole numbers of -2 .. 2: every sum is below 2^24 in float32 whatever the order,
so that the two calls agree to the bit with any tile and any parts.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# (tile, one launch of the gradient, parts); None: by the sizes
PLANS = [(None, None, None), (0, None, None), (1, 0, 3), (1, 1, 3), (2, 0, 2), (2, 1, None), (3, 0, None)]


def whole(*shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g).to("cuda", dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("counts,a,b", [([40, 3, 0, 130, 65, 9], 1, 4), ([40, 3, 0, 130, 65, 9], 3, 6),
                                        ([5] * 70, 33, 66), ([1, 0, 2, 4], 2, 4)],
                         ids=["1 to 3 of 6", "3 to 5 of 6", "33 to 65 of 70", "2 and 3 of 4"])
def test_run(counts, a, b, plan, dtype, monkeypatch):
    from selective_state_space_38_amd import expert_linear_bwd, expert_linear_fwd
    for name, v in zip(("SHAPE", "PAIR", "PARTS"), plan):
        if v is not None:
            monkeypatch.setenv(f"SSM_FORCE_PRODUCT_{name}", str(v))
    n, k = 75, 392
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    offsets, rows = torch.from_numpy(ends).cuda(), int(ends[-1]) + 7
    g = torch.Generator().manual_seed(9)
    token = torch.randint(0, 50, (rows,), generator=g, dtype=torch.int32).cuda()
    x, w = whole(50, k, dtype=dtype, seed=0), whole(len(counts), n, k, dtype=dtype, seed=1)
    bias, dout = whole(len(counts), n, dtype=torch.float32, seed=2), whole(rows, n, dtype=dtype, seed=3)
    part = offsets[a:b + 1].clone()
    here = slice(int(ends[a]), int(ends[b]))
    for act in (None, "silu"):
        whole_out, pre = expert_linear_fwd(x, w, offsets, token=token, bias=bias, activation=act, return_pre=True)
        kept = whole(rows, n, dtype=dtype, seed=4) + 100
        out = expert_linear_fwd(x, w[a:b].contiguous(), part, token=token, bias=bias[a:b].clone(),
                                activation=act, out=kept.clone())
        want = kept.clone()
        want[here] = whole_out[here]
        assert torch.equal(out, want)
    want = expert_linear_bwd(dout, x, w, offsets, token=token, bias=True)
    kept = whole(rows, k, dtype=dtype, seed=5) + 100
    got = expert_linear_bwd(dout, x, w[a:b].contiguous(), part, token=token, bias=True, dx=kept.clone())
    kept[here] = want["dx"][here]
    assert torch.equal(got["dx"], kept)
    assert torch.equal(got["dw"], want["dw"][a:b]) and torch.equal(got["dbias"], want["dbias"][a:b])
