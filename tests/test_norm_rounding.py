"""What moe_add_rmsnorm rounds: on rows of small integers, whose sum of squares is exact in binary32, everything up to the
last rounding of y to binary32 is compensated, so y is the formula's value rounded once to binary32, and then to bf16.

How many values may differ from that. The inverse root's Newton step leaves 3/8 of its start's error (2^-22) squared, and
the remainders carried along are rounded at 2^-24 of themselves: less than 2^-42 of y in all, so a value is rounded the
other way where it lies that near to a border of binary32 (steps of at least 2^-24): 2 * 2^-42 / 2^-24 = 2^-17 of them;
2^-14 is allowed. (Three rounded products instead give another binary32 value for 29 % of them.) Of bf16 values those
within half a binary32 step of a border between two (2^-25 to each side, of steps of at least 2^-8) go through the
border itself and half of them the wrong way: 2^-17; 2^-14 is allowed."""
import numpy as np
import pytest
import torch

import top_routing_expert_router_b200 as moe
from tests.test_norm_extremes import SHAPES

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -10


def _rounded(v, dtype):
    """v (binary64) rounded once to dtype, ties to even."""
    if dtype == torch.float32:
        return v.float().double()
    m, e = np.frexp(v.cpu().numpy())
    return torch.from_numpy(np.ldexp(np.round(m * 256) / 256, e)).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_values_are_rounded_once(dtype, rows, cols, residual):
    g = torch.Generator().manual_seed(cols)
    s = torch.randint(-15, 16, (rows, cols), generator=g).to(dtype).cuda()
    r = torch.randint(-100, 101, (rows, cols), generator=g).to(dtype).cuda() if residual else None
    x = s - r if residual else s  # exact: integers below 2^7
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(dtype).cuda()
    y = torch.empty_like(x)
    moe.moe_add_rmsnorm(x, w, EPS, y=y, residual=r)
    v = s.double()
    want = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * w.double()
    assert int((y.double() != _rounded(want, dtype)).sum()) <= 3 + rows * cols * 2.0 ** -14
    y = torch.empty_like(x)
    moe.moe_add_rmsnorm(x, None, EPS, y=y, residual=r)
    want = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
    # without a weight all values of one integer are alike in a row: a row's root within 2^-42 of a border would turn
    # them together, so rows with any difference are counted
    assert int((y.double() != _rounded(want, dtype)).any(-1).sum()) <= 3 + rows * 30 * 2.0 ** -14
