"""moe_add_rmsnorm on rows at the ends of binary32's range, against the formula in binary64.

Tolerance of y, relative to its own value: (51 / 2 + 2 + 3) * 2^-24, at most 31 * 2^-24, and one rounding to the output's type,
as tests/test_norm.py counts them. Beside it, absolutely: s / rms below 2^-126 is held in steps of 2^-149 before the
weight (product and remainder: a step), and so is a binary32 y; a bf16 y below 2^-126 has steps of 2^-133."""
import numpy as np
import pytest
import torch

import top_routing_expert_router_b200 as moe

pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
STEP = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
# every form: a row per warp, two warps, a block; streaming rows of a warp, 256 and 512 threads
SHAPES = [(2, 200), (9, 512), (300, 256), (300, 1024), (300, 2048), (300, 4096), (2, 7168), (300, 8192), (200, 16384), (150, 32768)]


def _powers(shape, lo, hi, g):
    """Values of either sign, their magnitudes spread evenly over 2^lo .. 2^hi."""
    v = torch.exp2(torch.empty(shape, dtype=torch.float64).uniform_(lo, hi, generator=g))
    return v * (1 - 2 * torch.randint(0, 2, shape, generator=g))


def _check(x, w, eps, y):
    s = x.double()
    eps = float(np.float32(eps))
    want = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    gain = w.double() if w is not None else torch.ones((), dtype=torch.float64, device="cuda")
    tol = ROUND[x.dtype]
    room = (31 * 2.0 ** -24 + tol) * (1 + tol) * (want * gain).abs() + 2 * 2.0 ** -149 * gain.abs() + STEP[x.dtype]
    assert ((y.double() - want * gain).abs() <= room).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_small_values_beside_huge_ones(dtype, rows, cols):
    """A row whose squares overflow still has its small values' digits: 2^-80 times them alone would not."""
    g = torch.Generator().manual_seed(rows + cols)
    x = _powers((rows, cols), -70, 30, g)
    x[:, 3] = _powers((rows,), 64.5, 127, g)
    x[0] = _powers((cols,), 120, 127, g)
    x = x.to(dtype).cuda()
    w = (1 + torch.randn(cols, generator=g)).to(dtype).cuda()
    for gain in (w, None):
        y = torch.full_like(x, float("nan"))
        moe.moe_add_rmsnorm(x, gain, 1e-6, y=y)
        _check(x, gain, 1e-6, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [1e34, 1e37, 3.4e38])
@pytest.mark.parametrize("rows,cols", [(2, 200), (9, 512), (300, 256), (300, 8192)])
def test_eps_beside_squares_that_overflow(dtype, eps, rows, cols):
    """eps counts however large: beside a sum of squares past binary32, and where its own sum with the mean is."""
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * 2.0 ** torch.linspace(40, 63.9, rows)[:, None]
    x = x.to(dtype).cuda()
    y = torch.full_like(x, float("nan"))
    moe.moe_add_rmsnorm(x, None, eps, y=y)
    _check(x, None, eps, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1e-36, 1e-29])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_tiny_eps_beside_squares_that_vanish(dtype, eps, rows, cols):
    """Rows of values whose squares are below binary32's range, of some within it, and of zeros."""
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * 2.0 ** torch.linspace(-90, -40, rows)[:, None]
    x[rows // 2] = 0
    w = (1 + torch.randn(cols, generator=g)).to(dtype).cuda()
    x = x.to(dtype).cuda()
    y = torch.full_like(x, float("nan"))
    moe.moe_add_rmsnorm(x, w, eps, y=y)
    _check(x, w, eps, y)
    assert (y[rows // 2] == 0).all()
