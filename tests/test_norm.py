"""Residual addition + root-mean-square norm + E4M3 output (moe_add_rmsnorm): refusals on the CPU, numerics on the
GPU against the formula in binary64 and the oracle's row quantiser.

Tolerance of y, relative to its own value. The sum of squares has only non-negative terms: 8 of a vector in a chain,
up to 4 vectors, 5 levels in a warp and up to 32 warps in a chain, 49 roundings of 2^-24 in all, and one for each
square's x + r taken twice: 51, halved by the root. The inverse root is rounded once, to within 2 * 2^-24 after its
Newton step; x + r and the two products add 3. So 31 * 2^-24, taken as 43, and one rounding to the output's type
(bf16: 2^-8, binary32: 2^-24)."""
import ctypes

import numpy as np
import pytest
import torch

import top_routing_expert_router_b200 as moe
from oracle import oracle as O
from tests import moe_harness as H

SUM_ERR = 43 * 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


# ---- refusals (no GPU needed) --------------------------------------------------------

A = 1 << 20  # stand-in addresses, never dereferenced
GOOD = dict(x=A, xs=256, r=2 * A, rs=256, w=3 * A, eps=1e-6, rows=4, cols=256, dtype=moe.MOE_BF16, s=4 * A, ss=256, y=5 * A,
            ys=256, q=6 * A, b=7 * A)


def _call(**kw):
    a = {**GOOD, **kw}
    return moe.lib_handle().moe_add_rmsnorm(a["x"], a["xs"], a["r"], a["rs"], a["w"], ctypes.c_float(a["eps"]), a["rows"], a["cols"],
                                            a["dtype"], a["s"], a["ss"], a["y"], a["ys"], a["q"], a["b"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), moe.MOE_ERR_INVALID_ARG),
    (dict(x=A + 2), moe.MOE_ERR_INVALID_ARG),                   # rows not on 16 bytes
    (dict(xs=248), moe.MOE_ERR_INVALID_ARG),                    # rows overlap
    (dict(xs=260), moe.MOE_ERR_INVALID_ARG),                    # second row off 16 bytes
    (dict(rs=0), moe.MOE_ERR_INVALID_ARG),
    (dict(ys=1 << 41), moe.MOE_ERR_INVALID_ARG),
    (dict(w=3 * A + 4), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=0.0), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (dict(rows=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(cols=0), moe.MOE_ERR_INVALID_ARG),
    (dict(cols=200), moe.MOE_ERR_INVALID_ARG),                  # codes need whole tiles
    (dict(cols=252, q=None, b=None), moe.MOE_ERR_UNSUPPORTED),
    (dict(cols=32768 + 128, xs=65536, rs=65536, ss=65536, ys=65536), moe.MOE_ERR_UNSUPPORTED),
    (dict(dtype=moe.MOE_FP8), moe.MOE_ERR_INVALID_ARG),
    (dict(b=None), moe.MOE_ERR_INVALID_ARG),                    # codes without scales
    (dict(y=None, q=None, b=None), moe.MOE_ERR_INVALID_ARG),    # nothing asked for
    (dict(y=4 * A), moe.MOE_ERR_INVALID_ARG),                   # y is sum_out
    (dict(s=A, ss=512), moe.MOE_ERR_INVALID_ARG),               # in place with another stride
])
def test_refusals(bad, code):
    assert _call(**bad) == code


def test_no_rows_is_a_no_op():
    assert _call(rows=0) == moe.MOE_OK
    assert _call(rows=0, x=None, y=None) == moe.MOE_OK


def test_binding_refuses_what_it_cannot_hand_over():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=x)                      # host tensors
    with pytest.raises(ValueError, match="like x"):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=x.float())
    with pytest.raises(ValueError, match="like x"):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=torch.zeros(256, 4, dtype=torch.bfloat16).T)
    with pytest.raises(ValueError, match="weight"):
        moe.moe_add_rmsnorm(x, w[:128], 1e-6, y=x)
    with pytest.raises(ValueError, match="codes"):
        moe.moe_add_rmsnorm(x, w, 1e-6, codes=torch.zeros(4, 256), scale_bytes=torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="x must"):
        moe.moe_add_rmsnorm(x.half(), w, 1e-6, y=x)


# ---- numerics ------------------------------------------------------------------------


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _strided(t, pad):
    big = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device="cuda")
    big[:, : t.shape[1]] = t
    return big, big[:, : t.shape[1]]


def _formula(x, r, w, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return s, y * w.double() if w is not None else y


def _check(x, r, w, eps, y=None, s=None):
    want_s, want_y = _formula(x, r, w, eps)
    tol = ROUND[x.dtype]
    if s is not None:
        assert ((s.double() - want_s).abs() <= (tol + 2.0 ** -24) * want_s.abs()).all()
    if y is not None:
        assert ((y.double() - want_y).abs() <= (SUM_ERR + tol) * (1 + tol) * want_y.abs() + 1e-40).all()


def _codes_of(y):
    """E4M3 codes and scale bytes of the rows of y, by the oracle (bf16) or the same rule in binary64 (binary32)."""
    if y.dtype == torch.bfloat16:
        return O.quantize_rows(H.to_np(y))
    t = y.cpu().double().unflatten(-1, (-1, 128))
    f, x = np.frexp(t.abs().amax(-1).numpy())
    e = torch.from_numpy(np.where(f == 0, 0, x - np.where(f <= 0.875, 9, 8)))
    q = (t * torch.exp2(-e.double())[..., None]).float().to(torch.float8_e4m3fn)  # exact: a power of two
    return q.flatten(-2).view(torch.uint8).numpy(), (e + 127).to(torch.uint8).numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 7168), (3, 200), (5, 264), (7, 512), (61, 5120), (149, 1160), (200, 128),
                                       (1000, 200), (2, 8192), (150, 8200), (3, 16392), (149, 32768), (2, 32768), (5000, 8),
                                       (3001, 256), (2000, 1280), (1500, 4224), (700, 8192), (900, 16384)])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, False)])
def test_matches_the_formula(dtype, rows, cols, residual, weight):
    x = _rand((rows, cols), dtype, 1)
    r = _rand((rows, cols), dtype, 2, 20.0) if residual else None
    w = _rand((cols,), dtype, 3) if weight else None
    y, s = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    codes = dict(codes=torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                 scale_bytes=torch.empty(rows, cols // 128, dtype=torch.uint8, device="cuda")) if cols % 128 == 0 else {}
    moe.moe_add_rmsnorm(x, w, 1e-5, y=y, residual=r, sum_out=s, **codes)
    _check(x, r, w, 1e-5, y, s)
    if codes:
        q, b = _codes_of(y)
        np.testing.assert_array_equal(codes["scale_bytes"].cpu().numpy(), b)
        np.testing.assert_array_equal(codes["codes"].cpu().numpy(), q)
        only = {k: torch.empty_like(v) for k, v in codes.items()}  # without y the codes are the same
        moe.moe_add_rmsnorm(x, w, 1e-5, residual=r, **only)
        assert all(torch.equal(only[k], codes[k]) for k in codes)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(37, 520), (1000, 104), (1000, 5000), (300, 1032)])
def test_strided_rows_and_untouched_padding(dtype, rows, cols):
    x, r = _rand((rows, cols), dtype, 4), _rand((rows, cols), dtype, 5)
    w = _rand((cols,), dtype, 6)
    (_, xv), (_, rv) = _strided(x, 24), _strided(r, 8)
    (yb, yv), (sb, sv) = _strided(torch.zeros_like(x), 16), _strided(torch.zeros_like(x), 40)
    moe.moe_add_rmsnorm(xv, w, 1e-6, y=yv, residual=rv, sum_out=sv)
    _check(x, r, w, 1e-6, yv, sv)
    assert (yb[:, cols:] == 7).all() and (sb[:, cols:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(3, 7168), (500, 1024), (1501, 256), (700, 7168), (400, 16384)])
def test_in_place(rows, cols):
    x, r = _rand((rows, cols), torch.bfloat16, 7), _rand((rows, cols), torch.bfloat16, 8)
    w = _rand((cols,), torch.bfloat16, 9)
    y, s = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, w, 1e-6, y=y, residual=r, sum_out=s)
    x2, r2 = x.clone(), r.clone()
    moe.moe_add_rmsnorm(x2, w, 1e-6, y=x2, residual=r2, sum_out=r2)  # the residual stream updated in place
    assert torch.equal(x2, y) and torch.equal(r2, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(2, 512), (9, 256), (9, 512), (300, 512), (300, 1024), (2, 7168), (300, 8192)])
def test_extreme_rows(dtype, rows, cols):
    """Zeros, values whose squares overflow or vanish in binary32, NaN and infinities: other rows keep their values."""
    x = _rand((rows, cols), dtype, 10)
    w = _rand((cols,), dtype, 11)
    y = torch.empty_like(x)
    x[0] = 0
    x[1] *= 2.0 ** 100
    moe.moe_add_rmsnorm(x, w, 1e-6, y=y)
    assert (y[0] == 0).all()
    _check(x, None, w, 1e-6, y)
    if rows < 5:
        return
    x[2] *= 2.0 ** -90
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    x[rows - 1, 0] = 3e38
    moe.moe_add_rmsnorm(x, w, 1e-6, y=y)
    assert y[3].isnan().all()
    assert y[4, 7].isnan() and (y[4, :7] == 0).all() and (y[4, 8:] == 0).all()
    fine = [i for i in range(rows) if i not in (3, 4)]
    _check(x[fine], None, w, 1e-6, y[fine])


@pytest.mark.gpu
def test_runs_in_a_graph_and_on_another_stream():
    x, r = _rand((16, 2048), torch.bfloat16, 12), _rand((16, 2048), torch.bfloat16, 13)
    w = _rand((2048,), torch.bfloat16, 14)
    y, s = torch.zeros_like(x), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=y, residual=r, sum_out=s)
    side.synchronize()
    _check(x, r, w, 1e-6, y, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=y, residual=r, sum_out=s)
    x.copy_(_rand((16, 2048), torch.bfloat16, 15))
    graph.replay()
    torch.cuda.synchronize()
    _check(x, r, w, 1e-6, y, s)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 7168), (300, 1024), (2000, 256), (400, 7168)])
def test_calls_at_once_and_outputs_left_out(rows, cols):
    x, r = _rand((rows, cols), torch.bfloat16, 16), _rand((rows, cols), torch.bfloat16, 17)
    w = _rand((cols,), torch.bfloat16, 18)
    y, s = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, w, 1e-6, y=y, residual=r, sum_out=s)
    outs = [torch.empty_like(x) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, t in zip(outs, streams):
            with torch.cuda.stream(t):
                moe.moe_add_rmsnorm(x, w, 1e-6, y=o, residual=r)  # no sum_out
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)
    z = x.clone()
    moe.moe_add_rmsnorm(z, w, 1e-6, y=outs[0], residual=z, sum_out=outs[1])  # the same rows twice: s = 2 x
    _check(z, z, w, 1e-6, outs[0], outs[1])
