"""The two-launch layer for few tokens (moe_layer_decode): refusals on the CPU; on the GPU every dtype and scoring
against the fp64 oracle, and the calls the documentation allows.

Tolerances of y are the layer parity tests' (2e-2 for bf16 and FP8, 1e-4 for binary32, relative to the larger of the
element and its row's rms). In bf16 the error is that of h and of y, each rounded by at most 2^-8 of itself: over a
row of sums that is a standard deviation of 2^-8 / sqrt(3) = 0.0023 of the rms from h, the largest of 64 x 512 such
values lying near 4.3 of them (0.0097), plus 2^-8 (0.0039) from y: 0.0136. (That is with h in one bf16 row, as in
FP8's tiles; bf16 experts keep 16 bits of it, which leaves y's part.) In binary32 the same with 2^-24 per
rounding, of which a sum of 7168 terms takes at most 7168 in a chain: 4.3e-4 at worst, about sqrt(7168) * 2^-24 =
5e-6 as roundings go; the largest sum below has 1032 terms (6.2e-5 at worst). Gates are sums in binary64 rounded once
to binary32: 2^-24, and 2^-22 allows for the two exponentials' own errors."""
import ctypes

import numpy as np
import pytest
import torch

import top_routing_expert_router_b200 as moe
from oracle import oracle as O
from synth import workloads as W
from tests import moe_harness as H

MATS = ("gate", "up", "down")


# ---- refusals (no GPU needed) --------------------------------------------------------


def _cfg(**kw):
    base = dict(d_model=512, n_routed=32, top_k=4, moe_intermediate_size=256, n_shared=1)
    return moe.make_config(**{**base, **kw})


def _call(cfg, n, x=256, xc=None, xs=None, w=None, y=256, idx=None, tw=None, counts=None, diag=None, ws=256, need=None):
    w = w or moe.moe_weights(*([256] * 14))
    need = moe.moe_workspace_size(cfg, max(n, 0)) if need is None else need
    return moe.lib_handle().moe_layer_decode(ctypes.byref(cfg), n, x, xc, xs, ctypes.byref(w), y, idx, tw, counts, diag, ws,
                                             need, None)


def test_refusals():
    bf, f8 = _cfg(), _cfg(dtype="fp8")
    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert _call(bf, 65) == un                                                      # more tokens than the form takes
    assert _call(_cfg(cap_policy="drop", capacity_factor=1.0), 4) == un
    assert _call(_cfg(top_k=33, n_routed=64), 4, need=1 << 30) == un
    assert _call(_cfg(moe_intermediate_size=1 << 27), 4, need=1 << 62) == un        # rows past 31 bits
    assert _call(_cfg(moe_intermediate_size=1 << 24, n_shared=128), 4, need=1 << 62) == un
    assert _call(bf, -1) == bad
    assert _call(bf, 4, x=None) == bad and _call(bf, 4, x=264) == bad
    assert _call(bf, 4, y=None) == bad and _call(bf, 4, y=260) == bad
    assert _call(bf, 4, idx=260) == bad and _call(bf, 4, tw=260) == bad
    assert _call(bf, 4, counts=258) == bad and _call(bf, 4, diag=260) == bad
    assert _call(bf, 4, ws=None) == bad and _call(bf, 4, ws=128) == bad
    assert _call(bf, 4, need=moe.moe_workspace_size(bf, 4) - 1) == moe.MOE_ERR_WORKSPACE
    assert _call(bf, 4, xc=256, xs=256) == bad                                      # codes without FP8 experts
    assert _call(f8, 4, xc=256) == bad and _call(f8, 4, xs=256) == bad              # one without the other
    assert _call(f8, 4, xc=264, xs=256) == bad
    no = moe.moe_weights(*([256] * 14))
    no.w_up = None
    assert _call(bf, 4, w=no) == bad
    no = moe.moe_weights(*([256] * 14))
    no.ws_down_scale = None
    assert _call(bf, 4, w=no, need=0) == moe.MOE_ERR_WORKSPACE and _call(f8, 4, w=no) == bad


@pytest.mark.parametrize("name", ["tiny_f32", "mixtral_small", "mixtral_8x7b", "deepseek_v3_small", "deepseek_v3_prefill",
                                  "deepseek_v3_decode_small_fp8", "deepseek_v3_decode_fp8_32e", "ragged_small"])
def test_one_workspace_serves_fewer_tokens_too(name):
    """A workspace is sized for the largest batch; every call of up to 64 tokens takes it."""
    cfg = H.cfg_for(W.get(name))
    size = [moe.moe_workspace_size(cfg, n) for n in [*range(1, 81), 100, 127, 128, 129, 200, 257, 500]]
    assert size[:64] == sorted(size[:64]) and min(size[64:]) >= size[63]
    for n in (1, 2, 7, 33, 64):  # (the refusal is of x, a null pointer)
        assert _call(cfg, n, x=None, need=size[79]) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (40, 32), (250, 5), (256, 8), (256, 1)])
def test_workspace_grows_with_the_tokens_for_every_shape(E, k):
    for d in (8, 136, 1032, 4096, 7168):
        for I in (8, 128, 1000, 2048, 14336):
            for shared in (0, 1, 3):
                for dtype in ("f32", "bf16", "fp8"):
                    if dtype == "fp8" and (d % 128 or I % 128 or I > 8192):
                        continue
                    cfg = moe.make_config(d_model=d, n_routed=E, top_k=k, moe_intermediate_size=I, n_shared=shared, dtype=dtype)
                    size = [moe.moe_workspace_size(cfg, n) for n in range(1, 67)]
                    assert size == sorted(size), (d, I, shared, dtype)


def test_binding_refuses_what_it_cannot_hand_over():
    cfg = _cfg()
    t = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_layer_decode(cfg, 4, t, moe.moe_weights(), t, torch.zeros(16, dtype=torch.uint8))


# ---- numerics ------------------------------------------------------------------------


def _weights(dev):
    if "w_gate_q" not in dev:
        return H.weights_for(dev)
    names = MATS + tuple("ws_" + k for k in MATS if "ws_gate_q" in dev)
    scales = {k: dev[("%s_s" if k.startswith("ws_") else "w_%s_s") % k] for k in names}
    return moe.make_weights(dev["w_r"], dev["w_gate_q"], dev["w_up_q"], dev["w_down_q"], dev.get("ws_gate_q"),
                            dev.get("ws_up_q"), dev.get("ws_down_q"), dev.get("bias"), scales=scales)


def _oracle(w, host):
    if w.dtype != "fp8":
        return O.layer(H.oracle_cfg(w), host["x"], host["w_r"], host["w_gate"], host["w_up"], host["w_down"],
                       host.get("bias"), host.get("ws_gate"), host.get("ws_up"), host.get("ws_down"))
    w8 = {k: (host["w_%s_q" % k], host["w_%s_s" % k]) for k in MATS}
    ws8 = {k: (host["ws_%s_q" % k], host["ws_%s_s" % k]) for k in MATS} if "ws_gate_q" in host else None
    return O.layer_fp8(H.oracle_cfg(w), host["x"], host["w_r"], host.get("bias"), w8, ws8)


class Call:
    """One workload's buffers; every output row past n and the workspace start as garbage."""

    def __init__(self, w, dev):
        self.w, self.dev, self.cfg, self.weights = w, dev, H.cfg_for(w), _weights(dev)
        self.ws = torch.full((moe.moe_workspace_size(self.cfg, w.n),), 0xFF, dtype=torch.uint8, device="cuda")
        self.y = torch.full((w.n + 3, w.d_model), 7.0, dtype=dev["x"].dtype, device="cuda")
        self.idx = torch.full((w.n + 3, w.top_k), -9, dtype=torch.int32, device="cuda")
        self.tw = torch.full((w.n + 3, w.top_k), -9.0, dtype=torch.float32, device="cuda")
        self.counts = torch.full((w.n_routed,), -9, dtype=torch.int32, device="cuda")
        self.diag = torch.full((8,), -9, dtype=torch.int32, device="cuda")

    def __call__(self, x=None, **kw):
        moe.moe_layer_decode(self.cfg, self.w.n, self.dev["x"] if x is None else x, self.weights, self.y, self.ws, self.idx,
                             self.tw, self.counts, self.diag, **kw)
        return self

    def check(self, r):
        n = self.w.n
        assert moe.moe_sync_status(self.ws) == moe.MOE_OK
        keep = ~r["exempt"]
        idx, tw, y = self.idx.cpu().numpy(), self.tw.cpu().numpy(), H.as_f64(self.y)
        np.testing.assert_array_equal(idx[:n][keep], r["topk_idx"][keep])
        np.testing.assert_allclose(tw[:n][keep], r["topk_w"][keep], rtol=2.0 ** -22, atol=0)
        assert H.rel_err(y[:n][keep], r["y"][keep]) <= H.TOL["f32" if self.w.dtype == "f32" else "bf16"]
        assert (idx[n:] == -9).all() and (tw[n:] == -9).all() and (y[n:] == 7).all()
        counts = np.bincount(idx[:n].ravel(), minlength=self.w.n_routed)
        np.testing.assert_array_equal(self.counts.cpu().numpy(), counts)
        assert self.diag.cpu().tolist() == [0, 0, 0, counts.max(), 0, -9, -9, -9]  # status and the rest are not touched


CASES = [("tiny_f32", n) for n in (1, 3, 64)] + [("mixtral_small", n) for n in (1, 2, 64)]
CASES += [("deepseek_v2_small", n) for n in (1, 17, 64)] + [("deepseek_v3_small", n) for n in (1, 5, 16, 33, 64)]
CASES += [("deepseek_v3_decode_small", n) for n in (1, 40)] + [("ragged_small", n) for n in (1, 7, 63)]
CASES += [("deepseek_v4_small", n) for n in (2, 64)] + [("tie_softmax", 64), ("tie_sigmoid", 64)]
CASES += [("fp8_ragged_small", n) for n in (1, 7, 64)] + [("deepseek_v3_decode_small_fp8", n) for n in (1, 16, 40)]
CASES += [("fp8_skewed_small", n) for n in (9, 64)]


def _get(name, n, **kw):
    w = W.get(name, n=n, **kw)
    return w, W.host_inputs(w), W.device_inputs(w)


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", CASES)
def test_layer_parity(name, n):
    w, host, dev = _get(name, n)
    Call(w, dev)().check(_oracle(w, host))


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("deepseek_v3_small", 16), ("deepseek_v3_small", 64), ("ragged_small", 7), ("mixtral_small", 33)])
def test_bf16_carries_one_rounding(name, n):
    """y is off by its own rounding (2^-8 of itself) and by h's 16 bits: 2^-16 of each term. Of 512 normal terms the
    magnitudes sum to 0.64 * 512 / sqrt(512) = 14.4 times the sum's rms, so 14.4 * 2^-16 = 2.2e-4 of it at worst; 2^-11
    (4.9e-4) leaves the binary32 sums (512 * 2^-24 = 3.1e-5 of the magnitudes' 14.4: 4.4e-4 if every one erred its way,
    2e-5 as roundings go) their part."""
    w, host, dev = _get(name, n)
    r, c = _oracle(w, host), Call(w, dev)()
    keep = ~r["exempt"]
    y, want = H.as_f64(c.y)[:n][keep], r["y"][keep]
    rms = np.sqrt(np.mean(want * want, axis=1, keepdims=True))
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * rms).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(n=6, d_model=8, n_routed=1, top_k=1, moe_intermediate_size=8, n_shared=0),     # one expert, the smallest matrices
    dict(n=5, d_model=24, n_routed=3, top_k=3, moe_intermediate_size=1000, n_shared=3),
    dict(n=64, d_model=1032, n_routed=33, top_k=32, moe_intermediate_size=136, n_shared=0),
    dict(n=2, d_model=136, n_routed=250, top_k=5, moe_intermediate_size=328, n_shared=2),
])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_odd_shapes(kw, dtype):
    w, host, dev = _get("ragged_small", dtype=dtype, **kw)
    Call(w, dev)().check(_oracle(w, host))


@pytest.mark.gpu
@pytest.mark.parametrize("name,kw", [
    ("ragged_small", dict(n=3, d_model=2568, n_routed=2, top_k=2, moe_intermediate_size=9608, n_shared=0)),
    ("fp8_ragged_small", dict(n=1, d_model=5120, n_routed=5, top_k=5, moe_intermediate_size=3840, n_shared=1)),
])
def test_long_tiles_in_halves(name, kw):
    """A little over one turn of the SMs, with long k axes: gate/up tiles in two parts, down tiles in several."""
    w, host, dev = _get(name, **kw)
    Call(w, dev)().check(_oracle(w, host))


@pytest.mark.gpu
@pytest.mark.parametrize("groups,kept,experts", [(2, 1, 6), (16, 3, 64), (3, 2, 201)])
def test_group_limits_off_32(groups, kept, experts):
    w, host, dev = _get("deepseek_v3_small", 19, n_group=groups, topk_group=kept, n_routed=experts, top_k=3)
    Call(w, dev)().check(_oracle(w, host))


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("tiny_f32", 9), ("deepseek_v3_small", 64), ("deepseek_v3_decode_small_fp8", 33)])
def test_same_results_every_time_and_same_routing_as_the_layer(name, n):
    w, _, dev = _get(name, n)
    a, b = Call(w, dev)(), Call(w, dev)()
    for _ in range(20):
        b()
    assert torch.equal(a.y, b.y) and torch.equal(a.idx, b.idx) and torch.equal(a.tw, b.tw)
    idx = torch.empty(n, w.top_k, dtype=torch.int32, device="cuda")
    y = torch.empty(n, w.d_model, dtype=dev["x"].dtype, device="cuda")
    moe.moe_layer_forward(a.cfg, n, dev["x"], a.weights, y, a.ws, topk_idx=idx)
    assert torch.equal(idx, a.idx[:n])
    assert H.rel_err(H.as_f64(a.y)[:n], H.as_f64(y)) <= 2 * H.TOL["f32" if w.dtype == "f32" else "bf16"]


@pytest.mark.gpu
def test_optional_outputs_left_out():
    w, _, dev = _get("deepseek_v3_small", 12)
    a, b = Call(w, dev)(), Call(w, dev)
    moe.moe_layer_decode(b.cfg, w.n, dev["x"], b.weights, b.y, b.ws)
    assert torch.equal(a.y, b.y)


@pytest.mark.gpu
def test_workspace_of_a_larger_batch():
    w, host, dev = _get("deepseek_v3_small", 5)
    c = Call(w, dev)
    c.ws = torch.full((moe.moe_workspace_size(c.cfg, 200),), 0xFF, dtype=torch.uint8, device="cuda")
    c().check(_oracle(w, host))


@pytest.mark.gpu
def test_no_tokens():
    w, _, dev = _get("ragged_small", 1)
    c = Call(w, dev)
    empty = torch.empty(0, w.d_model, dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_decode(c.cfg, 0, empty, c.weights, empty, c.ws, counts=c.counts, diag=c.diag)
    assert moe.moe_sync_status(c.ws) == moe.MOE_OK
    assert (c.counts == 0).all() and c.diag.cpu().tolist() == [0] * 5 + [-9] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["tiny_f32", "deepseek_v3_small", "deepseek_v3_decode_small_fp8"])
def test_nan_and_infinite_tokens_leave_the_others_alone(name):
    w, _, dev = _get(name, 20)
    a = Call(w, dev)()
    x = dev["x"].clone()
    x[3, 5] = float("nan")
    x[11] = float("inf")
    x[19, 0] = float("-inf")
    b = Call(w, dev)(x)
    assert moe.moe_sync_status(b.ws) == moe.MOE_OK
    fine = [t for t in range(20) if t not in (3, 11, 19)]
    assert torch.equal(a.y[fine], b.y[fine]) and torch.equal(a.idx[fine], b.idx[fine])
    got = b.idx[:20].cpu()
    assert ((got >= 0) & (got < w.n_routed)).all()
    assert b.y[3].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("deepseek_v3_small", 8), ("deepseek_v3_decode_small_fp8", 24)])
def test_graph_replay_sees_new_inputs(name, n):
    w, host, dev = _get(name, n)
    c = Call(w, dev)
    c()
    torch.cuda.synchronize()
    x = dev["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c(x)
    host2 = dict(host, x=W.host_inputs(w, seed=3, names=["x"])["x"])
    x.copy_(W.device_inputs(w, seed=3, names=["x"])["x"])
    for _ in range(3):
        graph.replay()
    c.check(_oracle(w, host2))


@pytest.mark.gpu
def test_overlapping_calls_on_streams():
    """Calls on several streams, each with its own workspace: none waits for blocks that the others keep out."""
    w, _, dev = _get("deepseek_v3_decode_small", 33)
    want = Call(w, dev)()
    calls = [Call(w, dev) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(25):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c()
    torch.cuda.synchronize()
    for c in calls:
        assert moe.moe_sync_status(c.ws) == moe.MOE_OK
        assert torch.equal(c.y, want.y) and torch.equal(c.idx, want.idx)


@pytest.mark.gpu
def test_workspace_shared_with_other_entry_points_in_turn():
    w, host, dev = _get("deepseek_v3_decode_small_fp8", 40)
    c = Call(w, dev)
    y = torch.empty(w.n, w.d_model, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        moe.moe_layer_forward(c.cfg, w.n, dev["x"], c.weights, y, c.ws)
        c()
    c.check(_oracle(w, host))


@pytest.mark.gpu
def test_calls_of_every_kind_at_once():
    """Both kernels' forms and the large-batch layer overlap on streams, each call with its own workspace."""
    kinds = [_get("tiny_f32", 40), _get("deepseek_v3_small", 64), _get("deepseek_v3_decode_small_fp8", 33), _get("mixtral_small", 1)]
    want = [Call(w, dev)() for w, _, dev in kinds]
    calls = [Call(w, dev) for w, _, dev in kinds]
    big, _, bdev = _get("deepseek_v3_decode_small", 128)
    bcfg, bw = H.cfg_for(big), _weights(bdev)
    bws = torch.empty(moe.moe_workspace_size(bcfg, big.n), dtype=torch.uint8, device="cuda")
    y0, y1 = (torch.empty(big.n, big.d_model, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_layer_forward(bcfg, big.n, bdev["x"], bw, y0, bws)
    streams = [torch.cuda.Stream() for _ in range(len(calls) + 1)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c()
        with torch.cuda.stream(streams[-1]):
            moe.moe_layer_forward(bcfg, big.n, bdev["x"], bw, y1, bws)
    torch.cuda.synchronize()
    for c, r in zip(calls, want):
        assert moe.moe_sync_status(c.ws) == moe.MOE_OK
        assert torch.equal(c.y, r.y) and torch.equal(c.idx, r.idx) and torch.equal(c.tw, r.tw)
    assert torch.equal(y0, y1)


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("tiny_f32", 6), ("deepseek_v3_small", 2), ("deepseek_v3_decode_small_fp8", 24)])
def test_captured_behind_a_copy_and_a_join(name, n):
    """Inside a graph the call follows a copy (no kernel) on its own stream and a norm on another one."""
    w, host, dev = _get(name, n)
    c = Call(w, dev)
    x, src, stale = dev["x"].clone(), dev["x"].clone(), torch.empty_like(dev["x"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(src)
        c(x)
        x.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            moe.moe_add_rmsnorm(src, None, 1e-6, y=stale)
            x.copy_(src)
        torch.cuda.current_stream().wait_stream(side)
        c(x)
    src.copy_(W.device_inputs(w, seed=3, names=["x"])["x"])
    for _ in range(3):
        x.fill_(1.0)
        graph.replay()
    c.check(_oracle(w, dict(host, x=W.host_inputs(w, seed=3, names=["x"])["x"])))


@pytest.mark.gpu
def test_two_graphs_take_turns_on_one_workspace():
    w, host, dev = _get("deepseek_v3_small", 48)
    w1, host1, dev1 = _get("deepseek_v3_small", 2)
    a, b = Call(w, dev), Call(w1, dev1)
    b.ws = a.ws
    graphs = []
    for c in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
    for _ in range(4):
        for g in graphs:
            g.replay()
    a.check(_oracle(w, host))
    b.check(_oracle(w1, host1))


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("tiny_f32", 2), ("tiny_f32", 64), ("deepseek_v3_small", 1), ("deepseek_v3_small", 64),
                                    ("deepseek_v3_decode_small_fp8", 40)])
def test_y_in_the_place_of_x(name, n):
    w, _, dev = _get(name, n)
    a = Call(w, dev)()
    for _ in range(5):
        x = dev["x"].clone()
        moe.moe_layer_decode(a.cfg, n, x, a.weights, x, a.ws)
        assert torch.equal(x, a.y[:n])


@pytest.mark.gpu
def test_most_slots_with_given_codes():
    w, host, dev = _get("fp8_ragged_small", 64, n_routed=40, top_k=32)
    codes = torch.empty(64, w.d_model, dtype=torch.uint8, device="cuda")
    sb = torch.empty(64, w.d_model // 128, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_fp8(dev["x"], codes, sb)
    Call(w, dev)(x_codes=codes, x_scale_bytes=sb).check(_oracle(w, host))


# ---- the step as it is used: residual add and norm, then the layer ---------------------


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("deepseek_v3_small", 3), ("deepseek_v3_decode_small_fp8", 1),
                                    ("deepseek_v3_decode_small_fp8", 40), ("fp8_ragged_small", 17)])
def test_norm_then_layer(name, n):
    w, host, dev = _get(name, n)
    c = Call(w, dev)
    g = torch.Generator(device="cuda").manual_seed(5)
    attn = torch.randn(n, w.d_model, device="cuda", generator=g).bfloat16()
    stream = (3 * torch.randn(n, w.d_model, device="cuda", generator=g)).bfloat16()
    gain = (1 + 0.1 * torch.randn(w.d_model, device="cuda", generator=g)).bfloat16()
    s = attn.double() + stream.double()
    x = torch.empty_like(attn)
    codes = torch.empty(n, w.d_model, dtype=torch.uint8, device="cuda") if w.dtype == "fp8" else None
    sb = torch.empty(n, w.d_model // 128, dtype=torch.uint8, device="cuda") if w.dtype == "fp8" else None
    moe.moe_add_rmsnorm(attn, gain, 1e-6, y=x, residual=stream, sum_out=stream, codes=codes, scale_bytes=sb)
    kw = dict(x_codes=codes, x_scale_bytes=sb) if codes is not None else {}
    c(x, **kw).check(_oracle(w, dict(host, x=H.to_np(x))))
    want = s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-6) * gain.double()
    assert ((x.double() - want).abs() <= 2.0 ** -7.9 * want.abs()).all()
    assert ((stream.double() - s).abs() <= 2.0 ** -7.99 * s.abs()).all()
    if codes is not None:  # the call's own quantisation of x gives the same bits
        d = Call(w, dev)(x)
        assert torch.equal(c.y, d.y)
