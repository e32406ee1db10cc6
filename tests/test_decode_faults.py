"""moe_layer_decode where it can go wrong: hand-overs between threads, waits that run out, workspaces, types."""
import pathlib
import re

import pytest
import torch

import top_routing_expert_router_b200 as moe
from synth import workloads as W
from tests import moe_harness as H
from tests.test_decode import Call

CSRC = pathlib.Path(moe.__file__).parent / "csrc"


# ---- hand-overs --------------------------------------------------------------------


def test_scale_bytes_are_read_behind_a_warp_barrier():
    """In the token warp lane 0 alone acquires the count of an expert's finished tiles; the other lanes read that expert's
    scale bytes. What orders their reads behind the acquire is a __syncwarp() (a shuffle does not), and no run shows its
    absence reliably: so the text is looked at."""
    text = (CSRC / "decode_tc.cu").read_text()
    acquire = text.index("wait_counter(a.ctr + kCtrExpert + tl.e")
    first_read = text.index("fetch(tl.kb0)", acquire)
    assert re.search(r"if \(!all\(ok\)\) break;\s*__syncwarp\(\);", text[acquire:first_read])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 24, 40])
def test_scale_bytes_of_an_earlier_call_are_not_seen(n):
    """Calls take turns on one workspace with tokens 2^12 apart, so that every scale byte of x and h changes each time."""
    w = W.get("deepseek_v3_decode_small_fp8", n=n)
    dev = W.device_inputs(w)
    loud = dev["x"] * 2.0 ** 12
    want = [Call(w, dev)(x).y for x in (dev["x"], loud)]
    c = Call(w, dev)
    for i in range(60):
        c(loud if i % 2 else dev["x"])
        assert torch.equal(c.y, want[i % 2])
    assert moe.moe_sync_status(c.ws) == moe.MOE_OK


# ---- types -------------------------------------------------------------------------


def _tensors(dtype, **kw):
    cfg = moe.make_config(d_model=512, n_routed=32, top_k=4, moe_intermediate_size=256, dtype=dtype)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    t = dict(x=torch.zeros(4, 512, dtype=act), y=torch.zeros(4, 512, dtype=act), topk_idx=torch.zeros(4, 4, dtype=torch.int32),
             topk_w=torch.zeros(4, 4), counts=torch.zeros(32, dtype=torch.int32), diag=torch.zeros(8, dtype=torch.int32))
    if dtype == "fp8":
        t.update(x_codes=torch.zeros(4, 512, dtype=torch.uint8), x_scale_bytes=torch.zeros(4, 4, dtype=torch.uint8))
    return cfg, {**t, **kw}


def _refusal(dtype, **kw):
    """What the binding says to host tensors, which it refuses at last for that."""
    cfg, t = _tensors(dtype, **kw)
    with pytest.raises(ValueError) as e:
        moe.moe_layer_decode(cfg, 4, t.pop("x"), moe.moe_weights(), t.pop("y"), torch.zeros(16, dtype=torch.uint8), **t)
    return str(e.value)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_binding_refuses_other_types(dtype):
    assert "CUDA" in _refusal(dtype)
    wrong = torch.bfloat16 if dtype == "f32" else torch.float32
    for name, t in [("x", torch.zeros(8, 512, dtype=wrong)), ("x", torch.zeros(8, 512, dtype=torch.float16)),
                    ("y", torch.zeros(8, 512, dtype=wrong)), ("topk_idx", torch.zeros(4, 4, dtype=torch.int64)),
                    ("topk_idx", torch.zeros(4, 4)), ("topk_w", torch.zeros(4, 4, dtype=torch.float64)),
                    ("counts", torch.zeros(32, dtype=torch.int64)), ("diag", torch.zeros(8, dtype=torch.int64))]:
        assert f"{name} is {t.dtype}" in _refusal(dtype, **{name: t})
    if dtype == "fp8":
        for name, kind in (("x_codes", torch.float8_e4m3fn), ("x_scale_bytes", torch.float8_e8m0fnu)):
            _, t = _tensors(dtype)
            assert "CUDA" in _refusal(dtype, **{name: t[name].view(kind)})
            assert f"{name} is" in _refusal(dtype, **{name: t[name].to(torch.int32)})
            assert f"{name} is" in _refusal(dtype, **{name: t[name].view(torch.float8_e5m2)})


def test_binding_refuses_what_is_too_small_or_strided():
    assert "y has" in _refusal("bf16", y=torch.zeros(3, 512, dtype=torch.bfloat16))
    assert "x has" in _refusal("bf16", x=torch.zeros(512, 4, dtype=torch.bfloat16).T)
    assert "topk_w has" in _refusal("f32", topk_w=torch.zeros(4, 3))


# ---- waits that run out ------------------------------------------------------------


BIG = dict(d_model=4096, n_routed=16, top_k=4, moe_intermediate_size=2048)


@pytest.mark.gpu
@pytest.mark.parametrize("stall", ["1", "2"])
@pytest.mark.parametrize("name,n,kw", [
    ("tiny_f32", 5, {}), ("tiny_f32", 64, dict(d_model=1024, moe_intermediate_size=1024)),
    ("ragged_small", 7, {}), ("ragged_small", 3, BIG), ("ragged_small", 64, BIG),
    ("fp8_ragged_small", 7, {}), ("fp8_ragged_small", 3, BIG), ("fp8_ragged_small", 40, BIG),
])
def test_abandoned_call_leaves_the_gpu_as_it_was(name, n, kw, stall, monkeypatch):
    """An expert's hidden rows are never reported finished (2: a token never decided): the waits for them end at their
    limit, the call leaves MOE_ERR_TIMEOUT, and neither the call right behind it nor the next one on its workspace
    sees anything of it."""
    w = W.get(name, n=n, **kw)
    dev = W.device_inputs(w)
    want, bad, good = Call(w, dev)(), Call(w, dev), Call(w, dev)
    torch.cuda.synchronize()
    for _ in range(5):
        monkeypatch.setenv("MOE_TEST_STALL", stall)
        bad()
        monkeypatch.delenv("MOE_TEST_STALL")
        good()
        assert moe.moe_sync_status(bad.ws) == moe.MOE_ERR_TIMEOUT
        assert moe.moe_sync_status(bad.ws) == moe.MOE_OK  # reading clears the word
        assert moe.moe_sync_status(good.ws) == moe.MOE_OK
        assert torch.equal(good.y, want.y) and torch.equal(good.idx, want.idx)
        assert (bad.y[n:] == 7).all()
        bad()
        assert moe.moe_sync_status(bad.ws) == moe.MOE_OK
        assert torch.equal(bad.y, want.y) and torch.equal(bad.idx, want.idx)


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("tiny_f32", 1), ("ragged_small", 1), ("fp8_ragged_small", 2)])
def test_abandoned_call_of_tokens_that_every_block_decides(name, n, monkeypatch):
    w = W.get(name, n=n)
    dev = W.device_inputs(w)
    want, c = Call(w, dev)(), Call(w, dev)
    monkeypatch.setenv("MOE_TEST_STALL", "1")
    c()
    assert moe.moe_sync_status(c.ws) == moe.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_TEST_STALL")
    c()
    assert moe.moe_sync_status(c.ws) == moe.MOE_OK and torch.equal(c.y, want.y)


# ---- workspace ---------------------------------------------------------------------


# Bytes for 1000 tokens before there was moe_layer_decode (and for fewer where they are the same still).
FORMER = {
    "tiny_f32": {1: 11264, 7: 35840, 64: 272128, 1000: 4166656},
    "mixtral_8x7b": {1000: 91194368},
    "deepseek_v3_small": {1000: 15774720},
    "deepseek_v3_prefill": {1000: 285342720},
    "deepseek_v3_decode_fp8_32e": {1: 8263424, 7: 10478336, 1000: 374758656},
    "ragged_small": {1000: 3130112},
}


@pytest.mark.parametrize("name", FORMER)
def test_a_batch_of_many_tokens_needs_no_more_for_the_decode_call(name):
    cfg = H.cfg_for(W.get(name))
    assert {n: moe.moe_workspace_size(cfg, n) for n in FORMER[name]} == FORMER[name]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["tiny_f32", "deepseek_v3_small", "deepseek_v3_decode_small_fp8"])
def test_stages_find_nothing_in_the_workspace(name):
    """moe_layer_decode writes where the other entry points have their scratch: between their calls it changes nothing."""
    w = W.get(name, n=64)
    dev = W.device_inputs(w)
    c, n, act = Call(w, dev), w.n, dev["x"].dtype
    c()
    want_decode = c.y.clone()

    def stages(between):
        idx, tw = torch.empty(n, w.top_k, dtype=torch.int32, device="cuda"), torch.empty(n, w.top_k, device="cuda")
        counts = torch.empty(w.n_routed, dtype=torch.int32, device="cuda")
        offs = torch.empty(w.n_routed + 1, dtype=torch.int32, device="cuda")
        perm, dest = (torch.empty(n * w.top_k, dtype=torch.int32, device="cuda") for _ in range(2))
        xp, eo = (torch.zeros(n * w.top_k, w.d_model, dtype=act, device="cuda") for _ in range(2))
        y = torch.empty(n, w.d_model, dtype=act, device="cuda")
        moe.moe_route(c.cfg, n, dev["x"], c.weights, idx, tw, counts, None, c.ws)
        between()
        moe.moe_permute(c.cfg, n, dev["x"], idx, offs, perm, dest, xp, c.ws)
        between()
        moe.moe_expert_ffn(c.cfg, n, xp, offs, c.weights, eo, c.ws)
        between()
        moe.moe_combine(c.cfg, n, eo, dest, tw, dev["x"], c.weights, y, c.ws)
        between()
        return idx, tw, counts, offs, dest, eo, y

    want = stages(lambda: None)
    got = stages(c)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(c.y, want_decode) and moe.moe_sync_status(c.ws) == moe.MOE_OK
