"""moe_layer_decode where it can go wrong: hand-overs between threads, waits that run out, workspaces, types."""
import pathlib
import re

import pytest
import torch

import top_routing_expert_router_b200 as moe
from synth import workloads as W
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
