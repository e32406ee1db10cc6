"""moe_layer_decode where tiles are cut along k: the rule's parts against their workspace on the CPU, and on the GPU
layers of every kind of cut against the oracle, and the shapes that are measured against their 64-bit definition.

Tolerances. bf16: 2^-8 of the element (y's rounding) plus 2^-8 of its row's rms. The second covers h and the sums: h carries
16 bits, 2^-16 of each term, and gate and up are chains of at most d / 16 = 1024 additions in the tensor cores, which may
drop up to 2^-23 of the sum each, 1.2e-4 of g and of u. All terms erring one way that is (2^-16 + 2 * 1.2e-4) * 0.64 *
sqrt(K) of the rms for K normal terms: at K = 2048, the longest here but one, 0.0074; as roundings go (they do not line
up: h's are random, the chains' common shrinkage scales the row by 2e-4) under a tenth of that, where 2^-8 is 0.0039. FP8 and
binary32: the layer parity tests' 2e-2 and 1e-4 of the larger of element and row rms. An FP8 code of h flips (by up to
2^-3 of its value) where h lies within its sums' error of a border between codes, at most one in 500, which is 0.125 *
sqrt(1 / 500) = 0.0056 of the rms in y, the largest of 10^5 near 4 of them. A binary32 lane sums K / 32 terms and 5
levels: 229 at K = 7168, as roundings go sqrt(229) * 2^-24 = 9e-7 of a sum, a chain's worst case 1.4e-5 of the terms' magnitudes."""
import ctypes
import importlib.util
import pathlib
import random

import numpy as np
import pytest
import torch

import top_routing_expert_router_b200 as moe
from synth import workloads as W
from tests import moe_harness as H
from tests.test_decode import Call, _oracle

DTYPE = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "fp8": moe.MOE_FP8}


class Splits(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("s1", "per1", "s1s", "per1s", "s2", "per2", "s2s", "per2s")]


class Rows(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("gu", "gus", "eo", "es")]


def _host(symbol, result):
    f = moe.lib_handle()[symbol]
    f.restype, f.argtypes = result, [ctypes.c_int64] + [ctypes.c_int32] * 6
    return f


decode_splits = _host("_ZN3moe13decode_splitsEliiiiii", Splits)
decode_rows = _host("_ZN3moe11decode_rowsEliiiiii", Rows)

# routed and shared gate/up parts, routed and shared down parts
CASES = [
    ("ragged_small", dict(n=29, d_model=7168, n_routed=5, top_k=2, moe_intermediate_size=512, n_shared=1), (7, 5, 1, 1)),
    ("ragged_small", dict(n=64, d_model=7168, n_routed=4, top_k=1, moe_intermediate_size=256, n_shared=1), (9, 4, 1, 1)),
    ("ragged_small", dict(n=13, d_model=7168, n_routed=3, top_k=1, moe_intermediate_size=264, n_shared=4), (12, 9, 1, 2)),
    ("ragged_small", dict(n=1, d_model=16384, n_routed=4, top_k=1, moe_intermediate_size=128, n_shared=1), (16, 16, 1, 1)),
    ("ragged_small", dict(n=6, d_model=4104, n_routed=8, top_k=2, moe_intermediate_size=200, n_shared=0), (9, 1, 1, 1)),
    ("ragged_small", dict(n=9, d_model=264, n_routed=2, top_k=2, moe_intermediate_size=4104, n_shared=0), (1, 1, 10, 1)),
    ("ragged_small", dict(n=33, d_model=520, n_routed=6, top_k=2, moe_intermediate_size=2056, n_shared=1), (1, 1, 5, 5)),
    ("fp8_ragged_small", dict(n=24, d_model=7168, n_routed=16, top_k=4, moe_intermediate_size=512, n_shared=1), (2, 5, 1, 1)),
    ("fp8_ragged_small", dict(n=24, d_model=4096, n_routed=4, top_k=2, moe_intermediate_size=256, n_shared=1), (4, 4, 1, 1)),
    ("fp8_ragged_small", dict(n=64, d_model=7168, n_routed=2, top_k=1, moe_intermediate_size=128, n_shared=1), (4, 4, 1, 1)),
    ("fp8_ragged_small", dict(n=7, d_model=16384, n_routed=2, top_k=1, moe_intermediate_size=256, n_shared=1), (16, 11, 1, 1)),
    ("fp8_skewed_small", dict(n=40, d_model=4096, n_routed=8, top_k=1, moe_intermediate_size=128, n_shared=1), (4, 4, 1, 1)),
    ("fp8_ragged_small", dict(n=17, d_model=384, n_routed=3, top_k=2, moe_intermediate_size=4096, n_shared=1), (1, 1, 4, 4)),
]
IDS = ["%s-%d-%d-%s" % (n.split("_")[0], k["n"], k["d_model"], "x".join(map(str, c))) for n, k, c in CASES]


def _splits_of(w):
    return decode_splits(w.n, w.d_model, w.n_routed, w.top_k, w.moe_intermediate_size, w.I_s, DTYPE[w.dtype])


@pytest.mark.parametrize("name,kw,cuts", CASES, ids=IDS)
def test_cases_are_cut_as_they_say(name, kw, cuts):
    s = _splits_of(W.get(name, **kw))
    assert (s.s1, s.s1s, s.s2, s.s2s) == cuts


def test_parts_cover_k_and_fit_the_workspace():
    """Every part holds some k block and all parts hold all of them; a workspace of n tokens holds the parts of fewer."""
    rng = random.Random(1)
    for _ in range(600):
        dtype = rng.choice(["bf16", "fp8"])
        unit, ke = (8, 64) if dtype == "bf16" else (128, 128)
        size = lambda most: unit * max(1, round(2 ** rng.uniform(0, np.log2(most / unit))))  # noqa: E731
        d, I, E = size(16384), size(16384), round(2 ** rng.uniform(0, 8))
        k, shared = rng.randint(1, min(E, 32)), rng.choice([0, 1, 2])
        Is, n = shared * I, rng.choice([1, 2, 3, 5, 8, 16, 33, 64])
        rows = decode_rows(n, d, E, k, I, Is, DTYPE[dtype])
        for m in range(1, n + 1):
            s = decode_splits(m, d, E, k, I, Is, DTYPE[dtype])
            for parts, per, length in ((s.s1, s.per1, d), (s.s2, s.per2, I)) + ((s.s1s, s.per1s, d), (s.s2s, s.per2s, Is)) * (Is > 0):
                blocks = -(-length // ke)
                assert (parts - 1) * per < blocks <= parts * per and (dtype == "bf16" or parts == 1 or per % 4 == 0)
            assert (m * k * s.s1 if s.s1 > 1 else 0) * I + (m * s.s1s if s.s1s > 1 else 0) * Is <= rows.gu * I + rows.gus * Is
            # (the shared parts start behind all of the routed ones' room)
            assert s.s1s == 1 or m * k * s.s1 * I + m * s.s1s * Is <= rows.gu * I + rows.gus * Is
            assert m * k * s.s2 <= rows.eo and (Is == 0 or m * s.s2s <= rows.es)


def _close(dtype, y, want):
    if dtype != "bf16":
        return H.rel_err(y, want) <= (1e-4 if dtype == "f32" else 2e-2)
    rms = np.sqrt(np.mean(want * want, axis=1, keepdims=True))
    return (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * rms).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name,kw,cuts", CASES, ids=IDS)
def test_layers_in_parts(name, kw, cuts):
    w = W.get(name, **kw)
    s = _splits_of(w)
    assert (s.s1, s.s1s, s.s2, s.s2s) == cuts
    r, c = _oracle(w, W.host_inputs(w)), Call(w, W.device_inputs(w))
    for _ in range(3):
        c().check(r)
    keep = ~r["exempt"]
    assert _close(w.dtype, H.as_f64(c.y)[: w.n][keep], r["y"][keep])


# ---- the shapes that are measured ----------------------------------------------------


def _operators():
    spec = importlib.util.spec_from_file_location("operators", pathlib.Path(__file__).parents[1] / "perf" / "operators.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


OPS = _operators()
LISTED = [c for c in OPS.listed() if c["op"] == "layer"]


def _drawn(seed):
    rng = random.Random(seed)
    while True:
        c = OPS.draw(rng)
        if c["op"] == "layer" and 3 * c["experts"] * c["d"] * c["inter"] < 1 << 29:
            return c


@pytest.mark.gpu
@pytest.mark.parametrize("case", LISTED + [_drawn(i) for i in range(12)], ids=lambda c: c.get("name", "drawn"))
def test_against_the_definition_in_64_bits(case):
    want = OPS.exact(case, 5)
    torch.cuda.empty_cache()
    got = OPS.run(OPS.prepare(case, 5))
    assert torch.equal(got["idx"].cpu(), want["idx"])
    np.testing.assert_allclose(got["gates"].cpu().numpy(), want["gates"].numpy(), rtol=2.0 ** -22, atol=0)
    assert _close(case["dtype"], H.as_f64(got["y"]), want["y"].cpu().numpy())
    torch.cuda.empty_cache()
