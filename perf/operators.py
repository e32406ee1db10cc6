"""Cases and plain forms of the serving-step operators around the sparse MoE layer:

* ``norm``: residual addition, root-mean-square norm and E4M3 output with one power-of-two scale per 1 x 128 tile
  (``moe_add_rmsnorm``);
* ``layer``: the whole sparse MoE layer for at most 64 tokens (``moe_layer_decode``).

``run`` computes them in elementary torch operations, or through the library where ``own`` is true; ``exact`` computes
the same definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases -------------------------------------------------------------------------


def _norm(name, rows, cols, dtype, residual, y, codes):
    return dict(name=name, op="norm", rows=rows, cols=cols, dtype=dtype, residual=residual, y=y, codes=codes)


def _layer(name, n, d, experts, k, inter, shared=0, groups=1, kept=1, score="softmax", renorm=False, rsf=1.0, dtype="bf16"):
    return dict(name=name, op="layer", n=n, d=d, experts=experts, k=k, inter=inter, shared=shared, groups=groups, kept=kept,
                score=score, renorm=renorm, rsf=rsf, dtype=dtype)


_V3 = dict(d=7168, experts=256, k=8, inter=2048, shared=1, groups=8, kept=4, score="sigmoid", renorm=True, rsf=2.5)


def listed():
    return [
        # one token of a decode step before an FP8 MoE layer: the router's bf16 row and the experts' codes
        _norm("norm_1x7168_bf16_fp8", 1, 7168, "bf16", True, True, True),
        # a decode batch, ragged row count
        _norm("norm_61x5120_bf16_fp8", 61, 5120, "bf16", True, True, True),
        # the first norm of a float32 model: no residual yet, a width off the 128 grid
        _norm("norm_1000x200_f32", 1000, 200, "f32", False, True, False),
        # a prefill batch between two bf16 layers
        _norm("norm_4096x4096_bf16", 4096, 4096, "bf16", True, True, False),
        # the largest prefill batch, feeding FP8 experts
        _norm("norm_16384x7168_bf16_fp8", 16384, 7168, "bf16", True, True, True),
        # the smallest layer: latency only
        _layer("layer_tiny_n1_f32", 1, 128, 8, 2, 256, dtype="f32"),
        # odd sizes, a shared expert
        _layer("layer_ragged_n7_bf16", 7, 200, 5, 2, 72, shared=1, renorm=True),
        # one sequence of a Mixtral-shaped model being decoded
        _layer("layer_mixtral_n1_bf16", 1, 4096, 8, 2, 14336, renorm=True),
        # a few sequences of a DeepSeek-V3-shaped model
        _layer("layer_v3_n4_bf16", 4, dtype="bf16", **_V3),
        # the largest batch the form takes: most experts active
        _layer("layer_v3_n64_bf16", 64, dtype="bf16", **_V3),
        # FP8 experts, one sequence and a batch
        _layer("layer_v3_n1_fp8", 1, dtype="fp8", **_V3),
        _layer("layer_v3_n24_fp8", 24, dtype="fp8", **_V3),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        codes = rng.random() < 0.5
        cols = 128 * _spread(rng, 1, 56) if codes else 8 * _spread(rng, 8, 896)
        rows = min(_spread(rng, 1, 16384), 16384 * 7168 // cols)
        return dict(op="norm", rows=rows, cols=cols, dtype=rng.choice(["f32", "bf16", "bf16"]),
                    residual=rng.random() < 0.7, y=not codes or rng.random() < 0.7, codes=codes)
    dtype = rng.choice(["f32", "bf16", "bf16", "fp8", "fp8"])
    score = rng.choice(["softmax", "sigmoid", "sqrtsoftplus"])
    groups = 1
    experts = _spread(rng, 4, 256)
    if score == "sigmoid" and rng.random() < 0.6:
        groups = rng.choice([2, 4, 8])
        experts = groups * max(2, experts // groups)
    kept = max(1, groups // 2)
    k = min(rng.choice([1, 2, 4, 6, 8, 11]), kept * (experts // groups))
    step = 128 if dtype == "fp8" else 8
    d = step * _spread(rng, max(1, 64 // step), 7168 // step)
    inter = step * _spread(rng, max(1, 64 // step), 4096 // step)
    size = 4 if dtype == "f32" else 2 if dtype == "bf16" else 1
    while 3 * experts * d * inter * size > 6 << 30:  # a drawn case costs no more than the largest listed one
        inter = max(step, inter // 2 // step * step)
    return dict(op="layer", n=_spread(rng, 1, 64), d=d, experts=experts, k=k, inter=inter, shared=rng.choice([0, 0, 1, 2]),
                groups=groups, kept=kept, score=score, renorm=rng.random() < 0.6, rsf=rng.choice([1.0, 2.5]), dtype=dtype)


# ---- inputs ------------------------------------------------------------------------


def _normal(g, shape, scale, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _fp8_matrix(g, *shape):
    """E4M3 codes of magnitude 0.25 to 3.75 and UE8M0 bytes per 128 x 128 block, of root mean square near fan_in^-1/2."""
    q = torch.empty(shape, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    q.bitwise_and_(0x9F).add_(0x28)  # a sign bit and a magnitude code in 0x28 .. 0x47
    e = math.floor(math.log2(1.0 / (1.69 * math.sqrt(shape[-1])))) + 127
    blocks = shape[:-2] + (-(-shape[-2] // 128), shape[-1] // 128)
    return q, torch.randint(e, e + 2, blocks, dtype=torch.uint8, device="cuda", generator=g)


def _prepare_norm(c, g):
    dt = DTYPES[c["dtype"]]
    rows, cols = c["rows"], c["cols"]
    s = dict(case=c)
    # a residual stream: a few channels far larger than the rest
    loud = 1.0 + 30.0 * (torch.rand(cols, device="cuda", generator=g) < 0.01)
    s["x"] = _normal(g, (rows, cols), 1.0, dt)
    s["residual"] = (_normal(g, (rows, cols), 1.0, dt) * loud).to(dt) if c["residual"] else None
    s["weight"] = (1.0 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(dt)
    if own:
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if c["y"] else None
        s["codes"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda") if c["codes"] else None
        s["scales"] = torch.empty(rows, cols // 128, dtype=torch.uint8, device="cuda") if c["codes"] else None
    return s


def _prepare_layer(c, g):
    n, d, E, I = c["n"], c["d"], c["experts"], c["inter"]
    act = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = dict(case=c, x=_normal(g, (n, d), 1.0, act), w_router=_normal(g, (E, d), d ** -0.5, act), bias=None)
    if c["score"] != "softmax":
        s["bias"] = torch.empty(E, device="cuda").uniform_(-0.1, 0.1, generator=g)
    shapes = dict(w_gate=(E, I, d), w_up=(E, I, d), w_down=(E, d, I))
    if c["shared"]:
        J = c["shared"] * I
        shapes.update(ws_gate=(J, d), ws_up=(J, d), ws_down=(d, J))
    for name, shape in shapes.items():
        if c["dtype"] == "fp8":
            s[name], s[name + "_scale"] = _fp8_matrix(g, *shape)
        else:
            s[name] = _normal(g, shape, shape[-1] ** -0.5, act)
    if own:
        import top_routing_expert_router_b200 as moe

        s["cfg"] = moe.make_config(d, E, c["k"], I, n_shared=c["shared"], n_group=c["groups"], topk_group=c["kept"],
                                   score_fn=c["score"], renormalize=c["renorm"], routed_scaling_factor=c["rsf"],
                                   dtype=c["dtype"])
        scales = {k: s[m + "_scale"] for k, m in (("gate", "w_gate"), ("up", "w_up"), ("down", "w_down"),
                                                  ("ws_gate", "ws_gate"), ("ws_up", "ws_up"), ("ws_down", "ws_down"))
                  if m + "_scale" in s}
        s["weights"] = moe.make_weights(s["w_router"], s["w_gate"], s["w_up"], s["w_down"], s.get("ws_gate"),
                                        s.get("ws_up"), s.get("ws_down"), s["bias"], scales=scales)
        s["ws"] = torch.empty(moe.moe_workspace_size(s["cfg"], n), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty_like(s["x"])
        s["idx"] = torch.empty(n, c["k"], dtype=torch.int32, device="cuda")
        s["gates"] = torch.empty(n, c["k"], dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_norm if case["op"] == "norm" else _prepare_layer)(case, g)


# ---- the operators -----------------------------------------------------------------


def _quantize(v):
    """E4M3 values and the exponents e of their 1 x 128 tiles: the smallest integer with max|v| <= 448 * 2^e."""
    t = v.unflatten(-1, (-1, 128))
    f, x = torch.frexp(t.abs().amax(-1))
    e = torch.where(f == 0, 0, x - torch.where(f <= 0.875, 9, 8))
    return torch.ldexp(t, -e[..., None]).to(torch.float8_e4m3fn).flatten(-2), e


def _dequantize(q, e):
    return torch.ldexp(q.float().unflatten(-1, (-1, 128)), e[..., None]).flatten(-2)


def _plain_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    v = s["x"].float()
    out = {}
    if s["residual"] is not None:
        v = v + s["residual"].float()
        out["sum"] = v.to(dt)
    y = (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()).to(dt)
    if c["y"]:
        out["y"] = y
    if c["codes"]:
        q, e = _quantize(y.float())
        out["codes"], out["scales"] = q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _route(c, logits, bias):
    """Experts in descending selection score (ties: the lower index first) and their gates, in the logits' precision."""
    if c["score"] == "softmax":
        score, chosen = torch.softmax(logits, -1), logits
    else:
        score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.sqrt(torch.logaddexp(logits, torch.zeros_like(logits)))
        chosen = score + bias
    if c["groups"] > 1:
        grouped = chosen.unflatten(-1, (c["groups"], -1))
        rank = torch.sort(grouped, dim=-1, descending=True).values
        order = torch.sort(rank[..., :2].sum(-1), dim=-1, descending=True, stable=True).indices[..., : c["kept"]]
        keep = torch.zeros_like(grouped[..., 0], dtype=torch.bool).scatter_(-1, order, True)
        chosen = torch.where(keep[..., None], grouped, -torch.inf).flatten(-2)
    idx = torch.sort(chosen, dim=-1, descending=True, stable=True).indices[..., : c["k"]]
    gates = score.gather(-1, idx)
    if c["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    return idx, gates * c["rsf"]


def _matrix(s, name, at=None):
    """A weight matrix (of the experts `at`, where given) in 32 bits."""
    w = s[name] if at is None else s[name][at]
    if s["case"]["dtype"] != "fp8":
        return w.float()
    e = (s[name + "_scale"] if at is None else s[name + "_scale"][at]).int() - 127
    e = e.repeat_interleave(128, -2)[..., : w.shape[-2], :]
    return _dequantize(w.view(torch.float8_e4m3fn), e)


def _operand(c, v):
    """An activation as it enters an expert matrix: FP8 experts take the E4M3 codes of its bf16 value."""
    return _dequantize(*_quantize(v.bfloat16().float())) if c["dtype"] == "fp8" else v


def _swiglu(c, x, gate, up, down):
    """x [d] through matrices [..., I, d], [..., I, d], [..., d, I]."""
    g = gate @ x
    h = _operand(c, g * torch.sigmoid(g) * (up @ x))
    return (down @ h[..., None])[..., 0]


def _plain_layer(s):
    c = s["case"]
    x = s["x"].float()
    # the logits in 64 bits: the experts' order is decided by small differences
    idx, gates = _route(c, s["x"].double() @ s["w_router"].double().T, None if s["bias"] is None else s["bias"].double())
    gates = gates.float()
    xq = _operand(c, x)
    shared = [_matrix(s, m) for m in ("ws_gate", "ws_up", "ws_down")] if c["shared"] else None
    rows = []
    for t in range(c["n"]):  # a token at a time: its k experts' matrices in 32 bits fit, the batch's would not
        out = _swiglu(c, xq[t], *(_matrix(s, m, idx[t]) for m in ("w_gate", "w_up", "w_down")))
        y = (gates[t][:, None] * out).sum(0)
        rows.append(y + _swiglu(c, xq[t], *shared) if shared else y)
    return {"y": torch.stack(rows).to(s["x"].dtype), "idx": idx.int(), "gates": gates}


def _own_norm(s):
    import top_routing_expert_router_b200 as moe

    moe.moe_add_rmsnorm(s["x"], s["weight"], EPS, y=s["y"], residual=s["residual"], sum_out=s["sum"], codes=s["codes"],
                        scale_bytes=s["scales"])
    out = {"sum": s["sum"], "y": s["y"]}
    if s["codes"] is not None:
        out["codes"], out["scales"] = s["codes"].view(torch.float8_e4m3fn), s["scales"].view(torch.float8_e8m0fnu)
    return out


def _own_layer(s):
    import top_routing_expert_router_b200 as moe

    moe.moe_layer_decode(s["cfg"], s["case"]["n"], s["x"], s["weights"], s["y"], s["ws"], topk_idx=s["idx"],
                         topk_w=s["gates"])
    return {"y": s["y"], "idx": s["idx"], "gates": s["gates"]}


def run(state):
    norm = state["case"]["op"] == "norm"
    if own:
        return _own_norm(state) if norm else _own_layer(state)
    return _plain_norm(state) if norm else _plain_layer(state)


# ---- the definitions in 64 bits ----------------------------------------------------


def _round_bits(v, bits, lowest):
    """v rounded to `bits` significant bits, ties to even; below 2^lowest in steps of 2^(lowest - bits + 1)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** lowest)))
    e = torch.where(torch.exp2(e) > v.abs().clamp_min(2.0 ** lowest), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= v.abs(), e + 1, e)
    step = torch.exp2(e - bits + 1)
    return torch.round(v / step) * step


def _tiles_64(v):
    """E4M3 values of v's 1 x 128 tiles and the tiles' scales, by the two inequalities that define the exponent."""
    t = v.reshape(*v.shape[:-1], -1, 128)
    top = t.abs().max(-1).values
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    scale = torch.where(top > 0, torch.exp2(e), torch.ones_like(e))
    return _round_bits(t / scale[..., None], 4, -6).reshape(v.shape), scale


def _exact_norm(s):
    c = s["case"]
    v = s["x"].double()
    out = {"sum": None, "y": None, "codes": None, "scales": None}
    if s["residual"] is not None:
        v = v + s["residual"].double()
        out["sum"] = v
    y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / c["cols"] + EPS) * s["weight"].double()
    if c["y"]:
        out["y"] = y
    if c["codes"]:
        bits = 8 if c["dtype"] == "bf16" else 24
        out["codes"], out["scales"] = _tiles_64(_round_bits(y, bits, -126))
    return out


def _wide(s, name, e=None):
    w = s[name] if e is None else s[name][e]
    if s["case"]["dtype"] != "fp8":
        return w.double()
    b = s[name + "_scale"] if e is None else s[name + "_scale"][e]
    scale = torch.exp2(b.double() - 127.0)
    scale = torch.kron(scale, torch.ones(128, 128, dtype=torch.float64, device=w.device))[: w.shape[0]]
    m = w.int()
    frac, ex, sign = (m & 7).double(), ((m >> 3) & 15).double(), 1.0 - 2.0 * (m >> 7).double()
    value = torch.where(ex > 0, torch.exp2(ex - 7) * (1 + frac / 8), frac * 2.0 ** -9)
    return sign * value * scale


def _exact_expert(s, x, names, e=None):
    fp8 = s["case"]["dtype"] == "fp8"

    def entering(v):
        if not fp8:
            return v
        q, scale = _tiles_64(_round_bits(v, 8, -126))
        return q * scale.repeat_interleave(128, -1)

    a = entering(x)
    g = a @ _wide(s, names[0], e).T
    h = g / (1.0 + torch.exp(-g)) * (a @ _wide(s, names[1], e).T)
    return entering(h) @ _wide(s, names[2], e).T


def _exact_layer(s):
    c = s["case"]
    n, E, G = c["n"], c["experts"], c["groups"]
    x = s["x"].double()
    logits = (x @ s["w_router"].double().T).cpu()
    if c["score"] == "softmax":
        p = torch.exp(logits - logits.max(-1, keepdim=True).values)
        score, sel = p / p.sum(-1, keepdim=True), logits
    else:
        score = 1.0 / (1.0 + torch.exp(-logits)) if c["score"] == "sigmoid" else torch.sqrt(torch.log1p(torch.exp(-logits.abs())) + logits.clamp_min(0))
        sel = score + s["bias"].double().cpu()
    y = torch.zeros(n, c["d"], dtype=torch.float64, device=x.device)
    idx, gates = torch.zeros(n, c["k"], dtype=torch.int32), torch.zeros(n, c["k"], dtype=torch.float64)
    held = {}
    for t in range(n):
        v = sel[t].tolist()
        allowed = range(E)
        if G > 1:
            per = E // G
            of = [sum(sorted(v[g * per:(g + 1) * per], reverse=True)[:2]) for g in range(G)]
            best = sorted(range(G), key=lambda g: (-of[g], g))[: c["kept"]]
            allowed = [e for e in range(E) if e // per in best]
        mine = sorted(allowed, key=lambda e: (-v[e], e))[: c["k"]]
        w = [float(score[t, e]) for e in mine]
        total = sum(w) if c["renorm"] else 1.0
        for j, e in enumerate(mine):
            idx[t, j], gates[t, j] = e, w[j] / total * c["rsf"]
            held.setdefault(e, []).append((t, float(gates[t, j])))
    for e, rows in held.items():
        at = torch.tensor([t for t, _ in rows], device=x.device)
        w = torch.tensor([g for _, g in rows], dtype=torch.float64, device=x.device)
        y[at] += w[:, None] * _exact_expert(s, x[at], ("w_gate", "w_up", "w_down"), e)
    if c["shared"]:
        y += _exact_expert(s, x, ("ws_gate", "ws_up", "ws_down"))
    return {"y": y, "idx": idx, "gates": gates}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_layer(s)


# ---- work --------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "norm":
        cells, b = c["rows"] * c["cols"], 4 if c["dtype"] == "f32" else 2
        moved = cells * b * (1 + 2 * c["residual"] + c["y"]) + c["cols"] * b
        return {"bytes": moved + c["codes"] * (cells + cells // 128), "flops": 5 * cells}
    n, d, E, k, I = c["n"], c["d"], c["experts"], c["k"], c["inter"]
    a = 4 if c["dtype"] == "f32" else 2
    w = {"f32": 4, "bf16": 2, "fp8": 1 + 1 / 16384}[c["dtype"]]
    active = E * (1.0 - (1.0 - k / E) ** n)  # expected distinct experts of n tokens under even routing
    weights = 3 * d * I * (active + c["shared"]) * w + E * d * a
    return {"bytes": weights + 2 * n * d * a + 8 * n * k, "flops": 2 * n * E * d + 6 * n * (k + c["shared"]) * d * I}
