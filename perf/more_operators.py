"""The operators of an expert block with microscaled 4-bit weights, as measured cases.

MXFP4 holds 32 consecutive inputs of a row as 4-bit floats (1 sign, 2 exponent,
1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) under one power of two.  A block of
a decoder takes the residual stream through a norm, a projection or a whole
expert layer, and back.  Each case is one of these calls:

  quantize  weights or activations to MXFP4, and back to the values they stand for
  product   y = x W^T with W in MXFP4, x in bf16 or in MXFP4 as well
  moe       router, selected experts and their weighted sum, for a few tokens
  norm      h + scale * gate * norm(f), its norm, in bf16 or in MXFP4

Where ``own`` is false, run() is plain torch in 32 bits (64 for router scores,
and for what is rounded to 4 bits after arithmetic); where it is true, it calls
the library.
"""

import math
import random

import torch

own = False

DEVICE = "cuda"
QUANTIZE, PRODUCT, MOE, NORM = "quantize", "product", "moe", "norm"
GROUP = 32


def listed():
    return [
        # activations of a few requests on their way into a 4-bit product: latency
        dict(name="quantize 5 rows bf16", op=QUANTIZE, n=5, k=8192, source="bf16"),
        # a checkpoint's fused gate and up projection, offline
        dict(name="quantize 8B w13 f32", op=QUANTIZE, n=28672, k=4096, source="f32"),
        # batch-1 decode, the 7B wqkv projection
        dict(name="product 1 token wqkv", op=PRODUCT, m=1, n=12288, k=4096, x="bf16", out="bf16"),
        # 5 drafted tokens through the 70B gate and up projection
        dict(name="product 5 tokens w13", op=PRODUCT, m=5, n=57344, k=8192, x="bf16", out="f32"),
        # a serving batch, odd, through the 8B down projection
        dict(name="product 47 tokens w2", op=PRODUCT, m=47, n=4096, k=14336, x="bf16", out="bf16"),
        # a prompt with bf16 activations through the 8B gate and up projection
        dict(name="product 2000 tokens w13", op=PRODUCT, m=2000, n=28672, k=4096, x="bf16", out="bf16"),
        # a long prompt with activations in 4 bits too, the 70B wqkv projection
        dict(name="product 4096 both in 4 bits", op=PRODUCT, m=4096, n=10240, k=8192, x="mxfp4", out="bf16"),
        # batch-1 decode through a Mixtral layer with int8 experts
        dict(name="moe 1 token 8 int8", op=MOE, tokens=1, experts=8, top=2, dim=4096, f=14336, weights="int8",
             scores="logits", out="f32"),
        # 6 tokens verify through a Mixtral layer with 4-bit experts
        dict(name="moe 6 tokens 8 mxfp4", op=MOE, tokens=6, experts=8, top=2, dim=4096, f=14336, weights="mxfp4",
             scores="router", out="bf16"),
        # a serving batch through a layer of many small experts
        dict(name="moe 61 tokens 128 mxfp4", op=MOE, tokens=61, experts=128, top=8, dim=2048, f=768, weights="mxfp4",
             scores="router", out="bf16"),
        # batch-1 decode, the residual around a block: latency
        dict(name="norm 1 row 4096", op=NORM, rows=1, dim=4096, h="bf16", f="f32", post=False, gate="none", u="bf16"),
        # a prompt's rows with norms on both sides, gated, into a 4-bit product
        dict(name="norm 4099 rows 8192 mxfp4", op=NORM, rows=4099, dim=8192, h="f32", f="bf16", post=True,
             gate="sigmoid", u="mxfp4"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    largest = max(work(c)["bytes"] for c in listed())
    most = max(work(c)["flops"] for c in listed())
    while True:
        c = _draw(rng)
        w = work(c)
        # all experts are resident, whichever run: no more than the largest listed layer's
        held = c["op"] != MOE or c["experts"] * c["dim"] * c["f"] <= 8 * 4096 * 14336
        if held and w["bytes"] <= 0.8 * largest and w["flops"] <= 0.8 * most:
            return c


def _draw(rng):
    op = rng.choice([QUANTIZE, PRODUCT, PRODUCT, PRODUCT, MOE, MOE, NORM])
    if op == QUANTIZE:
        return dict(op=op, n=_log(rng, 1, 40000), k=GROUP * _log(rng, 1, 896), source=rng.choice(["f32", "bf16"]))
    if op == PRODUCT:
        # short batches, or prompts
        m = rng.choice([1, 2, 3, 5, 8, _log(rng, 1, 128), _log(rng, 1, 128), _log(rng, 128, 5000)])
        return dict(op=op, m=m, n=_log(rng, 16, 60000), k=GROUP * _log(rng, 2, 896),
                    x=rng.choice(["bf16", "bf16", "mxfp4"]), out=rng.choice(["f32", "bf16"]))
    if op == MOE:
        experts, top = rng.choice([(8, 2), (8, 2), (4, 1), (16, 2), (32, 4), (64, 6), (128, 8), (60, 4)])
        return dict(op=op, tokens=rng.choice([1, 1, 2, 4, 8, _log(rng, 1, 64), rng.randint(1, 64)]), experts=experts,
                    top=top, dim=GROUP * _log(rng, 8, 160), f=GROUP * _log(rng, 8, 448),
                    weights=rng.choice(["int8", "mxfp4", "mxfp4"]), scores=rng.choice(["router", "router", "logits"]),
                    out=rng.choice(["f32", "bf16"]))
    return dict(op=op, rows=_log(rng, 1, 8192), dim=GROUP * _log(rng, 4, 512), h=rng.choice(["f32", "bf16"]),
                f=rng.choice(["f32", "bf16"]), post=rng.random() < 0.5, gate=rng.choice(["none", "plain", "sigmoid", "silu"]),
                u=rng.choice(["bf16", "bf16", "mxfp4"]))


def _mx(weights):
    """Bytes of that many weights in MXFP4."""
    return weights * (GROUP // 2 + 1) // GROUP


def _picked(case):
    """Experts in use, as expected of scores that favour none (all of them for many tokens)."""
    return case["experts"] * (1 - (1 - case["top"] / case["experts"]) ** case["tokens"])


def work(case):
    op = case["op"]
    if op == QUANTIZE:
        weights = case["n"] * case["k"]
        return {"bytes": weights * (4 if case["source"] == "f32" else 2) + _mx(weights) + 2 * weights,
                "flops": 2 * weights}
    if op == PRODUCT:
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (2 * m * k if case["x"] == "bf16" else _mx(m * k)) + _mx(n * k) +
                m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    if op == MOE:
        t, e, dim, f = case["tokens"], case["experts"], case["dim"], case["f"]
        one = (_mx(3 * dim * f) if case["weights"] == "mxfp4" else 3 * dim * f + 2 * (2 * f + dim))
        scores = 2 * e * dim if case["scores"] == "router" else 4 * t * e
        return {"bytes": int(_picked(case) * one) + scores + t * dim * (2 + (4 if case["out"] == "f32" else 2)),
                "flops": 6 * t * case["top"] * dim * f}
    values = case["rows"] * case["dim"]
    wide = {"f32": 4, "bf16": 2}
    return {"bytes": values * (2 * wide[case["h"]] + wide[case["f"]] + (0 if case["gate"] == "none" else 2) + 2) +
            (_mx(values) if case["u"] == "mxfp4" else 0), "flops": values * 10}


# --- inputs ----------------------------------------------------------------


def _normal(g, *shape, sigma=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEVICE).normal_(0.0, sigma, generator=g)


def _power(e):
    """2^e in 32 bits, e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _steps(v):
    """Nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with the sign of v: steps of a half up to 2, of one up to 4, of two up to
    6, ties to even."""
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(v.dtype)
    return (torch.round(v / step) * step).clamp(-6, 6)


def _codes(w):
    """Rows of floats in MXFP4: codes [n, k / 2] (even inputs low) and scale bytes [n, k / 32]."""
    n, k = w.shape
    groups = w.float().view(n, k // GROUP, GROUP)
    top = torch.frexp(groups.abs().amax(-1)).exponent - 1                   # floor(log2), for a group that is not 0
    power = (top - 2).clamp(min=-126)
    v = _steps(groups * _power(-power)[..., None])
    sizes = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEVICE)
    code = torch.bucketize(v.abs(), sizes, right=True, out_int32=True).to(torch.uint8)
    code |= torch.signbit(groups).to(torch.uint8) << 3
    code = code.view(n, k)
    return code[:, 0::2] | code[:, 1::2] << 4, (power + 127).to(torch.uint8)


def _weights(g, n, k, chunk=1 << 27):
    """Normal weights in MXFP4, made in parts."""
    q = torch.empty(n, k // 2, dtype=torch.uint8, device=DEVICE)
    scale = torch.empty(n, k // GROUP, dtype=torch.uint8, device=DEVICE)
    rows = max(1, chunk // k)
    for a in range(0, n, rows):
        b = min(n, a + rows)
        q[a:b], scale[a:b] = _codes(_normal(g, b - a, k, sigma=0.02))
    return q, scale


def _int8(g, n, k):
    q = torch.randint(-127, 128, (n, k), dtype=torch.int8, device=DEVICE, generator=g)
    scale = (torch.rand(n, generator=g, device=DEVICE) + 0.5) * (0.02 / 73)
    return q, scale.to(torch.bfloat16)


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = {"case": case}
    if op == QUANTIZE:
        n, k = case["n"], case["k"]
        s["w"] = _normal(g, n, k, sigma=0.02, dtype=torch.float32 if case["source"] == "f32" else torch.bfloat16)
        s["q"] = torch.empty(n, k // 2, dtype=torch.uint8, device=DEVICE)
        s["scale"] = torch.empty(n, k // GROUP, dtype=torch.uint8, device=DEVICE)
        s["y"] = torch.empty(n, k, dtype=torch.bfloat16, device=DEVICE)
    elif op == PRODUCT:
        m, n, k = case["m"], case["n"], case["k"]
        s["q"], s["scale"] = _weights(g, n, k)
        s["x"], s["x_scale"] = _normal(g, m, k), None
        if case["x"] == "mxfp4":
            s["x"], s["x_scale"] = _codes(s["x"])
        s["y"] = torch.empty(m, n, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=DEVICE)
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_gemm_mxfp4_prepare(s["x"], s["q"], s["scale"], s["y"], x_scale=s["x_scale"])
    elif op == MOE:
        t, e, dim, f, top = (case[x] for x in ("tokens", "experts", "dim", "f", "top"))
        make = _weights if case["weights"] == "mxfp4" else _int8
        s["w13"], s["s13"] = (x.view(e, 2 * f, *x.shape[1:]) for x in make(g, e * 2 * f, dim))
        s["w2"], s["s2"] = (x.view(e, dim, *x.shape[1:]) for x in make(g, e * dim, f))
        s["x"] = _normal(g, t, dim)
        s["router"] = _normal(g, e, dim, sigma=1.5 * dim ** -0.5)
        s["logits"] = _normal(g, t, e, sigma=1.5, dtype=torch.float32)
        s["router" if case["scores"] == "logits" else "logits"] = None
        s["y"] = torch.empty(t, dim, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=DEVICE)
        s["sel"] = torch.empty(t, top, dtype=torch.int32, device=DEVICE)
        s["gates"] = torch.empty(t, top, dtype=torch.float32, device=DEVICE)
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_moe_ffn_prepare(s["x"], s["w13"], s["s13"], s["w2"], s["s2"], s["y"], top=top,
                                              router=s["router"], logits=s["logits"], sel=s["sel"], gates=s["gates"])
    else:
        rows, dim = case["rows"], case["dim"]
        types = {"f32": torch.float32, "bf16": torch.bfloat16}
        s["h"] = _normal(g, rows, dim, sigma=3.0, dtype=types[case["h"]])
        s["f"] = _normal(g, rows, dim, dtype=types[case["f"]])
        s["f_norm"] = _normal(g, dim, sigma=0.1) + 1 if case["post"] else None
        s["norm"] = _normal(g, dim, sigma=0.1) + 1
        s["gate"] = None if case["gate"] == "none" else _normal(g, rows, dim)
        s["h_out"] = torch.empty_like(s["h"])
        s["u"] = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEVICE)
        s["q"] = torch.empty(rows, dim // 2, dtype=torch.uint8, device=DEVICE) if case["u"] == "mxfp4" else None
        s["scale"] = torch.empty(rows, dim // GROUP, dtype=torch.uint8, device=DEVICE) if case["u"] == "mxfp4" else None
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_block_norm_prepare(
                s["h"], h_out=s["h_out"], f=s["f"], f_norm=s["f_norm"], gate=s["gate"],
                gate_kind="plain" if case["gate"] == "none" else case["gate"], scale=0.75, norm=s["norm"],
                u=s["u"] if case["u"] == "bf16" else None, q=s["q"], q_scale=s["scale"], eps=1e-6)
    return s


# --- one pass --------------------------------------------------------------


def run(s):
    c = s["case"]
    if own:
        import weight_only_quantized_wq_amd as wq
        if c["op"] == QUANTIZE:
            f32 = c["source"] == "f32"
            wq.wq_quantize_mxfp4(s["w"] if f32 else None, None if f32 else s["w"], c["n"], c["k"], s["q"], s["scale"])
            wq.wq_dequantize_mxfp4(s["q"], s["scale"], c["n"], c["k"], None, s["y"])
            return s["y"]
        if c["op"] == PRODUCT:
            wq.wq_gemm_mxfp4_run(s["plan"])
            return s["y"]
        if c["op"] == MOE:
            wq.wq_moe_ffn_run(s["plan"])
            return {"y": s["y"], "sel": s["sel"], "gates": s["gates"]}
        wq.wq_block_norm_run(s["plan"])
        if c["u"] == "mxfp4":
            wq.wq_dequantize_mxfp4(s["q"], s["scale"], c["rows"], c["dim"], None, s["u"])
        return {"h": s["h_out"], "u": s["u"]}
    if c["op"] == QUANTIZE:
        return _values(*_codes(s["w"])).to(torch.bfloat16)
    if c["op"] == PRODUCT:
        x = s["x"].float() if s["x_scale"] is None else _values(s["x"], s["x_scale"])
        return (x @ _values(s["q"], s["scale"]).T).to(s["y"].dtype)
    if c["op"] == MOE:
        return _moe(s)
    return _norm(s)


def _values(q, scale):
    """What MXFP4 codes stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=DEVICE)
    code = torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], -1, GROUP)
    return (table[code.int()] * _power(scale.int() - 127)[..., None]).flatten(-2)


def _expert_weights(s, name, scale, e):
    w, sc = s[name][e], s[scale][e]
    return _values(w, sc) if s["case"]["weights"] == "mxfp4" else w.float() * sc.float()[..., None]


def _moe(s):
    c = s["case"]
    x, f = s["x"].float(), c["f"]
    # scores next to each other decide which experts run
    scores = s["logits"].double() if s["router"] is None else s["x"].double() @ s["router"].double().T
    order = torch.sort(scores, dim=-1, descending=True, stable=True)
    sel = order.indices[:, :c["top"]]
    gates = torch.softmax(order.values[:, :c["top"]], -1).float()
    y = torch.zeros(x.shape, device=DEVICE)
    if c["tokens"] * c["top"] < c["experts"]:
        # few rows: the weights that each (token, expert) uses
        for j in range(c["top"]):
            h = (_expert_weights(s, "w13", "s13", sel[:, j]) @ x[..., None])[..., 0]
            a = h[:, :f] / (1 + torch.exp(-h[:, :f])) * h[:, f:]
            y += gates[:, j, None] * (_expert_weights(s, "w2", "s2", sel[:, j]) @ a[..., None])[..., 0]
    else:
        # every expert over every token, those it is not for weighted by zero
        for e in range(c["experts"]):
            gate = ((sel == e) * gates).sum(-1, keepdim=True)
            h = x @ _expert_weights(s, "w13", "s13", e).T
            a = h[:, :f] / (1 + torch.exp(-h[:, :f])) * h[:, f:]
            y += gate * (a @ _expert_weights(s, "w2", "s2", e).T)
    return {"y": y.to(s["y"].dtype), "sel": sel.to(torch.int32), "gates": gates}


def _norm(s):
    c = s["case"]
    # 64 bits where the result is rounded to 4: values next to a border
    wide = torch.float64 if c["u"] == "mxfp4" else torch.float32
    f = s["f"].to(wide)
    if s["f_norm"] is not None:
        f = f / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6) * s["f_norm"].to(wide)
    if s["gate"] is not None:
        gate = s["gate"].to(wide)
        turned = 1 / (1 + torch.exp(-gate))
        f = f * {"plain": gate, "sigmoid": turned, "silu": gate * turned}[c["gate"]]
    h = s["h"].to(wide) + 0.75 * f
    u = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["norm"].to(wide)
    if c["u"] == "mxfp4":
        u = _rounded(u)
    return {"h": h.to(s["h"].dtype), "u": u.to(torch.bfloat16)}


def _rounded(u):
    """64-bit values as MXFP4 stands for them."""
    groups = u.view(u.shape[0], -1, GROUP)
    power = (torch.frexp(groups.abs().amax(-1, keepdim=True)).exponent - 3).clamp(min=-126)
    return (_steps(groups * _power(-power)) * _power(power)).view(u.shape)


# --- in 64 bits, from the definitions --------------------------------------


def _nearest(w):
    """Each group of 32 under its power of two, every value at the nearest of the fifteen that 4 bits hold."""
    w = w.double().reshape(-1, GROUP)
    largest = w.abs().amax(-1, keepdim=True)
    power = torch.floor(torch.log2(largest.clamp(min=2.0 ** -1000)))
    # log2 is rounded: make sure of 2^power <= largest < 2^(power + 1)
    power = torch.where(torch.pow(2.0, power) > largest, power - 1, power)
    power = torch.where(torch.pow(2.0, power + 1) <= largest, power + 1, power)
    unit = torch.pow(2.0, (power - 2).clamp(min=-127))
    size, best = (w / unit).abs(), torch.zeros_like(w)
    # (candidate, smallest size that rounds to it, whether a tie does)
    for value, border, tie in ((0.5, 0.25, False), (1.0, 0.75, True), (1.5, 1.25, False), (2.0, 1.75, True),
                               (3.0, 2.5, False), (4.0, 3.5, True), (6.0, 5.0, False)):
        best = torch.where((size >= border) if tie else (size > border), torch.full_like(best, value), best)
    return torch.copysign(best, w) * unit


def _stand_for(q, scale):
    """Values of MXFP4 rows from the bits: sign, exponent and mantissa of each code."""
    q = q.reshape(-1, q.shape[-1])
    code = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=DEVICE)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    exponent, mantissa = code >> 1 & 3, (code & 1).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.pow(2.0, (exponent - 1).double()))
    unit = torch.pow(2.0, scale.reshape(q.shape[0], -1).double() - 127).repeat_interleave(GROUP, 1)
    return torch.where(code >= 8, -size, size) * unit


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == QUANTIZE:
        w, rows = s["w"], max(1, (1 << 25) // case["k"])
        return torch.cat([_nearest(w[a:a + rows]) for a in range(0, w.shape[0], rows)]).view(w.shape)
    if case["op"] == PRODUCT:
        x = s["x"].double() if s["x_scale"] is None else _stand_for(s["x"], s["x_scale"])
        y, rows = torch.empty(s["y"].shape, dtype=torch.float64, device=DEVICE), 4096
        for a in range(0, case["n"], rows):
            y[:, a:a + rows] = torch.mm(x, _stand_for(s["q"][a:a + rows], s["scale"][a:a + rows]).t())
        return y
    if case["op"] == MOE:
        x, f = s["x"].double(), case["f"]

        def matrix(name, scale, e):
            if case["weights"] == "mxfp4":
                return _stand_for(s[name][e], s[scale][e])
            return s[name][e].double() * s[scale][e].double()[:, None]

        scores = s["logits"].double() if s["router"] is None else torch.mm(x, s["router"].double().t())
        rows = scores.cpu().tolist()
        picked = [sorted(range(len(r)), key=lambda e, r=r: (-r[e], e))[:case["top"]] for r in rows]
        weight = [[math.exp(r[e] - r[p[0]]) for e in p] for r, p in zip(rows, picked)]
        gates = [[v / sum(w) for v in w] for w in weight]
        y = torch.zeros(x.shape, dtype=torch.float64, device=DEVICE)
        for e in sorted({e for p in picked for e in p}):
            at = [(t, p.index(e)) for t, p in enumerate(picked) if e in p]
            who = torch.tensor([t for t, _ in at], device=DEVICE)
            share = torch.tensor([gates[t][j] for t, j in at], dtype=torch.float64, device=DEVICE)
            h = torch.mm(x[who], matrix("w13", "s13", e).t())
            a = h[:, :f] * torch.sigmoid(h[:, :f]) * h[:, f:]
            y[who] += share[:, None] * torch.mm(a, matrix("w2", "s2", e).t())
        return {"y": y, "sel": None, "gates": torch.tensor(gates, dtype=torch.float64, device=DEVICE)}
    h, f = s["h"].double(), s["f"].double()
    if case["post"]:
        f *= torch.rsqrt(f.square().mean(-1) + 1e-6)[:, None] * s["f_norm"].double()
    if case["gate"] != "none":
        gate = s["gate"].double()
        f *= gate if case["gate"] == "plain" else torch.sigmoid(gate) * (gate if case["gate"] == "silu" else 1)
    h += 0.75 * f
    u = h * torch.rsqrt(h.square().mean(-1) + 1e-6)[:, None] * s["norm"].double()
    return {"h": h, "u": _nearest(u).view(u.shape) if case["u"] == "mxfp4" else u}
