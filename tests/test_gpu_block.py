"""MXFP4 quantiser and products, the expert layer and the norm around a block on the GPU against oracle/block.py.

Tolerances, fixed before the first run.  A rounding to bf16 is off by at most
2^-8 of the value, one to fp32 by 2^-24.

* quantisation and its inverse: none, every code and value is exact.
* product: operands are exact in what the matrix cores take (bf16 pairs, or
  codes and scales), so a result differs by the roundings of its fp32 sum, at
  most (k + 16) 2^-23 of sum |x w| (additions that truncate count double), and
  one rounding to bf16 where that is asked for.
* expert layer: h1 and h3 as products; |silu'| <= 1.1 carries their errors to
  a = silu(h1) h3, whose own exp, quotient and products add 2^-19 |a|; a is
  carried in 24 bits (2^-23 |a|; 2^-16 |a| where only bf16 is asked for); the
  second product adds its sum's roundings, (3 f + 16) 2^-23 of sum |a w|, and
  the gate 2^-19; then a rounding to bf16.  Selections are exact.
* norm: fp32 elements through at most 16 roundings and an exp each (2^-19 of
  every term, |h| and |scale act(gate) norm(f)|), a factor good to 2^-19, a
  rounding to bf16; where MXFP4 is asked for the codes of the fp64 formula.
"""

import numpy as np
import pytest

from oracle import block

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_wq_amd as m
    return m


def bf16(a):
    """(float64 values of the nearest bf16, device tensor of them)"""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def f32(a):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.double().numpy(), t.cuda()


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def empty(*shape, dtype="float32", fill=None):
    import torch
    t = torch.empty(shape, dtype=getattr(torch, dtype), device="cuda")
    return t if fill is None else t.fill_(fill)


def within(got, want, allowed, what):
    off = np.abs(got - want) - allowed
    worst = np.unravel_index(np.nanargmax(off), off.shape) if off.size else None
    assert not off.size or (np.isfinite(got).all() and off[worst] <= 0), \
        f"{what}: {got[worst]} for {want[worst]} at {worst}, allowed {np.broadcast_to(allowed, off.shape)[worst]}"


def mx(rng, n, k, spread=3):
    """Random codes and scales around 1, as arrays; all 16 codes occur."""
    q = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    s = rng.integers(127 - spread, 128 + spread, (n, k // 32), dtype=np.uint8)
    return q, s


# --- quantisation ----------------------------------------------------------

GROUPS_AT = 32


def _borders(rng):
    """Groups whose values lie on, just below and just above every border, over the whole range of scales."""
    rows = []
    for e in list(range(-130, 126, 7)) + [-149, -148, -127, -126, -125, 124, 125]:
        base = np.arange(0, 64) / 8.0                       # in units of 2^e
        with np.errstate(over="ignore"):
            v = (base * 2.0 ** e).astype(np.float32)
        v = np.where(np.isfinite(v), v, np.finfo(np.float32).max).astype(np.float32)
        rows += [v, np.nextafter(v, np.float32(np.inf)), -np.nextafter(v, np.float32(0))]
    w = np.stack(rows).astype(np.float32)
    w[~np.isfinite(w)] = np.finfo(np.float32).max
    return rng.permuted(w, axis=1)


def _check_quantise(wq, w, tensor, source):
    n, k = w.shape
    q, s = empty(n, k // 2, dtype="uint8", fill=7), empty(n, k // 32, dtype="uint8", fill=7)
    wq.wq_quantize_mxfp4(*((tensor, None) if source == "f32" else (None, tensor)), n, k, q, s)
    want_q, want_s = block.mx_quantize(w)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)
    for kind in ("float32", "bfloat16"):
        y = empty(n, k, dtype=kind)
        wq.wq_dequantize_mxfp4(q, s, n, k, *((y, None) if kind == "float32" else (None, y)))
        assert np.array_equal(f64(y), block.mx_values(want_q, want_s), equal_nan=True)


@pytest.mark.parametrize("source", ["f32", "bf16"])
@pytest.mark.parametrize("n,k", [(1, 32), (3, 64), (5, 96), (37, 416), (2, 4096), (130, 1056)])
def test_quantise_random(wq, n, k, source):
    rng = np.random.default_rng(n * k)
    w, t = (f32 if source == "f32" else bf16)(rng.normal(0, 0.02, (n, k)))
    _check_quantise(wq, w, t, source)


@pytest.mark.parametrize("source", ["f32", "bf16"])
def test_quantise_at_every_border(wq, source):
    w, t = (f32 if source == "f32" else bf16)(_borders(np.random.default_rng(5)))
    if source == "bf16":
        w = np.where(np.isfinite(w), w, 0)              # the largest fp32 rounds past bf16's range
        import torch
        t = torch.where(torch.isfinite(t), t, torch.zeros_like(t))
    _check_quantise(wq, w, t, source)


@pytest.mark.parametrize("source", ["f32", "bf16"])
def test_quantise_zeros_infinities_and_nan(wq, source):
    w = np.random.default_rng(6).normal(0, 1, (4, 128))
    w[0] = 0.0
    w[0, 40] = -0.0
    w[1, 7], w[1, 70], w[2, 33], w[3, 127] = np.inf, -np.inf, np.nan, np.nan
    w, t = (f32 if source == "f32" else bf16)(w)
    _check_quantise(wq, w, t, source)


def test_every_code_under_every_scale(wq):
    q = np.tile(np.arange(0, 16, 2, dtype=np.uint8) | np.arange(1, 17, 2, dtype=np.uint8) << 4, (256, 2))
    s = np.arange(256, dtype=np.uint8)[:, None]
    with np.errstate(over="ignore"):
        want = block.mx_values(q, s).astype(np.float32).astype(np.float64)
    for kind in ("float32", "bfloat16"):
        y = empty(256, 32, dtype=kind)
        wq.wq_dequantize_mxfp4(up(q), up(s), 256, 32, *((y, None) if kind == "float32" else (None, y)))
        assert np.array_equal(f64(y), want, equal_nan=True)


# --- products --------------------------------------------------------------


def _product(wq, rng, m, n, k, xkind, out, pad=0):
    import torch
    q, s = mx(rng, n, k)
    w = block.mx_values(q, s)
    if xkind == "bf16":
        x, xt = bf16(rng.normal(0, 1, (m, k)))
        if pad:
            wide = torch.full((m, k + 8 * pad), float("nan"), dtype=torch.bfloat16, device="cuda")
            wide[:, :k] = xt
            xt = wide[:, :k]
        xs = None
    else:
        xq, xsc = mx(rng, m, k, spread=2)
        x, xt, xs = block.mx_values(xq, xsc), up(xq), up(xsc)
    both = out == "both"
    stride = n + 5 * pad
    wide = {kind: torch.full((m + 2, stride), 777.0, dtype=getattr(torch, kind), device="cuda") for kind in ("float32", "bfloat16")}
    y32, y16 = (wide[kind][1:m + 1, :n] for kind in ("float32", "bfloat16"))
    plan = wq.wq_gemm_mxfp4_prepare(xt, up(q), up(s), y32 if out != "bf16" else y16, y2=y16 if both else None, x_scale=xs)
    wq.wq_gemm_mxfp4_run(plan)
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    sums = (k + 16) * 2.0 ** -23 * size
    if out != "bf16":
        within(f64(y32), want, sums, "fp32")
    if out != "f32":
        within(f64(y16), want, sums + BF16 * (np.abs(want) + sums), "bf16")
    if both:
        assert torch.equal(y32.to(torch.bfloat16), y16)
    for kind in wide:
        written = torch.zeros_like(wide[kind], dtype=torch.bool)
        if out == "both" or (out == "f32") == (kind == "float32"):
            written[1:m + 1, :n] = True
        assert (wide[kind][~written] == 777.0).all()
    first = {kind: wide[kind].clone() for kind in wide}
    wq.wq_gemm_mxfp4_run(plan)
    assert all(torch.equal(first[kind], wide[kind]) for kind in wide), "a second run differs"


SHAPES = [(1, 1, 32), (1, 16, 64), (1, 17, 96), (2, 33, 128), (3, 100, 160), (4, 256, 512), (5, 129, 544), (8, 64, 1024),
          (7, 515, 1056), (9, 48, 2080), (15, 31, 512), (16, 1000, 4096), (1, 4100, 4096), (17, 70, 1504), (33, 130, 2048),
          (63, 257, 608), (64, 128, 8192), (65, 96, 160), (129, 515, 1056), (200, 300, 2560), (257, 260, 96), (515, 129, 640),
          (300, 260, 4096), (2051, 5600, 96), (1030, 12010, 64), (4100, 2900, 672),
          (2051, 5600, 512), (600, 20000, 1024), (500, 4000, 512), (500, 4000, 544),
          # tiles of 256 x 128, and large tiles over shares of k, with rows that end inside a stage and without
          (770, 5140, 1056), (1300, 1540, 2080), (1800, 1030, 4096), (770, 5140, 4128), (1800, 515, 8224), (770, 4100, 4096)]


@pytest.mark.parametrize("xkind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(wq, m, n, k, xkind):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    _product(wq, rng, m, n, k, xkind, ["f32", "bf16", "both"][(m + n) % 3], pad=(m + n) % 2)


# --- expert layer ----------------------------------------------------------


def _experts(rng, e, rows, k, weights):
    """(values [e, rows, k], device tensors)"""
    if weights == "mxfp4":
        q, s = mx(rng, e * rows, k, spread=2)
        v = block.mx_values(q, s).reshape(e, rows, k) * 2.0 ** -5
        s -= 5
        return v, (up(q.reshape(e, rows, -1)), up(s.reshape(e, rows, -1)))
    q = rng.integers(-127, 128, (e, rows, k), dtype=np.int8)
    s, st = bf16(rng.uniform(0.5, 1.5, (e, rows)) * 2.0 ** -9)
    return q * s[..., None], (up(q), st)


def _moe_allowed(x, w13, w2, sel, gates, want, parts, out):
    f, k = w2.shape[2], w13.shape[2]
    allowed = np.zeros(want.shape)
    for t in range(x.shape[0]):
        for e, g in zip(sel[t], gates[t]):
            h = w13[e] @ x[t]
            dh = (k + 16) * 2.0 ** -23 * (np.abs(w13[e]) @ np.abs(x[t]))
            a = np.abs(block.silu(h[:f]) * h[f:])
            da = 1.1 * dh[:f] * (np.abs(h[f:]) + dh[f:]) + np.abs(block.silu(h[:f])) * dh[f:] + a * 2.0 ** -19
            da += a * (2.0 ** -23 if parts == 3 else 2.0 ** -16)
            m = np.abs(w2[e])
            allowed[t] += g * (m @ da + ((3 * f + 16) * 2.0 ** -23 + 2.0 ** -19) * (m @ a))
    return allowed if out == "f32" else allowed + BF16 * (np.abs(want) + allowed)


def _moe(wq, rng, tokens, e, top, dim, f, weights, scores, out, renormalize=True, logits=None, pad=0, router=None):
    import torch
    w13, t13 = _experts(rng, e, 2 * f, dim, weights)
    w2, t2 = _experts(rng, e, dim, f, weights)
    x, xt = bf16(rng.normal(0, 1, (tokens, dim)))
    rt = lt = None
    if scores == "router":
        r, rt = bf16(rng.normal(0, 1.5 * dim ** -0.5, (e, dim)) if router is None else router)
        logits = x @ r.T
    else:
        logits, lt = f32(rng.normal(0, 1.5, (tokens, e)) if logits is None else logits)
    if pad:
        wide = torch.full((tokens, dim + 8 * pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :dim] = xt
        xt = wide[:, :dim]
    stride = dim + 3 * pad
    y32 = torch.full((tokens + 2, stride), 777.0, device="cuda")
    y16 = torch.full((tokens + 2, stride), 777.0, dtype=torch.bfloat16, device="cuda")
    a, b = y32[1:tokens + 1, :dim], y16[1:tokens + 1, :dim]
    sel, gates = empty(tokens, top, dtype="int32", fill=-1), empty(tokens, top, fill=-1)
    plan = wq.wq_moe_ffn_prepare(xt, *t13, *t2, a if out != "bf16" else b, y2=b if out == "both" else None, router=rt,
                                 logits=lt, top=top, renormalize=renormalize, sel=sel, gates=gates)
    wq.wq_moe_ffn_run(plan)
    want, want_sel, want_gates = block.moe_ffn(x, logits, w13, w2, top, renormalize)
    assert np.array_equal(sel.cpu().numpy(), want_sel)
    within(f64(gates), want_gates, 2.0 ** -19 * want_gates + 2.0 ** -126, "gates")
    parts = 2 if out == "bf16" else 3
    if out != "bf16":
        within(f64(a), want, _moe_allowed(x, w13, w2, want_sel, want_gates, want, parts, "f32"), "fp32")
    if out != "f32":
        within(f64(b), want, _moe_allowed(x, w13, w2, want_sel, want_gates, want, parts, "bf16"), "bf16")
    for t, used in ((y32, out != "bf16"), (y16, out != "f32")):
        written = torch.zeros_like(t, dtype=torch.bool)
        written[1:tokens + 1, :dim] = used
        assert (t[~written] == 777.0).all()
    first = y32.clone(), y16.clone(), sel.clone(), gates.clone()
    wq.wq_moe_ffn_run(plan)
    assert all(torch.equal(u, v) for u, v in zip(first, (y32, y16, sel, gates))), "a second run differs"


LAYERS = [(1, 8, 2, 256, 512), (1, 4, 1, 32, 32), (2, 8, 2, 544, 96), (3, 16, 4, 96, 160), (4, 8, 2, 1024, 352),
          (5, 8, 2, 64, 1056), (8, 60, 4, 128, 64), (9, 8, 2, 160, 96), (17, 4, 3, 64, 128), (33, 128, 8, 64, 32),
          (64, 3, 2, 96, 64), (64, 256, 16, 32, 32), (61, 1, 1, 64, 64)]


@pytest.mark.parametrize("weights", ["mxfp4", "int8"])
@pytest.mark.parametrize("tokens,e,top,dim,f", LAYERS)
def test_expert_layer(wq, tokens, e, top, dim, f, weights):
    rng = np.random.default_rng(tokens * 31 + e + dim + f)
    i = tokens + e + (weights == "int8")
    _moe(wq, rng, tokens, e, top, dim, f, weights, ["router", "logits"][i % 2], ["f32", "bf16", "both"][i % 3],
         renormalize=i % 5 != 0, pad=i % 2)


@pytest.mark.parametrize("weights", ["mxfp4", "int8"])
@pytest.mark.parametrize("tokens,e,top,dim,f", LAYERS + [(2, 8, 6, 64, 96), (16, 8, 2, 96, 1056), (50, 8, 2, 64, 512), (20, 64, 6, 64, 96)])
def test_a_bf16_result_is_the_rounded_fp32_result(wq, tokens, e, top, dim, f, weights):
    """What is carried between the products does not depend on the results' type."""
    import torch
    rng = np.random.default_rng(tokens * 5 + e + dim + f)
    _, t13 = _experts(rng, e, 2 * f, dim, weights)
    _, t2 = _experts(rng, e, dim, f, weights)
    _, x = bf16(rng.normal(0, 1, (tokens, dim)))
    _, logits = f32(rng.normal(0, 1.5, (tokens, e)))
    y32, y16 = empty(tokens, dim), empty(tokens, dim, dtype="bfloat16")
    for y in (y32, y16):
        wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x, *t13, *t2, y, logits=logits, top=top))
    assert torch.equal(y32.to(torch.bfloat16), y16)


@pytest.mark.parametrize("tokens", [1, 2, 9])
def test_int8_scales_at_an_odd_element(wq, tokens):
    """Scales that start behind one other bf16, as a slice of a checkpoint's buffer does."""
    import torch
    rng = np.random.default_rng(tokens)
    e, dim, f = 4, 48, 80
    w13, (q13, s13) = _experts(rng, e, 2 * f, dim, "int8")
    w2, (q2, s2) = _experts(rng, e, dim, f, "int8")
    x, xt = bf16(rng.normal(0, 1, (tokens, dim)))
    logits, lt = f32(rng.normal(0, 1.5, (tokens, e)))

    def behind(s):
        t = torch.full((s.numel() + 2,), float("nan"), dtype=s.dtype, device="cuda")
        t[1:-1] = s.flatten()
        return t[1:-1].view(s.shape)
    y = empty(tokens, dim)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(xt, q13, behind(s13), q2, behind(s2), y, logits=lt))
    want, sel, gates = block.moe_ffn(x, logits, w13, w2, 2)
    within(f64(y), want, _moe_allowed(x, w13, w2, sel, gates, want, 3, "f32"), "y")


@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_int8_experts_of_odd_sixteens(wq, tokens):
    _moe(wq, np.random.default_rng(tokens), tokens, 5, 2, 48, 272, "int8", "router", "f32")


@pytest.mark.parametrize("tokens", [2, 12])
def test_ties_infinities_and_nan_among_logits(wq, tokens):
    rng = np.random.default_rng(3)
    logits = rng.integers(-1, 2, (tokens, 70)).astype(np.float64)        # ties everywhere
    logits[0, 5] = -np.inf
    _moe(wq, rng, tokens, 70, 6, 32, 32, "mxfp4", "logits", "f32", logits=logits)


def test_equal_router_rows_tie_to_the_lower_index(wq):
    rng = np.random.default_rng(4)
    row = rng.normal(0, 0.1, (1, 64))
    _moe(wq, rng, 6, 9, 3, 64, 32, "int8", "router", "bf16", router=np.repeat(row, 9, 0))


@pytest.mark.parametrize("e,dim", [(22, 9216), (10, 32768), (129, 4096), (256, 1024), (9, 8192)])
def test_equal_router_rows_score_the_same_in_every_workgroup(wq, e, dim):
    """x with a few inputs 2^40 times the others, whose sums round: equal rows still tie, wherever they are summed."""
    import torch
    rng = np.random.default_rng(e + dim)
    x = rng.normal(0, 1, (64, dim))
    for row in x:
        row[rng.integers(0, dim, 4)] *= 2.0 ** 40
    _, x = bf16(x)
    _, router = bf16(np.repeat(rng.normal(0, 1, (1, dim)), e, 0))
    w13, w2 = torch.zeros(e, 32, dim, dtype=torch.int8, device="cuda"), torch.zeros(e, dim, 16, dtype=torch.int8, device="cuda")
    s13, s2 = torch.ones(e, 32, dtype=torch.bfloat16, device="cuda"), torch.ones(e, dim, dtype=torch.bfloat16, device="cuda")
    y, sel, gates = empty(64, dim), empty(64, 8, dtype="int32", fill=-1), empty(64, 8, fill=-1)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x, w13, s13, w2, s2, y, router=router, top=8, sel=sel, gates=gates))
    assert (sel.cpu() == torch.arange(8)).all() and (gates == 0.125).all()


@pytest.mark.parametrize("tokens", [2, 30])
def test_nan_logits_select_distinct_experts_in_range(wq, tokens):
    import torch
    w13, w2 = torch.zeros(4, 64, 32, dtype=torch.int8, device="cuda"), torch.zeros(4, 32, 32, dtype=torch.int8, device="cuda")
    s13, s2 = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(4, 32, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(tokens, 32, dtype=torch.bfloat16, device="cuda")
    logits = torch.full((tokens, 4), float("nan"), device="cuda")
    logits[1] = torch.tensor([float("nan"), 1.0, float("-inf"), float("nan")])
    sel, y = empty(tokens, 3, dtype="int32", fill=-1), empty(tokens, 32)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x, w13, s13, w2, s2, y, logits=logits, top=3, sel=sel))
    got = sel.cpu().tolist()
    assert got[0] == [0, 1, 2] and got[1] == [1, 2, 0]


@pytest.mark.parametrize("weights", ["mxfp4", "int8"])
@pytest.mark.parametrize("tokens,e,top", [(64, 64, 4), (37, 8, 2), (64, 2, 1), (23, 100, 3), (64, 16, 16), (6, 8, 1)])
def test_all_tokens_at_the_same_experts(wq, tokens, e, top, weights):
    """Routing as uneven as it gets, and every expert at once, where plans expect them alike."""
    logits = np.tile(np.random.default_rng(e).normal(0, 1.5, (1, e)), (tokens, 1))
    _moe(wq, np.random.default_rng(tokens + e), tokens, e, top, 64, 96, weights, "logits", "both", logits=logits)


def test_layers_in_turn_captured_over_one_workspace(wq):
    """Two layers of other sizes through one workspace, in a graph each, replayed in turn and after eager calls."""
    import torch
    rng = np.random.default_rng(21)
    sizes = [(30, 8, 2, 96, 256), (2, 16, 4, 160, 64), (1, 4, 2, 64, 352)]
    ws = torch.empty(max(wq.wq_moe_ffn_workspace_bytes(t, dim, f, e, top) for t, e, top, dim, f in sizes), dtype=torch.uint8,
                     device="cuda")
    plans, graphs, outs, wants = [], [], [], []
    for t, e, top, dim, f in sizes:
        w13, t13 = _experts(rng, e, 2 * f, dim, "mxfp4")
        w2, t2 = _experts(rng, e, dim, f, "mxfp4")
        x, xt = bf16(rng.normal(0, 1, (t, dim)))
        r, rt = bf16(rng.normal(0, dim ** -0.5, (e, dim)))
        y = empty(t, dim)
        plans.append(wq.wq_moe_ffn_prepare(xt, *t13, *t2, y, router=rt, top=top, workspace=ws))
        want, sel, gates = block.moe_ffn(x, x @ r.T, w13, w2, top)
        outs.append(y)
        wants.append((want, _moe_allowed(x, w13, w2, sel, gates, want, 3, "f32")))
    for p in plans:
        wq.wq_moe_ffn_run(p)
    torch.cuda.synchronize()
    for p in plans:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            wq.wq_moe_ffn_run(p)
    for _ in range(3):
        for y in outs:
            y.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for y, (want, allowed) in zip(outs, wants):
            within(f64(y), want, allowed, "replay")
        for y, p in zip(outs, plans):
            y.fill_(9)
            wq.wq_moe_ffn_run(p)
        torch.cuda.synchronize()
        for y, (want, allowed) in zip(outs, wants):
            within(f64(y), want, allowed, "call")


def test_large_activations_between_the_products_keep_their_values(wq):
    """silu(h1) h3 next to the largest fp32, which no bf16 rounded to nearest reaches."""
    import torch
    w13 = torch.zeros(1, 64, 32, dtype=torch.int8, device="cuda")
    w13[0, :, 0] = 1
    s13 = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    s13[0, 32:] = 1 + 2.0 ** -7
    w2 = torch.zeros(1, 32, 32, dtype=torch.int8, device="cuda")
    w2[0, torch.arange(32), torch.arange(32)] = 1
    s2 = torch.full((1, 32), 0.5, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(1, 32, dtype=torch.bfloat16, device="cuda")
    # 2^64 (1 - 2^-8): times itself and 1 + 2^-7 it is 2^128 (1 - 2^-14 + ...), past the largest bf16, 2^128 (1 - 2^-8),
    # and its rounding border, 2^128 (1 - 2^-9)
    x[0, 0] = 2.0 ** 64 * (1 - 2.0 ** -8)
    y = empty(1, 32)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x, w13, s13, w2, s2, y, logits=torch.zeros(1, 1, device="cuda"), top=1))
    a = float(x[0, 0].double()) ** 2 * (1 + 2.0 ** -7)
    assert 2.0 ** 128 * (1 - 2.0 ** -9) < a < float(torch.finfo(torch.float32).max)
    want = a * 0.5
    within(f64(y), np.full((1, 32), want), 2.0 ** -18 * want, "large")


# --- norm ------------------------------------------------------------------


def _block(wq, rng, rows, dim, h="f32", f="bf16", post=True, gate="sigmoid", u="bf16", out=True, norm=True, scale=0.75,
           eps=1e-6, pad=0, wide_gate=True, in_place=False, size=3.0):
    import torch
    make = {"f32": f32, "bf16": bf16}
    hv, ht = make[h](rng.normal(0, size, (rows, dim)))
    fv, ft = make[f](rng.normal(0, 1, (rows, dim))) if f else (None, None)
    pv, pt = bf16(rng.normal(1, 0.1, dim)) if f and post else (None, None)
    gv, gt = bf16(rng.normal(0, 2, (rows, dim) if wide_gate else dim)) if f and gate != "none" else (None, None)
    nv, nt = bf16(rng.normal(1, 0.1, dim)) if norm else (None, None)
    kind = "plain" if gate == "none" else gate

    def padded(t):
        if not pad or t is None or t.dim() < 2:
            return t
        w = torch.full((rows, dim + 8 * pad), float("nan"), dtype=t.dtype, device="cuda")
        w[:, :dim] = t
        return w[:, :dim]
    ht, ft, gt = padded(ht), padded(ft), padded(gt)
    ot = ht if in_place else padded(torch.zeros(rows, dim, dtype=ht.dtype, device="cuda")) if out else None
    ut = padded(torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")) if "bf16" in u else None
    q, qs = (empty(rows, dim // 2, dtype="uint8", fill=7), empty(rows, dim // 32, dtype="uint8", fill=7)) if "mxfp4" in u else (None, None)
    plan = wq.wq_block_norm_prepare(ht, h_out=ot, f=ft, f_norm=pt, gate=gt, gate_kind=kind, scale=scale, norm=nt, u=ut, q=q,
                                    q_scale=qs, eps=eps)
    wq.wq_block_norm_run(plan)
    # scale and eps are fp32 numbers
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    want_h, want_u = block.block_norm(hv, fv, pv, gv, kind, scale, nv, eps)
    added = want_h - hv
    dh = 2.0 ** -19 * (np.abs(hv) + np.abs(added)) + 1e-40
    if ot is not None:
        within(f64(ot), want_h, dh + (BF16 * (np.abs(want_h) + dh) if h == "bf16" else 0), "h")
    if ut is not None:
        r = np.abs(want_u / np.where(want_h == 0, 1, want_h))
        du = r * dh + 2.0 ** -18 * np.abs(want_u)
        within(f64(ut), want_u, du + BF16 * (np.abs(want_u) + du), "u")
    if q is not None:
        want_q, want_s = block.mx_quantize(want_u)
        assert np.array_equal(qs.cpu().numpy(), want_s)
        assert np.array_equal(q.cpu().numpy(), want_q)


NORMS = [(1, 8), (1, 4096), (2, 520), (3, 32), (5, 1024), (7, 2048), (13, 4104), (4, 8192), (2, 16384), (3, 20000), (1, 32768),
         (300, 64)]


@pytest.mark.parametrize("rows,dim", NORMS)
@pytest.mark.parametrize("gate", ["none", "plain", "sigmoid", "silu"])
def test_block_norm(wq, rows, dim, gate):
    rng = np.random.default_rng(rows + dim)
    i = rows + dim // 8
    u = ["bf16", "mxfp4", "bf16+mxfp4"][i % 3] if dim % 32 == 0 else "bf16"
    _block(wq, rng, rows, dim, h=["f32", "bf16"][i % 2], f=["bf16", "f32"][i // 2 % 2], post=i % 5 != 0, gate=gate, u=u,
           pad=i % 2, norm=i % 7 != 0, wide_gate=i % 4 != 1)


@pytest.mark.parametrize("h", ["f32", "bf16"])
def test_block_norm_in_place_without_f_and_without_norm(wq, h):
    rng = np.random.default_rng(1)
    _block(wq, rng, 9, 264, h=h, in_place=True)
    _block(wq, rng, 9, 264, h=h, f=None, out=False)
    _block(wq, rng, 9, 288, h=h, u="", norm=False)
    _block(wq, rng, 9, 288, h=h, u="mxfp4", out=False, norm=False, f=None)


@pytest.mark.parametrize("q", [False, True])
@pytest.mark.parametrize("h,out", [("f32", "bf16"), ("bf16", "f32")])
def test_block_norm_of_one_type_into_the_other(wq, h, out, q):
    import torch
    rng = np.random.default_rng(17)
    make = {"f32": f32, "bf16": bf16}
    hv, ht = make[h](rng.normal(0, 3, (5, 288)))
    fv, ft = make[out](rng.normal(0, 1, (5, 288)))
    got = empty(5, 288, dtype={"f32": "float32", "bf16": "bfloat16"}[out])
    codes, scale = (empty(5, 144, dtype="uint8"), empty(5, 9, dtype="uint8")) if q else (None, None)
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(ht, h_out=got, f=ft, scale=0.5, q=codes, q_scale=scale))
    want, u = block.block_norm(hv, fv, scale=0.5, eps=float(np.float32(1e-6)))
    # a product by a power of two and a sum, in fp32 or fp64, then the result's rounding
    within(f64(got), want, 2.0 ** -23 * np.abs(want) + (BF16 if out == "bf16" else 0) * np.abs(want) * (1 + 2.0 ** -23), out)
    if q:
        want_q, want_s = block.mx_quantize(u)
        assert np.array_equal(scale.cpu().numpy(), want_s) and np.array_equal(codes.cpu().numpy(), want_q)
    assert torch.equal(ht.double().cpu(), torch.from_numpy(hv))


@pytest.mark.parametrize("size", [1e-30, 1e30])
@pytest.mark.parametrize("u", ["bf16", "mxfp4"])
def test_block_norm_of_tiny_and_huge_rows(wq, size, u):
    _block(wq, np.random.default_rng(2), 3, 512, f=None, out=False, u=u, eps=0.0, size=size)


def test_zero_rows_and_rows_of_zeros(wq):
    import torch
    h, u = torch.zeros(2, 64, device="cuda"), empty(2, 64, dtype="bfloat16", fill=5)
    q, s = empty(2, 32, dtype="uint8", fill=7), empty(2, 2, dtype="uint8", fill=7)
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(h, u=u, q=q, q_scale=s))
    assert not u.any() and not q.any() and not s.any()
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(h[:0], u=u[:0]))


def test_an_infinity_or_nan_stays_in_its_row_and_group(wq):
    import torch
    h = torch.randn(3, 128, device="cuda")
    f = torch.zeros(3, 128, device="cuda")
    f[1, 40] = float("nan")
    out, u = torch.empty_like(h), empty(3, 128, dtype="bfloat16")
    q, s = empty(3, 64, dtype="uint8", fill=7), empty(3, 4, dtype="uint8", fill=7)
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(h, h_out=out, f=f, u=u, q=q, q_scale=s))
    bad = torch.isnan(out)
    assert bad[1, 40] and bad.sum() == 1
    assert torch.isnan(u[1]).all() and torch.isfinite(u[[0, 2]]).all()
    assert (s[1] == 255).all() and (q[1] == 0).all() and (s[[0, 2]] != 255).all()


# --- what must not reach other rows ----------------------------------------


@pytest.mark.parametrize("xkind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(4, 40, 96), (16, 40, 544), (40, 140, 1056), (2050, 5500, 96), (1300, 1540, 2080),
                                   (1800, 515, 8224)])
def test_infinities_and_nan_stay_in_their_rows_and_columns(wq, m, n, k, xkind):
    """Rows of x with NaN and infinities between rows without (rows that end inside a stage read on past their end), rows
    of W with a NaN group."""
    import torch
    rng = np.random.default_rng(m + k)
    q, s = mx(rng, n, k)
    s[1::7, -1] = 255
    if xkind == "bf16":
        x, xt = bf16(rng.normal(0, 1, (m, k)))
        xt[1::2] = float("nan")
        xt[2::4, 0] = float("inf")
        xs, bad = None, np.isnan(f64(xt)).any(1) | np.isinf(f64(xt)).any(1)
    else:
        xq, xsc = mx(rng, m, k, spread=2)
        xsc[1::2, 0] = 255
        x, xt, xs = block.mx_values(xq, xsc), up(xq), up(xsc)
        bad = np.isnan(x).any(1)
    y = empty(m, n, fill=5)
    wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(xt, up(q), up(s), y, x_scale=xs))
    got = f64(y)
    gone = (s == 255).any(1)
    assert np.isnan(got[:, gone]).all()
    fine = ~bad[:, None] & ~gone[None]
    w = block.mx_values(q, np.where(s == 255, 127, s))
    x = np.where(np.isfinite(x) & ~bad[:, None], x, 0)
    size = np.abs(x) @ np.abs(w).T
    within(np.where(fine, got, 0), np.where(fine, x @ w.T, 0), (k + 16) * 2.0 ** -23 * size, "rows beside")
    assert not np.isfinite(got[bad]).any()


def test_a_token_of_nan_leaves_the_others_alone(wq):
    rng = np.random.default_rng(8)
    w13, t13 = _experts(rng, 4, 2 * 64, 96, "mxfp4")
    w2, t2 = _experts(rng, 4, 96, 64, "mxfp4")
    x, xt = bf16(rng.normal(0, 1, (12, 96)))
    logits, lt = f32(rng.normal(0, 1, (12, 4)))
    xt[5] = float("nan")
    y = empty(12, 96)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(xt, *t13, *t2, y, logits=lt))
    x[5] = 0
    want, sel, gates = block.moe_ffn(x, logits, w13, w2, 2)
    got = f64(y)
    assert np.isnan(got[5]).all()
    got[5] = want[5] = 0
    within(got, want, _moe_allowed(x, w13, w2, sel, gates, want, 3, "f32"), "others")


def test_an_infinite_activation_between_the_products_is_no_nan_by_its_parts(wq):
    import torch
    w13 = torch.zeros(1, 64, 32, dtype=torch.int8, device="cuda")
    w13[0, :, 0] = 127
    s13 = torch.full((1, 64), 2.0 ** 100, dtype=torch.bfloat16, device="cuda")
    w2, s2 = torch.ones(1, 32, 32, dtype=torch.int8, device="cuda"), torch.ones(1, 32, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(2, 32, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([1.0, -1.0])
    y = empty(2, 32)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x, w13, s13, w2, s2, y, logits=torch.zeros(2, 1, device="cuda"), top=1))
    # silu(2^107) * 2^107 is infinite; silu(-2^107) is -0
    assert (y[0] == float("inf")).all() and (y[1] == 0).all()


# --- far offsets, streams, graphs, shared workspaces -----------------------


def test_offsets_past_32_bits(wq):
    """Weights of 4.6 GB: their last rows, for one row of x and for many; the quantiser over 4.4 billion values."""
    import torch
    n, k = 280000, 32768
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.randint(125, 130, (n, k // 32), dtype=torch.uint8, device="cuda")
    for m in (1, 20):
        x, xt = bf16(np.random.default_rng(m).normal(0, 1, (m, k)))
        y = empty(m, n)
        wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(xt, q, s, y))
        for rows in (slice(0, 40), slice(131060, 131090), slice(n - 40, n)):
            w = block.mx_values(q[rows].cpu().numpy(), s[rows].cpu().numpy())
            within(f64(y[:, rows]), x @ w.T, (k + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T), f"rows {rows}")
        del y
    del q, s
    n, k = 69000, 65536
    w = torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
    w[-1] = torch.arange(k, device="cuda").remainder(8).to(torch.bfloat16)
    q, s = empty(n, k // 2, dtype="uint8", fill=9), empty(n, k // 32, dtype="uint8", fill=9)
    wq.wq_quantize_mxfp4(None, w, n, k, q, s)
    want_q, want_s = block.mx_quantize(f64(w[-1:, :64]))
    assert np.array_equal(q[-1, :32].cpu().numpy(), want_q[0]) and np.array_equal(s[-1, -2:].cpu().numpy(), want_s[0])
    assert (q[:-1] == 0x66).all() and (s[:-1] == 125).all()
    wq.wq_dequantize_mxfp4(q, s, n, k, None, w)
    assert (w[:-1] == 1).all() and float(w[-1, -3]) == 4.0


def _layer_state(wq, seed, tokens=6, dim=256, f=192, e=8):
    """A block's buffers and plans: norm -> experts -> norm around them, into 4 bits -> product."""
    import torch
    rng = np.random.default_rng(seed)
    v = {}
    v["h"], h = f32(rng.normal(0, 2, (tokens, dim)))
    v["norm"], norm = bf16(rng.normal(1, 0.1, dim))
    v["post"], post = bf16(rng.normal(1, 0.1, dim))
    v["next"], nxt = bf16(rng.normal(1, 0.1, dim))
    v["router"], router = bf16(rng.normal(0, 0.1, (e, dim)))
    v["w13"], t13 = _experts(rng, e, 2 * f, dim, "mxfp4")
    v["w2"], t2 = _experts(rng, e, dim, f, "mxfp4")
    wf, wt = f32(rng.normal(0, 0.05, (320, dim)))
    q, s = empty(320, dim // 2, dtype="uint8"), empty(320, dim // 32, dtype="uint8")
    wq.wq_quantize_mxfp4(wt, None, 320, dim, q, s)
    v["w"] = block.mx_values(*block.mx_quantize(wf))
    b = dict(h=h, u=empty(tokens, dim, dtype="bfloat16"), f=empty(tokens, dim), out=empty(tokens, dim),
             uq=empty(tokens, dim // 2, dtype="uint8"), us=empty(tokens, dim // 32, dtype="uint8"), y=empty(tokens, 320))
    ws = torch.empty(max(wq.wq_moe_ffn_workspace_bytes(tokens, dim, f, e, 2), wq.wq_gemm_mxfp4_workspace_bytes(tokens, 320, dim)),
                     dtype=torch.uint8, device="cuda")
    plans = [
        (wq.wq_block_norm_run, wq.wq_block_norm_prepare(h, norm=norm, u=b["u"])),
        (wq.wq_moe_ffn_run, wq.wq_moe_ffn_prepare(b["u"], *t13, *t2, b["f"], router=router, workspace=ws)),
        (wq.wq_block_norm_run, wq.wq_block_norm_prepare(h, h_out=b["out"], f=b["f"], f_norm=post, scale=0.5, norm=nxt, q=b["uq"],
                                                        q_scale=b["us"])),
        (wq.wq_gemm_mxfp4_run, wq.wq_gemm_mxfp4_prepare(b["uq"], q, s, b["y"], x_scale=b["us"], workspace=ws)),
    ]
    return v, b, plans


def _check_layer(v, b):
    """Each step against the definition on what the step before it gave."""
    _, u = block.block_norm(v["h"], norm=v["norm"], eps=float(np.float32(1e-6)))
    within(f64(b["u"]), u, 2.0 ** -17 * np.abs(u) + BF16 * np.abs(u), "u")
    u = f64(b["u"])
    want, sel, gates = block.moe_ffn(u, u @ v["router"].T, v["w13"], v["w2"], 2)
    within(f64(b["f"]), want, _moe_allowed(u, v["w13"], v["w2"], sel, gates, want, 3, "f32"), "experts")
    out, nxt = block.block_norm(v["h"], f64(b["f"]), v["post"], scale=0.5, norm=v["next"], eps=float(np.float32(1e-6)))
    within(f64(b["out"]), out, 2.0 ** -24 * np.abs(out), "out")
    q, s = block.mx_quantize(nxt)
    assert np.array_equal(b["uq"].cpu().numpy(), q) and np.array_equal(b["us"].cpu().numpy(), s)
    x = block.mx_values(q, s)
    within(f64(b["y"]), x @ v["w"].T, (x.shape[1] + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(v["w"]).T), "y")


@pytest.mark.parametrize("tokens", [1, 6, 30])
def test_a_block_of_a_decoder(wq, tokens):
    v, b, plans = _layer_state(wq, tokens, tokens=tokens)
    for run, plan in plans:
        run(plan)
    _check_layer(v, b)


@pytest.mark.parametrize("tokens", [1, 6, 30])
def test_a_block_captured_and_replayed_over_other_contents(wq, tokens):
    import torch
    v, b, plans = _layer_state(wq, 50 + tokens, tokens=tokens)
    for run, plan in plans:
        run(plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for run, plan in plans:
            run(plan)
    for seed in range(3):
        v["h"], h = f32(np.random.default_rng(100 + seed).normal(0, 2, v["h"].shape))
        b["h"].copy_(h)
        for name in ("u", "f", "out", "uq", "us", "y"):
            b[name].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        _check_layer(v, b)
        got = {name: t.clone() for name, t in b.items()}
        for run, plan in plans:
            run(plan)
        torch.cuda.synchronize()
        assert all(torch.equal(got[name], t) for name, t in b.items()), "a replay differs from the calls"


def test_two_blocks_on_two_streams_and_one_workspace_per_stream(wq):
    import torch
    states = [_layer_state(wq, 70 + i, tokens=20) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, _, plans), stream in zip(states, streams):
            for run, plan in plans:
                run(plan, stream)
    torch.cuda.synchronize()
    for v, b, _ in states:
        _check_layer(v, b)


@pytest.mark.parametrize("m,n,k", [(40, 300, 4096), (1300, 1540, 2080)])
def test_split_products_share_a_workspace_on_one_stream(wq, m, n, k):
    """Shares of k meet in the workspace: two products in turn through one, and a capture of both."""
    import torch
    rng = np.random.default_rng(9)
    ws = torch.empty(wq.wq_gemm_mxfp4_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 4 * m * n                                    # there are shares
    plans, outs, wants = [], [], []
    for _ in range(2):
        q, s = mx(rng, n, k)
        x, xt = bf16(rng.normal(0, 1, (m, k)))
        y = empty(m, n)
        plans.append(wq.wq_gemm_mxfp4_prepare(xt, up(q), up(s), y, workspace=ws))
        w = block.mx_values(q, s)
        outs.append(y)
        wants.append((x @ w.T, (k + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)))
    for _ in range(2):
        for p in plans:
            wq.wq_gemm_mxfp4_run(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in plans:
            wq.wq_gemm_mxfp4_run(p)
    for _ in range(3):
        for y in outs:
            y.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for y, (want, allowed) in zip(outs, wants):
            within(f64(y), want, allowed, "y")


def test_empty_calls_touch_nothing(wq):
    import torch
    q, s = up(np.zeros((40, 32), np.uint8)), up(np.zeros((40, 2), np.uint8))
    x, y = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda"), empty(3, 40, fill=5)
    wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(x[:0], q, s, y[:0]))
    wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(x, q[:0], s[:0], y[:, :0]))
    wq.wq_quantize_mxfp4(None, x, 0, 64, q, s)
    w13, w2 = torch.zeros(4, 64, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, 64, 32, dtype=torch.int8, device="cuda")
    s13, s2 = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    out = empty(3, 64, fill=5)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x[:0], w13, s13, w2, s2, out[:0], logits=torch.zeros(0, 4, device="cuda")))
    torch.cuda.synchronize()
    assert (y == 5).all() and (out == 5).all()


def test_gates_past_what_an_exponential_holds(wq):
    """Gates of thousands, infinities and NaN, with results in bf16 and in 4 bits."""
    import torch
    rng = np.random.default_rng(11)
    f = rng.normal(0, 1, (1, 128))
    fv, ft = bf16(f)
    hv, ht = f32(rng.normal(0, 1, (1, 128)))
    g = rng.normal(0, 2, (1, 128))
    g[0, :8] = [1e4, -1e4, 800, -800, 88.8, -88.8, 3e38, -3e38]
    gv, gt = bf16(g)
    for kind in ("sigmoid", "silu"):
        with np.errstate(over="ignore"):
            want, u = block.block_norm(hv, fv, None, gv, kind, 1.0, None, float(np.float32(1e-6)))
        out, q, s = empty(1, 128), empty(1, 64, dtype="uint8"), empty(1, 4, dtype="uint8")
        for plan in (wq.wq_block_norm_prepare(ht, h_out=out, f=ft, gate=gt, gate_kind=kind),
                     wq.wq_block_norm_prepare(ht, h_out=out, f=ft, gate=gt, gate_kind=kind, q=q, q_scale=s)):
            wq.wq_block_norm_run(plan)
            got = f64(out)
            fine = np.abs(want) < 3e38
            within(np.where(fine, got, 0), np.where(fine, want, 0),
                   2.0 ** -19 * (np.abs(hv) + np.abs(np.where(fine, want, 0) - hv)), kind)
        if kind == "sigmoid":
            assert np.array_equal(q.cpu().numpy(), block.mx_quantize(u)[0])
    gt[0, 9] = float("nan")
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(ht, h_out=out, f=ft, gate=gt, gate_kind="sigmoid", q=q, q_scale=s))
    assert torch.isnan(out[0, 9]) and torch.isfinite(out[0, 10:]).all() and (s == 255).all()
    gt[0, 9], gt[0, 10] = float("-inf"), float("inf")
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(ht, h_out=out, f=ft, gate=gt, gate_kind="sigmoid", q=q, q_scale=s))
    within(f64(out[0, 9:11]), hv[0, 9:11] + np.array([0.0, fv[0, 10]]), 2.0 ** -20, "infinite gates")


def test_a_buffer_of_another_device_is_refused(wq):
    import torch

    class Elsewhere:
        """A tensor that says it is on the next device."""

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return self.t.get_device() + 1

    w, q, s = torch.zeros(2, 32, device="cuda"), empty(2, 16, dtype="uint8", fill=9), empty(2, 1, dtype="uint8", fill=9)
    for call in (lambda: wq.wq_quantize_mxfp4(Elsewhere(w), None, 2, 32, q, s),
                 lambda: wq.wq_quantize_mxfp4(w, None, 2, 32, q, Elsewhere(s), stream=torch.cuda.Stream()),
                 lambda: wq.wq_dequantize_mxfp4(Elsewhere(q), s, 2, 32, w)):
        with pytest.raises(ValueError, match="device"):
            call()
    torch.cuda.synchronize()
    assert (q == 9).all() and (s == 9).all() and (w == 0).all()


@pytest.mark.parametrize("post", [False, True])
def test_norms_of_rows_below_the_normal_range(wq, post):
    """Rows of a few units of 2^-149 without eps: results in bf16 are those of the formula, like any other row's."""
    import torch
    rng = np.random.default_rng(12)
    v = rng.integers(-511, 512, (3, 264)) * 2.0 ** -149
    xv, xt = f32(v)
    assert np.array_equal(xv, v)
    u = empty(3, 264, dtype="bfloat16")
    if post:
        # h' = 0 + norm(f), then as it is
        one = torch.ones(264, dtype=torch.bfloat16, device="cuda")
        plan = wq.wq_block_norm_prepare(torch.zeros(3, 264, device="cuda"), h_out=empty(3, 264), f=xt, f_norm=one, u=u, eps=0.0)
    else:
        plan = wq.wq_block_norm_prepare(xt, u=u, eps=0.0)
    wq.wq_block_norm_run(plan)
    want = v / np.sqrt((v * v).mean(1, keepdims=True))
    # a factor good to 2^-24 and a product each (twice with `post`), then bf16
    within(f64(u), want, (BF16 + 2.0 ** -20) * np.abs(want), "u")


def test_norms_of_as_many_rows_as_documented(wq):
    """2^24 rows of 520, more threads than one axis of a grid holds."""
    import torch
    rows, dim = 1 << 24, 520
    rng = np.random.default_rng(13)
    at = [0, 1, (1 << 20) - 1, 1 << 20, (1 << 23) + 5, rows - 2, rows - 1]
    h = torch.ones(rows, dim, dtype=torch.bfloat16, device="cuda")
    hv, ht = bf16(rng.normal(0, 3, (len(at), dim)))
    h[at] = ht
    u = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(h, u=u, eps=0.0))
    _, want = block.block_norm(hv, eps=0.0)
    within(f64(u[at]), want, (BF16 + 2.0 ** -18) * np.abs(want), "u")
    u[at] = 1
    # a row of ones stays one; by maximum and minimum, chunk by chunk
    for part in u.view(-1).split(1 << 30):
        assert float(part.max()) == 1 and float(part.min()) == 1


@pytest.mark.parametrize("xkind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(3, 70, 96), (16, 40, 544), (40, 140, 1056), (2050, 5500, 96)])
def test_products_of_scales_far_apart(wq, m, n, k, xkind):
    """Rows of W and of x from the smallest scales to the largest: a result is its own sum, not cut by either's range.
    Sums that end below 2^-126 may lose what is below it."""
    import torch
    rng = np.random.default_rng(m)
    q, s = mx(rng, n, k)
    s[:] = rng.choice(np.array([0, 1, 30, 90, 127, 160, 220, 250], np.uint8), (n, 1))
    w = block.mx_values(q, s)
    if xkind == "bf16":
        x, xt = bf16(rng.normal(0, 1, (m, k)) * 2.0 ** rng.choice([-120, -60, 0, 60, 119], (m, 1)))
        xs = None
    else:
        xq, xsc = mx(rng, m, k)
        xsc[:] = rng.choice(np.array([0, 2, 60, 127, 200, 246], np.uint8), (m, 1))
        x, xt, xs = block.mx_values(xq, xsc), up(xq), up(xsc)
    y = empty(m, n)
    wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(xt, up(q), up(s), y, x_scale=xs))
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    fine = size < 2.0 ** 127
    got = f64(y)
    within(np.where(fine, got, 0), np.where(fine, want, 0),
           np.where(fine, (k + 16) * 2.0 ** -23 * size + k * 2.0 ** -126, 0), "far scales")
    assert (np.abs(want[fine]) > 2.0 ** -100).any() and (np.abs(want[fine]) < 2.0 ** -120).any()


@pytest.mark.parametrize("xkind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(3, 70, 96), (16, 40, 544), (40, 140, 1056), (2050, 5500, 96), (300, 700, 1056)])
def test_weights_at_and_past_the_largest_finite_value(wq, m, n, k, xkind):
    """A group of scale byte 252, 253 or 254 in a row of W: past 2^128 a weight is infinite where x is bf16, and its own
    value where x is MXFP4, whose products are finite here."""
    rng = np.random.default_rng(m + n)
    q, s = mx(rng, n, k)
    for byte, first in ((252, 0), (253, 1), (254, 2)):
        s[first::4, byte % s.shape[1]] = byte
    w = block.mx_values(q, s)
    if xkind == "bf16":
        x, xt = bf16(rng.choice([-1.0, 1.0], (m, k)) * rng.uniform(1, 2, (m, k)) * 2.0 ** -30)
        xs = None
        lost = (np.abs(w) >= 2.0 ** 128).any(1)
        assert lost.any() and not lost[0::4].any()
    else:
        xq, xsc = mx(rng, m, k)
        xsc -= 30
        x, xt, xs, lost = block.mx_values(xq, xsc), up(xq), up(xsc), np.zeros(n, bool)
    y = empty(m, n)
    wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(xt, up(q), up(s), y, x_scale=xs))
    got, size = f64(y), np.abs(x) @ np.abs(w).T
    assert not np.isfinite(got[:, lost]).any()
    within(got[:, ~lost], (x @ w.T)[:, ~lost], (k + 16) * 2.0 ** -23 * size[:, ~lost], "weights to the end of the range")


@pytest.mark.parametrize("xkind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("m,n,k,stride", [(1 << 20, 40, 32, 32), (3, 1 << 24, 32, 32), (20, 70, 1 << 18, 1 << 18), (2, 70, 1 << 18, 1 << 18),
                                          (300, 80, 96, 1 << 22), (9, 80, 96, 1 << 22), (1 << 20, 300, 64, 64)])
def test_products_at_the_documented_limits(wq, m, n, k, stride, xkind):
    """As many rows, columns and inputs and as long a stride as documented; rows and columns here and there against 64
    bits."""
    import torch
    rng = np.random.default_rng(14)
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.randint(124, 131, (n, k // 32), dtype=torch.uint8, device="cuda")
    if xkind == "bf16":
        x = torch.empty(m, stride, dtype=torch.bfloat16, device="cuda")[:, :k]
        x.normal_()
        xs = None
    else:
        x = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device="cuda")
        xs = torch.randint(125, 130, (m, k // 32), dtype=torch.uint8, device="cuda")
    y = empty(m, n, dtype="bfloat16" if m * n > 1 << 26 else "float32")
    wq.wq_gemm_mxfp4_run(wq.wq_gemm_mxfp4_prepare(x, q, s, y, x_scale=xs))
    rows = np.unique(np.r_[0, m - 1, rng.integers(0, m, 40)])
    cols = np.unique(np.r_[0, n - 1, rng.integers(0, n, 60)])
    take = torch.from_numpy
    xv = f64(x[take(rows)]) if xs is None else block.mx_values(x[take(rows)].cpu().numpy(), xs[take(rows)].cpu().numpy())
    w = block.mx_values(q[take(cols)].cpu().numpy(), s[take(cols)].cpu().numpy())
    want, size = xv @ w.T, np.abs(xv) @ np.abs(w).T
    allowed = (k + 16) * 2.0 ** -23 * size
    if y.dtype == torch.bfloat16:
        allowed = allowed + BF16 * (np.abs(want) + allowed)
    within(f64(y[take(rows)][:, take(cols)]), want, allowed, "y")


def test_a_norm_of_one_row_at_the_longest_stride(wq):
    """Strides far past a row: the offsets of the last rows pass 32 bits."""
    import torch
    rows, dim, stride = 3, 64, 1 << 31
    rng = np.random.default_rng(15)
    hv, ht = bf16(rng.normal(0, 1, (rows, dim)))
    wide = torch.empty((rows - 1) * stride + dim, dtype=torch.bfloat16, device="cuda")
    h = wide.as_strided((rows, dim), (stride, 1))
    h.copy_(ht)
    u = torch.empty_like(wide).as_strided((rows, dim), (stride, 1))
    wq.wq_block_norm_run(wq.wq_block_norm_prepare(h, u=u, eps=0.0))
    _, want = block.block_norm(hv, eps=0.0)
    within(f64(u), want, (BF16 + 2.0 ** -18) * np.abs(want), "u")


@pytest.mark.parametrize("weights", ["int8", "mxfp4"])
@pytest.mark.parametrize("tokens", [1, 64])
def test_experts_at_the_documented_limits(wq, tokens, weights):
    """dim and f of 32768, the second expert's weights past 32 bits of offset: sampled columns against 64 bits."""
    import torch
    dim = f = 32768
    e = 2 if weights == "int8" else 3
    if weights == "int8":
        w13 = torch.randint(-127, 128, (e, 2 * f, dim), dtype=torch.int8, device="cuda")
        w2 = torch.randint(-127, 128, (e, dim, f), dtype=torch.int8, device="cuda")
        s13 = torch.full((e, 2 * f), 2.0 ** -14, dtype=torch.bfloat16, device="cuda")
        s2 = torch.full((e, dim), 2.0 ** -14, dtype=torch.bfloat16, device="cuda")

        def values(q, s):
            return q.double() * s.double()[:, None]
    else:
        w13 = torch.randint(0, 256, (e, 2 * f, dim // 2), dtype=torch.uint8, device="cuda")
        w2 = torch.randint(0, 256, (e, dim, f // 2), dtype=torch.uint8, device="cuda")
        s13 = torch.randint(117, 120, (e, 2 * f, dim // 32), dtype=torch.uint8, device="cuda")
        s2 = torch.randint(117, 120, (e, dim, f // 32), dtype=torch.uint8, device="cuda")
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")

        def values(q, s):
            v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).flatten(-2)
            return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)
    _, x = bf16(np.random.default_rng(16).normal(0, 1, (tokens, dim)))
    logits = torch.zeros(tokens, e, device="cuda")
    logits[:, e - 1] = 3
    y = empty(tokens, dim)
    wq.wq_moe_ffn_run(wq.wq_moe_ffn_prepare(x, w13, s13, w2, s2, y, logits=logits, top=1))
    h = []
    for half in range(2):
        parts = [x.double() @ values(w13[-1, r:r + 2048], s13[-1, r:r + 2048]).T for r in range(half * f, (half + 1) * f, 2048)]
        h.append(torch.cat(parts, 1))
    act = h[0] / (1 + torch.exp(-h[0])) * h[1]
    cols = torch.tensor([0, 1, 17, 4095, 20000, dim - 2, dim - 1], device="cuda")
    w = values(w2[-1, cols], s2[-1, cols])
    want, size = act @ w.T, act.abs() @ w.abs().T
    # sums of `dim` products behind act (its errors meet at random; here at most (dim + 16) 2^-23 of |x| |w13|, as in the
    # other layers' bound) and of 3 f parts
    biggest = values(w13[-1, :2048], s13[-1, :2048]).abs()
    d = (dim + 16) * 2.0 ** -23 * float((x.double().abs() @ biggest.T).max()) * 1.1
    da = 1.1 * d * (h[1].abs() + d) + act.abs() * 2.0 ** -19 + d * h[0].abs()
    allowed = da @ w.abs().T + ((3 * f + 16) * 2.0 ** -23 + 2.0 ** -19) * size
    within(f64(y[:, cols]), f64(want), f64(allowed), "y")
    # what the bound above is for: no piece of a sum is missing or doubled
    assert float((y[:, cols].double() - want).abs().max()) < 1e-3 * float(size.max())
