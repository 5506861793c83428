"""MXFP4 quantiser and products, the expert layer and the norm around a block on the GPU against oracle/block.py.

Tolerances, fixed before the first run.  A rounding to bf16 is off by at most
2^-8 of the value, one to fp32 by 2^-24.

* quantisation and its inverse: none, every code and value is exact.
* product: operands are exact in what the matrix cores take (bf16 pairs, or
  codes and scales), so a result differs by the roundings of its fp32 sum, at
  most (k + 16) 2^-23 of sum |x w| (additions that truncate count double), and
  one rounding to bf16 where that is asked for.
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
          (63, 257, 608), (64, 128, 8192), (65, 96, 160), (129, 515, 1056), (200, 300, 2560), (257, 260, 96), (515, 129, 640)]


@pytest.mark.parametrize("xkind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(wq, m, n, k, xkind):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    _product(wq, rng, m, n, k, xkind, ["f32", "bf16", "both"][(m + n) % 3], pad=(m + n) % 2)
