"""Pins of oracle/block.py by exact rational arithmetic and closed forms."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import block

SIZES = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]


def _code(size):
    """Nearest size by exact comparison; of two, the one with the even code."""
    best = min(range(8), key=lambda c: (abs(SIZES[c] - size), c % 2))
    return best


def _floor_log2(v):
    e = 0
    while Fraction(2) ** e > v:
        e -= 1
    while Fraction(2) ** (e + 1) <= v:
        e += 1
    return e


@pytest.mark.parametrize("seed", range(4))
def test_codes_are_the_nearest_by_exact_arithmetic(seed):
    rng = np.random.default_rng(seed)
    w = rng.normal(0, 2.0 ** rng.integers(-20, 20), (3, 64)).astype(np.float32).astype(np.float64)
    w[0, :32] = np.arange(32) / 8                       # every border and tie under one scale
    w[1, 5] = 0.0
    q, scale = block.mx_quantize(w)
    code = np.stack([q & 15, q >> 4], -1).reshape(3, 64)
    for r in range(3):
        for g in range(2):
            v = [Fraction(float(a)) for a in w[r, 32 * g:32 * g + 32]]
            e = max(_floor_log2(max(abs(a) for a in v)) - 2, -127)
            assert scale[r, g] == e + 127
            for a, c in zip(v, code[r, 32 * g:32 * g + 32]):
                assert _code(min(abs(a) / Fraction(2) ** e, Fraction(6))) == c & 7
                assert (c >> 3) == (a < 0)


def test_values_of_every_code_and_idempotence():
    q = np.zeros((1, 16), np.uint8)
    q[0, :8] = np.arange(0, 16, 2) | np.arange(1, 17, 2) << 4
    v = block.mx_values(q, np.array([[127]], np.uint8))[0]
    assert list(v[:16]) == [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]
    again, scale = block.mx_quantize(v[None])
    assert np.array_equal(again, q) and scale[0, 0] == 127
    assert np.isnan(block.mx_values(q, np.array([[255]], np.uint8))).all()


def test_scales_at_the_ends():
    for largest, byte in [(0.0, 0), (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125), (7.9, 127), (8.0, 128),
                          (float(np.finfo(np.float32).max), 252), (np.inf, 255), (np.nan, 255)]:
        assert block.mx_scale_byte(largest) == byte
    w = np.zeros((1, 32))
    w[0, 3] = np.nan
    q, scale = block.mx_quantize(w)
    assert scale[0, 0] == 255 and not q.any()


def test_routing_takes_ties_to_the_lower_index():
    sel, gates = block.route(np.array([1.0, 3.0, 3.0, 0.0]), 2)
    assert sel == [1, 2] and np.allclose(gates, 0.5)
    _, share = block.route(np.array([0.0, 0.0, 0.0, 0.0]), 2, renormalize=False)
    assert np.allclose(share, 0.25)


def test_expert_layer_of_identity_experts():
    dim = 32
    w13 = np.stack([np.concatenate([np.eye(dim) * 40, np.eye(dim)])] * 3)      # silu(40 x) ~ 40 x for x >= 1
    w2 = np.stack([np.eye(dim) * (e + 1) for e in range(3)])
    x = np.full((1, dim), 2.0)
    y, sel, gates = block.moe_ffn(x, np.array([[0.0, np.log(3.0), -50.0]]), w13, w2, 2)
    assert sel.tolist() == [[1, 0]] and np.allclose(gates, [[0.75, 0.25]])
    assert np.allclose(y, (0.75 * 2 + 0.25) * 160.0)


def test_block_norm_closed_forms():
    h = np.array([[3.0, 4.0]])
    out, u = block.block_norm(h, eps=0.0)
    assert np.array_equal(out, h) and np.allclose(u, h / np.sqrt(12.5))
    out, _ = block.block_norm(h, f=np.array([[1.0, -1.0]]), f_norm=np.array([2.0, 3.0]), gate=np.zeros((1, 2)),
                              gate_kind="sigmoid", scale=4.0, eps=0.0)
    assert np.allclose(out, [[3.0 + 4 * 0.5 * 2, 4.0 - 4 * 0.5 * 3]])
