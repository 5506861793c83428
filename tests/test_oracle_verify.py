"""Pins of oracle/verify.py that do not re-type its formulas: closed forms and invariants."""

import numpy as np
import pytest

from oracle import verify

RNG = np.random.default_rng(20)


def test_rotation_keeps_norms_and_depends_on_distance_only():
    freq, _ = verify.rope_frequencies("plain", 16, 1e4)
    for interleaved in (False, True):
        q, k = RNG.normal(size=(2, 20))
        def turned(x, p):
            return verify.norm_rope_head(x, p, freq, interleaved=interleaved)
        assert np.isclose(np.linalg.norm(turned(q, 77)), np.linalg.norm(q))
        assert np.isclose(turned(q, 105) @ turned(k, 98), turned(q, 7) @ turned(k, 0))
        assert np.array_equal(turned(q, 5)[16:], q[16:])
        assert np.allclose(turned(q, 0), q)


def test_layouts_are_permutations_of_each_other():
    freq, _ = verify.rope_frequencies("plain", 8, 1e4)
    x = RNG.normal(size=8)
    pairs = verify.norm_rope_head(x, 9, freq, interleaved=True)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    assert np.allclose(verify.norm_rope_head(x[order], 9, freq), pairs[order])


def test_norm_has_unit_mean_square():
    x = RNG.normal(size=64) * 17
    y = verify.norm_rope_head(x, 0, [], weight=np.ones(64), eps=0.0)
    assert np.isclose(np.mean(y * y), 1.0)


def test_frequencies_closed_forms():
    f, s = verify.rope_frequencies("plain", 4, 100.0)
    assert np.allclose(f, [1.0, 0.1]) and s == 1.0
    assert np.allclose(verify.rope_frequencies("linear", 4, 100.0, factor=8.0)[0], f / 8)
    # bands: a pair that turns often within the original length is kept, a slow one is stretched
    f, _ = verify.rope_frequencies("plain", 128, 5e5)
    g, _ = verify.rope_frequencies("bands", 128, 5e5, factor=8.0, low=1.0, high=4.0, original=8192)
    turns = 8192 * f / (2 * np.pi)
    assert np.allclose(g[turns > 4], f[turns > 4]) and np.allclose(g[turns < 1], f[turns < 1] / 8)
    assert np.all(np.diff(g) < 0)
    # ramp: the same ends, and the scale of the logits
    g, s = verify.rope_frequencies("ramp", 128, 1e4, factor=4.0, low=1.0, high=32.0, original=4096)
    f, _ = verify.rope_frequencies("plain", 128, 1e4)
    assert np.isclose(g[0], f[0]) and np.isclose(g[-1], f[-1] / 4) and np.all(g <= f + 1e-18) and np.all(g >= f / 4)
    assert np.isclose(s, 0.1 * np.log(4) + 1)


@pytest.mark.parametrize("rot_dim", [2, 10, 64, 128])
@pytest.mark.parametrize("kind,args", [("plain", {}), ("linear", dict(factor=3.5)),
                                       ("bands", dict(factor=8.0, low=1.0, high=4.0, original=8192.0)),
                                       ("ramp", dict(factor=16.0, low=1.0, high=32.0, original=4096.0))])
def test_library_frequencies(rot_dim, kind, args):
    """The library's table (host call, no GPU): fp64 rounded once, so half a step of fp32 and the differences of two
    pow's."""
    import weight_only_quantized_wq_amd as wq
    got, scale = wq.wq_rope_frequencies(rot_dim, 500000.0, kind, **args)
    want, s = verify.rope_frequencies(kind, rot_dim, 500000.0, **args)
    assert np.all(np.abs(got.numpy() - want) <= (2.0 ** -24 + 1e-12) * want)
    assert abs(scale - s) <= 2.0 ** -23


def _pool(pages, size, kv, dim):
    return RNG.normal(size=(pages, size, kv, dim)), RNG.normal(size=(pages, size, kv, dim))


def test_attention_of_one_position_is_its_value():
    k, v = _pool(3, 4, 2, 8)
    q = RNG.normal(size=(1, 4, 8))
    y, _ = verify.tree_attention(q, k, v, np.array([[2]]), [0, 1], [0], 0.3)
    assert np.allclose(y[0], np.repeat(v[2, 0], 2, axis=0))


def test_equal_keys_give_the_mean_of_what_is_seen():
    k, v = _pool(4, 4, 1, 8)
    k[:] = k[0, 0]
    table = np.array([[3, 1]])
    q = RNG.normal(size=(3, 1, 8))
    y, reach = verify.tree_attention(q, k, v, table, [0, 3], [3], 1.0, tree=[1, 3, 5])
    flat = np.concatenate([v[3], v[1]])[:, 0]
    assert np.allclose(y[0, 0], flat[:4].mean(0))
    assert np.allclose(y[1, 0], flat[:5].mean(0))
    assert np.allclose(y[2, 0], flat[[0, 1, 2, 3, 5]].mean(0))
    assert np.all(reach >= np.abs(y) - 1e-12)


def test_attention_rows_that_see_nothing_and_rows_left_alone():
    k, v = _pool(2, 4, 1, 8)
    q = RNG.normal(size=(4, 1, 8))
    y, _ = verify.tree_attention(q, k, v, np.array([[0], [9]]), [0, 1, 2], [0, 0], 1.0, tree=[0, 1, 1, 1])
    assert np.all(y[0] == 0) and np.all(y[1] == 0) and np.all(np.isnan(y[2:]))


def test_accept_moves_by_depth():
    k = np.arange(12.0).reshape(1, 3, 4, 1, 1)
    table, path = np.array([[1, 0]]), np.array([[0, 2, 3]])
    got, _ = verify.kv_accept(k, k.copy(), table, [2], path, [3])
    # positions 2, 3, 4 hold drafts 0, 2, 3 of positions 2 .. 5
    assert got.ravel().tolist() == [1.0, 1, 2, 3, 4, 5, 6, 0, 8, 9, 10, 11]
    same, _ = verify.kv_accept(k, k.copy(), table, [2], np.array([[0, 2, 2]]), [3])
    assert np.array_equal(same, k)


def test_lora_closed_forms():
    x = RNG.normal(size=(3, 8))
    a, b = np.zeros((2, 8, 8)), np.zeros((2, 8, 8))
    a[0] = b[0] = np.eye(8)
    a[1] = b[1] = 2 * np.eye(8)
    y, _, _ = verify.lora(x, a, b, [1, -1, 0], base=np.ones((3, 8)), ranks=[8, 3], scale=[1.0, 0.5])
    assert np.allclose(y[2], 1 + x[2]) and np.allclose(y[1], 1)
    assert np.allclose(y[0][:3], 1 + 2 * x[0][:3]) and np.allclose(y[0][3:], 1)
