"""The calls around a verify pass on the GPU against oracle/verify.py (fp64).

Tolerances, fixed before the first run.  A rounding to bf16 is off by at most
2^-8 of the value, one to fp32 by 2^-24.  Per element:

* rotation: one bf16 rounding, plus fp32 arithmetic on the pair (norm: a sum of
  dim squares, square root, quotient, two products; rotation: sin and cos good
  to 2^-22, two products) bounded by 2^-16 (|a| + |b|).
* attention: each weight is rounded to bf16 for the second product (2^-8 of it,
  so 2^-8 sum w|v|), scores carry dim fp32 roundings of sum |q k| * scale (at
  most 300 here: 2^-24 * 128 * 300 < 2^-8.7 in the worst case, a hundredth of
  that for random signs: 2^-10 sum w|v| is allowed), then one bf16 rounding.
* adapters: k + 8 fp32 roundings of the terms of A x carried through |B|, rank +
  8 of B h, doubled for products whose additions may truncate, one rounding of
  the sum with the base.
"""

import numpy as np
import pytest

from gpu_util import say
from oracle import verify

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


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def pages_for(rng, spans, page, extra=2, holes=False):
    """Table over positions [0, spans[r]) in no order; entries past a request's own are outside the pool."""
    width = max(1, max(-(-s // page) for s in spans))
    need = [-(-s // page) for s in spans]
    pages = sum(need) + extra
    order = rng.permutation(pages)
    table = np.full((len(spans), width), pages if rng.random() < 0.5 else -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, pages


def random_tree(rng, n):
    masks = []
    for j in range(n):
        parent = int(rng.integers(-1, j)) if j else -1
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
    return masks


def as_i64(masks):
    return np.array([m - (1 << 64) if m >> 63 else m for m in masks], np.int64)


class Attn:
    """One attention problem; `layout` "NHD" or "HND" (heads before positions in a page)."""

    def __init__(self, rng, lengths, counts, heads, kv, dim, page, tree=None, layout="NHD", pad_rows=0, scale=None):
        import torch
        self.kv, self.dim, self.heads, self.page = kv, dim, heads, page
        self.lengths, self.counts = list(lengths), list(counts)
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.tokens = int(self.starts[-1]) + pad_rows
        self.table, self.pages = pages_for(rng, [max(a, 0) + b for a, b in zip(lengths, counts)], page)
        shape = (self.pages, page, kv, dim)
        self.k64, k = bf16(rng.normal(size=shape))
        self.v64, v = bf16(rng.normal(size=shape))
        self.q64, self.q = bf16(rng.normal(size=(self.tokens, heads, dim)))
        if layout == "HND":
            k, v = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (k, v))
        self.k, self.v = k, v
        self.tree = None
        if tree is not None:
            masks = [m for n in counts for m in (tree(n) if callable(tree) else tree)] + [0] * pad_rows
            self.tree = masks
        self.scale = dim ** -0.5 if scale is None else scale
        self.y = torch.full((self.tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")

    def plan(self, wq, max_tokens=None, **kw):
        import torch
        tree = None if self.tree is None else torch.from_numpy(as_i64(self.tree)).cuda()
        return wq.wq_tree_attention_prepare(self.q, self.k, self.v, i32(self.table), i32(self.starts),
                                            i32(self.lengths), self.y, tree=tree, scale=self.scale,
                                            max_tokens=max_tokens or max(1, min(64, max(self.counts))), **kw)

    def want(self, max_tokens=64):
        return verify.tree_attention(self.q64, self.k64, self.v64, self.table, self.starts, self.lengths, self.scale,
                                     self.tree, max_tokens)

    def check(self, y=None, max_tokens=64):
        want, reach = self.want(max_tokens)
        got = f64(self.y if y is None else y)
        alone = np.isnan(want)
        assert np.all(got[alone] == 7.0), "rows of no request were written"
        tol = (BF16 + 2.0 ** -10) * reach + BF16 * np.abs(want) * (1 + BF16)
        off = np.where(alone, 0, np.abs(got - want) - tol)
        assert np.all(np.isfinite(got)) and np.all(off <= 0), (np.unravel_index(off.argmax(), off.shape), off.max())


def run(wq, p, **kw):
    import torch
    wq.wq_tree_attention_run(p.plan(wq, **kw))
    torch.cuda.synchronize()


# --- attention ---------------------------------------------------------------


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("heads,kv", [(4, 4), (8, 2), (7, 1)])
@pytest.mark.parametrize("page", [16, 13])
def test_attention_head_layouts(wq, dim, heads, kv, page):
    rng = np.random.default_rng(dim * 100 + heads * 10 + page)
    p = Attn(rng, [300, 0, 17, 129], [5, 3, 1, 8], heads, kv, dim, page, tree=lambda n: random_tree(rng, n))
    run(wq, p)
    p.check()


@pytest.mark.parametrize("length", [0, 1, 7, 31, 32, 33, 63, 127, 128, 129, 255, 1000, 4100])
@pytest.mark.parametrize("n", [1, 5])
def test_attention_lengths(wq, length, n):
    rng = np.random.default_rng(length * 7 + n)
    p = Attn(rng, [length], [n], 4, 2, 128, 16)
    run(wq, p)
    p.check()


@pytest.mark.parametrize("n,heads,kv", [(64, 8, 1), (64, 2, 2), (33, 8, 2), (17, 4, 4), (5, 64, 8), (2, 64, 1),
                                        (1, 64, 1), (16, 5, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_row_blocks(wq, n, heads, kv, dim):
    # rows per key head: less than a row tile, exactly one, several blocks
    rng = np.random.default_rng(n * heads + dim)
    p = Attn(rng, [450, 61], [n, max(1, n - 1)], heads, kv, dim, 32, tree=lambda m: random_tree(rng, m))
    run(wq, p)
    p.check()


def test_attention_256_with_many_rows(wq):
    rng = np.random.default_rng(256)
    p = Attn(rng, [400], [20], 8, 2, 256, 24, tree=lambda m: random_tree(rng, m))
    run(wq, p)
    p.check()


@pytest.mark.parametrize("page", [1, 3, 8, 40, 64, 100, 128, 1024])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_attention_pages_and_orders(wq, page, layout):
    rng = np.random.default_rng(page)
    p = Attn(rng, [333, 90], [4, 4], 8, 4, 128, page, layout=layout)
    run(wq, p)
    p.check()


def test_attention_rows_without_anything_to_see_and_unused_rows(wq):
    rng = np.random.default_rng(3)
    # a request without context whose tree shows nothing, one without tokens, rows behind the last request
    p = Attn(rng, [0, 50, -4, 20], [3, 0, 2, 2], 4, 2, 64, 16, tree=None, pad_rows=3)
    p.tree = [0, 1, 0, 0, 2, 3, 1, 5, 5, 5]
    run(wq, p)
    want, _ = p.want()
    assert np.all(want[0] == 0) and np.all(want[2:4] == 0)
    p.check()


def test_attention_bits_past_the_request_do_not_count(wq):
    rng = np.random.default_rng(4)
    p = Attn(rng, [40], [3], 2, 2, 64, 16)
    p.tree = [(1 << 64) - 1, 0xFFFF0002, 7]
    run(wq, p)
    p.check()


def test_attention_of_a_request_with_too_many_tokens_is_left_alone(wq):
    rng = np.random.default_rng(5)
    p = Attn(rng, [30, 30, 30], [2, 6, 3], 2, 2, 64, 16)
    run(wq, p, max_tokens=4)
    p.check(max_tokens=4)


def test_attention_bad_pages_hold_nothing(wq):
    rng = np.random.default_rng(6)
    for page in (16, 10):
        p = Attn(rng, [200, 100], [4, 4], 4, 2, 128, page)
        p.table[0, 2] = -1
        p.table[0, 5] = p.pages
        p.table[1, 0] = 0x7FFFFFFF
        run(wq, p)
        p.check()


def test_attention_length_past_the_table(wq):
    rng = np.random.default_rng(7)
    p = Attn(rng, [60], [2], 4, 2, 64, 16)
    p.lengths = [10 ** 9]
    run(wq, p)
    p.check()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_attention_what_a_row_does_not_see_does_not_change_it(wq, bad):
    import torch
    rng = np.random.default_rng(8)
    for page in (16, 10):
        p = Attn(rng, [150], [6], 8, 2, 128, page, tree=lambda n: [1, 3, 5, 11, 21, 33])
        run(wq, p)
        clean = p.y.clone()
        # poison: every position behind the request's last, and draft 3's own key and value
        k, v = p.k.clone(), p.v.clone()
        used = {(int(p.table[0, q // page]), q % page) for q in range(156)}
        for pg in range(p.pages):
            for row in range(page):
                if (pg, row) not in used:
                    k[pg, row], v[pg, row] = bad, bad
        at = int(p.table[0, 153 // page]), 153 % page
        k[at], v[at] = bad, bad
        p.k, p.v = k, v
        p.y.fill_(7.0)
        run(wq, p)
        same = [0, 1, 2, 4, 5]
        assert torch.equal(p.y[same], clean[same])
        assert not torch.isfinite(p.y[3]).any()


def test_attention_infinite_values_reach_the_rows_that_see_them(wq):
    import torch
    rng = np.random.default_rng(9)
    p = Attn(rng, [140], [4], 4, 2, 128, 16, tree=lambda n: [1, 3, 5, 13])
    at = int(p.table[0, 142 // 16]), 142 % 16
    p.v[at[0], at[1], 1, 5] = float("inf")
    p.v64 = p.v64.copy()
    run(wq, p)
    got = f64(p.y)
    hit = np.zeros(got.shape, bool)
    hit[2:4, 2:4, 5] = True           # tokens 2 and 3, the heads of key head 1, element 5
    assert np.all(got[hit] == np.inf) and np.all(np.isfinite(got[~hit]))
    want, reach = p.want()
    assert np.all((np.abs(got - want) <= (BF16 + 2.0 ** -10) * reach + BF16 * np.abs(want) * 1.01)[~hit])


def test_attention_large_scores(wq):
    # scores of +-1000: the running maximum is raised over and over
    rng = np.random.default_rng(10)
    p = Attn(rng, [700], [3], 4, 2, 64, 16, scale=0.125)
    p.q64, p.q = bf16(p.q64 * 3)
    ramp = np.linspace(0.1, 30, p.pages * 16).reshape(p.pages, 16, 1, 1)
    p.k64, p.k = bf16(p.k64 * ramp)
    run(wq, p)
    # weights of scores s carry an error of 64 * 2^-24 * |s| here, below 2^-8 for |s| < 1000
    want, reach = p.want()
    got = f64(p.y)
    assert np.all(np.abs(got - want) <= 2 * BF16 * reach + BF16 * np.abs(want) * 1.01)


def test_attention_ragged_batch_across_shares(wq):
    rng = np.random.default_rng(11)
    lengths = [0, 3000, 5, 129, 2048, 77, 1, 640, 128, 900, 31, 4000]
    counts = [1, 8, 3, 8, 2, 0, 8, 5, 1, 7, 8, 8]
    p = Attn(rng, lengths, counts, 8, 2, 128, 64, tree=lambda n: random_tree(rng, n), pad_rows=2)
    run(wq, p)
    p.check()


def test_attention_is_reproducible_and_follows_changed_buffers(wq):
    import torch
    rng = np.random.default_rng(12)
    p = Attn(rng, [1500, 900], [5, 5], 8, 2, 128, 16)
    plan = p.plan(wq)
    wq.wq_tree_attention_run(plan)
    first = p.y.clone()
    for _ in range(3):
        p.y.fill_(7.0)
        wq.wq_tree_attention_run(plan)
        assert torch.equal(p.y, first)
    lengths = plan.keep[5]
    lengths.copy_(i32([700, 33]))
    p.lengths = [700, 33]
    p.y.fill_(7.0)
    wq.wq_tree_attention_run(plan)
    torch.cuda.synchronize()
    p.check()


def test_attention_strided_rows(wq):
    import torch
    rng = np.random.default_rng(13)
    p = Attn(rng, [100, 40], [3, 2], 4, 2, 64, 16)
    wide = torch.full((p.tokens, 4 * 64 + 72), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 256] = p.q.view(p.tokens, 256)
    out = torch.full((p.tokens, 4 * 64 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    p.q, y = wide[:, 8:8 + 256], out[:, 16:16 + 256]
    p.y = y
    run(wq, p)
    p.check(y.reshape(p.tokens, 4, 64))
    assert torch.all(out[:, :16] == 7.0) and torch.all(out[:, 272:] == 7.0)


def test_attention_cache_past_32_bits(wq):
    """Pages that start past 2^32 elements (a pool of 8.9 GB, two pages of it used)."""
    import torch
    rng = np.random.default_rng(14)
    p = Attn(rng, [20], [3], 2, 2, 64, 16)
    pages = (1 << 32) // (16 * 2 * 64) + 70000
    k = torch.empty(pages, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    far = [pages - 1, pages - 30000]
    for i, pg in enumerate(far):
        k[pg], v[pg] = p.k[int(p.table[0, i])], p.v[int(p.table[0, i])]
    small = p.table.copy()
    p.k, p.v, p.table = k, v, np.array([far], np.int32)
    run(wq, p)
    p.table = small
    p.check()
    del k, v, p
    torch.cuda.empty_cache()


# --- norms, rotation, append -------------------------------------------------


def rope_case(wq, rng, lengths, counts, heads, kv, dim, rot, page, interleaved, norm, f32, positions=None, pad_rows=0,
              rot_scale=1.0, layout="NHD"):
    import torch
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    tokens = int(starts[-1]) + pad_rows
    table, pages = pages_for(rng, [max(a, 0) + b for a, b in zip(lengths, counts)], page)
    k64, k = bf16(rng.normal(size=(pages, page, kv, dim)))
    v64, v = bf16(rng.normal(size=(pages, page, kv, dim)))
    if layout == "HND":
        k, v = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (k, v))
    raw = rng.normal(size=(tokens, (heads + 2 * kv) * dim)).astype(np.float32)
    if f32:
        qkv64, qkv = raw.astype(np.float64), torch.from_numpy(raw).cuda()
    else:
        qkv64, qkv = bf16(raw)
    qn64, qn = bf16(1 + 0.2 * rng.normal(size=dim))
    kn64, kn = bf16(1 + 0.2 * rng.normal(size=dim))
    freq = wq.wq_rope_frequencies(rot, 10000.0)[0] if rot else None
    q = torch.full((tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = wq.wq_qkv_rope_prepare(qkv, q, k, v, i32(table), i32(starts), i32(lengths),
                                  None if freq is None else freq.cuda(),
                                  positions=None if positions is None else i32(positions),
                                  q_norm=qn if norm in ("both", "q") else None,
                                  k_norm=kn if norm in ("both", "k") else None, eps=1e-5, rot_scale=rot_scale,
                                  interleaved=interleaved)
    wq.wq_qkv_rope_run(plan)
    torch.cuda.synchronize()
    args = dict(positions=positions, q_norm=qn64 if norm in ("both", "q") else None,
                k_norm=kn64 if norm in ("both", "k") else None, eps=1e-5, rot_scale=rot_scale, interleaved=interleaved)
    f = [] if freq is None else freq.double().numpy()
    wq_, wk, wv = verify.qkv_rope(qkv64, k64, v64, table, starts, lengths, heads, f, **args)
    # magnitudes of a pair: the same call with the partner's part taken in absolute value is bounded by the pair's sum
    def pair(w):
        a, half = np.abs(w), rot // 2
        out = a.copy()
        if rot and interleaved:
            s = a[..., 0:rot:2] + a[..., 1:rot:2]
            out[..., 0:rot:2], out[..., 1:rot:2] = s, s
        elif rot:
            s = a[..., :half] + a[..., half:rot]
            out[..., :half], out[..., half:rot] = s, s
        return out * 1.5
    for got, want, what in ((q, wq_, "q"), (k, wk, "k"), (v, wv, "v")):
        got = f64(got)
        alone = np.isnan(want)
        assert np.all(got[alone] == 7.0), what
        want = np.where(alone, 7.0, want)
        off = np.abs(got - want) - BF16 * np.abs(want) - 2.0 ** -16 * pair(want)
        assert np.all(off <= 0), (what, np.unravel_index(off.argmax(), off.shape), off.max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["none", "both", "q", "k"])
@pytest.mark.parametrize("f32", [False, True])
def test_rope_kinds(wq, interleaved, norm, f32):
    rng = np.random.default_rng(40)
    rope_case(wq, rng, [5, 0, 100], [3, 1, 4], 8, 2, 128, 128, 16, interleaved, norm, f32)


@pytest.mark.parametrize("dim,rot", [(8, 8), (8, 2), (64, 64), (64, 32), (80, 32), (96, 24), (96, 96), (128, 20),
                                     (128, 0), (256, 256), (256, 64), (192, 6), (120, 120), (72, 70)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_dims(wq, dim, rot, interleaved):
    rng = np.random.default_rng(dim + rot)
    rope_case(wq, rng, [9, 30], [2, 3], 6, 3, dim, rot, 7, interleaved, "both", False, rot_scale=1.25)


def test_rope_far_positions_and_depths(wq):
    rng = np.random.default_rng(41)
    for positions in (None, [0, 131071, 2 ** 20 + 1, 2 ** 30, 5, -3, 77, 1000003]):
        rope_case(wq, rng, [3, 40], [4, 4], 4, 4, 64, 64, 16, False, "none", True, positions=positions)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page", [1, 16, 50])
def test_rope_pages_and_unused_rows(wq, layout, page):
    rng = np.random.default_rng(42)
    rope_case(wq, rng, [0, 49, -2, 7], [2, 0, 3, 1], 4, 1, 64, 64, page, False, "both", False, pad_rows=2,
              layout=layout)


def test_rope_many_requests_and_rows(wq):
    rng = np.random.default_rng(43)
    counts = [int(rng.integers(0, 4)) for _ in range(150)]
    rope_case(wq, rng, [int(rng.integers(0, 60)) for _ in counts], counts, 4, 2, 64, 32, 16, True, "q", False)


def test_rope_positions_without_a_page_are_dropped(wq):
    import torch
    rng = np.random.default_rng(44)
    k = torch.full((2, 4, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    qkv = torch.randn(6, 3 * 64, device="cuda")
    q = torch.full((6, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    # positions 2 .. 7: page 0 is the pool's page 1, page 1 is outside; request 1's start past its table
    plan = wq.wq_qkv_rope_prepare(qkv, q, k, v, i32([[1, 2], [0, -5]]), i32([0, 4, 6]), i32([2, 2 ** 31 - 1]))
    wq.wq_qkv_rope_run(plan)
    torch.cuda.synchronize()
    assert torch.equal(q.view(6, 64), qkv[:, :64].to(torch.bfloat16))
    want = torch.full_like(k, 7.0)
    want[1, 2:4, 0] = qkv[:2, 64:128].to(torch.bfloat16)
    assert torch.equal(k, want)


# --- accepted rows -----------------------------------------------------------


@pytest.mark.parametrize("layers,kv,dim,page", [(1, 8, 128, 16), (3, 2, 64, 5), (2, 3, 72, 1), (5, 32, 256, 64)])
def test_accept(wq, layers, kv, dim, page):
    import torch
    rng = np.random.default_rng(layers * 100 + page)
    lengths = [0, 33, 7, 100, 12, 5]
    paths = [[0, 1, 2, 5], [0, 3, 9, 30], [2, 3, 4, 63], [5, 5, 6, 7], [0, 2, 1, 8], [1, 2, 3, 4]]
    accepted = [4, 3, 4, 4, 4, 0]
    spans = [a + 64 for a in lengths]
    table, pages = pages_for(rng, spans, page)
    k = torch.from_numpy(rng.integers(-30000, 30000, (layers, pages, page, kv, dim)).astype(np.int16)).cuda()
    v = torch.from_numpy(rng.integers(-30000, 30000, (layers, pages, page, kv, dim)).astype(np.int16)).cuda()
    wk, wv = verify.kv_accept(k.cpu().numpy(), v.cpu().numpy(), table, lengths, np.array(paths), accepted)
    plan = wq.wq_kv_accept_prepare(k, v, i32(table), i32(lengths), i32(paths), i32(accepted))
    wq.wq_kv_accept_run(plan)
    torch.cuda.synchronize()
    assert np.array_equal(k.cpu().numpy(), wk) and np.array_equal(v.cpu().numpy(), wv)


def test_accept_long_paths_and_missing_pages(wq):
    import torch
    rng = np.random.default_rng(61)
    k = torch.from_numpy(rng.integers(-30000, 30000, (2, 40, 4, 2, 64)).astype(np.int16)).cuda()
    v = torch.flip(k, [1]).contiguous()
    table = np.stack([np.arange(18), np.arange(18, 36)]).astype(np.int32)
    table[0, 9] = -1
    table[1, 3] = 40
    path = np.stack([np.arange(64), np.sort(rng.permutation(66)[:64])]).astype(np.int32)
    path[0, 1:] += 1
    lengths, accepted = [3, 2], [64, 1000]
    wk, wv = verify.kv_accept(k.cpu().numpy(), v.cpu().numpy(), table, lengths, path, accepted)
    plan = wq.wq_kv_accept_prepare(k, v, i32(table), i32(lengths), i32(path), i32(accepted))
    wq.wq_kv_accept_run(plan)
    torch.cuda.synchronize()
    assert np.array_equal(k.cpu().numpy(), wk) and np.array_equal(v.cpu().numpy(), wv)


def test_accept_one_layer_with_heads_first(wq):
    import torch
    rng = np.random.default_rng(62)
    k = torch.randn(6, 2, 8, 64, device="cuda").to(torch.bfloat16).permute(0, 2, 1, 3)
    v = torch.randn(6, 2, 8, 64, device="cuda").to(torch.bfloat16).permute(0, 2, 1, 3)
    table, path = np.array([[4, 2, 0]], np.int32), np.array([[1, 4, 9]], np.int32)
    wk, wv = verify.kv_accept(f64(k)[None], f64(v)[None], table, [6], path, [3])
    plan = wq.wq_kv_accept_prepare(k, v, i32(table), i32([6]), i32(path), i32([3]))
    wq.wq_kv_accept_run(plan)
    torch.cuda.synchronize()
    assert np.array_equal(f64(k), wk[0]) and np.array_equal(f64(v), wv[0])


# --- adapters ----------------------------------------------------------------


def lora_case(wq, rng, adapter, adapters, rank, k, n, out=("f32",), base=True, ranks=None, scale=True, in_place=False,
              pad=0):
    import torch
    tokens = len(adapter)
    x64, x = bf16(rng.normal(size=(tokens, k)))
    a64, a = bf16(rng.normal(size=(adapters, rank, k)) / np.sqrt(k))
    b64, b = bf16(rng.normal(size=(adapters, n, rank)) / np.sqrt(rank))
    if ranks is not None:
        for c, r in enumerate(ranks):
            a[c, max(r, 0):] = float("nan")
            b[c, :, max(r, 0):] = float("inf")
    s = (rng.random(adapters) + 0.5).astype(np.float32) if scale else None
    bs = rng.normal(size=(tokens, n)).astype(np.float32) if base else None

    def rows(dtype):
        whole = torch.full((tokens, n + pad), 7.0, dtype=dtype, device="cuda")
        return whole, whole[:, :n]
    (w32, y32), (w16, y16) = rows(torch.float32), rows(torch.bfloat16)
    tb = torch.from_numpy(bs).cuda() if base else None
    if in_place:
        y32.copy_(tb)
        tb = y32
    outs = [{"f32": y32, "bf16": y16}[o] for o in out]
    plan = wq.wq_lora_prepare(x, a, b, i32(adapter), *outs, base=tb, ranks=None if ranks is None else i32(ranks),
                              scale=None if s is None else torch.from_numpy(s).cuda())
    wq.wq_lora_run(plan)
    torch.cuda.synchronize()
    want, deep, flat = verify.lora(x64, a64, b64, adapter, bs, ranks, s)
    tol = 2 * ((k + 8) * 2.0 ** -24 * deep + (3 * rank + 8) * 2.0 ** -24 * flat) + 2.0 ** -22 * np.abs(want)
    for o, y, w in (("f32", y32, w32), ("bf16", y16, w16)):
        if o in out:
            off = np.abs(f64(y) - want) - tol - (BF16 * np.abs(want) if o == "bf16" else 0)
            assert np.all(off <= 0), (o, np.unravel_index(off.argmax(), off.shape), off.max())
            assert torch.all(w[:, n:] == 7.0)
    return plan, (y32, y16)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 56, 64, 128])
@pytest.mark.parametrize("k,n", [(8, 1), (72, 50), (512, 64), (4096, 133), (1000, 2052)])
def test_lora_sizes(wq, rank, k, n):
    rng = np.random.default_rng(rank + k + n)
    lora_case(wq, rng, [1, 0, 1, 2, -1, 0], 3, rank, k, n)


@pytest.mark.parametrize("out", [("f32",), ("bf16",), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("base,in_place", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("pad", [0, 3, 4])
def test_lora_outputs(wq, out, base, in_place, pad):
    rng = np.random.default_rng(70)
    lora_case(wq, rng, [0, 1, -1, 1, 1], 2, 16, 256, 100, out=out, base=base, in_place=in_place and "f32" in out,
              pad=pad)


def test_lora_one_token(wq):
    rng = np.random.default_rng(71)
    lora_case(wq, rng, [5], 8, 16, 4096, 6144, out=("bf16",))
    lora_case(wq, rng, [-1], 8, 16, 4096, 6144, out=("bf16",))
    lora_case(wq, rng, [8], 8, 16, 64, 64, scale=False, base=False)
    lora_case(wq, rng, [0], 1, 8, 16384, 40)


def test_lora_ranks_that_end_anywhere(wq):
    rng = np.random.default_rng(72)
    lora_case(wq, rng, [0, 1, 2, 3, 4, 5, 0, 1], 6, 16, 128, 70, ranks=[16, 5, 0, -3, 9, 99])


@pytest.mark.parametrize("tokens,adapters", [(16, 1), (17, 1), (200, 3), (500, 40), (1000, 7), (4096, 2), (33, 4096)])
def test_lora_groups(wq, tokens, adapters):
    rng = np.random.default_rng(tokens + adapters)
    adapter = rng.integers(-1, adapters + 1, tokens)
    if adapters == 4096:
        adapter = rng.choice([0, 4095, 17], tokens)
    lora_case(wq, rng, adapter, adapters, 8, 64, 36)


def test_lora_rows_do_not_meet(wq):
    """NaN in one row of x, and in an adapter that another row uses, stays there."""
    import torch
    rng = np.random.default_rng(73)
    x = torch.randn(6, 128, device="cuda").to(torch.bfloat16)
    a = torch.randn(3, 16, 128, device="cuda").to(torch.bfloat16)
    b = torch.randn(3, 40, 16, device="cuda").to(torch.bfloat16)
    y, z = torch.zeros(6, 40, device="cuda"), torch.zeros(6, 40, device="cuda")
    adapter = i32([0, 0, 1, 2, 1, 0])
    wq.wq_lora_run(wq.wq_lora_prepare(x, a, b, adapter, y))
    x[1, 77], a[1, 3, 5], b[2, 9, 9] = float("nan"), float("inf"), float("nan")
    wq.wq_lora_run(wq.wq_lora_prepare(x, a, b, adapter, z))
    torch.cuda.synchronize()
    assert torch.equal(y[[0, 5]], z[[0, 5]])
    assert torch.isnan(z[1]).all() and torch.isnan(z[3, 9])
    keep = [i for i in range(40) if i != 9]
    assert torch.equal(y[3, keep], z[3, keep])


# --- empty calls, streams, graphs, devices -----------------------------------


def test_empty_batches(wq):
    import torch
    z = dict(dtype=torch.bfloat16, device="cuda")
    k = torch.full((2, 16, 2, 64), 7.0, **z)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    zero = i32([0])
    table = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    q, y = torch.empty(0, 4, 64, **z), torch.empty(0, 4, 64, **z)
    wq.wq_tree_attention_run(wq.wq_tree_attention_prepare(q, k, k.clone(), table, zero, none, y))
    wq.wq_qkv_rope_run(wq.wq_qkv_rope_prepare(torch.empty(0, 512, **z), q, k, k.clone(), table, zero, none))
    wq.wq_kv_accept_run(wq.wq_kv_accept_prepare(k, k.clone(), table, none, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), none))
    wq.wq_lora_run(wq.wq_lora_prepare(torch.empty(0, 64, **z), torch.zeros(1, 8, 64, **z), torch.zeros(1, 32, 8, **z), none,
                                      torch.empty(0, 32, **z)))
    wq.wq_lora_run(wq.wq_lora_prepare(torch.zeros(2, 64, **z), torch.zeros(1, 8, 64, **z), torch.empty(1, 0, 8, **z), i32([0, 0]),
                                      torch.empty(2, 0, **z)))
    torch.cuda.synchronize()
    assert torch.all(k == 7.0)


def test_prepare_refuses_what_does_not_fit(wq):
    import torch
    z = dict(dtype=torch.bfloat16, device="cuda")
    k, q = torch.zeros(2, 16, 2, 64, **z), torch.zeros(3, 4, 64, **z)
    args = [q, k, k, i32([[0]]), i32([0, 3]), i32([0]), q.clone()]

    def refuse(at, t, error=ValueError):
        with pytest.raises(error):
            wq.wq_tree_attention_prepare(*[t if i == at else a for i, a in enumerate(args)])
    refuse(0, q.float())
    refuse(0, q[:2])
    refuse(0, torch.zeros(3, 4, 56, **z))
    refuse(1, k[:, :8])
    refuse(1, k.cpu())
    refuse(3, i32([[0]]).long())
    refuse(3, i32([[0]])[:0])
    refuse(4, i32([0, 1, 3]))
    refuse(6, q.clone().transpose(0, 1))
    refuse(6, torch.zeros(3, 260, **z)[:, 2:258], wq.WQError)       # misaligned rows
    refuse(0, q.view(-1)[:512].view(8, 64).expand(8, 64))
    with pytest.raises(wq.WQError):
        wq.wq_tree_attention_prepare(*args, max_tokens=65)
    with pytest.raises(wq.WQError):
        wq.wq_tree_attention_prepare(*args, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        wq.wq_tree_attention_prepare(*args, tree=torch.zeros(2, dtype=torch.int64, device="cuda"))


class Layer:
    """The attention half of a verify pass: wqkv (int4, adapters) -> rope and append -> tree attention -> wo
    (int8, adapters) -> acceptance."""

    def __init__(self, wq, rng, lengths, counts, device="cuda"):
        import torch
        self.wq, self.heads, self.kv, self.dim, self.width = wq, 8, 2, 64, 512
        heads, kv, dim, width = self.heads, self.kv, self.dim, self.width
        self.m, out = sum(counts), (heads + 2 * kv) * dim
        self.counts, self.lengths = counts, lengths
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.wqkv = torch.from_numpy(rng.normal(size=(out, width)).astype(np.float32) * 0.05).cuda()
        self.wo = torch.from_numpy(rng.normal(size=(width, width)).astype(np.float32) * 0.05).cuda()
        self.p = torch.empty(out, width // 2, dtype=torch.uint8, device="cuda")
        self.sz = torch.empty(out, width // 32, 2, dtype=torch.int16, device="cuda")
        wq.wq_quantize_int4g32(self.wqkv, out, width, self.p, self.sz)
        self.o = torch.empty(width, width, dtype=torch.int8, device="cuda")
        self.os = torch.empty(width, dtype=torch.int16, device="cuda")
        wq.wq_quantize_int8(self.wo, width, width, self.o, self.os)
        _, self.x = bf16(rng.normal(size=(self.m, width)))
        ad = {}
        for name, n in (("qkv", out), ("o", width)):
            ad[name] = (bf16(rng.normal(size=(3, 16, width)) / 23)[1], bf16(rng.normal(size=(3, n, 16)) / 4)[1])
        self.ad = ad
        self.adapter = i32([[-1, 0, 2][r % 3] for r, n in enumerate(counts) for _ in range(n)])
        table, pages = pages_for(rng, [a + b for a, b in zip(lengths, counts)], 16)
        self.table_np = table
        self.table, self.dstarts, self.dlengths = i32(table), i32(self.starts), i32(lengths)
        self.k, self.v = (bf16(rng.normal(size=(pages, 16, kv, dim)))[1] for _ in range(2))
        masks, self.positions = [], []
        for r, n in enumerate(counts):
            t = random_tree(rng, n)
            masks += t
            self.positions += [lengths[r] + bin(x).count("1") - 1 for x in t]
        self.masks = masks
        self.tree = torch.from_numpy(as_i64(masks)).cuda()
        self.freq = wq.wq_rope_frequencies(dim, 10000.0)[0].cuda()
        self.qn, self.kn = (bf16(1 + 0.1 * rng.normal(size=dim))[1] for _ in range(2))
        e = dict(device="cuda")
        self.qkv = torch.empty(self.m, out, dtype=torch.float32, **e)
        self.q = torch.empty(self.m, heads, dim, dtype=torch.bfloat16, **e)
        self.y = torch.empty_like(self.q)
        self.z = torch.empty(self.m, width, dtype=torch.float32, **e)
        self.out = torch.empty(self.m, width, dtype=torch.float32, **e)
        self.lora_qkv = wq.wq_lora_prepare(self.x, *ad["qkv"], self.adapter, self.qkv, base=self.qkv)
        self.rope = wq.wq_qkv_rope_prepare(self.qkv, self.q, self.k, self.v, self.table, self.dstarts, self.dlengths,
                                           self.freq, positions=i32(self.positions), q_norm=self.qn, k_norm=self.kn)
        self.attn = wq.wq_tree_attention_prepare(self.q, self.k, self.v, self.table, self.dstarts, self.dlengths, self.y,
                                                 tree=self.tree, max_tokens=max(counts))
        self.lora_o = wq.wq_lora_prepare(self.y.view(self.m, width), *ad["o"], self.adapter, self.out, base=self.z)
        self.path = np.array([[0, min(2, n - 1)] if n > 1 else [0, 1] for n in counts], np.int32)
        self.accepted = [2 if n > 1 else 1 for n in counts]
        self.accept = wq.wq_kv_accept_prepare(self.k, self.v, self.table, self.dlengths, i32(self.path),
                                              i32(self.accepted))

    def step(self, stream=None):
        wq = self.wq
        wq.wq_gemm_smallM(self.x, self.m, self.p, self.sz, self.qkv.shape[1], self.width, self.qkv, None, stream)
        wq.wq_lora_run(self.lora_qkv, stream)
        wq.wq_qkv_rope_run(self.rope, stream)
        wq.wq_tree_attention_run(self.attn, stream)
        wq.wq_gemm_smallM_int8(self.y, self.m, self.o, self.os, self.width, self.width, self.z, None, stream)
        wq.wq_lora_run(self.lora_o, stream)

    def expected(self):
        """In fp64, rounding to bf16 where the calls do."""
        from oracle.matvec import gemm_small_m
        ad = self.adapter.cpu().numpy()
        x = f64(self.x)
        bits = self.x.view(__import__("torch").int16).cpu().numpy().view(np.uint16)
        qkv = gemm_small_m(bits, self.p.cpu().numpy(), self.sz.cpu().numpy().view(np.uint16))
        qkv, _, _ = verify.lora(x, *(f64(t) for t in self.ad["qkv"]), ad, qkv)
        q, k, v = verify.qkv_rope(qkv, f64(self.k), f64(self.v), self.table_np, self.starts, self.lengths, self.heads,
                                  self.freq.cpu().double().numpy(), self.positions, f64(self.qn), f64(self.kn))
        q, k, v = (bf16(t)[0] for t in (q, k, v))
        y, _ = verify.tree_attention(q, k, v, self.table_np, self.starts, self.lengths, self.dim ** -0.5, self.masks)
        y = bf16(y)[0].reshape(self.m, self.width)
        scale = (self.os.cpu().numpy().view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        z = y @ (self.o.cpu().numpy().astype(np.float64) * scale[:, None]).T
        z, _, _ = verify.lora(y, *(f64(t) for t in self.ad["o"]), ad, z)
        return z, k, v


def test_a_verify_pass_of_a_layer(wq):
    """Every call in a row as a user makes them, eager, on another stream and as a captured graph."""
    import torch
    rng = np.random.default_rng(90)
    lay = Layer(wq, rng, [37, 200], [5, 3])
    want, wk, wv = lay.expected()
    lay.step()
    torch.cuda.synchronize()
    # q, k, y are rounded to bf16 before they are used again: a value next to a border may fall to its other
    # side (2^-8 of it), so outputs are compared in the max norm with room for two such roundings
    def close(got):
        return np.abs(f64(got) - want).max() <= 4 * BF16 * np.abs(want).max()
    assert close(lay.out)
    assert np.all(np.abs(f64(lay.k) - wk) <= 2 * BF16 * np.abs(wk) + 1e-4)
    first = lay.out.clone()
    say("layer pass: max error", np.abs(f64(lay.out) - want).max() / np.abs(want).max())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lay.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lay.step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(lay.out, first)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.step()
    for i in range(4):
        lay.out.zero_()
        lay.q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.out, first), i
        torch.randn(1000, device="cuda").sum().item()
    # the graph reads lengths at replay
    lay.dlengths.copy_(i32([20, 100]))
    graph.replay()
    torch.cuda.synchronize()
    shorter = lay.out.clone()
    lay.out.zero_()
    lay.step()
    torch.cuda.synchronize()
    assert torch.equal(lay.out, shorter) and not torch.equal(shorter, first)
    lay.dlengths.copy_(i32(lay.lengths))
    lay.step()

    ak, av = verify.kv_accept(f64(lay.k)[None], f64(lay.v)[None], lay.table_np, lay.lengths, lay.path, lay.accepted)
    wq.wq_kv_accept_run(lay.accept)
    torch.cuda.synchronize()
    assert np.array_equal(f64(lay.k), ak[0]) and np.array_equal(f64(lay.v), av[0])


def test_two_plans_on_two_streams(wq):
    """Plans with workspaces of their own, at once."""
    import torch
    rng = np.random.default_rng(91)
    ps = [Attn(rng, [3000, 100], [5, 2], 8, 2, 128, 16), Attn(rng, [2500], [8], 8, 2, 128, 64)]
    plans = [p.plan(wq) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for plan, s in zip(plans, streams):
            wq.wq_tree_attention_run(plan, s)
    torch.cuda.synchronize()
    for p in ps:
        p.check()


def test_two_adapter_plans_on_two_streams(wq):
    import torch
    rng = np.random.default_rng(92)
    one, (y, _) = lora_case(wq, rng, [0, 1, 2, 0, -1], 3, 16, 2048, 3000)
    two, (z, _) = lora_case(wq, rng, [1] * 40, 2, 32, 1024, 2500)
    wy, wz = y.clone(), z.clone()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        y.zero_(), z.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            wq.wq_lora_run(one, s)
            wq.wq_lora_run(two, t)
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(z, wz)


# --- further shapes ----------------------------------------------------------


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("heads,n", [(4, 2), (16, 30)])
def test_attention_scales(wq, scale, heads, n):
    # a negative scale turns the order round, a zero one leaves the mean
    rng = np.random.default_rng(100)
    p = Attn(rng, [200, 3], [n, n], heads, 2, 64, 16, scale=scale, tree=lambda m: random_tree(rng, m))
    run(wq, p)
    p.check()


@pytest.mark.parametrize("requests", [65, 130, 600])
@pytest.mark.parametrize("heads", [2, 40])
def test_attention_many_requests(wq, requests, heads):
    rng = np.random.default_rng(requests)
    lengths = [int(rng.integers(0, 40)) for _ in range(requests)]
    lengths[requests // 2] = 1500
    counts = [int(rng.integers(0, 3)) for _ in range(requests)]
    counts[requests // 2] = 2
    p = Attn(rng, lengths, counts, heads, 2, 64, 16, pad_rows=1)
    run(wq, p)
    p.check()


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("page", [16, 11, 24])
def test_attention_wide_trees(wq, dim, page):
    rng = np.random.default_rng(dim + page)
    p = Attn(rng, [700, 0, 129], [64, 40, 1], 16, 2, dim, page, tree=lambda m: random_tree(rng, m))
    run(wq, p)
    p.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads,dim,page", [(4, 128, 16), (16, 128, 16), (64, 64, 16), (16, 96, 16), (8, 256, 16), (16, 128, 9)])
def test_attention_unseen_specials_in_every_kernel(wq, bad, heads, dim, page):
    """Draft 2 holds infinities or NaN that only its own row sees; 1200 positions cut the groups."""
    import torch
    rng = np.random.default_rng(dim + heads)
    p = Attn(rng, [1200], [6], heads, 2, dim, page, tree=lambda n: [1, 3, 5, 9, 27, 33])
    run(wq, p)
    clean = p.y.clone()
    at = int(p.table[0, 1202 // page]), 1202 % page
    p.k[at], p.v[at] = bad, bad
    p.y.fill_(7.0)
    run(wq, p)
    same = [0, 1, 3, 4, 5]
    assert torch.equal(p.y[same], clean[same])
    assert not torch.isfinite(p.y[2]).any()


def test_attention_shares_pages_between_requests(wq):
    rng = np.random.default_rng(101)
    p = Attn(rng, [160, 160], [2, 2], 4, 2, 64, 16)
    p.table[1, :10] = p.table[0, :10]        # a common prefix
    run(wq, p)
    p.check()


def test_attention_capture_with_a_workspace_of_its_own(wq):
    """A captured run and eager runs of another plan between its replays."""
    import torch
    rng = np.random.default_rng(102)
    a, b = Attn(rng, [3000], [5], 8, 2, 128, 16), Attn(rng, [2000, 40], [3, 8], 16, 2, 64, 16)
    need = wq.wq_tree_attention_workspace_bytes(1, 8, 2, 128, 5)
    pa = a.plan(wq, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    pb = b.plan(wq)
    wq.wq_tree_attention_run(pa)
    torch.cuda.synchronize()
    first = a.y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_tree_attention_run(pa)
    for _ in range(4):
        a.y.fill_(7.0)
        graph.replay()
        wq.wq_tree_attention_run(pb)
        torch.cuda.synchronize()
        assert torch.equal(a.y, first)
        b.check()


def test_a_plan_of_another_device_is_refused(wq):
    rng = np.random.default_rng(103)
    p = Attn(rng, [20], [2], 2, 2, 64, 16)
    plan = p.plan(wq)
    plan.device = 7                          # as if prepared on device 7
    with pytest.raises(wq.WQError, match="DEVICE"):
        wq.wq_tree_attention_run(plan, stream=0)
    with pytest.raises(wq.WQError, match="SHAPE"):
        wq.wq_tree_attention_prepare(p.q, p.k, p.v, i32(p.table), i32(p.starts), i32(p.lengths), p.q)


def test_rope_rows_of_no_request_and_queries_in_wide_rows(wq):
    import torch
    rng = np.random.default_rng(104)
    k = torch.full((3, 16, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.full((5, 4 * 64 + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    raw = torch.randn(5, 8 * 64 + 16, device="cuda")
    plan = wq.wq_qkv_rope_prepare(raw[:, 4:4 + 512], wide[:, 16:272], k, k.clone(), i32([[1, 2]]), i32([1, 4]), i32([3]))
    wq.wq_qkv_rope_run(plan)
    torch.cuda.synchronize()
    assert torch.equal(wide[1:4, 16:272], raw[1:4, 4:260].to(torch.bfloat16))
    assert torch.all(wide[0] == 7.0) and torch.all(wide[4] == 7.0)
    assert torch.all(wide[:, :16] == 7.0) and torch.all(wide[:, 272:] == 7.0)
    want = torch.full_like(k, 7.0)
    want[1, 3:6] = raw[1:4, 260:388].to(torch.bfloat16).view(3, 2, 64)
    assert torch.equal(k, want)


@pytest.mark.parametrize("tokens", [1, 2, 17, 31, 32, 33])
@pytest.mark.parametrize("rank,k", [(8, 64), (16, 1024), (16, 2048), (32, 1024), (16, 2056), (32, 4096)])
def test_lora_one_launch_and_two(wq, tokens, rank, k):
    # both sides of the rule that chooses one launch: 32 rows, rank * k of 32768
    rng = np.random.default_rng(tokens * rank + k)
    lora_case(wq, rng, rng.integers(-1, 5, tokens), 5, rank, k, 600, out=("f32", "bf16"), pad=1, ranks=[rank, 3, 8, 0, 99])


def test_lora_graph_follows_changed_adapters(wq):
    import torch
    rng = np.random.default_rng(105)
    for rank, k in ((16, 512), (32, 4096)):
        plan, (y, _) = lora_case(wq, rng, [0, 1, 2, 0, -1, 2, 1], 3, rank, k, 900)
        adapter = plan.keep[3]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            wq.wq_lora_run(plan)
        for _ in range(4):
            adapter.copy_(i32(rng.integers(-1, 3, 7)))
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone()
            y.zero_()
            wq.wq_lora_run(plan)
            torch.cuda.synchronize()
            assert torch.equal(got, y)


@pytest.mark.parametrize("dim,max_tokens", [(64, 1), (64, 64), (96, 64), (128, 8), (128, 64), (256, 64)])
def test_attention_of_the_most_requests(wq, dim, max_tokens):
    # whatever the number of requests leaves of LDS
    rng = np.random.default_rng(dim + max_tokens)
    lengths = [int(rng.integers(0, 9)) for _ in range(4096)]
    lengths[77] = 900
    counts = [int(rng.integers(0, 2)) for _ in range(4096)]
    counts[77], counts[4095] = 1, max_tokens
    p = Attn(rng, lengths, counts, 4, 2, dim, 8)
    run(wq, p, max_tokens=max_tokens)
    p.check()


@pytest.mark.parametrize("rank,out", [(16, "f32"), (16, "bf16"), (64, "f32"), (64, "bf16")])
def test_lora_sums_that_are_infinite_or_nearly(wq, rank, out):
    import torch
    rng = np.random.default_rng(rank)
    x, a = np.zeros((3, 64)), np.zeros((1, rank, 64))
    x[0, 0], x[1, 0], x[2, 0] = np.inf, -np.inf, 2.0 ** 127
    x[2, 1] = 2.0 ** 126
    a[0, :, 0], a[0, :, 1] = 1.0, 1.9921875            # row 2: A x = 1.99609375 * 2^127 rounds to no finite bf16
    b = rng.uniform(1, 2, size=(1, 40, rank)) * 2.0 ** -100
    b[0, 7], b[0, 8, 3] = -b[0, 7], -b[0, 8, 3]        # -inf, and inf - inf
    a64, at = bf16(a)
    b64, bt = bf16(b)
    y = torch.zeros(3, 40, device="cuda", dtype=torch.float32 if out == "f32" else torch.bfloat16)
    wq.wq_lora_run(wq.wq_lora_prepare(torch.from_numpy(x).to(torch.bfloat16).cuda(), at, bt, i32([0, 0, 0]), y))
    torch.cuda.synchronize()
    got = f64(y)
    h = 1.99609375 * 2.0 ** 127
    want = np.stack([np.inf * np.sign(b64[0]).sum(1), -np.inf * np.sign(b64[0]).sum(1), h * b64[0].sum(1)])
    want[:2, 8] = np.nan
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[:2, [i for i in range(40) if i != 8]], want[:2, [i for i in range(40) if i != 8]])
    reach = h * np.abs(b64[0]).sum(1)
    tol = (3 * rank + 8) * 2.0 ** -24 * reach + (BF16 * np.abs(want[2]) + 2.0 ** -16 * reach if out == "bf16" else 0)
    assert np.all(np.abs(got[2] - want[2]) <= tol)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("n,heads", [(1, 4), (5, 8), (40, 32)])
def test_attention_of_one_visible_position_is_its_value(wq, dim, n, heads):
    # the sum has the weight as the product has it, rounded
    rng = np.random.default_rng(dim + n)
    p = Attn(rng, [0, 0, 0], [n, n, n], heads, 4, dim, 16, tree=[1 << i for i in range(n)])
    run(wq, p)
    for r in range(3):
        for i in range(n):
            row = int(p.table[r][i // 16]), i % 16
            want = np.repeat(p.v64[row], heads // 4, axis=0)
            assert np.array_equal(f64(p.y[int(p.starts[r]) + i]), want)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("lengths", [(300, 0, 90), (2200, 1900, 2300)])
def test_attention_wide_trees_over_short_and_long_tables(wq, dim, lengths):
    # the rows times the positions of the table choose the kernel; one workspace size serves both
    rng = np.random.default_rng(dim + lengths[0])
    p = Attn(rng, lengths, [64, 33, 64], 64, 4, dim, 16, tree=lambda n: random_tree(rng, n))
    assert wq.wq_tree_attention_workspace_bytes(3, 64, 4, dim, 64) > wq.wq_tree_attention_workspace_bytes(3, 4, 4, dim, 64)
    run(wq, p, max_tokens=64)
    p.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 9), (96, 16), (128, 16), (128, 9), (128, 24)])
def test_attention_unseen_specials_of_wide_trees_over_long_tables(wq, bad, dim, page):
    """The same where blocks of the most rows are taken: draft 2 of the third request of four."""
    import torch
    rng = np.random.default_rng(dim + page)
    p = Attn(rng, [1300, 20, 1200, 1500], [6] * 4, 64, 2, dim, page, tree=[1, 3, 5, 9, 27, 33])
    run(wq, p, max_tokens=64)
    p.check()
    clean = p.y.clone()
    at = int(p.table[2, 1202 // page]), 1202 % page
    p.k[at], p.v[at] = bad, bad
    p.y.fill_(7.0)
    run(wq, p, max_tokens=64)
    same = [i for i in range(24) if i != 14]
    assert torch.equal(p.y[same], clean[same])
    assert not torch.isfinite(p.y[14]).any()


def test_attention_wide_trees_captured(wq):
    import torch
    rng = np.random.default_rng(55)
    p = Attn(rng, [1800, 700, 1500], [64, 40, 64], 64, 4, 128, 16, tree=lambda n: random_tree(rng, n))
    plan = p.plan(wq, max_tokens=64)
    wq.wq_tree_attention_run(plan)
    torch.cuda.synchronize()
    p.check()
    eager = p.y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_tree_attention_run(plan)
    for _ in range(3):
        p.y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y, eager)
        p.y.fill_(7.0)
        wq.wq_tree_attention_run(plan)
        torch.cuda.synchronize()
        assert torch.equal(p.y, eager)


@pytest.mark.parametrize("requests,heads,kv,dim,max_tokens", [(2048, 4, 2, 64, 64), (2048, 4, 2, 96, 64), (2048, 4, 2, 128, 64),
                                                             (256, 2, 1, 128, 3), (256, 2, 1, 96, 3), (257, 2, 1, 128, 3)])
def test_attention_where_a_kernel_takes_its_most_requests(wq, requests, heads, kv, dim, max_tokens):
    rng = np.random.default_rng(requests + dim)
    lengths = [int(rng.integers(0, 9)) for _ in range(requests)]
    lengths[77] = 900
    counts = [int(rng.integers(0, 3)) for _ in range(requests)]
    counts[77], counts[requests - 1] = 1, max_tokens
    p = Attn(rng, lengths, counts, heads, kv, dim, 8)
    run(wq, p, max_tokens=max_tokens)
    p.check()


@pytest.mark.parametrize("power", [20, 26, 34, 60, 90])
@pytest.mark.parametrize("lengths,counts,heads,kv,dim,page", [
    ([500], [1], 4, 4, 128, 16), ([1300, 40], [5, 3], 16, 2, 64, 11), ([900, 0, 2100], [16, 4, 9], 8, 1, 96, 16),
    ([700, 90], [33, 64], 8, 2, 128, 13), ([4100, 1900], [64, 64], 64, 2, 128, 16), ([1200], [7], 8, 2, 256, 16)])
def test_attention_scores_of_any_size(wq, power, lengths, counts, heads, kv, dim, page):
    """Every second token's scores are 2^power times as large.  Queries and keys are small integers, so that scores are
    exact and their weight is all on the largest, shared where several are equal, whatever the rounding of the product
    of score and scale (half a step of it is 2^power / 2^24)."""
    rng = np.random.default_rng(power + heads + dim)
    p = Attn(rng, lengths, counts, heads, kv, dim, page, tree=lambda n: random_tree(rng, n))
    p.k64, p.k = bf16(np.rint(1.5 * p.k64))
    q = np.rint(1.5 * p.q64)
    q[::2] *= 2.0 ** power
    p.q64, p.q = bf16(q)
    run(wq, p, max_tokens=64 if max(counts) > 16 else None)
    p.check()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("heads,kv,dim,n,page", [(4, 4, 128, 1, 16), (16, 2, 64, 5, 16), (16, 2, 128, 64, 16), (8, 2, 96, 3, 9),
                                                 (8, 2, 256, 3, 16)])
def test_attention_large_equal_scores_weigh_the_same(wq, sign, heads, kv, dim, n, page):
    """One key at every position: however large (or low) its score, the result is the mean of the values seen."""
    rng = np.random.default_rng(dim + n)
    p = Attn(rng, [1100, 30], [n, n], heads, kv, dim, page)
    p.k64, p.k = bf16(np.broadcast_to(p.k64[0, 0], p.k64.shape).copy())
    q = sign * np.sign(p.k64[0, 0]).repeat(heads // kv, axis=0) * np.abs(p.q64) * 2.0 ** 36
    p.q64, p.q = bf16(q)
    run(wq, p)
    want = np.zeros_like(p.q64)
    reach = np.zeros_like(p.q64)
    for r, length in enumerate(p.lengths):
        for j in range(n):
            at = np.arange(length + j + 1)
            v = p.v64[p.table[r, at // page], at % page].repeat(heads // kv, axis=1)
            want[p.starts[r] + j], reach[p.starts[r] + j] = v.mean(0), np.abs(v).mean(0)
    got = f64(p.y)
    # equal weights round alike and cancel; sums of 1164 values in fp32
    assert np.all(np.abs(got - want) <= BF16 * np.abs(want) + 2.0 ** -12 * reach)


@pytest.mark.parametrize("rank,k,tokens", [(16, 64, 3), (32, 512, 20), (8, 4104, 5), (64, 256, 40), (128, 96, 33)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_lora_infinite_weights_of_b(wq, rank, k, tokens, out):
    """B's infinities and NaN act on A x as a whole, not on each of the parts that carry it."""
    import torch
    rng = np.random.default_rng(rank + k)
    x = rng.normal(size=(tokens, k))
    a = rng.normal(size=(2, rank, k)) / np.sqrt(k)
    x[1], a[0, 0] = 0, 0
    x[1, 0], a[0, 0, 0] = 1.0, 2.0                     # row 1: A x is exactly 2 at rank 0, whose further parts are 0
    b = rng.normal(size=(2, 70, rank))
    x64, xt = bf16(x)
    a64, at = bf16(a)
    b64, _ = bf16(b)
    b64[0, 7, 0], b64[0, 65, 3], b64[0, 30, 5], b64[0, 31, 2] = np.inf, -np.inf, np.nan, np.inf
    b64[0, 40, 1], b64[0, 40, 4] = np.inf, -np.inf
    b64[1, 7, 6] = -np.inf
    adapter = np.array([0 if t % 5 != 4 else 1 for t in range(tokens)])
    adapter[2] = 1 if tokens < 4 else -1
    y = torch.zeros(tokens, 70, device="cuda", dtype=torch.float32 if out == "f32" else torch.bfloat16)
    base = rng.normal(size=(tokens, 70)).astype(np.float32)
    wq.wq_lora_run(wq.wq_lora_prepare(xt, at, torch.from_numpy(b64).to(torch.bfloat16).cuda(), i32(adapter), y,
                                      base=torch.from_numpy(base).cuda()))
    torch.cuda.synchronize()
    got = f64(y)
    for t, c in enumerate(adapter):
        want, tol = base[t].astype(np.float64), np.zeros(70)
        if c >= 0:
            h = a64[c] @ x64[t]
            assert np.abs(h).min() > 1e-5
            with np.errstate(invalid="ignore"):
                want = want + b64[c] @ h
            fine = np.where(np.isfinite(b64[c]), b64[c], 0)
            tol = 2 * ((k + 8) * 2.0 ** -24 * (np.abs(fine) @ (np.abs(a64[c]) @ np.abs(x64[t]))) +
                       (3 * rank + 8) * 2.0 ** -24 * (np.abs(fine) @ np.abs(h)))
            if out == "bf16":
                tol = tol + 2.0 ** -16 * (np.abs(fine) @ np.abs(h))
        assert np.array_equal(np.isnan(got[t]), np.isnan(want)), t
        inf = np.isinf(want)
        assert np.array_equal(got[t][inf], want[inf]), t
        ok = np.isfinite(want)
        tol = tol + 2.0 ** -22 * np.abs(want) + (BF16 * np.abs(want) if out == "bf16" else 0)
        assert np.all(np.abs(got[t][ok] - want[ok]) <= tol[ok]), t


@pytest.mark.parametrize("power", [-62, -64, -66, 40])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (20, False)])
def test_rope_norm_of_tiny_heads_without_eps(wq, power, f32, rot, interleaved):
    """mean(x^2) below 2^-126: its fp32 squares are good to 2^-18 of the sum (128 of them, each off by 2^-150 at most)."""
    import torch
    rng = np.random.default_rng(60)
    raw = rng.normal(size=(3, 4 * 128)) * 2.0 ** power
    qkv64, qkv = bf16(raw)
    if f32:
        qkv = qkv.float()
    _, k = bf16(np.zeros((1, 16, 1, 128)))
    v, q = k.clone(), torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    w64, w = bf16(1 + 0.2 * rng.normal(size=128))
    freq = wq.wq_rope_frequencies(rot, 10000.0)[0]
    wq.wq_qkv_rope_run(wq.wq_qkv_rope_prepare(qkv, q, k, v, i32([[0]]), i32([0, 3]), i32([2]), freq.cuda(), q_norm=w, k_norm=w,
                                              eps=0.0, interleaved=interleaved))
    torch.cuda.synchronize()
    wq_, wk, _ = verify.qkv_rope(qkv64, np.zeros((1, 16, 1, 128)), np.zeros((1, 16, 1, 128)), np.array([[0]]), [0, 3], [2], 2,
                                 freq.double().numpy(), q_norm=w64, k_norm=w64, eps=0.0, interleaved=interleaved)
    for got, want in ((f64(q), wq_), (f64(k)[:, 2:5], wk[:, 2:5])):
        pair = np.abs(want).max(axis=-1, keepdims=True)
        assert np.all(np.abs(got - want) <= BF16 * np.abs(want) + 2.0 ** -16 * 1.5 * pair)


@pytest.mark.parametrize("rank", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", [17, 32, 33, 100])
@pytest.mark.parametrize("out", [("bf16",), ("f32",)])
def test_lora_tiles_with_a_filled_second_half(wq, rank, rows, out):
    # more than 16 rows of one adapter, several shares of k, outputs that end inside a wave's 64
    rng = np.random.default_rng(rank * rows)
    adapter = rng.permutation([1] * rows + [0, 0, 2, -1, 3])
    lora_case(wq, rng, adapter, 3, rank, 2056, 133, out=out)
    lora_case(wq, rng, adapter, 3, rank, 1040, 333, out=out, ranks=[rank, rank - 3, 5], pad=3)


@pytest.mark.parametrize("rank,k", [(8, 512), (16, 1024), (32, 1024)])
@pytest.mark.parametrize("out", [("bf16",), ("f32",)])
def test_lora_tiles_with_a_filled_second_half_in_one_launch(wq, rank, k, out):
    rng = np.random.default_rng(rank * k)
    for rows in (17, 31, 32):
        lora_case(wq, rng, rng.permutation([1] * rows + [0] * (32 - rows)), 2, rank, k, 650, out=out, ranks=[rank, rank - 1])


@pytest.mark.parametrize("scale,power", [(0.0, 118), (2.0 ** -125, 118), (-(2.0 ** -125), 118), (2.0 ** -140, 118), (2.0 ** -110, 104)])
@pytest.mark.parametrize("heads,n", [(4, 2), (16, 30), (64, 64)])
def test_attention_scales_next_to_nothing(wq, scale, power, heads, n):
    # queries and keys are small integers times 2^power: scores up to 2^125 are exact, scaled ones about 1 or none
    rng = np.random.default_rng(n)
    p = Attn(rng, [900, 3], [n, n], heads, 2, 64, 16, scale=scale, tree=lambda m: random_tree(rng, m))
    p.k64, p.k = bf16(np.rint(p.k64))
    p.q64, p.q = bf16(np.rint(p.q64) * 2.0 ** power)
    run(wq, p)
    p.check()


def test_attention_plans_of_one_stream_share_a_workspace(wq):
    """As the layers of a model do: runs that follow each other, eager and in one captured graph."""
    import torch
    rng = np.random.default_rng(106)
    ps = [Attn(rng, [3000, 20], [5, 8], 8, 2, 128, 16), Attn(rng, [40, 2500], [8, 3], 8, 2, 128, 16)]
    ws = torch.empty(wq.wq_tree_attention_workspace_bytes(2, 8, 2, 128, 8), dtype=torch.uint8, device="cuda")
    plans = [p.plan(wq, max_tokens=8, workspace=ws) for p in ps]
    for plan in plans:
        wq.wq_tree_attention_run(plan)
    torch.cuda.synchronize()
    for p in ps:
        p.check()
    first = [p.y.clone() for p in ps]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for plan in plans:
            wq.wq_tree_attention_run(plan)
    for _ in range(3):
        for p in ps:
            p.y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.y, y) for p, y in zip(ps, first))
        torch.randn(1000, device="cuda").sum().item()


def test_accept_captured_follows_its_buffers(wq):
    import torch
    rng = np.random.default_rng(107)
    k0 = torch.from_numpy(rng.integers(-30000, 30000, (3, 20, 8, 2, 64)).astype(np.int16)).cuda()
    k, v = k0.clone(), torch.flip(k0, [1]).contiguous()
    v0 = v.clone()
    table = rng.permutation(20).astype(np.int32).reshape(2, 10)
    lengths, path, accepted = i32([3, 17]), i32([[0, 2, 5], [1, 3, 4]]), i32([3, 3])
    plan = wq.wq_kv_accept_prepare(k, v, i32(table), lengths, path, accepted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_kv_accept_run(plan)
    for l, p, n in (([3, 17], [[0, 2, 5], [1, 3, 4]], [3, 3]), ([0, 40], [[1, 2, 3], [0, 1, 7]], [2, 3]), ([9, 1], [[0, 4, 3], [2, 9, 30]], [3, 1])):
        lengths.copy_(i32(l)), path.copy_(i32(p)), accepted.copy_(i32(n))
        k.copy_(k0), v.copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        wk, wv = verify.kv_accept(k0.cpu().numpy(), v0.cpu().numpy(), table, l, np.array(p), n)
        assert np.array_equal(k.cpu().numpy(), wk) and np.array_equal(v.cpu().numpy(), wv)
