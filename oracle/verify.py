"""What stands between the linears of a verify pass, in fp64 from the definitions.

Values are float64 arrays (bf16 inputs decoded by the caller); nothing is
rounded here, so a test adds the roundings that the library documents.  Plain
loops over requests, rows and heads.
"""

import numpy as np


def rope_frequencies(kind, rot_dim, base, factor=1.0, low=1.0, high=4.0, original=8192.0):
    """Radians per position of each rotated pair, and the scale of cos and sin."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        turns = original * f / (2 * np.pi)          # turns within the original length
        if kind == "linear":
            f = f / factor
        elif kind == "bands":
            if turns < low:
                f = f / factor
            elif turns <= high:
                t = (turns - low) / (high - low)
                f = f * ((1 - t) / factor + t)
        elif kind == "ramp":
            def pair(n):
                return rot_dim * np.log(original / (2 * np.pi * n)) / (2 * np.log(base))
            a = min(max(np.floor(pair(high)), 0), rot_dim - 1)
            b = min(max(np.ceil(pair(low)), 0), rot_dim - 1)
            t = 0.0 if i <= a else 1.0 if i >= b else (i - a) / (b - a)
            f = f * (1 - t) + f / factor * t
        out.append(f)
    return np.array(out), (0.1 * np.log(factor) + 1.0 if kind == "ramp" else 1.0)


def norm_rope_head(x, position, freq, rot_scale=1.0, weight=None, eps=1e-6, interleaved=False):
    """One head [dim] of one token."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * weight
    out = x.copy()
    half = len(freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = float(position) * float(freq[i])
        out[a] = rot_scale * (x[a] * np.cos(t) - x[b] * np.sin(t))
        out[b] = rot_scale * (x[b] * np.cos(t) + x[a] * np.sin(t))
    return out


def cache_row(table, page_size, pages, request, position):
    """(page, row) of a position, or None if it holds nothing."""
    if position < 0 or position >= table.shape[1] * page_size:
        return None
    page = int(table[request, position // page_size])
    return (page, position % page_size) if 0 <= page < pages else None


def requests_of(starts, lengths, tokens):
    """(request, first row, rows, context length) of each request in order and range."""
    for r in range(len(lengths)):
        a, b = int(starts[r]), int(starts[r + 1])
        if 0 <= a <= b <= tokens:
            yield r, a, b - a, max(int(lengths[r]), 0)


def qkv_rope(qkv, k, v, table, starts, lengths, heads, freq, positions=None, q_norm=None, k_norm=None, eps=1e-6,
             rot_scale=1.0, interleaved=False):
    """qkv [tokens, (heads + 2 kv) * dim]; returns (q [tokens, heads, dim] with NaN in rows of no request, k, v)."""
    pages, page_size, kv, dim = k.shape
    k, v = k.astype(np.float64).copy(), v.astype(np.float64).copy()
    rows = np.asarray(qkv, np.float64).reshape(len(qkv), heads + 2 * kv, dim)
    q = np.full((len(qkv), heads, dim), np.nan)
    for r, a, n, length in requests_of(starts, lengths, len(qkv)):
        for j in range(n):
            t = a + j
            pos = length + j if positions is None else int(positions[t])
            turn = dict(position=pos, freq=freq, rot_scale=rot_scale, eps=eps, interleaved=interleaved)
            for h in range(heads):
                q[t, h] = norm_rope_head(rows[t, h], weight=q_norm, **turn)
            at = cache_row(table, page_size, pages, r, length + j)
            if at is not None:
                for h in range(kv):
                    k[at[0], at[1], h] = norm_rope_head(rows[t, heads + h], weight=k_norm, **turn)
                    v[at[0], at[1], h] = rows[t, heads + kv + h]
    return q, k, v


def tree_attention(q, k, v, table, starts, lengths, scale, tree=None, max_tokens=64):
    """q [tokens, heads, dim]; returns (y, weight) with y NaN in rows that are left alone and weight the sums of
    w |v| (how much a relative error of the weights can move y)."""
    pages, page_size, kv, dim = k.shape
    tokens, heads, _ = q.shape
    y = np.full((tokens, heads, dim), np.nan)
    reach = np.zeros((tokens, heads, dim))
    for r, a, n, length in requests_of(starts, lengths, tokens):
        if n > max_tokens:
            continue
        length = min(length, table.shape[1] * page_size)
        at = [cache_row(table, page_size, pages, r, p) for p in range(length + n)]
        for i in range(n):
            bits = (2 << i) - 1 if tree is None else int(tree[a + i])
            seen = [x for p, x in enumerate(at) if x is not None and (p < length or bits >> (p - length) & 1)]
            if not seen:
                y[a + i] = 0.0
                continue
            pg, row = np.array(seen).T
            for h in range(heads):
                keys, values = k[pg, row, h * kv // heads], v[pg, row, h * kv // heads]
                s = scale * (keys @ q[a + i, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                y[a + i, h] = w @ values
                reach[a + i, h] = w @ np.abs(values)
    return y, reach


def kv_accept(k, v, table, lengths, path, accepted):
    """k, v [layers, pages, page_size, ...], any dtype; returns the moved copies."""
    pages, page_size = k.shape[1:3]
    k0, v0, k, v = k, v, k.copy(), v.copy()
    for r, length in enumerate(lengths):
        length = max(int(length), 0)
        steps = [int(p) for p in path[r][:min(max(int(accepted[r]), 0), path.shape[1])]]
        if any(b <= a for a, b in zip([-1] + steps, steps)):
            continue
        for i, p in enumerate(steps):
            src = cache_row(table, page_size, pages, r, length + p)
            dst = cache_row(table, page_size, pages, r, length + i)
            if src is not None and dst is not None:
                k[:, dst[0], dst[1]] = k0[:, src[0], src[1]]
                v[:, dst[0], dst[1]] = v0[:, src[0], src[1]]
    return k, v


def lora(x, a, b, adapter, base=None, ranks=None, scale=None):
    """Returns (y, sums of the magnitudes of h's terms carried through B, of B h's terms)."""
    tokens, n = len(x), b.shape[1]
    y = np.zeros((tokens, n)) if base is None else np.asarray(base, np.float64).copy()
    deep, flat = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        c = int(adapter[t])
        if not 0 <= c < len(a):
            continue
        rank = a.shape[1] if ranks is None else min(max(int(ranks[c]), 0), a.shape[1])
        s = 1.0 if scale is None else float(scale[c])
        low, high = a[c, :rank].astype(np.float64), b[c, :, :rank].astype(np.float64)
        h = low @ x[t]
        y[t] += s * (high @ h)
        deep[t] = abs(s) * (np.abs(high) @ (np.abs(low) @ np.abs(x[t])))
        flat[t] = abs(s) * (np.abs(high) @ np.abs(h))
    return y, deep, flat
