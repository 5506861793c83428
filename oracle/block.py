"""An expert block with microscaled 4-bit weights, in fp64 from the definitions.

Values are float64 arrays (bf16 and fp32 inputs decoded by the caller).  Nothing
is rounded here but what is a 4-bit code by definition, so a test adds the
roundings that the library documents.
"""

import numpy as np

GROUP = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_scale_byte(largest):
    """Scale byte of a group whose largest magnitude this is."""
    if not np.isfinite(largest):
        return 255
    if largest == 0:
        return 0
    mantissa, exponent = np.frexp(largest)      # largest = mantissa * 2^exponent, mantissa in [0.5, 1)
    return int(max(exponent - 1 - 2, -127) + 127)


def mx_quantize(w):
    """[n, k] float64 -> codes u8 [n, k / 2] (even input low) and scale bytes u8 [n, k / 32]."""
    n, k = w.shape
    codes = np.zeros((n, k), np.uint8)
    scale = np.zeros((n, k // GROUP), np.uint8)
    for r in range(n):
        for g in range(k // GROUP):
            v = w[r, g * GROUP:(g + 1) * GROUP]
            scale[r, g] = mx_scale_byte(np.max(np.abs(v)) if np.all(np.isfinite(v)) else np.inf)
            if scale[r, g] == 255:
                continue
            size = np.abs(v) / 2.0 ** (int(scale[r, g]) - 127)          # exact
            # nearest of the eight sizes, of two equally near the even code
            off = np.abs(size[:, None] - VALUES)
            best = np.argmin(off, axis=1)
            tie = (best < 7) & (off[np.arange(GROUP), best] == off[np.arange(GROUP), np.minimum(best + 1, 7)])
            best = best + (tie & (best % 2 == 1))
            codes[r, g * GROUP:(g + 1) * GROUP] = best + 8 * np.signbit(v)
    return codes[:, 0::2] | codes[:, 1::2] << 4, scale


def mx_values(q, scale):
    """What codes stand for, float64 [..., k]."""
    code = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    size = VALUES[code & 7] * np.where(code >= 8, -1.0, 1.0)
    power = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return size * np.repeat(power, GROUP, axis=-1)


def silu(v):
    return v / (1 + np.exp(-v))


def route(logits, top, renormalize=True):
    """Selected experts (largest first, ties to the lower index) and gates of one token."""
    order = sorted(range(len(logits)), key=lambda e: (-logits[e], e))[:top]
    weight = np.exp(logits - np.max(logits))
    total = weight[order].sum() if renormalize else weight.sum()
    return order, weight[order] / total


def moe_ffn(x, logits, w13, w2, top, renormalize=True):
    """x [tokens, dim]; logits [tokens, e]; w13 [e, 2f, dim], w2 [e, dim, f] as values -> y, sel, gates."""
    f = w2.shape[2]
    y, sel, gates = np.zeros(x.shape), [], []
    for t in range(x.shape[0]):
        order, g = route(logits[t], top, renormalize)
        sel.append(order)
        gates.append(g)
        for e, share in zip(order, g):
            h = w13[e] @ x[t]
            y[t] += share * (w2[e] @ (silu(h[:f]) * h[f:]))
    return y, np.array(sel, np.int32), np.array(gates)


def block_norm(h, f=None, f_norm=None, gate=None, gate_kind="plain", scale=1.0, norm=None, eps=1e-6):
    """h + scale * act(gate) * norm(f), and its norm."""
    def rms(v, weight):
        return v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps) * weight
    if f is not None:
        if f_norm is not None:
            f = rms(f, f_norm)
        if gate is not None:
            turned = 1 / (1 + np.exp(-gate))
            f = f * {"plain": gate, "sigmoid": turned, "silu": gate * turned}[gate_kind]
        h = h + scale * f
    return h, rms(h, 1.0 if norm is None else norm)
