"""Oracle of the MXFP4 operators: coding, values, products, mixture of experts.

Codes and scales follow from the inputs alone (a division by a power of two is
exact), so they are compared bit for bit; everything else is float64.
"""
from __future__ import annotations

import numpy as np

__all__ = ["mx4_encode", "mx4_decode", "mx4_pack", "mx4_unpack", "moe_route", "moe_activation",
           "moe_layer"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_pack(q):
    """Codes 0..15 [R, K] -> bytes [R, K/2], the even element in the low half."""
    return (q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8)


def mx4_unpack(b):
    q = np.empty((b.shape[0], 2 * b.shape[1]), np.uint8)
    q[:, 0::2], q[:, 1::2] = b & 15, b >> 4
    return q


def mx4_encode(x):
    """float rows [R, K] -> (bytes [R, K/2], scale bytes [R, K/32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    with np.errstate(all="ignore"):
        most = np.abs(b).max(axis=2)
        bad = ~np.isfinite(b).all(axis=2)
        live = (most > 0) & ~bad
        e = np.where(live, np.frexp(np.where(live, most, 1.0))[1] - 1 - 2, -127)
        e = np.maximum(e, -127)
        y = np.where(bad[..., None], 0.0, b) / np.exp2(e.astype(np.float64))[..., None]
        a = np.abs(y)
    # the nearest value; of two equally near ones the even code
    d = np.abs(a[..., None] - E2M1)
    near = d == d.min(axis=-1, keepdims=True)
    odd = np.arange(8) % 2
    code = np.argmin(np.where(near, odd, 9), axis=-1).astype(np.uint8)
    code = np.where(a > 6, 7, code) + 8 * np.signbit(y).astype(np.uint8)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return mx4_pack(code.reshape(x.shape)), scale


def mx4_decode(codes, scales):
    """float64 values [R, K]."""
    q = mx4_unpack(codes)
    v = np.where(q & 8, -1.0, 1.0) * E2M1[q & 7]
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return v * np.repeat(s, 32, axis=1)


def moe_route(logits, top, renorm):
    """(experts [T, top], -1 for none; weights float64 [T, top], NaN in the rows
    that hold a NaN or +infinity)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids, w = np.full((T, top), -1), np.zeros((T, top))
    for t in range(T):
        if np.isnan(l[t]).any() or np.isposinf(l[t]).any():
            w[t] = np.nan
            continue
        order = sorted(range(E), key=lambda e: (-l[t, e], e))[:top]
        order = [e for e in order if not np.isneginf(l[t, e])]
        if not order:
            continue
        p = np.exp(l[t] - l[t, order[0]])
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[order] / (p[order].sum() if renorm else p.sum())
    return ids, w


def moe_activation(g, act):
    with np.errstate(over="ignore"):
        if act == 2:
            return np.maximum(g, 0.0) ** 2
        z = g if act == 0 else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
        return g / (1 + np.exp(-z))


def moe_layer(x, logits, top, w1, w2, act, renorm):
    """x [T, H]; w1 [E, 2 I, H] (gate rows, then up rows), w2 [E, H, I], float64 ->
    (out [T, H], and a bound's pieces: see the test that uses them)."""
    T, H = x.shape
    E, I = w2.shape[0], w2.shape[2]
    x = x.astype(np.float64)
    ids, w = moe_route(logits, top, renorm)
    out, err = np.zeros((T, H)), np.zeros((T, H))
    U = 2.0 ** -23
    for t in range(T):
        if np.isnan(w[t]).any():
            out[t] = np.nan
            continue
        for e, p in zip(ids[t], w[t]):
            if e < 0:
                continue
            g, u = w1[e, :I] @ x[t], w1[e, I:] @ x[t]
            # float32 sums of H terms, 16 or more to an addition
            n = (H / 16 + 16) * U
            dg, du = n * (np.abs(w1[e, :I]) @ np.abs(x[t])), n * (np.abs(w1[e, I:]) @ np.abs(x[t]))
            f = moe_activation(g, act)
            h = f * u
            # |act'| is at most 1.13 (silu, gelu), 2 g + its step (relu2); the activation's own
            # arithmetic: a few roundings, and the exponent's error through exp
            slope = 1.13 if act != 2 else 2 * (np.abs(g) + dg)
            z = np.abs(g) if act == 0 else 0 * g if act == 2 else 1.6 * (np.abs(g) + 0.045 * np.abs(g) ** 3)
            own = (16 + 4 * np.minimum(z, 100.0)) * U * np.abs(f)
            dh = np.abs(u) * (slope * dg + own) + np.abs(f) * du + dg * slope * du + 4 * U * np.abs(h)
            # two bfloat16 numbers: the first leaves at most half a step of 8 bits, 2^(e - 8) for h of
            # [2^e, 2^(e+1)), and of that the second at most half a step, 2^(e - 17)
            dh = dh + 2.0 ** -17 * np.abs(h)
            a = np.abs(w2[e])
            out[t] += p * (w2[e] @ h)
            err[t] += p * (a @ dh + (I / 16 + 64) * U * (a @ np.abs(h)))
    return out, err
