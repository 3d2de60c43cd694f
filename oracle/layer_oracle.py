"""Oracle of the operators between a decoder layer's products: residual norm to
8-bit rows, append to the paged 8-bit cache, attention over it.

Norm and attention are float64 throughout. The cache's codes and scales are
decided in float32, operation by operation in the order of their definition
(products and sums each rounded), so they are compared bit for bit.
"""
from __future__ import annotations

import numpy as np

from .w4_oracle import e4m3_decode, e4m3_encode

__all__ = ["rmsnorm_rows", "rope_f32", "code_scale", "encode_q8", "decode_q8", "PagedCache8",
           "attention_rows"]

f32 = np.float32


def rmsnorm_rows(x, w, residual, eps):
    """float64 (h, y): the residual sum and the normalised rows before coding."""
    h = x.astype(np.float64)
    if residual is not None:
        h = h + residual.astype(np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + float(f32(eps))) * w.astype(np.float64)
    return h, y


def rope_f32(x, table, pos, rot, style):
    """float32 rotation of x [T, H, D] at positions pos [T]; table [rows, rot]."""
    y = x.astype(f32).copy()
    if rot == 0:
        return y
    half = rot // 2
    c, s = table[pos, None, :half], table[pos, None, half:]
    ia, ib = ((slice(0, half), slice(half, rot)) if style == 0
              else (slice(0, rot, 2), slice(1, rot, 2)))
    a, b = x[..., ia].astype(f32), x[..., ib].astype(f32)
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def code_scale(m, kind):
    """float32 scale of a largest magnitude m (kind 0 INT8, 1 E4M3)."""
    m = f32(m)
    if not np.isfinite(m):
        return f32(np.nan)
    if m == 0:
        return f32(0)
    if kind == 0:
        return m / f32(127)
    f = m / f32(448)
    mant, e = np.frexp(f)
    s = np.ldexp(f32(1), int(e) - (1 if mant == 0.5 else 0)) if f > 0 else f32(0)
    return f32(max(s, f32(2.0 ** -126)))


def encode_q8(x, s, kind):
    """uint8 bit patterns of float32 x divided by the float32 scale s."""
    if not s > 0:
        return np.zeros(x.shape, np.uint8)
    y = (x.astype(f32) / f32(s)).astype(f32)
    if kind == 0:
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    return e4m3_encode(np.clip(y, f32(-448), f32(448)))


def decode_q8(b, kind):
    """float32 values of codes in units of the scale."""
    return (b.view(np.int8).astype(f32) if kind == 0 else e4m3_decode(b).astype(f32))


class PagedCache8:
    """The cache as token rows: codes [pages, heads, slot, DP] for keys and values."""

    def __init__(self, pages, page, heads, dim, dp, kind):
        self.page, self.dim, self.kind = page, dim, kind
        self.codes = [np.zeros((pages, heads, page, dp), np.uint8) for _ in range(2)]
        self.scale = [np.zeros((pages, heads), f32) for _ in range(2)]

    def append(self, rows, table, start):
        """rows: float32 (keys, values) [n, heads, dim] of one sequence whose first
        new position is start."""
        n = rows[0].shape[0]
        for which in range(2):
            codes, scale = self.codes[which], self.scale[which]
            for j in range(start // self.page, (start + n - 1) // self.page + 1):
                lo, hi = max(start, j * self.page), min(start + n, (j + 1) * self.page)
                lead, pid = lo - j * self.page, int(table[j])
                if not 0 <= pid < codes.shape[0]:
                    continue
                for h in range(codes.shape[1]):
                    new = rows[which][lo - start:hi - start, h]
                    mag = np.abs(new).max()
                    s = code_scale(mag, self.kind)
                    if lead:
                        old = scale[pid, h]
                        if np.isnan(old) or np.isnan(s):
                            s = f32(np.nan)
                        else:
                            s = max(s, old)
                            if old < s:
                                v = decode_q8(codes[pid, h, :lead], self.kind) * (old / s)
                                codes[pid, h, :lead] = (
                                    np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
                                    if self.kind == 0 else e4m3_encode(v.astype(f32)))
                    else:
                        codes[pid, h] = 0
                    codes[pid, h, lead:lead + hi - lo] = 0
                    codes[pid, h, lead:lead + hi - lo, :self.dim] = encode_q8(new, s, self.kind)
                    scale[pid, h] = s

    def rows(self, which, table, length, h):
        """float64 rows [length, dim] of one sequence and head."""
        ids = np.asarray(table[:-(-length // self.page)] if length else [], np.int64)
        c = decode_q8(self.codes[which][ids, h], self.kind).astype(np.float64)
        c = c * self.scale[which][ids, h].astype(np.float64)[:, None, None]
        return c.reshape(-1, c.shape[-1])[:length, :self.dim] if length else np.zeros((0, self.dim))


def attention_rows(q, k, v, limits, scale):
    """float64 (out, lse, sum_j w_j |v_j|, max |score terms|) of query rows q [R, D]
    over k, v [L, D]; row r sees the first limits[r] tokens."""
    R, D = q.shape
    out, lse = np.zeros((R, D)), np.full(R, -np.inf)
    absv, terms = np.zeros((R, D)), np.zeros(R)
    for r in range(R):
        n = max(0, int(limits[r]))
        if n == 0:
            continue
        s = scale * (k[:n] @ q[r].astype(np.float64))
        m = s.max()
        w = np.exp(s - m)
        lse[r] = m + np.log(w.sum())
        w = w / w.sum()
        out[r] = w @ v[:n]
        absv[r] = w @ np.abs(v[:n])
        terms[r] = abs(scale) * (np.abs(k[:n]) @ np.abs(q[r].astype(np.float64))).max()
    return out, lse, absv, terms
