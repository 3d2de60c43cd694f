"""Inputs of the MXFP4 operators whose products and sums are exact in float32 (and in the two
bfloat16 numbers that the expert layer keeps of h), so that a result has to be the definition's
rounded once: a bit lost, or an element left out or met twice, shows."""
import numpy as np

import oracle as O

# what ratio of the sum of magnitudes to the terms' unit a float32 sum holds in any order
EXACT = 2.0 ** 24


def exact_weights(rng, N, K, two=False):
    """Random codes, scales 1 (or 1 and 2): (codes, scales, values); the values' unit is 1/2."""
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (127 + (rng.integers(0, 2, (N, K // 32)) if two else np.zeros((N, K // 32), int))).astype(np.uint8)
    return codes, scales, O.mx4_decode(codes, scales)


class ExactLayer:
    """An expert layer with relu^2 whose gates are -1, 1 or 2 (one code that meets x[:, 0] = 1), `top`
    (a power of two) choices of equal weight and x of whole numbers up to `most`. `up` and `down` are
    powers of two that the up rows and the second product's weights carry."""

    def __init__(self, rng, T, H, I, E, top, most, up=0, down=-6):
        self.H, self.I, self.E, self.top, self.T = H, I, E, top, T
        gate = np.zeros((E, I, H // 2), np.uint8)
        gate[:, :, 0] = rng.choice(np.array([2, 10, 4], np.uint8), (E, I), p=[0.4, 0.2, 0.4])
        c, s, v = exact_weights(rng, E * I, H)
        self.c1 = np.concatenate([gate, c.reshape(E, I, -1)], 1).reshape(E * 2 * I, -1)
        self.s1 = np.concatenate([np.full((E, I, H // 32), 127), s.reshape(E, I, -1).astype(int) + up], 1).astype(np.uint8)
        self.s1 = self.s1.reshape(E * 2 * I, -1)
        self.c2, s2, v2 = exact_weights(rng, E * H, I)
        self.s2 = (s2.astype(int) + down).astype(np.uint8)
        self.x = rng.integers(-most, most + 1, (T, H)).astype(np.float16)
        self.x[:, 0] = 1
        self.chosen = np.stack([rng.permutation(E)[:top] for _ in range(T)])
        self.logits = rng.uniform(-9, -2, (T, E)).astype(np.float32)
        np.put_along_axis(self.logits, self.chosen, np.float32(0.5), 1)
        g = O.mx4_decode(gate.reshape(E * I, -1), np.full((E * I, H // 32), 127, np.uint8)).reshape(E, I, H)
        v, v2 = v.reshape(E, I, H), v2.reshape(E, H, I)
        self.h = np.zeros((T, top, I))                   # of 2^up / top
        self.out = np.zeros((T, H))
        size = np.zeros((T, H))
        x = self.x.astype(np.float64)
        for t in range(T):
            for j, e in enumerate(self.chosen[t]):
                u = v[e] @ x[t]
                assert (np.abs(v[e]) @ np.abs(x[t])).max() / 0.5 < EXACT
                self.h[t, j] = np.maximum(g[e] @ x[t], 0) ** 2 * u
                self.out[t] += v2[e] @ self.h[t, j]
                size[t] += np.abs(v2[e]) @ np.abs(self.h[t, j])
        assert size.max() / 0.25 < EXACT
        hi = bf16(self.h)
        assert np.array_equal(hi + bf16(self.h - hi), self.h)      # h is those two numbers
        self.v2 = v2
        self.factor = 2.0 ** (up + down) / top
        with np.errstate(over="ignore"):
            self.want = (self.out * self.factor).astype(np.float16)

    def of_hi_alone(self):
        """What the layer would give if h were one bfloat16 number."""
        out = np.zeros((self.T, self.H))
        for t in range(self.T):
            for j, e in enumerate(self.chosen[t]):
                out[t] += self.v2[e] @ bf16(self.h[t, j])
        return (out * self.factor).astype(np.float16)


def bf16(x):
    """Nearest bfloat16, ties to even (no subnormals)."""
    f, e = np.frexp(x)
    return np.ldexp(np.round(f * 256) / 256, e)


def dropped(a, w):
    """What the products of each run of eight along k may lose where the bits of a term below 2^-13
    of the largest one's power of two are dropped: float64 [M, N], for a [M, K], w [N, K]."""
    out = np.zeros((a.shape[0], w.shape[0]))
    for m in range(a.shape[0]):
        t = np.abs(a[m] * w).reshape(w.shape[0], -1, 8)
        unit = np.exp2(np.frexp(t.max(2))[1] - 1.0 - 13)
        out[m] = np.mod(t, unit[..., None]).sum((1, 2))
    return out


# (T, H, I, E, top, most): every way that the layer takes. One token and its choices among up to 64,
# 128 and 512 experts, pairs of strips a block, choices in a kernel of their own (hidden 16416),
# tokens as columns, rows of h, h in groups, two column operands.
LAYERS = [(1, 96, 160, 9, 4, 12), (1, 2048, 96, 60, 4, 3), (1, 2080, 160, 70, 2, 3), (1, 2048, 32, 140, 8, 3),
          (1, 64, 1056, 17, 16, 3), (1, 96, 1056, 100, 16, 2), (1, 64, 1056, 200, 16, 3), (1, 16416, 32, 3, 1, 1),
          (2, 2048, 96, 5, 4, 3), (7, 2144, 160, 100, 2, 3), (16, 2048, 32, 5, 4, 3), (16, 96, 160, 4, 1, 12),
          (17, 2048, 96, 9, 2, 3), (33, 96, 160, 4, 4, 12), (64, 160, 96, 3, 2, 9), (64, 64, 288, 70, 4, 12),
          (61, 320, 224, 16, 2, 6)]
