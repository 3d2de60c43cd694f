"""GPU: the decoder-layer operators at the edges of their arguments' ranges, against
the oracle."""
import numpy as np
import pytest

import oracle as O
from tests._helpers import say
from tests.test_gpu_layer import check_norm, dev, g, host  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


# one wave, four, eight and sixteen a row, rows read twice
WIDTHS = [8, 1000, 4096, 8192, 12288, 16384, 20000]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_norm_zero_rows_without_eps(g, dt, kind):  # noqa: F811
    """eps = 0: a row of zeros gets scale 0 and codes 0, its neighbours what they get alone."""
    rng = np.random.default_rng(1)
    for K in WIDTHS:
        x = rng.standard_normal((6, K)).astype(dt)
        w = (1 + 0.2 * rng.standard_normal(K)).astype(dt)
        x[1] = x[4] = 0
        r = -x
        r[[0, 2, 3, 5]] = 0
        r[1] = x[1]
        for res in (None, r):
            codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(
                dev(x), dev(w), None if res is None else dev(res), eps=0.0, q_dtype=kind))
            say("zero rows", K, dt.__name__, kind, scale[[1, 4]])
            assert not scale[[1, 4]].any() and not codes[[1, 4]].any()
            live = [0, 2, 3, 5]
            check_norm(codes[live], scale[live], x[live], w, None if res is None else res[live], 0.0,
                       kind, (K, dt, kind))
        # zeros after the weights: the same, whatever the root
        z = host(g.add_rmsnorm_q8(dev(x), dev(np.zeros(K, dt)), eps=0.0, q_dtype=kind)[1])
        assert not z.any()


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_float32_rows_of_any_magnitude(g, kind):  # noqa: F811
    """Rows whose squares leave float32 on either side, beside ordinary ones."""
    rng = np.random.default_rng(2)
    # magnitude of a row; with normal values and weights below 2, products stay finite and normal
    mags = np.array([1, 1e-34, 1e-28, 1e-22, 1e-19, 1e-15, 1e-7, 1e15, 1e18, 1e19, 1e20, 1e28, 1e36])
    for K in WIDTHS:
        base = rng.standard_normal((len(mags), K))
        base[:, 0] = 1
        x = (np.clip(base, -5, 5) * mags[:, None]).astype(np.float32)
        w = (1 + 0.2 * np.clip(rng.standard_normal(K), -4, 4)).astype(np.float32)
        r = (0.5 * x[:, ::-1]).copy()
        for eps in (0.0, 1e-44, 1e-36, 1e-5, 1e30):
            for res in (None, r):
                say("magnitudes", K, eps, kind, res is not None)
                codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(
                    dev(x), dev(w), None if res is None else dev(res), eps=eps, q_dtype=kind))
                assert np.isfinite(scale).all()
                check_norm(codes, scale, x, w, res, eps, kind, (K, eps, kind))


def test_norm_float32_row_at_the_largest_values(g):  # noqa: F811
    """Weights that bring the largest rows down and the smallest up."""
    rng = np.random.default_rng(3)
    for K in WIDTHS:
        s = np.sign(rng.standard_normal((1, K)))
        for h, w, eps in ((3e38, 1e-6, 0.0), (3e38, 1e-30, 1e-5), (1e-37, 100.0, 0.0), (1e-30, 1e20, 0.0)):
            x = (h * s).astype(np.float32)
            W = np.full(K, w, np.float32)
            codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(dev(x), dev(W), eps=eps))
            check_norm(codes, scale, x, W, None, eps, 0, (K, h, w, eps))
