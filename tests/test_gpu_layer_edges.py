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
