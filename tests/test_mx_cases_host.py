"""Host-only: the exact inputs of the MXFP4 tests tell h kept as two bfloat16 numbers from one."""
import numpy as np
import pytest

from tests._mx_cases import LAYERS, ExactLayer, bf16, dropped


@pytest.mark.parametrize("case", LAYERS)
def test_half_of_h_would_show(case):
    m = ExactLayer(np.random.default_rng(case[0] + case[1]), *case)
    assert np.isfinite(m.want).all()
    wrong = m.of_hi_alone() != m.want
    assert wrong.mean(1).min() > 0.05


def test_rounding_to_bfloat16():
    x = np.array([0.0, 1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -8 - 2.0 ** -20, 255.5])
    assert bf16(x).tolist() == [0.0, 1.0, 1.0, 1 + 2.0 ** -6, -1 - 2.0 ** -7, 256.0]


def test_dropped_bits():
    a = np.zeros((1, 16))
    a[0, :3], a[0, 8:10] = [256, 2.0 ** -5, 2.0 ** -6], [2.0 ** -6, 3 * 2.0 ** -20]
    assert dropped(a, np.ones((2, 16))).tolist() == [[2.0 ** -6 + 2.0 ** -20] * 2]
