"""GPU: NaN and infinity through the MXFP4 products and the mixture-of-experts layer:
each of them reaches what meets it, whatever the activation, the number of rows and the
result's type, and nothing else."""
import numpy as np
import pytest

import oracle as O
from tests.test_gpu_mx import Layer, check_product, dev, g, host, product, rows, tokens, weights  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("H", [96, 2048])
def test_moe_nan_in_one_matrix_of_an_expert(g, T, H, act):  # noqa: F811
    """A block of NaN in a gate row, an up row or a row of the second product: the first two reach
    every output of the expert's tokens, the last one column of them."""
    rng = np.random.default_rng(10 * T + act)
    I, E = 64, 4
    for row, second in ((5, False), (I + 9, False), (7, True)):
        m = Layer(g, rng, H, I, E)
        if second:
            m.s2[H * 1 + row, 1] = 255
        else:
            m.s1[2 * I * 1 + row, 1] = 255
        m.pack(g)
        x, logits = tokens(rng, T, H, E)
        logits[:, 1] = -9
        logits[0, 1] = 9
        y = host(m.check(g, x, logits, 2, act, what=f"row {row} second {second}"))
        want = np.zeros((T, H), bool)
        want[0, row if second else slice(None)] = True
        assert np.array_equal(np.isnan(y), want)


def spoil(x, rng):
    """NaN and both infinities in three rows of x; returns the rows."""
    at = rng.choice(x.shape[0], 3, replace=False)
    for r, v in zip(at, (np.nan, np.inf, -np.inf)):
        x[r, rng.integers(x.shape[1])] = v
    return at


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M", [4, 40, 64, 90, 300])
def test_products_of_weights_coded_from_nan(g, act, M):  # noqa: F811
    """Weights and 4-bit rows as quantize_mx4 codes them: a block that is NaN has codes of zero."""
    rng = np.random.default_rng(M)
    N, K = 70, 416
    w = rng.standard_normal((N, K)).astype(np.float32)
    bad = spoil(w, rng)
    t, a = rows(rng, act, M, K)
    lost = []
    if act == "a4":
        x = a.astype(np.float32)
        lost = spoil(x, rng)
        t = g.quantize_mx4(dev(x))
    Wp = g.prepack_mx4(*g.quantize_mx4(dev(w)))
    want = np.zeros((M, N), bool)
    want[:, bad] = want[lost] = True
    clean, kept = np.delete(np.arange(N), bad), np.delete(np.arange(M), lost)
    wv = O.mx4_decode(*O.mx4_encode(w))
    for half in (True, False):
        got = host(product(g, act)(*t, Wp, N, out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32, workspace=g.Workspace()))
        assert np.array_equal(np.isnan(got), want), (act, M, half)
        some, ref = got[np.ix_(kept, clean)].astype(np.float64), a[kept] @ wv[clean].T
        if half:                                         # past fp16: infinite, or its largest number
            over = np.abs(ref) > 65504
            assert (some * np.sign(ref) >= 65504)[over].all()
            some[over] = ref[over]
        check_product(some, a[kept], wv[clean], None, half, f"{act} {M} half {half}")


@pytest.mark.parametrize("M", [5, 64, 90, 300])
@pytest.mark.parametrize("half", [True, False])
def test_nan_of_8_bit_rows(g, M, half):  # noqa: F811
    rng = np.random.default_rng(M)
    N, K = 50, 416
    codes, scales = weights(rng, N, K)
    t, a = rows(rng, "a8", M, K)
    t[0][2, 7], t[0][3, K - 1], t[1][4] = 0x7F, 0xFF, float("nan")
    got = host(g.mx4a8_gemm(*t, g.prepack_mx4(dev(codes), dev(scales)), N, workspace=g.Workspace(),
                            out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32))
    want = np.zeros((M, N), bool)
    want[2:5] = True
    assert np.array_equal(np.isnan(got), want)
    kept = np.delete(np.arange(M), [2, 3, 4])
    check_product(got[kept], a[kept], O.mx4_decode(codes, scales), None, half, f"a8 {M}")


@pytest.mark.parametrize("T,H", [(1, 96), (1, 2048), (9, 2048), (20, 96), (64, 96)])
def test_moe_weights_coded_from_nan(g, T, H):  # noqa: F811
    rng = np.random.default_rng(T)
    I, E = 96, 3
    m = Layer(g, rng, H, I, E)
    w1, w2 = (rng.standard_normal(s).astype(np.float32) * 0.05 for s in ((E * 2 * I, H), (E * H, I)))
    w1[2 * I * 1 + 3, H - 1] = np.nan                    # expert 1: every output of its tokens
    w2[H * 2 + 11, 40] = np.inf                          # expert 2: one column of them
    (m.c1, m.s1), (m.c2, m.s2) = O.mx4_encode(w1), O.mx4_encode(w2)
    m.pack(g)
    m.p1, m.p2 = (g.prepack_mx4(*g.quantize_mx4(dev(w))) for w in (w1, w2))
    x, logits = tokens(rng, T, H, E)
    for act in (0, 1, 2):
        y = host(m.check(g, x, logits, 1, act, what=f"act {act}"))
        ids, _ = O.moe_route(logits, 1, True)
        want = np.repeat(ids == 1, H, 1)
        want[ids[:, 0] == 2, 11] = True
        assert np.array_equal(np.isnan(y), want)
