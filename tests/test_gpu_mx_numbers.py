"""GPU: MXFP4 products and the expert layer on inputs whose sums are exact, bit for bit, and what
8-bit rows lose where their products drop bits."""
import numpy as np
import pytest

import oracle as O
from tests._mx_cases import EXACT, LAYERS, ExactLayer, dropped, exact_weights
from tests.test_gpu_mx import STEP, dev, g, host, product, weights  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ mixture of experts
def run_exact(g, m):  # noqa: F811
    p1, p2 = (g.prepack_mx4(dev(c), dev(s)) for c, s in ((m.c1, m.s1), (m.c2, m.s2)))
    got = host(g.moe_mx4(dev(m.x), dev(m.logits), m.top, p1, p2, m.I, act=g.W4_ACT_RELU2, workspace=g.Workspace()))
    off = got != m.want
    assert not off.any(), f"{int(off.sum())} of {off.size} off: {got[off][:5]} for {m.want[off][:5]}"


@pytest.mark.parametrize("case", LAYERS)
def test_moe_of_exact_numbers(g, case):  # noqa: F811
    run_exact(g, ExactLayer(np.random.default_rng(case[0] + case[1]), *case))


@pytest.mark.parametrize("up,down", [(114, -127), (114, -126), (112, -118), (-100, 95), (-110, 105)])
@pytest.mark.parametrize("case", [(1, 2048, 96, 60, 4, 3), (5, 2048, 32, 9, 4, 3), (20, 96, 160, 9, 4, 12),
                                  (64, 160, 96, 3, 2, 9)])
def test_moe_to_the_ends_of_float32(g, case, up, down):  # noqa: F811
    """h near the largest and the smallest float32 numbers, weights down to 2^-128."""
    run_exact(g, ExactLayer(np.random.default_rng(case[0]), *case, up=up, down=down))


# ------------------------------------------------------------------ products
# rows kernels of one to four column operands and strips, every tile, split along k, two launches
PLANS = [(1, 4096, 2080), (16, 8192, 512), (17, 11008, 512), (32, 16000, 512), (48, 11008, 512), (64, 12000, 512),
         (65, 300, 2080), (130, 260, 1056), (200, 1100, 1024), (700, 8640, 640), (2048, 4096, 512), (2048, 8192, 512),
         (1000, 17001, 160), (2048, 11008, 160)]


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M,N,K", PLANS)
def test_products_of_exact_numbers(g, act, M, N, K):  # noqa: F811
    rng = np.random.default_rng(M + N)
    codes, scales, w = exact_weights(rng, N, K, two=True)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    scale = np.ones(M, np.float32)
    if act == "a4":
        ca, sa, a = exact_weights(rng, M, K, two=True)
        t = (dev(ca), dev(sa))
    else:
        a = rng.integers(-4, 5, (M, K)).astype(np.float64)
        t = (dev(a.astype(np.float16)),)
    if act == "a8":
        # the terms of eight neighbours span less than 2^13: nothing is dropped
        scale = np.exp2(rng.integers(-2, 3, M)).astype(np.float32)
        f8 = torch.from_numpy(a).to(torch.float8_e4m3fn)
        assert torch.equal(f8.double(), torch.from_numpy(a))
        t = (f8.cuda(), dev(scale))
    assert K * np.abs(a).max() * np.abs(w).max() / 0.25 < EXACT
    want = (torch.from_numpy(a).float() @ torch.from_numpy(w).float().T).numpy() * scale[:, None]
    bias = rng.integers(-64, 65, N).astype(np.float16)
    ws = g.Workspace()
    for half in (True, False):
        got = host(product(g, act)(*t, Wp, N, bias=dev(bias), out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32,
                                   workspace=ws))
        right = (want + bias.astype(np.float32)).astype(np.float16) if half else want
        off = got != right
        assert not off.any(), f"half {half}: {int(off.sum())} of {off.size} off"


@pytest.mark.parametrize("M,N,K", [(5, 333, 1056), (20, 700, 320), (45, 100, 2080), (64, 260, 512), (90, 130, 2080),
                                   (130, 260, 416), (257, 300, 256)])
def test_8_bit_rows_lose_no_more_than_the_bits_dropped(g, M, N, K):  # noqa: F811
    """Codes of every size. Beyond the result's half step: each term may lose its bits below 2^-13 of the
    largest of its eight; float32 sums as in the products' other tests."""
    rng = np.random.default_rng(M)
    codes, scales = weights(rng, N, K)
    w = O.mx4_decode(codes, scales)
    rows = rng.integers(0, 256, (M, K), dtype=np.uint8)
    rows[(rows & 127) == 127] = 0
    a = O.e4m3_decode(rows).astype(np.float64)
    got = host(g.mx4a8_gemm(dev(rows), dev(np.ones(M, np.float32)), g.prepack_mx4(dev(codes), dev(scales)), N,
                            workspace=g.Workspace())).astype(np.float64)
    ref, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    tol = dropped(a, w) + (K / 16 + 16) * STEP * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    over = np.abs(ref) > 65000
    off = (np.abs(got - ref) > tol) & ~over
    assert over.mean() < 0.1
    assert not off.any(), f"{int(off.sum())} off, worst {np.max((np.abs(got - ref) / tol)[~over])}"


@pytest.mark.parametrize("M,N,K", [(1, 4096, 1024), (16, 8192, 512), (17, 11008, 512), (32, 16000, 512), (45, 3200, 2048),
                                   (64, 12000, 512), (65, 300, 2080), (200, 1100, 1024), (700, 8640, 640),
                                   (2048, 4096, 512), (2048, 8192, 512), (1000, 17001, 512)])
def test_8_bit_rows_of_normal_data(g, M, N, K):  # noqa: F811
    """The bias takes the result away, rounded to fp16, so that fp16 holds what is left of the float32 sum
    to 2^-22 of the result; one row, M times.

    Norm: 8e-6 of the result's for the dropped bits, and a step of a partial sum for each of K / 16 + 16
    additions, whose norms, for terms of any sign, are at most the result's; 2^-21 for the rounding of
    what is left."""
    rng = np.random.default_rng(N + K)
    codes, scales = O.mx4_encode(rng.standard_normal((N, K)) * K ** -0.5)
    w = O.mx4_decode(codes, scales)
    x = rng.standard_normal((1, K)).astype(np.float32)
    scale = (np.abs(x).max() / 448).astype(np.float32)
    f8 = (torch.from_numpy(x) / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    a = f8.double().numpy() * float(scale)
    ref = (a @ w.T)[0]
    bias = -ref.astype(np.float16)
    got = host(g.mx4a8_gemm(f8.cuda().repeat(M, 1), dev(np.full(M, scale)), g.prepack_mx4(dev(codes), dev(scales)), N,
                            bias=dev(bias), workspace=g.Workspace()))
    assert (got == got[0]).all()
    err = np.linalg.norm(got[0].astype(np.float64) - (ref + bias.astype(np.float64))) / np.linalg.norm(ref)
    assert err <= 8e-6 + (K / 16 + 16) * STEP + 2.0 ** -21, err
    print(f"{err:.3g} of the norm", flush=True)


# ------------------------------------------------------------------ far from one
@pytest.mark.parametrize("M", [3, 40, 100])
@pytest.mark.parametrize("low,up", [(-24, 14), (-24, -3), (-20, 0)])
def test_fp16_rows_of_subnormal_numbers(g, M, low, up):  # noqa: F811
    """Rows of whole multiples of 2^low, results down to fp16's subnormals: the sum rounded once."""
    rng = np.random.default_rng(M)
    N, K = 70, 544
    codes, scales, w = exact_weights(rng, N, K)
    a = rng.integers(-4, 5, (M, K)).astype(np.float64) * 2.0 ** low
    t = dev(a.astype(np.float16))
    assert np.array_equal(host(t).astype(np.float64), a)
    Wp = g.prepack_mx4(dev(codes), dev((scales.astype(int) + up).astype(np.uint8)))
    want = a @ w.T * 2.0 ** up
    for half in (True, False):
        got = host(g.mx4a16_gemm(t, Wp, N, out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32, workspace=g.Workspace()))
        assert np.array_equal(got, want.astype(np.float16 if half else np.float32)), half


@pytest.mark.parametrize("M", [3, 40, 100])
@pytest.mark.parametrize("low,up", [(-127, 120), (-126, 126), (-107, 100), (-60, 40), (60, -70), (110, -115)])
def test_8_bit_rows_far_from_one(g, M, low, up):  # noqa: F811
    """Weights and the rows' scale far apart; E4M3's least numbers, of which 2^-9 is one unit."""
    rng = np.random.default_rng(M)
    N, K = 70, 544
    codes, scales, w = exact_weights(rng, N, K)
    a = rng.integers(-7, 8, (M, K)) / 512.0
    f8 = torch.from_numpy(a).to(torch.float8_e4m3fn)
    assert torch.equal(f8.double(), torch.from_numpy(a))
    Wp = g.prepack_mx4(dev(codes), dev((scales.astype(int) + low).astype(np.uint8)))
    want = a @ w.T * 2.0 ** (low + up)
    for half in (True, False):
        got = host(g.mx4a8_gemm(f8.cuda(), dev(np.full(M, 2.0 ** up, np.float32)), Wp, N, workspace=g.Workspace(),
                                out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32))
        assert np.array_equal(got, want.astype(np.float16 if half else np.float32)), (half, got[0, :4], want[0, :4])


@pytest.mark.parametrize("M", [3, 40, 100])
@pytest.mark.parametrize("low,up", [(-127, 127), (127, -127), (-100, 95), (-60, -60), (80, 30)])
def test_4_bit_rows_far_from_one(g, M, low, up):  # noqa: F811
    rng = np.random.default_rng(M)
    N, K = 70, 544
    codes, scales, w = exact_weights(rng, N, K)
    ca, sa, a = exact_weights(rng, M, K)
    Wp = g.prepack_mx4(dev(codes), dev((scales.astype(int) + low).astype(np.uint8)))
    want = a @ w.T * 2.0 ** (low + up)
    got = host(g.mx4a4_gemm(dev(ca), dev((sa.astype(int) + up).astype(np.uint8)), Wp, N, out_dtype=g.W4_OUT_F32,
                            workspace=g.Workspace()))
    assert np.array_equal(got, want.astype(np.float32)), (got[0, :4], want[0, :4])
