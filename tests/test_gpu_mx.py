"""GPU: MXFP4 coding, products on MXFP4 weights and the mixture-of-experts layer,
through the public entry points, against the float64 oracle."""
import numpy as np
import pytest

import oracle as O
from tests._helpers import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23       # float32 spacing; sums in the matrix cores are taken to this, not to half of it


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_nibble_unpack_amd as G
    G.load()
    return G


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def guarded(x, fill):
    """x on the device with `fill` bytes directly behind it (what a read past the end would meet)."""
    raw = np.ascontiguousarray(x)
    buf = torch.full((raw.nbytes + 4096,), fill, dtype=torch.uint8, device="cuda")
    buf[:raw.nbytes] = torch.from_numpy(raw.view(np.uint8).reshape(-1)).cuda()
    return buf[:raw.nbytes].view(torch.from_numpy(raw).dtype).view(raw.shape)


# ------------------------------------------------------------------ coding
def values(rng, R, K, dt):
    x = rng.standard_normal((R, K)) * np.exp(rng.standard_normal((R, 1)))
    if dt == np.float32:
        x = x * np.exp2(rng.integers(-60, 60, (R, K // 32)).repeat(32, 1).astype(float))
    # ties and borders: quarters of small powers of two
    x[:, ::5] = rng.integers(-32, 33, x[:, ::5].shape) / 4 * 2.0 ** rng.integers(-3, 4)
    return x.astype(dt)


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (1, 4096), (7, 96), (33, 8640), (257, 1056), (1000, 320)])
def test_coding_is_the_definition_s(g, R, K, dt):
    x = values(np.random.default_rng(R * K), R, K, dt)
    codes, scales = g.quantize_mx4(dev(x))
    want = O.mx4_encode(x)
    assert np.array_equal(host(scales), want[1]) and np.array_equal(host(codes), want[0])
    v = O.mx4_decode(*want)
    assert np.array_equal(host(g.dequantize_mx4(codes, scales, torch.float32)), v.astype(np.float32))
    with np.errstate(over="ignore"):
        half = v.astype(np.float32).astype(np.float16)
    assert np.array_equal(host(g.dequantize_mx4(codes, scales)), half)


def special_rows(dt):
    f = np.finfo(dt)
    x = np.zeros((14, 64), dt)
    x[1, 3] = f.max
    x[2] = f.smallest_subnormal
    x[3, 40] = f.smallest_normal
    x[4, :7] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[4, 8], x[5, 31], x[6, 32] = 4, np.inf, -np.inf
    x[7, 0] = np.nan
    x[8, 5], x[8, 6] = np.nan, np.inf
    x[9] = -x[9]
    x[10] = np.nextafter(dt(8), dt(0))
    x[11] = -f.max
    x[12, ::2], x[12, 1::2] = f.smallest_normal, -f.smallest_subnormal
    x[13] = np.linspace(-6, 6, 64)
    return x


@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_coding_of_special_values(g, dt):
    x = special_rows(dt)
    codes, scales = g.quantize_mx4(dev(x))
    want = O.mx4_encode(x)
    assert np.array_equal(host(scales), want[1])
    assert np.array_equal(host(codes), want[0])
    v = host(g.dequantize_mx4(codes, scales, torch.float32))
    assert np.array_equal(v, O.mx4_decode(*want).astype(np.float32), equal_nan=True)


def test_decoding_of_every_code_and_scale(g):
    q = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    codes, scales = O.mx4_pack(q), np.arange(256, dtype=np.uint8)[:, None]
    want = O.mx4_decode(codes, scales)
    with np.errstate(over="ignore"):
        assert np.array_equal(host(g.dequantize_mx4(dev(codes), dev(scales), torch.float32)),
                              want.astype(np.float32), equal_nan=True)
        assert np.array_equal(host(g.dequantize_mx4(dev(codes), dev(scales))),
                              want.astype(np.float32).astype(np.float16), equal_nan=True)


@pytest.mark.parametrize("N,K", [(1, 32), (16, 128), (17, 160), (100, 640), (333, 8640)])
def test_packing_and_back(g, N, K):
    rng = np.random.default_rng(N)
    codes, scales = (rng.integers(0, 256, s, dtype=np.uint8) for s in ((N, K // 2), (N, K // 32)))
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    assert Wp.numel() == g.prepack_mx4_bytes(N, K)
    c, s = g.unprepack_mx4(Wp, N, K)
    assert np.array_equal(host(c), codes) and np.array_equal(host(s), scales)


# ------------------------------------------------------------------ products
def weights(rng, N, K, spread=2):
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (120 + rng.integers(-spread, spread + 1, (N, K // 32))).astype(np.uint8)
    return codes, scales


def rows(rng, act, M, K):
    """(call's tensors, float64 values)."""
    x = (rng.standard_normal((M, K)) * np.exp(0.7 * rng.standard_normal(K))).astype(np.float16)
    if act == "a16":
        return (guarded(x, 0xFF),), x.astype(np.float64)
    if act == "a8":
        codes = rng.integers(0, 256, (M, K), dtype=np.uint8)
        codes[(codes & 127) == 127] = 0                  # the NaN codes
        scale = np.exp(rng.standard_normal(M)).astype(np.float32)
        return (guarded(codes, 0xFF), dev(scale)), O.e4m3_decode(codes).astype(np.float64) * scale[:, None]
    codes, scales = O.mx4_encode(x)
    return (guarded(codes, 0xFF), guarded(scales, 0xFF)), O.mx4_decode(codes, scales)


def product(g, act):
    return {"a16": g.mx4a16_gemm, "a8": g.mx4a8_gemm, "a4": g.mx4a4_gemm}[act]


def check_product(got, a, w, bias, half, what):
    """Half a step of the result's type, and of float32 sums: at least 16 terms go
    into an addition, and each addition is off by at most a step of the sum of
    magnitudes (the partial sums' bound); 16 more for the split sums, the scales
    and the bias. E4M3 rows with an fp16 result: of eight neighbours along k each
    may lose 2^-13 of the largest, 2^-10 of the sum of magnitudes in all."""
    ref, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    if bias is not None and half:
        ref, mag = ref + bias, mag + np.abs(bias)
    tol = (a.shape[1] / 16 + 16) * STEP * mag + np.abs(ref) * 2.0 ** (-11 if half else -24)
    tol = tol + (2.0 ** -25 if half else 0) + (2.0 ** -10 * mag if half and what.startswith("a8") else 0)
    err = np.abs(got.astype(np.float64) - ref)
    assert np.isfinite(got).all(), what
    assert np.all(err <= tol), f"{what}: worst {np.max(err / tol)} of the bound, {int((err > tol).sum())} off"


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("N,K", [(1, 32), (16, 64), (17, 96), (100, 128), (40, 2080), (333, 416), (260, 1056)])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 130, 257, 400])
def test_products(g, act, M, N, K):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    codes, scales = weights(rng, N, K)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    w = O.mx4_decode(codes, scales)
    t, a = rows(rng, act, M, K)
    bias = rng.standard_normal(N).astype(np.float16)
    ws = g.Workspace()
    for b, half in ((None, True), (bias, True), (bias, False)):
        got = product(g, act)(*t, Wp, N, bias=None if b is None else dev(b),
                              out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32, workspace=ws)
        check_product(host(got), a, w, None if b is None else b.astype(np.float64), half,
                      f"{act} {M}x{N}x{K} bias {b is not None} half {half}")


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 3200, 8640), (48, 1024, 11008), (200, 1100, 3200),
                                   (700, 8640, 640), (2048, 4096, 512)])
def test_products_at_real_sizes(g, act, M, N, K):
    rng = np.random.default_rng(M)
    codes, scales = weights(rng, N, K)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    t, a = rows(rng, act, M, K)
    got = product(g, act)(*t, Wp, N, workspace=g.Workspace())
    check_product(host(got), a, O.mx4_decode(codes, scales), None, True, f"{act} {M}x{N}x{K}")
    again = product(g, act)(*t, Wp, N, workspace=g.Workspace())
    assert torch.equal(got, again)                       # bits repeat
    say("ok", act, M, N, K)


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M,N,K", [(65, 300, 8640), (40, 12500, 2080), (128, 130, 4128)])
def test_products_split_along_k(g, act, M, N, K):
    op = {"a16": g.W4_MX_A16, "a8": g.W4_MX_A8, "a4": g.W4_MX_A4}[act]
    rng = np.random.default_rng(N)
    codes, scales = weights(rng, N, K)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    w = O.mx4_decode(codes, scales)
    t, a = rows(rng, act, M, K)
    need = g.mx4_workspace_bytes(op, M, N, K)
    assert (need > 16384) == (N < 1000)                  # the wide one has tiles enough
    raw = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    raw[16384:] = 0xFF                                   # only the counters have to be zero
    for half in (True, False):
        got = product(g, act)(*t, Wp, N, out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32, workspace=raw)
        check_product(host(got), a, w, None, half, f"{act} {M}x{N}x{K} half {half}")
        assert not raw[:16384].any()
    if need:
        for short in (raw[:need - 1], raw[:16384]):
            with pytest.raises(g.W4Error):
                product(g, act)(*t, Wp, N, workspace=short)


@pytest.mark.parametrize("act", ["a8", "a4"])
@pytest.mark.parametrize("M,N,K", [(1000, 17001, 160), (1000, 20011, 96), (2000, 9000, 160), (2048, 11008, 64)])
def test_products_in_two_launches(g, act, M, N, K):
    """Sizes whose whole rounds of large tiles leave columns for smaller ones."""
    rng = np.random.default_rng(N)
    codes, scales = weights(rng, N, K)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    w = O.mx4_decode(codes, scales)
    t, a = rows(rng, act, M, K)
    bias = rng.standard_normal(N).astype(np.float16)
    for half in (True, False):
        guard = torch.full((M * N + 64,), 7.0, dtype=torch.float16 if half else torch.float32, device="cuda")
        got = product(g, act)(*t, Wp, N, bias=dev(bias), out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32,
                              C=guard[:M * N].view(M, N))
        check_product(host(got), a, w, bias.astype(np.float64), half, f"{act} {M}x{N}x{K} half {half}")
        assert (guard[M * N:] == 7).all()


@pytest.mark.parametrize("M", [7, 70, 300])
@pytest.mark.parametrize("K", [512, 544])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_a4_scales_at_any_address(g, M, K, off):
    rng = np.random.default_rng(off)
    N = 48
    codes, scales = weights(rng, N, K)
    t, a = rows(rng, "a4", M, K)
    s = torch.full((M * K // 32 + off,), 255, dtype=torch.uint8, device="cuda")[off:].view(M, K // 32)
    s.copy_(t[1])
    got = g.mx4a4_gemm(t[0], s, g.prepack_mx4(dev(codes), dev(scales)), N, out_dtype=g.W4_OUT_F32,
                       workspace=g.Workspace())
    check_product(host(got), a, O.mx4_decode(codes, scales), None, False, "a4")


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M", [3, 100])
def test_scales_of_any_size(g, act, M):
    """Scales far apart in a row and between rows; float32 out, so nothing overflows."""
    rng = np.random.default_rng(5)
    N, K = 48, 512
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (rng.integers(-15, 16, (N, K // 32)) + rng.integers(70, 180, N)[:, None]).astype(np.uint8)
    codes[3, :16] = 0
    scales[3, 0] = 254                                   # a block of zeros with a huge scale
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    t, a = rows(rng, act, M, K)
    got = product(g, act)(*t, Wp, N, out_dtype=g.W4_OUT_F32)
    check_product(host(got), a, O.mx4_decode(codes, scales), None, False, act)


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M", [3, 100])
def test_blocks_of_zeros_whatever_their_scale(g, act, M):
    rng = np.random.default_rng(7)
    N, K = 20, 256 * 32
    codes = rng.choice(np.array([0, 8, 128], np.uint8), (N, K // 2))          # +0 and -0
    scales = np.tile(np.append(np.arange(255), 0), (N, 1)).astype(np.uint8)
    for n in range(N - 1):                               # one block that is not zeros; the last row has none
        codes[n, 16 * 255:] = rng.integers(0, 256, 16)
        scales[n, 255] = 100 + 3 * n
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    t, a = rows(rng, act, M, K)
    for half in (True, False):
        got = product(g, act)(*t, Wp, N, out_dtype=g.W4_OUT_F16 if half else g.W4_OUT_F32, workspace=g.Workspace())
        assert torch.isfinite(got[:, N - 1]).all() and not got[:, N - 1].any()
        if not half:
            check_product(host(got), a, O.mx4_decode(codes, scales), None, False, act)


@pytest.mark.parametrize("M", [2, 66])
def test_weights_past_4_gib(g, M):
    """Rows of zeros but for the first and the last strips."""
    rng = np.random.default_rng(M)
    N, K, R = (1 << 20) + 5, 8320, 40
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(N, K // 32, dtype=torch.uint8, device="cuda")
    c, s = weights(rng, 2 * R, K)
    for x, y in ((codes, c), (scales, s)):
        x[:R] = dev(y[:R])
        x[N - R:] = dev(y[R:])
    Wp = g.prepack_mx4(codes, scales)
    assert Wp.numel() > 1 << 32
    w = O.mx4_decode(c, s)
    for act in ("a16", "a8", "a4"):
        t, a = rows(rng, act, M, K)
        got = product(g, act)(*t, Wp, N, workspace=g.Workspace())
        check_product(host(torch.cat((got[:, :R], got[:, N - R:]), 1)), a, w, None, True, act)
        assert not got[:, R:N - R].any()
    c2, s2 = g.unprepack_mx4(Wp, N, K)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_rows_past_4_gib(g):
    rng = np.random.default_rng(2)
    M, N, K, R = 262144 + 9, 33, 8320, 300
    codes, scales = weights(rng, N, K)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    w = O.mx4_decode(codes, scales)
    x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    some = rng.standard_normal((R, K)).astype(np.float16)
    x[M - R:] = dev(some)
    got = g.mx4a16_gemm(x, Wp, N, workspace=g.Workspace())
    check_product(host(got[M - R:]), some.astype(np.float64), w, None, True, "a16")
    assert not got[:M - R].any()
    # coded, back, and their product
    qc, qs = g.quantize_mx4(x)
    wc, ws_ = O.mx4_encode(some)
    assert np.array_equal(host(qc[M - R:]), wc) and np.array_equal(host(qs[M - R:]), ws_)
    back = g.dequantize_mx4(qc, qs)
    assert np.array_equal(host(back[M - R:]), O.mx4_decode(wc, ws_).astype(np.float16)) and not back[:M - R].any()
    got = g.mx4a4_gemm(qc, qs, Wp, N, workspace=g.Workspace())
    check_product(host(got[M - R:]), O.mx4_decode(wc, ws_), w, None, True, "a4")


@pytest.mark.parametrize("M", [3, 100])
def test_a16_blocks_far_below_their_row(g, M):
    """Blocks below 2^-35 of their row's largest scale are rounded to 2^-36 of it."""
    rng = np.random.default_rng(6)
    N, K = 16, 256
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = rng.integers(60, 131, (N, K // 32)).astype(np.uint8)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    t, a = rows(rng, "a16", M, K)
    w = O.mx4_decode(codes, scales)
    got = host(g.mx4a16_gemm(*t, Wp, N, out_dtype=g.W4_OUT_F32)).astype(np.float64)
    mag = np.abs(a) @ np.abs(w).T
    top = np.exp2(scales.max(1).astype(float) - 127)
    tol = (K / 16 + 16) * STEP * mag + np.abs(a).sum(1)[:, None] * top * 2.0 ** -36
    assert np.all(np.abs(got - a @ w.T) <= tol)


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
@pytest.mark.parametrize("M", [5, 90])
def test_nan_reaches_what_meets_it_and_no_more(g, act, M):
    rng = np.random.default_rng(9)
    N, K = 50, 416
    codes, scales = weights(rng, N, K)
    scales[20, 3] = 255
    t, _ = rows(rng, act, M, K)
    if act == "a16":
        t[0][2, 7] = float("nan")
        t[0][4, 100] = float("inf")
    elif act == "a8":
        t[0][2, 7] = 0x7F
        t[1][4] = float("nan")
    else:
        t[1][2, 1] = 255
        t[1][4, 12] = 255
    got = host(product(g, act)(*t, g.prepack_mx4(dev(codes), dev(scales)), N))
    bad = ~np.isfinite(got)
    want = np.zeros((M, N), bool)
    want[:, 20] = want[2] = want[4] = True
    if act == "a16":
        # infinity times zero codes is NaN, times others infinite: not finite either way
        assert np.isnan(got[2]).all() and np.isnan(got[:, 20]).all()
    else:
        assert np.isnan(got[want]).all()
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
def test_products_on_a_stream_into_given_outputs_and_in_a_graph(g, act):
    rng = np.random.default_rng(11)
    for M, N, K in ((4, 96, 1024), (200, 96, 1024)):
        codes, scales = weights(rng, N, K)
        Wp = g.prepack_mx4(dev(codes), dev(scales))
        t, a = rows(rng, act, M, K)
        ws, ws2 = g.Workspace(), g.Workspace()
        want = product(g, act)(*t, Wp, N, workspace=ws)
        C = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        assert product(g, act)(*t, Wp, N, C=C, workspace=ws2, stream=s) is C
        s.synchronize()
        assert torch.equal(C, want)
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                product(g, act)(*t, Wp, N, C=C, workspace=ws2)
        for _ in range(3):
            C.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(C, want)
            assert torch.equal(product(g, act)(*t, Wp, N, workspace=ws), want)


def test_no_rows(g):
    codes, scales = weights(np.random.default_rng(0), 16, 64)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    assert g.mx4a16_gemm(torch.empty(0, 64, dtype=torch.float16, device="cuda"), Wp, 16).shape == (0, 16)
    c, s = g.quantize_mx4(torch.empty(0, 64, device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    m = Layer(g, np.random.default_rng(1), 64, 32, 2)
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    assert g.moe_mx4(x, torch.empty(0, 2, device="cuda"), 1, m.p1, m.p2, 32).shape == (0, 64)


def test_refusals_of_tensors(g):
    codes, scales = weights(np.random.default_rng(0), 16, 64)
    Wp = g.prepack_mx4(dev(codes), dev(scales))
    x = torch.zeros(2, 64, dtype=torch.float16, device="cuda")
    u8 = torch.zeros(2, 64, dtype=torch.uint8, device="cuda")
    sc = torch.ones(2, device="cuda")
    for call in (lambda: g.mx4a16_gemm(x.float(), Wp, 16), lambda: g.mx4a16_gemm(x, Wp, 17),
                 lambda: g.mx4a16_gemm(x, Wp[:100], 16), lambda: g.mx4a16_gemm(x, Wp, 16, bias=sc),
                 lambda: g.mx4a16_gemm(x, Wp, 16, C=torch.zeros(2, 17, device="cuda").half()),
                 lambda: g.mx4a16_gemm(x[:, ::2], Wp, 16), lambda: g.mx4a16_gemm(x, Wp.cpu(), 16),
                 lambda: g.mx4a8_gemm(u8, sc[:1], Wp, 16), lambda: g.mx4a8_gemm(u8, sc.half(), Wp, 16),
                 lambda: g.mx4a8_gemm(u8, None, Wp, 16), lambda: g.mx4a4_gemm(u8[:, :32].contiguous(), u8, Wp, 16),
                 lambda: g.quantize_mx4(x.bfloat16()), lambda: g.quantize_mx4(x[0]),
                 lambda: g.quantize_mx4(x, out=(u8, u8)), lambda: g.dequantize_mx4(u8, u8),
                 lambda: g.moe_mx4(x, torch.zeros(3, 4, device="cuda"), 2, Wp, Wp, 32),
                 lambda: g.moe_mx4(x, torch.zeros(2, 4, device="cuda"), 2, Wp, Wp, 32),
                 lambda: g.moe_mx4(x, torch.zeros(2, 4, device="cuda").bfloat16(), 2, Wp, Wp, 32)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.quantize_mx4(torch.zeros(2, 48, device="cuda")),
                 lambda: g.mx4a16_gemm(x, Wp, 16, out_dtype=g.W4_OUT_I32),
                 lambda: g.moe_mx4(x, torch.zeros(2, 4, device="cuda"), 2, Wp, Wp, 48)):
        with pytest.raises(g.W4Error):
            call()


# ------------------------------------------------------------------ mixture of experts
class Layer:
    def __init__(self, g, rng, H, I, E):
        self.H, self.I, self.E = H, I, E
        self.c1, self.s1 = weights(rng, E * 2 * I, H)
        self.c2, self.s2 = weights(rng, E * H, I)
        self.pack(g)

    def pack(self, g):
        self.p1, self.p2 = (g.prepack_mx4(dev(c), dev(s)) for c, s in ((self.c1, self.s1), (self.c2, self.s2)))
        self.w1 = O.mx4_decode(self.c1, self.s1).reshape(self.E, 2 * self.I, self.H)
        self.w2 = O.mx4_decode(self.c2, self.s2).reshape(self.E, self.H, self.I)

    def check(self, g, x, logits, top, act=0, renorm=True, ws=None, what=""):
        got = g.moe_mx4(dev(x), dev(logits), top, self.p1, self.p2, self.I, act=act, renormalize=renorm,
                        workspace=g.Workspace() if ws is None else ws)
        ref, err = O.moe_layer(x, logits, top, self.w1, self.w2, act, renorm)
        y = host(got).astype(np.float64)
        nan = np.isnan(ref)
        assert np.array_equal(np.isnan(y), nan), what
        # the result's half step; weights of the softmax: 64 roundings of float32
        tol = err + (2.0 ** -11 + 64 * STEP) * np.abs(ref) + 2.0 ** -25
        over = np.abs(ref) + err > 65504
        with np.errstate(invalid="ignore"):
            off = (np.abs(y - ref) > tol) & ~nan & ~over
        assert not off.any(), f"{what}: {int(off.sum())} off, worst {np.max((np.abs(y - ref) / tol)[off])}"
        return got


def tokens(rng, T, H, E, dt=np.float32):
    return (0.05 * rng.standard_normal((T, H))).astype(np.float16), (1.5 * rng.standard_normal((T, E))).astype(dt)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("H,I,E,top", [(64, 32, 4, 2), (160, 96, 9, 3), (416, 288, 1, 1), (1024, 512, 5, 5),
                                       (96, 64, 70, 8)])
def test_moe(g, T, H, I, E, top):
    rng = np.random.default_rng(T + H)
    m = Layer(g, rng, H, I, E)
    ws = g.Workspace()
    for act, renorm, dt in ((0, True, np.float32), (1, False, np.float16), (2, True, np.float16)):
        m.check(g, *tokens(rng, T, H, E, dt), top, act, renorm, ws, f"T {T} H {H} I {I} E {E} act {act}")


@pytest.mark.parametrize("T", [1, 2, 5, 16, 17])
@pytest.mark.parametrize("H,I,E,top", [(2080, 96, 5, 3), (2048, 32, 140, 6), (2144, 160, 100, 1)])
def test_moe_wide_hidden(g, T, H, I, E, top):
    """hidden at which a few tokens are the columns of the second product, and the choices
    among more than 64 and more than 128 experts."""
    rng = np.random.default_rng(T + H)
    m = Layer(g, rng, H, I, E)
    ws = g.Workspace()
    for renorm, dt in ((True, np.float32), (False, np.float16)):
        m.check(g, *tokens(rng, T, H, E, dt), top, 0, renorm, ws, f"T {T} H {H}")
    x, logits = tokens(rng, T, H, E)
    logits[-1] = -np.inf
    assert not host(m.check(g, x, logits, top, ws=ws))[-1].any()
    logits[-1, E // 2] = np.nan
    m.check(g, x, logits, top, ws=ws)
    logits[-1] = 1.0
    m.check(g, x, logits, top, ws=ws)


def test_moe_one_token_longer_than_the_first_product_keeps(g):
    rng = np.random.default_rng(8)
    m = Layer(g, rng, 16416, 32, 3)
    m.check(g, *tokens(rng, 1, 16416, 3), 2)


@pytest.mark.parametrize("T", [1, 6, 16, 40, 64])
@pytest.mark.parametrize("H,I,E,top", [(96, 160, 4, 3), (2048, 96, 4, 3), (160, 224, 16, 16), (64, 96, 60, 2)])
def test_moe_on_a_workspace_of_nan(g, T, H, I, E, top):
    """Only the counters have to be zero; some choices are none, and exactly the bytes asked for are there."""
    rng = np.random.default_rng(T + E)
    m = Layer(g, rng, H, I, E)
    x, logits = tokens(rng, T, H, E)
    logits[rng.random((T, E)) < 0.5] = -np.inf
    need = g.moe_mx4_workspace_bytes(T, H, I, E, top)
    raw = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    raw[:16384] = 0
    m.check(g, x, logits, top, ws=raw[:need])
    assert not raw[:16384].any() and (raw[need:] == 255).all()
    with pytest.raises(g.W4Error):
        m.check(g, x, logits, top, ws=raw[:need - 1])


@pytest.mark.parametrize("T", [4, 64])
def test_moe_most_choices(g, T):
    rng = np.random.default_rng(9)
    m = Layer(g, rng, 64, 32, 512)
    m.check(g, *tokens(rng, T, 64, 512), 16)


@pytest.mark.parametrize("T", [1, 3, 20])
def test_moe_experts_past_4_gib(g, T):
    """512 experts of zeros but for the first, one between and the last."""
    rng = np.random.default_rng(T)
    H, I, E, used = 8192, 2080, 512, [0, 300, 511]

    def fill(rows, K):
        c = torch.zeros(E * rows, K // 2, dtype=torch.uint8, device="cuda")
        s = torch.zeros(E * rows, K // 32, dtype=torch.uint8, device="cuda")
        hc, hs = weights(rng, len(used) * rows, K)
        for i, e in enumerate(used):
            c[e * rows:(e + 1) * rows] = dev(hc[i * rows:(i + 1) * rows])
            s[e * rows:(e + 1) * rows] = dev(hs[i * rows:(i + 1) * rows])
        return g.prepack_mx4(c, s), O.mx4_decode(hc, hs).reshape(len(used), rows, K)

    p1, w1 = fill(2 * I, H)
    p2, w2 = fill(H, I)
    assert min(p1.numel(), p2.numel()) > 1 << 32
    m = Layer.__new__(Layer)
    m.H, m.I, m.E, m.p1, m.p2, m.w1, m.w2 = H, I, E, p1, p2, w1, w2
    x, few = tokens(rng, T, H, len(used))
    logits = np.full((T, E), -np.inf, np.float32)
    logits[:, used] = few
    got = g.moe_mx4(dev(x), dev(logits), 2, p1, p2, I, workspace=g.Workspace())
    ref, err = O.moe_layer(x, few, 2, w1, w2, 0, True)
    tol = err + (2.0 ** -11 + 64 * STEP) * np.abs(ref) + 2.0 ** -25
    assert np.all(np.abs(host(got).astype(np.float64) - ref) <= tol)


@pytest.mark.parametrize("T,H", [(1, 96), (1, 2048), (9, 96), (9, 2048), (40, 160)])
def test_moe_into_its_input(g, T, H):
    rng = np.random.default_rng(T)
    m = Layer(g, rng, H, 64, 4)
    x, logits = tokens(rng, T, H, 4)
    want = m.check(g, x, logits, 2)
    for _ in range(3):
        y = dev(x)
        assert g.moe_mx4(y, dev(logits), 2, m.p1, m.p2, 64, workspace=g.Workspace(), out=y) is y
        assert torch.equal(y, want)


@pytest.mark.parametrize("T", [2, 20])
def test_moe_rows_of_zeros_whatever_their_scale(g, T):
    rng = np.random.default_rng(3)
    m = Layer(g, rng, 8192, 32, 2)
    m.c1[5] = 0
    m.s1[5] = np.append(np.arange(255), 116)
    m.pack(g)
    m.check(g, *tokens(rng, T, 8192, 2), 2)


@pytest.mark.parametrize("T", [5, 40])
def test_moe_every_token_on_one_expert(g, T):
    rng = np.random.default_rng(1)
    m = Layer(g, rng, 160, 96, 6)
    x, logits = tokens(rng, T, 160, 6)
    logits[:, 4] = 9
    m.check(g, x, logits, 1, what="one expert")


@pytest.mark.parametrize("T", [6, 30, 64])
def test_moe_ties_masks_and_nan(g, T):
    rng = np.random.default_rng(2)
    E = 130
    m = Layer(g, rng, 96, 64, E)
    x, logits = tokens(rng, T, 96, E)
    logits[0] = 0.5                                      # all alike: the first experts
    logits[1] = -np.inf
    logits[1, 77] = -3                                   # one left
    logits[2] = -np.inf                                  # none
    logits[3, 9] = np.nan
    logits[4, 100] = np.inf
    logits[5, ::2], logits[5, 1::2] = 0.0, -0.0          # equal
    for renorm in (True, False):
        y = host(m.check(g, x, logits, 4, renorm=renorm, what="masks"))
        assert not y[2].any() and np.isnan(y[3:5]).all()


@pytest.mark.parametrize("T", [3, 20])
def test_moe_no_token_chooses(g, T):
    rng = np.random.default_rng(3)
    m = Layer(g, rng, 64, 32, 3)
    x, logits = tokens(rng, T, 64, 3)
    ws = g.Workspace()
    assert not host(m.check(g, x, np.full_like(logits, -np.inf), 2, ws=ws)).any()
    m.check(g, x, logits, 2, ws=ws, what="afterwards")


@pytest.mark.parametrize("size", [1e-4, 60.0])
@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("act", [0, 2])
def test_moe_small_and_large_activations(g, T, size, act):
    """h below fp16's normal range, and far above its range where the weights bring it back."""
    rng = np.random.default_rng(4)
    m = Layer(g, rng, 128, 160, 4)
    shift = -12 if size > 1 else 12
    m.s2 = (m.s2.astype(int) + shift).astype(np.uint8)
    m.pack(g)
    x = (size * rng.standard_normal((T, 128))).astype(np.float16)
    m.check(g, x, rng.standard_normal((T, 4)).astype(np.float32), 2, act, what=f"size {size}")


@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("H", [96, 2048])
def test_moe_nan_weights_reach_the_expert_s_tokens_only(g, T, H):
    rng = np.random.default_rng(5)
    m = Layer(g, rng, H, 64, 4)
    m.s1[2 * 64 * 1 + 5, 1] = 255                        # expert 1, a gate row
    m.s2[H * 3 + 7, 1] = 255                             # expert 3, a row of its output
    m.pack(g)
    x, logits = tokens(rng, T, H, 4)
    logits[:, 1] = -9
    logits[0, 1] = 9
    logits[:, 3] = -9
    logits[1, 3] = 9
    y = host(g.moe_mx4(dev(x), dev(logits), 2, m.p1, m.p2, 64, workspace=g.Workspace()))
    want = np.zeros((T, H), bool)
    want[0] = True
    want[1, 7] = True
    assert np.array_equal(np.isnan(y), want)


@pytest.mark.parametrize("T", [1, 6, 12, 48])
def test_moe_repeats_on_streams_and_in_graphs(g, T):
    rng = np.random.default_rng(6)
    m = Layer(g, rng, 256, 160, 8)
    x, logits = (dev(v) for v in tokens(rng, T, 256, 8))
    ws, ws2 = g.Workspace(), g.Workspace()

    def call(**k):
        return g.moe_mx4(x, logits, 3, m.p1, m.p2, 160, **k)
    want = call(workspace=ws)
    for _ in range(3):
        assert torch.equal(call(workspace=ws), want)
    out = torch.full_like(x, 3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert call(workspace=ws2, out=out, stream=s) is out
    s.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(workspace=ws2, out=out)
    first = x.clone()
    for i in range(3):
        x.copy_(first * (i + 1))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call(workspace=ws))
    # the workspace serves a product afterwards: its counters are zero
    assert not ws.buf[:16384].any()


# ------------------------------------------------------------------ together
def test_a_step_of_a_layer_in_a_graph(g):
    """What a decode step runs between its attention and its residual: norm to E4M3 rows, their
    product, rows to MXFP4, their product, the router's product on fp16 rows, the experts;
    replayed with other inputs, two streams at once with a workspace each."""
    rng = np.random.default_rng(21)
    T, H, I, E, top = 12, 512, 160, 8, 3
    w = {n: weights(rng, r, H) for n, r in (("a", H), ("b", H), ("r", E))}
    packed = {n: g.prepack_mx4(dev(c), dev(s)) for n, (c, s) in w.items()}
    m = Layer(g, rng, H, I, E)
    gain = (1 + 0.1 * rng.standard_normal(H)).astype(np.float16)
    dgain = dev(gain)

    def step(x, res, ws):
        rows, scale, res = g.add_rmsnorm_q8(x, dgain, res, q_dtype=g.W4_Q_F8)
        y = g.mx4a8_gemm(rows, scale, packed["a"], H, workspace=ws)
        z = g.mx4a4_gemm(*g.quantize_mx4(y), packed["b"], H, workspace=ws)
        logits = g.mx4a16_gemm(z, packed["r"], E, out_dtype=g.W4_OUT_F32, workspace=ws)
        return g.moe_mx4(z, logits, top, m.p1, m.p2, I, workspace=ws), rows, scale, y, z, logits

    xs = [(dev(rng.standard_normal((T, H)).astype(np.float16)), dev(rng.standard_normal((T, H)).astype(np.float16)))
          for _ in range(3)]
    eager = [step(x, r, g.Workspace()) for x, r in xs]
    # each stage against the oracle, on the inputs that it got
    for out, rows_, scale, y, z, logits in eager:
        a8 = O.e4m3_decode(host(rows_)).astype(np.float64) * host(scale)[:, None]
        check_product(host(y), a8, O.mx4_decode(*w["a"]), None, True, "a8")
        a4 = O.mx4_decode(*O.mx4_encode(host(y)))
        check_product(host(z), a4, O.mx4_decode(*w["b"]), None, True, "a4")
        check_product(host(logits), host(z).astype(np.float64), O.mx4_decode(*w["r"]), None, False, "a16")
        m.check(g, host(z), host(logits), top)
    graphs = []
    for x, r in xs[:2]:
        s, ws = torch.cuda.Stream(), g.Workspace()
        s.wait_stream(torch.cuda.current_stream())
        x, r = x.clone(), r.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            step(x, r, ws)                               # allocates the workspace
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out = step(x, r, ws)[0]
        graphs.append((graph, s, x, r, out, ws))
    for i in range(3):
        for n, (graph, s, x, r, out, _) in enumerate(graphs):
            x.copy_(xs[(i + n) % 3][0])
            r.copy_(xs[(i + n) % 3][1])
        torch.cuda.synchronize()
        for graph, s, *_ in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for n, (*_, out, ws) in enumerate(graphs):
            assert torch.equal(out, eager[(i + n) % 3][0])
            assert not ws.buf[:16384].any()
