"""Host-only checks of the MXFP4 operators: header, library and binding agree, bad
arguments are rejected before a launch, the oracle's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import gemv_nibble_unpack_amd as G
import oracle as O
from gemv_nibble_unpack_amd import _lib as L

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "gemv_nibble_unpack_mx.h")
P = ctypes.c_void_p(0x7F0000000000)
MIS = ctypes.c_void_p(0x7F0000000004)
ODD = ctypes.c_void_p(0x7F0000000001)


def test_header_and_library_agree():
    text = open(HEADER).read()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", code, flags=re.M))
    assert names == set(L.MX_SIGNATURES)
    for n in names:
        assert hasattr(G.load(), n) and hasattr(G, n), n
    for name, value in re.findall(r"#define\s+(W4_\w+)\s+(\d+)", text):
        assert int(value) == getattr(L, name) == getattr(G, name), name


def calls(f, ok):
    def call(**at):
        a = list(ok)
        for k, v in at.items():
            a[int(k[1:])] = v
        return f(*a)
    return call


@pytest.mark.parametrize("name", ["quantize_mx4", "dequantize_mx4"])
def test_coding_refusals(name):
    first = name == "quantize_mx4"
    dt, r, k = (1, 2, 3) if first else (4, 2, 3)
    call = calls(getattr(G.load(), name), [P, 0, 2, 64, P, P, None] if first else [P, P, 2, 64, 0, P, None])
    for i in (0, 4, 5) if first else (0, 1, 5):
        assert call(**{f"_{i}": None}) == L.W4_ERR_NULL, i
    assert call(**{f"_{dt}": 2}) == L.W4_ERR_ARG and call(**{f"_{dt}": -1}) == L.W4_ERR_ARG
    for K in (0, 16, 33, 48, -32, L.W4_MAX_K + 16):
        assert call(**{f"_{k}": K}) == L.W4_ERR_SHAPE, K
    assert call(**{f"_{r}": -1}) == L.W4_ERR_SHAPE
    for i in (0, 4) if first else (0, 5):
        assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, i
    assert call(**{f"_{r}": 0, "_0": None}) == L.W4_OK


def test_prepack_refusals():
    for name, ok, n, k, codes, packed in (("prepack_mx4", [P, P, 5, 64, P, None], 2, 3, 0, 4),
                                          ("unprepack_mx4", [P, 5, 64, P, P, None], 1, 2, 3, 0)):
        call = calls(getattr(G.load(), name), ok)
        for i, v in enumerate(ok[:5]):
            if v is P:
                assert call(**{f"_{i}": None}) == L.W4_ERR_NULL, (name, i)
        for v in (0, -1, (1 << 30) + 1):
            assert call(**{f"_{n}": v}) == L.W4_ERR_SHAPE, (name, v)
        for v in (0, 16, 40, L.W4_MAX_K + 16):
            assert call(**{f"_{k}": v}) == L.W4_ERR_SHAPE, (name, v)
        for i in (codes, packed):
            assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, (name, i)
    assert G.prepack_mx4_bytes(0, 64) == G.prepack_mx4_bytes(5, 48) == 0
    # codes in whole tiles, a word of scales for each lane and four tiles, a byte a row
    assert G.prepack_mx4_bytes(1, 32) == 1024 + 256 + 16
    assert G.prepack_mx4_bytes(33, 640) == 3 * (5 * 1024 + 2 * 256 + 16)


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
def test_product_refusals(act):
    s = [] if act == "a16" else [P]
    o = len(s)
    ok = [P, *s, P, P, P, 0, 3, 40, 64, None, 0, None]
    call = calls(getattr(G.load(), f"mx4{act}_gemm"), ok)
    for i in [0, *([1] if s else []), 1 + o, 3 + o]:
        assert call(**{f"_{i}": None}) == L.W4_ERR_NULL, i
    for v in (2, 3, -1):
        assert call(**{f"_{4 + o}": v}) == L.W4_ERR_ARG
    for i, v in ((5, -1), (5, (1 << 30) + 1), (6, 0), (6, (1 << 30) + 1), (7, 48), (7, 0), (7, L.W4_MAX_K + 16)):
        assert call(**{f"_{i + o}": v}) == L.W4_ERR_SHAPE, (i, v)
    for i in (0, 1 + o, 3 + o, 8 + o):
        assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, i
    assert call(**{f"_{2 + o}": ODD}) == L.W4_ERR_ALIGN
    if act == "a8":
        assert call(_1=ODD) == L.W4_ERR_ALIGN
    assert call(**{f"_{5 + o}": 0, "_0": None}) == L.W4_OK


@pytest.mark.parametrize("act", ["a16", "a8", "a4"])
def test_products_of_too_many_tiles(act):
    s = [] if act == "a16" else [P]
    for M, N in ((1 << 30, 1 << 30), (1 << 30, 4096), (300, 1 << 30)):
        st = getattr(G.load(), f"mx4{act}_gemm")(P, *s, P, None, P, 0, M, N, 32, None, 0, None)
        assert st == L.W4_ERR_SHAPE and G.mx4_workspace_bytes(int(act == "a8") + 2 * (act == "a4"), M, N, 32) == 0


#      x  logits dt T  H   I   E  k  ren act w1 w2 out ws nb stream
MOE = [P, P, 1, 3, 64, 96, 8, 2, 1, 0, P, P, P, P, 1 << 30, None]


def test_moe_refusals():
    call = calls(G.load().moe_mx4, MOE)
    for i in (0, 1, 10, 11, 12):
        assert call(**{f"_{i}": None}) == L.W4_ERR_NULL, i
    for i, v in ((2, 2), (2, -1), (9, 3), (9, -1)):
        assert call(**{f"_{i}": v}) == L.W4_ERR_ARG, (i, v)
    for i, v in ((3, -1), (3, 65), (4, 0), (4, 48), (4, L.W4_MAX_K + 16), (5, 16), (5, 0), (5, L.W4_MAX_K + 16),
                 (6, 0), (6, 513), (7, 0), (7, 9), (7, 17)):
        assert call(**{f"_{i}": v}) == L.W4_ERR_SHAPE, (i, v)
    assert call(_6=40, _7=17) == L.W4_ERR_SHAPE
    for i in (0, 10, 11, 12, 13):
        assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, i
    assert call(_1=ODD) == L.W4_ERR_ALIGN
    assert call(_13=None) == L.W4_ERR_WORKSPACE and call(_14=4096) == L.W4_ERR_WORKSPACE
    assert call(_3=0, _0=None) == L.W4_OK


def test_moe_workspace():
    f = G.moe_mx4_workspace_bytes
    assert f(0, 64, 64, 4, 2) == f(65, 64, 64, 4, 2) == f(1, 64, 48, 4, 2) == f(1, 64, 64, 4, 5) == 0
    assert f(1, 64, 64, 4, 2) >= 16384 + 2 * 64 * 4
    assert f(64, 4096, 1536, 64, 4) >= 256 * (4096 + 1536) * 4


def test_wrappers_refuse():
    torch = pytest.importorskip("torch")
    u = torch.zeros(2, 32, dtype=torch.uint8)
    for call in (lambda: G.quantize_mx4(torch.zeros(2, 64)), lambda: G.dequantize_mx4(u, u[:, :2].contiguous()),
                 lambda: G.prepack_mx4(u, u[:, :2].contiguous()), lambda: G.unprepack_mx4(u, 16, 64),
                 lambda: G.dequantize_mx4(u, u, dtype=torch.bfloat16),
                 lambda: G.mx4a16_gemm(torch.zeros(2, 64).half(), u, 16),
                 lambda: G.moe_mx4(torch.zeros(2, 64).half(), torch.zeros(2, 4), 2, u, u, 64,
                                   workspace=torch.zeros(4))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the oracle's pins
def test_every_code_decodes_to_its_value():
    q = np.tile(np.arange(16, dtype=np.uint8), 2)[None]
    v = O.mx4_decode(O.mx4_pack(q), np.array([[127]], np.uint8))[0]
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert v[:8].tolist() == want and v[8:16].tolist() == [-x for x in want]
    assert O.mx4_decode(O.mx4_pack(q), np.array([[130]], np.uint8))[0, 7] == 48
    assert np.isnan(O.mx4_decode(O.mx4_pack(q), np.array([[255]], np.uint8))).all()
    assert np.array_equal(O.mx4_unpack(O.mx4_pack(q)), q)


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32))
    x[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    codes, scale = O.mx4_encode(x)
    v = O.mx4_decode(codes, scale)[0]
    assert scale[0, 0] == 127 and v[:9].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, -4]
    x[0, 1:9] = [0.2501, 0.7499, 1.2501, 1.7499, 2.5001, 3.4999, 5.0001, -7.9]
    assert O.mx4_decode(*O.mx4_encode(x))[0, :9].tolist() == [4, 0.5, 0.5, 1.5, 1.5, 3, 3, 6, -6]


def test_scales():
    for m, byte in ((0.0, 0), (6.0, 127), (4.0, 127), (3.99, 126), (8.0, 128), (2.0 ** 127, 252), (2.0 ** -126, 0),
                    (2.0 ** -149, 0), (2.0 ** -124, 1), (np.inf, 255), (np.nan, 255)):
        x = np.zeros((1, 32))
        x[0, 5] = m
        codes, scale = O.mx4_encode(x)
        assert scale[0, 0] == byte, m
        if byte == 255:
            assert not codes.any()


def test_route_closed_forms():
    ids, w = O.moe_route([[0.0, np.log(3.0), 0.0], [1.0, 1.0, 1.0]], 2, True)
    assert ids.tolist() == [[1, 0], [0, 1]] and np.allclose(w, [[0.75, 0.25], [0.5, 0.5]])
    ids, w = O.moe_route([[0.0, np.log(2.0), 0.0, -np.inf]], 2, False)
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = O.moe_route([[-np.inf] * 3, [1.0, -np.inf, -np.inf], [np.nan, 0, 0], [np.inf, 0, 0]], 2, True)
    assert ids.tolist() == [[-1, -1], [0, -1], [-1, -1], [-1, -1]]
    assert w[:2].tolist() == [[0, 0], [1, 0]] and np.isnan(w[2:]).all()


def test_layer_closed_form():
    # one expert, identity-like weights: out = relu(x)^2 * x
    x = np.array([[1.0, -2.0, 3.0]])
    w1, w2 = np.concatenate([np.eye(3), np.eye(3)])[None], np.eye(3)[None]
    out, _ = O.moe_layer(x, [[0.3]], 1, w1, w2, 2, True)
    assert out.tolist() == [[1.0, 0.0, 27.0]]
