"""Host-only checks of the decoder-layer operators: header, library and binding
agree, bad arguments are rejected before a launch, the oracle's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import gemv_nibble_unpack_amd as G
import oracle as O
from gemv_nibble_unpack_amd import _lib as L

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include",
                      "gemv_nibble_unpack_layer.h")
P = ctypes.c_void_p(0x7F0000000000)
MIS = ctypes.c_void_p(0x7F0000000002)


def test_header_and_library_agree():
    text = open(HEADER).read()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", code, flags=re.M))
    assert names == set(L.LAYER_SIGNATURES)
    for n in names:
        assert hasattr(G.load(), n) and hasattr(G, n), n
    for name in ("W4_Q_I8", "W4_Q_F8", "W4_ROPE_HALF", "W4_ROPE_INTERLEAVED", "W4_MAX_HEAD_DIM"):
        m = re.search(rf"#define\s+{name}\s+(\d+)", text)
        assert int(m.group(1)) == getattr(L, name) == getattr(G, name), name
    assert L.W4_ATTN_WORKSPACE_MAX == 64 << 20


def test_norm_refusals():
    f = G.load().add_rmsnorm_q8
    ok = [P, None, P, 0, 2, 64, 1e-5, 0, None, P, P, None]

    def call(**at):
        a = list(ok)
        for k, v in at.items():
            a[int(k[1:])] = v
        return f(*a)
    assert call(_0=None) == L.W4_ERR_NULL and call(_2=None) == L.W4_ERR_NULL
    assert call(_9=None) == L.W4_ERR_NULL and call(_10=None) == L.W4_ERR_NULL
    assert call(_3=2) == L.W4_ERR_ARG and call(_7=2) == L.W4_ERR_ARG
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(_6=eps) == L.W4_ERR_ARG
    for K in (0, 4, 12, L.W4_MAX_K + 8, -8):
        assert call(_5=K) == L.W4_ERR_SHAPE
    assert call(_4=-1) == L.W4_ERR_SHAPE
    for i in (0, 1, 2, 8, 9, 10):
        assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, i
    assert call(_4=0, _0=None) == L.W4_OK


#               q  k  v  dt qs   ks   vs   rope rows rot st ip    len tab B  T  mq col Hq Hkv D  page pages kind
APPEND = [P, P, P, 0, 512, 512, 512, P, 99, 64, 0, None, P, P, 2, 2, 1, 4, 8, 4, 64, 16, 9, 0,
          P, P, P, P, P, None]


def test_append_refusals():
    f = G.load().rope_append_kv8

    def call(**at):
        a = list(APPEND)
        for k, v in at.items():
            a[int(k[1:])] = v
        return f(*a)
    for i in (1, 2, 7, 12, 13, 24, 25, 26, 27, 28):
        assert call(**{f"_{i}": None}) == L.W4_ERR_NULL, i
    for i, v in ((3, 2), (10, 2), (23, 5)):
        assert call(**{f"_{i}": v}) == L.W4_ERR_ARG, i
    for i, v in ((4, 500), (5, 255), (6, 258), (8, 0), (9, 6), (9, 68), (9, -4), (14, -1), (15, 3),
                 (16, -1), (17, 0), (18, 6), (19, 0), (20, 6), (20, 260), (21, 8), (21, 48), (22, 0)):
        assert call(**{f"_{i}": v}) == L.W4_ERR_SHAPE, (i, v)
    for i in (0, 1, 2, 7, 24, 25):
        assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, i
    assert call(_28=MIS) == L.W4_ERR_ALIGN
    assert call(_14=0, _15=0, _1=None) == L.W4_OK
    assert call(_16=0) == L.W4_OK


#       q  qs   kc vc ks vs ip    len tab B  T  mq mkv col Hq Hkv D  page pages kind scale out lse ws nb
ATTN = [P, 512, P, P, P, P, None, P, P, 2, 2, 1, 64, 4, 8, 4, 64, 16, 9, 0, 0.125, P, None, None, 0,
        None]


def test_attention_refusals():
    f = G.load().paged_attn_kv8

    def call(**at):
        a = list(ATTN)
        for k, v in at.items():
            a[int(k[1:])] = v
        return f(*a)
    for i in (0, 2, 3, 4, 5, 7, 8, 21):
        assert call(**{f"_{i}": None}) == L.W4_ERR_NULL, i
    for i, v in ((19, 2), (20, float("nan")), (20, float("inf"))):
        assert call(**{f"_{i}": v}) == L.W4_ERR_ARG, i
    for i, v in ((1, 500), (1, 514), (9, -1), (10, 3), (11, -1), (12, -1), (12, (1 << 30) + 1), (13, 0),
                 (14, 6), (15, 0), (16, 6), (16, 260), (17, 24), (17, 256), (18, 0)):
        assert call(**{f"_{i}": v}) == L.W4_ERR_SHAPE, (i, v)
    for i in (0, 2, 3, 4, 21, 23):
        assert call(**{f"_{i}": MIS}) == L.W4_ERR_ALIGN, i
    assert call(_9=0, _10=0, _0=None) == L.W4_OK
    assert call(_11=0) == L.W4_OK
    assert call(_12=1 << 20) == L.W4_ERR_WORKSPACE
    assert call(_12=1 << 20, _23=P, _24=4096) == L.W4_ERR_WORKSPACE


def test_workspace_sizes():
    f = G.paged_attn_kv8_workspace_bytes
    assert f(1, 1, 1, 64, 8, 8, 128) == 0                  # one block a head: nothing to join
    assert f(1, 1, 1, 131072, 32, 8, 128) > 16384
    assert f(1, 1, 1, 131072, 32, 7, 128) == 0             # invalid
    for B in (1, 2, 3, 7, 31, 127, 255, 256, 700, 1023, 2000, 5000):
        for Hq, Hkv in ((1, 1), (8, 8), (32, 8), (40, 1), (32, 32)):
            for D in (64, 128, 256):
                for mq in (1, 2, 5, 64, 2048):
                    for kv in (1, 300, 4096, 131072, 1 << 30):
                        assert f(B, B * mq, mq, kv, Hq, Hkv, D) <= L.W4_ATTN_WORKSPACE_MAX


def test_padded_dims():
    want = {4: 64, 64: 64, 68: 96, 96: 96, 100: 128, 128: 128, 132: 192, 192: 192, 196: 256, 256: 256,
            0: 0, 6: 0, 260: 0, -4: 0}
    for d, p in want.items():
        assert G.kv8_padded_dim(d) == p
    with pytest.raises(G.W4Error):
        G.kv8_alloc(1, 16, 1, 300, device="cpu")


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        G.add_rmsnorm_q8(torch.zeros(2, 64), torch.zeros(64))
    c = G.kv8_alloc(2, 16, 2, 64, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        G.rope_append_kv8(x, x, x, *c, i[None], i)
    with pytest.raises(ValueError):
        G.paged_attn_kv8(x, *c, i[None], i, 16)


# ------------------------------------------------------------------ the oracle's pins
def test_scale_rules():
    assert O.code_scale(254.0, 0) == np.float32(2.0) and O.code_scale(0.0, 0) == 0
    for k in range(-20, 20):
        assert O.code_scale(448.0 * 2.0 ** k, 1) == 2.0 ** k
        assert O.code_scale(449.0 * 2.0 ** k, 1) == 2.0 ** (k + 1)
        assert O.code_scale(225.0 * 2.0 ** k, 1) == 2.0 ** k
    assert O.code_scale(1e-44, 1) == np.float32(2.0 ** -126)
    assert np.isnan(O.code_scale(np.inf, 0)) and np.isnan(O.code_scale(np.nan, 1))


@pytest.mark.parametrize("kind", [0, 1])
def test_oracle_cache_holds_what_was_appended(kind):
    rng = np.random.default_rng(0)
    c = O.PagedCache8(4, 16, 2, 8, 64, kind)
    rows = rng.standard_normal((40, 2, 8)).astype(np.float32) * np.linspace(1, 6, 40)[:, None, None]
    rows = rows.astype(np.float32)
    table = [2, 0, 3]
    at = 0
    for n in (5, 1, 1, 20, 1, 12):
        c.append((rows[at:at + n], -rows[at:at + n]), table, at)
        at += n
    for h in range(2):
        k, v = c.rows(0, table, 40, h), c.rows(1, table, 40, h)
        s = np.repeat(c.scale[0][table, h], 16)[:40, None]
        # half a step when written and half a step for each re-coding of the page
        step = 1.0 if kind == 0 else np.maximum(np.abs(rows[:, h]) / s, 2.0 ** -6) / 8
        assert np.all(np.abs(k - rows[:, h]) <= (0.5 * 6 if kind == 0 else 0.6) * step * s)
        assert np.array_equal(k, -v)


def test_oracle_rope_turns_pairs():
    x = np.arange(8, dtype=np.float32)[None, None]
    tab = np.array([[0.0, 0.0, 1.0, 1.0]], np.float32)      # a quarter turn of two pairs
    assert O.rope_f32(x, tab, [0], 4, 0)[0, 0].tolist() == [-2, -3, 0, 1, 4, 5, 6, 7]
    assert O.rope_f32(x, tab, [0], 4, 1)[0, 0].tolist() == [-1, 0, -3, 2, 4, 5, 6, 7]


def test_oracle_attention_closed_forms():
    k = np.zeros((5, 4))
    v = np.arange(20.0).reshape(5, 4)
    q = np.ones((3, 4), np.float16)
    out, lse, absv, _ = O.attention_rows(q, k, v, [5, 2, 0], 0.5)
    assert np.allclose(out[0], v.mean(0)) and np.allclose(out[1], v[:2].mean(0)) and not out[2].any()
    assert np.allclose(lse[:2], np.log([5, 2])) and np.isneginf(lse[2])
    # one dominating key
    k[3] = 100
    assert np.allclose(O.attention_rows(q[:1], k, v, [5], 0.5)[0], v[3])
