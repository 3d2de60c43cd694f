"""Host-only: the layer operators refuse tensors that lie on different devices. Fake
tensors stand for device ones: a refusal comes before any memory is touched."""
import pytest

import gemv_nibble_unpack_amd as G

torch = pytest.importorskip("torch")
fake = pytest.importorskip("torch._subclasses.fake_tensor")


def mixed(names, where, spec):
    """The tensors of `spec` on cuda:0, the one called `where` on cuda:1."""
    with fake.FakeTensorMode():
        return {n: torch.empty(*spec[n][0], dtype=spec[n][1], device="cuda:1" if n == where else "cuda:0")
                for n in names}


F16, F32, I8, I32 = torch.float16, torch.float32, torch.int8, torch.int32
CACHE = {"kc": ((4, 2, 16, 64), I8), "vc": ((4, 2, 64, 16), I8), "ks": ((4, 2), F32), "vs": ((4, 2), F32),
         "table": ((1, 2), I32), "len": ((1,), I32), "indptr": ((2,), I32)}
NORM = {"x": ((2, 64), F16), "w": ((64,), F16), "r": ((2, 64), F16), "ro": ((2, 64), F16),
        "codes": ((2, 64), I8), "scale": ((2,), F32)}
APPEND = {"k": ((3, 2, 64), F16), "q": ((3, 4, 64), F16), "v": ((3, 2, 64), F16), **CACHE,
          "rope": ((40, 64), F32), "q_out": ((3, 4, 64), F16)}
ATTN = {"q": ((3, 4, 64), F16), **CACHE, "lse": ((3, 4), F32), "ws": ((1 << 20,), torch.uint8),
        "out": ((3, 4, 64), F16)}


def refuses(call):
    with pytest.raises(ValueError, match="one device"):
        call()


@pytest.mark.parametrize("where", list(NORM)[1:])
def test_norm(where):
    t = mixed(NORM, where, NORM)
    refuses(lambda: G.add_rmsnorm_q8(t["x"], t["w"], t["r"], residual_out=t["ro"], out=(t["codes"], t["scale"])))


@pytest.mark.parametrize("where", list(APPEND)[1:])
def test_append(where):
    t = mixed(APPEND, where, APPEND)
    refuses(lambda: G.rope_append_kv8(t["q"], t["k"], t["v"], t["kc"], t["vc"], t["ks"], t["vs"], t["table"],
                                      t["len"], q_indptr=t["indptr"], max_q=3, rope=t["rope"], q_out=t["q_out"]))


@pytest.mark.parametrize("where", list(ATTN)[1:])
def test_attention(where):
    t = mixed(ATTN, where, ATTN)
    refuses(lambda: G.paged_attn_kv8(t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["table"], t["len"], 32,
                                     q_indptr=t["indptr"], max_q=3, lse=t["lse"], workspace=t["ws"],
                                     out=t["out"]))


@pytest.mark.parametrize("given", ["codes", "scale", "both", "none"])
def test_norm_outputs_left_out_come_from_the_pool_of_the_call_s_stream(given, monkeypatch):
    from gemv_nibble_unpack_amd import layer
    t = mixed(NORM, None, NORM)
    stream = type("Stream", (), {"cuda_stream": 5})()
    seen = {}

    class Bind:
        @staticmethod
        def add_rmsnorm_q8(x, w, r, eps, kind, ro, codes, scales, raw):
            seen.update(codes=codes, scales=scales, ro=ro, raw=raw)
            return codes, scales, ro
    monkeypatch.setattr(layer, "_BIND", Bind)
    monkeypatch.setattr(layer, "_empty", lambda shape, dtype, dev, s: ("made", tuple(shape) if shape != 2 else 2,
                                                                       dtype, s))
    out = {"codes": (t["codes"], None), "scale": (None, t["scale"]), "both": (t["codes"], t["scale"]),
           "none": None}[given]
    layer.add_rmsnorm_q8(t["x"], t["w"], t["r"], out=out, stream=stream)
    assert seen["raw"] == 5 and seen["ro"] == ("made", (2, 64), F16, stream)
    assert seen["codes"] is t["codes"] if given in ("codes", "both") else seen["codes"] == \
        ("made", (2, 64), I8, stream)
    assert seen["scales"] is t["scale"] if given in ("scale", "both") else seen["scales"] == \
        ("made", 2, F32, stream)
