"""Host-only: the MXFP4 operators refuse tensors that lie on different devices, and
take outputs left out from the pool of the call's stream. Fake tensors stand for
device ones: a refusal comes before any memory is touched."""
import pytest

import gemv_nibble_unpack_amd as G

torch = pytest.importorskip("torch")
fake = pytest.importorskip("torch._subclasses.fake_tensor")

F16, F32, U8 = torch.float16, torch.float32, torch.uint8
N, K = 32, 64
PACKED = G.prepack_mx4_bytes(N, K)
A16 = {"A": ((3, K), F16), "Wp": ((PACKED,), U8), "bias": ((N,), F16), "ws": ((1 << 20,), U8), "C": ((3, N), F16)}
A8 = {"A": ((3, K), U8), "s": ((3,), F32), **{k: A16[k] for k in ("Wp", "bias", "ws", "C")}}
A4 = {"A": ((3, K // 2), U8), "s": ((3, K // 32), U8), **{k: A16[k] for k in ("Wp", "bias", "ws", "C")}}
QUANT = {"x": ((3, K), F16), "codes": ((3, K // 2), U8), "scales": ((3, K // 32), U8)}
DEQUANT = {"codes": ((3, K // 2), U8), "scales": ((3, K // 32), U8), "out": ((3, K), F16)}
H, I, E = 64, 32, 4
MOE = {"x": ((3, H), F16), "logits": ((3, E), F32), "w1": ((G.prepack_mx4_bytes(E * 2 * I, H),), U8),
       "w2": ((G.prepack_mx4_bytes(E * H, I),), U8), "ws": ((1 << 20,), U8), "out": ((3, H), F16)}


def mixed(spec, where):
    """The tensors of `spec` on cuda:0, the one called `where` on cuda:1."""
    with fake.FakeTensorMode():
        return {n: torch.empty(*s, dtype=d, device="cuda:1" if n == where else "cuda:0") for n, (s, d) in spec.items()}


CALLS = {
    "a16": (A16, lambda t: G.mx4a16_gemm(t["A"], t["Wp"], N, bias=t["bias"], workspace=t["ws"], C=t["C"])),
    "a8": (A8, lambda t: G.mx4a8_gemm(t["A"], t["s"], t["Wp"], N, bias=t["bias"], workspace=t["ws"], C=t["C"])),
    "a4": (A4, lambda t: G.mx4a4_gemm(t["A"], t["s"], t["Wp"], N, bias=t["bias"], workspace=t["ws"], C=t["C"])),
    "quantize": (QUANT, lambda t: G.quantize_mx4(t["x"], out=(t["codes"], t["scales"]))),
    "dequantize": (DEQUANT, lambda t: G.dequantize_mx4(t["codes"], t["scales"], out=t["out"])),
    "moe": (MOE, lambda t: G.moe_mx4(t["x"], t["logits"], 2, t["w1"], t["w2"], I, workspace=t["ws"], out=t["out"])),
}


@pytest.mark.parametrize("name,where", [(n, w) for n, (spec, _) in CALLS.items() for w in list(spec)[1:]])
def test_one_device(name, where):
    spec, call = CALLS[name]
    with pytest.raises(ValueError, match="one device"):
        call(mixed(spec, where))


def test_prepack_one_device():
    t = mixed(DEQUANT, "scales")
    with pytest.raises(ValueError, match="one device"):
        G.prepack_mx4(t["codes"], t["scales"])


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_left_out_come_from_the_pool_of_the_call_s_stream(name, monkeypatch):
    from gemv_nibble_unpack_amd import mx
    spec, _ = CALLS[name]
    t = mixed(spec, None)
    stream = type("Stream", (), {"cuda_stream": 5})()
    made = []

    def empty(shape, dtype, dev, s):
        assert s is stream
        made.append(tuple(shape))
        return "made"

    class Bind:
        def __getattr__(self, _):
            return lambda *a: a
    monkeypatch.setattr(mx, "_empty", empty)
    monkeypatch.setattr(mx, "_bind", lambda: Bind())
    call = {"a16": lambda: G.mx4a16_gemm(t["A"], t["Wp"], N, workspace=t["ws"], stream=stream),
            "a8": lambda: G.mx4a8_gemm(t["A"], t["s"], t["Wp"], N, workspace=t["ws"], stream=stream),
            "a4": lambda: G.mx4a4_gemm(t["A"], t["s"], t["Wp"], N, workspace=t["ws"], stream=stream),
            "quantize": lambda: G.quantize_mx4(t["x"], stream=stream),
            "dequantize": lambda: G.dequantize_mx4(t["codes"], t["scales"], stream=stream),
            "moe": lambda: G.moe_mx4(t["x"], t["logits"], 2, t["w1"], t["w2"], I, workspace=t["ws"], stream=stream)}
    args = call[name]()
    want = {"a16": [(3, N)], "a8": [(3, N)], "a4": [(3, N)], "quantize": [(3, K // 2), (3, K // 32)],
            "dequantize": [(3, K)], "moe": [(3, H)]}
    plain = [a for a in args if isinstance(a, (int, str))]
    assert made == want[name] and plain.count("made") == len(made) and 5 in plain
