"""GPU: the layer with MXFP4 weights and experts runs, and its tokens taken one at a
time in a graph are those of eager steps, bit for bit."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer
    yield expert_layer
    sys.path.pop(0)


def test_example_runs(example, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["expert_layer.py", "--hidden", "512", "--heads", "8", "--kv-heads", "2",
                                      "--inner", "160", "--experts", "6", "--top-k", "2", "--prompt", "150",
                                      "--tokens", "5"])
    example.main()
    out = capsys.readouterr().out
    assert "prompt of 150" in out and "us a token" in out


def test_graph_repeats_eager_steps(example):
    def run(graphed):
        layer = example.ExpertLayer(256, 4, 2, 96, 5, 2, 64, seed=3)
        gen = torch.Generator(device="cuda").manual_seed(4)
        x = torch.randn(1, 256, device="cuda", dtype=torch.float16, generator=gen)
        r = torch.zeros_like(x)
        kv_len = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = []

        def step():
            kv_len.add_(1)
            r.zero_()
            return layer.forward(x, r, kv_len)
        if not graphed:
            for _ in range(6):
                x.copy_(step())
                outs.append(x.clone())
            return outs
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            stream.wait_stream(torch.cuda.default_stream())
            step()                                       # allocates
            kv_len.zero_()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                x.copy_(step())
        torch.cuda.synchronize()
        for _ in range(6):
            graph.replay()
            outs.append(x.clone())
            torch.cuda.synchronize()
        return outs
    for a, b in zip(run(False), run(True)):
        assert torch.isfinite(a).all() and torch.equal(a, b)
