"""One decoder layer on the low-bit products and the operators between them.

    python examples/decoder_layer.py [--hidden 4096 --heads 32 --kv-heads 8 --prompt 500 --tokens 64]

INT4 weights, INT8 activations and an INT8 paged KV cache; random weights. A
prompt goes through the layer in one call, then tokens one at a time, each
decode step replayed as one graph (lengths advance on the device). The layer:

    residual += previous output;  rows = INT8(norm(residual))     add_rmsnorm_q8
    qkv       = rows x Wqkv                                       w4a8_gemm
    q, cache  = rotated queries, keys and values appended         rope_append_kv8
    o         = attention of the new tokens over the cache        paged_attn_kv8
    out       = INT8(o) x Wo                                      w4a8_gemm_fused_act
    residual += out;  rows = INT8(norm(residual))                 add_rmsnorm_q8
    gate, up  = rows x Wgu                                        w4a8_gemm
    output    = INT8(relu(gate)^2 * up) x Wd                      w4a8_gemm_fused_act
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_nibble_unpack_amd as G  # noqa: E402


class DecoderLayer:
    def __init__(self, hidden, heads, kv_heads, inner, max_tokens, sequences=1, page=64, seed=0):
        self.hidden, self.heads, self.kv_heads = hidden, heads, kv_heads
        self.dim = hidden // heads
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5
            codes, scale, _ = G.quantize_pack_w4(w)
            return G.prepack_w(G.W4_LAYOUT_W4A8, codes, n, k), scale, n

        self.qkv = weight((heads + 2 * kv_heads) * self.dim, hidden)
        self.o, self.gate_up, self.down = weight(hidden, hidden), weight(2 * inner, hidden), weight(hidden, inner)
        self.norm1, self.norm2 = (
            (1 + 0.1 * torch.randn(hidden, device="cuda", generator=gen)).half() for _ in range(2))
        # angles in float64; a long context would stretch the positions here
        half = self.dim // 2
        angle = torch.arange(max_tokens, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        columns = -(-max_tokens // page)
        self.cache = G.kv8_alloc(columns * sequences, page, kv_heads, self.dim)
        self.table = torch.arange(columns * sequences, dtype=torch.int32, device="cuda").view(sequences, columns)
        self.max_tokens = max_tokens
        self.workspace = G.Workspace()

    def _rows(self, rows, scale, w):
        return G.w4a8_gemm(rows, scale, w[0], w[1], w[2], workspace=self.workspace)

    def _float_rows(self, x, w):
        return G.w4a8_gemm_fused_act(x, w[0], w[1], w[2], workspace=self.workspace)

    def forward(self, x, residual, kv_len, q_indptr=None, max_q=1):
        """x [tokens, hidden] fp16 and the residual stream, which is updated in place;
        kv_len counts the new tokens. Returns the layer's output [tokens, hidden]."""
        rows, scale, _ = G.add_rmsnorm_q8(x, self.norm1, residual, residual_out=residual)
        qkv = self._rows(rows, scale, self.qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = G.rope_append_kv8(q, k, v, *self.cache, self.table, kv_len, q_indptr=q_indptr, max_q=max_q,
                              rope=self.rope)
        o = G.paged_attn_kv8(q, *self.cache, self.table, kv_len, self.max_tokens, q_indptr=q_indptr,
                             max_q=max_q, workspace=self.workspace)
        out = self._float_rows(o.view(x.shape[0], self.hidden), self.o)
        rows, scale, _ = G.add_rmsnorm_q8(out, self.norm2, residual, residual_out=residual)
        gate, up = self._rows(rows, scale, self.gate_up).chunk(2, 1)
        return self._float_rows((torch.relu(gate).square() * up).contiguous(), self.down)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--inner", type=int, default=11008)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    layer = DecoderLayer(a.hidden, a.heads, a.kv_heads, a.inner, a.prompt + a.tokens)
    x = torch.randn(a.prompt, a.hidden, device="cuda", dtype=torch.float16)
    res = torch.zeros_like(x)
    kv_len = torch.tensor([a.prompt], dtype=torch.int32, device="cuda")
    y = layer.forward(x, res, kv_len, torch.tensor([0, a.prompt], dtype=torch.int32, device="cuda"), a.prompt)
    torch.cuda.synchronize()
    print(f"prompt of {a.prompt}: output rms {y.float().square().mean().sqrt().item():.3f}", flush=True)

    # decode steps: one token in, the layer's output fed back, as a replayed graph
    x1, r1 = y[-1:].clone(), torch.zeros(1, a.hidden, dtype=torch.float16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        kv_len.add_(1)
        layer.forward(x1, r1.clone(), kv_len)          # allocates, outside the capture
        kv_len.sub_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        kv_len.add_(1)
        r1.zero_()
        x1.copy_(layer.forward(x1, r1, kv_len))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    for _ in range(a.tokens):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert int(kv_len) == a.prompt + a.tokens and bool(torch.isfinite(x1).all())
    print(f"{a.tokens} tokens: {begin.elapsed_time(end) / a.tokens * 1e3:.1f} us a token and layer", flush=True)


if __name__ == "__main__":
    main()
