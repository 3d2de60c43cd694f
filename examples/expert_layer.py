"""One decoder layer with MXFP4 weights and a mixture of experts.

    python examples/expert_layer.py [--hidden 4096 --heads 32 --kv-heads 8 --experts 64 --top-k 4]

The layer of decoder_layer.py with other products (random weights, an FP8 paged cache):

    residual += previous output;  rows = E4M3(norm(residual))     add_rmsnorm_q8
    qkv       = rows x Wqkv                                       mx4a8_gemm
    q, cache  = rotated queries, keys and values appended         rope_append_kv8
    o         = attention of the new tokens over the cache        paged_attn_kv8
    out       = MXFP4(o) x Wo                                     quantize_mx4, mx4a4_gemm
    residual += out;  x = norm(residual), fp16                    (torch)
    logits    = x x Wr, float32                                   mx4a16_gemm
    output    = the chosen experts' weighted sum                  moe_mx4, 64 tokens at a time
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_nibble_unpack_amd as G  # noqa: E402


class ExpertLayer:
    def __init__(self, hidden, heads, kv_heads, inner, experts, top_k, max_tokens, page=64, seed=0):
        self.hidden, self.heads, self.kv_heads = hidden, heads, kv_heads
        self.inner, self.experts, self.top_k = inner, experts, top_k
        self.dim = hidden // heads
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5
            return G.prepack_mx4(*G.quantize_mx4(w))

        self.qkv_rows = (heads + 2 * kv_heads) * self.dim
        self.qkv, self.o, self.router = weight(self.qkv_rows, hidden), weight(hidden, hidden), weight(experts, hidden)
        self.gate_up, self.down = weight(experts * 2 * inner, hidden), weight(experts * hidden, inner)
        self.norm1, self.norm2 = (
            (1 + 0.1 * torch.randn(hidden, device="cuda", generator=gen)).half() for _ in range(2))
        half = self.dim // 2
        angle = torch.arange(max_tokens, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        columns = -(-max_tokens // page)
        self.cache = G.kv8_alloc(columns, page, kv_heads, self.dim, G.W4_Q_F8)
        self.table = torch.arange(columns, dtype=torch.int32, device="cuda").view(1, columns)
        self.max_tokens = max_tokens
        self.workspace = G.Workspace()

    def mlp(self, x):
        """x fp16 [tokens, hidden] through the router and its experts."""
        logits = G.mx4a16_gemm(x, self.router, self.experts, out_dtype=G.W4_OUT_F32, workspace=self.workspace)
        out = torch.empty_like(x)
        for t in range(0, x.shape[0], 64):
            G.moe_mx4(x[t:t + 64], logits[t:t + 64], self.top_k, self.gate_up, self.down, self.inner,
                      workspace=self.workspace, out=out[t:t + 64])
        return out

    def forward(self, x, residual, kv_len, q_indptr=None, max_q=1):
        """x [tokens, hidden] fp16 and the residual stream, which is updated in place;
        kv_len counts the new tokens. Returns the layer's output [tokens, hidden]."""
        rows, scale, _ = G.add_rmsnorm_q8(x, self.norm1, residual, q_dtype=G.W4_Q_F8, residual_out=residual)
        qkv = G.mx4a8_gemm(rows, scale, self.qkv, self.qkv_rows, workspace=self.workspace)
        q, k, v = qkv.view(x.shape[0], -1, self.dim).split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = G.rope_append_kv8(q, k, v, *self.cache, self.table, kv_len, q_indptr=q_indptr, max_q=max_q,
                              rope=self.rope)
        o = G.paged_attn_kv8(q, *self.cache, self.table, kv_len, self.max_tokens, q_indptr=q_indptr,
                             max_q=max_q, workspace=self.workspace)
        codes, scales = G.quantize_mx4(o.view(x.shape[0], self.hidden))
        residual.add_(G.mx4a4_gemm(codes, scales, self.o, self.hidden, workspace=self.workspace))
        h = residual.float()
        h = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-5) * self.norm2
        return self.mlp(h.half())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--inner", type=int, default=1536)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    layer = ExpertLayer(a.hidden, a.heads, a.kv_heads, a.inner, a.experts, a.top_k, a.prompt + a.tokens)
    x = torch.randn(a.prompt, a.hidden, device="cuda", dtype=torch.float16)
    kv_len = torch.tensor([a.prompt], dtype=torch.int32, device="cuda")
    y = layer.forward(x, torch.zeros_like(x), kv_len,
                      torch.tensor([0, a.prompt], dtype=torch.int32, device="cuda"), a.prompt)
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
