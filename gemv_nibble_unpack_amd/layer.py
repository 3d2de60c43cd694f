"""torch-tensor wrappers of the decoder-layer operators (marshalling only; the
semantics are in ``include/gemv_nibble_unpack_layer.h``, the checks of the
tensors in ``csrc_layer/bind.cpp``)."""
from __future__ import annotations

import torch

from . import _lib as L
from .api import Workspace, _dev, _empty

_BIND = None


def _bind():
    """The compiled marshalling module (csrc_layer/bind.cpp), loaded once."""
    global _BIND
    if _BIND is None:
        L.load()
        try:
            from . import _layer_bind
        except ImportError as e:
            raise L.LibraryMissing(
                f"the compiled module _layer_bind cannot be loaded ({e}): build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')") from e
        _BIND = _layer_bind
    return _BIND


def add_rmsnorm_q8(x, weight, residual=None, eps=1e-5, q_dtype=L.W4_Q_I8, residual_out=None,
                   out=None, stream=None):
    """fp16/float32 x [M,K] (+ residual) -> (codes [M,K] int8 or uint8 E4M3, scales
    float32 [M], the residual sum [M,K]). Without a residual the sum is x itself
    and is returned as given. ``residual_out`` may be x or residual; ``out`` is a
    (codes, scales) pair to write into."""
    codes, scales = (None, None) if out is None else out
    raw = None
    if stream is not None:      # outputs come from the pool of the call's stream
        raw = stream.cuda_stream
        if residual is not None and residual_out is None:
            residual_out = _empty(x.shape, x.dtype, _dev(x), stream)
        if codes is None:
            codes = _empty(x.shape, torch.int8 if q_dtype == L.W4_Q_I8 else torch.uint8, _dev(x),
                           stream)
        if scales is None:
            scales = _empty(x.shape[0], torch.float32, _dev(x), stream)
    r = (_BIND or _bind()).add_rmsnorm_q8(x, weight, residual, eps, q_dtype, residual_out, codes,
                                          scales, raw)
    if type(r) is int:
        L.check("add_rmsnorm_q8", r)
    return r


def kv8_padded_dim(head_dim):
    """The padded head dim of a cache, or 0 for a head_dim that is not served."""
    return int(L.load().kv8_padded_dim(head_dim))


def kv8_alloc(num_pages, page_size, kv_heads, head_dim, q_dtype=L.W4_Q_I8, device="cuda"):
    """A zeroed cache: (k_codes [pages, heads, page, DP], v_codes [pages, heads,
    DP, page], k_scale, v_scale float32 [pages, heads])."""
    dp = kv8_padded_dim(head_dim)
    if dp == 0:
        raise L.W4Error("kv8_alloc", L.W4_ERR_SHAPE)
    dt = torch.int8 if q_dtype == L.W4_Q_I8 else torch.uint8
    return (torch.zeros(num_pages, kv_heads, page_size, dp, dtype=dt, device=device),
            torch.zeros(num_pages, kv_heads, dp, page_size, dtype=dt, device=device),
            torch.zeros(num_pages, kv_heads, dtype=torch.float32, device=device),
            torch.zeros(num_pages, kv_heads, dtype=torch.float32, device=device))


def rope_append_kv8(q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, q_indptr=None,
                    max_q=1, rope=None, style=L.W4_ROPE_HALF, q_out=None, stream=None):
    """Rotate the new q [T,Hq,D] and k [T,Hkv,D] by their positions and write k
    and v [T,Hkv,D] into the 8-bit cache; returns the rotated q as fp16 [T,Hq,D]
    (None for q None). Tokens may be strided (slices of a fused projection).
    ``rope`` is float32 [positions, rot_dim] (cosines, then sines) or None;
    ``kv_len`` counts the new tokens; ``q_indptr`` None: one token a sequence."""
    raw = None
    if stream is not None:
        raw = stream.cuda_stream
        if q is not None and q_out is None:
            q_out = _empty(q.shape, torch.float16, q.device, stream)
    r = (_BIND or _bind()).rope_append_kv8(q, k, v, k_cache, v_cache, k_scale, v_scale, page_table,
                                           kv_len, q_indptr, max_q, rope, style, q_out, raw)
    if type(r) is int:
        L.check("rope_append_kv8", r)
    return r


def paged_attn_kv8_workspace_bytes(batch, tokens, max_q, max_kv, q_heads, kv_heads, head_dim):
    """Workspace bytes of a paged_attn_kv8 call with these sizes."""
    return int(L.load().paged_attn_kv8_workspace_bytes(batch, tokens, max_q, max_kv, q_heads,
                                                       kv_heads, head_dim))


def paged_attn_kv8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, max_kv, q_indptr=None,
                   max_q=1, scale=None, lse=None, workspace=None, out=None, stream=None):
    """Causal attention of the new tokens q fp16 [T,Hq,D] over the 8-bit cache ->
    fp16 [T,Hq,D]. ``scale`` defaults to D**-0.5; ``lse`` is an optional float32
    [T,Hq] output; ``workspace`` a Workspace or a zeroed uint8 device tensor."""
    if workspace is None or isinstance(workspace, Workspace):
        need = paged_attn_kv8_workspace_bytes(kv_len.shape[0], q.shape[0], max_q, max_kv, q.shape[1],
                                              k_cache.shape[1], q.shape[2])
        workspace = (workspace or Workspace(q.device)).get(need, stream) if need else None
    raw = None
    if stream is not None:
        raw = stream.cuda_stream
        if out is None:
            out = _empty(q.shape, torch.float16, q.device, stream)
    r = (_BIND or _bind()).paged_attn_kv8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len,
                                          max_kv, q_indptr, max_q, scale, lse, workspace, out, raw)
    if type(r) is int:
        L.check("paged_attn_kv8", r)
    return r
