"""torch-tensor wrappers of the decoder-layer operators (marshalling only; the
semantics are in ``include/gemv_nibble_unpack_layer.h``)."""
from __future__ import annotations

import torch

from . import _lib as L
from .api import Workspace, _dev, _empty, _ptr

_IN = {torch.float16: L.W4_IN_F16, torch.float32: L.W4_IN_F32}
_CODES = {torch.int8: L.W4_Q_I8, torch.uint8: L.W4_Q_F8}


def _raw_stream(stream):
    """The HIP stream a call runs on (None: the current torch stream)."""
    return torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream


def _new(shape, dtype, dev, stream):
    if stream is None:          # the current stream's pool: torch's default
        return torch.empty(shape, dtype=dtype, device=dev)
    return _empty(shape, dtype, dev, stream)


def _in_dtype(t, name):
    dt = _IN.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float16 or float32")
    return dt


def add_rmsnorm_q8(x, weight, residual=None, eps=1e-5, q_dtype=L.W4_Q_I8, residual_out=None,
                   out=None, stream=None):
    """fp16/float32 x [M,K] (+ residual) -> (codes [M,K] int8 or uint8 E4M3, scales
    float32 [M], the residual sum [M,K]). Without a residual the sum is x itself
    and is returned as given. ``residual_out`` may be x or residual; ``out`` is a
    (codes, scales) pair to write into."""
    dev = _dev(x)
    M, K = x.shape
    dt = _in_dtype(x, "x")
    _dev(weight)
    if weight.dtype != x.dtype or weight.numel() != K:
        raise ValueError("weight must be [K] of x's type")
    if residual is not None:
        _dev(residual)
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ValueError("residual must have x's shape and type")
        if residual_out is None:
            residual_out = _new((M, K), x.dtype, dev, stream)
    if residual_out is not None:
        _dev(residual_out)
        if residual_out.dtype != x.dtype or residual_out.shape != x.shape:
            raise ValueError("residual_out must have x's shape and type")
    if out is None:
        codes = _new((M, K), torch.int8 if q_dtype == L.W4_Q_I8 else torch.uint8, dev, stream)
        scales = _new((M,), torch.float32, dev, stream)
    else:
        codes, scales = out
        _dev(codes), _dev(scales)
        if (codes.shape != x.shape or codes.element_size() != 1 or scales.dtype != torch.float32
                or scales.numel() != M):
            raise ValueError("out must be ([M,K] one-byte codes, float32 [M])")
    L.check("add_rmsnorm_q8", L.load().add_rmsnorm_q8(
        x.data_ptr(), _ptr(residual), weight.data_ptr(), dt, M, K, eps, q_dtype, _ptr(residual_out),
        codes.data_ptr(), scales.data_ptr(), _raw_stream(stream)))
    return codes, scales, x if residual_out is None else residual_out


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


def _cache(kc, vc, ks, vs, kv_heads, head_dim):
    """(pages, page size, code kind) of a cache, checked against the heads."""
    pages, heads, page, dp = kc.shape
    kind = _CODES.get(kc.dtype)
    if kind is None or vc.dtype != kc.dtype:
        raise ValueError("cache codes must be int8 (INT8) or uint8 (E4M3), keys and values alike")
    if heads != kv_heads or dp != kv8_padded_dim(head_dim) or vc.shape != (pages, heads, dp, page):
        raise ValueError("cache shapes do not match the heads: keys [pages, heads, page, DP], "
                         "values [pages, heads, DP, page]")
    if ks.shape != (pages, heads) or vs.shape != (pages, heads) or \
            ks.dtype != torch.float32 or vs.dtype != torch.float32:
        raise ValueError("cache scales must be float32 [pages, heads]")
    if not (kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous() and kc.is_cuda and vc.is_cuda and ks.is_cuda and vs.is_cuda):
        raise ValueError("expected contiguous device tensors")
    return pages, page, kind


def _batch(page_table, kv_len, q_indptr):
    B = kv_len.shape[0]
    if page_table.dtype != torch.int32 or kv_len.dtype != torch.int32 or \
            (q_indptr is not None and (q_indptr.dtype != torch.int32
                                       or q_indptr.shape != (B + 1,))):
        raise ValueError("page_table, kv_len [batch] and q_indptr [batch + 1] must be int32")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [batch, columns]")
    if not (page_table.is_contiguous() and kv_len.is_contiguous() and page_table.is_cuda
            and kv_len.is_cuda) or (q_indptr is not None and not (q_indptr.is_contiguous()
                                                                  and q_indptr.is_cuda)):
        raise ValueError("expected contiguous device tensors")
    return B, page_table.shape[1]


def _token_stride(t, name):
    """Elements between tokens of [tokens, heads, dim] whose heads are dense."""
    s = t.stride()
    if t.dim() != 3 or s[2] != 1 or (s[1] != t.shape[2] and t.shape[1] > 1) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor [tokens, heads, dim] with dense heads")
    return s[0] if t.shape[0] > 1 else max(s[0], t.shape[1] * t.shape[2])


def rope_append_kv8(q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, q_indptr=None,
                    max_q=1, rope=None, style=L.W4_ROPE_HALF, q_out=None, stream=None):
    """Rotate the new q [T,Hq,D] and k [T,Hkv,D] by their positions and write k
    and v [T,Hkv,D] into the 8-bit cache; returns the rotated q as fp16 [T,Hq,D]
    (None for q None). Tokens may be strided (slices of a fused projection).
    ``rope`` is float32 [positions, rot_dim] (cosines, then sines) or None;
    ``kv_len`` counts the new tokens; ``q_indptr`` None: one token a sequence."""
    T, Hkv, D = k.shape
    dt = _in_dtype(k, "k")
    pages, page, kind = _cache(k_cache, v_cache, k_scale, v_scale, Hkv, D)
    B, cols = _batch(page_table, kv_len, q_indptr)
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must have one shape and type")
    Hq, qs = Hkv, 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != D or q.dtype != k.dtype:
            raise ValueError("q must be [tokens, q_heads, dim] of k's type")
        Hq, qs = q.shape[1], _token_stride(q, "q")
        if q_out is None:
            q_out = _new((T, Hq, D), torch.float16, q.device, stream)
        elif q_out.shape != q.shape or q_out.dtype != torch.float16 or not q_out.is_contiguous() \
                or not q_out.is_cuda:
            raise ValueError("q_out must be a dense float16 device tensor of q's shape")
    rows = rot = 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 2:
            raise ValueError("rope must be float32 [positions, rot_dim]")
        _dev(rope)
        rows, rot = rope.shape
    L.check("rope_append_kv8", L.load().rope_append_kv8(
        _ptr(q), k.data_ptr(), v.data_ptr(), dt, qs, _token_stride(k, "k"), _token_stride(v, "v"),
        _ptr(rope), rows, rot, style, _ptr(q_indptr), kv_len.data_ptr(), page_table.data_ptr(),
        B, T, max_q, cols, Hq, Hkv, D, page, pages, kind, k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), None if q is None else q_out.data_ptr(),
        _raw_stream(stream)))
    return q_out if q is not None else None


def paged_attn_kv8_workspace_bytes(batch, tokens, max_q, max_kv, q_heads, kv_heads, head_dim):
    """Workspace bytes of a paged_attn_kv8 call with these sizes."""
    return int(L.load().paged_attn_kv8_workspace_bytes(batch, tokens, max_q, max_kv, q_heads,
                                                       kv_heads, head_dim))


def paged_attn_kv8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, max_kv, q_indptr=None,
                   max_q=1, scale=None, lse=None, workspace=None, out=None, stream=None):
    """Causal attention of the new tokens q fp16 [T,Hq,D] over the 8-bit cache ->
    fp16 [T,Hq,D]. ``scale`` defaults to D**-0.5; ``lse`` is an optional float32
    [T,Hq] output; ``workspace`` a Workspace or a zeroed uint8 device tensor."""
    T, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    if q.dtype != torch.float16:
        raise ValueError("q must be float16")
    pages, page, kind = _cache(k_cache, v_cache, k_scale, v_scale, Hkv, D)
    B, cols = _batch(page_table, kv_len, q_indptr)
    if out is None:
        out = _new((T, Hq, D), torch.float16, q.device, stream)
    elif out.shape != q.shape or out.dtype != torch.float16 or not out.is_contiguous() \
            or not out.is_cuda:
        raise ValueError("out must be a dense float16 device tensor of q's shape")
    if lse is not None and (lse.shape != (T, Hq) or lse.dtype != torch.float32
                            or not lse.is_contiguous() or not lse.is_cuda):
        raise ValueError("lse must be a dense float32 device tensor [tokens, q_heads]")
    lib = L.load()
    buf, nb = None, 0
    if workspace is None or isinstance(workspace, Workspace):
        need = int(lib.paged_attn_kv8_workspace_bytes(B, T, max_q, max_kv, Hq, Hkv, D))
        if need:
            buf = (workspace or Workspace(q.device)).get(need, stream)
            nb = buf.numel()
    else:
        buf, nb = workspace, workspace.numel() * workspace.element_size()
    L.check("paged_attn_kv8", lib.paged_attn_kv8(
        q.data_ptr(), _token_stride(q, "q"), k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), _ptr(q_indptr), kv_len.data_ptr(),
        page_table.data_ptr(), B, T, max_q, max_kv, cols, Hq, Hkv, D, page, pages, kind,
        D ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse), _ptr(buf), nb,
        _raw_stream(stream)))
    return out
