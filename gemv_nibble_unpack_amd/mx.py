"""torch-tensor wrappers of the MXFP4 operators (marshalling only; the semantics
are in ``include/gemv_nibble_unpack_mx.h``, the checks of the tensors in
``csrc_mx/bind_mx.hpp``)."""
from __future__ import annotations

import torch

from . import _lib as L
from .api import Workspace, _dev, _empty, _ptr, _stream
from .layer import _bind


def _done(name, r):
    if type(r) is int:
        L.check(name, r)
    return r


def quantize_mx4(x, out=None, stream=None):
    """fp16/float32 x [R,K] -> (codes uint8 [R,K/2], E8M0 scales uint8 [R,K/32]);
    ``out`` is such a pair to write into."""
    codes, scales = (None, None) if out is None else out
    raw = None
    if stream is not None:
        raw = stream.cuda_stream
        if x.dim() == 2:
            R, K = x.shape
            if codes is None:
                codes = _empty((R, K // 2), torch.uint8, _dev(x), stream)
            if scales is None:
                scales = _empty((R, K // 32), torch.uint8, _dev(x), stream)
    return _done("quantize_mx4", _bind().quantize_mx4(x, codes, scales, raw))


def dequantize_mx4(codes, scales, dtype=torch.float16, out=None, stream=None):
    """MXFP4 rows -> torch.float16 or torch.float32 [R,K]."""
    if dtype not in (torch.float16, torch.float32):
        raise ValueError("dtype must be torch.float16 or torch.float32")
    raw = None
    if stream is not None:
        raw = stream.cuda_stream
        if out is None:
            out = _empty((codes.shape[0], 2 * codes.shape[1]), dtype, _dev(codes), stream)
    return _done("dequantize_mx4",
                 _bind().dequantize_mx4(codes, scales, int(dtype == torch.float32), out, raw))


def prepack_mx4_bytes(N, K):
    """Bytes of the packed weights of an [N,K] matrix (0: not served)."""
    return int(L.load().prepack_mx4_bytes(N, K))


def prepack_mx4(codes, scales, stream=None):
    """Codes [N,K/2] and scales [N,K/32] of weights -> the packed uint8 buffer that
    the products read."""
    dev = _dev(codes)
    if _dev(scales) != dev:
        raise ValueError("all tensors must be on one device")
    if (codes.dim() != 2 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or
            tuple(scales.shape) != (codes.shape[0], codes.shape[1] // 16) or codes.shape[1] % 16):
        raise ValueError("MXFP4 rows are uint8 codes [rows, K / 2] and uint8 scales [rows, K / 32]")
    N, K = codes.shape[0], 2 * codes.shape[1]
    nbytes = prepack_mx4_bytes(N, K)
    if nbytes == 0:
        raise L.W4Error("prepack_mx4", L.W4_ERR_SHAPE)
    with torch.cuda.device(dev):
        Wp = _empty(nbytes, torch.uint8, dev, stream)
        L.check("prepack_mx4", L.load().prepack_mx4(_ptr(codes), _ptr(scales), N, K, _ptr(Wp),
                                                    _stream(stream)))
    return Wp


def unprepack_mx4(Wp, N, K, stream=None):
    """Inverse of prepack_mx4 -> (codes [N,K/2], scales [N,K/32])."""
    dev = _dev(Wp)
    nbytes = prepack_mx4_bytes(N, K)
    if nbytes == 0:
        raise L.W4Error("unprepack_mx4", L.W4_ERR_SHAPE)
    if Wp.nbytes < nbytes:
        raise ValueError("Wp is not prepack_mx4's of an [N, K] matrix")
    with torch.cuda.device(dev):
        codes = _empty((N, K // 2), torch.uint8, dev, stream)
        scales = _empty((N, K // 32), torch.uint8, dev, stream)
        L.check("unprepack_mx4", L.load().unprepack_mx4(_ptr(Wp), N, K, _ptr(codes), _ptr(scales),
                                                        _stream(stream)))
    return codes, scales


def mx4_workspace_bytes(op, M, N, K):
    """Workspace bytes of a product (op W4_MX_A16, W4_MX_A8 or W4_MX_A4)."""
    return int(L.load().mx4_workspace_bytes(op, M, N, K))


_NEED = {}


def _space(key, ask, workspace, device, stream):
    """The tensor that a call's workspace is: None if it needs none."""
    if workspace is not None and not isinstance(workspace, Workspace):
        return workspace
    need = _NEED.get(key)
    if need is None:
        if len(_NEED) > 4096:
            _NEED.clear()
        need = _NEED[key] = ask(*key[1:])
    return (workspace or Workspace(device)).get(need, stream) if need else None


def _product(name, op, A, scales, Wp, N, K, bias, out_dtype, workspace, C, stream):
    M = A.shape[0]
    raw = None
    if stream is not None:
        raw = stream.cuda_stream
        if C is None:
            C = _empty((M, N), torch.float32 if out_dtype == L.W4_OUT_F32 else torch.float16, _dev(A),
                       stream)
    ws = _space(("gemm", op, M, N, K), mx4_workspace_bytes, workspace, A.device, stream)
    return _done(name, _bind().mx4_gemm(op, A, scales, Wp, N, bias, out_dtype, ws, C, raw))


def mx4a16_gemm(A, Wp, N, bias=None, out_dtype=L.W4_OUT_F16, workspace=None, C=None, stream=None):
    """fp16 A [M,K] x MXFP4 weights -> C [M,N]; ``workspace`` a Workspace or a zeroed
    uint8 device tensor."""
    return _product("mx4a16_gemm", L.W4_MX_A16, A, None, Wp, N, A.shape[-1], bias, out_dtype, workspace,
                    C, stream)


def mx4a8_gemm(Aq, a_scale, Wp, N, bias=None, out_dtype=L.W4_OUT_F16, workspace=None, C=None,
               stream=None):
    """E4M3 codes Aq [M,K] with a float32 scale a row (add_rmsnorm_q8, quantize_f8) x
    MXFP4 weights -> C [M,N]."""
    return _product("mx4a8_gemm", L.W4_MX_A8, Aq, a_scale, Wp, N, Aq.shape[-1], bias, out_dtype,
                    workspace, C, stream)


def mx4a4_gemm(Aq, a_scales, Wp, N, bias=None, out_dtype=L.W4_OUT_F16, workspace=None, C=None,
               stream=None):
    """MXFP4 rows (quantize_mx4) Aq [M,K/2], a_scales [M,K/32] x MXFP4 weights -> C [M,N]."""
    return _product("mx4a4_gemm", L.W4_MX_A4, Aq, a_scales, Wp, N, 2 * Aq.shape[-1], bias, out_dtype,
                    workspace, C, stream)


def moe_mx4_workspace_bytes(tokens, hidden, inner, experts, top_k):
    """Workspace bytes of a moe_mx4 call with these sizes."""
    return int(L.load().moe_mx4_workspace_bytes(tokens, hidden, inner, experts, top_k))


def moe_mx4(x, logits, top_k, w_gate_up, w_down, inner, act=L.W4_ACT_SILU, renormalize=True,
            workspace=None, out=None, stream=None):
    """A mixture-of-experts layer: fp16 x [T,H] and the router's logits [T,E] -> fp16
    [T,H]. ``w_gate_up`` and ``w_down`` are prepack_mx4's of [E*2*inner,H] and
    [E*H,inner]; ``act`` a W4_ACT_*."""
    raw = None
    if stream is not None:
        raw = stream.cuda_stream
        if out is None:
            out = _empty(x.shape, torch.float16, _dev(x), stream)
    ws = _space(("moe", x.shape[0], x.shape[-1], inner, logits.shape[-1], top_k),
                moe_mx4_workspace_bytes, workspace, x.device, stream)
    return _done("moe_mx4", _bind().moe_mx4(x, logits, top_k, w_gate_up, w_down, inner, act,
                                            int(bool(renormalize)), ws, out, raw))
