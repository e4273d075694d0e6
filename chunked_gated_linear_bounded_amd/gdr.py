"""The gated delta rule: one log-decay per token and value head, key heads shared by groups of value
heads (kda_gdr_* of include/kda.h).

    S_t = e^{g_t} S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = scale S_t q_t

Argument marshalling only, as the rest of the package: q, k, v, g and beta may be strided views whose
last dimension is contiguous (for instance [B,T,H,d] projections transposed to [B,H,T,d])."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import KDA_OK, KdaError, _DTYPES, _empty, _on_device, _stream_of, lib

_S3 = ctypes.c_longlong * 3


def _view(t, name, dtype, dev, inner=True):
    """Checks a strided input; returns (pointer, element strides of all but the last dimension)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dev.type != "cuda" or t.device != dev:
        raise ValueError("%s must be a GPU tensor on %s, is on %s" % (name, dev, t.device))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    s = t.stride()
    if inner:
        if s[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0:
            raise ValueError("the last dimension of %s must be contiguous" % name)
        s = s[:-1]
    return t.data_ptr(), _S3(*s) if len(s) == 3 else _S3(*((0,) * (3 - len(s)) + s))


def _plain(t, name, dtype, dev, shape):
    """Checks a contiguous tensor of a given shape (or None); returns its pointer."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev or t.dtype != dtype:
        raise ValueError("%s must be %s on %s, is %s on %s" % (name, dtype, dev, t.dtype, t.device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, has %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _shapes(q, k, v, g, beta, cu_seqlens):
    """(leading dims, N, Hk, H, T, dk, dv) of a batch [B,H,T,d] or of a packed stream [H,T,d]."""
    if not all(isinstance(t, torch.Tensor) for t in (q, k, v, g, beta)):
        raise TypeError("q, k, v, g and beta must be torch.Tensors")
    if q.dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % q.dtype)
    dims = 4 if cu_seqlens is None else 3
    if q.dim() != dims or v.dim() != dims:
        raise ValueError("q and v must have %d dimensions" % dims)
    lead, (Hk, T, dk), (H, dv) = tuple(q.shape[:-3]), q.shape[-3:], (v.shape[-3], v.shape[-1])
    if k.shape != q.shape or tuple(v.shape) != lead + (H, T, dv) or tuple(g.shape) != lead + (H, T) or \
            beta.shape != g.shape:
        raise ValueError("shape mismatch")
    if Hk < 1 or H % Hk:
        raise ValueError("%d value heads cannot share %d key heads" % (H, Hk))
    if cu_seqlens is None:
        return lead, lead[0], Hk, H, T, dk, dv
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 boundaries")
    return lead, cu_seqlens.numel() - 1, Hk, H, T, dk, dv


def gdr_workspace_bytes(N, Hk, H, T, dk, dv, dtype, packed=False, backward=False) -> int:
    """Bytes of workspace for a call on N sequences (packed: N documents in a stream of T tokens)."""
    io = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib().kda_gdr_workspace_bytes(int(backward), int(packed), N, Hk, H, T, dk, dv, io))


def _workspace(workspace, need, dev, stream):
    if workspace is None:
        return _empty(max(need, 1), torch.uint8, dev, stream)
    _plain(workspace, "workspace", torch.uint8, dev, workspace.shape)
    return workspace


def _fwd(q, k, v, g, beta, cu_seqlens, scale, out, final_state, return_final_state, initial_state, workspace, stream):
    lead, N, Hk, H, T, dk, dv = _shapes(q, k, v, g, beta, cu_seqlens)
    dtype, dev = q.dtype, q.device
    args = []
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        args += _view(t, name, dtype, dev)
    for t, name in ((g, "g"), (beta, "beta")):
        args += _view(t, name, dtype, dev, inner=False)
    cu = None if cu_seqlens is None else _plain(cu_seqlens, "cu_seqlens", torch.int32, dev, (N + 1,))
    s0 = _plain(initial_state, "initial_state", torch.float32, dev, (N, H, dv, dk))
    with _on_device(dev):
        if out is None:
            out = _empty(lead + (H, T, dv), dtype, dev, stream)
        if final_state is None and return_final_state:
            final_state = _empty((N, H, dv, dk), torch.float32, dev, stream)
        po = _plain(out, "out", dtype, dev, lead + (H, T, dv))
        pf = _plain(final_state, "final_state", torch.float32, dev, (N, H, dv, dk))
        workspace = _workspace(workspace, gdr_workspace_bytes(N, Hk, H, T, dk, dv, dtype, cu is not None), dev, stream)
        st = lib().kda_gdr_chunk_fwd(*args, cu, N, Hk, H, T, dk, dv, _DTYPES[dtype], float(scale), s0, po, pf,
                                     workspace.data_ptr(), workspace.numel(), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_gdr_chunk_fwd", st)
    return (out, final_state) if return_final_state else out


def gdr_chunk_fwd(q, k, v, g, beta, scale=1.0, out=None, final_state=None, return_final_state=False, initial_state=None,
                  workspace=None, stream=None):
    """Chunked forward.  q, k [B,Hk,T,dk]; v [B,H,T,dv]; g (log-decay, <= 0) and beta [B,H,T]; all
    bf16 or all float32; T any length; value head h uses key head h // (H / Hk).  Returns out
    [B,H,T,dv] (and the float32 final state [B,H,dv,dk] when asked for)."""
    return _fwd(q, k, v, g, beta, None, scale, out, final_state, return_final_state, initial_state, workspace, stream)


def gdr_chunk_fwd_varlen(q, k, v, g, beta, cu_seqlens, scale=1.0, out=None, final_state=None, return_final_state=False,
                         initial_state=None, workspace=None, stream=None):
    """Packed documents: q, k [Hk,T,dk]; v [H,T,dv]; g, beta [H,T]; cu_seqlens int32 [N+1] on the GPU.
    Each document runs from its own state, initial_state / final_state [N,H,dv,dk].  Rows of out
    behind the last document are not written."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _fwd(q, k, v, g, beta, cu_seqlens, scale, out, final_state, return_final_state, initial_state, workspace,
                stream)


def _bwd(q, k, v, g, beta, dout, cu_seqlens, scale, initial_state, dfinal_state, workspace, stream, want_dinitial):
    lead, N, Hk, H, T, dk, dv = _shapes(q, k, v, g, beta, cu_seqlens)
    dtype, dev = q.dtype, q.device
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a torch.Tensor")
    if dout.shape != v.shape:
        raise ValueError("dout must have v's shape")
    args = []
    for t, name, inner in ((q, "q", True), (k, "k", True), (v, "v", True), (g, "g", False), (beta, "beta", False),
                           (dout, "dout", True)):
        args += _view(t, name, dtype, dev, inner)
    cu = None if cu_seqlens is None else _plain(cu_seqlens, "cu_seqlens", torch.int32, dev, (N + 1,))
    s0 = _plain(initial_state, "initial_state", torch.float32, dev, (N, H, dv, dk))
    df = _plain(dfinal_state, "dfinal_state", torch.float32, dev, (N, H, dv, dk))
    with _on_device(dev):
        out = {n: _empty(shape, dtype, dev, stream) for n, shape in (
            ("dq", q.shape), ("dk", q.shape), ("dv", v.shape), ("dg", g.shape), ("dbeta", g.shape))}
        out["dinitial_state"] = _empty((N, H, dv, dk), torch.float32, dev, stream) if want_dinitial else None
        need = gdr_workspace_bytes(N, Hk, H, T, dk, dv, dtype, cu is not None, backward=True)
        workspace = _workspace(workspace, need, dev, stream)
        st = lib().kda_gdr_chunk_bwd(*args, cu, N, Hk, H, T, dk, dv, _DTYPES[dtype], float(scale), s0, df,
                                     *(None if t is None else t.data_ptr() for t in out.values()),
                                     workspace.data_ptr(), workspace.numel(), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_gdr_chunk_bwd", st)
    return out


def gdr_chunk_bwd(q, k, v, g, beta, dout, scale=1.0, initial_state=None, dfinal_state=None, workspace=None, stream=None,
                  want_dinitial=True):
    """Gradients of sum(dout * out) + sum(dfinal_state * final_state) of gdr_chunk_fwd, from its inputs
    alone.  Returns a dict of dq, dk (summed over the value heads that share a key head), dv, dg, dbeta
    in the inputs' dtype and dinitial_state in float32 (None unless want_dinitial)."""
    return _bwd(q, k, v, g, beta, dout, None, scale, initial_state, dfinal_state, workspace, stream, want_dinitial)


def gdr_chunk_bwd_varlen(q, k, v, g, beta, dout, cu_seqlens, scale=1.0, initial_state=None, dfinal_state=None,
                         workspace=None, stream=None, want_dinitial=True):
    """gdr_chunk_bwd of packed documents (gdr_chunk_fwd_varlen).  Tokens behind the last document get
    zero gradients."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _bwd(q, k, v, g, beta, dout, cu_seqlens, scale, initial_state, dfinal_state, workspace, stream, want_dinitial)


class GdrChunkFunction(torch.autograd.Function):
    """out, final_state = GdrChunkFunction.apply(q, k, v, g, beta, scale, initial_state, cu_seqlens): the
    chunked forward with its backward, for a batch or (cu_seqlens given) for packed documents.  Once
    differentiable: a gradient of the gradients is an error."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale=1.0, initial_state=None, cu_seqlens=None):
        out, fs = _fwd(q, k, v, g, beta, cu_seqlens, scale, None, None, True, initial_state, None, None)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.scale = scale
        return out, fs

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dfinal):
        q, k, v, g, beta, s0, cu = ctx.saved_tensors
        d = _bwd(q, k, v, g, beta, dout.contiguous(), cu, ctx.scale, s0, dfinal.contiguous(), None, None,
                 s0 is not None and ctx.needs_input_grad[6])
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], None, d["dinitial_state"], None


def gdr_decode_step(q, k, v, g, beta, state, scale=1.0, out=None, stream=None):
    """One token per (batch, value head): q, k [B,Hk,dk]; v [B,H,dv]; g, beta [B,H] (all bf16 or all
    float32, contiguous); state float32 [B,H,dv,dk], updated in place.  Returns out [B,H,dv]."""
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("q and v must be torch.Tensors")
    dtype, dev = q.dtype, q.device
    if dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dtype)
    if dev.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must have 3 dimensions")
    (B, Hk, dk), (H, dv) = q.shape, v.shape[1:]
    if Hk < 1 or H % Hk:
        raise ValueError("%d value heads cannot share %d key heads" % (H, Hk))
    ptrs = [_plain(t, name, dtype, dev, shape) for t, name, shape in (
        (q, "q", (B, Hk, dk)), (k, "k", (B, Hk, dk)), (v, "v", (B, H, dv)), (g, "g", (B, H)), (beta, "beta", (B, H)))]
    ps = _plain(state, "state", torch.float32, dev, (B, H, dv, dk))
    with _on_device(dev):
        if out is None:
            out = _empty((B, H, dv), dtype, dev, stream)
        st = lib().kda_gdr_decode_step(*ptrs, B, Hk, H, dk, dv, _DTYPES[dtype], float(scale), ps,
                                       _plain(out, "out", dtype, dev, (B, H, dv)), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_gdr_decode_step", st)
    return out
