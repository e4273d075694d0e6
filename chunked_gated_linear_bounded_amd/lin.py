"""Linear attention with one log-decay per token and value head, key heads shared by groups of value heads
(kda_lin_* of include/kda.h).

    S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t

Argument marshalling only, as the rest of the package: q, k and v may be strided views whose last
dimension is contiguous, g any view (a constant per head: slopes[:, None].expand(B, H, T))."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import KDA_OK, KdaError, _DTYPES, _empty, _on_device, _stream_of, lib
from .gdr import _plain, _view, _workspace


def _shapes(q, k, v, g, cu_seqlens):
    """(leading dims, N, Hk, H, T, dk, dv) of a batch [B,H,T,d] or of a packed stream [H,T,d]."""
    if not all(isinstance(t, torch.Tensor) for t in (q, k, v, g)):
        raise TypeError("q, k, v and g must be torch.Tensors")
    if q.dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % q.dtype)
    if g.dtype != q.dtype and g.dtype != torch.float32:
        raise ValueError("g has dtype %s, expected %s or float32" % (g.dtype, q.dtype))
    dims = 4 if cu_seqlens is None else 3
    if q.dim() != dims or v.dim() != dims:
        raise ValueError("q and v must have %d dimensions" % dims)
    lead, (Hk, T, dk), (H, dv) = tuple(q.shape[:-3]), q.shape[-3:], (v.shape[-3], v.shape[-1])
    if k.shape != q.shape or tuple(v.shape) != lead + (H, T, dv) or tuple(g.shape) != lead + (H, T):
        raise ValueError("shape mismatch")
    if Hk < 1 or H % Hk:
        raise ValueError("%d value heads cannot share %d key heads" % (H, Hk))
    if cu_seqlens is None:
        return lead, lead[0], Hk, H, T, dk, dv
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 boundaries")
    return lead, cu_seqlens.numel() - 1, Hk, H, T, dk, dv


def lin_workspace_bytes(N, Hk, H, T, dk, dv, dtype, packed=False, backward=False, end_state=True) -> int:
    """Bytes of workspace for a call on N sequences (packed: N documents in a stream of T tokens); of a
    backward that is not given dfinal_state, or not asked for dg, less with end_state=False."""
    io = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib().kda_lin_workspace_bytes((1 if end_state else 2) if backward else 0, int(packed), N, Hk, H, T, dk, dv, io))


def _fwd(q, k, v, g, cu_seqlens, scale, out, final_state, return_final_state, initial_state, workspace, stream):
    lead, N, Hk, H, T, dk, dv = _shapes(q, k, v, g, cu_seqlens)
    dtype, dev = q.dtype, q.device
    args = []
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        args += _view(t, name, dtype, dev)
    args += _view(g, "g", g.dtype, dev, inner=False)
    cu = None if cu_seqlens is None else _plain(cu_seqlens, "cu_seqlens", torch.int32, dev, (N + 1,))
    s0 = _plain(initial_state, "initial_state", torch.float32, dev, (N, H, dv, dk))
    po = _plain(out, "out", dtype, dev, lead + (H, T, dv))
    pf = _plain(final_state, "final_state", torch.float32, dev, (N, H, dv, dk))
    L, io = lib(), _DTYPES[dtype]
    with _on_device(dev):
        if out is None:
            out = _empty(lead + (H, T, dv), dtype, dev, stream)
            po = out.data_ptr()
        if final_state is None and return_final_state:
            final_state = _empty((N, H, dv, dk), torch.float32, dev, stream)
            pf = final_state.data_ptr()
        need = L.kda_lin_workspace_bytes(0, int(cu is not None), N, Hk, H, T, dk, dv, io)
        room = (None, 0)
        if need or workspace is not None:
            workspace = _workspace(workspace, need, dev, stream)
            room = (workspace.data_ptr(), workspace.numel())
        st = L.kda_lin_chunk_fwd(*args, cu, N, Hk, H, T, dk, dv, io, _DTYPES[g.dtype], float(scale), s0, po, pf, *room,
                                 _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_lin_chunk_fwd", st)
    return (out, final_state) if return_final_state else out


def lin_chunk_fwd(q, k, v, g, scale=1.0, out=None, final_state=None, return_final_state=False, initial_state=None,
                  workspace=None, stream=None):
    """Chunked forward.  q, k [B,Hk,T,dk]; v [B,H,T,dv], all bf16 or all float32; g (log-decay, <= 0)
    [B,H,T] in their dtype or float32; T any length; value head h uses key head h // (H / Hk).  Returns
    out [B,H,T,dv] (and the float32 final state [B,H,dv,dk] when asked for)."""
    return _fwd(q, k, v, g, None, scale, out, final_state, return_final_state, initial_state, workspace, stream)


def lin_chunk_fwd_varlen(q, k, v, g, cu_seqlens, scale=1.0, out=None, final_state=None, return_final_state=False,
                         initial_state=None, workspace=None, stream=None):
    """Packed documents: q, k [Hk,T,dk]; v [H,T,dv]; g [H,T]; cu_seqlens int32 [N+1] on the GPU.  Each
    document runs from its own state, initial_state / final_state [N,H,dv,dk].  Rows of out behind the
    last document are not written."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _fwd(q, k, v, g, cu_seqlens, scale, out, final_state, return_final_state, initial_state, workspace, stream)


def _bwd(q, k, v, g, dout, cu_seqlens, scale, initial_state, dfinal_state, workspace, stream, want_dg, want_dinitial):
    lead, N, Hk, H, T, dk, dv = _shapes(q, k, v, g, cu_seqlens)
    dtype, dev = q.dtype, q.device
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a torch.Tensor")
    if dout.shape != v.shape:
        raise ValueError("dout must have v's shape")
    args = []
    for t, name, inner in ((q, "q", True), (k, "k", True), (v, "v", True), (g, "g", False), (dout, "dout", True)):
        args += _view(t, name, g.dtype if name == "g" else dtype, dev, inner)
    cu = None if cu_seqlens is None else _plain(cu_seqlens, "cu_seqlens", torch.int32, dev, (N + 1,))
    s0 = _plain(initial_state, "initial_state", torch.float32, dev, (N, H, dv, dk))
    df = _plain(dfinal_state, "dfinal_state", torch.float32, dev, (N, H, dv, dk))
    with _on_device(dev):
        out = {n: _empty(shape, dt, dev, stream) if want else None for n, shape, dt, want in (
            ("dq", q.shape, dtype, True), ("dk", q.shape, dtype, True), ("dv", v.shape, dtype, True),
            ("dg", g.shape, g.dtype, want_dg), ("dinitial_state", (N, H, dv, dk), torch.float32, want_dinitial))}
        need = lin_workspace_bytes(N, Hk, H, T, dk, dv, dtype, cu is not None, backward=True, end_state=want_dg and df is not None)
        workspace = _workspace(workspace, need, dev, stream)
        st = lib().kda_lin_chunk_bwd(*args, cu, N, Hk, H, T, dk, dv, _DTYPES[dtype], _DTYPES[g.dtype], float(scale), s0, df,
                                     *(None if t is None else t.data_ptr() for t in out.values()),
                                     workspace.data_ptr(), workspace.numel(), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_lin_chunk_bwd", st)
    return out


def lin_chunk_bwd(q, k, v, g, dout, scale=1.0, initial_state=None, dfinal_state=None, workspace=None, stream=None,
                  want_dg=True, want_dinitial=True):
    """Gradients of sum(dout * out) + sum(dfinal_state * final_state) of lin_chunk_fwd, from its inputs
    alone.  Returns a dict of dq, dk (summed over the value heads that share a key head), dv in the
    inputs' dtype, dg in g's (None unless want_dg: constant decays need none) and dinitial_state in
    float32 (None unless want_dinitial)."""
    return _bwd(q, k, v, g, dout, None, scale, initial_state, dfinal_state, workspace, stream, want_dg, want_dinitial)


def lin_chunk_bwd_varlen(q, k, v, g, dout, cu_seqlens, scale=1.0, initial_state=None, dfinal_state=None, workspace=None,
                         stream=None, want_dg=True, want_dinitial=True):
    """lin_chunk_bwd of packed documents (lin_chunk_fwd_varlen).  Tokens behind the last document get zero
    gradients."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _bwd(q, k, v, g, dout, cu_seqlens, scale, initial_state, dfinal_state, workspace, stream, want_dg, want_dinitial)


class LinChunkFunction(torch.autograd.Function):
    """out, final_state = LinChunkFunction.apply(q, k, v, g, scale, initial_state, cu_seqlens): the chunked
    forward with its backward, for a batch or (cu_seqlens given) for packed documents.  Once
    differentiable: a gradient of the gradients is an error.  So is, with gradients enabled, a capture into a
    graph with leaves among the inputs: a leaf gathers its gradient on the stream it was first used on, and
    where an eager graph of it lives that is not the captured one, which ends the process.  lin_chunk_fwd and
    lin_chunk_bwd may be captured, and under no_grad this function."""

    @classmethod
    def apply(cls, *args):
        # (here, because forward itself runs with gradients disabled)
        if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad and t.is_leaf for t in args) and \
                torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a leaf's gradient cannot be captured here: capture lin_chunk_fwd and lin_chunk_bwd")
        return super().apply(*args)

    @staticmethod
    def forward(ctx, q, k, v, g, scale=1.0, initial_state=None, cu_seqlens=None):
        out, fs = _fwd(q, k, v, g, cu_seqlens, scale, None, None, True, initial_state, None, None)
        ctx.set_materialize_grads(False)  # an end state that nobody used costs the backward nothing
        ctx.save_for_backward(q, k, v, g, initial_state, cu_seqlens)
        ctx.scale = scale
        return out, fs

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dfinal):
        q, k, v, g, s0, cu = ctx.saved_tensors
        if dout is None and dfinal is None:
            return (None,) * 7
        dout = v.new_zeros(v.shape) if dout is None else dout.contiguous()
        d = _bwd(q, k, v, g, dout, cu, ctx.scale, s0, None if dfinal is None else dfinal.contiguous(), None, None, ctx.needs_input_grad[3],
                 s0 is not None and ctx.needs_input_grad[5])
        return d["dq"], d["dk"], d["dv"], d["dg"], None, d["dinitial_state"], None


def lin_decode_step(q, k, v, g, state, scale=1.0, out=None, stream=None):
    """One token per (batch, value head): q, k [B,Hk,dk]; v [B,H,dv] (all bf16 or all float32); g [B,H] in
    their dtype or float32; all contiguous; state float32 [B,H,dv,dk], updated in place.  Returns out
    [B,H,dv]."""
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor) or not isinstance(g, torch.Tensor):
        raise TypeError("q, v and g must be torch.Tensors")
    dtype, dev = q.dtype, q.device
    if dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dtype)
    if g.dtype != dtype and g.dtype != torch.float32:
        raise ValueError("g has dtype %s, expected %s or float32" % (g.dtype, dtype))
    if dev.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must have 3 dimensions")
    (B, Hk, dk), (H, dv) = q.shape, v.shape[1:]
    if Hk < 1 or H % Hk:
        raise ValueError("%d value heads cannot share %d key heads" % (H, Hk))
    ptrs = [_plain(t, name, dt, dev, shape) for t, name, dt, shape in (
        (q, "q", dtype, (B, Hk, dk)), (k, "k", dtype, (B, Hk, dk)), (v, "v", dtype, (B, H, dv)), (g, "g", g.dtype, (B, H)))]
    ps = _plain(state, "state", torch.float32, dev, (B, H, dv, dk))
    with _on_device(dev):
        if out is None:
            out = _empty((B, H, dv), dtype, dev, stream)
        st = lib().kda_lin_decode_step(*ptrs, B, Hk, H, dk, dv, _DTYPES[dtype], _DTYPES[g.dtype], float(scale), ps,
                                       _plain(out, "out", dtype, dev, (B, H, dv)), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_lin_decode_step", st)
    return out
