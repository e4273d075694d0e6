"""Latent attention: causal softmax attention whose keys and values come from one latent vector a token
(kda_latent_* of include/kda.h).  Expanded form for prefill and training, absorbed form for decoding.

Argument marshalling only.  The inputs of the expanded form may be strided views whose last dimension
is contiguous: with kv [B,S,H,dn+dn] from the up-projection of the latents, k = kv[..., :dn].transpose(1, 2)
and v = kv[..., dn:].transpose(1, 2) are taken as they are."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import KDA_OK, KdaError, _DTYPES, _empty, _on_device, _stream_of, lib
from .gdr import _S3, _plain, _view, _workspace


def _shapes(q, k, v, k_rope, cu_q, cu_k):
    """(leading dims, N, H, T, S, dn, dr) of a batch ([B,H,T,d] ...) or of packed streams ([H,T,d] ...)."""
    if not all(isinstance(t, torch.Tensor) for t in (q, k, v, k_rope)):
        raise TypeError("q, k, v and k_rope must be torch.Tensors")
    if q.dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % q.dtype)
    dims = 4 if cu_q is None else 3
    if q.dim() != dims or k.dim() != dims or k_rope.dim() != dims - 1:
        raise ValueError("q, k and k_rope must have %d, %d and %d dimensions" % (dims, dims, dims - 1))
    lead, (H, T, d), (S, dn), dr = tuple(q.shape[:-3]), q.shape[-3:], k.shape[-2:], k_rope.shape[-1]
    if tuple(k.shape) != lead + (H, S, dn) or v.shape != k.shape or tuple(k_rope.shape) != lead + (S, dr) or d != dn + dr:
        raise ValueError("shape mismatch")
    if cu_q is None:
        return lead, lead[0], H, T, S, dn, dr
    for t in (cu_q, cu_k):
        if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.numel() < 2 or t.shape != cu_q.shape:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must be 1-D tensors of N + 1 boundaries each")
    return lead, cu_q.numel() - 1, H, T, S, dn, dr


def _inputs(q, k, v, k_rope, cu_q, cu_k, N):
    dtype, dev = q.dtype, q.device
    args = []
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        args += _view(t, name, dtype, dev)
    args += _rope(k_rope, dtype, dev)
    for t, name in ((cu_q, "cu_seqlens_q"), (cu_k, "cu_seqlens_k")):
        args.append(None if t is None else _plain(t, name, torch.int32, dev, (N + 1,)))
    return args


def _rope(t, dtype, dev):
    """k_rope [B,S,dr] or [S,dr]: strides b, (no head), t."""
    ptr, _ = _view(t, "k_rope", dtype, dev)
    st = t.stride()[:-1]
    return ptr, _S3(st[0] if len(st) == 2 else 0, 0, st[-1])


def _fwd(q, k, v, k_rope, cu_q, cu_k, scale, out, lse, return_lse, stream):
    lead, N, H, T, S, dn, dr = _shapes(q, k, v, k_rope, cu_q, cu_k)
    dtype, dev = q.dtype, q.device
    args = _inputs(q, k, v, k_rope, cu_q, cu_k, N)
    scale = (dn + dr) ** -0.5 if scale is None else scale
    with _on_device(dev):
        if out is None:
            out = _empty(lead + (H, T, dn), dtype, dev, stream)
        if lse is None:
            lse = _empty(lead + (H, T), torch.float32, dev, stream)
        st = lib().kda_latent_attn_fwd(*args, N, H, T, S, dn, dr, _DTYPES[dtype], float(scale),
                                       _plain(out, "out", dtype, dev, lead + (H, T, dn)),
                                       _plain(lse, "lse", torch.float32, dev, lead + (H, T)), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_latent_attn_fwd", st)
    return (out, lse) if return_lse else out


def latent_attn_fwd(q, k, v, k_rope, scale=None, out=None, lse=None, return_lse=False, stream=None):
    """Expanded form: q [B,H,T,dn+dr]; k, v [B,H,S,dn]; k_rope [B,S,dr], shared by the heads; all bf16 or
    all float32.  Causal, the last query at the last key (S >= T: T queries behind a prefix).  scale
    defaults to (dn + dr)^-0.5.  Returns out [B,H,T,dn] (and the float32 log-sum-exps [B,H,T])."""
    return _fwd(q, k, v, k_rope, None, None, scale, out, lse, return_lse, stream)


def latent_attn_fwd_varlen(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, scale=None, out=None, lse=None, return_lse=False,
                           stream=None):
    """Packed sequences: q [H,T,dn+dr]; k, v [H,S,dn]; k_rope [S,dr]; boundaries int32 [N+1] on the GPU.
    Rows of out and lse behind the last sequence are not written."""
    if cu_seqlens_q is None or cu_seqlens_k is None:
        raise TypeError("cu_seqlens_q and cu_seqlens_k must be torch.Tensors")
    return _fwd(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, scale, out, lse, return_lse, stream)


def latent_bwd_workspace_bytes(N, H, T, S, dn, dr, dtype, packed=False) -> int:
    io = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib().kda_latent_attn_bwd_workspace_bytes(int(packed), N, H, T, S, dn, dr, io))


def _bwd(q, k, v, k_rope, out, lse, dout, cu_q, cu_k, scale, workspace, stream):
    lead, N, H, T, S, dn, dr = _shapes(q, k, v, k_rope, cu_q, cu_k)
    dtype, dev = q.dtype, q.device
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a torch.Tensor")
    if tuple(dout.shape) != lead + (H, T, dn):
        raise ValueError("dout must have out's shape")
    args = _inputs(q, k, v, k_rope, cu_q, cu_k, N)
    kept = [_plain(out, "out", dtype, dev, lead + (H, T, dn)), _plain(lse, "lse", torch.float32, dev, lead + (H, T))]
    if None in kept:
        raise TypeError("out and lse of the forward are needed")
    scale = (dn + dr) ** -0.5 if scale is None else scale
    with _on_device(dev):
        g = {n: _empty(shape, dtype, dev, stream) for n, shape in (
            ("dq", q.shape), ("dk", k.shape), ("dv", v.shape), ("dk_rope", k_rope.shape))}
        workspace = _workspace(workspace, latent_bwd_workspace_bytes(N, H, T, S, dn, dr, dtype, cu_q is not None), dev, stream)
        st = lib().kda_latent_attn_bwd(*args[:8], *kept, *_view(dout, "dout", dtype, dev), *args[8:], N, H, T, S, dn, dr,
                                       _DTYPES[dtype], float(scale), *(t.data_ptr() for t in g.values()),
                                       workspace.data_ptr(), workspace.numel(), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_latent_attn_bwd", st)
    return g


def latent_attn_bwd(q, k, v, k_rope, out, lse, dout, scale=None, workspace=None, stream=None):
    """Gradients of sum(dout * out), from latent_attn_fwd's inputs, out and lse: a dict of dq, dk, dv and
    dk_rope (summed over the heads) in the inputs' dtype."""
    return _bwd(q, k, v, k_rope, out, lse, dout, None, None, scale, workspace, stream)


def latent_attn_bwd_varlen(q, k, v, k_rope, out, lse, dout, cu_seqlens_q, cu_seqlens_k, scale=None, workspace=None,
                           stream=None):
    """latent_attn_bwd of packed sequences.  Tokens that no sequence covers get zero gradients."""
    if cu_seqlens_q is None or cu_seqlens_k is None:
        raise TypeError("cu_seqlens_q and cu_seqlens_k must be torch.Tensors")
    return _bwd(q, k, v, k_rope, out, lse, dout, cu_seqlens_q, cu_seqlens_k, scale, workspace, stream)


class LatentAttnFunction(torch.autograd.Function):
    """out = LatentAttnFunction.apply(q, k, v, k_rope, scale, cu_seqlens_q, cu_seqlens_k): the expanded form
    with its backward, for a batch or (boundaries given) for packed sequences.  Once differentiable: a
    gradient of the gradients is an error."""

    @staticmethod
    def forward(ctx, q, k, v, k_rope, scale=None, cu_seqlens_q=None, cu_seqlens_k=None):
        out, lse = _fwd(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, scale, None, None, True, None)
        ctx.save_for_backward(q, k, v, k_rope, out, lse, cu_seqlens_q, cu_seqlens_k)
        ctx.scale = scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        *x, out, lse, cu_q, cu_k = ctx.saved_tensors
        g = _bwd(*x, out, lse, dout.contiguous(), cu_q, cu_k, ctx.scale, None, None)
        return g["dq"], g["dk"], g["dv"], g["dk_rope"], None, None, None


def latent_decode_workspace_bytes(B, H, page, max_pages, dc, dr, dtype) -> int:
    io = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib().kda_latent_decode_workspace_bytes(B, H, page, max_pages, dc, dr, io))


def latent_decode_step(q, cache, block_table, lengths, scale, dc=512, out=None, lse=None, return_lse=False, workspace=None,
                       stream=None):
    """Absorbed form, one token per sequence: q [B,H,dc+dr] (the query multiplied into the latent's space,
    and its rotary part); cache [pages,page,dc+dr], whose first dc channels are also the values;
    block_table int32 [B,max_pages]; lengths int32 [B].  scale is the expanded form's, (dn + dr)^-0.5.
    Returns out [B,H,dc] (and the float32 log-sum-exps [B,H])."""
    if not isinstance(q, torch.Tensor) or not isinstance(cache, torch.Tensor) or not isinstance(block_table, torch.Tensor):
        raise TypeError("q, cache and block_table must be torch.Tensors")
    dtype, dev = q.dtype, q.device
    if dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dtype)
    if dev.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    if q.dim() != 3 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q, cache and block_table must have 3, 3 and 2 dimensions")
    (B, H, D), (pages, page), max_pages = q.shape, cache.shape[:2], block_table.shape[1]
    ptrs = [_plain(q, "q", dtype, dev, (B, H, D)), _plain(cache, "cache", dtype, dev, (pages, page, D)),
            _plain(block_table, "block_table", torch.int32, dev, (B, max_pages)),
            _plain(lengths, "lengths", torch.int32, dev, (B,))]
    with _on_device(dev):
        if out is None:
            out = _empty((B, H, dc), dtype, dev, stream)
        if lse is None:
            lse = _empty((B, H), torch.float32, dev, stream)
        need = latent_decode_workspace_bytes(B, H, page, max_pages, dc, D - dc, dtype)
        workspace = _workspace(workspace, need, dev, stream)
        st = lib().kda_latent_decode_step(*ptrs, B, H, pages, page, max_pages, dc, D - dc, _DTYPES[dtype], float(scale),
                                          _plain(out, "out", dtype, dev, (B, H, dc)),
                                          _plain(lse, "lse", torch.float32, dev, (B, H)),
                                          workspace.data_ptr(), workspace.numel(), _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_latent_decode_step", st)
    return (out, lse) if return_lse else out


def _append(latent, k_rope, cache, block_table, lengths, freqs, cu_seqlens, norm_weight, eps, positions, counts, interleaved, q_rope, q,
            stream):
    if not all(isinstance(t, torch.Tensor) for t in (latent, k_rope, cache, block_table)):
        raise TypeError("latent, k_rope, cache and block_table must be torch.Tensors")
    dtype, dev = cache.dtype, cache.device
    if dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dtype)
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q go together")
    dims = 3 if cu_seqlens is None else 2
    if latent.dim() != dims or k_rope.dim() != dims or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("latent, k_rope, cache and block_table must have %d, %d, 3 and 2 dimensions" % (dims, dims))
    lead, dc, dr, (pages, page), (N, max_pages) = tuple(latent.shape[:-1]), latent.shape[-1], k_rope.shape[-1], cache.shape[:2], block_table.shape
    if tuple(k_rope.shape[:-1]) != lead or cache.shape[2] != dc + dr or (cu_seqlens is None and lead[0] != N):
        raise ValueError("shape mismatch")
    T, H = lead[-1], 0
    if q_rope is not None:
        if not isinstance(q_rope, torch.Tensor) or not isinstance(q, torch.Tensor):
            raise TypeError("q_rope and q must be torch.Tensors")
        if q_rope.dim() != dims + 1 or tuple(q_rope.shape[:-2]) != lead or q_rope.shape[-1] != dr:
            raise ValueError("q_rope must have shape %s, has %s" % (lead + ("H", dr), tuple(q_rope.shape)))
        H = q_rope.shape[-2]
    pl, sl = _view(latent, "latent", dtype, dev)
    pk, sk = _view(k_rope, "k_rope", dtype, dev)
    pr, sr = _view(q_rope, "q_rope", dtype, dev) if q_rope is not None else (None, None)
    # (.., b, t) and (b, t, h) as the library's (b, h, t)
    for s in (sl, sk):
        s[0], s[1] = s[1], 0
    if sr is not None:
        sr[1], sr[2] = sr[2], sr[1]
    args = [_plain(cache, "cache", dtype, dev, (pages, page, dc + dr)),
            _plain(block_table, "block_table", torch.int32, dev, (N, max_pages)), _plain(lengths, "lengths", torch.int32, dev, (N,)),
            _plain(freqs, "freqs", torch.float32, dev, (dr // 2,)), _plain(norm_weight, "norm_weight", dtype, dev, (dc,)), float(eps),
            _plain(positions, "positions", torch.int32, dev, lead), _plain(counts, "counts", torch.int32, dev, (N,)),
            pr, sr, _plain(q, "q", dtype, dev, lead + (H, dc + dr)),
            None if cu_seqlens is None else _plain(cu_seqlens, "cu_seqlens", torch.int32, dev, (N + 1,))]
    with _on_device(dev):
        st = lib().kda_latent_append(pl, sl, pk, sk, *args, N, T, H, pages, page, max_pages, dc, dr, _DTYPES[dtype], int(bool(interleaved)),
                                     _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_latent_append", st)
    return cache


def latent_append(latent, k_rope, cache, block_table, lengths, freqs, norm_weight=None, eps=1e-6, positions=None, counts=None,
                  interleaved=True, q_rope=None, q=None, stream=None):
    """Writes T new tokens a sequence into the paged cache that latent_decode_step and latent_tree_step read:
    latent [B,T,dc], normalised by its root mean square and norm_weight [dc] where that is given, and
    k_rope [B,T,dr], rotated; both may be strided views (the two parts of one projection).  lengths int32
    [B] are those with the new tokens; counts int32 [B] how many of T are tokens (all by default): token i
    becomes row lengths[b] - counts[b] + i.  A pair turns by position * freqs[i] (float32 [dr / 2]);
    positions int32 [B,T], by default the rows'; pairs are neighbours (interleaved) or dr / 2 apart.  With
    q_rope [B,T,H,dr], the queries' rotary part, its rotation goes into the last dr channels of q
    [B,T,H,dc+dr].  Returns cache."""
    return _append(latent, k_rope, cache, block_table, lengths, freqs, None, norm_weight, eps, positions, counts, interleaved, q_rope, q,
                   stream)


def latent_append_varlen(latent, k_rope, cache, block_table, lengths, freqs, cu_seqlens, norm_weight=None, eps=1e-6, positions=None,
                         interleaved=True, q_rope=None, q=None, stream=None):
    """latent_append of packed sequences: latent [T,dc], k_rope [T,dr], positions [T], q_rope [T,H,dr], q
    [T,H,dc+dr]; boundaries int32 [N+1] on the GPU.  Tokens that no sequence covers are not written."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _append(latent, k_rope, cache, block_table, lengths, freqs, cu_seqlens, norm_weight, eps, positions, None, interleaved, q_rope, q,
                   stream)


def latent_tree_workspace_bytes(B, T, H, page, max_pages, dc, dr, dtype) -> int:
    io = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib().kda_latent_tree_workspace_bytes(B, T, H, page, max_pages, dc, dr, io))


def latent_tree_step(q, cache, block_table, lengths, tree_mask, scale, dc=512, counts=None, out=None, lse=None, return_lse=False,
                     workspace=None, stream=None):
    """Absorbed form, up to 64 drafted tokens per sequence, whose rows are the last of the cache
    (latent_append): q [B,T,H,dc+dr]; cache, block_table, lengths and scale as for latent_decode_step, lengths
    with the drafted tokens.  Every drafted token sees the rows before them, and of theirs those whose bits
    are set in its tree_mask (int64 [B,T]; bit j: the token j of the sequence, its own among them: a chain
    has 2 << i - 1).  counts int32 [B]: how many of T are tokens (all by default); the others give zeros.
    Returns out [B,T,H,dc] (and the float32 log-sum-exps [B,T,H])."""
    if not all(isinstance(t, torch.Tensor) for t in (q, cache, block_table, tree_mask)):
        raise TypeError("q, cache, block_table and tree_mask must be torch.Tensors")
    dtype, dev = q.dtype, q.device
    if dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dtype)
    if dev.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    if q.dim() != 4 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q, cache and block_table must have 4, 3 and 2 dimensions")
    (B, T, H, D), (pages, page), max_pages = q.shape, cache.shape[:2], block_table.shape[1]
    ptrs = [_plain(q, "q", dtype, dev, (B, T, H, D)), _plain(cache, "cache", dtype, dev, (pages, page, D)),
            _plain(block_table, "block_table", torch.int32, dev, (B, max_pages)),
            _plain(lengths, "lengths", torch.int32, dev, (B,)), _plain(counts, "counts", torch.int32, dev, (B,)),
            _plain(tree_mask, "tree_mask", torch.int64, dev, (B, T))]
    po, pl = _plain(out, "out", dtype, dev, (B, T, H, dc)), _plain(lse, "lse", torch.float32, dev, (B, T, H))
    L, io = lib(), _DTYPES[dtype]
    with _on_device(dev):
        if out is None:
            out = _empty((B, T, H, dc), dtype, dev, stream)
            po = out.data_ptr()
        if lse is None:
            lse = _empty((B, T, H), torch.float32, dev, stream)
            pl = lse.data_ptr()
        need = L.kda_latent_tree_workspace_bytes(B, T, H, page, max_pages, dc, D - dc, io)
        room = (None, 0)
        if need or workspace is not None:
            workspace = _workspace(workspace, need, dev, stream)
            room = (workspace.data_ptr(), workspace.numel())
        st = L.kda_latent_tree_step(*ptrs, B, T, H, pages, page, max_pages, dc, D - dc, io, float(scale), po, pl, *room,
                                    _stream_of(stream, dev))
    if st != KDA_OK:
        raise KdaError("kda_latent_tree_step", st)
    return (out, lse) if return_lse else out
