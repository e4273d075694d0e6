"""Refusals of latent attention's entry points, without a GPU."""
import ctypes

import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first
OK, E_NULL, E_SHAPE, E_DTYPE, E_WS, E_ALIGN, E_SCALE = 0, -1, -2, -3, -6, -8, -11
S3 = ctypes.c_longlong * 3


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(k=None), E_NULL), (dict(kr=None), E_NULL), (dict(out=None), E_NULL), (dict(lse=None), E_NULL),
    (dict(cq=FAKE), E_NULL), (dict(ck=FAKE), E_NULL), (dict(io=2), E_DTYPE), (dict(N=0), E_SHAPE), (dict(H=0), E_SHAPE),
    (dict(T=-1), E_SHAPE), (dict(S=-1), E_SHAPE), (dict(dn=96), E_SHAPE), (dict(dr=16), E_SHAPE), (dict(H=70000), E_SHAPE),
    (dict(N=70000), E_SHAPE), (dict(N=1 << 30, cq=FAKE, ck=FAKE), E_SHAPE), (dict(scale=0.0), E_SCALE),
    (dict(scale=-1.0), E_SCALE), (dict(scale=float("nan")), E_SCALE), (dict(scale=float("inf")), E_SCALE),
    (dict(q=FAKE + 8), E_ALIGN), (dict(lse=FAKE + 2), E_ALIGN), (dict(ks=S3(0, 0, 132)), E_ALIGN),
    (dict(krs=S3(0, 0, 68)), E_ALIGN), (dict(io=1, vs=S3(0, 2, 128)), E_ALIGN),
    (dict(ks=S3(0, 0, 1 << 24)), E_SHAPE), (dict(io=1, qs=S3(0, 0, 1 << 23)), E_SHAPE), (dict(vs=S3(0, 0, -128)), E_SHAPE),
    (dict(krs=S3(0, 0, 1 << 40)), E_SHAPE), (dict(T=0, q=None, out=None, lse=None), OK),
])
def test_forward_refusals(kw, want):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, kr=FAKE, krs=None, cq=None, ck=None, N=2, H=4, T=100, S=120,
             dn=128, dr=64, io=0, scale=0.1, out=FAKE, lse=FAKE)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_latent_attn_fwd(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), E_NULL), (dict(lse=None), E_NULL), (dict(do=None), E_NULL), (dict(dkr=None), E_NULL), (dict(io=5), E_DTYPE),
    (dict(dr=48), E_SHAPE), (dict(scale=0.0), E_SCALE), (dict(do=FAKE + 4), E_ALIGN), (dict(dos=S3(0, 0, 129)), E_ALIGN),
    (dict(dq=FAKE + 8), E_ALIGN), (dict(ws=None), E_WS), (dict(wsb=1000), E_WS), (dict(ws=FAKE + 4), E_ALIGN),
    (dict(dos=S3(0, 0, 1 << 24)), E_SHAPE), (dict(dos=S3(0, 0, -128)), E_SHAPE), (dict(T=0, S=0, ws=None, wsb=0), OK),
])
def test_backward_refusals(kw, want):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, kr=FAKE, krs=None, out=FAKE, lse=FAKE, do=FAKE, dos=None, cq=None,
             ck=None, N=2, H=4, T=100, S=120, dn=128, dr=64, io=0, scale=0.1, dq=FAKE, dk=FAKE, dv=FAKE, dkr=FAKE, ws=FAKE,
             wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_latent_attn_bwd(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(table=None), E_NULL), (dict(lse=None), E_NULL), (dict(io=2), E_DTYPE), (dict(B=0), E_SHAPE),
    (dict(H=0), E_SHAPE), (dict(pages=0), E_SHAPE), (dict(page=0), E_SHAPE), (dict(max_pages=0), E_SHAPE),
    (dict(page=1 << 20, max_pages=1 << 12), E_SHAPE), (dict(dc=384), E_SHAPE), (dict(dr=32), E_SHAPE), (dict(scale=0.0), E_SCALE),
    (dict(cache=FAKE + 8), E_ALIGN), (dict(lengths=FAKE + 2), E_ALIGN), (dict(ws=None), E_WS), (dict(wsb=16), E_WS),
])
def test_decode_refusals(kw, want):
    a = dict(q=FAKE, cache=FAKE, table=FAKE, lengths=FAKE, B=2, H=16, pages=50, page=64, max_pages=20, dc=512, dr=64, io=0,
             scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_latent_decode_step(*a.values(), None) == want


def test_workspace_bytes():
    # delta, in whole 256 bytes, and the heads' float32 partials of the rotary part's gradient
    assert kda.latent_bwd_workspace_bytes(2, 4, 100, 120, 128, 64, torch.bfloat16) == 3328 + 2 * 4 * 120 * 64 * 4
    assert kda.latent_bwd_workspace_bytes(3, 4, 100, 120, 64, 32, torch.float32, packed=True) == 1792 + 4 * 120 * 32 * 4
    assert kda.latent_bwd_workspace_bytes(2, 4, 100, 120, 100, 64, torch.bfloat16) == 0
    # one part per 64 keys of the longest sequence, as long as the chip has room for it
    assert kda.latent_decode_workspace_bytes(2, 16, 64, 5, 512, 64, torch.bfloat16) == 2 * 5 * 16 * 513 * 4
    assert kda.latent_decode_workspace_bytes(1024, 128, 64, 100, 512, 64, torch.bfloat16) == 0
    assert kda.latent_decode_workspace_bytes(2, 16, 64, 1, 512, 64, torch.bfloat16) == 0


def test_binding_refusals():
    q, k, r = torch.zeros(1, 2, 8, 192), torch.zeros(1, 2, 8, 128), torch.zeros(1, 8, 64)
    cu = torch.zeros(2, dtype=torch.int32)
    for bad in ((q, k, k, r), (q.half(), k.half(), k.half(), r.half()), (q[..., :128], k, k, r), (q, k, k[..., :64], r), (q[0], k, k, r)):
        with pytest.raises(ValueError):
            kda.latent_attn_fwd(*bad)
    with pytest.raises(TypeError):
        kda.latent_attn_fwd(q, k, None, r)
    with pytest.raises(TypeError):
        kda.latent_attn_fwd_varlen(q[0], k[0], k[0], r[0], cu, None)
    with pytest.raises(ValueError):
        kda.latent_attn_fwd_varlen(q[0], k[0], k[0], r[0], cu, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.latent_attn_bwd(q, k, k, r, k, q[..., 0], k[:, :1])
    with pytest.raises(ValueError):
        kda.latent_decode_step(q[0], torch.zeros(4, 16, 192), torch.zeros(2, 4, dtype=torch.int32), cu, 0.1)
