"""Refusals of the gated delta rule's entry points, without a GPU: status codes of the C ABI before
anything is launched, and the binding's checks."""
import ctypes

import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first
OK, E_NULL, E_SHAPE, E_DTYPE, E_WS, E_ALIGN, E_SCALE = 0, -1, -2, -3, -6, -8, -11
S3 = ctypes.c_longlong * 3


def _fwd(**kw):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, g=FAKE, gs=None, b=FAKE, bs=None, cu=None, N=2, Hk=2, H=4,
             T=100, dk=128, dv=64, io=0, scale=1.0, s0=None, out=FAKE, fs=None, ws=FAKE, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return kda.lib().kda_gdr_chunk_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(v=None), E_NULL), (dict(b=None), E_NULL), (dict(out=None), E_NULL),
    (dict(io=3), E_DTYPE), (dict(N=0), E_SHAPE), (dict(Hk=0), E_SHAPE), (dict(H=0), E_SHAPE), (dict(Hk=3), E_SHAPE),
    (dict(T=-1), E_SHAPE), (dict(dk=96), E_SHAPE), (dict(dv=32), E_SHAPE), (dict(N=70000), E_SHAPE), (dict(H=70000), E_SHAPE),
    (dict(N=1 << 30, cu=FAKE), E_SHAPE), (dict(scale=float("nan")), E_SCALE), (dict(scale=float("inf")), E_SCALE),
    (dict(q=FAKE + 8), E_ALIGN), (dict(v=FAKE + 8), E_ALIGN), (dict(vs=S3(25600, 6400, 65)), E_ALIGN), (dict(g=FAKE + 1), E_ALIGN), (dict(cu=FAKE + 2), E_ALIGN),
    (dict(s0=FAKE + 8), E_ALIGN), (dict(fs=FAKE + 4), E_ALIGN), (dict(qs=S3(25600, 12800, 132)), E_ALIGN),
    (dict(ks=S3(25600, 4, 128)), E_ALIGN), (dict(io=1, ks=S3(0, 6, 128)), E_ALIGN),
    (dict(ws=None), E_WS), (dict(wsb=1000), E_WS), (dict(ws=FAKE + 8), E_ALIGN),
    (dict(T=0, q=None, k=None, v=None, g=None, b=None, out=None, ws=None, wsb=0), OK),
])
def test_forward_refusals(kw, want):
    assert _fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(state=None), E_NULL), (dict(io=2), E_DTYPE), (dict(B=0), E_SHAPE), (dict(Hk=3), E_SHAPE),
    (dict(dk=32), E_SHAPE), (dict(scale=float("nan")), E_SCALE), (dict(v=FAKE + 8), E_ALIGN), (dict(state=FAKE + 4), E_ALIGN),
])
def test_decode_refusals(kw, want):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, b=FAKE, B=2, Hk=2, H=4, dk=128, dv=128, io=0, scale=1.0, state=FAKE, out=FAKE)
    a.update(kw)
    assert kda.lib().kda_gdr_decode_step(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), E_NULL), (dict(do=None), E_NULL), (dict(dq=None), E_NULL), (dict(db=None), E_NULL), (dict(io=2), E_DTYPE),
    (dict(Hk=3), E_SHAPE), (dict(T=-5), E_SHAPE), (dict(dv=96), E_SHAPE), (dict(scale=float("inf")), E_SCALE),
    (dict(do=FAKE + 4), E_ALIGN), (dict(dos=S3(25600, 6400, 65)), E_ALIGN), (dict(dk_=FAKE + 8), E_ALIGN),
    (dict(df=FAKE + 4), E_ALIGN), (dict(ds=FAKE + 8), E_ALIGN), (dict(wsb=1 << 20), E_WS),
    (dict(T=0, q=None, k=None, v=None, g=None, b=None, do=None, dq=None, dk_=None, dv_=None, dg=None, db=None, ws=None, wsb=0), OK),
])
def test_backward_refusals(kw, want):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, g=FAKE, gs=None, b=FAKE, bs=None, do=FAKE, dos=None, cu=None,
             N=2, Hk=2, H=4, T=100, dk=128, dv=64, io=0, scale=1.0, s0=None, df=None, dq=FAKE, dk_=FAKE, dv_=FAKE, dg=FAKE,
             db=FAKE, ds=None, ws=FAKE, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_gdr_chunk_bwd(*a.values(), None) == want


def test_workspace_bytes():
    # key records: 256 bytes and the fp16 pieces of K and Q; value records: 1 KiB and the six causal
    # fragments of T (two pieces) and M
    key, val = 256 + 2 * 64 * 128 * 2, 1024 + 3 * 6144
    assert kda.gdr_workspace_bytes(2, 4, 8, 130, 128, 128, torch.bfloat16) == 2 * 3 * (4 * key + 8 * val)
    assert kda.gdr_workspace_bytes(5, 4, 8, 130, 128, 128, torch.bfloat16, packed=True) == 7 * (4 * key + 8 * val)
    key, val = 256 + 4 * 64 * 64 * 2, 1024 + 4 * 6144
    assert kda.gdr_workspace_bytes(1, 1, 1, 1, 64, 64, torch.float32) == key + val
    # backward: M in two pieces, and per 16 columns what the two passes keep
    key, val, kept = 256 + 2 * 64 * 128 * 2, 1024 + 4 * 6144, 256 + 4096 + 2048
    assert kda.gdr_workspace_bytes(2, 4, 8, 130, 128, 64, torch.bfloat16, backward=True) == \
        2 * 3 * (4 * key + 8 * (val + 2 * 4 * kept))
    assert kda.gdr_workspace_bytes(1, 3, 4, 64, 64, 64, torch.float32) == 0
    assert kda.gdr_workspace_bytes(1, 1, 1, 0, 64, 64, torch.float32) == 0


def test_binding_refusals():
    x = torch.zeros(1, 2, 8, 64)
    b = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd(x, x, x, b, b)  # host tensors
    with pytest.raises(TypeError):
        kda.gdr_chunk_fwd(x, x, None, b, b)
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd(x.half(), x.half(), x.half(), b.half(), b.half())
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd(x[0], x[0], x[0], b[0], b[0])
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd(x, x[:, :1], x, b, b)
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd(x.expand(1, 2, 8, 64), x, torch.zeros(1, 3, 8, 64), torch.zeros(1, 3, 8), torch.zeros(1, 3, 8))
    with pytest.raises(TypeError):
        kda.gdr_chunk_fwd_varlen(x[0], x[0], x[0], b[0], b[0], None)
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd_varlen(x[0], x[0], x[0], b[0], b[0], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.gdr_chunk_bwd(x, x, x, b, b, x[..., :32])
    with pytest.raises(TypeError):
        kda.gdr_chunk_bwd(x, x, x, b, b, None)
    with pytest.raises(ValueError):
        kda.gdr_decode_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], b[..., 0], b[..., 0], torch.zeros(1, 2, 64, 64))
