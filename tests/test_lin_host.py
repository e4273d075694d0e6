"""Refusals of decayed linear attention's entry points, without a GPU: status codes of the C ABI before
anything is launched, and the binding's checks."""
import ctypes

import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first
OK, E_NULL, E_SHAPE, E_DTYPE, E_WS, E_ALIGN, E_SCALE = 0, -1, -2, -3, -6, -8, -11
S3 = ctypes.c_longlong * 3
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(v=None), E_NULL), (dict(g=None), E_NULL), (dict(out=None), E_NULL),
    (dict(io=3), E_DTYPE), (dict(gt=2), E_DTYPE), (dict(io=1, gt=0), E_DTYPE), (dict(N=0), E_SHAPE), (dict(Hk=0), E_SHAPE),
    (dict(H=0), E_SHAPE), (dict(Hk=3), E_SHAPE), (dict(T=-1), E_SHAPE), (dict(dk=96), E_SHAPE), (dict(dv=32), E_SHAPE),
    (dict(N=70000), E_SHAPE), (dict(H=70000), E_SHAPE), (dict(N=1 << 30, cu=FAKE), E_SHAPE), (dict(scale=float("nan")), E_SCALE),
    (dict(scale=float("inf")), E_SCALE), (dict(q=FAKE + 8), E_ALIGN), (dict(v=FAKE + 8), E_ALIGN), (dict(vs=S3(25600, 6400, 65)), E_ALIGN),
    (dict(g=FAKE + 2), E_ALIGN), (dict(gt=0, g=FAKE + 1), E_ALIGN), (dict(cu=FAKE + 2), E_ALIGN), (dict(s0=FAKE + 8), E_ALIGN),
    (dict(fs=FAKE + 4), E_ALIGN), (dict(qs=S3(25600, 12800, 132)), E_ALIGN), (dict(ks=S3(25600, 4, 128)), E_ALIGN),
    (dict(io=1, ks=S3(0, 6, 128)), E_ALIGN), (dict(ks=S3(0, 0, -128)), E_SHAPE), (dict(vs=S3(0, 0, 1 << 24)), E_SHAPE),
    (dict(io=1, qs=S3(0, 0, 1 << 23)), E_SHAPE), (dict(T=3000, ws=None), E_WS), (dict(T=3000, wsb=1000), E_WS), (dict(ws=FAKE + 8), E_ALIGN),
    (dict(T=0, q=None, k=None, v=None, g=None, out=None, ws=None, wsb=0), OK),
])
def test_forward_refusals(kw, want):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, g=FAKE, gs=None, cu=None, N=2, Hk=2, H=4, T=100, dk=128, dv=64, io=0, gt=1,
             scale=1.0, s0=None, out=FAKE, fs=None, ws=FAKE, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_lin_chunk_fwd(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), E_NULL), (dict(do=None), E_NULL), (dict(dq=None), E_NULL), (dict(dv_=None), E_NULL), (dict(io=2), E_DTYPE),
    (dict(io=1, gt=0), E_DTYPE), (dict(Hk=3), E_SHAPE), (dict(T=-5), E_SHAPE), (dict(dv=96), E_SHAPE), (dict(scale=float("inf")), E_SCALE),
    (dict(do=FAKE + 4), E_ALIGN), (dict(dos=S3(25600, 6400, 65)), E_ALIGN), (dict(dos=S3(25600, 6400, -64)), E_SHAPE), (dict(dk_=FAKE + 8), E_ALIGN),
    (dict(dg=FAKE + 2), E_ALIGN), (dict(df=FAKE + 4), E_ALIGN), (dict(ds=FAKE + 8), E_ALIGN), (dict(wsb=1 << 18), E_WS),
    (dict(T=0, q=None, k=None, v=None, g=None, do=None, dq=None, dk_=None, dv_=None, dg=None), OK),
])
def test_backward_refusals(kw, want):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, g=FAKE, gs=None, do=FAKE, dos=None, cu=None, N=2, Hk=2, H=4, T=100, dk=128,
             dv=64, io=0, gt=1, scale=1.0, s0=None, df=None, dq=FAKE, dk_=FAKE, dv_=FAKE, dg=FAKE, ds=None, ws=FAKE, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_lin_chunk_bwd(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(state=None), E_NULL), (dict(io=2), E_DTYPE), (dict(io=1, gt=0), E_DTYPE), (dict(B=0), E_SHAPE),
    (dict(Hk=3), E_SHAPE), (dict(dk=32), E_SHAPE), (dict(scale=float("nan")), E_SCALE), (dict(v=FAKE + 8), E_ALIGN),
    (dict(state=FAKE + 4), E_ALIGN), (dict(g=FAKE + 2), E_ALIGN), (dict(B=1 << 21, Hk=1, H=1), E_SHAPE),
])
def test_one_token_refusals(kw, want):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, B=2, Hk=2, H=4, dk=128, dv=128, io=0, gt=1, scale=1.0, state=FAKE, out=FAKE)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_lin_decode_step(*a.values(), None) == want


def test_workspace_bytes():
    # one segment a sequence: none.  Else the segments' states and decays
    assert kda.lin_workspace_bytes(2, 4, 8, 256, 128, 128, BF) == 0
    assert kda.lin_workspace_bytes(2, 4, 8, 257, 128, 128, BF) == 2 * 8 * 5 * 128 * 128 * 4 + 2 * 8 * 5 * 4
    assert kda.lin_workspace_bytes(5, 4, 8, 300, 64, 128, BF, packed=True) == 9 * 8 * 64 * 128 * 4 + 9 * 8 * 4
    assert kda.lin_workspace_bytes(1, 3, 4, 64, 64, 64, F32) == 0
    assert kda.lin_workspace_bytes(1, 3, 4, 1000, 64, 64, F32) == 0  # 3 and 4 heads
    assert kda.lin_workspace_bytes(1, 1, 1, 1, 64, 64, F32, backward=True) > 2 * 64 * 64 * 4
    # value heads' float32 partials of dq and dk where key heads are shared
    a, b = (kda.lin_workspace_bytes(1, hk, 4, 640, 64, 64, BF, backward=True) for hk in (4, 2))
    assert b - a == 2 * 4 * 640 * 64 * 4


@pytest.mark.parametrize("N,H,T,packed,fits", [
    ((1 << 22) - 1, 1, 64, True, True), (1 << 22, 1, 64, True, False),                # 2^22 sequences and heads of 64 x 64
    (1, 1, (1 << 28) - 64, False, True), (1, 1, 1 << 28, False, False),                # 2^24 pieces of 16 tokens
])
def test_launch_limits(N, H, T, packed, fits):
    d = 64
    assert (kda.lin_workspace_bytes(N, 1, H, T, d, d, BF, packed=packed, backward=True) > 0) == fits


def test_binding_refusals():
    x, g = torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8)
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x, x, x, g)  # host tensors
    with pytest.raises(TypeError):
        kda.lin_chunk_fwd(x, x, None, g)
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x.half(), x.half(), x.half(), g.half())
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x, x, x, g.bfloat16())  # g below the other tensors' type
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x[0], x[0], x[0], g[0])
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x, x[:, :1], x, g)
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x, x, torch.zeros(1, 3, 8, 64), torch.zeros(1, 3, 8))
    with pytest.raises(TypeError):
        kda.lin_chunk_fwd_varlen(x[0], x[0], x[0], g[0], None)
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd_varlen(x[0], x[0], x[0], g[0], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.lin_chunk_bwd(x, x, x, g, x[..., :32])
    with pytest.raises(TypeError):
        kda.lin_chunk_bwd(x, x, x, g, None)
    with pytest.raises(TypeError):
        kda.lin_chunk_bwd_varlen(x[0], x[0], x[0], g[0], x[0], None)
    with pytest.raises(ValueError):
        kda.lin_decode_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g[..., 0], torch.zeros(1, 2, 64, 64))


def test_leaves_are_not_captured(monkeypatch):
    """A leaf gathers its gradient on another stream than the captured one where an eager graph of it lives."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    x, g = torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8)
    with pytest.raises(RuntimeError, match="leaf"):
        kda.LinChunkFunction.apply(x, x, x.clone().requires_grad_(), g)
    with pytest.raises(ValueError):  # none: as far as the check of the device
        kda.LinChunkFunction.apply(x, x, x.clone().requires_grad_() * 1, g)
