"""Refusals of the paged latent cache's writer and of drafted tokens' attention, without a GPU: status codes
of the C ABI before anything is launched, and the binding's checks."""
import ctypes

import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first
OK, E_NULL, E_SHAPE, E_DTYPE, E_WS, E_ALIGN, E_SCALE = 0, -1, -2, -3, -6, -8, -11
S3 = ctypes.c_longlong * 3
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("kw,want", [
    (dict(lat=None), E_NULL), (dict(kr=None), E_NULL), (dict(cache=None), E_NULL), (dict(table=None), E_NULL), (dict(lengths=None), E_NULL),
    (dict(freqs=None), E_NULL), (dict(qr=None), E_NULL), (dict(q=None), E_NULL), (dict(cu=FAKE, counts=FAKE), E_NULL),
    (dict(io=2), E_DTYPE), (dict(N=0), E_SHAPE), (dict(T=-1), E_SHAPE), (dict(H=-1), E_SHAPE), (dict(H=70000), E_SHAPE), (dict(pages=0), E_SHAPE),
    (dict(page=0), E_SHAPE), (dict(mp=0), E_SHAPE), (dict(mp=1 << 30), E_SHAPE), (dict(dc=128), E_SHAPE), (dict(dr=32), E_SHAPE),
    (dict(T=1 << 26), E_SHAPE), (dict(eps=float("nan")), E_SCALE), (dict(eps=-1e-6), E_SCALE), (dict(eps=float("inf")), E_SCALE),
    (dict(lat=FAKE + 8), E_ALIGN), (dict(kr=FAKE + 8), E_ALIGN), (dict(ls=S3(0, 0, 513)), E_ALIGN), (dict(ks=S3(4, 0, 64)), E_ALIGN),
    (dict(qs=S3(0, 68, 640)), E_ALIGN), (dict(io=1, ls=S3(0, 0, 514)), E_ALIGN), (dict(cache=FAKE + 8), E_ALIGN), (dict(w=FAKE + 2), E_ALIGN),
    (dict(q=FAKE + 8), E_ALIGN), (dict(pos=FAKE + 2), E_ALIGN), (dict(counts=FAKE + 1), E_ALIGN), (dict(cu=FAKE + 2, counts=None), E_ALIGN),
    (dict(T=0, lat=None, kr=None, qr=None, q=None), OK),
])
def test_append_refusals(kw, want):
    a = dict(lat=FAKE, ls=None, kr=FAKE, ks=None, cache=FAKE, table=FAKE, lengths=FAKE, freqs=FAKE, w=FAKE, eps=1e-6, pos=None, counts=None, qr=FAKE,
             qs=None, q=FAKE, cu=None, N=2, T=10, H=4, pages=8, page=16, mp=4, dc=512, dr=64, io=0, inter=1)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_latent_append(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E_NULL), (dict(cache=None), E_NULL), (dict(table=None), E_NULL), (dict(lengths=None), E_NULL), (dict(mask=None), E_NULL),
    (dict(out=None), E_NULL), (dict(lse=None), E_NULL), (dict(io=2), E_DTYPE), (dict(B=0), E_SHAPE), (dict(B=70000), E_SHAPE), (dict(T=0), E_SHAPE),
    (dict(T=65), E_SHAPE), (dict(H=0), E_SHAPE), (dict(H=70000), E_SHAPE), (dict(pages=0), E_SHAPE), (dict(page=0), E_SHAPE), (dict(mp=0), E_SHAPE),
    (dict(mp=1 << 30), E_SHAPE), (dict(dc=128), E_SHAPE), (dict(dr=32), E_SHAPE), (dict(B=65535, T=64, H=65535), E_SHAPE),
    (dict(scale=0.0), E_SCALE), (dict(scale=float("nan")), E_SCALE), (dict(q=FAKE + 8), E_ALIGN), (dict(cache=FAKE + 4), E_ALIGN),
    (dict(mask=FAKE + 4), E_ALIGN), (dict(counts=FAKE + 2), E_ALIGN), (dict(out=FAKE + 8), E_ALIGN), (dict(lse=FAKE + 2), E_ALIGN),
    (dict(ws=None), E_WS), (dict(wsb=100), E_WS), (dict(ws=FAKE + 8), E_ALIGN),
])
def test_tree_refusals(kw, want):
    a = dict(q=FAKE, cache=FAKE, table=FAKE, lengths=FAKE, counts=None, mask=FAKE, B=2, T=4, H=16, pages=99, page=64, mp=40, dc=512, dr=64, io=0,
             scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    assert kda.lib().kda_latent_tree_step(*a.values(), None) == want


def test_tree_workspace_bytes():
    # nothing from 1024 units (of 64 rows) on, and where a last round of units leaves few CUs idle; else two
    # units' rows of out and lse for each of up to 256 work-groups, and the sequences' first tiles
    assert kda.latent_tree_workspace_bytes(64, 32, 128, 64, 40, 512, 64, BF) == 0
    assert kda.latent_tree_workspace_bytes(16, 32, 128, 64, 40, 512, 64, BF) == 0
    assert kda.latent_tree_workspace_bytes(12, 32, 128, 64, 40, 512, 64, BF) == 0
    assert kda.latent_tree_workspace_bytes(13, 32, 128, 64, 40, 512, 64, BF) == 2 * 256 * 64 * 513 * 4 + 15 * 4
    # few tiles: 16 rows a unit, and no more work-groups than tiles
    assert kda.latent_tree_workspace_bytes(1, 5, 16, 64, 40, 512, 64, BF) == 2 * 200 * 16 * 513 * 4 + 3 * 4
    assert kda.latent_tree_workspace_bytes(1, 1, 3, 64, 1, 256, 64, F32) == 0  # one tile
    assert kda.latent_tree_workspace_bytes(1, 65, 16, 64, 40, 512, 64, BF) == 0


def test_binding_refusals():
    lat, kr, cache = torch.zeros(2, 3, 512), torch.zeros(2, 3, 64), torch.zeros(9, 16, 576)
    table, lengths, freqs = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(32)
    args = (lat, kr, cache, table, lengths, freqs)
    for bad, at in ((None, 0), (None, 2), (None, 3)):
        with pytest.raises(TypeError):
            kda.latent_append(*(bad if i == at else t for i, t in enumerate(args)))
    with pytest.raises(ValueError):
        kda.latent_append(*args)  # host tensors
    with pytest.raises(ValueError):
        kda.latent_append(lat.half(), kr.half(), cache.half(), table, lengths, freqs)
    with pytest.raises(ValueError):
        kda.latent_append(lat[:1], kr, *args[2:])
    with pytest.raises(ValueError):
        kda.latent_append(lat[..., :256], kr, *args[2:])
    with pytest.raises(ValueError):
        kda.latent_append(*args, q_rope=torch.zeros(2, 3, 4, 64))  # and no q
    with pytest.raises(ValueError):
        kda.latent_append(*args, q_rope=torch.zeros(2, 4, 4, 64), q=torch.zeros(2, 3, 4, 576))
    with pytest.raises(TypeError):
        kda.latent_append_varlen(lat[0], kr[0], *args[2:], None)
    with pytest.raises(ValueError):
        kda.latent_append_varlen(*args, torch.zeros(3, dtype=torch.int32))
    q, mask = torch.zeros(2, 3, 4, 576), torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError):
        kda.latent_tree_step(q, cache, table, lengths, mask, 0.1)
    with pytest.raises(TypeError):
        kda.latent_tree_step(q, cache, table, lengths, None, 0.1)
    with pytest.raises(ValueError):
        kda.latent_tree_step(q[0], cache, table, lengths, mask, 0.1)
