"""Latent attention on the GPU outside the ordinary: values that are not finite, long histories in many
parts, views with rows further apart than they are long, large scores.  Bounds as in test_gpu_latent.py."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from test_gpu_latent import _check, _check_all, inputs, one, split

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


@pytest.mark.parametrize("pages", [1, 5])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_absorbed_shows_what_is_not_finite(dtype, pages):
    """One part and several (64 rows each): a NaN or a score that overflows, in a query or in one row of
    the cache inside the length, makes that head's or that sequence's outputs NaN; the others keep theirs."""
    B, H, dc, page = 5, 16, 256, 64
    gen = torch.Generator().manual_seed(pages)
    cache = torch.randn(B * pages, page, dc + 64, generator=gen).to(dtype)
    q = (torch.randn(B, H, dc + 64, generator=gen) * 0.5).to(dtype)
    table = torch.arange(B * pages).reshape(B, pages).to(torch.int32)
    n = pages * page - 3
    at = 64 * (pages // 2) + 9
    dirty, dq = cache.clone(), q.clone()
    dirty[table[1, at // page].long(), at % page, 300] = NAN
    dirty[table[2, at // page].long(), at % page, 7] = INF
    dirty[table[3, at // page].long(), at % page] = 1e30
    dq[3, 0], dq[3, 1:] = 1e30, 1e-30
    dq[4, 2, 11] = NAN
    out, lse = kda.latent_decode_step(dq.cuda(), dirty.cuda(), table.cuda(), torch.full((B,), n, dtype=torch.int32, device="cuda"), 0.07,
                                      dc=dc, return_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(out[2]).any(-1).all() and not torch.isfinite(out[2, :, 7]).any()
    assert torch.isnan(out[3, 0]).all() and torch.isnan(lse[3, 0])
    assert torch.isnan(out[4, 2]).all() and torch.isnan(lse[4, 2])
    rows = cache.reshape(B, -1, dc + 64)[:, :n]
    for b, h in ((0, 0), (0, 15), (4, 1), (4, 3)):
        ref = one(q[b, h][None], rows[b], rows[b][:, :dc], 0.07, dtype)
        _check(out[b, h][None], *ref["out"], "out %d %d" % (b, h))
        _check(lse[b, h][None], *ref["lse"], "lse %d %d" % (b, h))


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_expanded_shows_what_is_not_finite(dtype, T):
    """A NaN in a query: NaN in that row's output and log-sum-exp, the other rows as they are."""
    q, kv, r, _ = inputs((1,), 2, T, T, 64, 32, dtype, T)
    k, v = split(kv, 64)
    dirty = q.clone()
    dirty[0, 1, 17, 3] = NAN
    out, lse = kda.latent_attn_fwd(dirty.cuda(), *split(kv.cuda(), 64), r.cuda(), return_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 1, 17]).all() and torch.isnan(lse[0, 1, 17])
    for h in range(2):
        ref = one(q[0, h], torch.cat([k[0, h], r[0]], -1), v[0, h], 96 ** -0.5, dtype)
        keep = [i for i in range(T) if (h, i) != (1, 17)]
        _check(out[0, h, keep], *(t[keep] for t in ref["out"]), "out")
        _check(lse[0, h, keep], *(t[keep] for t in ref["lse"]), "lse")


def test_second_derivatives_are_refused():
    q, kv, r, _ = inputs((1,), 1, 40, 40, 64, 32, F32, 3)
    leaf = [t.cuda().requires_grad_() for t in (q, *(t.contiguous() for t in split(kv, 64)), r)]
    first = torch.autograd.grad(kda.LatentAttnFunction.apply(*leaf).square().sum(), leaf[2], create_graph=True)[0]
    with pytest.raises(RuntimeError):
        (first.square().sum() + leaf[0].sum()).backward()


@pytest.mark.parametrize("T,dims", [(70, (0, 1)), (1, (0, 2))])
def test_strides_of_dimensions_of_one(T, dims):
    """A stride of 13 in dimensions of one: no row's start depends on it."""
    H = 1 if 1 in dims else 3
    q, kv, r, do = inputs((1,), H, T, T, 64, 32, BF, 5)
    a = [t.cuda().contiguous() for t in (q, *split(kv, 64), r, do)]
    loose = lambda t, d: t.as_strided(t.shape, [13 if i in d else s for i, s in enumerate(t.stride())])
    b = [loose(t, dims if t.dim() == 4 else (0,)) for t in a]
    got = []
    for x in (a, b):
        out, lse = kda.latent_attn_fwd(*x[:4], return_lse=True)
        got.append([out, lse, *kda.latent_attn_bwd(*x[:4], out, lse, x[4]).values()])
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(*got))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,S", [(70, 70), (40, 200)])
def test_wide_rows(T, S, dtype):
    """k_rope as a slice of the down-projection's output [B,S,dc+dr], q as one of wider rows, dout
    transposed from [B,T,H,d]."""
    dn, dr, dc, B, H = 128, 64, 96, 2, 3
    q, kv, r, do = inputs((B,), H, T, S, dn, dr, dtype, 31)
    gen = torch.Generator().manual_seed(1)
    down = torch.randn(B, S, dc + dr, generator=gen).to(dtype)
    down[..., dc:] = r
    qw = torch.randn(B, T, H, dn + dr + 32, generator=gen).to(dtype)
    qw[..., :dn + dr] = q.transpose(1, 2)
    k, v = split(kv, dn)
    dev = (qw.cuda()[..., :dn + dr].transpose(1, 2), *split(kv.cuda(), dn), down.cuda()[..., dc:])
    dd = do.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    assert not any(t.is_contiguous() for t in (*dev, dd))
    out, lse = kda.latent_attn_fwd(*dev, return_lse=True)
    g = kda.latent_attn_bwd(*dev, out, lse, dd)
    torch.cuda.synchronize()
    for b in range(B):
        _check_all(q[b], k[b], v[b], r[b], do[b], (dn + dr) ** -0.5, dtype, out[b], lse[b], {n: t[b] for n, t in g.items()}, "%d " % b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,n", [(1, 16, 9000), (2, 5, 4500)])
def test_absorbed_long_history(B, H, n, dtype):
    """One or two users with more rows than the largest number of parts has 64-row shares of."""
    dc, page = 512, 64
    gen = torch.Generator().manual_seed(n)
    M = -(-n // page)
    cache = torch.randn(B * M, page, dc + 64, generator=gen).to(dtype)
    table = torch.randperm(B * M, generator=gen).reshape(B, M)
    q = (torch.randn(B, H, dc + 64, generator=gen) * 0.5).to(dtype)
    lens = [n - 777 * b for b in range(B)]
    out, lse = kda.latent_decode_step(q.cuda(), cache.cuda(), table.to(torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.07,
                                      dc=dc, return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        rows = cache[table[b]].reshape(-1, dc + 64)[:lens[b]]
        for h in (0, H - 1):
            ref = one(q[b, h][None], rows, rows[:, :dc], 0.07, dtype)
            _check(out[b, h][None], *ref["out"], "out %d %d" % (b, h))
            _check(lse[b, h][None], *ref["lse"], "lse %d %d" % (b, h))


def test_large_scores():
    """Scores of a few hundred with bf16 inputs: one or two keys have all of a row's weight."""
    q, kv, r, do = inputs((1,), 2, 200, 200, 128, 64, BF, 5)
    q = q * 32
    k, v = split(kv, 128)
    dev = (q.cuda(), *split(kv.cuda(), 128), r.cuda())
    out, lse = kda.latent_attn_fwd(*dev, return_lse=True)
    g = kda.latent_attn_bwd(*dev, out, lse, do.cuda())
    torch.cuda.synchronize()
    _check_all(q[0], k[0], v[0], r[0], do[0], 192 ** -0.5, BF, out[0], lse[0], {n: t[0] for n, t in g.items()})
