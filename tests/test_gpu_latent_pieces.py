"""Drafted tokens over histories that many work-groups share, on the GPU: every tile of keys shows in the
result by itself (latent_pieces_util.py; test_latent_pieces_host.py shows what is noticed)."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import latent_pieces_util as P
from tests.test_gpu_latent_serving import BF, F32, HALF, attend, check

pytestmark = pytest.mark.gpu
SCALE = 0.07


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,dc,page,lens", [
    (1, 2, 8, 512, 64, [20011]), (1, 1, 1, 512, 16, [32768]), (1, 2, 8, 256, 64, [16384]),  # more pieces of a unit than a wave has lanes
    (1, 3, 21, 512, 64, [9001]), (2, 3, 20, 256, 1, [6001, 9]), (3, 2, 128, 512, 64, [3000, 1, 2500]), (5, 4, 16, 512, 7, [700, 64, 129, 0, 1000]),
    (24, 2, 24, 256, 64, [64 * (1 + 7 * i % 40) - i for i in range(24)]),
])
def test_every_tile_counts(B, T, H, dc, page, lens, dtype):
    gen = torch.Generator().manual_seed(7)
    mp = (max(lens) + page - 1) // page
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32)
    cache, q = torch.full((B * mp, page, dc + 64), float("nan"), dtype=dtype), P.queries(B, T, H, dc, dtype, gen)
    rows = [P.history(n, dc, dtype, gen) for n in lens]
    for b, n in enumerate(lens):
        j = torch.arange(n)
        cache[table[b, j // page].long(), j % page] = rows[b]
    mask = torch.tensor([[(2 << i) - 1 for i in range(T)]] * B, dtype=torch.int64)
    out, lse = kda.latent_tree_step(q.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), mask.cuda(), SCALE, dc=dc,
                                    return_lse=True)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        for i in range(T):
            seen = rows[b][:max(0, n - T + i + 1)]
            ref, tol, lref, _ = attend(q[b, i], seen, SCALE, dc, dtype)
            check(out[b, i], ref, tol, "out %d %d" % (b, i))
            check(lse[b, i], lref, P.lse_bound(q[b, i], seen, SCALE, lref), "lse %d %d" % (b, i))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [1e5, 1e9, 4e10, 1e14, 1e30])
@pytest.mark.parametrize("B,T,H,n", [(1, 1, 2, 30), (2, 3, 16, 700), (1, 2, 64, 1500)])
def test_scores_far_out(B, T, H, n, size, dtype):
    """Scores up to 1e30, whose steps are far above a float32's rounding of them: all weight is on the largest,
    wherever it stands, and the log-sum-exp is that score."""
    dc, page = 512, 64
    gen = torch.Generator().manual_seed(9)
    mp = (n + page - 1) // page
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32)
    rows = torch.randn(B, mp * page, dc + 64, generator=gen)
    # channel dc: 1, 2, .. 128 times size, in any order; two rows share the largest at most
    rows[..., dc:] = 0
    rows[..., dc] = torch.stack([torch.randperm(mp * page, generator=gen) % 128 for _ in range(B)]) * 1.0
    top = [int(torch.randint(0, n - T + 1, (1,), generator=gen)) for _ in range(B)]
    for b in range(B):
        rows[b, top[b], dc] = 160.0
    rows = rows.to(dtype)
    q = torch.zeros(B, T, H, dc + 64)
    q[..., dc] = size / 16
    q = q.to(dtype)
    cache = torch.empty(B * mp, page, dc + 64, dtype=dtype)
    cache[table.long().flatten()] = rows.reshape(B * mp, page, dc + 64)
    mask = torch.tensor([[(2 << i) - 1 for i in range(T)]] * B, dtype=torch.int64)
    scale = 0.07
    out, lse = kda.latent_tree_step(q.cuda(), cache.cuda(), table.cuda(), torch.full((B,), n, dtype=torch.int32).cuda(), mask.cuda(), scale, return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        want = rows[b, top[b], :dc].double().expand(T, H, dc)
        # the weight is one, rounded once more with the result; a score is rounded twice, its logarithm three times
        check(out[b], want, HALF[dtype] * want.abs() * 1.01 + 2.0 ** -22 * want.abs(), "out %d" % b)
        score = 160.0 * float(q[0, 0, 0, dc]) * scale
        check(lse[b], torch.full((T, H), score, dtype=torch.float64), torch.full((T, H), 2.0 ** -21 * score, dtype=torch.float64), "lse %d" % b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-38, 1e-6, 0.5])
def test_scales(scale, dtype):
    """From scales that leave every row the same weight on."""
    B, T, H, dc, page, n = 2, 3, 20, 256, 16, 500
    gen = torch.Generator().manual_seed(12)
    mp = -(-n // page)
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32)
    cache = torch.randn(B * mp, page, dc + 64, generator=gen).to(dtype)
    q = torch.randn(B, T, H, dc + 64, generator=gen).to(dtype)
    mask = torch.tensor([[1, 3, 5]] * B, dtype=torch.int64)
    out, lse = kda.latent_tree_step(q.cuda(), cache.cuda(), table.cuda(), torch.full((B,), n, dtype=torch.int32).cuda(), mask.cuda(), scale, dc=dc,
                                    return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        rows = cache[table[b].long()].reshape(-1, dc + 64)[:n]
        for i, see in enumerate(((0,), (0, 1), (0, 2))):
            ref, tol, lref, ltol = attend(q[b, i], rows[list(range(n - T)) + [n - T + j for j in see]], scale, dc, dtype)
            check(out[b, i], ref, tol, "out %d %d" % (b, i))
            check(lse[b, i], lref, ltol, "lse %d %d" % (b, i))
