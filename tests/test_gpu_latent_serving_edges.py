"""The paged latent cache on the GPU outside the ordinary: odd views, caches beyond 32-bit offsets, long
histories in many pieces, many short sequences, workspaces that hold anything, streams; and a decoder's
layers together, linear attention's state beside the latent cache.  Bounds as in
test_gpu_latent_serving.py and lin_util.py."""
import math

import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import lin_util as U
from tests.test_gpu_latent_serving import BF, F32, HALF, attend, case, check, normed, run_tree, tree, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def paged(B, mp, page, dc, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32).cuda()
    return table, torch.randn(B * mp, page, dc + 64, generator=gen).to(dtype).cuda(), gen


# ------------------------------------------------------------------------------------- appending


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_append_odd_views(interleaved, dtype):
    """The queries' rotary part turned where it lies; latents backwards in memory, broadcast keys, strides of
    dimensions of one: the same bits as from copies."""
    B, T, H, dc, page = 2, 5, 40, 256, 8
    _, qfull, freqs, weight, gen = case(B, T, H, dc, dtype, 7)
    table, cache, _ = paged(B, 4, page, dc, dtype, 8)
    lengths = torch.tensor([9, 5], dtype=torch.int32).cuda()
    lat = torch.randn(B, T, dc, generator=gen).to(dtype).cuda()
    kr = torch.randn(64, generator=gen).to(dtype).cuda().expand(B, T, 64)
    back = lat.flip(0, 1).contiguous()
    # (torch has no negative strides: those go to the library below)
    wide = torch.empty(B, T, 3, dc, dtype=dtype).cuda()
    wide[:, :, 1] = lat
    q = torch.randn(B, T, H, dc + 64, generator=gen).to(dtype).cuda()
    q1, q2, c1, c2 = q.clone(), q.clone(), cache.clone(), cache.clone()
    kda.latent_append(wide[:, :, 1], kr, c1, table, lengths, freqs.cuda(), norm_weight=weight.cuda(), interleaved=interleaved, q_rope=q1[..., dc:], q=q1)
    kda.latent_append(lat, kr.contiguous(), c2, table, lengths, freqs.cuda(), norm_weight=weight.cuda(), interleaved=interleaved,
                      q_rope=q[..., dc:].contiguous(), q=q2)
    torch.cuda.synchronize()
    assert torch.equal(c1, c2) and torch.equal(q1, q2) and torch.equal(q1[..., :dc], q[..., :dc]) and not torch.equal(c1, cache)
    # backwards in memory, through the library's own strides
    c3, q3 = cache.clone(), q.clone()
    S3, size = kda.gdr._S3, back.element_size()
    fd, wd, qr = freqs.cuda(), weight.cuda(), q[..., dc:].contiguous()  # held: the call takes their addresses
    st = kda.lib().kda_latent_append(
        back.data_ptr() + (B * T - 1) * dc * size, S3(-T * dc, 0, -dc), kr.data_ptr(), S3(0, 0, 0), c3.data_ptr(), table.data_ptr(),
        lengths.data_ptr(), fd.data_ptr(), wd.data_ptr(), 1e-6, None, None, qr.data_ptr(), None,
        q3.data_ptr(), None, B, T, H, cache.shape[0], page, 4, dc, 64, int(dtype == F32), int(interleaved),
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(c3, c2) and torch.equal(q3, q2)
    one = lat[:1, :1].as_strided((1, 1, dc), (13, 7, 1))
    c4, c5 = cache.clone(), cache.clone()
    kda.latent_append(one, kr[:1, :1], c4, table[:1], lengths[:1], freqs.cuda(), interleaved=interleaved)
    kda.latent_append(lat[:1, :1].contiguous(), kr[:1, :1].contiguous(), c5, table[:1], lengths[:1], freqs.cuda(), interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(c4, c5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_positions_and_norms_far_out(dtype):
    """Positions from the least to the greatest of int32; rows of zeros, of tiny and of large values."""
    B, T, dc, page = 1, 6, 512, 16
    _, _, freqs, weight, gen = case(B, T, 0, dc, dtype, 11)
    table, cache, _ = paged(B, 1, page, dc, dtype, 12)
    x = torch.randn(B, T, dc + 64, generator=gen)
    x = (x * torch.tensor([0.0, 1e-18, 1e-3, 1.0, 1e3, 1e15])[None, :, None]).to(dtype)
    pos = torch.tensor([[-2 ** 31, -1, 0, 1, 2 ** 24 + 1, 2 ** 31 - 1]], dtype=torch.int32)
    xd = x.cuda()
    kda.latent_append(xd[..., :dc], xd[..., dc:], cache, table, torch.tensor([T], dtype=torch.int32).cuda(), freqs.cuda(), norm_weight=weight.cuda(),
                      eps=1e-6, positions=pos.cuda())
    torch.cuda.synchronize()
    for i in range(T):
        row = cache[int(table[0, 0]), i]
        check(row[:dc], *normed(x[0, i, :dc], weight, 1e-6, dtype), "latent %d" % i)
        check(row[dc:], *turned(x[0, i, dc:], pos[0, i], freqs, True, dtype), "rotary %d" % i)


def test_append_shows_what_is_not_finite():
    """A NaN in a token: its own row (a NaN in the latent: all of it that is normalised)."""
    B, T, dc, page = 1, 4, 256, 16
    x, _, freqs, weight, _ = case(B, T, 0, dc, BF, 13)
    table, cache, _ = paged(B, 1, page, dc, BF, 14)
    x[0, 1, 3], x[0, 2, dc + 10] = float("nan"), float("inf")
    xd = x.cuda()
    kda.latent_append(xd[..., :dc], xd[..., dc:], cache, table, torch.tensor([T], dtype=torch.int32).cuda(), freqs.cuda(), norm_weight=weight.cuda())
    rows = cache[int(table[0, 0])]
    assert torch.isnan(rows[1, :dc]).all() and torch.isfinite(rows[1, dc:]).all()
    bad = ~torch.isfinite(rows[2])
    assert bool(bad[dc + 10] | bad[dc + 11]) and int(bad.sum()) <= 2 and torch.isfinite(rows[[0, 3]]).all()


# ------------------------------------------------------------------------------------- large, long, many


def test_beyond_32_bit_offsets():
    """A cache of more than 2^31 elements: rows written on its last pages, read by drafted tokens."""
    dc, page, H, T = 512, 64, 16, 3
    pages = (1 << 31) // (page * (dc + 64)) + 9
    cache = torch.empty(pages, page, dc + 64, dtype=BF, device="cuda")
    gen = torch.Generator().manual_seed(2)
    n = 3 * page + 5
    table = torch.tensor([[pages - 1, 0, pages - 3, pages - 2]], dtype=torch.int32).cuda()
    x = torch.randn(1, n, dc + 64, generator=gen).to(BF)
    xd, freqs, lengths = x.cuda(), torch.zeros(32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    kda.latent_append(xd[..., :dc], xd[..., dc:], cache, table, lengths, freqs)
    torch.cuda.synchronize()
    for j in (0, page, 2 * page + 1, n - 1):  # frequencies of zero: rows as they were
        assert torch.equal(cache[int(table[0, j // page]), j % page].cpu(), x[0, j])
    q = (torch.randn(1, T, H, dc + 64, generator=gen) * 0.5).to(BF)
    out, lse = kda.latent_tree_step(q.cuda(), cache, table, lengths, torch.tensor([[1, 3, 5]]).cuda(), 0.07, return_lse=True)
    torch.cuda.synchronize()
    for i, see in enumerate(((0,), (0, 1), (0, 2))):
        ref, tol, lref, ltol = attend(q[0, i], x[0, list(range(n - T)) + [n - T + j for j in see]], 0.07, dc, BF)
        check(out[0, i], ref, tol, "out %d" % i)
        check(lse[0, i], lref, ltol, "lse %d" % i)


@pytest.mark.parametrize("dtype,B,T,H,dc,page,lens", [
    (BF, 1, 2, 8, 512, 64, [20011]),            # one unit in more pieces than a wave has lanes
    (BF, 2, 3, 20, 256, 1, [6001, 9]),
    (F32, 1, 2, 16, 512, 64, [9001]),
    (BF, 3, 2, 128, 512, 64, [3000, 1, 2500]),  # units of 64 rows that end inside work-groups' shares
])
def test_tree_long_history(dtype, B, T, H, dc, page, lens):
    run_tree(B, T, H, dc, page, lens, dtype, 31)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_many_short_sequences(dtype):
    """As many units as fill the card: a work-group each, no pieces."""
    B, T, H, dc, page, mp = 1030, 2, 3, 256, 8, 3
    table, cache, gen = paged(B, mp, page, dc, dtype, 41)
    lengths = torch.randint(0, mp * page + 1, (B,), generator=gen, dtype=torch.int32)
    q = (torch.randn(B, T, H, dc + 64, generator=gen) * 0.5).to(dtype)
    mask = torch.tensor([[1, 3]] * B, dtype=torch.int64).cuda()
    assert kda.latent_tree_workspace_bytes(B, T, H, page, mp, dc, 64, dtype) == 0
    out, lse = kda.latent_tree_step(q.cuda(), cache, table, lengths.cuda(), mask, 0.07, dc=dc, return_lse=True)
    torch.cuda.synchronize()
    rows = cache.cpu()[table.cpu().long()].reshape(B, mp * page, dc + 64)
    for b in (0, 1, 2, 500, 777, B - 2, B - 1):
        n = int(lengths[b])
        for i in range(T):
            see = [j for j in range(n) if j <= n - T + i]
            ref, tol, lref, ltol = attend(q[b, i], rows[b, see], 0.07, dc, dtype)
            check(out[b, i], ref, tol, "out %d %d" % (b, i))
            check(lse[b, i], lref, ltol, "lse %d %d" % (b, i))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_workspace_streams_and_same_bits(dtype):
    """A workspace of NaN, larger than needed, gives a fresh one's bits; two calls at once on two streams too."""
    B, T, H, dc, page, mp = 2, 5, 20, 512, 16, 40
    table, cache, gen = paged(B, mp, page, dc, dtype, 51)
    lengths = torch.tensor([600, 77], dtype=torch.int32).cuda()
    qs = [(torch.randn(B, T, H, dc + 64, generator=gen) * 0.5).to(dtype).cuda() for _ in range(2)]
    mask = torch.tensor([tree(T, gen)[1] for _ in range(B)], dtype=torch.int64).cuda()
    step = lambda q, **kw: kda.latent_tree_step(q, cache, table, lengths, mask, 0.07, return_lse=True, **kw)
    want = [step(q) for q in qs]
    need = kda.latent_tree_workspace_bytes(B, T, H, page, mp, dc, 64, dtype)
    assert need > 0
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    got = [step(q, workspace=ws) for q in qs]
    torch.cuda.synchronize()
    assert bool((ws[need:] == 255).all())
    streams = [torch.cuda.Stream() for _ in qs]
    there = [step(q, stream=s) for q, s in zip(qs, streams)]
    torch.cuda.synchronize()
    for a in (got, there):
        assert all(torch.equal(x, y) for g, w in zip(a, want) for x, y in zip(g, w))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_large_scores(dtype):
    """Scores of hundreds whose maximum grows along the history, and one key that outweighs all."""
    B, T, H, dc, page, n = 1, 2, 24, 256, 64, 900
    table, cache, gen = paged(B, 15, page, dc, dtype, 61)
    grow = torch.linspace(0.1, 8, 15 * page).reshape(15, page, 1)
    cache[table[0].long()] = (cache[table[0].long()].cpu() * grow).to(dtype).cuda()
    q = torch.randn(B, T, H, dc + 64, generator=gen).to(dtype)
    out, lse = kda.latent_tree_step(q.cuda(), cache, table, torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([[1, 3]]).cuda(), 1.0,
                                    dc=dc, return_lse=True)
    torch.cuda.synchronize()
    rows = cache.cpu()[table[0].cpu().long()].reshape(-1, dc + 64)
    for i in range(T):
        ref, tol, lref, ltol = attend(q[0, i], rows[:n - T + i + 1], 1.0, dc, dtype)
        check(out[0, i], ref, tol, "out %d" % i)
        check(lse[0, i], lref, ltol, "lse %d" % i)


# ------------------------------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", [BF, F32])
def test_hybrid_decoder(dtype):
    """A layer of linear attention, whose output is projected into a layer of latent attention: two prompts
    packed, then four drafted tokens a sequence, of which the first two stay, then a plain token.  Every
    kernel's result against float64 of what it was given; the drafted tokens' linear states come from the
    prompts' by the one-token step."""
    H, d, dc, Hq, page, scale, lens = 2, 64, 256, 8, 16, 0.07, [70, 19]
    B, D, dev = len(lens), 2 * 64, "cuda"
    gen = torch.Generator().manual_seed(71)
    cu = [0, lens[0], sum(lens)]
    wl, wq = ((torch.randn(D, n, generator=gen) * D ** -0.5).to(dtype).to(dev) for n in (dc + 64, Hq * (dc + 64)))
    freqs, weight = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float(), torch.ones(dc, dtype=dtype)
    table, cache, _ = paged(B, 8, page, dc, dtype, 72)
    q, k, v, g = U.inputs(0, H, H, cu[-1] + 5 * B, d, d, dtype, 73, packed=True)
    x = [t.to(dev) for t in (q, k, v, g)]
    # the linear layer over the prompts
    out, S = kda.lin_chunk_fwd_varlen(*(t[:, :cu[-1]] for t in x), torch.tensor(cu, dtype=torch.int32).cuda(), scale=scale, return_final_state=True)
    want = {}
    for b in range(B):
        s = slice(cu[b], cu[b + 1])
        for h in range(H):
            want[b, h] = U.one(q[h, s], k[h, s], v[h, s], g[h, s], scale, dtype, dtype)
            U.check(out[h, s], *want[b, h]["out"], "prompt %d %d" % (b, h))
            U.check(S[b, h], *want[b, h]["final_state"], "state %d %d" % (b, h))
    # into the cache
    hid = out.transpose(0, 1).reshape(-1, D)
    lat = hid @ wl
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()
    kda.latent_append_varlen(lat[:, :dc], lat[:, dc:], cache, table, lengths, freqs.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                             norm_weight=weight.cuda())
    place = lambda b, j: (int(table[b, j // page]), j % page)
    for b in range(B):
        for j in (0, lens[b] - 1):
            row = cache[place(b, j)]
            check(row[:dc], *normed(lat[cu[b] + j, :dc].cpu(), weight, 1e-6, dtype), "latent %d %d" % (b, j))
            check(row[dc:], *turned(lat[cu[b] + j, dc:].cpu(), torch.tensor(float(j)), freqs, True, dtype), "rotary %d %d" % (b, j))

    def tokens(state, first, n):
        """n tokens a sequence from number `first` on through the linear layer; [B,n,D] and the states."""
        hs = []
        for i in range(first, first + n):
            at = [cu[-1] + 5 * b + i for b in range(B)]
            y = [t[:, at].transpose(0, 1).contiguous() for t in x]
            hs.append(kda.lin_decode_step(*y, state, scale=scale).reshape(B, 1, D))
        return torch.cat(hs, 1), state

    # four drafted tokens: 0 - 1 - 2 and 0 - 3, all of the same linear state here
    T, bits, depth = 4, [1, 3, 7, 9], [0, 1, 2, 1]
    before = S.clone()
    hid, _ = tokens(S.clone(), 0, T)
    new = hid @ wl
    qq = (hid @ wq).reshape(B, T, Hq, dc + 64)
    pos = (lengths[:, None] + torch.tensor(depth, dtype=torch.int32).cuda()).contiguous()
    raw = qq.clone()
    kda.latent_append(new[..., :dc], new[..., dc:], cache, table, lengths + T, freqs.cuda(), norm_weight=weight.cuda(), positions=pos,
                      q_rope=qq[..., dc:], q=qq)
    mask = torch.tensor([bits] * B, dtype=torch.int64).cuda()
    o, lse = kda.latent_tree_step(qq, cache, table, lengths + T, mask, scale, dc=dc, return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        rows = torch.stack([cache[place(b, j)] for j in range(lens[b] + T)]).cpu()
        for i in range(T):
            check(qq[b, i, :, dc:], *turned(raw[b, i, :, dc:].cpu(), pos[b, i].cpu().expand(Hq), freqs, True, dtype), "q %d %d" % (b, i))
            see = list(range(lens[b])) + [lens[b] + j for j in range(T) if bits[i] >> j & 1]
            ref, tol, lref, ltol = attend(qq[b, i].cpu(), rows[see], scale, dc, dtype)
            check(o[b, i], ref, tol, "out %d %d" % (b, i))
            check(lse[b, i], lref, ltol, "lse %d %d" % (b, i))
    # the first two stay: their rows are in place; the state goes on from the prompt's; one more token
    assert torch.equal(S, before)
    _, S = tokens(S, 0, 2)
    hid, S = tokens(S, 4, 1)
    now = lengths + 3
    new, qq = hid @ wl, (hid @ wq).reshape(B, 1, Hq, dc + 64)
    kda.latent_append(new[..., :dc], new[..., dc:], cache, table, now, freqs.cuda(), norm_weight=weight.cuda(), q_rope=qq[..., dc:], q=qq)
    o, lse = kda.latent_decode_step(qq[:, 0].contiguous(), cache, table, now, scale, dc=dc, return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        rows = torch.stack([cache[place(b, j)] for j in range(lens[b] + 3)]).cpu()
        ref, tol, lref, ltol = attend(qq[b, 0].cpu(), rows, scale, dc, dtype)
        check(o[b], ref, tol, "plain out %d" % b)
        check(lse[b], lref, ltol, "plain lse %d" % b)
        sel = [cu[-1] + 5 * b + i for i in (0, 1, 4)]
        for h in range(H):
            y = [torch.cat([t[h, cu[b]:cu[b + 1]], t[h, sel]]) for t in (q, k, v, g)]
            U.check(S[b, h], *U.one(*y, scale, dtype, dtype)["final_state"], "state at the end %d %d" % (b, h))
