"""The paged latent cache on the GPU: tokens written into it (norm, rotation, rows through the block
table), drafted tokens against it, and a speculative step that uses both, against float64.

Bounds.  A written value is rounded once to its type.  The norm is a float32 sum of dc squares, off by dc
2^-24 of itself at most, so its root by half of that, and a few roundings; a rotated value is x cos - y sin
of an angle that is off by 2^-53 of position * freq and by the rounding of half a turn (2^-24 pi), cosine
and sine by two steps.  Attention: a score is a sum of D products in float32, each off by 2^-24 of the sum by
magnitude; p takes a score's error over as a relative one, with 2^-21 for the exponential and the sums;
with bf16 inputs p is rounded to bf16 (2^-8) as an operand."""
import math

import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def check(got, ref, tol, what):
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.equal(torch.isinf(got), torch.isinf(ref)) and not torch.isnan(got).any(), what
    d = torch.where(torch.isinf(ref), 0.0, (got - ref).abs())
    worst = float((d / (tol + 1e-30)).max()) if d.numel() else 0.0
    print("  %s: worst %.3f of the bound" % (what, worst), flush=True)
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


# ------------------------------------------------------------------------------------- appending


def turned(x, pos, freqs, interleaved, dtype):
    """x [.., dr] turned by pos [..] (float64), and the bound."""
    x, a = x.double(), pos.double()[..., None] * freqs.double()
    e = a.abs() * 2.0 ** -52 + 2.0 ** -21
    c, s = torch.cos(a), torch.sin(a)
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    y, z, size = u * c - v * s, u * s + v * c, (u.abs() + v.abs()) * e
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat([p, q], -1))
    y = join(y, z)
    return y, HALF[dtype] * y.abs() * 1.01 + join(size, size)


def normed(c, w, eps, dtype):
    c = c.double()
    if w is None:
        return c, 0.0 * c
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps) * w.double()
    return y, (HALF[dtype] * 1.01 + (c.shape[-1] / 2 + 8) * 2.0 ** -24) * y.abs()


def case(B, T, H, dc, dtype, seed, packed=False):
    gen = torch.Generator().manual_seed(seed)
    lead = (T,) if packed else (B, T)
    both = (torch.randn(*lead, dc + 64, generator=gen) * 2).to(dtype)
    qfull = torch.randn(*lead, H, 128 + 64, generator=gen).to(dtype)
    return both, qfull, (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float(), (1 + 0.1 * torch.randn(dc, generator=gen)).to(dtype), gen


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,T,H,dc,page,norm,ragged", [
    (1, 1, 1, 512, 64, True, False), (5, 1, 128, 512, 64, True, False), (3, 7, 5, 256, 16, False, True), (2, 70, 33, 512, 1, True, True),
    (4, 3, 0, 256, 7, True, True),
])
def test_append(B, T, H, dc, page, norm, ragged, interleaved, dtype):
    both, qfull, freqs, weight, gen = case(B, T, H, dc, dtype, 3)
    counts = torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32) if ragged else None
    n = counts if ragged else torch.full((B,), T, dtype=torch.int32)
    lengths = torch.randint(0, 100, (B,), generator=gen, dtype=torch.int32) + n
    mp = (int(lengths.max()) + page - 1) // page + 1
    table = torch.randperm(B * mp + 2, generator=gen)[:B * mp].reshape(B, mp).to(torch.int32)
    old = torch.randn(B * mp + 2, page, dc + 64, generator=gen).to(dtype)
    pos = torch.randint(0, 2 ** 31 - 1, (B, T), generator=gen, dtype=torch.int32) if ragged else None
    cache, x, qd = old.cuda(), both.cuda(), qfull.cuda()
    oldq = torch.randn(B, T, H, dc + 64, generator=gen).to(dtype)
    q = oldq.cuda()
    more = dict(q_rope=qd[..., 128:], q=q) if H else {}
    got = kda.latent_append(x[..., :dc], x[..., dc:], cache, table.cuda(), lengths.cuda(), freqs.cuda(), norm_weight=weight.cuda() if norm else None,
                            eps=1e-5, positions=None if pos is None else pos.cuda(), counts=None if counts is None else counts.cuda(),
                            interleaved=interleaved, **more)
    torch.cuda.synchronize()
    assert got is cache
    ref, tol, qref, qtol = old.double(), torch.zeros(old.shape, dtype=torch.float64), oldq.double(), torch.zeros(oldq.shape, dtype=torch.float64)
    for b in range(B):
        for i in range(int(n[b])):
            row = int(lengths[b] - n[b]) + i
            at = (int(table[b, row // page]), row % page)
            p = torch.tensor(float(row if pos is None else pos[b, i]), dtype=torch.float64)
            for y, lo, hi in ((normed(both[b, i, :dc], weight if norm else None, 1e-5, dtype), 0, dc),
                              (turned(both[b, i, dc:], p, freqs, interleaved, dtype), dc, dc + 64)):
                ref[at][lo:hi], tol[at][lo:hi] = y
            qref[b, i, :, dc:], qtol[b, i, :, dc:] = turned(qfull[b, i, :, 128:], p.expand(H), freqs, interleaved, dtype)
    check(cache, ref, tol, "cache")
    if H:
        check(q, qref, qtol, "q")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_packed(dtype):
    """Ragged prompts, empty ones, rows in front of and behind the sequences; the boundaries of the batch form."""
    lens, dc, page, H, lead = [3, 0, 70, 1, 0], 512, 16, 3, 2
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N = cu[-1] + 3, len(lens)
    both, qfull, freqs, weight, gen = case(0, T, H, dc, dtype, 5, packed=True)
    lengths = torch.tensor([n + 11 * i for i, n in enumerate(lens)], dtype=torch.int32)
    table = torch.randperm(N * 8, generator=gen).reshape(N, 8).to(torch.int32)
    old = torch.zeros(N * 8, page, dc + 64, dtype=dtype)
    cache, x, qd, q = old.cuda(), both.cuda(), qfull.cuda(), torch.full((T, H, dc + 64), 5.0, dtype=dtype).cuda()
    kda.latent_append_varlen(x[..., :dc], x[..., dc:], cache, table.cuda(), lengths.cuda(), freqs.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                             norm_weight=weight.cuda(), q_rope=qd[..., 128:], q=q)
    torch.cuda.synchronize()
    ref, tol = old.double(), torch.zeros(old.shape, dtype=torch.float64)
    qref, qtol = torch.full((T, H, dc + 64), 5.0, dtype=torch.float64), torch.zeros(T, H, dc + 64, dtype=torch.float64)
    for b in range(N):
        for i in range(lens[b]):
            t, row = cu[b] + i, int(lengths[b]) - lens[b] + i
            at = (int(table[b, row // page]), row % page)
            p = torch.tensor(float(row), dtype=torch.float64)
            ref[at][:dc], tol[at][:dc] = normed(both[t, :dc], weight, 1e-6, dtype)
            ref[at][dc:], tol[at][dc:] = turned(both[t, dc:], p, freqs, True, dtype)
            qref[t, :, dc:], qtol[t, :, dc:] = turned(qfull[t, :, 128:], p.expand(H), freqs, True, dtype)
    check(cache, ref, tol, "cache")
    check(q, qref, qtol, "q")


def test_append_leaves_what_is_out_of_range():
    """Rows that are negative, behind the table or on pages outside the cache: nothing but their own rows'
    places is missing, and queries turn all the same."""
    dc, page, dtype = 256, 4, BF
    both, qfull, freqs, _, gen = case(4, 6, 2, dc, dtype, 9)
    lengths = torch.tensor([3, 10, 6, -5], dtype=torch.int32)  # rows -3 .. 2; 4 .. 9 of 8; bad pages; -11 .. -6
    table = torch.tensor([[0, 1], [2, 3], [-1, 99], [4, 5]], dtype=torch.int32)
    cache, x, qd, q = torch.zeros(6, page, dc + 64, dtype=dtype).cuda(), both.cuda(), qfull.cuda(), torch.zeros(4, 6, 2, dc + 64, dtype=dtype).cuda()
    kda.latent_append(x[..., :dc], x[..., dc:], cache, table.cuda(), lengths.cuda(), freqs.cuda(), q_rope=qd[..., 128:], q=q)
    torch.cuda.synchronize()
    want = torch.zeros(6, page, dc, dtype=dtype)
    for i in range(3):
        want[0, i] = both[0, 3 + i, :dc]
    for i in range(4):
        want[3, i] = both[1, i, :dc]
    assert torch.equal(cache[..., :dc].cpu(), want)
    assert bool((q[..., dc:].abs().sum(-1) > 0).all())


# ------------------------------------------------------------------------------------- drafted tokens


def tree(T, gen):
    """Random parents, and the bits of each node's ancestors and its own."""
    parents, bits = [], []
    for i in range(T):
        p = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
        parents.append(p)
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return parents, bits


def signed(x):
    return x - (1 << 64) if x >> 63 else x


def attend(q, rows, scale, dc, dtype):
    """out and lse of one token's heads against its visible rows, and their bounds."""
    q, rows = q.double(), rows.double()
    if not rows.shape[0]:
        z = torch.zeros(q.shape[0], dc, dtype=torch.float64)
        return z, z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64), torch.zeros(q.shape[0], dtype=torch.float64)
    s = q @ rows.T * scale
    size = float((q.abs() @ rows.abs().T).max()) * scale
    e = 2 * q.shape[1] * 2.0 ** -24 * size + 2.0 ** -21
    r = HALF[dtype] + e if dtype == BF else e
    p, lse = torch.softmax(s, -1), torch.logsumexp(s, -1)
    out = p @ rows[:, :dc]
    return out, HALF[dtype] * out.abs() * 1.01 + 2 * r * (p @ rows[:, :dc].abs()), lse, e * (1 + size) + 2.0 ** -22 * lse.abs()


def run_tree(B, T, H, dc, page, lens, dtype, seed, counts=None, masks=None, out_of=None):
    gen = torch.Generator().manual_seed(seed)
    mp = max(1, (max(max(lens), 1) + page - 1) // page)
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32)
    cache = torch.randn(B * mp, page, dc + 64, generator=gen).to(dtype)
    q = (torch.randn(B, T, H, dc + 64, generator=gen) * 0.5).to(dtype)
    if masks is None:
        masks = [tree(T, gen)[1] for _ in range(B)]
    mask = torch.tensor([[signed(x) for x in m] for m in masks], dtype=torch.int64)
    lengths = torch.tensor(lens, dtype=torch.int32)
    args = [t.cuda() for t in (q, cache, table, lengths, mask)]
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    out, lse = kda.latent_tree_step(*args, 0.07, dc=dc, counts=c, return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        rows = torch.cat([cache[int(table[b, j // page]), j % page][None] for j in range(lens[b])]) if lens[b] else cache[0, :0]
        n = T if counts is None else counts[b]
        base = lens[b] - n
        for i in range(T):
            see = [j for j in range(lens[b]) if j < base or masks[b][i] >> (j - base) & 1] if i < n else []
            ref, tol, lref, ltol = attend(q[b, i], rows[see], 0.07, dc, dtype)
            check(out[b, i], ref, tol, "out %d %d" % (b, i))
            check(lse[b, i], lref, ltol, "lse %d %d" % (b, i))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,dc,page,lens", [
    (1, 1, 1, 512, 64, [1]), (2, 1, 16, 512, 64, [5, 130]), (1, 4, 16, 512, 16, [4]), (3, 5, 16, 256, 64, [5, 64, 300]),
    (1, 3, 5, 512, 7, [200]), (2, 2, 16, 256, 1, [63, 65]), (1, 64, 2, 512, 64, [64]), (1, 64, 1, 256, 16, [129]),
    (2, 9, 13, 512, 128, [500, 20]), (1, 2, 128, 512, 64, [1100]), (1, 33, 4, 256, 64, [700]),
])
def test_tree(B, T, H, dc, page, lens, dtype):
    run_tree(B, T, H, dc, page, lens, dtype, 7 + T)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_padded_batch_and_empty_rows(dtype):
    """Counts from none to all, lengths of zero, shorter than the count and as long, bits that leave a row
    nothing, bits behind the count."""
    full = (1 << 64) - 1
    run_tree(6, 4, 3, 256, 16, [0, 40, 3, 2, 4, 33], dtype, 17, counts=[2, 0, 1, 4, 4, 3],
             masks=[[1, 3, 7, 15], [1, 3, 7, 15], [0, full, 0, 0], [1, 2, 4, full], [0, 0, full, 8], [0, full, 1 << 63, 5]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_of_one_is_the_one_token_step(dtype):
    B, H, dc, page, n = 3, 20, 512, 64, 333
    gen = torch.Generator().manual_seed(3)
    mp = 6
    table, cache = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32).cuda(), torch.randn(B * mp, page, 576, generator=gen).to(dtype).cuda()
    q, lengths = torch.randn(B, 1, H, 576, generator=gen).to(dtype).cuda(), torch.tensor([n, 1, 64], dtype=torch.int32).cuda()
    one = torch.ones(B, 1, dtype=torch.int64).cuda()
    out, lse = kda.latent_tree_step(q, cache, table, lengths, one, 0.05, return_lse=True)
    out1, lse1 = kda.latent_decode_step(q[:, 0].contiguous(), cache, table, lengths, 0.05, return_lse=True)
    torch.cuda.synchronize()
    # either is off by one rounding of p and one of the result
    assert float((out[:, 0].double() - out1.double()).abs().max()) <= 4 * (HALF[dtype] + 2.0 ** -18) * float(cache.abs().max())
    assert float((lse[:, 0] - lse1).abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,n", [(2, 30), (40, 700)])
def test_tree_bad_rows_reach_who_sees_them(H, n, dtype, bad):
    """A drafted row that is not finite: NaN in the tokens that see it, the others as without it.  Rows past
    the length hold NaN as well and are nobody's."""
    B, T, dc, page = 1, 4, 512, 16
    gen = torch.Generator().manual_seed(4)
    mp = (n + page - 1) // page + 1
    table = torch.randperm(mp, generator=gen).reshape(B, mp).to(torch.int32)
    cache = torch.randn(mp, page, 576, generator=gen).to(dtype)
    q = torch.randn(B, T, H, 576, generator=gen).to(dtype).cuda()
    mask = torch.tensor([[1, 2, 5, 10]], dtype=torch.int64).cuda()  # two chains: 0 - 2, 1 - 3
    lengths = torch.tensor([n], dtype=torch.int32).cuda()
    for j in range(n, mp * page):
        cache[int(table[0, j // page]), j % page] = float("nan")
    ref, lref = kda.latent_tree_step(q, cache.cuda(), table.cuda(), lengths, mask, 0.04, return_lse=True)
    assert torch.isfinite(ref).all() and torch.isfinite(lref).all()
    row = n - T + 1  # token 1's
    for ch in (3, 540):
        c = cache.clone()
        c[int(table[0, row // page]), row % page, ch] = bad
        out, lse = kda.latent_tree_step(q, c.cuda(), table.cuda(), lengths, mask, 0.04, return_lse=True)
        torch.cuda.synchronize()
        for i in range(T):
            if i in (1, 3):
                assert torch.isnan(out[0, i]).all() and torch.isnan(lse[0, i]).all(), i
            else:
                assert torch.equal(out[0, i], ref[0, i]) and torch.equal(lse[0, i], lref[0, i]), i
    q2 = q.clone()
    q2[0, 2, 1, 7] = bad  # one head of one token
    out, lse = kda.latent_tree_step(q2, cache.cuda(), table.cuda(), lengths, mask, 0.04, return_lse=True)
    assert torch.isnan(out[0, 2, 1]).all() and torch.isnan(lse[0, 2, 1])
    out[0, 2, 1], lse[0, 2, 1] = ref[0, 2, 1], lref[0, 2, 1]
    assert torch.equal(out, ref) and torch.equal(lse, lref)


def test_tree_contents_out_of_range():
    """Pages outside the cache, lengths beyond the table and below zero, counts beyond T: no access outside,
    finite results from a finite cache."""
    B, T, H, dc, page, mp = 4, 3, 4, 256, 16, 3
    cache = torch.randn(5, page, dc + 64).to(BF).cuda()
    table = torch.tensor([[0, 99, -7], [2 ** 31 - 1, 1, 2], [0, 1, 2], [3, 4, -2 ** 31]], dtype=torch.int32).cuda()
    lengths = torch.tensor([48, 2 ** 31 - 1, -5, 40], dtype=torch.int32).cuda()
    counts = torch.tensor([2 ** 31 - 1, 3, 1, -4], dtype=torch.int32).cuda()
    mask = torch.full((B, T), -1, dtype=torch.int64).cuda()
    out, lse = kda.latent_tree_step(torch.randn(B, T, H, dc + 64).to(BF).cuda(), cache, table, lengths, mask, 0.1, dc=dc, counts=counts, return_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    assert torch.isfinite(lse[:2]).all() and bool((lse[2:] == -math.inf).all()) and bool((out[2:] == 0).all())


# ------------------------------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", [BF, F32])
def test_speculative_step(dtype):
    """Prompts into the cache, then a tree of drafted tokens behind them, then the accepted path again as
    plain tokens: the drafted nodes of that path got what a chain of single steps gets."""
    B, H, dc, page, scale = 2, 8, 512, 16, (128 + 64) ** -0.5
    gen = torch.Generator().manual_seed(8)
    prompt, mp = [37, 5], 8
    cache = torch.zeros(B * mp, page, dc + 64, dtype=dtype).cuda()
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32).cuda()
    freqs = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()
    weight = torch.ones(dc, dtype=dtype).cuda()
    x = torch.randn(sum(prompt), dc + 64, generator=gen).to(dtype).cuda()
    cu, lengths = torch.tensor([0, prompt[0], sum(prompt)], dtype=torch.int32).cuda(), torch.tensor(prompt, dtype=torch.int32).cuda()
    kda.latent_append_varlen(x[:, :dc], x[:, dc:], cache, table, lengths, freqs, cu, norm_weight=weight)
    # a tree: 0 - 1 - 3, 0 - 2; positions go by depth
    T, bits, depth = 4, [1, 3, 5, 11], [0, 1, 1, 2]
    new = torch.randn(B, T, dc + 64, generator=gen).to(dtype).cuda()
    qr = torch.randn(B, T, H, 64, generator=gen).to(dtype).cuda()
    q = torch.randn(B, T, H, dc + 64, generator=gen).to(dtype).cuda()
    pos = (lengths[:, None] + torch.tensor(depth, dtype=torch.int32).cuda()[None]).contiguous()
    kda.latent_append(new[..., :dc], new[..., dc:], cache, table, lengths + T, freqs, norm_weight=weight, positions=pos, q_rope=qr, q=q)
    mask = torch.tensor([bits] * B, dtype=torch.int64).cuda()
    out, lse = kda.latent_tree_step(q, cache, table, lengths + T, mask, scale, return_lse=True)
    # accepted: 0, 1, 3
    path = [0, 1, 3]
    for k, i in enumerate(path):
        now = lengths + k + 1
        q1 = q[:, i:i + 1].clone()
        kda.latent_append(new[:, i:i + 1, :dc], new[:, i:i + 1, dc:], cache, table, now, freqs, norm_weight=weight, q_rope=qr[:, i:i + 1], q=q1)
        assert torch.equal(q1, q[:, i:i + 1]), "a drafted token stands where the plain one does"
        o, l = kda.latent_decode_step(q1[:, 0].contiguous(), cache, table, now, scale, return_lse=True)
        torch.cuda.synchronize()
        size = float(cache[..., :dc].abs().max())
        assert float((o.double() - out[:, i].double()).abs().max()) <= 4 * (HALF[dtype] + 2.0 ** -18) * size, i
        assert float((l - lse[:, i]).abs().max()) <= 2.0 ** -16, i


def test_captured_step_replays():
    """Append and tree in one captured graph, replayed on new inputs with eager work between: every replay has
    the eager call's bits."""
    B, T, H, dc, page, mp = 2, 3, 16, 512, 16, 20
    gen = torch.Generator().manual_seed(6)
    table = torch.randperm(B * mp, generator=gen).reshape(B, mp).to(torch.int32).cuda()
    base = torch.randn(B * mp, page, dc + 64, generator=gen).to(BF).cuda()
    freqs, lengths = torch.rand(32, generator=gen).cuda(), torch.tensor([300, 20], dtype=torch.int32).cuda()
    mask = torch.tensor([[1, 3, 5]] * B, dtype=torch.int64).cuda()
    x, qr, q = (torch.zeros(*s, dtype=BF).cuda() for s in ((B, T, dc + 64), (B, T, H, 64), (B, T, H, dc + 64)))
    out, lse = torch.zeros(B, T, H, dc, dtype=BF).cuda(), torch.zeros(B, T, H).cuda()
    ws = torch.zeros(max(1, kda.latent_tree_workspace_bytes(B, T, H, page, mp, dc, 64, BF)), dtype=torch.uint8).cuda()
    cache = base.clone()

    def step(cache, q, out, lse, ws):
        kda.latent_append(x[..., :dc], x[..., dc:], cache, table, lengths, freqs, q_rope=qr, q=q)
        kda.latent_tree_step(q, cache, table, lengths, mask, 0.1, out=out, lse=lse, workspace=ws)

    step(cache, q, out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, q, out, lse, ws)
    for k in range(4):
        for t in (x, qr, q):
            t.copy_(torch.randn(t.shape, generator=gen).to(BF))
        want = [base.clone(), q.clone(), torch.zeros_like(out), torch.zeros_like(lse)]
        step(*want, ws.clone())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref, n in zip((cache, q, out, lse), want, ("cache", "q", "out", "lse")):
            assert torch.equal(got, ref), "%s of replay %d" % (n, k)
