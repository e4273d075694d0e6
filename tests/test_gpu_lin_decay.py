"""The log-decays' gradient of linear attention on the GPU, element by element and in norm against the sum that
it is, over segments of one chunk and of several, states, shared heads, packed documents and decays from none
to -inf.  lin_decay_util.py derives the bounds; test_lin_decay_host.py shows what they notice."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import lin_decay_util as D
from tests import lin_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def states(N, H, dv, dk, seed, which):
    gen = torch.Generator().manual_seed(seed)
    s0, df = (torch.randn(N, H, dv, dk, generator=gen) for _ in range(2))
    return s0 if which in ("both", "start") else None, df if which in ("both", "end") else None


def cuda(*x):
    return [None if t is None else t.cuda() for t in x]


@pytest.mark.parametrize("dtype,g32", [(BF, False), (BF, True), (F32, True)])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv,which,rate", [
    (1, 1, 1, 1, 64, 64, "both", -3), (1, 1, 2, 2, 128, 64, "both", -3), (1, 2, 2, 64, 64, 128, "both", -3), (1, 1, 2, 65, 128, 128, "none", -3),
    (2, 1, 2, 200, 64, 64, "end", -3),                                                   # a segment of four chunks (bf16)
    (1, 1, 2, 257, 128, 128, "both", -3), (1, 2, 4, 319, 64, 64, "start", -3), (1, 1, 2, 700, 128, 128, "none", -3),
    (1, 2, 2, 1030, 64, 128, "both", -3), (1, 1, 2, 2049, 128, 64, "end", -3),           # segments of one chunk
    (1, 1, 2, 1030, 64, 64, "both", -8), (2, 1, 1, 700, 128, 128, "both", -12),          # decays of next to nothing
    (4, 8, 32, 1100, 128, 64, "both", -3), (16, 8, 16, 833, 64, 128, "both", -4),        # full cards: segments of several chunks
    (1, 64, 128, 1500, 64, 64, "none", -4),
])
def test_batch(B, Hk, H, T, dk, dv, which, rate, dtype, g32):
    q, k, v, g = U.inputs(B, Hk, H, T, dk, dv, dtype, 110 + T, rate=float(rate), g32=g32)
    do = U.inputs(B, Hk, H, T, dk, dv, dtype, 111 + T)[2]
    s0, df = states(B, H, dv, dk, T, which)
    scale, r = dk ** -0.5, H // Hk
    i, e = cuda(s0, df)
    got = kda.lin_chunk_bwd(*cuda(q, k, v, g, do), scale=scale, initial_state=i, dfinal_state=e)["dg"]
    torch.cuda.synchronize()
    assert got.dtype == g.dtype
    for b, h in sorted({(0, 0), (B - 1, H - 1), (B // 2, H // 2)}):
        ref = D.dg(q[b, h // r], k[b, h // r], v[b, h], g[b, h], scale, dtype, g.dtype, None if s0 is None else s0[b, h], do[b, h],
                   None if df is None else df[b, h])
        D.check(got[b, h], ref, g.dtype, "%d %d" % (b, h))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hk,H,dk,dv,which,lens", [
    (1, 2, 128, 128, "both", [1, 300, 0, 64, 530, 3, 0]), (2, 2, 64, 64, "end", [70, 257, 1, 128]), (1, 1, 64, 128, "start", [3] * 40 + [200, 65]),
    (32, 32, 64, 64, "both", [1, 700, 64, 2049, 0, 385, 1500, 3]), (16, 32, 128, 64, "none", [900, 5, 64, 1300, 129]),
    (32, 32, 64, 64, "both", [9] * 60 + [700, 130, 1200] + [1] * 30),  # more documents than segments
])
def test_packed(Hk, H, dk, dv, which, lens, dtype):
    cu = [3]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N, r = cu[-1] + 9, len(lens), H // Hk
    q, k, v, g = U.inputs(0, Hk, H, T, dk, dv, dtype, 121, packed=True)
    do = U.inputs(0, Hk, H, T, dk, dv, dtype, 122, packed=True)[2]
    s0, df = states(N, H, dv, dk, 3, which)
    i, e = cuda(s0, df)
    got = kda.lin_chunk_bwd_varlen(*cuda(q, k, v, g, do), torch.tensor(cu, dtype=torch.int32).cuda(), scale=0.1, initial_state=i, dfinal_state=e)["dg"]
    torch.cuda.synchronize()
    for n in range(N):
        s = slice(cu[n], cu[n + 1])
        if lens[n] == 0 or lens[n] < 10 and n % 7:
            continue
        for h in sorted({0, H - 1}):
            ref = D.dg(q[h // r, s], k[h // r, s], v[h, s], g[h, s], 0.1, dtype, dtype, None if s0 is None else s0[n, h], do[h, s],
                       None if df is None else df[n, h])
            D.check(got[h, s], ref, dtype, "document %d head %d" % (n, h))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["none", "strong", "inf", "mixed", "head", "one token forgets"])
def test_decays(kind, dtype):
    B, H, T, d = 1, 2, 700, 64
    q, k, v, _ = U.inputs(B, H, H, T, d, d, dtype, 131)
    do = U.inputs(B, H, H, T, d, d, dtype, 132)[2]
    gen = torch.Generator().manual_seed(5)
    g = {"none": torch.zeros(B, H, T), "strong": -20 * torch.rand(B, H, T, generator=gen),
         "inf": torch.where(torch.rand(B, H, T, generator=gen) < 0.05, -float("inf"), -0.01),
         "mixed": torch.where(torch.rand(B, H, T, generator=gen) < 0.3, -300.0, -0.001),
         "head": torch.tensor([-0.3, -0.002])[:, None], "one token forgets": torch.full((B, H, T), -0.001)}[kind]
    if kind == "one token forgets":
        g[..., 100], g[..., 640] = -9.0, -30.0
    g = g.expand(B, H, T) if kind == "head" else g.to(dtype)
    s0, df = states(B, H, d, d, 9, "both")
    gd = torch.tensor([-0.3, -0.002]).cuda()[:, None].expand(B, H, T) if kind == "head" else g.cuda()
    got = kda.lin_chunk_bwd(*cuda(q, k, v), gd, do.cuda(), scale=0.125, initial_state=s0.cuda(), dfinal_state=df.cuda())["dg"]
    torch.cuda.synchronize()
    for h in range(H):
        D.check(got[0, h], D.dg(q[0, h], k[0, h], v[0, h], g[0, h], 0.125, dtype, g.dtype, s0[0, h], do[0, h], df[0, h]), g.dtype, "head %d" % h)
