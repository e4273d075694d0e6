"""Decayed linear attention on the GPU against float64, pair of tokens by pair: forward, backward and the
one-token step, over lengths from none on, segments that end inside and at a chunk, shared key heads, start
states, packed documents, strides, decays from none to -inf.  lin_util.py derives the bounds."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import lin_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def cuda(*x):
    return [None if t is None else t.cuda() for t in x]


def states(B, H, dv, dk, seed, want=True):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(B, H, dv, dk, generator=gen) if want else None for _ in range(2)]


def run_batch(q, k, v, g, scale, s0, do, df, want_dg=True):
    """Everything of a batch, as {name: tensor [B, ...]}; q .. on the GPU."""
    out, fs = kda.lin_chunk_fwd(q, k, v, g, scale=scale, initial_state=s0, return_final_state=True)
    d = kda.lin_chunk_bwd(q, k, v, g, do, scale=scale, initial_state=s0, dfinal_state=df, want_dg=want_dg)
    torch.cuda.synchronize()
    return {"out": out, "final_state": fs, **{n: t for n, t in d.items() if t is not None}}


def check_batch(x, q, k, v, g, scale, s0, do, df, what=""):
    B, H = v.shape[:2]
    r = H // q.shape[1]
    for b in range(B):
        U.check_sequence({n: t[b] for n, t in x.items()}, "%s%d " % (what, b), H, r, lambda h: U.one(
            q[b, h // r], k[b, h // r], v[b, h], g[b, h], scale, q.dtype, g.dtype, None if s0 is None else s0[b, h], do[b, h],
            None if df is None else df[b, h]), q.dtype, g.dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv,state", [
    (1, 1, 1, 1, 128, 128, True), (2, 1, 2, 2, 64, 64, False), (1, 2, 2, 37, 64, 128, True), (1, 1, 1, 63, 128, 64, False),
    (1, 1, 3, 64, 128, 128, True), (1, 2, 4, 65, 64, 64, True), (1, 1, 1, 128, 128, 64, True), (2, 1, 1, 256, 64, 128, False),
    (1, 1, 2, 257, 128, 128, True), (1, 1, 1, 319, 64, 64, True), (1, 1, 2, 700, 128, 128, True), (1, 2, 2, 1030, 64, 128, False),
])
def test_batch(B, Hk, H, T, dk, dv, state, dtype):
    q, k, v, g = U.inputs(B, Hk, H, T, dk, dv, dtype, 10 + T, g32=T % 2 == 0)
    do = U.inputs(B, Hk, H, T, dk, dv, dtype, 11 + T)[2]
    s0, df = states(B, H, dv, dk, T, state)
    x = run_batch(*cuda(q, k, v, g), dk ** -0.5, *cuda(s0, do, df))
    assert x["out"].dtype == dtype and x["final_state"].dtype == F32 and x["dg"].dtype == g.dtype
    check_batch(x, q, k, v, g, dk ** -0.5, s0, do, df)


@pytest.mark.parametrize("dtype,Hk,H,dk,dv,lens", [
    (BF, 1, 2, 128, 128, [1, 300, 0, 64, 530, 3, 0]), (F32, 2, 2, 64, 64, [70, 257, 1]), (BF, 2, 4, 64, 128, [0, 0, 5]),
    (F32, 1, 2, 128, 64, [300, 256, 128, 0]), (BF, 1, 1, 64, 64, [3] * 40),
])
def test_packed(dtype, Hk, H, dk, dv, lens):
    lead, tail = 3, 70  # rows in front of and behind the documents
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N, r = cu[-1] + tail, len(lens), H // Hk
    q, k, v, g = U.inputs(0, Hk, H, T, dk, dv, dtype, 5, packed=True)
    do = U.inputs(0, Hk, H, T, dk, dv, dtype, 6, packed=True)[2]
    s0, df = states(N, H, dv, dk, 3)
    for t in (q, k, v, do):  # not part of any document
        t[:, :lead], t[:, cu[-1]:] = float("nan"), float("inf")
    g[:, :lead], g[:, cu[-1]:] = float("nan"), float("nan")
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    out = torch.full((H, T, dv), 7.0, dtype=dtype).cuda()
    qd, kd, vd, gd = cuda(q, k, v, g)
    sd, dd, fd = cuda(s0, do, df)
    _, fs = kda.lin_chunk_fwd_varlen(qd, kd, vd, gd, c, scale=0.1, out=out, initial_state=sd, return_final_state=True)
    d = kda.lin_chunk_bwd_varlen(qd, kd, vd, gd, dd, c, scale=0.1, initial_state=sd, dfinal_state=fd)
    d2 = kda.lin_chunk_bwd_varlen(qd, kd, vd, gd, dd, c, scale=0.1, initial_state=sd, dfinal_state=fd, want_dg=False)
    torch.cuda.synchronize()
    for x in (out[:, :lead], out[:, cu[-1]:]):
        assert bool((x == 7.0).all()), "rows outside the documents were written"
    for n in ("dq", "dk", "dv", "dg"):
        for x in (d[n][:, :lead], d[n][:, cu[-1]:]):
            assert bool((x == 0).all()), "%s outside the documents" % n
    for n in ("dq", "dk", "dv", "dinitial_state"):
        assert torch.isfinite(d2[n]).all() and float((d2[n] - d[n]).abs().max()) <= 2.0 ** -7 * float(d[n].abs().max() + 1e-30), n
    assert d2["dg"] is None
    for i in range(N):
        s = slice(cu[i], cu[i + 1])
        x = {"out": out[:, s], "final_state": fs[i], **{n: d[n][:, s] for n in ("dq", "dk", "dv", "dg")}, "dinitial_state": d["dinitial_state"][i]}
        U.check_sequence(x, "%d " % i, H, r, lambda h: U.one(q[h // r, s], k[h // r, s], v[h, s], g[h, s], 0.1, dtype, g.dtype, s0[i, h],
                                                               do[h, s], df[i, h]), dtype, g.dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0, 1, 100, 600])
def test_no_gradient_of_the_end_state(T, dtype):
    """dfinal_state left out, no dinitial wanted, and the other way round."""
    q, k, v, g = U.inputs(1, 1, 2, T, 64, 64, dtype, 3)
    do = U.inputs(1, 1, 2, T, 64, 64, dtype, 4)[2]
    s0, df = states(1, 2, 64, 64, 8)
    x = cuda(q, k, v, g)
    sd, dd, fd = cuda(s0, do, df)
    a = kda.lin_chunk_bwd(*x, dd, scale=0.2, initial_state=sd, want_dinitial=False)
    b = kda.lin_chunk_bwd(*x, dd, scale=0.2, initial_state=sd, dfinal_state=fd)
    c = kda.lin_chunk_bwd(*x, dd, scale=0.2)
    torch.cuda.synchronize()
    assert a["dinitial_state"] is None
    a.pop("dinitial_state")
    for got, s, f in ((a, s0, None), (b, s0, df), (c, None, None)):
        check_batch(got, q, k, v, g, 0.2, s, do, f)
    if T == 0:
        assert torch.equal(b["dinitial_state"].cpu(), df) and bool((c["dinitial_state"] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["none", "strong", "inf", "mixed", "head"])
def test_decays(kind, dtype):
    """No decay at all; decays that forget at once; resets by -inf; both side by side; a constant per head
    in float32, expanded."""
    B, H, T, d = 1, 2, 330, 64
    q, k, v, _ = U.inputs(B, H, H, T, d, d, dtype, 21)
    do = U.inputs(B, H, H, T, d, d, dtype, 22)[2]
    gen = torch.Generator().manual_seed(5)
    g = {"none": torch.zeros(B, H, T), "strong": -20 * torch.rand(B, H, T, generator=gen), "inf": torch.where(
        torch.rand(B, H, T, generator=gen) < 0.05, -float("inf"), -0.01), "mixed": torch.where(
        torch.rand(B, H, T, generator=gen) < 0.3, -300.0, -0.001), "head": torch.tensor([-0.3, -0.002])[:, None]}[kind]
    g = g.expand(B, H, T) if kind == "head" else g.to(dtype)
    s0, df = states(B, H, d, d, 9)
    gd = torch.tensor([-0.3, -0.002]).cuda()[:, None].expand(B, H, T) if kind == "head" else g.cuda()
    x = run_batch(*cuda(q, k, v), gd, 0.125, *cuda(s0, do, df))
    check_batch(x, q, k, v, g, 0.125, s0, do, df)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_views(dtype):
    """[B,T,H,d] projections, one tensor for all of them, g and dout strided too; the same bits as with
    contiguous copies."""
    B, Hk, H, T, d = 2, 2, 4, 150, 64
    gen = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, T, 2 * Hk + H, d, generator=gen).to(dtype).cuda()
    q, k, v = (t.transpose(1, 2) for t in qkv.split([Hk, Hk, H], 2))
    g = (-torch.rand(B, T, H, generator=gen)).to(dtype).cuda().transpose(1, 2)
    do = torch.randn(B, T, H, d, generator=gen).to(dtype).cuda().transpose(1, 2)
    a = run_batch(q, k, v, g, 0.3, None, do, None)
    c = run_batch(*(t.contiguous() for t in (q, k, v, g)), 0.3, None, do.contiguous(), None)
    for n in a:
        assert torch.equal(a[n], c[n]), n
    check_batch({n: t for n, t in a.items()}, *(t.cpu() for t in (q, k, v, g)), 0.3, None, do.cpu(), None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 6, 128, 64), (2, 4, 4, 64, 128), (5, 1, 8, 128, 128)])
def test_one_token(B, Hk, H, dk, dv, dtype):
    q, k, v, g = (t[:, :, 0].contiguous() for t in U.inputs(B, Hk, H, 1, dk, dv, dtype, 31, g32=B == 3))
    s0 = states(B, H, dv, dk, 1)[0]
    S = s0.cuda()
    out = kda.lin_decode_step(*cuda(q, k, v, g), S, scale=0.25)
    torch.cuda.synchronize()
    r = H // Hk
    for b in range(B):
        U.check_sequence({"out": out[b][:, None], "final_state": S[b]}, "%d " % b, H, r, lambda h: U.one(
            q[b, h // r][None], k[b, h // r][None], v[b, h][None], g[b, h][None], 0.25, dtype, g.dtype, s0[b, h]), dtype, g.dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_in_pieces_then_tokens(dtype):
    """A prompt in two pieces, the state in place, then token by token, against the whole sequence."""
    B, H, T, d = 1, 2, 90, 64
    q, k, v, g = U.inputs(B, H, H, T, d, d, dtype, 41)
    x = cuda(q, k, v, g)
    S = torch.zeros(B, H, d, d).cuda()
    outs = [kda.lin_chunk_fwd(*(t[:, :, a:b] for t in x), scale=0.1, initial_state=S, final_state=S) for a, b in ((0, 50), (50, 85))]
    for t in range(85, T):
        outs.append(kda.lin_decode_step(*(y[:, :, t].contiguous() for y in x), S, scale=0.1)[:, :, None])
    out = torch.cat(outs, 2)
    torch.cuda.synchronize()
    check_batch({"out": out, "final_state": S}, q, k, v, g, 0.1, None, v, None)


def test_gradients_against_differences():
    """Directional differences of the forward, in float32, against the backward's gradients."""
    B, Hk, H, T, d = 1, 1, 2, 300, 64
    q, k, v, g = cuda(*U.inputs(B, Hk, H, T, d, d, F32, 51))
    s0, df = cuda(*states(B, H, d, d, 6))
    do = U.inputs(B, Hk, H, T, d, d, F32, 52)[2].cuda()
    grads = kda.lin_chunk_bwd(q, k, v, g, do, scale=0.1, initial_state=s0, dfinal_state=df)

    def loss(q, k, v, g, s0):
        out, fs = kda.lin_chunk_fwd(q, k, v, g, scale=0.1, initial_state=s0, return_final_state=True)
        return float((out.double() * do.double()).sum() + (fs.double() * df.double()).sum())

    gen = torch.Generator().manual_seed(1)
    leaves = [q, k, v, g, s0]
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dinitial_state")):
        step = torch.randn(leaves[i].shape, generator=gen).cuda() * (1e-2 * leaves[i].abs() if name == "dg" else 1e-2)
        up, down = (loss(*(t + s * step if j == i else t for j, t in enumerate(leaves))) for s in (1, -1))
        want = float((grads[name].double() * step.double()).sum())
        # out is linear or quadratic in q, k, v and s0 (central differences are exact), third order in g's
        # steps of 1 %; float32 sums of some 40,000 terms leave 2^-24 sqrt of them of the sum by magnitude
        size = float((grads[name].double() * step.double()).abs().sum())
        print("  %s: differences %.6e, gradient %.6e, by magnitude %.2e" % (name, (up - down) / 2, want, size), flush=True)
        assert abs((up - down) / 2 - want) <= 1e-3 * size, name


def test_autograd():
    """LinChunkFunction: the entry points' gradients; a constant per head gets the sum over its tokens;
    a second derivative is refused."""
    B, H, T, d = 2, 2, 70, 64
    q, k, v, _ = (t.cuda() for t in U.inputs(B, H, H, T, d, d, F32, 61))
    slope = torch.tensor([-0.1, -0.02]).cuda().requires_grad_()
    g = slope[:, None].expand(B, H, T)
    x = [t.requires_grad_() for t in (q, k, v)]
    out, fs = kda.LinChunkFunction.apply(*x, g, 0.1)
    (out.sum() + fs.square().sum()).backward()
    d2 = kda.lin_chunk_bwd(*(t.detach() for t in (*x, g)), torch.ones_like(out), scale=0.1, dfinal_state=2 * fs.detach())
    for t, n in zip(x, ("dq", "dk", "dv")):
        assert torch.equal(t.grad, d2[n]), n
    # the sum over batch entries and tokens, in another order
    assert torch.allclose(slope.grad, d2["dg"].sum((0, 2)), rtol=1e-4)
    out, _ = kda.LinChunkFunction.apply(*x, slope.detach()[:, None].expand(B, H, T), 0.1)
    first, = torch.autograd.grad(out.sum(), x[0], create_graph=True)
    with pytest.raises(RuntimeError):
        first.sum().backward()


def test_same_bits_again():
    q, k, v, g = cuda(*U.inputs(1, 2, 4, 777, 128, 128, BF, 71))
    do = U.inputs(1, 2, 4, 777, 128, 128, BF, 72)[2].cuda()
    a, b = (run_batch(q, k, v, g, 0.1, None, do, None) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n
