"""Gradients of the gated delta rule on the GPU: against the adjoint of the token recurrence in
float64, against differences of the float64 forward, through autograd, packed documents, shared key
heads, graph capture."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from gdr_util import HALF, inputs, recurrent

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def reference(x, dout, scale, S0, dfin):
    """Gradients by autograd through the float64 token recurrence (elementary steps only)."""
    leaf = [t.double().requires_grad_() for t in x] + [S0.double().requires_grad_()]
    q, k, v, g, beta, S = leaf
    r = v.shape[1] // k.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    loss = 0.0
    for t in range(v.shape[2]):
        S = torch.exp(g[:, :, t])[..., None, None] * S
        w = beta[:, :, t, None] * (v[:, :, t] - (S * k[:, :, t, None]).sum(-1))
        S = S + w[..., None] * k[:, :, t, None]
        loss = loss + (dout[:, :, t].double() * scale * (S * q[:, :, t, None]).sum(-1)).sum()
    if dfin is not None:
        loss = loss + (S * dfin.double()).sum()
    return torch.autograd.grad(loss, leaf)


def compare(got, ref, dtype, what):
    """One rounding to the gradient's type, and what the stages round before: with bf16 inputs about
    eight fp16 roundings (P, U, dP', dX, X1, X2, dO's products, b) of 2^-11 each on terms whose sum of
    squares is the gradient's, so 8 * 2^-11 of its RMS over a head, times 4 for the largest of the
    elements; with float32 inputs 22 bits cut off in their place, and sums of 192 terms in float32.
    dg sums up to 64 rows of such terms and takes the factor 8 (sqrt 64) for it.  The initial state's
    gradient comes from 22-bit operands with either type."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    rms = ref.square().mean().sqrt()
    low = dtype == BF and what != "dinitial_state"
    eps = 8 * 2.0 ** -11 if low else 8 * 2.0 ** -21 + 192 * 2.0 ** -24
    tol = eps * 4 * (8 if what == "dg" else 1) * rms + (HALF[dtype] if low else 2.0 ** -24) * ref.abs() + 1e-30
    d = (got - ref).abs()
    print("  %s: worst %.3f of the bound, relative norm %.2e" % (what, float((d / tol).max()), float(d.norm() / ref.norm())), flush=True)
    assert (d <= tol).all(), "%s: %.3f of the bound" % (what, float((d / tol).max()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv", [
    (1, 1, 1, 1, 64, 64), (1, 1, 2, 3, 128, 64), (2, 2, 2, 63, 64, 128), (1, 2, 4, 64, 128, 128), (1, 1, 3, 65, 128, 128),
    (1, 2, 2, 127, 64, 64), (2, 1, 4, 150, 128, 128), (3, 4, 16, 70, 128, 128), (3, 4, 12, 195, 64, 128),
    (5, 7, 14, 66, 64, 128),
])
def test_gradients(B, Hk, H, T, dk, dv, dtype):
    x = inputs(B, Hk, H, T, dk, dv, dtype, 7 + T)
    gen = torch.Generator().manual_seed(T)
    dout = torch.randn(B, H, T, dv, generator=gen).to(dtype)
    S0, dfin = (torch.randn(B, H, dv, dk, generator=gen) * 0.5 for _ in range(2))
    if T % 2 == 0:
        dfin = None
    got = kda.gdr_chunk_bwd(*(t.cuda() for t in x), dout.cuda(), scale=dk ** -0.5, initial_state=S0.cuda(),
                            dfinal_state=None if dfin is None else dfin.cuda())
    for name, ref in zip(NAMES, reference(x, dout, dk ** -0.5, S0, dfin)):
        compare(got[name], ref, dtype, name)


@pytest.mark.parametrize("what", ["keys", "queries", "values", "dout"])
def test_zeros(what):
    """An operand that is zero throughout the middle chunk: the bounds that the others' exponents come
    from hold there too, and the initial state's gradient keeps its 22 bits."""
    x = list(inputs(1, 1, 2, 192, 128, 64, F32, 31, rate=-5.0))
    gen = torch.Generator().manual_seed(2)
    dout, S0, dfin = (torch.randn(1, 2, *s, generator=gen) for s in ((192, 64), (64, 128), (64, 128)))
    {"keys": x[1], "queries": x[0], "values": x[2], "dout": dout}[what][:, :, 64:128] = 0.0
    got = kda.gdr_chunk_bwd(*(t.cuda() for t in x), dout.cuda(), scale=128 ** -0.5, initial_state=S0.cuda(), dfinal_state=dfin.cuda())
    for name, ref in zip(NAMES, reference(x, dout, 128 ** -0.5, S0, dfin)):
        compare(got[name], ref, F32, name)


def test_differences():
    """The float32 gradients against central differences of the float64 token recurrence, along random
    directions of each input: the difference's own error is h^2 times a third derivative of the order
    of the value, h = 1e-4."""
    x = inputs(1, 1, 2, 70, 64, 64, F32, 3)
    gen = torch.Generator().manual_seed(5)
    dout, S0 = torch.randn(1, 2, 70, 64, generator=gen), torch.randn(1, 2, 64, 64, generator=gen) * 0.5
    got = kda.gdr_chunk_bwd(*(t.cuda() for t in x), dout.cuda(), initial_state=S0.cuda())
    args = [t.double() for t in x] + [S0.double()]

    def loss(a):
        return float((recurrent(*a[:5], 1.0, a[5])[0] * dout.double()).sum())

    for i, name in enumerate(NAMES):
        u = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        u /= u.norm()
        h = 1e-4
        up, down = ([a + s * h * u if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        d, want = (loss(up) - loss(down)) / (2 * h), float((got[name].double().cpu() * u).sum())
        size = float(got[name].double().norm())
        assert abs(d - want) <= 1e-5 * size + 1e-6, (name, d, want)


def test_autograd_and_shared_heads():
    """loss.backward() through GdrChunkFunction, on strided leaves, gives what the entry point gives."""
    x = inputs(2, 2, 4, 100, 128, 128, BF, 9)
    gen = torch.Generator().manual_seed(1)
    dout, dfin = torch.randn(2, 4, 100, 128, generator=gen).to(BF).cuda(), torch.randn(2, 4, 128, 128, generator=gen).cuda()
    S0 = torch.zeros(2, 4, 128, 128, device="cuda", requires_grad=True)
    leaf = [t.transpose(1, 2).contiguous().cuda().requires_grad_() for t in x]
    out, fs = kda.GdrChunkFunction.apply(*(t.transpose(1, 2) for t in leaf), 0.5, S0)
    ((out * dout).sum(dtype=torch.float32) + (fs * dfin).sum()).backward()
    want = kda.gdr_chunk_bwd(*(t.cuda() for t in x), dout, scale=0.5, initial_state=S0.detach(), dfinal_state=dfin)
    for t, name in zip(leaf, NAMES):
        assert torch.equal(t.grad.transpose(1, 2), want[name]), name
    assert torch.equal(S0.grad, want["dinitial_state"])
    # no gradient of the state wanted, only one output used
    leaf = [t.cuda().requires_grad_() for t in x]
    kda.GdrChunkFunction.apply(*leaf)[0].float().sum().backward()
    assert all(t.grad is not None and torch.isfinite(t.grad).all() for t in leaf)


@pytest.mark.parametrize("dtype,lengths", [(BF, [1, 64, 0, 65, 30]), (F32, [0, 70, 5]), (BF, [0, 0])])
def test_packed(dtype, lengths):
    a0, T, Hk, H, dk, dv = 3, sum(lengths) + 10, 1, 2, 64, 128  # 3 tokens in front of, 7 behind the documents
    x = inputs(1, Hk, H, T, dk, dv, dtype, 17, packed=True)
    cu = a0 + torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32)
    N, gen = len(lengths), torch.Generator().manual_seed(2)
    dout = torch.randn(H, T, dv, generator=gen).to(dtype)
    S0, dfin = (torch.randn(N, H, dv, dk, generator=gen) * 0.5 for _ in range(2))
    got = kda.gdr_chunk_bwd_varlen(*(t.cuda() for t in x), dout.cuda(), cu.cuda(), initial_state=S0.cuda(), dfinal_state=dfin.cuda())
    end = int(cu[-1])
    for name in NAMES[:5]:
        assert not got[name][:, :a0].any() and not got[name][:, end:].any(), name
    for i, (a, b) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        if a == b:
            assert torch.equal(got["dinitial_state"][i].cpu(), dfin[i])
            continue
        ref = reference([t[:, a:b][None] for t in x], dout[None, :, a:b], 1.0, S0[i][None], dfin[i][None])
        for name, t in zip(NAMES, ref):
            compare(got[name][i][None] if name == "dinitial_state" else got[name][None, :, a:b], t, dtype, name)


def test_captured():
    """Forward and backward in a graph, replayed on other inputs with eager work in between; the same
    inputs give the same bits."""
    xs = [[t.cuda() for t in inputs(2, 2, 4, 200, 128, 128, BF, s)] for s in (61, 62)]
    dout = torch.randn(2, 4, 200, 128, device="cuda").to(BF)
    want = [kda.gdr_chunk_bwd(*x, dout) for x in xs]
    buf = [t.clone() for t in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.gdr_chunk_fwd(*buf)
        got = kda.gdr_chunk_bwd(*buf, dout)
    for i in (0, 1, 0, 1):
        for t, s in zip(buf, xs[i]):
            t.copy_(s)
        graph.replay()
        again = kda.gdr_chunk_bwd(*xs[1 - i], dout)
        torch.cuda.synchronize()
        for name in NAMES:
            assert torch.equal(got[name], want[i][name]) and torch.equal(again[name], want[1 - i][name]), name
        assert torch.isfinite(out).all()
