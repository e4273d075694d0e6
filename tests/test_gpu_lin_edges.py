"""Decayed linear attention on the GPU outside the ordinary: values that are not finite, views with odd
strides and beyond 32-bit offsets, workspaces that hold anything, streams, captured graphs.  Bounds as in
lin_util.py."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import lin_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GRADS = ("dq", "dk", "dv", "dg", "dinitial_state")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def both(q, k, v, g, do, s0=None, df=None, scale=0.1, **kw):
    """Forward and backward: {name: tensor}."""
    out, fs = kda.lin_chunk_fwd(q, k, v, g, scale=scale, initial_state=s0, return_final_state=True, **kw)
    return {"out": out, "final_state": fs, **kda.lin_chunk_bwd(q, k, v, g, do, scale=scale, initial_state=s0, dfinal_state=df, **kw)}


def case(B, Hk, H, T, dk, dv, dtype, seed):
    x = U.inputs(B, Hk, H, T, dk, dv, dtype, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    do = torch.randn(B, H, T, dv, generator=gen).to(dtype)
    s0, df = (torch.randn(B, H, dv, dk, generator=gen) for _ in range(2))
    return [t.cuda() for t in (*x, do, s0, df)]


def same(a, b, what=""):
    for n in b:
        assert torch.equal(a[n], b[n]), what + n


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,dk,dv", [(300, 64, 128), (130, 128, 64)])
def test_what_is_not_finite(T, dk, dv, dtype, bad):
    """In q: its token's outputs; in v: its channel from its chunk on; in k or g = NaN: its head's.  Other
    heads, channels and earlier chunks keep their bits."""
    t, c0 = 100, 64
    x = U.inputs(1, 2, 2, T, dk, dv, dtype, 3)
    ref, rs = kda.lin_chunk_fwd(*(y.cuda() for y in x), scale=0.1, return_final_state=True)
    for i, name in enumerate("qkvg"):
        y = [z.clone() for z in x]
        at = (0, 1, t) + ((5,) if name != "g" else ())
        if name == "g" and bad != bad:
            y[i][at] = bad
        elif name == "g":
            continue  # -inf is a decay to zero; above zero there is nothing to hold to
        else:
            y[i][at] = bad
        out, fs = kda.lin_chunk_fwd(*(z.cuda() for z in y), scale=0.1, return_final_state=True)
        torch.cuda.synchronize()
        assert torch.equal(out[0, 0], ref[0, 0]) and torch.equal(fs[0, 0], rs[0, 0]), name
        assert torch.equal(out[0, 1, :c0], ref[0, 1, :c0]), name
        assert not torch.isfinite(out[0, 1, t]).any() if name != "v" else not torch.isfinite(out[0, 1, t, 5]), name
        if name == "q":
            rest = [j for j in range(T) if j != t]
            assert torch.equal(out[0, 1, rest], ref[0, 1, rest]) and torch.equal(fs, rs)
        elif name == "v":
            rest = [j for j in range(dv) if j != 5]
            assert torch.equal(out[0, 1][:, rest], ref[0, 1][:, rest]) and torch.equal(fs[0, 1, rest], rs[0, 1, rest])
            assert not torch.isfinite(out[0, 1, t:, 5]).any() and not torch.isfinite(fs[0, 1, 5]).any()


def loose(t, dims):
    """t with a stride of 13 in dimensions of one, which no row's start depends on."""
    t = t.contiguous()
    assert all(t.shape[i] == 1 for i in dims)
    return t.as_strided(t.shape, [13 if i in dims else s for i, s in enumerate(t.stride())])


@pytest.mark.parametrize("T,dims", [(330, (0, 1)), (1, (0, 2))])
def test_strides_of_dimensions_of_one(T, dims):
    H = 1 if 1 in dims else 3
    q, k, v, g, do, s0, df = case(1, H, H, T, 64, 64, BF, 13)
    same(both(*(loose(t, dims) for t in (q, k, v, g, do)), s0, df), both(q, k, v, g, do, s0, df))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_share_memory(dtype):
    """Heads, batch entries and tokens broadcast (strides of zero), windows that overlap, batch and heads
    backwards in memory: the same bits as copies."""
    B, H, T, d = 2, 2, 333, 64
    gen = torch.Generator().manual_seed(4)
    wide = torch.randn(T * 8 + d, generator=gen).to(dtype).cuda()
    q = torch.randn(d, generator=gen).to(dtype).cuda().expand(B, H, T, d)
    k = wide.as_strided((B, H, T, d), (0, 8, 8, 1))
    v = torch.randn(B, 1, T, d, generator=gen).to(dtype).cuda().expand(B, H, T, d)
    g = (-torch.rand(1, H, 1, generator=gen)).cuda().expand(B, H, T)
    do = torch.randn(1, 1, 1, d, generator=gen).to(dtype).cuda().expand(B, H, T, d)
    x = (q, k, v, g, do)
    same(both(*x), both(*(t.contiguous() for t in x)))


def test_offsets_beyond_32_bits():
    """Batch entries more than 2^31 elements apart in memory."""
    B, H, T, d, far = 2, 2, 130, 64, (1 << 31) + 64
    room = torch.empty(far + 5 * H * T * d, dtype=BF, device="cuda")
    q, k, v, g, do, *_ = case(B, H, H, T, d, d, BF, 17)
    views, at = [], 0
    for t in (q, k, v, do):
        w = room.as_strided(t.shape, (far, T * d, d, 1), at)
        w.copy_(t)
        views.append(w)
        at += H * T * d
    same(both(views[0], views[1], views[2], g, views[3]), both(q, k, v, g, do))


def test_more_than_2_to_the_31_elements():
    """One sequence of 2^22 + 77 tokens, 8 heads: decays of e^-1 a token forget what is more than a hundred
    tokens back, so the last rows are those of the last tokens alone (e^-900 of what came before)."""
    H, T, d, tail = 8, (1 << 22) + 77, 64, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, H, T, d, generator=gen, device="cuda", dtype=BF) for _ in range(3))
    g = torch.full((1, H, 1), -1.0, device="cuda").expand(1, H, T)
    out, fs = kda.lin_chunk_fwd(q, k, v, g, scale=0.1, return_final_state=True)
    torch.cuda.synchronize()
    for h in (0, H - 1):
        x = [t[0, h, -tail:].cpu() for t in (q, k, v, g)]
        ref = U.one(*x, 0.1, BF, F32)
        U.check(out[0, h, -100:], ref["out"][0][-100:], ref["out"][1][-100:], "out %d" % h, BF)
        U.check(fs[0, h], *ref["final_state"], "final_state %d" % h, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [64, 257, 1100])
def test_workspaces_may_hold_anything(T, dtype):
    """One workspace for all calls, of NaN before each, larger than needed; as with fresh ones."""
    q, k, v, g, do, s0, df = case(1, 1, 2, T, 128, 64, dtype, T)
    need = max(kda.lin_workspace_bytes(1, 1, 2, T, 128, 64, dtype, backward=b) for b in (False, True))
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    want = both(q, k, v, g, do, s0, df)
    out, fs = kda.lin_chunk_fwd(q, k, v, g, scale=0.1, initial_state=s0, return_final_state=True, workspace=ws)
    assert bool((ws[need:] == 255).all())
    ws.fill_(255)
    d = kda.lin_chunk_bwd(q, k, v, g, do, scale=0.1, initial_state=s0, dfinal_state=df, workspace=ws)
    assert bool((ws[need:] == 255).all())
    same({"out": out, "final_state": fs, **d}, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_calls_at_once_on_other_streams(dtype):
    xs = [case(1, 2, 4, 900, 128, 128, dtype, s) for s in (1, 2)]
    want = [both(*x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [both(*x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        same(a, b)


def test_captured():
    """Forward, backward and a one-token step in two graphs that share a workspace, replayed in turn on other
    inputs with eager calls in between."""
    xs = [case(2, 2, 4, 300, 64, 128, BF, s) for s in (5, 6)]
    token = [torch.randn(*s, device="cuda").to(BF) for s in ((2, 2, 64), (2, 2, 64), (2, 4, 128))]

    def step(x, ws=None):
        r = both(*x, workspace=ws)
        r["state"] = r["final_state"] * 1
        r["token"] = kda.lin_decode_step(*token, x[3][:, :, 0].contiguous(), r["state"], scale=0.2)
        return r

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    bufs = [[t.clone() for t in x] for x in xs]
    ws = torch.full((kda.lin_workspace_bytes(2, 2, 4, 300, 64, 128, BF, backward=True),), 255, dtype=torch.uint8, device="cuda")
    graphs, res = [torch.cuda.CUDAGraph() for _ in xs], []
    for graph, buf in zip(graphs, bufs):
        with torch.cuda.graph(graph):
            res.append(step(buf, ws))
    for k in range(4):
        for j, graph in enumerate(graphs):
            i = (j + k) % 2
            for t, s in zip(bufs[j], xs[i]):
                t.copy_(s)
            graph.replay()
            same(step(xs[1 - i]), want[1 - i], "eager ")
            torch.cuda.synchronize()
            same(res[j], want[i], "replay %d of graph %d " % (k, j))


def test_function_of_packed_documents():
    """LinChunkFunction of documents with start states, the end states unused, bf16 with float32 decays."""
    H, d, cu = 2, 64, [0, 70, 70, 401]
    q, k, v, g = (t.cuda() for t in U.inputs(0, 1, H, cu[-1], d, d, BF, 8, packed=True, g32=True))
    s0 = torch.randn(3, H, d, d, device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    do = torch.randn_like(v)
    x = [t.clone().requires_grad_() for t in (q, k, v, g, s0)]
    out, _ = kda.LinChunkFunction.apply(*x[:4], 0.1, x[4], c)
    out.backward(do)
    want = kda.lin_chunk_bwd_varlen(q, k, v, g, do, c, scale=0.1, initial_state=s0, dfinal_state=torch.zeros_like(s0))
    assert torch.equal(out.detach(), kda.lin_chunk_fwd_varlen(q, k, v, g, c, scale=0.1, initial_state=s0))
    for t, n in zip(x, GRADS):
        assert torch.equal(t.grad, want[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_far_apart(dtype):
    """Keys and values of a few large and many small channels, start states of 1e4."""
    q, k, v, g, do, s0, df = (t.cpu() for t in case(1, 1, 1, 200, 64, 64, dtype, 23))
    scale = torch.logspace(-4, 3, 64)
    k, v, s0 = (k * scale).to(dtype), (v * scale.flip(0)).to(dtype), s0 * 1e4
    got = both(*(t.cuda() for t in (q, k, v, g, do, s0, df)))
    torch.cuda.synchronize()
    ref = U.one(q[0, 0], k[0, 0], v[0, 0], g[0, 0], 0.1, dtype, dtype, s0[0, 0], do[0, 0], df[0, 0])
    for n, (value, bound) in ref.items():
        U.check(got[n][0, 0], value, bound + U.HALF[dtype] * value.abs() * 1.01, n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv", [
    (8, 4, 8, 1297, 64, 64),     # 21 chunks a head: segments of six, six, six and three (float32: of three)
    (4, 8, 32, 1100, 128, 64),   # 18: nine and nine, key heads shared by four
    (16, 16, 32, 450, 64, 128),  # eight: all of a sequence in one
    (1, 64, 128, 833, 128, 128),  # 14: seven and seven, the last of one row
])
def test_segments_of_several_chunks(B, Hk, H, T, dk, dv, dtype):
    """Full cards, where a segment is several chunks: the first and the last key head against float64."""
    q, k, v, g, do, s0, df = (t.cpu() for t in case(B, Hk, H, T, dk, dv, dtype, 31))
    got = both(*(t.cuda() for t in (q, k, v, g, do, s0, df)))
    torch.cuda.synchronize()
    r = H // Hk
    for b, j in ((0, 0), (B - 1, Hk - 1)):
        x = {n: t[b, j:j + 1] if n in ("dq", "dk") else t[b, j * r:(j + 1) * r] for n, t in got.items()}
        U.check_sequence(x, "%d %d " % (b, j), r, r, lambda h: U.one(
            q[b, j], k[b, j], v[b, j * r + h], g[b, j * r + h], 0.1, dtype, g.dtype, s0[b, j * r + h], do[b, j * r + h], df[b, j * r + h]),
            dtype, g.dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_segments_of_several_chunks(dtype):
    """Documents of one row to many segments in a stream that fills the card."""
    H, d, lens = 32, 64, [1, 700, 64, 2049, 0, 385, 1500, 3]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N = cu[-1], len(lens)
    q, k, v, g = U.inputs(0, H, H, T, d, d, dtype, 33, packed=True)
    do = U.inputs(0, H, H, T, d, d, dtype, 34, packed=True)[2]
    gen = torch.Generator().manual_seed(35)
    s0, df = (torch.randn(N, H, d, d, generator=gen) for _ in range(2))
    x = [t.cuda() for t in (q, k, v, g)]
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    out, fs = kda.lin_chunk_fwd_varlen(*x, c, scale=0.1, initial_state=s0.cuda(), return_final_state=True)
    grads = kda.lin_chunk_bwd_varlen(*x, do.cuda(), c, scale=0.1, initial_state=s0.cuda(), dfinal_state=df.cuda())
    torch.cuda.synchronize()
    for i in range(N):
        s = slice(cu[i], cu[i + 1])
        for h0 in (0, H - 1):
            got = {"out": out[h0:h0 + 1, s], "final_state": fs[i, h0:h0 + 1], "dinitial_state": grads["dinitial_state"][i, h0:h0 + 1],
                   **{n: grads[n][h0:h0 + 1, s] for n in ("dq", "dk", "dv", "dg")}}
            U.check_sequence(got, "%d %d " % (i, h0), 1, 1, lambda h: U.one(q[h0, s], k[h0, s], v[h0, s], g[h0, s], 0.1, dtype, dtype,
                                                                             s0[i, h0], do[h0, s], df[i, h0]), dtype, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_tokens(dtype):
    """A batch of none, a stream of none and a stream of empty documents: end states are the start states."""
    H, d = 2, 64
    q = torch.zeros(3, H, 0, d, dtype=dtype, device="cuda")
    s0 = torch.randn(3, H, d, d, device="cuda")
    out, fs = kda.lin_chunk_fwd(q, q, q, q[..., 0], initial_state=s0, return_final_state=True)
    assert out.shape == q.shape and torch.equal(fs, s0)
    out, fs = kda.lin_chunk_fwd(q, q, q, q[..., 0], return_final_state=True)
    assert bool((fs == 0).all())
    c = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, fs = kda.lin_chunk_fwd_varlen(q[0], q[0], q[0], q[0, ..., 0], c, initial_state=s0, return_final_state=True)
    assert out.shape == q[0].shape and torch.equal(fs, s0)
    x, g = torch.randn(H, 90, d, device="cuda").to(dtype), torch.zeros(H, 90, device="cuda")
    out, fs = kda.lin_chunk_fwd_varlen(x, x, x, g, c, out=torch.full_like(x, 7), initial_state=s0, return_final_state=True)
    grads = kda.lin_chunk_bwd_varlen(x, x, x, g, x, c, initial_state=s0, dfinal_state=s0)
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and torch.equal(fs, s0) and torch.equal(grads["dinitial_state"], s0)
    assert all(bool((grads[n] == 0).all()) for n in ("dq", "dk", "dv", "dg"))


def test_boundaries_out_of_order():
    """Boundaries below zero, behind the stream and going back: no access outside, and documents that stand by
    themselves get what they get alone."""
    H, T, d = 2, 200, 64
    q, k, v, g, do, *_ = (t[0] if t.dim() == 4 or t.dim() == 3 else t for t in case(1, H, H, T, d, d, BF, 41))
    c = torch.tensor([-50, 70, 30, 30, 10 ** 6], dtype=torch.int32, device="cuda")
    out, fs = kda.lin_chunk_fwd_varlen(q, k, v, g, c, scale=0.1, return_final_state=True)
    kda.lin_chunk_bwd_varlen(q, k, v, g, do, c, scale=0.1)
    torch.cuda.synchronize()
    assert torch.isfinite(fs).all()
    c = torch.tensor([-50, 70, 10 ** 6], dtype=torch.int32, device="cuda")
    out, fs = kda.lin_chunk_fwd_varlen(q, k, v, g, c, scale=0.1, return_final_state=True)
    want = kda.lin_chunk_fwd_varlen(q, k, v, g, torch.tensor([0, 70, T], dtype=torch.int32, device="cuda"), scale=0.1, return_final_state=True)
    assert torch.equal(out, want[0]) and torch.equal(fs, want[1])
