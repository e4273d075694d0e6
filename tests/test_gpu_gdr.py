"""The gated delta rule on the GPU against the float64 token recurrence (gdr_util.py says where the
bounds come from): chunked forward over lengths from one token on, short last chunks, shared key
heads, strides, packed documents, initial states, extreme decays; the one-token step."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from gdr_util import check, chunk_terms, inputs, out_bound, recurrent, state_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def _state(N, H, dv, dk, seed):
    return torch.randn(N, H, dv, dk, generator=torch.Generator().manual_seed(seed)) * 0.5


def _check_fwd(x, out, fs, scale, S0, what=""):
    ref, S = recurrent(*x, scale, S0)
    for b in range(ref.shape[0]):
        inter, intra, size = chunk_terms(*(t[b] for t in x), scale, None if S0 is None else S0[b])
        check(out[b], ref[b], out_bound(ref[b], inter, intra, x[0].dtype), "%sout %d" % (what, b))
        check(fs[b], S[b], state_bound(size), "%sstate %d" % (what, b))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv", [
    (1, 1, 1, 1, 64, 64), (1, 1, 2, 2, 128, 64), (2, 2, 2, 63, 64, 128), (1, 2, 4, 64, 128, 128), (1, 1, 3, 65, 128, 128),
    (1, 2, 2, 127, 64, 64), (2, 1, 4, 200, 128, 128), (1, 1, 1, 513, 128, 128),
])
def test_forward(B, Hk, H, T, dk, dv, dtype):
    x = inputs(B, Hk, H, T, dk, dv, dtype, 11 + T)
    S0 = _state(B, H, dv, dk, T) if T % 2 else None
    out, fs = kda.gdr_chunk_fwd(*(t.cuda() for t in x), scale=dk ** -0.5, return_final_state=True,
                                initial_state=None if S0 is None else S0.cuda())
    _check_fwd(x, out, fs, dk ** -0.5, S0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_waves_per_work_group(dtype):
    """Enough heads for each number of waves in a work-group of the state stage."""
    for B, H in ((1, 8), (4, 16), (8, 16)):
        x = inputs(B, H, H, 70, 64, 128, dtype, B + H)
        out, fs = kda.gdr_chunk_fwd(*(t.cuda() for t in x), return_final_state=True)
        _check_fwd(x, out, fs, 1.0, None, "%d " % (B * H))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,T", [(128, 200), (64, 129), (128, 5)])
def test_two_column_tiles(dk, T, dtype):
    """More than 256 slices of 16 value columns, 32 a work-group but for dk = 64 in bf16; a start state."""
    B, H, dv = 3, 12, 128
    x = inputs(B, 4, H, T, dk, dv, dtype, dk + T)
    S0 = _state(B, H, dv, dk, T)
    out, fs = kda.gdr_chunk_fwd(*(t.cuda() for t in x), scale=dk ** -0.5, return_final_state=True, initial_state=S0.cuda())
    _check_fwd(x, out, fs, dk ** -0.5, S0)


def test_strided_views():
    """Projections as a model leaves them: [B,T,H,d] seen as [B,H,T,d], g and beta interleaved."""
    x = inputs(2, 2, 4, 77, 128, 64, BF, 3)
    q, k, v = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in x[:3])
    gb = torch.stack(x[3:], -1).transpose(1, 2).contiguous().cuda()
    g, beta = gb[..., 0].transpose(1, 2), gb[..., 1].transpose(1, 2)
    assert not q.is_contiguous() and not g.is_contiguous()
    a = kda.gdr_chunk_fwd(q, k, v, g, beta, return_final_state=True)
    b = kda.gdr_chunk_fwd(*(t.cuda() for t in x), return_final_state=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,lengths", [
    (BF, [1, 63, 64, 65, 0, 130, 7]), (F32, [0, 5, 100, 0]), (BF, [0, 0]), (F32, [128]), (BF, [1] * 40),
])
def test_packed(dtype, lengths):
    T, Hk, H, dk, dv = sum(lengths) + 9, 2, 4, 128, 64  # nine rows behind the last document
    x = inputs(1, Hk, H, T, dk, dv, dtype, 21, packed=True)
    cu = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32)
    S0 = _state(len(lengths), H, dv, dk, 5)
    out = torch.full((H, T, dv), 7.0, dtype=dtype, device="cuda")
    _, fs = kda.gdr_chunk_fwd_varlen(*(t.cuda() for t in x), cu.cuda(), scale=0.7, out=out, return_final_state=True,
                                     initial_state=S0.cuda())
    assert (out[:, int(cu[-1]):] == 7.0).all()
    for n, (a, b) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        if a == b:
            assert torch.equal(fs[n].cpu(), S0[n])
            continue
        _check_fwd([t[:, a:b][None] for t in x], out[None, :, a:b], fs[None, n], 0.7, S0[n][None], "doc %d " % n)


def test_bad_boundaries_stay_inside():
    """Boundaries outside the contract are clipped on the device: finite, unspecified results."""
    x = inputs(1, 1, 2, 150, 64, 64, BF, 5, packed=True)
    for cu in ([-5, 70, 900], [100, 20, 150], [150, 150, 0], [2 ** 31 - 1, -2 ** 31, 64]):
        fs = kda.gdr_chunk_fwd_varlen(*(t.cuda() for t in x), torch.tensor(cu, dtype=torch.int32).cuda(),
                                      return_final_state=True)[1]
        torch.cuda.synchronize()
        assert fs.shape == (2, 2, 64, 64)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays(dtype):
    """No decay, decays to zero (-inf among them) in the middle of a chunk, and a large one early in
    a chunk, behind which small ones must keep their precision."""
    x = list(inputs(1, 1, 4, 150, 64, 64, dtype, 9))
    g = x[3].clone()
    g[0, 0] = 0
    g[0, 1, 70] = float("-inf")
    g[0, 1, 71] = -2e4
    g[0, 2, 64:] = -0.001
    g[0, 2, 65] = -900.0
    g[0, 3] = -30.0
    x[3] = g
    out, fs = kda.gdr_chunk_fwd(*(t.cuda() for t in x), return_final_state=True)
    _check_fwd(x, out, fs, 1.0, None)


def test_magnitudes():
    """Values far from one: powers of two scale out exactly (block exponents), zeros stay zeros."""
    x = inputs(1, 1, 2, 100, 128, 128, BF, 13)
    a = kda.gdr_chunk_fwd(*(t.cuda() for t in x), return_final_state=True)
    y = [x[0] * 2.0 ** -40, x[1], x[2] * 2.0 ** 60, x[3], x[4]]
    b = kda.gdr_chunk_fwd(*(t.cuda() for t in y), return_final_state=True)
    assert torch.equal(a[0].double() * 2.0 ** 20, b[0].double()) and torch.equal(a[1].double() * 2.0 ** 60, b[1].double())
    z = [torch.zeros_like(t) for t in x]
    out, fs = kda.gdr_chunk_fwd(*(t.cuda() for t in z), return_final_state=True)
    assert not out.any() and not fs.any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 6, 128, 64), (2, 4, 4, 64, 128), (5, 2, 4, 128, 128)])
def test_decode_step(B, Hk, H, dk, dv, dtype):
    x = inputs(B, Hk, H, 3, dk, dv, dtype, 31)
    S0 = _state(B, H, dv, dk, 8)
    S = S0.cuda()
    scale = dk ** -0.5
    for t in range(3):
        o = kda.gdr_decode_step(*(y[:, :, t].contiguous().cuda() for y in x), S, scale=scale)
        ref, Sr = recurrent(*(y[:, :, :t + 1] for y in x), scale, S0)
        inter = scale * x[0][:, :, t].double().norm(dim=-1).repeat_interleave(H // Hk, 1)[..., None] * Sr.norm(dim=-1)
        # float32 sums of dk terms in every token so far, then one rounding
        check(o, ref[:, :, t], 2.0 ** -8 * ref[:, :, t].abs() * (dtype == BF) + (t + 1) * (dk + 8) * 2.0 ** -24 * inter * 4,
              "out %d" % t)
        check(S, Sr, (t + 1) * (dk + 8) * 2.0 ** -24 * Sr.abs().amax((-1, -2), keepdim=True).expand_as(Sr) * 4, "state %d" % t)


def test_prefill_then_decode():
    """A sequence in pieces: a chunked prefill, its state handed to one-token steps, against one
    chunked pass over everything."""
    T, n = 150, 6
    x = inputs(2, 2, 4, T + n, 128, 128, BF, 41)
    d = [t.cuda() for t in x]
    full, fs = kda.gdr_chunk_fwd(*d, return_final_state=True)
    out, S = kda.gdr_chunk_fwd(*(t[:, :, :T] for t in d), return_final_state=True)
    steps = [kda.gdr_decode_step(*(t[:, :, T + i].contiguous() for t in d), S) for i in range(n)]
    got = torch.cat([out, torch.stack(steps, 2)], 2)
    _check_fwd(x, got, S, 1.0, None)
    assert torch.equal(got[:, :, :128], full[:, :, :128])


def test_two_streams_and_graph():
    """Two calls at once on two streams, and a captured call replayed on new inputs."""
    xs = [[t.cuda() for t in inputs(2, 2, 4, 300, 128, 128, BF, s)] for s in (51, 52)]
    want = [kda.gdr_chunk_fwd(*x, return_final_state=True) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [kda.gdr_chunk_fwd(*x, return_final_state=True, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    buf = [t.clone() for t in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = kda.gdr_chunk_fwd(*buf, return_final_state=True)
    for i in (1, 0, 1):
        for t, s in zip(buf, xs[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want[i][0]) and torch.equal(res[1], want[i][1])
