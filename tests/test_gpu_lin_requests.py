"""Decayed linear attention on the GPU: what else a call asks for, and where it is called from, leave its
results alone."""
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


@pytest.mark.parametrize("dtype", [BF, F32])
def test_function_captured_without_gradients(dtype):
    """LinChunkFunction under no_grad with a parameter as its start state: captured, replayed on other inputs
    and with another start state, with eager calls in between."""
    H, T, d = 2, 200, 64
    xs = [[t.cuda() for t in U.inputs(1, H, H, T, d, d, dtype, s)] for s in (1, 2)]
    s0 = torch.randn(1, H, d, d, device="cuda").requires_grad_()
    buf = [t.clone() for t in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad():
        kda.LinChunkFunction.apply(*buf, 0.1, s0)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out, fs = kda.LinChunkFunction.apply(*buf, 0.1, s0)
        for k in range(4):
            for t, s in zip(buf, xs[k % 2]):
                t.copy_(s)
            s0.mul_(0.5)
            graph.replay()
            want = kda.lin_chunk_fwd(*xs[k % 2], scale=0.1, initial_state=s0, return_final_state=True)
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(fs, want[1]), k


def case(B, Hk, H, T, d, dtype, seed, packed=False):
    x = U.inputs(B, Hk, H, T, d, d, dtype, seed, packed=packed)
    do = U.inputs(B, Hk, H, T, d, d, dtype, seed + 1, packed=packed)[2]
    return [t.cuda() for t in (*x, do)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,H,T,d,lens", [
    (2, 1, 2, 200, 64, None), (1, 2, 2, 256, 128, None),   # four chunks of a sequence that is one segment
    (1, 1, 2, 700, 128, None),                              # eleven segments
    (16, 16, 32, 450, 64, None),                            # a full card: all of a sequence in one segment again
    (0, 1, 2, 240, 64, [70, 0, 130, 40]), (0, 32, 32, 3000, 64, [100, 64, 700, 1, 2135]),
])
def test_the_same_bits_whatever_is_asked_for(B, Hk, H, T, d, lens, dtype):
    """out with and without the end state; every gradient with and without dinitial_state, and with the end
    state's gradient left out or zeros; dv and dinitial_state with and without dg."""
    q, k, v, g, do = case(B, Hk, H, T, d, dtype, 81, packed=lens is not None)
    N = B if lens is None else len(lens)
    if lens is None:
        more, fwd, bwd = (), kda.lin_chunk_fwd, kda.lin_chunk_bwd
    else:
        more, fwd, bwd = (torch.tensor([0, *lens], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda(),), kda.lin_chunk_fwd_varlen, kda.lin_chunk_bwd_varlen
    s0 = torch.randn(N, H, d, d, device="cuda")
    for init in (None, s0):
        a = fwd(q, k, v, g, *more, scale=0.1, initial_state=init)
        b, _ = fwd(q, k, v, g, *more, scale=0.1, initial_state=init, return_final_state=True)
        torch.cuda.synchronize()
        assert torch.equal(a, b), "out"
        back = lambda **kw: bwd(q, k, v, g, do, *more, scale=0.1, initial_state=init, **kw)
        want = back()
        for kw in (dict(want_dinitial=False), dict(dfinal_state=torch.zeros_like(s0)), dict(want_dg=False),
                   dict(dfinal_state=torch.zeros_like(s0), want_dinitial=False)):
            got = back(**kw)
            torch.cuda.synchronize()
            for n, t in got.items():
                if t is not None and not (n in ("dq", "dk") and "want_dg" in kw):
                    assert torch.equal(t, want[n]), (n, kw.keys())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("used", ["out", "state", "both"])
def test_function_with_one_of_its_results(used, dtype):
    """Gradients through LinChunkFunction of its output, its end state or both: the entry points' bits."""
    q, k, v, g, do = case(2, 1, 2, 200, 64, dtype, 91)
    s0, df = (torch.randn(2, 2, 64, 64, device="cuda") for _ in range(2))
    x = [t.clone().requires_grad_() for t in (q, k, v, g, s0)]
    out, fs = kda.LinChunkFunction.apply(*x[:4], 0.1, x[4])
    loss = 0.0
    if used != "state":
        loss = loss + (out * do).sum()
    if used != "out":
        loss = loss + (fs * df).sum()
    got = torch.autograd.grad(loss, x)
    want = kda.lin_chunk_bwd(q, k, v, g, torch.zeros_like(do) if used == "state" else do, scale=0.1, initial_state=s0,
                             dfinal_state=None if used == "out" else df)
    torch.cuda.synchronize()
    for t, n in zip(got, ("dq", "dk", "dv", "dg", "dinitial_state")):
        assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,lens", [(200, None), (700, None), (0, [70, 0, 300, 1, 64, 500]), (0, [9] * 40 + [300, 65] + [0] * 9)])
def test_states_in_place(T, lens, dtype):
    """The end states written over the start states: as into other memory, also of many segments and of documents
    of one and of many side by side."""
    H, d = 2, 64
    N, total = (2, T) if lens is None else (len(lens), sum(lens))
    q, k, v, g, _ = case(2, 1, H, total, d, dtype, 101, packed=lens is not None)
    s0 = torch.randn(N, H, d, d, device="cuda")
    more = () if lens is None else (torch.tensor([0, *lens], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda(),)
    fwd = kda.lin_chunk_fwd if lens is None else kda.lin_chunk_fwd_varlen
    want, last = fwd(q, k, v, g, *more, scale=0.1, initial_state=s0, return_final_state=True)
    state = s0.clone()
    got = fwd(q, k, v, g, *more, scale=0.1, initial_state=state, final_state=state)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(state, last)
