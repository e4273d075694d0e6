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
