"""Decayed linear attention's forward beyond 2^28 tokens and heads on the GPU, which its backward refuses.  Bounds as
in lin_util.py."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import lin_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_more_than_2_to_the_28_tokens_and_heads():
    """128 heads of 2^21 + 64 tokens that share their keys and values, a decay for each head: at e^-0.9 a token
    and below the last rows are those of the last thousand tokens alone."""
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    H, T, d, tail = 128, (1 << 21) + 64, 64, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, 1, T, d, generator=gen, device="cuda", dtype=BF) for _ in range(3))
    slopes = -0.9 - 0.01 * torch.arange(H, device="cuda", dtype=F32)
    g = slopes[None, :, None].expand(1, H, T)
    s0 = torch.randn(1, H, d, d, generator=gen, device="cuda")
    out, fs = kda.lin_chunk_fwd(q, k, v.expand(1, H, T, d), g, scale=0.1, initial_state=s0, return_final_state=True)
    torch.cuda.synchronize()
    for h in (0, 63, H - 1):
        x = [t[0, 0, -tail:].cpu() for t in (q, k, v)] + [g[0, h, -tail:].cpu()]
        ref = U.one(*x, 0.1, BF, F32)
        U.check(out[0, h, -100:], ref["out"][0][-100:], ref["out"][1][-100:], "out %d" % h, BF)
        U.check(fs[0, h], *ref["final_state"], "final_state %d" % h, F32)
        x = [t[0, 0, :130].cpu() for t in (q, k, v)] + [g[0, h, :130].cpu()]
        U.check(out[0, h, :130], *U.one(*x, 0.1, BF, F32, s0[0, h].cpu())["out"], "first rows %d" % h, BF)
