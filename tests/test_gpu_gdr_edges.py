"""The gated delta rule on the GPU where the magnitudes inside a chunk are uneven: keys that end before
the chunk does, betas and keys far from one, value channels that are zero or hold an infinity.  The
bounds are those of gdr_util.py and test_gpu_gdr_bwd.py."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from gdr_util import check, chunk_terms, inputs, out_bound, recurrent, state_bound
from test_gpu_gdr_bwd import NAMES, compare, reference

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# sequences, key heads, value heads, dv: one and two column tiles a work-group at dk = 128
SIZES = [(1, 1, 2, 64), (3, 4, 12, 128)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def _check_fwd(x, out, fs, scale, channels=slice(None)):
    """`channels`: the value channels that are compared."""
    ref, S = recurrent(*x, scale)
    for b in range(ref.shape[0]):
        inter, intra, size = chunk_terms(*(t[b] for t in x), scale)
        bound = out_bound(ref[b], inter, intra, x[0].dtype)
        check(out[b][..., channels], ref[b][..., channels], bound[..., channels], "out %d" % b)
        check(fs[b][:, channels], S[b][:, channels], state_bound(size)[:, channels], "state %d" % b)


def _fwd_and_grads(x, dout, scale, skip=()):
    """Forward against the recurrence, gradients (no start state) against its adjoint."""
    dtype, (B, H, T, dv), dk = x[0].dtype, x[2].shape, x[0].shape[-1]
    d = [t.cuda() for t in x]
    out, fs = kda.gdr_chunk_fwd(*d, scale=scale, return_final_state=True)
    _check_fwd(x, out, fs, scale)
    got = kda.gdr_chunk_bwd(*d, dout.cuda(), scale=scale)
    for name, ref in zip(NAMES, reference(x, dout, scale, torch.zeros(B, H, dv, dk), None)):
        if name not in skip:
            compare(got[name], ref, dtype, name)


def _tail(sizes, dtype, decay):
    """Keys and values stop after 30 tokens of the first chunk while the state goes on decaying, and no
    value comes afterwards: what follows is as small as the state is then."""
    B, Hk, H, dv = sizes
    x = inputs(B, Hk, H, 150, 128, dv, dtype, 71, rate=-6.0)
    x[1][:, :, 30:64] = 0.0
    x[2][:, :, 30:] = 0.0
    x[3][:, :, 30:64] = decay
    dout = torch.randn(B, H, 150, dv, generator=torch.Generator().manual_seed(3)).to(dtype)
    dout[:, :, :64] = 0.0  # the gradients of q, g and beta are then as small as the state, too
    return x, dout


@pytest.mark.parametrize("decay", [-0.1, -0.2])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_end_before_the_chunk(dtype, sizes, decay):
    _fwd_and_grads(*_tail(sizes, dtype, decay), 128 ** -0.5)


@pytest.mark.parametrize("norm", [0.3, 1e-3, 300.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_beta_far_from_one(dtype, norm):
    """Keys of another norm, and betas that keep beta |k|^2 below one: up to 10, to 9e5, to 1e-5."""
    x = list(inputs(2, 2, 4, 150, 128, 64, dtype, 81))
    x[1] = (x[1].double() * norm).to(dtype)
    x[4] = (x[4].double() * 0.9 / norm ** 2).to(dtype)
    dout = torch.randn(2, 4, 150, 64, generator=torch.Generator().manual_seed(4)).to(dtype)
    _fwd_and_grads(x, dout, 128 ** -0.5)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_zero_channels(dtype, sizes):
    """Heads padded with zero channels (values and gradients of 16 or 32 columns), beside small values
    and small gradients."""
    B, Hk, H, dv = sizes
    x = inputs(B, Hk, H, 150, 128, dv, dtype, 91)
    dout = torch.randn(B, H, 150, dv, generator=torch.Generator().manual_seed(5)).to(dtype)
    for t in (x[2], dout):
        t *= 2.0 ** -20
        t[..., -32:] = 0.0
    _fwd_and_grads(x, dout, 128 ** -0.5)
